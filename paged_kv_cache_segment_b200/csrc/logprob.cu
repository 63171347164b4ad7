// logprob.cu - tf_logprob_rows: log probabilities of given tokens, entropy and
// top alternatives of logit rows, in one pass over the logits.
//
// With m the row's largest logit, d = x - m, c = scale * log2(e), l = sum 2^(c d)
// and t = sum 2^(c d) d:
//   log p(x) = scale * d - ln l,  lse = scale * m + ln l,  H = ln l - scale * t / l.
// d <= 0, so both terms of H are >= 0 and nothing cancels; d is exact or rounded
// once, where x * c - m * c would carry the rounding of m * c into every term.
//
// A CTA (512 threads) owns a row's columns, or 1/CL of them with a cluster of CL
// CTAs a row when there are few rows.  It walks them in chunks that a thread
// holds in registers (four 16-byte vectors), the next chunk's loads in flight
// while the current one folds, across the row's end too.  Vectors are aligned to
// 16 bytes whatever the row's own alignment: the grid of vectors starts up to 15
// bytes before the row, and only the vectors that cross its ends load by element.
//
// Top k: elements are ordered by a 64-bit key, the value's order-preserving image
// above the complement of the column, so keys are distinct and ties go to the
// lower column.  The 32 half-warps keep the largest key each has seen; the
// smallest of those 32 is a threshold that at least 32 >= k elements reach, so
// only elements at or above it can be among the top k.  They are few (a few
// dozen to a few hundred of a row) and go to a list in shared memory, from which
// the k largest are ranked by counting.  A chunk that would overflow the list (a
// half-warp that holds only masked columns leaves the threshold at nothing) is
// searched by k block-wide maxima instead: slower, but never wrong.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "api_common.h"
#include "tf_common.cuh"
#include "tf_internal.h"

namespace cg = cooperative_groups;

namespace tfp {
namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpBatch = 4;       // 16-byte vectors a thread holds of a chunk
constexpr int kLpMaxTop = 32;
constexpr int kLpGroups = 2 * kLpWarps;  // half-warps, each with its largest key
constexpr int kLpList = 1024;            // candidates of a row
constexpr int kLpMaxCluster = 8;
static_assert(kLpGroups >= kLpMaxTop, "the threshold needs a group for every alternative");

struct LogprobParams {
    const void *logits;
    int n_rows, n_cols;
    int64_t ld;
    float scale;
    const int32_t *tokens;
    int n_tokens;
    float *token_logprobs, *entropy, *lse;
    int top_k;
    int32_t *top_ids;
    float *top_logprobs;
    uint8_t *flags;
    uint32_t *status;
};

// Order-preserving image of a float (-0 as +0), 0 for -infinity, and back.
__device__ __forceinline__ uint32_t key32(float x) {
    if (x == -INFINITY) return 0u;
    const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unkey32(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ uint64_t key64(float x, int col) {
    const uint32_t k = key32(x);
    return k == 0u ? 0ull : ((uint64_t)k << 32) | (uint32_t)~col;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A row's running statistics: the largest logit, sum 2^(c (x - m)), and the same
// sum weighted by x - m.
struct Stat {
    float m, l, t;
    __device__ __forceinline__ void to(float M, float c) {  // M >= m
        if (m != -INFINITY) {  // (no unmasked column yet: l and t are 0, or NaN)
            const float r = ex2((m - M) * c);
            // (r = 0: the old terms are gone, and l * (m - M) may have overflowed)
            t = M == m ? t : (r > 0.f ? (t + l * (m - M)) * r : 0.f);
            l *= r;
        }
        m = M;
    }
};
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float M = fmaxf(a.m, b.m);
    if (M == -INFINITY) return {M, a.l + b.l, a.t + b.t};  // a NaN stays
    a.to(M, c);
    b.to(M, c);
    return {M, a.l + b.l, a.t + b.t};
}

// Ranks the n distinct keys of `list` and puts the k largest, largest first,
// into `top` (0 past the n-th).  The whole CTA calls it.
__device__ __forceinline__ void rank_top(const uint64_t *list, int n, int k, uint64_t *top) {
    for (int i = threadIdx.x; i < n; i += kLpThreads) {
        const uint64_t mine = list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += list[j] > mine ? 1 : 0;
        if (rank < k) top[rank] = mine;
    }
    for (int i = n + threadIdx.x; i < k; i += kLpThreads) top[i] = 0ull;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kPer = 4;  // elements of a 16-byte vector
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int e) { return __uint_as_float(w[e]); }
    static __device__ __forceinline__ float load(const float *p) { return __ldg(p); }
    static __device__ __forceinline__ void put(uint32_t (&w)[4], int e, float x) { w[e] = __float_as_uint(x); }
};
template <>
struct Elem<uint16_t> {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int e) {
        return (e & 1) ? bf16_hi_to_f32(w[e >> 1]) : bf16_lo_to_f32(w[e >> 1]);
    }
    static __device__ __forceinline__ float load(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
    static __device__ __forceinline__ void put(uint32_t (&w)[4], int e, float x) {
        const uint32_t b = __float_as_uint(x) >> 16;
        w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (b << 16) : (w[e >> 1] & 0xffff0000u) | b;
    }
};

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 2) logprob_kernel(const LogprobParams p) {
    using E = Elem<T>;
    constexpr int EPV = E::kPer;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ Stat w_stat[kLpWarps];
    __shared__ uint64_t s_group[2][kLpGroups];
    __shared__ uint64_t s_list[TOP ? kLpList : 1], s_top[kLpMaxTop], s_best[kLpWarps];
    __shared__ int s_n;
    // rank 0's slots, filled by every CTA of the cluster, two buffers by row parity
    __shared__ Stat x_stat[2][kLpMaxCluster];
    __shared__ uint64_t x_top[2][TOP ? kLpMaxCluster * kLpMaxTop : 1];
    if (CL > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    bool joined = CL == 1;
    const float c = p.scale * kLog2e;
    const int K = p.top_k;

    // this CTA's vectors [v0, v1) of a row; vector v holds columns v * EPV - mis ...
    struct Row {
        const T *at;
        int mis, v0, v1, n_chunks;
    };
    auto open = [&](int r) {
        Row w;
        w.at = static_cast<const T *>(p.logits) + (int64_t)r * p.ld;
        w.mis = (int)((reinterpret_cast<uintptr_t>(w.at) & 15u) / sizeof(T));
        const int nv = (w.mis + p.n_cols + EPV - 1) / EPV, per = (nv + CL - 1) / CL;
        w.v0 = min(nv, rank * per);
        w.v1 = min(nv, w.v0 + per);
        w.n_chunks = max(1, (w.v1 - w.v0 + kLpBatch * kLpThreads - 1) / (kLpBatch * kLpThreads));
        return w;
    };
    auto load = [&](const Row &w, int chunk, uint32_t (&x)[kLpBatch][4]) {
#pragma unroll
        for (int k = 0; k < kLpBatch; ++k) {
            const int v = w.v0 + (chunk * kLpBatch + k) * kLpThreads + tid;
            const int c0 = v * EPV - w.mis;
            if (v < w.v1 && c0 >= 0 && c0 + EPV <= p.n_cols) {
                const uint4 y = __ldg(reinterpret_cast<const uint4 *>(w.at + c0));
                x[k][0] = y.x;
                x[k][1] = y.y;
                x[k][2] = y.z;
                x[k][3] = y.w;
            } else {
                const uint32_t none = EPV == 4 ? 0xff800000u : 0xff80ff80u;
                x[k][0] = x[k][1] = x[k][2] = x[k][3] = none;
                if (v < w.v1) {
#pragma unroll
                    for (int e = 0; e < EPV; ++e)
                        if (c0 + e >= 0 && c0 + e < p.n_cols) E::put(x[k], e, E::load(w.at + c0 + e));
                }
            }
        }
    };

    uint32_t cur[kLpBatch][4], nxt[kLpBatch][4];
    int row = blockIdx.y, it = 0;
    if (row >= p.n_rows) {
        if (!joined) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        return;  // (the whole cluster: its CTAs share blockIdx.y)
    }
    Row w = open(row);
    load(w, 0, cur);
    for (; row < p.n_rows; row += gridDim.y, ++it) {
        Stat st{-INFINITY, 0.f, 0.f};
        uint64_t group_best = 0, tau = 0;  // this half-warp's largest key, the threshold
        const int next_row = row + (int)gridDim.y;
        Row wn = w;
        if constexpr (TOP) {
            if (tid == 0) s_n = 0;
        }
        for (int ch = 0; ch < w.n_chunks; ++ch) {
            // the next chunk's loads, of this row or the next one
            if (ch + 1 < w.n_chunks) {
                load(w, ch + 1, nxt);
            } else if (next_row < p.n_rows) {
                wn = open(next_row);
                load(wn, 0, nxt);
            }
            // ---- statistics
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
                for (int e = 0; e < EPV; ++e) mx = fmaxf(mx, E::get(cur[k], e));
            if (mx > st.m) st.to(mx, c);
            // (all masked so far: the reference is 0, every term 2^-inf = 0 or a NaN)
            const float ref = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    const float d = max_nan(E::get(cur[k], e) - ref, -FLT_MAX);  // a masked column: 0 * finite
                    const float q = ex2(d * c);
                    st.l += q;
                    st.t = fmaf(q, d, st.t);
                }
            if constexpr (TOP) {
                // ---- candidates of this chunk
                auto col_of = [&](int k, int e) {
                    return (w.v0 + (ch * kLpBatch + k) * kLpThreads + tid) * EPV - w.mis + e;
                };
                uint64_t best = 0;
                if (key32(mx) != 0u && key32(mx) >= (uint32_t)(tau >> 32)) {
                    int col = INT_MAX;
#pragma unroll
                    for (int k = kLpBatch - 1; k >= 0; --k)
#pragma unroll
                        for (int e = EPV - 1; e >= 0; --e)
                            if (E::get(cur[k], e) == mx) col = col_of(k, e);
                    best = key64(mx, col);
                }
                uint64_t gb = best;
#pragma unroll
                for (int o = 8; o; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, gb, o);
                    gb = y > gb ? y : gb;
                }
                group_best = gb > group_best ? gb : group_best;
                if ((lane & 15) == 0) s_group[ch & 1][warp * 2 + (lane >> 4)] = group_best;
                __syncthreads();
                const int n_before = s_n;
                tau = s_group[ch & 1][lane];
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, tau, o);
                    tau = y < tau ? y : tau;
                }
                __syncthreads();  // every thread has read s_n
                if (best != 0 && best >= tau) {
#pragma unroll
                    for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
                        for (int e = 0; e < EPV; ++e) {
                            const uint64_t y = key64(E::get(cur[k], e), col_of(k, e));
                            if (y != 0 && y >= tau) {
                                const int at = atomicAdd(&s_n, 1);
                                if (at < kLpList) s_list[at] = y;
                            }
                        }
                }
                __syncthreads();
                if (s_n > kLpList) {
                    // too many: k block-wide maxima over the chunk and the list as it was
                    uint64_t last = ~0ull;
                    for (int q = 0; q < K; ++q) {
                        uint64_t b = 0;
#pragma unroll
                        for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
                            for (int e = 0; e < EPV; ++e) {
                                const uint64_t y = key64(E::get(cur[k], e), col_of(k, e));
                                if (y < last && y > b) b = y;
                            }
                        for (int i = tid; i < n_before; i += kLpThreads) {
                            const uint64_t y = s_list[i];
                            if (y < last && y > b) b = y;
                        }
#pragma unroll
                        for (int o = 16; o; o >>= 1) {
                            const uint64_t y = __shfl_xor_sync(0xffffffffu, b, o);
                            b = y > b ? y : b;
                        }
                        if (lane == 0) s_best[warp] = b;
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < kLpWarps; ++i) b = s_best[i] > b ? s_best[i] : b;
                        if (tid == 0) s_top[q] = b;
                        last = b;
                        __syncthreads();
                        if (b == 0) {  // no more elements
                            for (int i = q + 1 + tid; i < K; i += kLpThreads) s_top[i] = 0ull;
                            break;
                        }
                    }
                    __syncthreads();
                    if (tid < K) s_list[tid] = s_top[tid];
                    __syncthreads();
                    if (tid == 0) {
                        int n = 0;
                        while (n < K && s_list[n] != 0) ++n;
                        s_n = n;
                    }
                    __syncthreads();
                } else if (s_n > kLpList / 2 && ch + 1 < w.n_chunks) {
                    // keep the k largest
                    const int n = s_n;
                    rank_top(s_list, n, K, s_top);
                    __syncthreads();
                    if (tid < K) s_list[tid] = s_top[tid];
                    if (tid == 0) s_n = K;
                    __syncthreads();
                }
            }
            if (ch + 1 < w.n_chunks) {
#pragma unroll
                for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) cur[k][e] = nxt[k][e];
            }
        }
        // ---- the CTA's statistics and top k
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const Stat y{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.l, o),
                         __shfl_xor_sync(0xffffffffu, st.t, o)};
            st = join(st, y, c);
        }
        if (lane == 0) w_stat[warp] = st;
        if constexpr (TOP) rank_top(s_list, s_n, K, s_top);
        if (!joined) {  // remote shared memory only once every CTA of the cluster runs
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
            joined = true;
        }
        __syncthreads();
        Stat all = w_stat[0];
#pragma unroll
        for (int i = 1; i < kLpWarps; ++i) all = join(all, w_stat[i], c);
        if (CL > 1) {
            const int buf = it & 1;
            if (tid == 0) *cluster.map_shared_rank(&x_stat[buf][rank], 0) = all;
            if constexpr (TOP) {
                if (tid < K) *cluster.map_shared_rank(&x_top[buf][rank * K + tid], 0) = s_top[tid];
            }
            cluster.sync();
            if (rank == 0) {
                all = x_stat[buf][0];
                for (int i = 1; i < CL; ++i) all = join(all, x_stat[buf][i], c);
                if constexpr (TOP) {
                    // empty places (0) share a rank past every real key
                    for (int i = tid; i < CL * K; i += kLpThreads) {
                        const uint64_t mine = x_top[buf][i];
                        int r = 0;
                        for (int j = 0; j < CL * K; ++j) r += x_top[buf][j] > mine ? 1 : 0;
                        if (mine != 0 && r < K) s_top[r] = mine;
                    }
                    int have = 0;
                    for (int j = 0; j < CL * K; ++j) have += x_top[buf][j] != 0 ? 1 : 0;
                    if (tid >= have && tid < K) s_top[tid] = 0ull;
                    __syncthreads();
                }
            }
        }
        if (rank == 0) {
            const bool bad = !(all.l > 0.f) || !isfinite(all.l) || !isfinite(all.m);
            const float nan = __int_as_float(0x7fc00000);
            const float log_l = logf(all.l);
            if (tid == 0) {
                if (p.entropy) p.entropy[row] = bad ? nan : log_l - p.scale * (all.t / all.l);
                if (p.lse) p.lse[row] = bad ? nan : fmaf(p.scale, all.m, log_l);
                p.flags[row] = bad ? 1 : 0;
            }
            for (int i = tid; i < p.n_tokens; i += kLpThreads) {
                const int64_t at = (int64_t)row * p.n_tokens + i;
                const int tok = p.tokens[at];
                float lp = nan;
                if (tok < 0 || tok >= p.n_cols)
                    atomicOr(p.status, TF_DEV_BAD_TOKEN);
                else if (!bad)
                    lp = (E::load(w.at + tok) - all.m) * p.scale - log_l;
                p.token_logprobs[at] = lp;
            }
            if constexpr (TOP) {
                if (tid < K) {
                    const uint64_t y = s_top[tid];
                    const int64_t at = (int64_t)row * K + tid;
                    p.top_ids[at] = (bad || y == 0) ? -1 : (int)~(uint32_t)y;
                    p.top_logprobs[at] =
                        bad ? nan : (y == 0 ? -INFINITY : (unkey32((uint32_t)(y >> 32)) - all.m) * p.scale - log_l);
                }
            }
        }
        __syncthreads();  // the shared arrays serve the next row
        w = wn;
#pragma unroll
        for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) cur[k][e] = nxt[k][e];
    }
}

template <typename T, bool TOP>
cudaError_t launch_logprob(const LogprobParams &p, cudaStream_t st) {
    // few rows: a cluster a row, so that the row's columns spread over the SMs;
    // a CTA keeps at least one chunk's worth of columns
    const int chunk = Elem<T>::kPer * kLpBatch * kLpThreads;
    const int sms = device_sms();
    int cl = 1;
    while (cl < kLpMaxCluster && (int64_t)p.n_rows * cl < 2 * sms && (int64_t)cl * chunk < p.n_cols) cl *= 2;
    const int64_t groups = (int64_t)2 * sms / cl > 0 ? (int64_t)2 * sms / cl : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)cl, (unsigned)(p.n_rows < groups ? p.n_rows : groups));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<T, TOP>, p);
}

}  // namespace
}  // namespace tfp

using namespace tfp;

extern "C" tf_status tf_logprob_rows(const void *logits, int32_t logits_dtype, int32_t n_rows, int32_t n_cols,
                                     int64_t ld, float scale, const int32_t *tokens, int32_t n_tokens,
                                     float *token_logprobs, float *entropy, float *lse, int32_t top_k,
                                     int32_t *top_ids, float *top_logprobs, uint8_t *flags, uint32_t *status,
                                     tf_stream_t stream) {
    if (n_rows < 0 || n_cols <= 0 || ld < n_cols || n_tokens < 0 || top_k < 0 || !(scale >= 0x1p-64f) ||
        !(scale <= 0x1p64f) || (logits_dtype != TF_OUT_F32 && logits_dtype != TF_OUT_BF16))
        return TF_ERR_ARG;
    if (top_k > kLpMaxTop || n_cols > (1 << 24)) return TF_ERR_UNSUPPORTED;
    if (n_rows == 0) return TF_OK;
    if (!logits || !flags || !status || (n_tokens > 0 && (!tokens || !token_logprobs)) ||
        (top_k > 0 && (!top_ids || !top_logprobs)))
        return TF_ERR_ARG;
    const uintptr_t size = logits_dtype == TF_OUT_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % size != 0) return TF_ERR_ALIGN;
    LogprobParams p{logits, n_rows, n_cols, ld, scale, tokens, n_tokens, token_logprobs, entropy, lse, top_k, top_ids,
                    top_logprobs, flags, status};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (logits_dtype == TF_OUT_F32)
        return cuda_status(top_k ? launch_logprob<float, true>(p, st) : launch_logprob<float, false>(p, st));
    return cuda_status(top_k ? launch_logprob<uint16_t, true>(p, st) : launch_logprob<uint16_t, false>(p, st));
}
