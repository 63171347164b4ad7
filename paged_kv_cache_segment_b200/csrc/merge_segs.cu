// merge_segs.cu - the merge of tf_paged_attn_q8 and tf_paged_attn_shared: a
// stream's partials, and its rows' prefix's, into f32 or bf16 output rows.
//
// Per (row, head): M = max m_c, L = sum e^(m_c - M) l_c, out = sum e^(m_c - M)
// o_c / L over the partials with l_c > 0 of up to two sets, a flag when a
// partial's is set, the output is nonfinite or no partial holds a key.  A row's
// partial counts follow from its table entries, so no slot past them is read
// and none needs a marker; only rows the table names are written.
//
// One warp owns a (row, head) and 128 of its columns (float4 a lane; two warps
// at head dim 256), and loads up to sixteen partials' rows in one round: the
// kernel is a few microseconds of latency (its data, written just before, sits
// in L2), so what counts is how few round trips a warp makes.  Where a row may
// have more partials than that, a block of eight warps shares a (row,
// head), each warp (pair) every fourth or eighth round, and joins them in shared
// memory (one stream of 32,000 keys in 63 partials: 20 us with its decode kernel,
// 33 us with a warp for all of them; at 16 partials or fewer one round is shorter
// than the join).  It launches as a programmatic dependent of the partial kernel and
// reads the tables, which that kernel never writes, before it waits for the
// partials.
#include <cstdint>
#include <cuda_runtime.h>

#include "tf_common.cuh"
#include "tf_internal.h"

namespace tfp {
namespace {

// Partials an entry's rows have (0: a bad entry, no keys, or more rows than the
// partials' launch was sized for or more keys than a call takes, which this kernel reports).
__device__ __forceinline__ int seg_parts(const tf_seg &e, const PartSet &s, const MergeSegsParams &p, bool full) {
    if (e.n_rows > s.max_rows || e.n_keys > kMaxKeys) {
        atomicOr(p.status, TF_DEV_BAD_SEG);
        return 0;
    }
    const bool bad = e.q_row < 0 || e.n_rows < 0 || (int64_t)e.q_row + e.n_rows > p.n_rows_total ||
                     e.n_keys < (full ? 1 : e.n_rows) || e.pt_base < 0 || e.n_pages < 0 ||
                     (int64_t)e.pt_base + e.n_pages > p.pt_len ||
                     (int64_t)e.n_keys > ((int64_t)e.n_pages << p.log2_page);
    if (bad) return 0;
    int64_t len = s.split_keys;
    if (len <= 0) {
        len = ((int64_t)e.n_keys + s.n_splits - 1) / s.n_splits;
        len = ((len + (1 << p.log2_page) - 1) >> p.log2_page) << p.log2_page;
    }
    const int64_t n = ((int64_t)e.n_keys + len - 1) / len;
    return n <= s.n_splits ? (int)n : 0;
}

template <int D, bool BF16, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 256 : 128) merge_segs_kernel(const MergeSegsParams p) {
    constexpr int SL = D > 128 ? D / 128 : 1;  // warps across a (row, head)'s columns
    constexpr int DW = D / SL;                 // columns a warp
    constexpr int CH = WIDE ? 8 : 16;          // partials in flight
    constexpr int WAYS = WIDE ? 8 / SL : 1;    // warps along its partials
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sl = warp % SL, way = WIDE ? warp / SL : 0;
    // row of the stream x head
    const int64_t u = WIDE ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (4 / SL) + warp / SL;
    const tf_seg e = p.segs[blockIdx.y];
    const int i = (int)(u / p.hq), h = (int)(u - (int64_t)i * p.hq);
    // (all warps of a unit leave together)
    if (i >= min(e.n_rows, p.own.max_rows) || e.q_row < 0 || (int64_t)e.q_row + i >= p.n_rows_total) {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // no grid of this kernel ends before the partials' does
        return;
    }
    const int row = e.q_row + i;
    const int n_own = seg_parts(e, p.own, p, p.full != 0);
    bool bad = n_own == 0;
    int n_pre = 0;
    for (int b = 0; b < p.n_prefixes; b += 32) {  // the prefix whose rows hold this one
        tf_seg x{};
        if (b + lane < p.n_prefixes) x = p.prefixes[b + lane];
        const bool mine = x.n_rows > 0 && row >= x.q_row && row - x.q_row < x.n_rows;
        int n = 0;
        if (mine) n = seg_parts(x, p.prefix, p, true);
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        if (who) {
            n_pre = __shfl_sync(0xffffffffu, n, __ffs(who) - 1);
            bad |= n_pre == 0;
            break;
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // a partial kernel whose wait ran out left partials unwritten
    bad |= (*p.status & TF_DEV_TIMEOUT) != 0;
    const int64_t unit = (int64_t)row * p.hq + h;
    const int d0 = sl * DW + lane * 4;
    const bool col = lane * 4 < DW;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, L = 0.f;
    uint32_t f = bad ? 1u : 0u;
    const int total = bad ? 0 : n_pre + n_own;
    for (int c0 = way * CH; c0 < total; c0 += WAYS * CH) {
        float4 v[CH];
        float mc = -INFINITY, lc = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = c0 + k;
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < total && col) {
                const bool pre = c < n_pre;
                const float *o = pre ? p.prefix.o : p.own.o;
                const int64_t at = unit * (pre ? p.prefix.n_splits : p.own.n_splits) + (pre ? c : c - n_pre);
                v[k] = *reinterpret_cast<const float4 *>(o + at * D + d0);
            }
        }
        if (lane < CH && c0 + lane < total) {
            const int c = c0 + lane;
            const bool pre = c < n_pre;
            const PartSet &s = pre ? p.prefix : p.own;
            const int64_t at = unit * s.n_splits + (pre ? c : c - n_pre);
            mc = s.m[at];
            lc = s.l[at];
            f |= s.flag[at];
        }
        const bool live = lc > 0.f;
        float mx = live ? mc : -INFINITY;
#pragma unroll
        for (int x = CH / 2; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        mx = __shfl_sync(0xffffffffu, mx, 0);
        const float Mn = fmaxf(M, mx);
        if (Mn != -INFINITY) {
            const float r = M == -INFINITY ? 0.f : ex2((M - Mn) * kLog2e);
            L *= r;
            acc.x *= r;
            acc.y *= r;
            acc.z *= r;
            acc.w *= r;
            M = Mn;
        }
        const float w = live ? ex2((mc - M) * kLog2e) : 0.f;
        L += w * lc;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            // a partial without a key is never multiplied in: its o may be unwritten
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (wk != 0.f) {
                acc.x += wk * v[k].x;
                acc.y += wk * v[k].y;
                acc.z += wk * v[k].z;
                acc.w += wk * v[k].w;
            }
        }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        L += __shfl_xor_sync(0xffffffffu, L, x);
        f |= __shfl_xor_sync(0xffffffffu, f, x);
    }
    if constexpr (WIDE) {
        // the ways meet in the first one's warps
        __shared__ float4 s_acc[8][32];
        __shared__ float s_m[8], s_l[8];
        __shared__ uint32_t s_f[8];
        s_acc[warp][lane] = acc;
        if (lane == 0) {
            s_m[warp] = M;
            s_l[warp] = L;
            s_f[warp] = f;
        }
        __syncthreads();
        if (way != 0) return;
        float Mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < WAYS; ++k) Mx = fmaxf(Mx, s_m[k * SL + sl]);
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        L = 0.f;
#pragma unroll
        for (int k = 0; k < WAYS; ++k) {
            const int x = k * SL + sl;
            const float w = s_m[x] == -INFINITY ? 0.f : ex2((s_m[x] - Mx) * kLog2e);
            const float4 a = s_acc[x][lane];
            acc.x += w * a.x;
            acc.y += w * a.y;
            acc.z += w * a.z;
            acc.w += w * a.w;
            L += w * s_l[x];
            f |= s_f[x];
        }
    }
    acc.x /= L;
    acc.y /= L;
    acc.z /= L;
    acc.w /= L;
    bool nf = !(L > 0.f) || !isfinite(L);
    if (col) nf |= !isfinite(acc.x) || !isfinite(acc.y) || !isfinite(acc.z) || !isfinite(acc.w);
    uint32_t nfw = __any_sync(0xffffffffu, nf) ? 1u : 0u;
    if constexpr (SL > 1) {  // the other half's columns
        __shared__ uint32_t s_nf[4];
        if (lane == 0) s_nf[warp] = nfw;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (WIDE ? 0 : warp / SL)), "r"(32 * SL) : "memory");
#pragma unroll
        for (int k = 0; k < SL; ++k) nfw |= s_nf[(WIDE ? 0 : warp / SL) * SL + k];
    }
    f |= nfw;
    if (f) {
        const float qnan = __int_as_float(0x7fc00000);
        acc = make_float4(qnan, qnan, qnan, qnan);
    }
    if (col) {
        if constexpr (BF16) {
            const uint2 b = f ? make_uint2(0x7fc07fc0u, 0x7fc07fc0u)
                              : make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + unit * D + d0) = b;
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + unit * D + d0) = acc;
        }
    }
    if (lane == 0 && sl == 0) p.flags[unit] = (uint8_t)(f ? 1 : 0);
}

template <int D, bool BF16, bool WIDE>
cudaError_t launch_t(const MergeSegsParams &p, cudaStream_t st) {
    constexpr int units = WIDE ? 1 : (D > 128 ? 4 / (D / 128) : 4);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((int64_t)p.own.max_rows * p.hq + units - 1) / units), (unsigned)p.n_segs);
    cfg.blockDim = dim3(WIDE ? 256 : 128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge_segs_kernel<D, BF16, WIDE>, p);
}

template <int D>
cudaError_t launch_d(const MergeSegsParams &p, cudaStream_t st) {
    const bool wide = p.own.n_splits + (p.n_prefixes > 0 ? p.prefix.n_splits : 0) > 16;
    if (p.out_bf16) return wide ? launch_t<D, true, true>(p, st) : launch_t<D, true, false>(p, st);
    return wide ? launch_t<D, false, true>(p, st) : launch_t<D, false, false>(p, st);
}

}  // namespace

cudaError_t launch_merge_segs(const MergeSegsParams &p, int head_dim, cudaStream_t st) {
    if (p.n_segs == 0 || p.own.max_rows == 0) return cudaSuccess;
    switch (head_dim) {
        case 64: return launch_d<64>(p, st);
        case 128: return launch_d<128>(p, st);
        case 256: return launch_d<256>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tfp
