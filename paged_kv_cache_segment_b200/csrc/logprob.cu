// logprob.cu - tf_logprob_rows: log probabilities of given tokens, entropy and
// top alternatives of logit rows, in one pass over the logits.
//
// With m the row's largest logit, d = x - m, c = scale * log2(e), l = sum 2^(c d)
// and t = sum 2^(c d) d:
//   log p(x) = scale * d - ln l,  lse = scale * m + ln l,  H = ln l - scale * t / l.
// d <= 0, so both terms of H are >= 0 and nothing cancels; d is exact or rounded
// once, where x * c - m * c would carry the rounding of m * c into every term.
// Every thread keeps its own m, l and t; they are joined once a row.
//
// A row's columns are walked in chunks that a thread holds in registers (four
// 16-byte vectors), the next chunk's loads in flight while the current one folds,
// and without a barrier inside the row.  Vectors are aligned to 16 bytes whatever
// the row's own alignment: the grid of vectors starts up to 15 bytes before the
// row, and only the vectors that cross its ends load by element.
//
// Top k: elements are ordered by a 64-bit key, the value's order-preserving image
// above the complement of the column, so keys are distinct and ties go to the
// lower column.  During the pass a thread keeps only its largest value (and which
// chunk it came from, and the largest of its other chunks).  The k-th largest of
// some groups' largest values is a threshold that at least k elements reach, and
// few others do: only the chunks that reach it, nearly always one a thread, are
// read again, from L2, and the elements that reach it go to a list that is ranked
// by counting.  A list that overflows means ties (a mask of the type's lowest
// value, a row of equal logits): then the elements above the threshold are listed,
// and the columns equal to it in order until there are k.  If even the former
// overflow (columns left to a few threads only) the k largest keys are taken one
// at a time: slow, but never wrong.
//
// The logits are read once, so HBM bounds many rows; few rows, and the end of
// every row (a threshold, a second look, a ranking: 3 us), are latency.
//  - CTA mode: a CTA a row, several CTAs an SM so that one's row end hides behind
//    the others' streaming; with few rows 1,024 threads and a cluster of up to
//    eight CTAs a row, whose statistics and lists meet in distributed shared memory.
//  - warp mode, for short rows: a warp streams and ends a row of its own.
// Measured (bf16): 1,024 rows x 128,000 columns 59 us with 5 alternatives (262 MB,
// 4.4 TB/s), 68 with 20, 51 without; 62 rows with 20 14 us (12.5 with the logits in
// L2); one row of 128,000 f32 with 5 9 us; 20,000 rows x 3,000 51 us by warps, 151 by
// CTAs.  A persistent
// form with a warp of each CTA for the row ends was slower (75 us): one warp is
// slow at them.  So were five or six smaller CTAs an SM (56-60 us without
// alternatives).
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

constexpr int kLpBatch = 4;  // 16-byte vectors a thread holds of a chunk
constexpr int kLpMaxTop = 32;
constexpr int kLpMaxCluster = 8;
constexpr int kLpList = 1024;  // candidates of a row's columns in a CTA

// Threads a group, each group with its largest value: 64 groups of 128 or 256
// threads, 128 of more, at least kLpMaxTop of them.  With fewer columns than would
// fill that many groups the list holds them all (1,024-thread CTAs have more).
template <int NT>
constexpr int lp_group() { return NT == 128 ? 2 : (NT == 1024 ? 8 : 4); }
static_assert(kLpMaxTop * 4 * 8 <= kLpList, "a row without k filled groups must fit the list");

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

// A masked column (-infinity) enters the sums as this finite value, whose term
// is 0 and whose product with 0 is 0: x - m stays finite while m < 2^127 (past
// 2^128 - 2^126 it would be -infinity, and 0 times it NaN).  It also stands in
// for logits below it.  So a thread whose maximum is not far above it, or is
// 2^127 or more, takes the careful form instead, where x - m itself is clamped.
constexpr float kLpFloor = -0x1p126f, kLpLow = -0x1p125f, kLpHigh = 0x1p127f;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kPer = 4;  // elements of a 16-byte vector
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int e) { return __uint_as_float(w[e]); }
    // elements 2 i and 2 i + 1, no lower than kLpFloor (a NaN stays)
    static __device__ __forceinline__ uint64_t pair(const uint32_t (&w)[4], int i) {
        return pk2(max_nan(get(w, 2 * i), kLpFloor), max_nan(get(w, 2 * i + 1), kLpFloor));
    }
    // the largest of a vector's elements (NaN ignored)
    static __device__ __forceinline__ float most(const uint32_t (&w)[4]) {
        return fmaxf(fmaxf(get(w, 0), get(w, 1)), fmaxf(get(w, 2), get(w, 3)));
    }
    static __device__ __forceinline__ float load(const float *p) { return __ldg(p); }
    static __device__ __forceinline__ void put(uint32_t (&w)[4], int e, float x) { w[e] = __float_as_uint(x); }
};
template <>
struct Elem<uint16_t> {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int e) {
        return (e & 1) ? bf16_hi_to_f32(w[e >> 1]) : bf16_lo_to_f32(w[e >> 1]);
    }
    static __device__ __forceinline__ uint64_t pair(const uint32_t (&w)[4], int i) {
        uint32_t y;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w[i]), "r"(0xfe80fe80u));  // kLpFloor in bf16
        return pk2(bf16_lo_to_f32(y), bf16_hi_to_f32(y));
    }
    static __device__ __forceinline__ float most(const uint32_t (&w)[4]) {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w[0]), "r"(w[1]));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w[2]), "r"(w[3]));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return fmaxf(bf16_lo_to_f32(a), bf16_hi_to_f32(a));
    }
    static __device__ __forceinline__ float load(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
    static __device__ __forceinline__ void put(uint32_t (&w)[4], int e, float x) {
        const uint32_t b = __float_as_uint(x) >> 16;
        w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (b << 16) : (w[e >> 1] & 0xffff0000u) | b;
    }
};

// One row's columns, or a CTA's share of them: vectors [v0, v1), vector v holding
// columns v * kPer - mis and on; columns outside the row are masked.
template <typename T>
struct RowView {
    static constexpr int kPer = Elem<T>::kPer;
    const T *at;
    int mis, v0, v1, n_cols;

    RowView() = default;
    __device__ __forceinline__ RowView(const LogprobParams &p, int64_t row, int rank, int cl) {
        at = static_cast<const T *>(p.logits) + row * p.ld;
        n_cols = p.n_cols;
        mis = (int)((reinterpret_cast<uintptr_t>(at) & 15u) / sizeof(T));
        const int nv = (mis + n_cols + kPer - 1) / kPer, per = (nv + cl - 1) / cl;
        v0 = min(nv, rank * per);
        v1 = min(nv, v0 + per);
    }
    __device__ __forceinline__ void vec(int v, uint32_t (&x)[4]) const {
        const int c0 = v * kPer - mis;
        if (v < v1 && c0 >= 0 && c0 + kPer <= n_cols) {
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(at + c0));
            x[0] = y.x;
            x[1] = y.y;
            x[2] = y.z;
            x[3] = y.w;
        } else {
            x[0] = x[1] = x[2] = x[3] = kPer == 4 ? 0xff800000u : 0xff80ff80u;
            if (v < v1) {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (c0 + e >= 0 && c0 + e < n_cols) Elem<T>::put(x, e, Elem<T>::load(at + c0 + e));
            }
        }
    }
    // chunk `c` of thread `tid` of `nt`
    __device__ __forceinline__ void chunk(int c, int tid, int nt, uint32_t (&x)[kLpBatch][4]) const {
        const int v = v0 + c * kLpBatch * nt;  // the chunk's first vector
        if (v * kPer - mis >= 0 && v + kLpBatch * nt <= v1 && (v + kLpBatch * nt) * kPer - mis <= n_cols) {
            const uint4 *src = reinterpret_cast<const uint4 *>(at + (v * kPer - mis)) + tid;  // all inside the row
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k) {
                const uint4 y = __ldg(src + k * nt);
                x[k][0] = y.x;
                x[k][1] = y.y;
                x[k][2] = y.z;
                x[k][3] = y.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k) vec(v + k * nt + tid, x[k]);
        }
    }
    __device__ __forceinline__ int chunks(int nt) const {
        return max(1, (v1 - v0 + kLpBatch * nt - 1) / (kLpBatch * nt));
    }
};

// Folds a chunk into a thread's statistics; the chunk's largest value.
template <typename T>
__device__ __forceinline__ float fold(Stat &st, const uint32_t (&x)[kLpBatch][4], float c) {
    using E = Elem<T>;
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kLpBatch; ++k) mx = fmaxf(mx, E::most(x[k]));
    if (mx > st.m) st.to(mx, c);
    if ((st.m > kLpLow && st.m < kLpHigh) || st.m == -INFINITY) {
        // (all masked so far: the reference is 0, every term 0 or a NaN)
        const float ref = st.m == -INFINITY ? 0.f : -st.m;
        const uint64_t ref2 = pk2(ref, ref), c2 = pk2(c, c);
        uint64_t l2 = pk2(st.l, 0.f), t2 = pk2(st.t, 0.f);
#pragma unroll
        for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
            for (int e = 0; e < E::kPer / 2; ++e) {
                const uint64_t d2 = add2(E::pair(x[k], e), ref2);
                float y0, y1;
                unpk2(mul2(d2, c2), y0, y1);
                const uint64_t q2 = pk2(ex2(y0), ex2(y1));
                l2 = add2(l2, q2);
                t2 = fma2(q2, d2, t2);
            }
        float a, b;
        unpk2(l2, a, b);
        st.l = a + b;
        unpk2(t2, a, b);
        st.t = a + b;
    } else {
#pragma unroll
        for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
            for (int e = 0; e < E::kPer; ++e) {
                // (a masked column, or one more than FLT_MAX below: 0 * finite)
                const float d = max_nan(E::get(x[k], e) - st.m, -FLT_MAX);
                const float q = ex2(d * c);
                st.l += q;
                st.t = fmaf(q, d, st.t);
            }
    }
    return mx;
}

// A warp appends the columns equal to `tau`, lowest first, to a list of n keys
// until it has K; the new count.
template <typename T>
__device__ __forceinline__ int take_equal(const RowView<T> &w, float tau, uint64_t *list, int n, int K) {
    using E = Elem<T>;
    const int lane = threadIdx.x & 31;
    for (int v = w.v0; n < K && v < w.v1; v += 32) {
        uint32_t x[4];
        w.vec(v + lane, x);
        const int c0 = (v + lane) * E::kPer - w.mis;
        int mine = 0;
#pragma unroll
        for (int e = 0; e < E::kPer; ++e) mine += E::get(x, e) == tau ? 1 : 0;
        int before = mine;  // equal columns in this and the lower lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        const int found = __shfl_sync(0xffffffffu, before, 31);
        before -= mine;
#pragma unroll
        for (int e = 0; e < E::kPer; ++e)
            if (E::get(x, e) == tau) {
                if (n + before < K) list[n + before] = key64(tau, c0 + e);
                ++before;
            }
        n = min(K, n + found);
    }
    return n;
}

// Shared memory of a warp that ends a row.
template <int LIST>
struct FinishBuf {
    uint64_t list[LIST], top[kLpMaxTop];
    uint8_t hits[32];
    int n;
};

// A warp ends a row of its own, `own` being the lane's statistics and, if DEEP,
// `other` the largest of another part of the lane's columns.  Returns the joined
// ones; with TOP the K largest keys are in b.top, largest first, 0 past the
// unmasked columns.
template <typename T, bool TOP, bool DEEP, int LIST>
__device__ __forceinline__ Stat finish(const RowView<T> &w, const Stat &own, float other, FinishBuf<LIST> &b, int K,
                                       float c) {
    using E = Elem<T>;
    constexpr int EPV = E::kPer;
    const int lane = threadIdx.x & 31;
    Stat all = own;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Stat y{__shfl_xor_sync(0xffffffffu, all.m, o), __shfl_xor_sync(0xffffffffu, all.l, o),
                     __shfl_xor_sync(0xffffffffu, all.t, o)};
        all = join(all, y, c);
    }
    const float lm = own.m;  // the lane's largest
    if constexpr (TOP) {
        // ---- the threshold: the K-th largest of the lanes' largest values (equal ones rank by lane),
        // if DEEP of two a lane: of one, some 18 elements reach it for K = 14 but 130 for K = 32
        int r = 0, r2 = 0;
        if constexpr (!DEEP) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float y = __shfl_sync(0xffffffffu, lm, j);
                r += (y > lm || (y == lm && j < lane)) ? 1 : 0;
            }
            r2 = 32;
        } else {
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {  // (the others after every largest of the same value)
                const float y = __shfl_sync(0xffffffffu, lm, j), z = __shfl_sync(0xffffffffu, other, j);
                r += ((y > lm || (y == lm && j < lane)) ? 1 : 0) + (z > lm ? 1 : 0);
                r2 += (y >= other ? 1 : 0) + ((z > other || (z == other && j < lane)) ? 1 : 0);
            }
        }
        const uint32_t one = __ballot_sync(0xffffffffu, r == K - 1), two = __ballot_sync(0xffffffffu, r2 == K - 1);
        const float tau = one ? __shfl_sync(0xffffffffu, lm, __ffs(one) - 1)
                              : __shfl_sync(0xffffffffu, other, two ? __ffs(two) - 1 : 0);
        const int nk = (w.v1 - w.v0 + 31) / 32;  // vectors a lane
        // the lanes whose largest value is at least `want` (above it, if strict)
        auto find = [&](float want, bool strict) -> int {
            __syncwarp();
            const bool hit = (strict ? lm > want : lm >= want) && lm > -INFINITY;
            const uint32_t who = __ballot_sync(0xffffffffu, hit);
            if (hit) b.hits[__popc(who & ((1u << lane) - 1u))] = (uint8_t)lane;
            if (lane == 0) b.n = 0;
            __syncwarp();
            return __popc(who);
        };
        // a vector's elements at least (above, if strict) `want`, to the list
        auto take = [&](const uint32_t (&x)[4], int v, float want, bool strict) {
            const float most = E::most(x);
            if (!(strict ? most > want : most >= want) || most == -INFINITY) return;
            const int c0 = v * EPV - w.mis;
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const float y = E::get(x, e);
                if ((strict ? y > want : y >= want) && y > -INFINITY) {
                    const int at = atomicAdd(&b.n, 1);
                    if (at < LIST) b.list[at] = key64(y, c0 + e);
                }
            }
        };
        // those lanes' vectors, four a lane in flight; false if the list overflows
        auto look = [&](int n_hits, float want, bool strict) -> bool {
            const int total = n_hits * nk;
            for (int base = 0; base < total; base += 4 * 32) {
                uint32_t x[4][4];
                int v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int idx = base + 32 * k + lane, h = idx / nk;
                    v[k] = idx < total ? w.v0 + b.hits[h] + (idx - h * nk) * 32 : w.v1;
                    w.vec(v[k], x[k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) take(x[k], v[k], want, strict);
                __syncwarp();
                const int n = b.n;
                __syncwarp();
                if (n > LIST) return false;
            }
            return true;
        };
        bool ok = look(find(tau, false), tau, false);
        if (!ok && tau > -INFINITY) {
            // ties: what is above the threshold, then the first columns equal to it
            ok = look(find(tau, true), tau, true);
            int n = b.n;
            if (ok) n = take_equal(w, tau, b.list, n, K);
            __syncwarp();
            if (lane == 0 && ok) b.n = n;
            __syncwarp();
        }
        if (ok) {
            // ---- rank by counting: a key a lane
            const int n = b.n;
            for (int i = lane; i < ((n + 31) & ~31); i += 32) {
                const uint64_t mine = i < n ? b.list[i] : ~0ull;
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) rank += b.list[j] > mine ? 1 : 0;
                if (i < n && rank < K) b.top[rank] = mine;
            }
            for (int i = n + lane; i < K; i += 32) b.top[i] = 0ull;
        } else {
            // ---- one at a time: the largest key below the last one taken, a lane's share each
            uint64_t last = ~0ull, best = 0;
            bool stale = true;
            for (int q = 0; q < K; ++q) {
                if (stale) {
                    best = 0;
                    for (int v = w.v0 + lane; v < w.v1; v += 32 * kLpBatch) {
                        uint32_t x[kLpBatch][4];
#pragma unroll
                        for (int k = 0; k < kLpBatch; ++k) w.vec(v + 32 * k, x[k]);
#pragma unroll
                        for (int k = 0; k < kLpBatch; ++k)
#pragma unroll
                            for (int e = 0; e < EPV; ++e) {
                                const uint64_t y = key64(E::get(x[k], e), (v + 32 * k) * EPV - w.mis + e);
                                if (y < last && y > best) best = y;
                            }
                    }
                }
                __syncwarp();
                uint64_t top = best;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, top, o);
                    top = y > top ? y : top;
                }
                if (lane == 0) b.top[q] = top;
                last = top;
                stale = top != 0 && top == best;
            }
        }
        __syncwarp();
    }
    return all;
}

// A row's first 32 given tokens and their logits, a lane each, fetched while the
// row is read: after it the two loads, one behind the other, were a call's tail
// (one row of 128,000 f32 with 5: 8.6 us; 10.5 before this and the join of a
// cluster's lists by a thread a (key, list)).
struct GivenToken {
    int tok = -1;
    float x = 0.f;

    __device__ __forceinline__ void ask(const LogprobParams &p, int64_t row, bool here) {
        const int lane = threadIdx.x & 31;
        if (here && lane < p.n_tokens) tok = __ldg(p.tokens + row * p.n_tokens + lane);
    }
    template <typename T>
    __device__ __forceinline__ void fetch(const LogprobParams &p, const T *at) {
        if (tok >= 0 && tok < p.n_cols) x = Elem<T>::load(at + tok);
    }
};

// One warp writes a row's outputs.
template <typename T, bool TOP>
__device__ __forceinline__ void write_row(const LogprobParams &p, int64_t row, const Stat &all, const uint64_t *top,
                                          const GivenToken &given) {
    const int lane = threadIdx.x & 31, K = p.top_k;
    const bool bad = !(all.l > 0.f) || !isfinite(all.l) || !isfinite(all.m);
    const float nan = __int_as_float(0x7fc00000);
    const float log_l = logf(all.l);
    auto log_p = [&](float x) {
        float y = (x - all.m) * p.scale;
        // (a logit more than FLT_MAX below the largest: halved, the distance is a float again)
        if (y == -INFINITY && x != -INFINITY) y = (0.5f * x - 0.5f * all.m) * (2.f * p.scale);
        return y - log_l;
    };
    if (lane == 0) {
        if (p.entropy) p.entropy[row] = bad ? nan : log_l - p.scale * (all.t / all.l);
        if (p.lse) p.lse[row] = bad ? nan : fmaf(p.scale, all.m, log_l);
        p.flags[row] = bad ? 1 : 0;
    }
    const T *at = static_cast<const T *>(p.logits) + row * p.ld;
    for (int i = lane; i < p.n_tokens; i += 32) {
        const int64_t to = row * p.n_tokens + i;
        GivenToken g = given;
        if (i >= 32) {
            g.tok = p.tokens[to];
            g.fetch(p, at);
        }
        float lp = nan;
        if (g.tok < 0 || g.tok >= p.n_cols)
            atomicOr(p.status, TF_DEV_BAD_TOKEN);
        else if (!bad)
            lp = log_p(g.x);
        p.token_logprobs[to] = lp;
    }
    if constexpr (TOP) {
        if (lane < K) {
            const uint64_t y = top[lane];
            const int64_t to = row * K + lane;
            p.top_ids[to] = (bad || y == 0) ? -1 : (int)~(uint32_t)y;
            p.top_logprobs[to] =
                bad ? nan : (y == 0 ? -INFINITY : log_p(unkey32((uint32_t)(y >> 32))));
        }
    }
}

// ---- CTA mode: a CTA a row, or a cluster of CL
// Ranks the n distinct keys of `list` and puts the k largest, largest first,
// into `top` (0 past the n-th): a warp a key, 32 of the others at a time.
template <int NT>
__device__ __forceinline__ void rank_top(const uint64_t *list, int n, int k, uint64_t *top) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < n; i += NT / 32) {
        const uint64_t mine = list[i];
        int rank = 0;
        for (int j = 0; j < n; j += 32)
            rank += __popc(__ballot_sync(0xffffffffu, j + lane < n && list[min(j + lane, n - 1)] > mine));
        if (lane == 0 && rank < k) top[rank] = mine;
    }
    for (int i = n + threadIdx.x; i < k; i += NT) top[i] = 0ull;
}

// The K largest keys of a row's part whose list of columns that reach `tau` did not
// hold them all: ties.  A CTA lists what is above `tau`, then the columns equal to
// it, lowest first, until there are K; if that does not fit either it takes the keys
// one at a time.  (Seldom called, and apart from the kernel, which is short of
// registers: inside it the kernel spills, and rows without ties take 3% longer.)
template <typename T, int NT>
__device__ __noinline__ void top_of_ties(const T *at, int v0, int v1, int n_cols, float tau, uint64_t *list,
                                         int *count, uint64_t *best_of, int K, uint64_t *top) {
    using E = Elem<T>;
    const int tid = threadIdx.x;
    RowView<T> w;
    w.at = at;
    w.mis = (int)((reinterpret_cast<uintptr_t>(at) & 15u) / sizeof(T));
    w.v0 = v0;
    w.v1 = v1;
    w.n_cols = n_cols;
    auto all = [&](auto &&each) {  // the part's vectors, a batch at a time
        for (int v = v0 + tid; v < v1; v += kLpBatch * NT) {
            uint32_t x[kLpBatch][4];
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k) w.vec(v + k * NT, x[k]);
#pragma unroll
            for (int k = 0; k < kLpBatch; ++k) each(x[k], (v + k * NT) * E::kPer - w.mis);
        }
    };
    __syncthreads();  // every thread has read the count
    if (tid == 0) *count = 0;
    __syncthreads();
    if (tau > -INFINITY) {
        all([&](const uint32_t(&x)[4], int c0) {
            if (!(E::most(x) > tau)) return;
#pragma unroll
            for (int e = 0; e < E::kPer; ++e) {
                const float y = E::get(x, e);
                if (y > tau) {
                    const int i = atomicAdd(count, 1);
                    if (i < kLpList) list[i] = key64(y, c0 + e);
                }
            }
        });
        __syncthreads();
        int n = *count;
        if (n <= kLpList) {
            __syncthreads();
            if (tid < 32) {
                n = take_equal(w, tau, list, n, K);
                if (tid == 0) *count = n;
            }
            __syncthreads();
            rank_top<NT>(list, *count, K, top);
            return;
        }
    }
    uint64_t best = 0;
    auto look = [&](uint64_t below) {  // this thread's largest key below the last one taken
        best = 0;
        all([&](const uint32_t(&x)[4], int c0) {
#pragma unroll
            for (int e = 0; e < E::kPer; ++e) {
                const uint64_t key = key64(E::get(x, e), c0 + e);
                if (key < below && key > best) best = key;
            }
        });
    };
    look(~0ull);
    for (int q = 0; q < K; ++q) {
        uint64_t b = best;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const uint64_t y = __shfl_xor_sync(0xffffffffu, b, o);
            b = y > b ? y : b;
        }
        if ((tid & 31) == 0) best_of[tid >> 5] = b;
        __syncthreads();
        for (int i = 0; i < NT / 32; ++i) b = best_of[i] > b ? best_of[i] : b;
        if (tid == 0) top[q] = b;
        if (b != 0 && b == best) look(b);
        __syncthreads();
    }
}

template <typename T, bool TOP, int NT>
__global__ void __launch_bounds__(NT, NT >= 1024 ? 1 : 1024 / NT) logprob_kernel(const LogprobParams p) {
    using E = Elem<T>;
    constexpr int EPV = E::kPer;
    constexpr int NW = NT / 32, GT = lp_group<NT>(), NG = NT / GT;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ Stat w_stat[NW];
    __shared__ float s_group[TOP ? NG : 1], s_tau;
    __shared__ uint64_t s_list[TOP ? kLpList : 1], s_top[kLpMaxTop], s_best[NW];
    __shared__ int s_n;
    // rank 0's slots, filled by every CTA of the cluster
    __shared__ Stat x_stat[kLpMaxCluster];
    __shared__ uint64_t x_top[TOP ? kLpMaxCluster * kLpMaxTop : 1];
    // remote shared memory only once every CTA of the cluster runs: arrive here, wait before the first store
    if (CL > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const float c = p.scale * kLog2e;
    const int K = p.top_k;

    const int64_t row = blockIdx.x / (unsigned)CL;
    const RowView<T> w(p, row, rank, CL);
    const int n_chunks = w.chunks(NT);
    Stat st{-INFINITY, 0.f, 0.f};
    uint32_t cur[kLpBatch][4];
    w.chunk(0, tid, NT, cur);
    GivenToken given;
    given.ask(p, row, rank == 0 && warp == 0);
    if constexpr (TOP) {
        if (tid == 0) s_n = 0;
    }
    // the thread's chunk with its largest value, the largest of its other chunks
    int best_ch = 0;
    float second = -INFINITY;
    auto step = [&](const uint32_t (&x)[kLpBatch][4], int ch) {
        const float before = st.m, mx = fold<T>(st, x, c);
        if constexpr (TOP) {
            second = fmaxf(second, fminf(before, mx));
            best_ch = mx > before ? ch : best_ch;
        }
    };
    for (int ch = 0; ch < n_chunks; ch += 2) {
        uint32_t nxt[kLpBatch][4];
        if (ch + 1 < n_chunks) w.chunk(ch + 1, tid, NT, nxt);
        step(cur, ch);
        if (ch + 1 < n_chunks) {
            if (ch + 2 < n_chunks) w.chunk(ch + 2, tid, NT, cur);
            step(nxt, ch + 1);
        }
    }

    given.fetch(p, w.at);
    // ---- the CTA's statistics
    {
        Stat all = st;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const Stat y{__shfl_xor_sync(0xffffffffu, all.m, o), __shfl_xor_sync(0xffffffffu, all.l, o),
                         __shfl_xor_sync(0xffffffffu, all.t, o)};
            all = join(all, y, c);
        }
        if (lane == 0) w_stat[warp] = all;
    }
    if constexpr (TOP) {
        const float mine = st.m;  // this thread's largest logit
        // ---- the threshold: the K-th largest of the groups' largest values
        float gm = mine;
#pragma unroll
        for (int o = 1; o < GT; o <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
        if (tid % GT == 0) s_group[tid / GT] = gm;
        __syncthreads();
        {
            float v[NG / 32];
#pragma unroll
            for (int i = 0; i < NG / 32; ++i) v[i] = s_group[32 * i + lane];
#pragma unroll
            for (int j = 0; j < NG / NW; ++j) {
                const int g = warp * (NG / NW) + j;
                const float x = s_group[g];
                int r = 0;
#pragma unroll
                for (int i = 0; i < NG / 32; ++i)  // equal values rank by place
                    r += __popc(__ballot_sync(0xffffffffu, v[i] > x || (v[i] == x && 32 * i + lane < g)));
                if (lane == 0 && r == K - 1) s_tau = x;
            }
        }
        __syncthreads();
        const float tau = s_tau;
        // ---- the threads that reach it have their columns read again
        {
            auto push = [&](const uint32_t (&x)[4], int v) {
                const float most = E::most(x);
                if (!(most >= tau) || most == -INFINITY) return;
                const int c0 = v * EPV - w.mis;
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    const float y = E::get(x, e);
                    if (y >= tau && y > -INFINITY) {
                        const int i = atomicAdd(&s_n, 1);
                        if (i < kLpList) s_list[i] = key64(y, c0 + e);
                    }
                }
            };
            const bool hit = mine >= tau && mine > -INFINITY, more = second >= tau;
            // most have one chunk that reaches it: its vectors, eight threads' at a time
            uint32_t one = __ballot_sync(0xffffffffu, hit && !more);
            while (one) {
                int from = -1;  // lane 4 i + k: vector k of the i-th such thread
                for (int i = 0; i < 32 / kLpBatch && one; ++i, one &= one - 1)
                    if (lane / kLpBatch == i) from = __ffs(one) - 1;
                const int ch = __shfl_sync(0xffffffffu, best_ch, from < 0 ? 0 : from);
                if (from >= 0) {
                    const int v = w.v0 + (ch * kLpBatch + lane % kLpBatch) * NT + warp * 32 + from;
                    uint32_t x[4];
                    w.vec(v, x);
                    push(x, v);
                }
            }
            // the others' vectors, a vector a lane
            for (uint32_t all = __ballot_sync(0xffffffffu, hit && more); all; all &= all - 1) {
                const int first = w.v0 + warp * 32 + __ffs(all) - 1;
                for (int v = first + lane * NT; v - lane * NT < w.v1; v += 2 * 32 * NT) {
                    uint32_t x[2][4];
                    w.vec(v, x[0]);
                    w.vec(v + 32 * NT, x[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) push(x[k], v + k * 32 * NT);
                }
                // (a list that has overflowed is of no use: stop)
                if (*static_cast<volatile int *>(&s_n) > kLpList) break;
            }
        }
        __syncthreads();
        const int listed = s_n;
        if (listed > kLpList) {
            top_of_ties<T, NT>(w.at, w.v0, w.v1, w.n_cols, tau, s_list, &s_n, s_best, K, s_top);
        } else {
            rank_top<NT>(s_list, listed, K, s_top);
        }
    }
    __syncthreads();
    Stat all{-INFINITY, 0.f, 0.f};
    if (warp == 0) {
        if (lane < NW) all = w_stat[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const Stat y{__shfl_xor_sync(0xffffffffu, all.m, o), __shfl_xor_sync(0xffffffffu, all.l, o),
                         __shfl_xor_sync(0xffffffffu, all.t, o)};
            all = join(all, y, c);
        }
    }
    if (CL > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid == 0) *cluster.map_shared_rank(&x_stat[rank], 0) = all;
        if constexpr (TOP) {
            if (tid < K) *cluster.map_shared_rank(&x_top[rank * K + tid], 0) = s_top[tid];
        }
        cluster.sync();
        if (rank != 0) return;
        if (warp == 0) {
            all = lane < CL ? x_stat[lane] : Stat{-INFINITY, 0.f, 0.f};
#pragma unroll
            for (int o = kLpMaxCluster / 2; o; o >>= 1) {
                const Stat y{__shfl_xor_sync(0xffffffffu, all.m, o), __shfl_xor_sync(0xffffffffu, all.l, o),
                             __shfl_xor_sync(0xffffffffu, all.t, o)};
                all = join(all, y, c);
            }
        }
        if constexpr (TOP) {
            // a key's rank: its place in its own sorted list and, in each of the
            // others, how many are larger, a thread a list (CL is a power of two);
            // empty places (0) come last
            for (int i = tid; i < ((CL * K * CL + 31) & ~31); i += NT) {
                const int a = i % CL, key = min(i / CL, CL * K - 1), own = key / K;
                const uint64_t mine = x_top[key];
                const uint64_t *list = x_top + a * K;
                int lo = 0, hi = K;  // list[0 .. lo) before mine
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    // equal only when both are empty: by list, so that every place is taken once
                    if (list[mid] > mine || (list[mid] == mine && a < own))
                        lo = mid + 1;
                    else
                        hi = mid;
                }
                int r = a == own ? key % K : lo;
                for (int o = 1; o < CL; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
                if (a == 0 && i < CL * K * CL && r < K) s_top[r] = mine;
            }
            __syncthreads();
        }
    }
    // ---- warp 0 writes the row
    if (warp != 0) return;
    all.m = __shfl_sync(0xffffffffu, all.m, 0);
    all.l = __shfl_sync(0xffffffffu, all.l, 0);
    write_row<T, TOP>(p, row, all, s_top, given);
}

// ---- warp mode: a warp a row
constexpr int kLpWarpRows = 8;   // warps a CTA
constexpr int kLpWarpList = 256;

// DEEP: many alternatives, see finish().
template <typename T, bool TOP, bool DEEP>
__global__ void __launch_bounds__(kLpWarpRows * 32, 4) logprob_warp_kernel(const LogprobParams p) {
    __shared__ FinishBuf<TOP ? kLpWarpList : 1> s_fin[kLpWarpRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float c = p.scale * kLog2e;
    const int64_t row = (int64_t)blockIdx.x * kLpWarpRows + warp;
    if (row >= p.n_rows) return;
    const RowView<T> w(p, row, 0, 1);
    Stat st{-INFINITY, 0.f, 0.f};
    float other = -INFINITY;  // the largest outside the chunk with the lane's largest
    uint32_t a[kLpBatch][4], b[kLpBatch][4];
    const int n_chunks = w.chunks(32);
    w.chunk(0, lane, 32, a);
    GivenToken given;
    given.ask(p, row, true);
    auto step = [&](const uint32_t (&x)[kLpBatch][4]) {
        const float before = st.m, mx = fold<T>(st, x, c);
        if constexpr (DEEP) other = fmaxf(other, fminf(before, mx));
    };
    for (int ch = 0; ch < n_chunks; ch += 2) {
        if (ch + 1 < n_chunks) w.chunk(ch + 1, lane, 32, b);
        step(a);
        if (ch + 1 < n_chunks) {
            if (ch + 2 < n_chunks) w.chunk(ch + 2, lane, 32, a);
            step(b);
        }
    }
    if (DEEP && n_chunks == 1) {
        // of one chunk, the second of its vectors' largest: a row may fill two vectors only (60,000 rows x 512 with 32:
        // 158 us; 340 when it was the smaller of the two halves' largest, of which such rows have one)
        static_assert(kLpBatch == 4, "the second of four");
        const float v0 = Elem<T>::most(a[0]), v1 = Elem<T>::most(a[1]);
        const float v2 = Elem<T>::most(a[2]), v3 = Elem<T>::most(a[3]);
        other = max3(fminf(v0, v1), fminf(v2, v3), fminf(fmaxf(v0, v1), fmaxf(v2, v3)));
    }
    given.fetch(p, w.at);
    const Stat all = finish<T, TOP, DEEP>(w, st, other, s_fin[warp], p.top_k, c);
    write_row<T, TOP>(p, row, all, s_fin[warp].top, given);
}

template <typename T, bool TOP, int NT>
cudaError_t launch_cta(const LogprobParams &p, int cl, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.n_rows * (unsigned)cl);
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<T, TOP, NT>, p);
}

template <typename T, bool TOP>
cudaError_t launch_logprob(const LogprobParams &p, cudaStream_t st) {
    const int sms = device_sms();
    const int chunk = Elem<T>::kPer * kLpBatch;  // columns a thread holds
    // short rows (up to four chunks of a warp): a warp a row (60,000 rows x 1,000 with 5: 91 us; 356 by CTAs of 64)
    if (p.n_cols <= 4 * 32 * chunk && p.n_rows > 4 * sms) {
        const int64_t grid = ((int64_t)p.n_rows + kLpWarpRows - 1) / kLpWarpRows;
        // (20,000 rows x 3,000 with 32: 102 us deep, 298 not; 60,000 x 1,000 with 20: 140 and 134)
        if (TOP && p.top_k > 24)
            logprob_warp_kernel<T, TOP, TOP><<<(unsigned)grid, kLpWarpRows * 32, 0, st>>>(p);
        else
            logprob_warp_kernel<T, TOP, false><<<(unsigned)grid, kLpWarpRows * 32, 0, st>>>(p);
        return cudaGetLastError();
    }
    // many rows: eight CTAs an SM where a row is short (4,000 rows x 32,000 with 20: 85 us, 106 by four), else four
    // (1,024 x 128,000 with 20: 68 us, 71 by eight)
    if (p.n_rows > 4 * sms && p.n_cols <= 2 * 1024 * chunk) return launch_cta<T, TOP, 128>(p, 1, st);
    if (p.n_rows > 2 * sms || p.n_cols <= 256 * chunk) return launch_cta<T, TOP, 256>(p, 1, st);
    if (p.n_rows > sms) return launch_cta<T, TOP, 512>(p, 1, st);
    // a CTA an SM: a cluster a row while there are SMs for it and columns to fill its threads (62 rows x 128,000 with
    // 20: 14 us; two more by clusters of four CTAs of 512, two an SM)
    int cl = 1;
    while (cl < kLpMaxCluster && p.n_rows * 2 * cl <= sms && cl * 1024 * chunk < p.n_cols) cl *= 2;
    return launch_cta<T, TOP, 1024>(p, cl, st);
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
