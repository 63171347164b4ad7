// decode_q8.cu - split-KV partials over an 8-bit cache for decode-shaped work
// (at most 8 queries per (stream, kv-head)): a persistent, warp-specialized
// kernel, the 8-bit counterpart of the one in decode_ws.cu, whose work items,
// order, barriers and abort path it shares.
//
// HBM bounds it: a (key, kv-head) is 2 (D + 1) bytes, about half of bf16's, so
// each key also has half the time, and the kernel is built to spend few
// instructions on one.
//  - The producer warp's lane 0 issues TMA boxes of codes (one per page and
//    128-byte slab, swizzled) into a ring of 64-key stages; its lanes copy the
//    tile's scale bytes beside them in 8-byte pieces (cp.async, which arrive on
//    the same barrier), 8 keys being the smallest page.
//  - Codes go to the tensor cores as f16: exact, one conversion instruction per
//    two codes.  With the keys as the MMA's M side a warp converts each code of
//    its 16 keys once for all 8 queries.  The order of the contraction's columns
//    and of the output's rows is free, so the fragments are taken as the bytes
//    lie: a thread's four bytes of K are its k columns (2t, 2t+1, 2t+8, 2t+9)
//    as columns 4t .. 4t+3, with Q's fragment in the same order; a transposed
//    pair of V bytes is rows g and g + 8 as columns 2g and 2g + 1.
//  - Q is bf16; a query's row is scaled by a power of two so that its largest
//    element is in [2^14, 2^15) and fed as f16, exact for every element within
//    2^-29 of the largest and off by 2^-40 of it below that.
//  - Scales never touch the codes.  K's multiplies the score.  V's joins the
//    weight: with s_j the score and e_j the value's scale, both in base 2,
//    l = sum 2^(s_j - m) and o = sum 2^((s_j - m) + (e_j - r)) c_j, r being a whole
//    number, so that e_j - r is exact and a weight carries the rounding of s_j - m
//    alone, whatever the value rows' sizes.  It is fed as f16 hi + f16 lo (two MMAs
//    into one fp32 accumulator; see kRefLift for what they hold).
//  - The references move only when a term would pass 2^15, so a tile takes one
//    vote instead of two butterfly maxima.
// Measured (partials and merge): 16 streams of 1,024-8,192 keys, 32/8 heads, D 128
// (123 MB) in 31.7 us, 3.9 TB/s, 30 of them this kernel; D 256 33.6 us, D 64 42.5 us
// for as many bytes (a key there has a quarter of the time; four CTAs an SM, where
// three took 45 us); one stream of 32,000 keys 20.7 us; two streams of 37 and 70
// keys, written directly, 7.2 us.  By stamps in a copy a CTA of the first has its first
// tile after 4.8 us (table, page ids, copies, one after another), then takes 20 tiles
// of 0.97 us and 1.5 us to combine and write: 26 us in the middle, 28 at the slowest.
// Of a tile's 1,830 cycles its warps wait 290 for the copies (D 64 570 of 1,740, D 256
// 560 of 2,560): what holds it is the codes' way through the MMAs, more than the loads.
// Tried and not kept: four CTAs an SM at D 128 with two stages each (36 us where three
// took 30), one with three stages at D 256 (43 us, 32).
#include <atomic>
#include <cfloat>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tf_common.cuh"
#include "tf_internal.h"
#include "tf_q8.cuh"
#include "tf_sm100.cuh"
#include "tma_host.h"
#include "ws_items.cuh"

namespace tfp {
namespace {

template <int D>
struct Q8Cfg {
    static constexpr int NC = 4;  // consumer warps, 16 keys of a tile each
    static constexpr int kThreads = (NC + 1) * 32;
    static constexpr int TK = 16 * NC;
    static constexpr int kRow = D < 128 ? D : 128;  // bytes of a slab's row
    static constexpr int kSlab = TK * kRow;
    static constexpr int kSlabs = D / kRow;
    static constexpr int kTileBytes = kSlabs * kSlab;
    // codes of K, codes of V, scale bytes of K and of V, to a multiple of 1,024
    static constexpr int kOffScale = 2 * kTileBytes;
    static constexpr int kStageBytes = kOffScale + 1024;
    static constexpr int kStages = D == 256 ? 2 : (D == 128 ? 3 : 4);
    static constexpr int kNQ = 2;
    static constexpr int kPrefixMax = 256;
    static constexpr int kMinBlocks = D == 256 ? 2 : (D == 128 ? 3 : 4);
    static constexpr int kQBytes = kWsQ * D * 2;
    static constexpr int kCombStride = D + 4;  // floats a query row of the combine buffer
    static constexpr int kCombBytes = (NC / 2) * kWsQ * kCombStride * 4;
    static constexpr int kOffQ = kStages * kStageBytes;
    static constexpr int kOffComb = kOffQ + kNQ * kQBytes;
    static constexpr int kOffPrefix = kOffComb + kCombBytes;
    static constexpr int kSmem = kOffPrefix + 3 * (kPrefixMax + 1) * 4 + 1024;
};

// Byte offset of 16-byte chunk c (of a slab) of row r: the TMA swizzle's.
template <int D>
__device__ __forceinline__ uint32_t q8_chunk(int r, int c) {
    using C = Q8Cfg<D>;
    if constexpr (C::kRow == 128)
        return (uint32_t)((c >> 3) * C::kSlab + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    else
        return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void cp_async_8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival on `bar` once its cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// DIRECT: one split a stream, so an item's rows are final and go to p.out.
template <int D, int TYPE, bool DIRECT>
__global__ void __launch_bounds__(Q8Cfg<D>::kThreads, Q8Cfg<D>::kMinBlocks)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const WsParams p) {
    using C = Q8Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[C::kStages], empty_bar[C::kStages];
    __shared__ __align__(8) uint64_t qfull_bar[C::kNQ], qempty_bar[C::kNQ];
    __shared__ uint32_t s_meta[C::kStages];
    __shared__ WsItem s_item[C::kNQ];
    __shared__ float comb_m[C::NC / 2][kWsQ], comb_r[C::NC / 2][kWsQ], comb_l[C::NC / 2][kWsQ];
    __shared__ uint32_t comb_f[C::NC / 2][kWsQ];
    __shared__ int s_total, s_full;
    __shared__ int s_bucket[kWsBuckets];
    __shared__ uint32_t s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t lim = p.wait_ns ? p.wait_ns : 2000000000ull;  // every bounded wait's limit
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    unsigned char *base_ptr = smem_raw + (sbase - sraw);
    int *prefix = reinterpret_cast<int *>(base_ptr + C::kOffPrefix);
    int *prefix_full = prefix + (C::kPrefixMax + 1);
    int *tail_order = prefix_full + (C::kPrefixMax + 1);
    float *comb_o = reinterpret_cast<float *>(base_ptr + C::kOffComb);

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&full_bar[i]), 1 + 32);  // lane 0's expect_tx, every lane's scale bytes
            mbar_init(smem_u32(&empty_bar[i]), C::NC);
        }
        for (int i = 0; i < C::kNQ; ++i) {
            mbar_init(smem_u32(&qfull_bar[i]), 1);
            mbar_init(smem_u32(&qempty_bar[i]), C::NC);
        }
        fence_barrier_init();
        s_abort = 0;
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 1) {
        // the page table's first 16 KB into L2 while warp 0 works out the items
        const int n = min(p.pt_len, 4096);
        for (int i = lane * 32; i < n; i += 32 * 32) prefetch_l2(p.page_table + i);
    }
    if (warp == 0)
        ws_build_order<false, C::TK>(p, lane, prefix, prefix_full, tail_order, s_bucket, &s_total, &s_full);
    __syncthreads();
    const int total = s_total, n_full = s_full;
    const int bid = (int)blockIdx.x, grid = (int)gridDim.x;

    // final rows that no item writes: NaN, flagged
    auto flag_rows = [&](int q_row, int rows, int h0, int heads, int from, int step) {
        for (int x = from; x < rows * heads * D; x += step) {
            const int q = x / D, i = q / heads;
            const int64_t unit = (int64_t)(q_row + i) * p.hq + h0 + (q - i * heads);
            if (p.out_bf16)
                static_cast<uint16_t *>(p.out)[unit * D + x % D] = 0x7fc0;
            else
                static_cast<float *>(p.out)[unit * D + x % D] = __int_as_float(0x7fc00000);
            if (x % D == 0) p.out_flags[unit] = 1;
        }
    };
    if (warp == C::NC) {
        // ---- producer warp: the items in order, a tile a stage; page ids come
        // a window of 32 at a time, the next item's before this one's tiles
        if (!p.test_idle) {
            const int P = 1 << p.log2_page, BR = P < C::TK ? P : C::TK, n_box = C::TK / BR;
            auto load_window = [&](const WsItem &w, int w0) -> int {
                const int idx = w0 + lane;
                return idx < w.n_pg ? p.page_table[w.pt_base + idx] : -2;
            };
            uint32_t tc = 0, qc = 0;
            bool ok = true;
            auto publish = [&](const WsItem &w) -> bool {
                const uint32_t qs = qc % C::kNQ;
                if (qc >= (uint32_t)C::kNQ && !mbar_wait(smem_u32(&qempty_bar[qs]), ((qc / C::kNQ) - 1) & 1, lim))
                    return false;
                if (lane == 0) {
                    s_item[qs] = w;
                    const uint32_t qdst = sbase + C::kOffQ + qs * C::kQBytes;
                    const uint32_t qbytes = (uint32_t)(p.group * D * 2);
                    mbar_arrive_expect_tx(smem_u32(&qfull_bar[qs]), qbytes * w.n_rows);
                    for (int i = 0; i < w.n_rows; ++i)
                        bulk_load(qdst + i * qbytes, p.q + ((int64_t)(w.q_row + i) * p.hq + w.g * p.group) * D,
                                  qbytes, smem_u32(&qfull_bar[qs]));
                }
                ++qc;
                return true;
            };
            int k = 0, L = ws_snake(0, bid, grid);
            WsItem it{};
            int win = 0, w0 = 0;
            if (L < total) {
                it = ws_resolve<false>(p, prefix, prefix_full, tail_order, n_full, L);
                w0 = it.key_lo >> p.log2_page;
                win = load_window(it, w0);
                ok = publish(it);
            }
            while (L < total && ok) {
                const int L_next = ws_snake(k + 1, bid, grid);
                WsItem nx{};
                int win_next = 0, w0_next = 0;
                bool sent_next = false;
                auto prep_next = [&]() -> bool {
                    sent_next = true;
                    if (L_next >= total) return true;
                    nx = ws_resolve<false>(p, prefix, prefix_full, tail_order, n_full, L_next);
                    w0_next = nx.key_lo >> p.log2_page;
                    win_next = load_window(nx, w0_next);
                    return publish(nx);
                };
                for (int j0 = it.key_lo; j0 < it.key_hi;) {
                    const int rows = min(C::TK, it.key_hi - j0);
                    const uint32_t st = tc % C::kStages;
                    if (tc >= (uint32_t)C::kStages &&
                        !mbar_wait(smem_u32(&empty_bar[st]), ((tc / C::kStages) - 1) & 1, lim)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dK = sbase + st * C::kStageBytes, dV = dK + C::kTileBytes;
                    const uint32_t fb = smem_u32(&full_bar[st]);
                    if (((j0 + rows - 1) >> p.log2_page) - w0 >= 32) {  // past the window: slide it
                        w0 = j0 >> p.log2_page;
                        win = load_window(it, w0);
                    }
                    // lanes 0-7: the 8-byte pieces of K's scale bytes, 8-15: V's
                    {
                        const int key0 = j0 + (lane & 7) * 8;
                        const int id = __shfl_sync(0xffffffffu, win, ((key0 >> p.log2_page) - w0) & 31);
                        if (lane < 16 && key0 < j0 + rows && id >= 0 && id < p.n_pages) {
                            const uint8_t *src = (lane < 8 ? p.k_scale : p.v_scale) +
                                                 (((int64_t)id * p.hkv + it.g) << p.log2_page) + (key0 & (P - 1));
                            cp_async_8(dK + C::kOffScale + (lane < 8 ? 0 : C::TK) + (lane & 7) * 8, src);
                        }
                    }
                    int pid[C::TK / 8];
                    uint32_t bad = 0, bytes = 0;
                    for (int b = 0; b < n_box; ++b) {
                        const int key0 = j0 + b * BR;
                        const int id = __shfl_sync(0xffffffffu, win, ((key0 >> p.log2_page) - w0) & 31);
                        pid[b] = -1;
                        if (key0 < j0 + rows) {
                            if (id < 0 || id >= p.n_pages)
                                bad = 1;
                            else {
                                pid[b] = id;
                                bytes += 2u * BR * C::kRow * C::kSlabs;
                            }
                        }
                    }
                    if (lane == 0) {
                        s_meta[st] = bad;
                        mbar_arrive_expect_tx(fb, bytes);
                        for (int b = 0; b < n_box; ++b) {
                            if (pid[b] < 0) continue;
                            const int slot = (j0 + b * BR) & (P - 1);
#pragma unroll
                            for (int s = 0; s < C::kSlabs; ++s) {
                                tma_load_4d(dK + s * C::kSlab + b * BR * C::kRow, &tmK, fb, C::kRow * s, slot, it.g,
                                            pid[b]);
                                tma_load_4d(dV + s * C::kSlab + b * BR * C::kRow, &tmV, fb, C::kRow * s, slot, it.g,
                                            pid[b]);
                            }
                        }
                        if (bad) atomicOr(p.status, TF_DEV_BAD_PAGE);
                    }
                    cp_async_arrive(fb);
                    ++tc;
                    j0 += rows;
                    if (!sent_next && !prep_next()) {
                        ok = false;
                        break;
                    }
                }
                if (ok && !sent_next && !prep_next()) ok = false;
                L = L_next;
                ++k;
                it = nx;
                win = win_next;
                w0 = w0_next;
            }
            if (!ok && lane == 0) {
                atomicOr(p.status, TF_DEV_TIMEOUT);
                s_abort = 1;
            }
        }
        if constexpr (DIRECT) {
            for (int s = bid; s < p.n_segs; s += grid)
                if (prefix[s + 1] == prefix[s]) {  // an entry found bad (or with no rows)
                    // its rows that the launch holds, as the merge flags them
                    const tf_seg e = p.segs[s];
                    const int rows = e.q_row < 0 ? 0 : min(min(e.n_rows, p.max_rows), p.n_rows_total - e.q_row);
                    if (rows > 0) flag_rows(e.q_row, rows, 0, p.hq, lane, 32);
                }
        }
        cp_async_commit();
        cp_async_wait<0>();  // no scale byte is in flight when this CTA ends
        // (the merge, which waits for this grid; final rows have none, and another launch need not wait)
        if constexpr (!DIRECT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    } else {
        // ---- consumer warps
        const int gq = lane >> 2, t4 = lane & 3;
        uint32_t tc = 0, qc = 0;
        for (int k = 0, L = ws_snake(0, bid, grid); L < total; L = ws_snake(++k, bid, grid)) {
            const uint32_t qs = qc % C::kNQ;
            const bool q_ok = mbar_wait(smem_u32(&qfull_bar[qs]), (qc / C::kNQ) & 1, lim);
            WsItem it = s_item[qs];
            if (!q_ok) it.key_lo = it.key_hi = 0;
            const int q_item = it.n_rows * p.group;
            // query gq's columns 16 c + 4 t4 .. + 3 as f16, scaled so the row's
            // largest magnitude is in [2^14, 2^15)
            uint32_t qb[D / 16][2];
            float fq;  // scale * log2(e) over that power of two
            {
                const unsigned char *qrow = base_ptr + C::kOffQ + qs * C::kQBytes + gq * (D * 2) + t4 * 8;
                uint32_t amax = 0;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint2 w = make_uint2(0u, 0u);
                    if (gq < q_item) w = *reinterpret_cast<const uint2 *>(qrow + c * 32);
                    qb[c][0] = w.x;
                    qb[c][1] = w.y;
                    amax = max(amax, max(max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu),
                                         max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu)));
                }
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^e, e = 14 - exponent of amax, at most 120 so that 2^-e is normal
                const int e = min(120, 14 + 127 - (int)(amax >> 7));
                const float up = __uint_as_float((uint32_t)(e + 127) << 23);
                fq = p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
                if (amax >= 0x7f80u) fq = __int_as_float(0x7fc00000);  // a nonfinite query: every score NaN
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        qb[c][x] = pack_f16x2(bf16_lo_to_f32(qb[c][x]) * up, bf16_hi_to_f32(qb[c][x]) * up);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&qempty_bar[qs]));
            ++qc;

            // per-thread state: queries 2 t4 and 2 t4 + 1; o's rows: columns 16 u + 2 gq (+ 1)
            const int qa = 2 * t4, qb_ = qa + 1;
            const float fa = __shfl_sync(0xffffffffu, fq, 4 * qa), fb_ = __shfl_sync(0xffffffffu, fq, 4 * qb_);
            const int lim_a = qa < q_item ? min(it.key_hi, it.causal0 + qa / p.group) : it.key_hi;
            const int lim_b = qb_ < q_item ? min(it.key_hi, it.causal0 + qb_ / p.group) : it.key_hi;
            float o[D / 16][4];
#pragma unroll
            for (int u = 0; u < D / 16; ++u) o[u][0] = o[u][1] = o[u][2] = o[u][3] = 0.f;
            // m: reference of the scores (-FLT_MAX before the first key, so nothing is
            // special-cased); m + r: that of score + value scale (base 2 both)
            float m0 = -FLT_MAX, m1 = -FLT_MAX, r0 = 0.f, r1 = 0.f, l0 = 0.f, l1 = 0.f;
            float n0 = INFINITY, n1 = INFINITY;  // the smallest scores (-inf: an overflow, flagged)
            uint32_t e0 = 0, e1 = 0, tb0 = 0, tb1 = 0, badp = 0, vtop = 0;
            const uint64_t f2 = pk2(fa, fb_);
            const int kb = warp * 16;
            bool aborted = !q_ok;

            for (int j0 = it.key_lo; j0 < it.key_hi;) {
                const int rows = min(C::TK, it.key_hi - j0);
                const uint32_t st = tc % C::kStages;
                if (!mbar_wait(smem_u32(&full_bar[st]), (tc / C::kStages) & 1, lim)) {
                    aborted = true;
                    break;
                }
                badp |= s_meta[st];
                const uint32_t sK = sbase + st * C::kStageBytes, sV = sK + C::kTileBytes;
                bool wrote = false;
                if (kb < rows) {
                    if (kb + 16 > rows) {
                        // value rows past the tile's keys hold other rows' codes: zero them
                        unsigned char *vrows = base_ptr + st * C::kStageBytes + C::kTileBytes;
                        for (int x = lane; x < 16 * (D / 16); x += 32) {
                            const int r = kb + x / (D / 16), ch = x % (D / 16);
                            if (r >= rows)
                                *reinterpret_cast<uint4 *>(vrows + q8_chunk<D>(r, ch)) = make_uint4(0, 0, 0, 0);
                        }
                        wrote = true;
                        __syncwarp();
                    }
                    // ---- S^T = K Q^T for this warp's 16 keys (two accumulators halve the MMA chain)
                    float s4[4] = {0.f, 0.f, 0.f, 0.f}, s5[4] = {0.f, 0.f, 0.f, 0.f};
                    const int lr = kb + (lane & 7) + (((lane >> 3) & 1) << 3), lc = lane >> 4;
#pragma unroll
                    for (int c = 0; c < D / 16; c += 2) {
                        uint32_t w[4], a[4];
                        ldsm_x4(sK + q8_chunk<D>(lr, c + lc), w[0], w[1], w[2], w[3]);
                        q8_to_f16<TYPE>(w[0], a[0], a[2]);
                        q8_to_f16<TYPE>(w[1], a[1], a[3]);
                        mma_f16(s4, a[0], a[1], a[2], a[3], qb[c][0], qb[c][1]);
                        q8_to_f16<TYPE>(w[2], a[0], a[2]);
                        q8_to_f16<TYPE>(w[3], a[1], a[3]);
                        mma_f16(s5, a[0], a[1], a[2], a[3], qb[c + 1][0], qb[c + 1][1]);
                    }
                    // ---- scores and value exponents of keys kb + gq and kb + gq + 8
                    const unsigned char *sc = base_ptr + st * C::kStageBytes + C::kOffScale + kb + gq;
                    const uint32_t eka = sc[0], ekb = sc[8], eva = sc[C::TK], evb = sc[C::TK + 8];
                    // (a marked row's scale is inf here: inf * 0, its codes' sum, is NaN)
                    const float ska = __uint_as_float(eka << 23), skb = __uint_as_float(ekb << 23);
                    uint64_t xa = mul2(add2(pk2(s4[0], s4[1]), pk2(s5[0], s5[1])), mul2(pk2(ska, ska), f2));
                    uint64_t xb = mul2(add2(pk2(s4[2], s4[3]), pk2(s5[2], s5[3])), mul2(pk2(skb, skb), f2));
                    float fva = (float)((int)eva - kE8Bias), fvb = (float)((int)evb - kE8Bias);
                    if (kb + 16 <= rows && j0 + kb + 16 <= it.full_hi) {
                        // every query sees these keys: NaN and +inf reach l, -inf is caught
                        // here, a marked value row at the end
                        float x0, x1, x2, x3;
                        unpk2(xa, x0, x1);
                        unpk2(xb, x2, x3);
                        n0 = min3(n0, x0, x2);
                        n1 = min3(n1, x1, x3);
                        vtop = max(vtop, max(eva, evb));
                    } else {
                        const int ra = kb + gq, rb = ra + 8, ka = j0 + ra, kbk = j0 + rb;
                        const bool va0 = ra < rows && ka < lim_a, va1 = ra < rows && ka < lim_b;
                        const bool vb0 = rb < rows && kbk < lim_a, vb1 = rb < rows && kbk < lim_b;
                        float x0, x1, x2, x3;
                        unpk2(xa, x0, x1);
                        unpk2(xb, x2, x3);
                        e0 = max(e0, max(va0 ? exp_bits(x0) : 0u, vb0 ? exp_bits(x2) : 0u));
                        e1 = max(e1, max(va1 ? exp_bits(x1) : 0u, vb1 ? exp_bits(x3) : 0u));
                        // a value row marked nonfinite flags the queries that see it and weighs nothing
                        if (eva == kE8Nan) {
                            tb0 |= va0;
                            tb1 |= va1;
                            fva = -INFINITY;
                        }
                        if (evb == kE8Nan) {
                            tb0 |= vb0;
                            tb1 |= vb1;
                            fvb = -INFINITY;
                        }
                        xa = pk2(va0 ? x0 : -INFINITY, va1 ? x1 : -INFINITY);
                        xb = pk2(vb0 ? x2 : -INFINITY, vb1 ? x3 : -INFINITY);
                    }
                    // ---- exponents over the references, which move when one would pass 2^15
                    uint64_t da, db, ga, gb;
                    float d0, d1, d2, d3, g0, g1, g2, g3;
                    auto over = [&]() {
                        const uint64_t nm = pk2(-m0, -m1), nr = pk2(-r0, -r1);
                        da = add2(xa, nm);
                        db = add2(xb, nm);
                        ga = add2(da, add2(pk2(fva, fva), nr));
                        gb = add2(db, add2(pk2(fvb, fvb), nr));
                        unpk2(da, d0, d1);
                        unpk2(db, d2, d3);
                        unpk2(ga, g0, g1);
                        unpk2(gb, g2, g3);
                    };
                    over();
                    const float most = max3(max3(d0, d1, d2), max3(d3, g0, g1), fmaxf(g2, g3));
                    if (__any_sync(0xffffffffu, most > kRefTop)) {
                        float x0, x1, x2, x3;
                        unpk2(xa, x0, x1);
                        unpk2(xb, x2, x3);
                        auto rows_max = [](float &a, float &b) {  // over the warp's keys
#pragma unroll
                            for (int s = 4; s < 32; s <<= 1) {
                                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
                                b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, s));
                            }
                        };
                        // to the tile's largest score and, beside it (large scores would round the
                        // exponents away), score + scale; the factors of what was summed so far
                        float a0 = fmaxf(x0, x2), a1 = fmaxf(x1, x3);
                        rows_max(a0, a1);
                        a0 = fmaxf(m0, a0 - kRefLift);
                        a1 = fmaxf(m1, a1 - kRefLift);
                        float b0 = fmaxf(x0 - a0 + fva, x2 - a0 + fvb), b1 = fmaxf(x1 - a1 + fva, x3 - a1 + fvb);
                        rows_max(b0, b1);
                        auto move = [](float &m, float &r, float n, float both, float &fo) -> float {
                            const float down = m - n, rn = fmaxf(ceilf(both) - kRefLift, ceilf(down + r));
                            fo = ex2(down + (r - rn));
                            m = n;
                            r = rn;
                            return ex2(down);
                        };
                        float h0, h1;
                        l0 *= move(m0, r0, a0, b0, h0);
                        l1 *= move(m1, r1, a1, b1, h1);
#pragma unroll
                        for (int u = 0; u < D / 16; ++u) {
                            o[u][0] *= h0;
                            o[u][1] *= h1;
                            o[u][2] *= h0;
                            o[u][3] *= h1;
                        }
                        over();
                    }
                    l0 += ex2(d0) + ex2(d2);
                    l1 += ex2(d1) + ex2(d3);
                    const float w0 = ex2(g0), w1 = ex2(g1), w2 = ex2(g2), w3 = ex2(g3);
                    // W^T fragments: (keys 2t4.., query gq) from (key gq.., queries 2t4..), hi and lo
                    const uint32_t h01 = pack_f16x2(w0, w1), h23 = pack_f16x2(w2, w3);
                    const float2 f01 = f16x2_to_f32(h01), f23 = f16x2_to_f32(h23);
                    const uint32_t bh0 = movmatrix_t(h01), bh1 = movmatrix_t(h23);
                    const uint32_t bl0 = movmatrix_t(pack_f16x2(w0 - f01.x, w1 - f01.y));
                    const uint32_t bl1 = movmatrix_t(pack_f16x2(w2 - f23.x, w3 - f23.y));
                    // ---- O^T += V^T W^T: a tile's 16 keys apart, added with rounding (the MMA
                    // truncates its sums: with all keys in one accumulator the 16-stream step at
                    // D 128 is off by 9.4e-7 of its norm instead of 3.4e-7; it took 30.3 us, 31.4 now)
                    auto add = [&](int u, const uint32_t (&a)[4]) {
                        float t[4];
                        mma_f16_new(t, a[0], a[1], a[2], a[3], bl0, bl1);
                        mma_f16(t, a[0], a[1], a[2], a[3], bh0, bh1);
                        unpk2(add2(pk2(o[u][0], o[u][1]), pk2(t[0], t[1])), o[u][0], o[u][1]);
                        unpk2(add2(pk2(o[u][2], o[u][3]), pk2(t[2], t[3])), o[u][2], o[u][3]);
                    };
#pragma unroll
                    for (int u = 0; u < D / 16; u += 2) {
                        uint32_t w[4], a[4];
                        ldsm_x4_t(sV + q8_chunk<D>(lr, u + lc), w[0], w[1], w[2], w[3]);
                        q8_to_f16_pairs<TYPE>(w[0], a[0], a[1]);
                        q8_to_f16_pairs<TYPE>(w[1], a[2], a[3]);
                        add(u, a);
                        q8_to_f16_pairs<TYPE>(w[2], a[0], a[1]);
                        q8_to_f16_pairs<TYPE>(w[3], a[2], a[3]);
                        add(u + 1, a);
                    }
                }
                __syncwarp();
                if (wrote) fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&empty_bar[st]));
                ++tc;
                j0 += rows;
            }
            if (named_bar_red_or(1, C::NC * 32, aborted)) {  // every consumer warp leaves together
                if (tid == 0) {
                    atomicOr(p.status, TF_DEV_TIMEOUT);
                    s_abort = 1;
                }
                break;
            }

            // ---- combine the four warps (tree through shared memory) and write
            tb0 |= (n0 == -INFINITY || vtop == kE8Nan) ? 1u : 0u;
            tb1 |= (n1 == -INFINITY || vtop == kE8Nan) ? 1u : 0u;
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, s);
                l1 += __shfl_xor_sync(0xffffffffu, l1, s);
                e0 = max(e0, __shfl_xor_sync(0xffffffffu, e0, s));
                e1 = max(e1, __shfl_xor_sync(0xffffffffu, e1, s));
                tb0 |= __shfl_xor_sync(0xffffffffu, tb0, s);
                tb1 |= __shfl_xor_sync(0xffffffffu, tb1, s);
            }
            uint32_t f0 = (e0 == 0x7f800000u) | tb0 | badp, f1 = (e1 == 0x7f800000u) | tb1 | badp;
            auto put = [&](int slot) {
                float *dst = comb_o + slot * kWsQ * C::kCombStride;
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {
                    *reinterpret_cast<float2 *>(dst + qa * C::kCombStride + 16 * u + 2 * gq) =
                        make_float2(o[u][0], o[u][2]);
                    *reinterpret_cast<float2 *>(dst + qb_ * C::kCombStride + 16 * u + 2 * gq) =
                        make_float2(o[u][1], o[u][3]);
                }
                if (gq == 0) {
                    comb_m[slot][qa] = m0;
                    comb_m[slot][qb_] = m1;
                    comb_r[slot][qa] = r0;
                    comb_r[slot][qb_] = r1;
                    comb_l[slot][qa] = l0;
                    comb_l[slot][qb_] = l1;
                    comb_f[slot][qa] = f0;
                    comb_f[slot][qb_] = f1;
                }
            };
            auto take = [&](int slot) {
                const float *src = comb_o + slot * kWsQ * C::kCombStride;
                f0 |= comb_f[slot][qa];
                f1 |= comb_f[slot][qb_];
                // this warp's and the slot's sums at the larger references: the joined l, the weights of o
                // (r need not be whole any more)
                auto pair = [](float &m, float &r, float l, float om, float orr, float ol, float &mine,
                               float &theirs) -> float {
                    const float n = fmaxf(m, om), dm = m - n, dt = om - n;
                    const float rm = dm + r, rt = dt + orr, rn = fmaxf(rm, rt);
                    mine = ex2(rm - rn);
                    theirs = ex2(rt - rn);
                    m = n;
                    r = rn;
                    return l * ex2(dm) + ol * ex2(dt);
                };
                float a0, b0, a1, b1;
                l0 = pair(m0, r0, l0, comb_m[slot][qa], comb_r[slot][qa], comb_l[slot][qa], a0, b0);
                l1 = pair(m1, r1, l1, comb_m[slot][qb_], comb_r[slot][qb_], comb_l[slot][qb_], a1, b1);
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {
                    const float2 y = *reinterpret_cast<const float2 *>(src + qa * C::kCombStride + 16 * u + 2 * gq);
                    const float2 z = *reinterpret_cast<const float2 *>(src + qb_ * C::kCombStride + 16 * u + 2 * gq);
                    o[u][0] = o[u][0] * a0 + y.x * b0;
                    o[u][2] = o[u][2] * a0 + y.y * b0;
                    o[u][1] = o[u][1] * a1 + z.x * b1;
                    o[u][3] = o[u][3] * a1 + z.y * b1;
                }
            };
            if (warp >= 2) put(warp - 2);
            named_bar_sync(1, C::NC * 32);
            if (warp < 2) {
                take(warp);
                named_bar_sync(2, 64);  // warp 0 has read slot 0: warp 1 may refill it
                if (warp == 1) put(0);
                named_bar_sync(2, 64);
            }
            if (warp == 0) {
                take(0);
                // o in units of 2^m, as the merge wants it (in two steps: 2^r itself
                // may be past the floats where o is small)
                const float g0 = ex2(0.5f * r0), g1 = ex2(0.5f * r1);
                bool nf0 = !isfinite(l0), nf1 = !isfinite(l1);
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {
                    o[u][0] = o[u][0] * g0 * g0;
                    o[u][1] = o[u][1] * g1 * g1;
                    o[u][2] = o[u][2] * g0 * g0;
                    o[u][3] = o[u][3] * g1 * g1;
                    nf0 |= !isfinite(o[u][0]) || !isfinite(o[u][2]);
                    nf1 |= !isfinite(o[u][1]) || !isfinite(o[u][3]);
                }
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) {
                    nf0 |= __shfl_xor_sync(0xffffffffu, nf0, s);
                    nf1 |= __shfl_xor_sync(0xffffffffu, nf1, s);
                }
                f0 |= nf0;
                f1 |= nf1;
                auto write = [&](int qq, float m, float l, uint32_t f, int c) {
                    if (qq >= q_item) return;
                    const int i = qq / p.group, hl = qq - i * p.group;
                    const int64_t unit = (int64_t)(it.q_row + i) * p.hq + it.g * p.group + hl;
                    if constexpr (DIRECT) {
                        const bool bad = f || !(l > 0.f);
                        const float nan = __int_as_float(0x7fc00000);
#pragma unroll
                        for (int u = 0; u < D / 16; ++u) {
                            const float y = o[u][c] / l, z = o[u][c + 2] / l;
                            const int64_t to = unit * D + 16 * u + 2 * gq;
                            if (p.out_bf16)
                                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + to) =
                                    bad ? 0x7fc07fc0u : pack_bf16x2(y, z);
                            else
                                *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + to) =
                                    bad ? make_float2(nan, nan) : make_float2(y, z);
                        }
                        if (gq == 0) p.out_flags[unit] = (uint8_t)(bad ? 1 : 0);
                    } else {
                        const int64_t at = unit * p.n_splits_max + it.c;
                        float *dst = p.part_o + at * D + 2 * gq;
#pragma unroll
                        for (int u = 0; u < D / 16; ++u)
                            *reinterpret_cast<float2 *>(dst + 16 * u) = make_float2(o[u][c], o[u][c + 2]);
                        if (gq == 0) {
                            p.part_m[at] = m == -FLT_MAX ? -INFINITY : m * kLn2;
                            p.part_l[at] = l;
                            p.part_flag[at] = (uint8_t)(f ? 1 : 0);
                        }
                    }
                };
                write(qa, m0, l0, f0, 0);
                write(qb_, m1, l1, f1, 1);
            }
        }
    }

    // ---- a CTA that gave up leaves only when its copies have landed (each
    // barrier gets a bounded wait for the phase it is in)
    __syncthreads();
    if (DIRECT && s_abort)  // its rows are final, and some of them unwritten
        for (int k = 0, L = ws_snake(0, bid, grid); L < total; L = ws_snake(++k, bid, grid)) {
            const WsItem it = ws_resolve<false>(p, prefix, prefix_full, tail_order, n_full, L);
            flag_rows(it.q_row, it.n_rows, it.g * p.group, p.group, tid, C::kThreads);
        }
    if (s_abort && tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_wait(smem_u32(&full_bar[i]), 0u, 20000000ull);
            mbar_wait(smem_u32(&full_bar[i]), 1u, 20000000ull);
        }
        for (int i = 0; i < C::kNQ; ++i) {
            mbar_wait(smem_u32(&qfull_bar[i]), 0u, 20000000ull);
            mbar_wait(smem_u32(&qfull_bar[i]), 1u, 20000000ull);
        }
    }
}

// CTAs of a full launch on the current device: its SMs times the CTAs an SM
// holds, looked up once a device.
template <int D, int TYPE, bool DIRECT>
int grid_cap() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cap[kMaxDevices];  // 0: not looked up yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    const int known = cap[dev].load(std::memory_order_relaxed);
    if (known > 0) return known;
    int n = 148, per_sm = 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
    if (cudaFuncSetAttribute(decode_q8_kernel<D, TYPE, DIRECT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Q8Cfg<D>::kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, decode_q8_kernel<D, TYPE, DIRECT>, Q8Cfg<D>::kThreads,
                                                      Q8Cfg<D>::kSmem) != cudaSuccess ||
        per_sm < 1)
        per_sm = 1;
    cap[dev].store(n * per_sm, std::memory_order_relaxed);
    return n * per_sm;
}

template <int D, int TYPE, bool DIRECT>
cudaError_t launch_t(const WsParams &p, const void *k, const void *v, int64_t n_items_bound, cudaStream_t st) {
    using C = Q8Cfg<D>;
    CUtensorMap mk, mv;
    const int P = 1 << p.log2_page, BR = P < C::TK ? P : C::TK;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)P, (cuuint64_t)p.hkv, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)P * D, (cuuint64_t)p.hkv * P * D};
    const cuuint32_t box[4] = {(cuuint32_t)C::kRow, (cuuint32_t)BR, 1, 1};
    if (!make_tensor_map_u8(&mk, k, 4, dims, strides, box, C::kRow)) return cudaErrorInvalidValue;
    if (!make_tensor_map_u8(&mv, v, 4, dims, strides, box, C::kRow)) return cudaErrorInvalidValue;
    auto kern = decode_q8_kernel<D, TYPE, DIRECT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    int64_t grid = grid_cap<D, TYPE, DIRECT>();
    if (n_items_bound < grid) grid = n_items_bound < 1 ? 1 : n_items_bound;
    WsParams q = p;
    if (const uint64_t runout = test_wait_runout_ns()) {
        q.test_idle = 1;
        q.wait_ns = runout;
    }
    kern<<<(unsigned)grid, C::kThreads, C::kSmem, st>>>(mk, mv, q);
    return cudaGetLastError();
}

}  // namespace

bool decode_q8_supported(int head_dim, int n_segs) {
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && n_segs >= 1 && n_segs <= Q8Cfg<128>::kPrefixMax;
}

int decode_q8_grid(int head_dim, int kv_type) {
    const bool e = kv_type == TF_KV_E4M3;
    switch (head_dim) {
        case 64: return e ? grid_cap<64, TF_KV_E4M3, false>() : grid_cap<64, TF_KV_INT8, false>();
        case 128: return e ? grid_cap<128, TF_KV_E4M3, false>() : grid_cap<128, TF_KV_INT8, false>();
        default: return e ? grid_cap<256, TF_KV_E4M3, false>() : grid_cap<256, TF_KV_INT8, false>();
    }
}

template <int D, int TYPE>
static cudaError_t launch_d(const WsParams &p, const void *k, const void *v, int64_t n_items_bound, cudaStream_t st) {
    return p.out ? launch_t<D, TYPE, true>(p, k, v, n_items_bound, st)
                 : launch_t<D, TYPE, false>(p, k, v, n_items_bound, st);
}

cudaError_t launch_decode_q8(const WsParams &p, int head_dim, int kv_type, const void *k, const void *v,
                             int64_t n_items_bound, cudaStream_t st) {
    const bool e = kv_type == TF_KV_E4M3;
    switch (head_dim) {
        case 64: return e ? launch_d<64, TF_KV_E4M3>(p, k, v, n_items_bound, st)
                          : launch_d<64, TF_KV_INT8>(p, k, v, n_items_bound, st);
        case 128: return e ? launch_d<128, TF_KV_E4M3>(p, k, v, n_items_bound, st)
                           : launch_d<128, TF_KV_INT8>(p, k, v, n_items_bound, st);
        case 256: return e ? launch_d<256, TF_KV_E4M3>(p, k, v, n_items_bound, st)
                           : launch_d<256, TF_KV_INT8>(p, k, v, n_items_bound, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tfp
