// verify_q8.cu - split-KV partials over an 8-bit cache for more than 8 queries
// a kv-head (verify rounds, blocks) on the 5th-generation tensor cores: the
// 8-bit counterpart of prompt_tc.cu's partial kernel, whose work split, barriers,
// softmax roles and abort path it follows.
//
// One CTA computes 128 queries (128/G rows x the G q-heads of a kv-head) over a
// split of the keys, 64 at a time.  Eighteen warps:
//  - a load warp brings a tile's codes by bulk copies (a page's slots of a
//    kv-head are contiguous) and its scale bytes (8-byte cp.async) into raw
//    buffers;
//  - eight converter warps turn codes into f16 tiles in the tensor cores' swizzled
//    layout (exact, one conversion instruction per two codes) and the scale bytes
//    into two floats a key: 2^e of K, and e itself of V;
//  - an MMA warp issues S = Q K^T and O += W V (both f16 with fp32 accumulators
//    in tensor memory, Q and W as the tensor-memory operand);
//  - eight softmax warps, two threads a query row, as in prompt_tc.cu.
// The numerics are those of decode_q8.cu: Q's rows scaled by a power of two into
// f16, K's scale multiplying the score, V's joining the weight, whose sum o
// keeps a reference of its own (W = f16 hi + f16 lo: see kRefLift).  So
// the converters never multiply, and an element costs them about one
// instruction: with bf16 tiles that carry the scales it would be four.
//
// Measured: 8 streams of 1-16 rows over 2,048-16,384 keys, 16/2 heads, D 256, int8
// (87 MB) in 52 us, 50 of them this kernel, by stamps in a copy: a CTA starts within
// 3 us of the first, has its first scores after 6.5, the second tile's 2.5 later and
// 17 more tiles at 1.75, then 2 us for the last W V and 3 of epilogue; the middle one
// of the full CTAs is done after 46, the last after 50.  The softmax warps are what a
// tile waits for: of 3,300 cycles with the stamps (3,000 without) they work 3,050, to
// the maxima 1,030, the references 360, the weights 1,360, in tensor memory 300.  The
// tensor pipe is active 29% of the kernel, shared memory's 27%, the issue slots 37%.
// (At D 128 a tile takes 1.6 us, at D 64 1.55: the softmax is the same.)
// Tried when it took 46-51 us: four converter warps took 64 where eight took 51;
// slower or no faster were four converter warps for K and four for V, fetching the
// next codes before converting the last, sixteen softmax warps, registers moved to
// them from the converters, one poll of the MMA warp for all three barriers.
// One split a stream is written as final rows (18 streams of 10-16 rows over 20-121
// keys, 64/8 heads, D 128: 14 us, 25 with partials and a merge; over 900-1,100 keys
// 36 us).
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tf_common.cuh"
#include "tf_internal.h"
#include "tf_q8.cuh"
#include "tf_sm100.cuh"

namespace tfp {
namespace {

constexpr int kSoftmax = 256;                       // threads of the eight softmax warps
constexpr int kMmaWarp = 8, kLoadWarp = 9, kConvWarp = 10, kConvWarps = 8;
constexpr int kVqThreads = (kConvWarp + kConvWarps) * 32;
constexpr int kTmemBar = 6;                         // named barriers: 1 softmax, 2-5 softmax pairs
constexpr int kM = 128, kN = 64;                    // queries a CTA, keys a tile
constexpr int kSlab = kN * 128;                     // 64 keys x 64 columns of f16
constexpr int kStages = 2;                          // f16 K and V tiles
constexpr int kFactors = 4;                         // tiles whose per-key factors are kept
constexpr uint32_t kColS0 = 0, kColS1 = 64, kColQ = 128, kColO = 256;
constexpr int kPids = 1024;                         // page ids held in shared memory

template <int D>
struct VqCfg {
    static constexpr int kSlabs = D / 64;
    static constexpr int kTile = kSlabs * kSlab;    // an f16 tile
    static constexpr int kRaw = kN * D;             // a tile of codes
    static constexpr int kRawStages = D == 256 ? 2 : 4;
    static constexpr int kRawK = kRaw + 128;        // with K's and V's 64 scale bytes
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kStages * kTile;
    static constexpr int kOffRaw = 2 * kStages * kTile;
    static constexpr int kOffRawV = kOffRaw + kRawStages * kRawK;
    static constexpr int kOffFactor = kOffRawV + kRawStages * kRaw;  // float [kFactors][3][kN]
    static constexpr int kOffPid = kOffFactor + kFactors * 3 * kN * 4;
    static constexpr int kSmem = kOffPid + kPids * 4 + 1024;
};

// barrier slots
constexpr int kBarQ = 0;                                 // Q in tensor memory
constexpr int kBarRawK = 1;                              // [4] K's codes and both scale bytes landed
constexpr int kBarRawV = kBarRawK + 4;                   // [4] V's codes landed
constexpr int kBarRawKFree = kBarRawV + 4;               // [4] the converters have read them
constexpr int kBarRawVFree = kBarRawKFree + 4;
constexpr int kBarKFull = kBarRawVFree + 4;              // [kStages] f16 tile written
constexpr int kBarVFull = kBarKFull + kStages;
constexpr int kBarKFree = kBarVFull + kStages;           // [kStages] the MMA that read it is done
constexpr int kBarVFree = kBarKFree + kStages;
constexpr int kBarS = kBarVFree + kStages;               // [2] QK done
constexpr int kBarW = kBarS + 2;                         // [2] weights written
constexpr int kBarO = kBarW + 2;                         // [2] W V done
constexpr int kNumBars = kBarO + 2;

// Instruction descriptor, kind::f16: f16 x f16 -> f32.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ bool vq_wait(uint32_t bar, uint32_t phase, volatile uint32_t *abort_flag, uint64_t lim) {
    if (*abort_flag) return false;
    if (mbar_wait(bar, phase, lim)) return true;
    *abort_flag = 1;
    return false;
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kVqThreads, 1) verify_q8_kernel(const Q8TcParams p) {
    using C = VqCfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[kNumBars];
    __shared__ uint32_t s_tmem, s_err, s_abort;
    __shared__ float s_xmax[2][2][kM];      // [tile parity][column half][row]: the largest score
    __shared__ float s_ymax[2][kM];         // [column half][row]: the largest score + value exponent
    __shared__ float s_xl[2][kM];           // [column half][row]: final partial sums
    __shared__ uint32_t s_x[2][2][kM];      // [exchange][column half][row]: row maxima of Q, findings
    __shared__ uint32_t s_vnan[kFactors][2];  // value rows marked nonfinite, a bit a key
    __shared__ uint32_t s_vmax[kFactors][2];  // the largest scale byte of the others

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t lim = p.wait_ns ? p.wait_ns : 2000000000ull;  // every bounded wait's limit
    // the merge may start: it waits for this grid.  Final rows have none, and what
    // follows on the stream need not wait (a prompt chunk does not): no early start then.
    if (!p.out) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *base_ptr = smem_raw + (sbase - smem_u32(smem_raw));
    auto sK = [&](int s) { return sbase + C::kOffK + s * C::kTile; };
    auto sV = [&](int s) { return sbase + C::kOffV + s * C::kTile; };
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    float *factor = reinterpret_cast<float *>(base_ptr + C::kOffFactor);
    volatile uint32_t *abort_flag = &s_abort;
    bool sent_row = false;

    // ---- the work item: a stream, a kv-head, a split of its keys, a tile of 128/G rows
    const int G = p.group, RT = kM / p.group, g = (int)blockIdx.y;
    const int P = 1 << p.log2_page, BR = P < kN ? P : kN, n_box = kN / BR;
    const int split = (int)blockIdx.x / p.n_qt, qt = p.n_qt - 1 - (int)blockIdx.x % p.n_qt;
    const tf_seg e = p.segs[blockIdx.z];
    const int q_row = e.q_row, T = e.n_rows, N = e.n_keys, pt_base = e.pt_base, n_pg = e.n_pages;
    // final rows of the tile that the launch holds flagged, as the merge would where there is one
    auto flag_rows = [&]() {
        if (q_row < 0) return;
        const int64_t lo = (int64_t)q_row + (int64_t)qt * RT;
        const int64_t hi = min((int64_t)q_row + min((int64_t)min(T, p.max_rows), (int64_t)(qt + 1) * RT),
                               (int64_t)p.n_rows_total);
        for (int64_t x = tid; x < (hi - lo) * G * D; x += kVqThreads) {
            const int64_t r = x / (G * D), c = x - r * (G * D);  // a row's G heads lie together
            const int64_t at = ((lo + r) * p.hq + g * G) * D + c;
            if (p.out_bf16)
                static_cast<uint16_t *>(p.out)[at] = 0x7fc0;
            else
                static_cast<float *>(p.out)[at] = __int_as_float(0x7fc00000);
            if (c % D == 0) p.out_flags[at / D] = 1;
        }
    };
    {
        const bool bad = q_row < 0 || T < 0 || (int64_t)q_row + T > p.n_rows_total ||
                         N < (p.full ? (T > 0 ? 1 : 0) : T) || pt_base < 0 || n_pg < 0 ||
                         (int64_t)pt_base + n_pg > p.pt_len || T > p.max_rows || N > kMaxKeys;
        uint32_t bit = 0;
        if (bad)
            bit = TF_DEV_BAD_SEG;
        else if ((int64_t)N > ((int64_t)n_pg << p.log2_page))
            bit = TF_DEV_PAST_PAGES;
        else if (T > 0 && ((int64_t)N + p.split_keys - 1) / p.split_keys > p.n_splits)
            bit = TF_DEV_SPLITS;
        if (bit) {
            if (tid == 0) atomicOr(p.status, bit);
            if (p.out) flag_rows();
            return;
        }
    }
    const int64_t key_lo64 = (int64_t)split * p.split_keys;
    if (qt * RT >= T || key_lo64 >= N) return;  // the merge knows how many partials a row has
    const int key_lo = (int)key_lo64;
    const int key_hi = (int)min((int64_t)N, key_lo64 + p.split_keys);
    const int row0 = qt * RT, rows_here = min(RT, T - row0);
    const int causal0 = p.full ? N : N - T + 1;  // row i sees keys [0, causal0 + i), with full all N
    const int key_hi_eff = p.full ? key_hi : min(key_hi, causal0 + row0 + rows_here - 1);
    const int full_hi = min(key_hi_eff, causal0 + (p.full ? 0 : row0));  // keys every row of the tile sees
    const int n_tiles = key_hi_eff > key_lo ? (key_hi_eff - key_lo + kN - 1) / kN : 0;
    if (n_tiles == 0) {
        // no row of the tile sees a key of this split
        for (int r = tid; r < rows_here * G; r += kVqThreads) {
            const int64_t at = ((int64_t)(q_row + row0 + r / G) * p.hq + g * G + r % G) * p.n_splits + split;
            p.part_m[at] = -INFINITY;
            p.part_l[at] = 0.f;
            p.part_flag[at] = 0;
        }
        return;
    }

    int *pids = reinterpret_cast<int *>(base_ptr + C::kOffPid);
    const int pg_lo = key_lo >> p.log2_page;
    {
        const int n_pid = min((int)(((int64_t)key_hi_eff + P - 1) >> p.log2_page), n_pg) - pg_lo;
        for (int i = tid; i < n_pid && i < kPids; i += kVqThreads) {
            const int id = p.page_table[pt_base + pg_lo + i];
            pids[i] = (id < 0 || id >= p.n_pages) ? -1 : id;
        }
    }
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t count = 1;
            if (i >= kBarS && i < kBarS + 2) count = 2;
            if (i == kBarQ || (i >= kBarW && i < kBarW + 2)) count = kSoftmax / 32;
            if (i >= kBarRawK && i < kBarRawV) count = 1 + 32;  // expect_tx, every lane's scale bytes
            if (i >= kBarRawKFree && i < kBarKFree) count = kConvWarps;  // raw free, K and V tiles written
            mbar_init(bar(i), count);
        }
        fence_barrier_init();
        s_err = 0;
        s_abort = 0;
    }
    __syncthreads();
    uint32_t tmem = 0;
    auto take_tmem = [&]() {  // the softmax warps and the MMA warp
        if (warp == 0) {
            tmem_alloc(smem_u32(&s_tmem), 512);
            tmem_relinquish();
        }
        tc_fence_before();
        named_bar_sync(kTmemBar, kSoftmax + 32);
        tc_fence_after();
        tmem = s_tmem;
    };
    auto wwait = [&](uint32_t b, uint32_t phase) { return __all_sync(0xffffffffu, vq_wait(b, phase, abort_flag, lim)); };

    if (warp == kLoadWarp) {
        // ================= load warp: codes by bulk copies, one per page (or
        // 64-key span of a larger page); scale bytes, K's and V's, in 8-byte
        // pieces with K's codes.  K goes a tile ahead of V, as it is converted.
        auto page_of = [&](int key) -> int {
            const int idx = key >> p.log2_page;
            if (idx >= n_pg) return -1;
            const int id = idx - pg_lo < kPids ? pids[idx - pg_lo] : p.page_table[pt_base + idx];
            return id < 0 || id >= p.n_pages ? -1 : id;
        };
        auto issue = [&](int t, bool is_v) -> bool {
            const int s = t % C::kRawStages, kt = key_lo + t * kN;
            if (t >= C::kRawStages &&
                !wwait(bar((is_v ? kBarRawVFree : kBarRawKFree) + s), (uint32_t)((t / C::kRawStages - 1) & 1)))
                return false;
            const uint32_t dst = sbase + (is_v ? C::kOffRawV + s * C::kRaw : C::kOffRaw + s * C::kRawK);
            const uint32_t full = bar((is_v ? kBarRawV : kBarRawK) + s);
            if (!is_v) {  // lanes 0-7: K's scale bytes, 8-15: V's
                const int key0 = kt + (lane & 7) * 8;
                const int id = lane < 16 && key0 < key_hi_eff ? page_of(key0) : -1;
                if (id >= 0) {
                    const uint8_t *src = (lane < 8 ? p.k_scale : p.v_scale) +
                                         (((int64_t)id * p.hkv + g) << p.log2_page) + (key0 & (P - 1));
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(
                                     dst + C::kRaw + (lane < 8 ? 0 : kN) + (lane & 7) * 8),
                                 "l"(src)
                                 : "memory");
                }
            }
            const int key0 = kt + lane * BR;  // lane i < n_box: box i
            int id = -1;
            if (lane < n_box && key0 < key_hi_eff) {
                id = page_of(key0);
                if (id < 0) {
                    s_err = 1;
                    atomicOr(p.status, TF_DEV_BAD_PAGE);
                }
            }
            const uint32_t live = __ballot_sync(0xffffffffu, id >= 0);
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)__popc(live) * (uint32_t)(BR * D));
            __syncwarp();
            if (id >= 0) {
                const int64_t src = ((((int64_t)id * p.hkv + g) << p.log2_page) + (key0 & (P - 1))) * D;
                bulk_load(dst + lane * BR * D, (is_v ? p.v_codes : p.k_codes) + src, (uint32_t)(BR * D), full);
            }
            if (!is_v) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(full) : "memory");
            return true;
        };
        // (under the timeout test hook it issues nothing: the other warps' waits run out)
        bool ok = !p.test_idle && issue(0, false);
        for (int t = 0; t < n_tiles && ok; ++t) {
            if (t + 1 < n_tiles) ok = issue(t + 1, false);
            if (ok) ok = issue(t, true);
        }
        cp_async_commit();
        cp_async_wait<0>();  // no scale byte is in flight when this CTA ends
    } else if (warp >= kConvWarp) {
        // ================= converter warps: a 16-byte chunk of a key's codes
        // becomes two 16-byte chunks of f16.  A thread keeps its column and its
        // row modulo 8, so every address is a base and a constant step.  Of eight
        // neighbouring lanes four take 64 codes of one key and four the next 64
        // codes of the key after it: the loads then cover 128 bytes of banks, and
        // the swizzle puts the two keys' stores on even and odd bank groups.
        const int ct = tid - kConvWarp * 32;
        const int c4 = ct & 3, hi = (ct >> 2) & 1, rest = ct >> 3;
        constexpr int kPairs = C::kSlabs > 1 ? C::kSlabs / 2 : 1;  // pairs of slabs
        const int flip = C::kSlabs > 1 ? rest & 1 : 0;
        const int sl = C::kSlabs > 1 ? 2 * ((rest >> 1) % kPairs) + (hi ^ flip) : 0;
        const int r0 = 2 * (C::kSlabs > 1 ? (rest >> 1) / kPairs : rest) + hi;  // first row
        constexpr int kStep = C::kSlabs > 1 ? 4 * kConvWarps / kPairs : 8 * kConvWarps;  // rows from one to the next
        const uint32_t src0 = (uint32_t)(r0 * D + sl * 64 + c4 * 16);
        const uint32_t dst0 = (uint32_t)(sl * kSlab + r0 * 128);
        const uint32_t at0 = dst0 + (((2 * c4) ^ (r0 & 7)) << 4), at1 = dst0 + (((2 * c4 + 1) ^ (r0 & 7)) << 4);
        auto convert = [&](const unsigned char *src, unsigned char *dst, int rows) {
            uint4 w[kN / kStep];
#pragma unroll
            for (int i = 0; i < kN / kStep; ++i) {
                w[i] = *reinterpret_cast<const uint4 *>(src + src0 + i * kStep * D);
            }
            if (rows < kN) {
#pragma unroll
                for (int i = 0; i < kN / kStep; ++i)
                    if (r0 + i * kStep >= rows) w[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kN / kStep; ++i) {
                uint4 h0, h1;
                q8_to_f16<TYPE>(w[i].x, h0.x, h0.y);
                q8_to_f16<TYPE>(w[i].y, h0.z, h0.w);
                q8_to_f16<TYPE>(w[i].z, h1.x, h1.y);
                q8_to_f16<TYPE>(w[i].w, h1.z, h1.w);
                *reinterpret_cast<uint4 *>(dst + at0 + i * kStep * 128) = h0;
                *reinterpret_cast<uint4 *>(dst + at1 + i * kStep * 128) = h1;
            }
        };
        auto convert_k = [&](int t) -> bool {
            const int s = t % C::kRawStages, f = t % kStages;
            if (!wwait(bar(kBarRawK + s), (uint32_t)((t / C::kRawStages) & 1))) return false;
            // the tile is free once QK(t - stages) is done; by then softmax(t - kFactors) is too
            if (t >= kStages && !wwait(bar(kBarKFree + f), (uint32_t)((t / kStages - 1) & 1))) return false;
            const unsigned char *raw = base_ptr + C::kOffRaw + s * C::kRawK;
            const int rows = key_hi_eff - (key_lo + t * kN);  // keys past it: codes 0 (their scores are masked)
            if (ct < kN) {
                const uint32_t ek = raw[C::kRaw + ct], ev = raw[C::kRaw + kN + ct];
                const bool nan = ev == kE8Nan;
                float *fk = factor + (t % kFactors) * 3 * kN;
                fk[ct] = e8m0_f32(ek);
                fk[kN + ct] = nan ? -INFINITY : (float)((int)ev - kE8Bias);
                fk[2 * kN + ct] = nan || ct >= rows ? 0.f : e8m0_f32(ev);
                const uint32_t nans = __ballot_sync(0xffffffffu, nan);
                const uint32_t top = __reduce_max_sync(0xffffffffu, nan || ct >= rows ? 0u : ev);
                if (lane == 0) {
                    s_vnan[t % kFactors][ct >> 5] = nans;
                    s_vmax[t % kFactors][ct >> 5] = top;
                }
            }
            convert(raw, base_ptr + C::kOffK + f * C::kTile, rows);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kBarKFull + f));
                mbar_arrive(bar(kBarRawKFree + s));
            }
            return true;
        };
        auto convert_v = [&](int t) -> bool {
            const int s = t % C::kRawStages, f = t % kStages;
            if (!wwait(bar(kBarRawV + s), (uint32_t)((t / C::kRawStages) & 1))) return false;
            if (t >= kStages && !wwait(bar(kBarVFree + f), (uint32_t)((t / kStages - 1) & 1))) return false;
            convert(base_ptr + C::kOffRawV + s * C::kRaw, base_ptr + C::kOffV + f * C::kTile,
                    key_hi_eff - (key_lo + t * kN));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kBarVFull + f));
                mbar_arrive(bar(kBarRawVFree + s));
            }
            return true;
        };
        // K a tile ahead of V: QK(t + 1) is then ready to run while softmax(t) does
        bool ok = convert_k(0);
        for (int t = 0; t < n_tiles && ok; ++t) {
            if (t + 1 < n_tiles) ok = convert_k(t + 1);
            if (ok) ok = convert_v(t);
        }
    } else if (warp == kMmaWarp) {
        // ================= MMA warp: lane 0 issues every tcgen05.mma
        take_tmem();
        const uint32_t idesc_qk = idesc_f16(kM, kN, false), idesc_wv = idesc_f16(kM, D, true);
        auto issue_qk = [&](int t) {
            if (lane == 0) {
                const int b = t & 1, s = t % kStages;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int sl = k >> 2, kk = k & 3;
                    const uint64_t bd = umma_desc_sw128(sK(s) + sl * kSlab + kk * 32, 16, 1024);
                    umma_ts(tmem + (b ? kColS1 : kColS0), tmem + kColQ + k * 8, bd, idesc_qk, k > 0 ? 1u : 0u);
                }
                umma_commit(bar(kBarS + b));
                umma_commit(bar(kBarKFree + s));
                mbar_arrive(bar(kBarS + b));  // hands on the converters' factors, acquired with the K tile
            }
            __syncwarp();
        };
        auto issue_wv = [&](int j) {
            if (lane == 0) {
                const int b = j & 1, s = j % kStages;
                tc_fence_after();
                const uint32_t sb = tmem + (b ? kColS1 : kColS0);
#pragma unroll
                for (int kk = 0; kk < kN / 16; ++kk) {
                    const uint64_t bd = umma_desc_sw128(sV(s) + kk * 16 * 128, kSlab, 1024);
                    umma_ts(tmem + kColO, sb + kk * 8, bd, idesc_wv, (j > 0 || kk > 0) ? 1u : 0u);
                    umma_ts(tmem + kColO, sb + 32 + kk * 8, bd, idesc_wv, 1u);
                }
                umma_commit(bar(kBarO + b));
                umma_commit(bar(kBarVFree + s));
            }
            __syncwarp();
        };
        auto ready = [&](uint32_t bb, uint32_t phase) { return __all_sync(0xffffffffu, mbar_test_wait(bb, phase)); };
        if (wwait(bar(kBarQ), 0) && wwait(bar(kBarKFull), 0)) issue_qk(0);
        for (int j = 0; j < n_tiles && !*abort_flag; ++j) {
            // QK(j + 1) and W V(j) touch different S buffers: whichever is ready goes first
            const int b = j & 1, s = j % kStages, j1 = j + 1;
            bool need_qk = j1 < n_tiles, need_wv = true;
            const uint64_t t_poll = global_ns();
            while (need_qk || need_wv) {
                bool moved = false;
                if (need_qk && ready(bar(kBarKFull + j1 % kStages), (uint32_t)((j1 / kStages) & 1))) {
                    issue_qk(j1);
                    need_qk = false;
                    moved = true;
                }
                if (need_wv && ready(bar(kBarW + b), (uint32_t)((j >> 1) & 1)) &&
                    ready(bar(kBarVFull + s), (uint32_t)((j / kStages) & 1))) {
                    issue_wv(j);
                    need_wv = false;
                    moved = true;
                }
                if (!moved) {
                    if (__any_sync(0xffffffffu, *abort_flag != 0 || global_ns() - t_poll > lim)) {
                        *abort_flag = 1;
                        break;
                    }
                    __nanosleep(32);
                }
            }
        }
    } else {
        // ================= softmax warps: row qi of the tile, keys 32 h .. 32 h + 31 of each key tile
        const int quad = warp & 3, h = warp >> 2, qi = quad * 32 + lane;
        const int row_i = row0 + qi / G;
        const bool valid_row = row_i < T;
        const int lim_k = valid_row && !p.full ? min(key_hi_eff, causal0 + row_i) : key_hi_eff;
        const uint32_t pair_bar = 2 + quad;
        // m_ref: reference of the scores; m_ref + r_ref: that of score + value exponent (base 2
        // both; r_ref apart, or exponents would round away beside large scores)
        float m_ref = -INFINITY, r_ref = -INFINITY, l_run = 0.f;
        uint32_t emax = 0, tail_bad = 0, lane_base = 0;
        float fq;  // scale * log2(e) over the row's power of two

        // Q into tensor memory as f16, this thread's half of its row; the row's
        // largest magnitude goes to [2^14, 2^15); rows past the stream are zero
        {
            constexpr int kWH = D / 4;  // 32-bit words a half row
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + ((int64_t)(q_row + (valid_row ? row_i : 0)) * p.hq + g * G + qi % G) * D + h * (D / 2));
            uint32_t w[kWH / 16][16];
            uint32_t amax = 0;
#pragma unroll
            for (int v = 0; v < kWH / 4; ++v) {
                const uint4 x = valid_row ? __ldg(src + v) : make_uint4(0u, 0u, 0u, 0u);
                w[v >> 2][4 * (v & 3)] = x.x;
                w[v >> 2][4 * (v & 3) + 1] = x.y;
                w[v >> 2][4 * (v & 3) + 2] = x.z;
                w[v >> 2][4 * (v & 3) + 3] = x.w;
            }
#pragma unroll
            for (int c = 0; c < kWH / 16; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    amax = max(amax, max(w[c][i] & 0x7fffu, (w[c][i] >> 16) & 0x7fffu));
            s_x[0][h][qi] = amax;
            named_bar_sync(pair_bar, 64);
            amax = max(amax, s_x[0][h ^ 1][qi]);
            // (no more than keeps fq normal)
            const int ex = min(min(120, 14 + 127 - (int)(amax >> 7)),
                               126 + (int)(exp_bits(p.scale_log2) >> 23) - 127);
            const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
            fq = p.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
            if (amax >= 0x7f80u) tail_bad = 1;  // a nonfinite query
#pragma unroll
            for (int c = 0; c < kWH / 16; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[c][i] = pack_f16x2(bf16_lo_to_f32(w[c][i]) * up, bf16_hi_to_f32(w[c][i]) * up);
            take_tmem();
            lane_base = tmem + ((uint32_t)(quad * 32) << 16);
#pragma unroll
            for (int c = 0; c < kWH / 16; ++c) tmem_st16(lane_base + kColQ + h * kWH + c * 16, w[c]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarQ));
        }

        for (int j = 0; j < n_tiles; ++j) {
            const int b = j & 1, kt = key_lo + j * kN;
            const uint32_t colS = b ? kColS1 : kColS0;
            const int kh = kt + 32 * h;
            const bool there = vq_wait(bar(kBarS + b), (uint32_t)((j >> 1) & 1), abort_flag, lim);
            tc_fence_after();
            float sv[32];
            {
                uint32_t r[32];
                tmem_ld32(lane_base + colS + 32 * h, r);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) sv[c] = __uint_as_float(r[c]);
            }
            // scores in base 2, rounded (large ones, unrounded, may lie any distance from a reference
            // of their own rounding), and their largest
            const int fs = j % kFactors;
            const float4 *fk = reinterpret_cast<const float4 *>(factor + fs * 3 * kN + 32 * h);
            const float4 *fv = fk + kN / 4, *vs = fk + 2 * (kN / 4);
            const uint32_t vnan = s_vnan[fs][h];
            float mx = -INFINITY;
            const uint64_t fq2 = pk2(fq, fq);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 k4 = fk[q];
                unpk2(mul2(mul2(pk2(sv[4 * q], sv[4 * q + 1]), pk2(k4.x, k4.y)), fq2), sv[4 * q], sv[4 * q + 1]);
                unpk2(mul2(mul2(pk2(sv[4 * q + 2], sv[4 * q + 3]), pk2(k4.z, k4.w)), fq2), sv[4 * q + 2],
                      sv[4 * q + 3]);
            }
            if (kt + kN > full_hi) {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const bool vis = kh + c < lim_k;
                    emax = max(emax, vis ? exp_bits(sv[c]) : 0u);
                    sv[c] = vis ? sv[c] : -INFINITY;
                }
            } else {
                float mn = INFINITY;
#pragma unroll
                for (int c = 0; c < 32; c += 2) mn = min3(mn, sv[c], sv[c + 1]);
                if (mn == -INFINITY) emax = 0x7f800000u;  // (NaN and +inf reach the row sum)
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) mx = max3(mx, sv[c], sv[c + 1]);
            if (vnan) {  // value rows marked nonfinite: flag the rows that see one
#pragma unroll 1
                for (uint32_t v = vnan; v; v &= v - 1)
                    if (kh + __ffs(v) - 1 < lim_k) tail_bad = 1;
            }
            // (NaN where the wait for the scores gave up, for both warps of the pair: no reference
            // moves.  They have to decide alike below, where they meet at a barrier, and s_vmax
            // is the same for both only while the tile's scores are there)
            s_xmax[b][h][qi] = there ? mx : __int_as_float(0x7fc00000);
            named_bar_sync(pair_bar, 64);
            mx = max_nan(there ? mx : __int_as_float(0x7fc00000), s_xmax[b][h ^ 1][qi]);
            // lazy references: they move when a term would pass 2^15 (both halves see
            // the same maxima, so they move together)
            if (mx - m_ref > kRefTop) {
                const float n = mx - kRefLift, down = m_ref - n;
                l_run *= ex2(down);
                r_ref += down;
                m_ref = n;
            }
            const float mu = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t nmu2 = pk2(-mu, -mu);
            float alpha = 1.f;
            // score + value exponent is at most mx + vmax: its own maximum is
            // looked for only when that bound is past the reference
            const float vmax = (float)((int)max(s_vmax[fs][0], s_vmax[fs][1]) - kE8Bias);
            if (__any_sync(0xffffffffu, mx - mu + vmax - r_ref > kRefTop)) {
                float my = -INFINITY;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 v4 = fv[q];
                    float y0, y1, y2, y3;
                    unpk2(add2(add2(pk2(sv[4 * q], sv[4 * q + 1]), nmu2), pk2(v4.x, v4.y)), y0, y1);
                    unpk2(add2(add2(pk2(sv[4 * q + 2], sv[4 * q + 3]), nmu2), pk2(v4.z, v4.w)), y2, y3);
                    my = max3(my, max3(y0, y1, y2), y3);
                }
                s_ymax[h][qi] = my;
                named_bar_sync(pair_bar, 64);
                my = fmaxf(my, s_ymax[h ^ 1][qi]);
                if (my - r_ref > kRefTop) {
                    alpha = ex2(r_ref - (my - kRefLift));
                    r_ref = my - kRefLift;
                }
            }
            const float ru = r_ref == -INFINITY ? 0.f : r_ref;
            {
                uint32_t hi[16], lo[16];
                uint64_t ls2 = 0;  // two zeros
                auto split = [&](int c, float w0, float w1) {
                    hi[c / 2] = pack_f16x2(w0, w1);
                    const float2 f = f16x2_to_f32(hi[c / 2]);
                    lo[c / 2] = pack_f16x2(w0 - f.x, w1 - f.y);
                };
                if (__all_sync(0xffffffffu, vmax - ru <= 90.f)) {
                    // a weight is its probability times 2^(e - ru): a probability
                    // below the floats would give one below 2^-36
                    const float rho = ex2(-ru);
                    const uint64_t rho2 = pk2(rho, rho);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 s4 = vs[q];
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const int c = 4 * q + i;
                            float p0, p1, w0, w1;
                            unpk2(add2(pk2(sv[c], sv[c + 1]), nmu2), p0, p1);
                            const uint64_t p2 = pk2(ex2(p0), ex2(p1));
                            ls2 = add2(ls2, p2);
                            unpk2(mul2(p2, mul2(i ? pk2(s4.z, s4.w) : pk2(s4.x, s4.y), rho2)), w0, w1);
                            split(c, w0, w1);
                        }
                    }
                } else {
                    const uint64_t nru2 = pk2(-ru, -ru);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 v4 = fv[q];
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const int c = 4 * q + i;
                            const uint64_t d2 = add2(pk2(sv[c], sv[c + 1]), nmu2);
                            float p0, p1, w0, w1;
                            unpk2(d2, p0, p1);
                            ls2 = add2(ls2, pk2(ex2(p0), ex2(p1)));
                            unpk2(add2(d2, add2(i ? pk2(v4.z, v4.w) : pk2(v4.x, v4.y), nru2)), w0, w1);
                            split(c, ex2(w0), ex2(w1));
                        }
                    }
                }
                float ls0, ls1;
                unpk2(ls2, ls0, ls1);
                l_run += ls0 + ls1;
                tmem_st16(lane_base + colS + 32 + 16 * h, lo);
                tmem_st16(lane_base + colS + 16 * h, hi);
            }
            // O holds the tiles before this one: rescale it once W V(j - 1) is done
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                vq_wait(bar(kBarO + ((j - 1) & 1)), (uint32_t)(((j - 1) >> 1) & 1), abort_flag, lim);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t r[32];
                    const uint32_t col = kColO + h * (D / 2) + c * 32;
                    tmem_ld32(lane_base + col, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int w = 0; w < 32; ++w) r[w] = __float_as_uint(__uint_as_float(r[w]) * alpha);
                    tmem_st32(lane_base + col, r);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarW + b));
        }

        // ---- epilogue: o in units of 2^m, each half stores its D/2 columns
        vq_wait(bar(kBarO + ((n_tiles - 1) & 1)), (uint32_t)(((n_tiles - 1) >> 1) & 1), abort_flag, lim);
        tc_fence_after();
        const bool aborted = *abort_flag != 0;
        s_xl[h][qi] = l_run;
        s_x[1][h][qi] = (emax == 0x7f800000u ? 1u : 0u) | tail_bad;
        named_bar_sync(pair_bar, 64);
        const float l_sum = s_xl[0][qi] + s_xl[1][qi];
        uint32_t bad = s_x[1][0][qi] | s_x[1][1][qi] | s_err | (aborted ? 1u : 0u) | (isfinite(l_sum) ? 0u : 1u);
        const int64_t at = ((int64_t)(q_row + row_i) * p.hq + g * G + qi % G) * p.n_splits + split;
        // 2^r in two steps: it may itself be past the floats where o is small
        const float gf = r_ref == -INFINITY ? 0.f : ex2(0.5f * r_ref);
        const int d0 = h * (D / 2);
        if (p.out) {
            // ---- one split: normalise, look the row over, write it
            const float il = 1.f / l_sum;
            auto load = [&](int cc, float(&o)[32]) {
                uint32_t r[32];
                tmem_ld32(lane_base + kColO + d0 + cc * 32, r);
                tmem_wait_ld();
#pragma unroll
                for (int w = 0; w < 32; ++w) o[w] = __uint_as_float(r[w]) * gf * gf * il;
            };
            uint32_t obad = 0;
#pragma unroll 1
            for (int cc = 0; cc < D / 64; ++cc) {
                float o[32];
                load(cc, o);
#pragma unroll
                for (int w = 0; w < 32; ++w) obad |= !isfinite(o[w]);
            }
            s_x[0][h][qi] = obad;
            named_bar_sync(pair_bar, 64);
            bad |= s_x[0][0][qi] | s_x[0][1][qi] | (l_sum > 0.f ? 0u : 1u);
#pragma unroll 1
            for (int cc = 0; cc < D / 64; ++cc) {
                float o[32];
                load(cc, o);
                if (!valid_row) continue;
#pragma unroll
                for (int w = 0; w < 32; ++w) o[w] = bad ? __int_as_float(0x7fc00000) : o[w];
                if (!p.out_bf16) {
                    float4 *d4 = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at * D + d0 + cc * 32);
#pragma unroll
                    for (int w = 0; w < 8; ++w) d4[w] = make_float4(o[4 * w], o[4 * w + 1], o[4 * w + 2], o[4 * w + 3]);
                } else {
                    uint4 *d4 = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at * D + d0 + cc * 32);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        d4[w] = bad ? make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u)
                                    : make_uint4(pack_bf16x2(o[8 * w], o[8 * w + 1]),
                                                 pack_bf16x2(o[8 * w + 2], o[8 * w + 3]),
                                                 pack_bf16x2(o[8 * w + 4], o[8 * w + 5]),
                                                 pack_bf16x2(o[8 * w + 6], o[8 * w + 7]));
                }
            }
            if (valid_row && h == 0) p.out_flags[at] = (uint8_t)(bad ? 1 : 0);
        } else {
            const bool staged = rows_here * G >= 64;  // see prompt_tc.cu: many rows leave by bulk copies
            uint32_t *stage = reinterpret_cast<uint32_t *>(base_ptr + C::kOffK) + qi * (D + 4) + d0;
            uint32_t *gout = reinterpret_cast<uint32_t *>(p.part_o + at * D + d0);
            const bool direct = !staged && valid_row && !aborted;
            uint32_t obad = 0;
#pragma unroll 1
            for (int cc = 0; cc < D / 64; ++cc) {
                uint32_t r[32];
                tmem_ld32(lane_base + kColO + d0 + cc * 32, r);
                tmem_wait_ld();
                float o[32];
#pragma unroll
                for (int w = 0; w < 32; ++w) {
                    o[w] = __uint_as_float(r[w]) * gf * gf;
                    obad |= !isfinite(o[w]);
                }
                if ((staged && !aborted) || direct) {
                    float4 *d4 = reinterpret_cast<float4 *>((staged ? stage : gout) + cc * 32);
#pragma unroll
                    for (int w = 0; w < 8; ++w) d4[w] = make_float4(o[4 * w], o[4 * w + 1], o[4 * w + 2], o[4 * w + 3]);
                }
            }
            s_x[0][h][qi] = obad;
            named_bar_sync(pair_bar, 64);
            bad |= s_x[0][0][qi] | s_x[0][1][qi];
            if (staged && valid_row && !aborted) {
                fence_proxy_async_smem();
                bulk_store(gout, smem_u32(stage), (uint32_t)(D / 2) * 4u);
                bulk_commit();
                sent_row = true;
            }
            if (valid_row && h == 0) {
                p.part_m[at] = m_ref == -INFINITY ? -INFINITY : m_ref * kLn2;
                p.part_l[at] = l_sum;
                p.part_flag[at] = (uint8_t)(bad ? 1 : 0);
            }
        }
    }
    // everyone: report a timeout, give in-flight work a bounded chance to land,
    // release tensor memory
    __syncthreads();
    if (s_abort) {
        if (tid == 0) atomicOr(p.status, TF_DEV_TIMEOUT);
        if (tid == 0)
            for (int i = 0; i < kNumBars; ++i) {
                mbar_wait(bar(i), 0u, 20000000ull);
                mbar_wait(bar(i), 1u, 20000000ull);
            }
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (sent_row) bulk_wait_read();
}

template <int D, int TYPE>
cudaError_t launch_t(const Q8TcParams &p, int n_segs, cudaStream_t st) {
    using C = VqCfg<D>;
    auto kern = verify_q8_kernel<D, TYPE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    Q8TcParams q = p;
    if (const uint64_t runout = test_wait_runout_ns()) {
        q.test_idle = 1;
        q.wait_ns = runout;
    }
    const dim3 grid((unsigned)(p.n_qt * p.n_splits), (unsigned)p.hkv, (unsigned)n_segs);
    kern<<<grid, kVqThreads, C::kSmem, st>>>(q);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Q8TcParams &p, int kv_type, int n_segs, cudaStream_t st) {
    return kv_type == TF_KV_E4M3 ? launch_t<D, TF_KV_E4M3>(p, n_segs, st) : launch_t<D, TF_KV_INT8>(p, n_segs, st);
}

}  // namespace

bool verify_q8_supported(int head_dim, int group, int split_keys) {
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && group <= 128 && 128 % group == 0 &&
           split_keys > 0 && split_keys % kN == 0;
}

cudaError_t launch_verify_q8(const Q8TcParams &p, int head_dim, int kv_type, int n_segs, cudaStream_t st) {
    switch (head_dim) {
        case 64: return launch_d<64>(p, kv_type, n_segs, st);
        case 128: return launch_d<128>(p, kv_type, n_segs, st);
        case 256: return launch_d<256>(p, kv_type, n_segs, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tfp
