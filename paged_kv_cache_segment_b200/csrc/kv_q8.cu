// kv_q8.cu - the 8-bit cache written and read: new K/V rows quantised into
// their pages (tf_kv_append_q8) and cached keys read back into bf16 pages
// (tf_kv_read_q8).
//
// Per (row, kv-head) of K and of V, with amax = max |x_d| and Q = 448 or 127:
// k = min{k >= -100 : amax <= Q 2^k}, e = k + 127, code_d = rne(x_d 2^-k); and
// back x_d = code_d 2^(e - 127).  Scaling by a power of two is exact, so is the
// read-back in bf16, and the codes follow from the formula bit for bit.
//
// Both move rows and do next to no arithmetic: per (row, kv-head) of K and of V
// 2 D bytes of bf16 on one side and D + 1 bytes on the other, so HBM bounds
// them (and the launch, for a decode step's few rows).  Measured: 15,000 rows x 4
// kv-heads x D 256 appended (92.3 MB) in 22.1 us, 4.2 TB/s; 12,288 keys of the
// same heads read back (75.6 MB) in 15.9 us, 4.8 TB/s; 16 rows x 8 x 128 in 1.9 us.
// One unit a thread instead of four took 23.5 and 17.1 us; rounding to int8 by a
// conversion instead of the addition 0.6 us more.  A group of D / 8 lanes
// owns a (row, kv-head): every lane moves one 16-byte chunk of bf16 of K and
// one of V and the 8-byte runs of codes they become, so each side is whole
// contiguous runs of D (codes) or 2 D (bf16) bytes and both tensors' loads are
// in flight at once; with enough rows a group takes four.  The row's largest magnitude is an integer maximum of the
// bf16 magnitude patterns over the group (its order is the values' order, and
// the all-ones exponent of a NaN or an infinity tops every finite pattern).
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "api_common.h"
#include "tf_internal.h"
#include "tf_q8.cuh"

namespace tfp {
namespace {

constexpr int kQ8Threads = 256;

struct KvQ8Params {
    const uint16_t *k_rows, *v_rows;  // append: bf16 [n_rows_total][hkv][D]
    uint8_t *k_codes, *v_codes;       // u8 [n_pages][hkv][P][D]
    uint8_t *k_scale, *v_scale;       // u8 [n_pages][hkv][P]
    uint16_t *k_pool, *v_pool;        // read: bf16 [n_pages_dst][hkv][P][D]
    int n_rows_total, max_rows, hkv, n_pages, n_pages_dst, log2_page, pt_len;  // max_rows: that the grid holds
    const int32_t *page_table, *dst_page_table;
    const tf_seg *segs;
    uint32_t *status;
};

// Stream blockIdx.y's entry; false (and the status bit) when it is bad.
__device__ __forceinline__ bool kv_q8_seg(const KvQ8Params &p, bool rows_used, tf_seg &e) {
    e = p.segs[blockIdx.y];
    uint32_t bit = 0;
    if ((rows_used && (e.q_row < 0 || (int64_t)e.q_row + e.n_rows > p.n_rows_total)) || e.n_rows < 0 || e.n_rows > p.max_rows ||
        e.n_keys < e.n_rows || e.pt_base < 0 || e.n_pages < 0 || (int64_t)e.pt_base + e.n_pages > p.pt_len)
        bit = TF_DEV_BAD_SEG;
    else if ((int64_t)e.n_keys > ((int64_t)e.n_pages << p.log2_page))
        bit = TF_DEV_PAST_PAGES;
    if (bit && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, bit);
    return bit == 0;
}

// Unit (row, kv-head) `k` of this group's U: its row and head, or live = false.
struct Unit {
    int i, g;
    bool live;
};
template <int L, int U>
__device__ __forceinline__ Unit unit_of(const KvQ8Params &p, int n_rows, int k) {
    constexpr uint32_t kGroups = kQ8Threads / L;
    const uint32_t u = (blockIdx.x * U + k) * kGroups + threadIdx.x / L, n = (uint32_t)n_rows * (uint32_t)p.hkv;
    Unit x;
    x.live = u < n;
    x.i = x.live ? (int)(u / (uint32_t)p.hkv) : 0;
    x.g = x.live ? (int)(u - (uint32_t)x.i * (uint32_t)p.hkv) : 0;
    return x;
}

template <int D, int TYPE, int U>
__global__ void __launch_bounds__(kQ8Threads) kv_append_q8_kernel(const KvQ8Params p) {
    constexpr int L = D / 8;  // lanes of a group
    tf_seg e;
    if (!kv_q8_seg(p, true, e)) return;
    const int lane = threadIdx.x % L;
    // every unit's rows and page ids first
    uint4 x[U][2];
    int page[U];
    Unit w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        w[k] = unit_of<L, U>(p, e.n_rows, k);
        x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
        page[k] = -1;
        if (w[k].live) {
            const int64_t src = ((int64_t)(e.q_row + w[k].i) * p.hkv + w[k].g) * D + lane * 8;
            x[k][0] = __ldg(reinterpret_cast<const uint4 *>(p.k_rows + src));
            x[k][1] = __ldg(reinterpret_cast<const uint4 *>(p.v_rows + src));
            page[k] = p.page_table[e.pt_base + ((e.n_keys - e.n_rows + w[k].i) >> p.log2_page)];
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const bool ok = w[k].live && page[k] >= 0 && page[k] < p.n_pages;
        if (w[k].live && !ok && lane == 0) atomicOr(p.status, TF_DEV_BAD_PAGE);
        const int j = e.n_keys - e.n_rows + w[k].i;
        const int64_t slot = (((int64_t)page[k] * p.hkv + w[k].g) << p.log2_page) | (j & ((1 << p.log2_page) - 1));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t v[4] = {x[k][t].x, x[k][t].y, x[k][t].z, x[k][t].w};
            uint32_t amax = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) amax = max(amax, max(v[q] & 0x7fffu, (v[q] >> 16) & 0x7fffu));
#pragma unroll
            for (int o = L / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const bool nf = amax >= 0x7f80u;
            const int k2 = q8_exponent<TYPE>(amax);
            const float s = __uint_as_float((uint32_t)(kE8Bias - k2) << 23);  // 2^-k2, exact
            uint2 c;
            c.x = q8_encode4<TYPE>(bf16_lo_to_f32(v[0]), bf16_hi_to_f32(v[0]), bf16_lo_to_f32(v[1]),
                                   bf16_hi_to_f32(v[1]), s);
            c.y = q8_encode4<TYPE>(bf16_lo_to_f32(v[2]), bf16_hi_to_f32(v[2]), bf16_lo_to_f32(v[3]),
                                   bf16_hi_to_f32(v[3]), s);
            if (nf) c = make_uint2(0u, 0u);
            if (ok) {
                reinterpret_cast<uint2 *>((t ? p.v_codes : p.k_codes) + slot * D)[lane] = c;
                if (lane == 0) (t ? p.v_scale : p.k_scale)[slot] = (uint8_t)(nf ? kE8Nan : (uint32_t)(k2 + kE8Bias));
            }
        }
    }
}

template <int D, int TYPE, int U>
__global__ void __launch_bounds__(kQ8Threads) kv_read_q8_kernel(const KvQ8Params p) {
    constexpr int L = D / 8;
    tf_seg e;
    if (!kv_q8_seg(p, false, e)) return;
    const int lane = threadIdx.x % L;
    Unit w[U];
    int page[U], to[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        w[k] = unit_of<L, U>(p, e.n_rows, k);
        page[k] = to[k] = -1;
        if (w[k].live) {
            const int at = e.pt_base + ((e.n_keys - e.n_rows + w[k].i) >> p.log2_page);
            page[k] = p.page_table[at];
            to[k] = p.dst_page_table[at];
        }
    }
    uint2 ck[U], cv[U];
    uint32_t ek[U], ev[U];
    int64_t dst[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const bool bad = page[k] < 0 || page[k] >= p.n_pages || to[k] < 0 || to[k] >= p.n_pages_dst;
        if (w[k].live && bad && lane == 0) atomicOr(p.status, TF_DEV_BAD_PAGE);
        w[k].live = w[k].live && !bad;
        const int in_page = (e.n_keys - e.n_rows + w[k].i) & ((1 << p.log2_page) - 1);
        const int64_t src = (((int64_t)page[k] * p.hkv + w[k].g) << p.log2_page) | in_page;
        dst[k] = (((int64_t)to[k] * p.hkv + w[k].g) << p.log2_page) | in_page;
        if (w[k].live) {
            ck[k] = __ldg(reinterpret_cast<const uint2 *>(p.k_codes + src * D) + lane);
            cv[k] = __ldg(reinterpret_cast<const uint2 *>(p.v_codes + src * D) + lane);
            ek[k] = __ldg(p.k_scale + src);
            ev[k] = __ldg(p.v_scale + src);
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (!w[k].live) continue;
        reinterpret_cast<uint4 *>(p.k_pool + dst[k] * D)[lane] = q8_to_bf16x8<TYPE>(ck[k], e8m0_f32(ek[k]));
        reinterpret_cast<uint4 *>(p.v_pool + dst[k] * D)[lane] = q8_to_bf16x8<TYPE>(cv[k], e8m0_f32(ev[k]));
    }
}

template <int D, int TYPE, int U>
cudaError_t launch_kv_q8_u(const KvQ8Params &p, bool read, int n_segs, int64_t units, cudaStream_t st) {
    constexpr int kGroups = kQ8Threads / (D / 8) * U;
    const dim3 grid((unsigned)((units + kGroups - 1) / kGroups), (unsigned)n_segs);
    if (read)
        kv_read_q8_kernel<D, TYPE, U><<<grid, kQ8Threads, 0, st>>>(p);
    else
        kv_append_q8_kernel<D, TYPE, U><<<grid, kQ8Threads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int D, int TYPE>
cudaError_t launch_kv_q8(const KvQ8Params &p, bool read, int n_segs, int max_rows, cudaStream_t st) {
    const int64_t units = (int64_t)max_rows * p.hkv;
    // several units a thread, their loads in flight together, once that still fills the GPU (15,000 rows: 22.1 us
    // against 23.5 with one; 16 rows: one, so that they spread over the SMs)
    const int64_t wave = (int64_t)device_sms() * (2048 / (D / 8));  // units of one a group on every SM
    if (units * n_segs >= 4 * wave) return launch_kv_q8_u<D, TYPE, 4>(p, read, n_segs, units, st);
    return launch_kv_q8_u<D, TYPE, 1>(p, read, n_segs, units, st);
}

template <int TYPE>
cudaError_t launch_kv_q8_d(const KvQ8Params &p, bool read, int head_dim, int n_segs, int max_rows, cudaStream_t st) {
    switch (head_dim) {
        case 64: return launch_kv_q8<64, TYPE>(p, read, n_segs, max_rows, st);
        case 128: return launch_kv_q8<128, TYPE>(p, read, n_segs, max_rows, st);
        case 256: return launch_kv_q8<256, TYPE>(p, read, n_segs, max_rows, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kv_q8_t(const KvQ8Params &p, bool read, const tf_q8_cache &c, int n_segs, int max_rows,
                           cudaStream_t st) {
    return c.kv_type == TF_KV_E4M3 ? launch_kv_q8_d<TF_KV_E4M3>(p, read, c.head_dim, n_segs, max_rows, st)
                                   : launch_kv_q8_d<TF_KV_INT8>(p, read, c.head_dim, n_segs, max_rows, st);
}

KvQ8Params cache_params(const tf_q8_cache &c) {
    KvQ8Params p{};
    p.k_codes = static_cast<uint8_t *>(c.k_codes);
    p.v_codes = static_cast<uint8_t *>(c.v_codes);
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.hkv = c.n_kv_heads;
    p.n_pages = c.n_pages;
    p.log2_page = log2_exact(c.page_size);
    return p;
}

}  // namespace
}  // namespace tfp

using namespace tfp;

extern "C" {

tf_status tf_kv_append_q8(const void *k_rows, const void *v_rows, int32_t n_rows_total,
                          const tf_q8_cache *cache_host, const int32_t *page_table, int32_t page_table_len,
                          const tf_seg *segs, int32_t n_segs, const tf_seg *segs_host, const int32_t *page_table_host,
                          uint32_t *status, tf_stream_t stream) {
    if (!cache_host || n_rows_total < 0 || page_table_len < 0 || n_segs < 0) return TF_ERR_ARG;
    const tf_q8_cache c = *cache_host;
    tf_status rc = check_q8_shape(c);
    if (rc != TF_OK) return rc;
    if (n_segs > 65535) return TF_ERR_UNSUPPORTED;
    if (n_segs == 0 || n_rows_total == 0) return TF_OK;
    if (!k_rows || !v_rows || !page_table || !segs || !status || !q8_pointers(c)) return TF_ERR_ARG;
    if (!aligned16(k_rows) || !aligned16(v_rows) || !q8_aligned(c)) return TF_ERR_ALIGN;
    int max_rows = n_rows_total;
    if (segs_host) {
        rc = check_segs_host(segs_host, n_segs, n_rows_total, page_table_len, c.page_size, c.n_pages, page_table_host,
                             0, 0, &max_rows);
        if (rc != TF_OK) return rc;
        if (max_rows == 0) return TF_OK;
    }
    if ((int64_t)max_rows * c.n_kv_heads > ((int64_t)1 << 30)) return TF_ERR_UNSUPPORTED;
    KvQ8Params p = cache_params(c);
    p.k_rows = static_cast<const uint16_t *>(k_rows);
    p.v_rows = static_cast<const uint16_t *>(v_rows);
    p.n_rows_total = n_rows_total;
    p.max_rows = max_rows;
    p.pt_len = page_table_len;
    p.page_table = page_table;
    p.segs = segs;
    p.status = status;
    return cuda_status(launch_kv_q8_t(p, false, c, n_segs, max_rows, reinterpret_cast<cudaStream_t>(stream)));
}

tf_status tf_kv_read_q8(const tf_q8_cache *cache_host, const int32_t *page_table, int32_t page_table_len,
                        const tf_seg *segs, int32_t n_segs, const tf_seg *segs_host, const int32_t *page_table_host,
                        void *k_pool, void *v_pool, int32_t n_pages_dst, const int32_t *dst_page_table,
                        const int32_t *dst_page_table_host, uint32_t *status, tf_stream_t stream) {
    if (!cache_host || page_table_len < 0 || n_segs < 0 || n_pages_dst < 0) return TF_ERR_ARG;
    const tf_q8_cache c = *cache_host;
    tf_status rc = check_q8_shape(c);
    if (rc != TF_OK) return rc;
    if (n_segs > 65535) return TF_ERR_UNSUPPORTED;
    if (n_segs == 0) return TF_OK;
    if (!page_table || !dst_page_table || !segs || !status || !k_pool || !v_pool || !q8_pointers(c)) return TF_ERR_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !q8_aligned(c)) return TF_ERR_ALIGN;
    // without a host table a stream may have as many keys as its pages hold
    int64_t max_rows = (int64_t)page_table_len * c.page_size;
    if (segs_host) {
        max_rows = 0;
        for (int s = 0; s < n_segs; ++s) {
            tf_seg e = segs_host[s];
            e.q_row = 0;  // not used by this call
            int rows = 0;
            rc = check_segs_host(&e, 1, INT_MAX, page_table_len, c.page_size, c.n_pages, page_table_host, 0, 0, &rows);
            if (rc == TF_OK && dst_page_table_host)
                rc = check_segs_host(&e, 1, INT_MAX, page_table_len, c.page_size, n_pages_dst, dst_page_table_host, 0,
                                     0, &rows);
            if (rc != TF_OK) return rc;
            if (rows > max_rows) max_rows = rows;
        }
    }
    if (max_rows == 0) return TF_OK;
    if (max_rows * c.n_kv_heads > ((int64_t)1 << 30)) return TF_ERR_UNSUPPORTED;
    KvQ8Params p = cache_params(c);
    p.k_pool = static_cast<uint16_t *>(k_pool);
    p.v_pool = static_cast<uint16_t *>(v_pool);
    p.n_pages_dst = n_pages_dst;
    p.max_rows = (int)max_rows;
    p.pt_len = page_table_len;
    p.page_table = page_table;
    p.dst_page_table = dst_page_table;
    p.segs = segs;
    p.status = status;
    return cuda_status(launch_kv_q8_t(p, true, c, n_segs, (int)max_rows, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
