// api_common.h - argument checks, split sizes and workspace layouts shared by the
// extern "C" entry points.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tfserve.h"
#include "tf_internal.h"

namespace tfp {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int log2_exact(int x) {
    if (x <= 0 || (x & (x - 1))) return -1;
    int r = 0;
    while ((1 << r) < x) ++r;
    return r;
}

inline bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

inline tf_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TF_OK : TF_ERR_CUDA; }

inline int split_len(int n_keys, int split_keys, int n_splits_max, int page_size) {
    return split_keys > 0 ? split_keys : even_split(n_keys, n_splits_max, log2_exact(page_size));
}

// Checks of a host copy of a segment table; see tf_paged_attn_decode.
inline tf_status check_segs_host(const tf_seg *sh, int n_segs, int n_rows_total, int page_table_len, int page_size,
                          int n_pages, const int32_t *pt_host, int split_keys, int n_splits_max, int *max_rows,
                          bool full = false) {
    int mr = 0;
    for (int s = 0; s < n_segs; ++s) {
        const tf_seg e = sh[s];
        if (e.q_row < 0 || e.n_rows < 0 || (int64_t)e.q_row + e.n_rows > n_rows_total ||
            e.n_keys < (full ? (e.n_rows > 0 ? 1 : 0) : e.n_rows) ||
            e.pt_base < 0 || e.n_pages < 0 || (int64_t)e.pt_base + e.n_pages > page_table_len)
            return TF_ERR_ARG;
        if ((int64_t)e.n_keys > (int64_t)e.n_pages * page_size) return TF_ERR_PAST_PAGES;
        if (e.n_rows > 0 && n_splits_max > 0) {
            const int per = split_len(e.n_keys, split_keys, n_splits_max, page_size);
            if (splits_of(e.n_keys, per) > n_splits_max) return TF_ERR_ARG;
        }
        if (pt_host) {
            const int used = (e.n_keys + page_size - 1) / page_size;
            for (int k = 0; k < used; ++k) {
                const int pid = pt_host[e.pt_base + k];
                if (pid < 0 || pid >= n_pages) return TF_ERR_BAD_PAGE;
            }
        }
        if (e.n_rows > mr) mr = e.n_rows;
    }
    *max_rows = mr;
    return TF_OK;
}

// Whether no entry has more keys than the serving calls take.
inline bool keys_taken(const tf_seg *sh, int n_segs) {
    for (int s = 0; s < n_segs; ++s)
        if (sh[s].n_keys > kMaxKeys) return false;
    return true;
}

// An 8-bit cache's type and sizes, its pointers, their alignment.
inline tf_status check_q8_shape(const tf_q8_cache &c) {
    if (c.n_pages < 0 || c.n_kv_heads <= 0 || (c.kv_type != TF_KV_E4M3 && c.kv_type != TF_KV_INT8)) return TF_ERR_ARG;
    const int lp = log2_exact(c.page_size);
    return head_dim_ok(c.head_dim) && lp >= 3 && lp <= 10 ? TF_OK : TF_ERR_UNSUPPORTED;
}

// Bytes of partials [n_rows_total][n_q_heads][n_splits]: o, m, l, flag, each
// part's start a multiple of 16 bytes from the last.  More than 2^60: that many.
constexpr size_t kTooManyBytes = (size_t)1 << 60;
inline size_t part_bytes(int64_t n_rows_total, int n_q_heads, int head_dim, int n_splits) {
    const double all = (double)n_rows_total * n_q_heads * n_splits * ((double)head_dim * 4 + 9);
    if (all > (double)kTooManyBytes) return kTooManyBytes;
    const size_t parts = (size_t)n_rows_total * n_q_heads * n_splits;
    return (parts * ((size_t)head_dim * 4 + 9) + 255) / 256 * 256;
}
struct PartBuffers {
    float *o, *m, *l;
    uint8_t *flag;
};
inline PartBuffers part_buffers(void *at, int64_t n_rows_total, int n_q_heads, int head_dim, int n_splits) {
    const size_t parts = (size_t)n_rows_total * n_q_heads * n_splits;
    PartBuffers b;
    b.o = static_cast<float *>(at);
    b.m = b.o + parts * head_dim;
    b.l = b.m + parts;
    b.flag = reinterpret_cast<uint8_t *>(b.l + parts);
    return b;
}

inline bool q8_pointers(const tf_q8_cache &c) { return c.k_codes && c.v_codes && c.k_scale && c.v_scale; }
inline bool q8_aligned(const tf_q8_cache &c) {
    return aligned16(c.k_codes) && aligned16(c.v_codes) && aligned16(c.k_scale) && aligned16(c.v_scale);
}

// SMs of the current device.
inline int device_sms() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                  cudaSuccess || n < 1)
        n = 148;
    return n;
}

// The most keys of a stream with rows (at least 1).
inline int longest_keys(const tf_seg *sh, int n_segs) {
    int n = 1;
    for (int s = 0; s < n_segs; ++s)
        if (sh[s].n_rows > 0 && sh[s].n_keys > n) n = sh[s].n_keys;
    return n;
}

// The least split worth a CTA of its own: one 64-key tile, more for a longer stream,
// whose partials the merge has to read; two tiles where that leaves one split and the
// kernel needs no merge (`direct`).  8-bit, 1 stream, us by splits of 64, 128 and 256:
// 8 rows, D 256, 512 keys 14.5, 15.7 and 18.6; 4,096 keys 18.8, 16.9 and 20.2; 8,000
// 20.3 by 128 or 256; 100 keys 14.3, 13.2 direct; one row, D 128, 600 keys 9.0, 9.3
// and 10.8.  (2 one-row streams of 353-2,000 keys behind a
// short prefix, 16/8 heads: 17.7 against 24.2 by 256; 15 streams of 2,000 behind 3 of
// 846 lose 1.4 to a wider merge.)
inline int least_split(int longest, bool direct) {
    if (direct && longest <= 128) return 128;
    return longest <= 2048 ? 64 : longest <= 8192 ? 128 : 256;
}

// The longest split chosen for the tensor-core kernels.  Their unit truncates its sums,
// twice every 16 keys (hi and lo weights), each time by less than a step, 2^-23, of a sum
// that grows evenly: a partial of n keys loses up to n 2^-27 of its sum, 2^-14 here
// (20,000 keys in one split: 1.2e-4 measured over an 8-bit cache, 6e-5 over bf16).
// A chunk of 1,024 rows over 13,312 keys (D 256, 16/2 heads) takes 383 us in two such
// splits, 342 in one; 20 streams of 9,000-10,000 keys (D 64, 8 kv-heads: 160 CTAs) 312
// in two, 360 in one, 80 rows behind 20 bf16 prefixes of as many 227 and 297.
constexpr int kLongestSplit = 8192;

// A split size for kernels of one CTA an SM with a fixed cost a CTA (start-up
// and epilogue, some eight 64-key tiles' worth): the smallest whole number of
// tiles that leaves one wave of CTAs (streams x kv-heads x query tiles x splits)
// on the SMs, since a second wave pays the fixed cost again; one split a stream
// where even that is more.  No split is longer than `most` keys, as far as n_splits_max allows.
inline int one_wave_split(const tf_seg *sh, int n_segs, int n_kv_heads, int rows_per_tile, int n_sms, int least,
                          int n_splits_max, int64_t most = kMaxKeys) {
    const int64_t longest = longest_keys(sh, n_segs);
    auto ctas = [&](int64_t tiles) {
        int64_t n = 0;
        for (int s = 0; s < n_segs; ++s)
            if (sh[s].n_rows > 0)
                n += ((int64_t)sh[s].n_keys + tiles * 64 - 1) / (tiles * 64) *
                     (((int64_t)sh[s].n_rows + rows_per_tile - 1) / rows_per_tile) * n_kv_heads;
        return n;
    };
    const int64_t fit = (longest + n_splits_max - 1) / n_splits_max;
    int64_t lo = (least > fit ? least : fit) + 63, hi = (longest + 63) / 64;
    lo /= 64;
    if (hi < lo) hi = lo;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (ctas(mid) <= n_sms)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo * 64 > most) {  // even splits of up to `most`
        const int64_t n = (longest + most - 1) / most, len = (longest + n - 1) / n;
        lo = ((len > fit ? len : fit) + 63) / 64;
    }
    return lo > (0x40000000 >> 6) ? 0x40000000 : (int)(lo * 64);
}

// A split size for the persistent decode kernels (`slots` CTAs taking items one
// after another): one wave of items when that is balanced, that is when its
// longest item is near the slots' average load; otherwise half of that load, up
// to `most` keys, since the items of a CTA follow one another without a new start.
inline int decode_split(const tf_seg *sh, int n_segs, int n_kv_heads, int64_t slots, int most, int least,
                        int n_splits_max) {
    const int one = one_wave_split(sh, n_segs, n_kv_heads, 1 << 30, (int)slots, least, n_splits_max);
    int64_t tiles = 0;
    for (int s = 0; s < n_segs; ++s)
        if (sh[s].n_rows > 0) tiles += ((int64_t)sh[s].n_keys + 63) / 64 * n_kv_heads;
    const int64_t load = tiles / slots;  // tiles a CTA
    if (one / 64 <= load + load / 3 + 2) return one;
    const int64_t fit = ((int64_t)longest_keys(sh, n_segs) + n_splits_max - 1) / n_splits_max;
    int64_t len = load / 2 * 64;
    if (len > most) len = most;
    if (len < 256) len = 256;
    if (len < fit) len = (fit + 63) / 64 * 64;
    return (int)len;
}

}  // namespace tfp
