// api_q8.cu - tf_paged_attn_q8: attention over an 8-bit cache, partials and
// merge in one call (include/tfserve.h).  Argument checks on the host, then
// two stream-ordered launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "api_common.h"
#include "tf_internal.h"

using namespace tfp;

extern "C" {

size_t tf_paged_attn_q8_workspace_bytes(int32_t n_rows_total, int32_t n_q_heads, int32_t head_dim,
                                        int32_t n_splits_max) {
    if (n_rows_total < 0 || n_q_heads <= 0 || head_dim <= 0 || n_splits_max <= 0) return 0;
    const size_t n = part_bytes(n_rows_total, n_q_heads, head_dim, n_splits_max);
    return n < kTooManyBytes ? n : 0;
}

tf_status tf_paged_attn_q8(const void *q, int32_t n_rows_total, int32_t n_q_heads, const tf_q8_cache *cache_host,
                           const int32_t *page_table, int32_t page_table_len, const tf_seg *segs, int32_t n_segs,
                           const tf_seg *segs_host, const int32_t *page_table_host, float scale, int32_t full,
                           int32_t split_keys, int32_t n_splits_max, void *workspace, size_t workspace_bytes,
                           void *out, int32_t out_dtype, uint8_t *flags, uint32_t *status, tf_stream_t stream) {
    if (!cache_host || n_rows_total < 0 || n_q_heads <= 0 || page_table_len < 0 || n_segs < 0 || split_keys < 0 ||
        n_splits_max <= 0 || !(scale > 0.f) || !std::isfinite(scale) || (out_dtype != TF_OUT_F32 && out_dtype != TF_OUT_BF16))
        return TF_ERR_ARG;
    const tf_q8_cache c = *cache_host;
    tf_status rc = check_q8_shape(c);
    if (rc != TF_OK) return rc;
    if (n_q_heads % c.n_kv_heads != 0 || (split_keys > 0 && split_keys < 16)) return TF_ERR_UNSUPPORTED;
    if (n_segs > 65535 || n_splits_max > (1 << 24)) return TF_ERR_UNSUPPORTED;
    if (n_segs == 0 || n_rows_total == 0) return TF_OK;
    if (!q || !page_table || !segs || !workspace || !out || !flags || !status || !q8_pointers(c)) return TF_ERR_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !q8_aligned(c)) return TF_ERR_ALIGN;
    if (workspace_bytes < part_bytes(n_rows_total, n_q_heads, c.head_dim, n_splits_max))
        return TF_ERR_WORKSPACE;
    const int group = n_q_heads / c.n_kv_heads;
    int max_rows = n_rows_total, splits = n_splits_max, split = split_keys;
    bool ws = false;  // decode-shaped: the warp-specialized kernel
    if (segs_host) {
        if (!keys_taken(segs_host, n_segs)) return TF_ERR_UNSUPPORTED;
        rc = check_segs_host(segs_host, n_segs, n_rows_total, page_table_len, c.page_size, c.n_pages, page_table_host,
                             split_keys, n_splits_max, &max_rows, full != 0);
        if (rc != TF_OK) return rc;
        if (max_rows == 0) return TF_OK;
        ws = (int64_t)max_rows * group <= 8 && decode_q8_supported(c.head_dim, n_segs) &&
             (split == 0 || split % std::min(c.page_size, 64) == 0);
        // (64 streams of 256-4,096 keys take 70 us in one split each, 60 us in splits of 1,280 keys; 16 of
        // 1,024-8,192 take 31 us in one wave of 1,152, 36.5 in splits of 768)
        const int least = least_split(longest_keys(segs_host, n_segs), true);
        if (split == 0)
            split = ws ? decode_split(segs_host, n_segs, c.n_kv_heads, decode_q8_grid(c.head_dim, c.kv_type), 1280,
                                      least, n_splits_max)
                       : one_wave_split(segs_host, n_segs, c.n_kv_heads, std::max(1, 128 / group), device_sms(), least,
                                        n_splits_max, kLongestSplit);
        // the partial slots (and, in the tensor-core kernel, the CTAs) that the longest stream takes
        splits = (int)(((int64_t)longest_keys(segs_host, n_segs) + split - 1) / split);
    }
    const int64_t n_qgroups = ((int64_t)max_rows * group + 63) / 64;
    if (n_qgroups * c.n_kv_heads > 65535 || (int64_t)max_rows * n_q_heads > ((int64_t)1 << 31))
        return TF_ERR_UNSUPPORTED;
    const PartBuffers b = part_buffers(workspace, n_rows_total, n_q_heads, c.head_dim, splits);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

    const int lp = log2_exact(c.page_size);
    const float scale_log2 = scale * 1.4426950408889634f;
    cudaError_t e = cudaSuccess;
    bool direct = false;  // the kernel writes the final rows
    if (ws) {
        WsParams w{};
        w.q = static_cast<const uint16_t *>(q);
        w.n_rows_total = n_rows_total;
        w.hq = n_q_heads;
        w.hkv = c.n_kv_heads;
        w.group = group;
        w.n_segs = n_segs;
        w.segs = segs;
        w.page_table = page_table;
        w.n_pages = c.n_pages;
        w.log2_page = lp;
        w.pt_len = page_table_len;
        w.k_scale = c.k_scale;
        w.v_scale = c.v_scale;
        w.max_rows = max_rows;
        w.max_keys = kMaxKeys;
        w.scale_log2 = scale_log2;
        w.split_keys = split;
        w.n_splits_max = splits;
        w.full = full ? 1 : 0;
        w.part_o = b.o;
        w.part_m = b.m;
        w.part_l = b.l;
        w.part_flag = b.flag;
        w.status = status;
        if (splits == 1) {  // nothing to merge
            w.out = out;
            w.out_bf16 = out_dtype == TF_OUT_BF16;
            w.out_flags = flags;
            direct = true;
        }
        int64_t items = 0;
        for (int s = 0; s < n_segs; ++s)
            if (segs_host[s].n_rows > 0)
                items += ((int64_t)segs_host[s].n_keys + split - 1) / split * c.n_kv_heads;
        e = launch_decode_q8(w, c.head_dim, c.kv_type, c.k_codes, c.v_codes, items, st);
    } else if (verify_q8_supported(c.head_dim, group, split)) {
        // more queries a kv-head (a verify round, a block): the tensor-core kernel
        Q8TcParams t{};
        t.q = static_cast<const uint16_t *>(q);
        t.k_codes = static_cast<const uint8_t *>(c.k_codes);
        t.v_codes = static_cast<const uint8_t *>(c.v_codes);
        t.k_scale = c.k_scale;
        t.v_scale = c.v_scale;
        t.page_table = page_table;
        t.segs = segs;
        t.n_rows_total = n_rows_total;
        t.hq = n_q_heads;
        t.hkv = c.n_kv_heads;
        t.group = group;
        t.n_pages = c.n_pages;
        t.log2_page = lp;
        t.pt_len = page_table_len;
        t.scale_log2 = scale_log2;
        t.split_keys = split;
        t.n_splits = splits;
        t.n_qt = (max_rows + 128 / group - 1) / (128 / group);
        t.full = full ? 1 : 0;
        t.part_o = b.o;
        t.part_m = b.m;
        t.part_l = b.l;
        t.part_flag = b.flag;
        if (splits == 1) {  // nothing to merge
            t.out = out;
            t.out_bf16 = out_dtype == TF_OUT_BF16;
            t.out_flags = flags;
        }
        t.max_rows = max_rows;
        t.status = status;
        direct = splits == 1;
        if ((int64_t)t.n_qt * splits > 0x7fffffff || c.n_kv_heads > 65535) return TF_ERR_UNSUPPORTED;
        e = launch_verify_q8(t, c.head_dim, c.kv_type, n_segs, st);
    } else {
        AttnParams p{};
        p.q = static_cast<const uint16_t *>(q);
        p.n_rows_total = n_rows_total;
        p.hq = n_q_heads;
        p.hkv = c.n_kv_heads;
        p.group = group;
        p.k_codes = static_cast<const uint8_t *>(c.k_codes);
        p.v_codes = static_cast<const uint8_t *>(c.v_codes);
        p.k_scale = c.k_scale;
        p.v_scale = c.v_scale;
        p.kv_type = c.kv_type;
        p.n_pages = c.n_pages;
        p.log2_page = lp;
        p.pt_len = page_table_len;
        p.max_keys = kMaxKeys;
        p.max_rows = max_rows;
        p.page_table = page_table;
        p.segs = segs;
        p.scale_log2 = scale_log2;
        p.split_keys = split;
        p.n_splits_max = splits;
        p.n_qgroups = (int)n_qgroups;
        p.full = full ? 1 : 0;
        p.part_o = b.o;
        p.part_m = b.m;
        p.part_l = b.l;
        p.part_flag = b.flag;
        p.status = status;
        const dim3 grid((unsigned)splits, (unsigned)(n_qgroups * c.n_kv_heads), (unsigned)n_segs);
        e = launch_attn_partial(p, c.head_dim, false, false, grid, st);
    }
    if (e != cudaSuccess) return TF_ERR_CUDA;
    if (direct) return TF_OK;

    MergeSegsParams m{};
    m.own = PartSet{b.o, b.m, b.l, b.flag, splits, split, max_rows};
    m.segs = segs;
    m.n_segs = n_segs;
    m.n_rows_total = n_rows_total;
    m.hq = n_q_heads;
    m.log2_page = lp;
    m.pt_len = page_table_len;
    m.full = full ? 1 : 0;
    m.out = out;
    m.out_bf16 = out_dtype == TF_OUT_BF16;
    m.flags = flags;
    m.status = status;
    return cuda_status(launch_merge_segs(m, c.head_dim, st));
}

}  // extern "C"
