// api_shared.cu - tf_paged_attn_shared: attention of streams that share long
// prefixes (include/tfserve.h).  The rows of a prefix form one segment whose
// keys every row sees, so the prefix's partials come from the FULL partial
// kernels with all of those rows as queries and its keys are read once for
// them; the streams' own keys take the causal ones, and one merge joins both
// sets.  With p, q the two sets' (m, l, o) of a row, M = max(m_p, m_q):
//   out = (2^(m_p - M) o_p + 2^(m_q - M) o_q) / (2^(m_p - M) l_p + 2^(m_q - M) l_q).
//
// The streams' partials go first and the prefixes' beside them, as the
// programmatic dependent: the prefixes' CTAs fill the SMs that the others leave
// (7 streams x 1-5 rows behind prefixes of 500-1,300 keys, D 256: both kernels on
// disjoint SMs, 16.9 us against 28.4 one after the other).  64 one-row streams of
// 16-1,024 keys behind 8,192 (32/8 heads, D 128) take 60 us: some 30 of the decode
// kernel at the HBM rate (134 MB), 26 of the tensor-core kernel, 4 of the merge.
// Those two do not overlap more than at the seam: the decode kernel's two CTAs an
// SM leave no shared memory for the other, and with one CTA an SM beside it the
// decode kernel took 66 us.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>
#include <cuda_runtime.h>

#include "api_common.h"
#include "tf_internal.h"

using namespace tfp;

namespace {

// Whether two entries name one row.  (No exception may leave a C entry: without
// memory for the sort every pair is compared.)
bool rows_overlap(const tf_seg *host, int n) {
    std::unique_ptr<int64_t[]> runs(new (std::nothrow) int64_t[n]);  // first row, row count
    int m = 0;
    for (int a = 0; a < n; ++a) {
        if (host[a].n_rows == 0) continue;
        if (runs) runs[m++] = ((int64_t)host[a].q_row << 32) | host[a].n_rows;
        for (int b = runs ? n : 0; b < a; ++b)
            if (host[a].q_row < host[b].q_row + host[b].n_rows && host[b].q_row < host[a].q_row + host[a].n_rows &&
                host[b].n_rows > 0)
                return true;
    }
    std::sort(runs.get(), runs.get() + m);
    for (int a = 1; a < m; ++a)
        if ((runs[a] >> 32) < (runs[a - 1] >> 32) + (runs[a - 1] & 0x7fffffff)) return true;
    return false;
}

}  // namespace

extern "C" {

size_t tf_paged_attn_shared_workspace_bytes(int32_t n_rows_total, int32_t n_q_heads, int32_t head_dim,
                                            int32_t n_prefix_splits, int32_t n_splits_max) {
    if (n_rows_total < 0 || n_q_heads <= 0 || head_dim <= 0 || n_prefix_splits <= 0 || n_splits_max <= 0) return 0;
    const size_t n = part_bytes(n_rows_total, n_q_heads, head_dim, n_prefix_splits) +
                     part_bytes(n_rows_total, n_q_heads, head_dim, n_splits_max);
    return n < kTooManyBytes ? n : 0;
}

tf_status tf_paged_attn_shared(const void *q, int32_t n_rows_total, int32_t n_q_heads, const void *k_pool,
                               const void *v_pool, int32_t n_pages, int32_t page_size, int32_t n_kv_heads,
                               int32_t head_dim, const int32_t *page_table, int32_t page_table_len,
                               const tf_seg *prefixes, int32_t n_prefixes, const tf_seg *prefixes_host,
                               const tf_seg *segs, int32_t n_segs, const tf_seg *segs_host,
                               const int32_t *page_table_host, float scale, int32_t split_keys,
                               int32_t n_prefix_splits, int32_t n_splits_max, void *workspace, size_t workspace_bytes,
                               void *out, int32_t out_dtype, uint8_t *flags, uint32_t *status, tf_stream_t stream) {
    if (n_rows_total < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_pages < 0 || page_table_len < 0 ||
        n_prefixes < 0 || n_segs < 0 || split_keys < 0 || n_prefix_splits <= 0 || n_splits_max <= 0 ||
        !(scale > 0.f) || !std::isfinite(scale) || (out_dtype != TF_OUT_F32 && out_dtype != TF_OUT_BF16))
        return TF_ERR_ARG;
    const int lp = log2_exact(page_size);
    if (n_q_heads % n_kv_heads != 0 || !head_dim_ok(head_dim) || lp < 3 || lp > 10 ||
        (split_keys > 0 && split_keys < 16) || n_segs > 65535 || n_prefixes > 65535 || n_splits_max > (1 << 24) ||
        n_prefix_splits > (1 << 24))
        return TF_ERR_UNSUPPORTED;
    if (n_segs == 0 || n_rows_total == 0) return TF_OK;
    if (!q || !k_pool || !v_pool || !page_table || (n_prefixes > 0 && !prefixes) || !segs || !workspace || !out ||
        !flags || !status)
        return TF_ERR_ARG;
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned16(workspace))
        return TF_ERR_ALIGN;
    if (workspace_bytes < part_bytes(n_rows_total, n_q_heads, head_dim, n_prefix_splits) +
                              part_bytes(n_rows_total, n_q_heads, head_dim, n_splits_max))
        return TF_ERR_WORKSPACE;
    const int group = n_q_heads / n_kv_heads;
    int max_rows = n_rows_total, own_splits = n_splits_max, own_split = split_keys;
    int pre_rows = n_rows_total, pre_splits = n_prefix_splits, pre_split = split_keys;
    // a table's checks, its split size and the partial slots it needs
    auto plan = [&](const tf_seg *host, int n, bool full, int &rows, int &splits, int &split) -> tf_status {
        if (!keys_taken(host, n)) return TF_ERR_UNSUPPORTED;
        const tf_status rc = check_segs_host(host, n, n_rows_total, page_table_len, page_size, n_pages,
                                             page_table_host, split_keys, splits, &rows, full);
        if (rc != TF_OK || rows == 0) return rc;
        // the tensor-core kernel (prefixes, and more than 8 queries a kv-head) in one wave: 8,192 keys x 256 queries
        // take 26 us in 1,024-key splits (128 CTAs), 30 in 512 and in 1,280; the decode kernel two CTAs an SM
        const int least = least_split(longest_keys(host, n), false);
        if (split == 0)
            split = (int64_t)rows * group > 8
                        ? one_wave_split(host, n, n_kv_heads, std::max(1, 128 / group), device_sms(), least, splits,
                                         kLongestSplit)
                        : decode_split(host, n, n_kv_heads, device_sms() * 2, 1024, least, splits);
        splits = (int)(((int64_t)longest_keys(host, n) + split - 1) / split);
        return TF_OK;
    };
    if (segs_host) {
        const tf_status rc = plan(segs_host, n_segs, false, max_rows, own_splits, own_split);
        if (rc != TF_OK) return rc;
    }
    if (prefixes_host && n_prefixes > 0) {
        const tf_status rc = plan(prefixes_host, n_prefixes, true, pre_rows, pre_splits, pre_split);
        if (rc != TF_OK) return rc;
        // a row belongs to one prefix
        if (n_prefixes > 1 && rows_overlap(prefixes_host, n_prefixes)) return TF_ERR_ARG;
    }
    if (max_rows == 0) return TF_OK;
    // what either partial launch would refuse, before the first one
    const int64_t most_rows = n_prefixes > 0 ? std::max(max_rows, pre_rows) : max_rows;
    if ((most_rows * group + 63) / 64 * n_kv_heads > 65535 || most_rows * n_q_heads > ((int64_t)1 << 31))
        return TF_ERR_UNSUPPORTED;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const PartBuffers pre = part_buffers(ws, n_rows_total, n_q_heads, head_dim, pre_splits);
    const PartBuffers own = part_buffers(ws + part_bytes(n_rows_total, n_q_heads, head_dim, n_prefix_splits),
                                         n_rows_total, n_q_heads, head_dim, own_splits);
    const tf_status rc = paged_partials(false, q, n_rows_total, n_q_heads, k_pool, v_pool, n_pages, page_size,
                                        n_kv_heads, head_dim, page_table, page_table_len, segs, n_segs, segs_host,
                                        page_table_host, scale, own_split, own_splits, own.o, own.m, own.l, own.flag,
                                        status, stream, false, kMaxKeys, true);
    if (rc != TF_OK) return rc;

    if (n_prefixes > 0 && pre_rows > 0) {
        const tf_status rc = paged_partials(true, q, n_rows_total, n_q_heads, k_pool, v_pool, n_pages, page_size,
                                            n_kv_heads, head_dim, page_table, page_table_len, prefixes, n_prefixes,
                                            prefixes_host, page_table_host, scale, pre_split, pre_splits, pre.o,
                                            pre.m, pre.l, pre.flag, status, stream, true, kMaxKeys, true);
        if (rc != TF_OK) return rc;
    }
    MergeSegsParams m{};
    m.own = PartSet{own.o, own.m, own.l, own.flag, own_splits, own_split, max_rows};
    m.prefix = PartSet{pre.o, pre.m, pre.l, pre.flag, pre_splits, pre_split, pre_rows};
    m.segs = segs;
    m.prefixes = prefixes;
    m.n_segs = n_segs;
    m.n_prefixes = n_prefixes;
    m.n_rows_total = n_rows_total;
    m.hq = n_q_heads;
    m.log2_page = lp;
    m.pt_len = page_table_len;
    m.out = out;
    m.out_bf16 = out_dtype == TF_OUT_BF16;
    m.flags = flags;
    m.status = status;
    return cuda_status(launch_merge_segs(m, head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
