// tf_internal.h - parameter blocks and launchers shared between the C-ABI
// entry points (api.cu) and the kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tfpaged.h"

namespace tfp {

// The most keys of a stream (or prefix) in tf_paged_attn_q8 and
// tf_paged_attn_shared: keys and their tiles' ends then stay below 2^31.
constexpr int kMaxKeys = 1 << 30;

// The keys a partial covers where none are given: n_keys in n_splits parts,
// rounded up to whole pages.
__host__ __device__ inline int even_split(int n_keys, int n_splits, int log2_page) {
    const uint32_t per = ((uint32_t)n_keys + (uint32_t)n_splits - 1u) / (uint32_t)n_splits;
    const uint32_t len = (per + (1u << log2_page) - 1u) >> log2_page << log2_page;
    return len > 0x7fffffffu ? 0x7fffffff : (int)len;
}
// Partials of `per` keys that n_keys take (a sum of two ints may pass 2^31, not 2^32).
__host__ __device__ inline int splits_of(int n_keys, int per) {
    return (int)(((uint32_t)n_keys + (uint32_t)per - 1u) / (uint32_t)per);
}
// The end of the partial that starts at key_lo.
__host__ __device__ inline int split_end(int n_keys, int key_lo, int per) {
    return per < n_keys - key_lo ? key_lo + per : n_keys;
}

// Parameters of the split-KV attention kernel (paged or ring source).
struct AttnParams {
    const uint16_t *q;
    int n_rows_total, hq, hkv, group;
    const uint16_t *k, *v;  // pool [pages][Hkv][P][D] or ring [slots][Hkv][D]
    // an 8-bit cache (kv_type TF_KV_*, 0: none): codes [pages][Hkv][P][D], scale bytes [pages][Hkv][P]
    const uint8_t *k_codes, *v_codes, *k_scale, *v_scale;
    int kv_type;
    // paged source
    int n_pages, log2_page, pt_len;
    int max_keys;  // an entry of more is bad
    int max_rows;  // so is one of more rows (0: any number)
    const int32_t *page_table;
    const tf_seg *segs;
    tf_seg seg0;     // used instead of segs[0] when seg_inline != 0 (one-stream prompt calls)
    int seg_inline;
    // ring source
    const tf_ring_seg *rsegs;
    int64_t ring_slots_total;
    float scale_log2;  // scale * log2(e)
    int split_keys, n_splits_max, n_qgroups;
    int full;  // every row sees all of its stream's keys (no causal count)
    // partial outputs [unit][n_splits_max](*D)
    float *part_o, *part_m, *part_l;
    uint8_t *part_flag;
    // direct outputs [row][Hq](*D)
    void *out;
    int out_bf16;
    uint8_t *out_flags;
    uint32_t *status;
};

struct MergeParams {
    const float *part_o, *part_m, *part_l;
    const uint8_t *part_flag;
    int64_t n_units;  // units of partials (rows x heads, or ring entries x heads)
    int n_parts, hq, n_rows_total;
    const tf_ring_seg *rsegs;  // ring merge: unit s * Hq + h writes row rsegs[s].q_row
    int split_slots;           // ring merge: partials of entry s are ceil(n_valid / split_slots)
    int64_t ring_slots_total;
    // tree merge: unit (s * tree_nodes + i) * Hq + h writes row tsegs[s].q_row + i
    const tf_tree_seg *tsegs;
    int tree_nodes;
    int n_parents;
    float *out;
    uint8_t *flags;
};

// Parameters of the tensor-core prompt kernel (one stream's chunk).
struct PromptTcParams {
    const uint16_t *q;                         // bf16 [n_rows_total][hq][D]
    int q_row, n_rows, n_keys, pt_base, n_pg;  // the prompt chunk's segment
    const int32_t *page_table;
    int n_pages, log2_page, hq, hkv, group, n_rows_total;
    float scale_log2;
    // prompt: final rows
    void *out;
    int out_bf16;
    uint8_t *out_flags;
    // split-KV partials: segment table, splits, q-tiles of the grid, outputs
    const tf_seg *segs;
    int pt_len, split_keys, n_splits_max, n_qt;
    int max_keys;  // an entry of more is bad
    int max_rows;  // so is one of more rows (0: any number)
    int full;  // every row sees all of its stream's keys (no causal count)
    // partials that run beside the partial kernel launched before this one: as
    // its programmatic dependent, waiting for that grid only at the end, so that
    // what depends on this launch depends on both
    int beside;
    float *part_o, *part_m, *part_l;
    uint8_t *part_flag;
    uint32_t *status;
    // draft trees over rings: one table entry per tree; partials are laid
    // out by query row like the paged partials
    const tf_tree_seg *tsegs;
    const int32_t *parents;
    int n_parents;
    int64_t ring_slots_total;
    // the timeout test hook (tf_wait_limit_test): the TMA warp issues nothing
    // and every bounded wait gives up after wait_ns (0: the 2 s default)
    int test_idle;
    uint64_t wait_ns;
};

// Parameters of the tensor-core partial kernel over an 8-bit cache.
struct Q8TcParams {
    const uint16_t *q;  // bf16 [n_rows_total][hq][D]
    const uint8_t *k_codes, *v_codes, *k_scale, *v_scale;
    const int32_t *page_table;
    const tf_seg *segs;
    int n_rows_total, hq, hkv, group, n_pages, log2_page, pt_len;
    float scale_log2;
    int split_keys, n_splits, n_qt;  // n_qt: 128-query tiles of the longest stream's rows
    int max_rows;                    // rows of a stream the launch holds
    int full;
    float *part_o, *part_m, *part_l;
    uint8_t *part_flag;
    // one split a stream: the final rows instead of partials
    void *out;
    int out_bf16;
    uint8_t *out_flags;
    uint32_t *status;
    int test_idle;  // the timeout test hook, as in PromptTcParams
    uint64_t wait_ns;
};

// Parameters of the KV append (rows into their pages).
struct AppendParams {
    const uint16_t *k_rows, *v_rows;  // bf16 [n_rows_total][hkv][D]
    uint16_t *k_pool, *v_pool;        // bf16 [n_pages][hkv][P][D]
    int n_rows_total, hkv, n_pages, log2_page, pt_len;
    const int32_t *page_table;
    const tf_seg *segs;
    uint32_t *status;
};

// Parameters of the warp-specialized decode kernel (paged or ring source).
struct WsParams {
    const uint16_t *q;
    int n_rows_total, hq, hkv, group;
    int n_segs;
    // paged
    const tf_seg *segs;
    const int32_t *page_table;
    int n_pages, log2_page, pt_len;
    int max_keys;  // an entry of more is bad
    // ring
    const tf_ring_seg *rsegs;
    int64_t ring_slots_total;
    // an 8-bit cache's scale bytes [pages][Hkv][P]
    const uint8_t *k_scale, *v_scale;
    // an 8-bit cache, one split a stream: the final rows instead of partials
    void *out;
    int out_bf16;
    uint8_t *out_flags;
    int max_rows;  // rows of a stream the launch holds (0: any that fit an item)
    float scale_log2;
    int split_keys, n_splits_max;
    int full;  // every row sees all of its stream's keys (no causal count)
    float *part_o, *part_m, *part_l;
    uint8_t *part_flag;
    uint32_t *status;
    // the timeout test hook (tf_wait_limit_test): the producer issues nothing
    // and every bounded wait gives up after wait_ns (0: the 2 s default)
    int test_idle;
    uint64_t wait_ns;
};

struct ArgmaxParams {
    const uint16_t *logits;
    int n_rows, n_cols;
    int64_t ld;
    int32_t *ids;
    uint8_t *flags;
};

// The timeout test hook: while set (tf_wait_limit_test), the warp-specialized
// and tensor-core kernels launched on this host thread issue no loads and
// give up their bounded waits after this many nanoseconds (0: hook off).
uint64_t test_wait_runout_ns();

// Split-KV partials of tf_paged_attn_decode / tf_paged_attn_block, arguments
// checked (csrc/api.cu).  `beside`: the launch before it on the stream is another
// call of this function, whose outputs it neither reads nor writes; the
// tensor-core kernel then runs beside it (PromptTcParams::beside).  `max_keys`: the
// most keys an entry on the device may have (a host table is the caller's to check).
// `held`: an entry on the device with more rows than the host table's is bad.
tf_status paged_partials(bool full, const void *q, int32_t n_rows_total, int32_t n_q_heads, const void *k_pool,
                         const void *v_pool, int32_t n_pages, int32_t page_size, int32_t n_kv_heads, int32_t head_dim,
                         const int32_t *page_table, int32_t page_table_len, const tf_seg *segs, int32_t n_segs,
                         const tf_seg *segs_host, const int32_t *page_table_host, float scale, int32_t split_keys,
                         int32_t n_splits_max, float *part_o, float *part_m, float *part_l, uint8_t *part_flag,
                         uint32_t *status, tf_stream_t stream, bool beside = false, int max_keys = 0x7fffffff,
                         bool held = false);

// Partials of one kind for the merge of tf_paged_attn_q8 and
// tf_paged_attn_shared: arrays [n_rows_total][hq][n_splits](*D), of which a row
// of an entry with N keys has ceil(N / len), len being the split rule's.  The
// launch that wrote them held max_rows rows of an entry.
struct PartSet {
    const float *o, *m, *l;
    const uint8_t *flag;
    int n_splits, split_keys, max_rows;
};
struct MergeSegsParams {
    PartSet own, prefix;
    const tf_seg *segs, *prefixes;
    int n_segs, n_prefixes;  // n_prefixes = 0: no prefix partials
    int n_rows_total, hq, log2_page, pt_len;
    int full;
    void *out;
    int out_bf16;
    uint8_t *flags;
    uint32_t *status;
};
cudaError_t launch_merge_segs(const MergeSegsParams &p, int head_dim, cudaStream_t st);

cudaError_t launch_attn_partial(const AttnParams &p, int head_dim, bool ring, bool direct, dim3 grid,
                                cudaStream_t st);
enum MergeMode { kMergeRows = 0, kMergeRing = 1, kMergeTree = 2 };
cudaError_t launch_merge(const MergeParams &p, int head_dim, int mode, cudaStream_t st);
cudaError_t launch_argmax(const ArgmaxParams &p, bool vec, bool early, cudaStream_t st);
bool prompt_tc_supported(int head_dim, int group, int page_size);
bool decode_ws_supported(int head_dim, int n_segs);
cudaError_t launch_decode_ws(const WsParams &p, int head_dim, bool ring, const void *k, const void *v,
                             int64_t n_items_bound, cudaStream_t st);
bool decode_q8_supported(int head_dim, int n_segs);
int decode_q8_grid(int head_dim, int kv_type);  // CTAs of a full launch on the current device
cudaError_t launch_decode_q8(const WsParams &p, int head_dim, int kv_type, const void *k, const void *v,
                             int64_t n_items_bound, cudaStream_t st);
bool verify_q8_supported(int head_dim, int group, int split_keys);
cudaError_t launch_verify_q8(const Q8TcParams &p, int head_dim, int kv_type, int n_segs, cudaStream_t st);
cudaError_t launch_kv_append(const AppendParams &p, int head_dim, int n_segs, int max_rows, cudaStream_t st);
cudaError_t launch_prompt_tc(const PromptTcParams &p, int head_dim, const void *k, const void *v, cudaStream_t st);
bool partial_tc_supported(int head_dim, int group, int page_size, int split_keys);
cudaError_t launch_partial_tc(const PromptTcParams &p, int head_dim, const void *k, const void *v, int n_segs,
                              cudaStream_t st);

constexpr int kArgmaxCluster = 2;

// The most nodes a draft tree may have (a node's ancestors are a 64-bit mask).
constexpr int kTreeMaxNodes = 64;

// Splits of a draft tree's keys: the keys [0, n_valid + n_nodes) run from
// slot start = (head - n_valid) mod size; those at or past wrap_at = size -
// start sit at slot key - wrap_at.  Splits never cross the wrap: the first
// run [0, na) and the second [na, N) are cut into split_slots-key pieces.
struct TreeSplits {
    int start, wrap_at, n_keys, na, sa, n_sp;
};
__host__ __device__ inline TreeSplits tree_splits(const tf_tree_seg &e, int split_slots) {
    TreeSplits t;
    t.start = e.head - e.n_valid;
    if (t.start < 0) t.start += e.size;
    t.wrap_at = e.size - t.start;
    t.n_keys = e.n_valid + e.n_nodes;
    t.na = t.n_keys < t.wrap_at ? t.n_keys : t.wrap_at;
    t.sa = (t.na + split_slots - 1) / split_slots;
    t.n_sp = t.sa + (t.n_keys - t.na + split_slots - 1) / split_slots;
    return t;
}
// An entry the tree kernels can read: sizes and ranges only (the parents are
// checked as each node's path is walked).
__host__ __device__ inline bool tree_seg_ok(const tf_tree_seg &e, int n_rows_total, int n_parents,
                                            int64_t ring_slots_total) {
    return e.n_nodes >= 1 && e.n_nodes <= kTreeMaxNodes && e.n_valid >= 0 && e.size > 0 &&
           (int64_t)e.n_valid + e.n_nodes <= e.size && e.head >= 0 && e.head < e.size && e.base >= 0 &&
           e.base + e.size <= ring_slots_total && e.q_row >= 0 && (int64_t)e.q_row + e.n_nodes <= n_rows_total &&
           e.parent_base >= 0 && (int64_t)e.parent_base + e.n_nodes <= n_parents;
}
bool tree_tc_supported(int head_dim, int group);
cudaError_t launch_tree_tc(const PromptTcParams &p, int head_dim, const void *k, const void *v, int n_segs,
                           cudaStream_t st);

}  // namespace tfp
