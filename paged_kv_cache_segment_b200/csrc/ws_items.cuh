// ws_items.cuh - the work items of the persistent decode kernels: (stream or
// ring row, kv-head, split), which of them exist, and the order in which the
// CTAs take them.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "tf_internal.h"

namespace tfp {

constexpr int kWsQ = 8;         // queries per item (the MMA's N)
constexpr int kWsBuckets = 64;  // tail lengths, in tiles (longer tails share the top bucket)

struct WsItem {
    int s, g, c;
    int q_row, n_rows, n_keys;
    int key_lo, key_hi, full_hi, causal0;
    int pt_base, n_pg;             // paged
    int64_t base;                  // ring
    int size, start, wrap_at;      // ring: keys j >= wrap_at sit at slots j - wrap_at
};

// Stream s's entry and the number of its non-empty partials (0 if the entry is
// invalid or has no rows).  `bits` collects TF_DEV_* codes.
template <bool RING>
__device__ __forceinline__ int ws_stream_splits(const WsParams &p, int s, uint32_t &bits) {
    if constexpr (RING) {
        const tf_ring_seg e = p.rsegs[s];
        const bool bad = e.q_row < 0 || e.q_row >= p.n_rows_total || e.size <= 0 || e.n_valid < 1 ||
                         e.n_valid > e.size || e.head < 0 || e.head >= e.size || e.base < 0 ||
                         e.base + e.size > p.ring_slots_total;
        if (bad) {
            bits |= TF_DEV_BAD_SEG;
            return 0;
        }
        const int n = (e.n_valid + p.split_keys - 1) / p.split_keys;
        if (n > p.n_splits_max) {
            bits |= TF_DEV_SPLITS;
            return 0;
        }
        return n;
    } else {
        const tf_seg e = p.segs[s];
        const bool bad = e.q_row < 0 || e.n_rows < 0 || (int64_t)e.q_row + e.n_rows > p.n_rows_total ||
                         e.n_keys < (p.full ? (e.n_rows > 0 ? 1 : 0) : e.n_rows) || e.pt_base < 0 || e.n_pages < 0 ||
                         (int64_t)e.pt_base + e.n_pages > p.pt_len ||
                         e.n_keys > p.max_keys || (p.max_rows > 0 && e.n_rows > p.max_rows);
        if (bad) {
            bits |= TF_DEV_BAD_SEG;
            return 0;
        }
        if ((int64_t)e.n_keys > ((int64_t)e.n_pages << p.log2_page)) {
            bits |= TF_DEV_PAST_PAGES;
            return 0;
        }
        if (e.n_rows == 0 || e.n_rows * p.group > kWsQ) return 0;
        int per = p.split_keys;
        if (per <= 0) per = even_split(e.n_keys, p.n_splits_max, p.log2_page);
        const int n = splits_of(e.n_keys, per);
        if (n > p.n_splits_max) {
            bits |= TF_DEV_SPLITS;
            return 0;
        }
        return n;
    }
}

// Work order.  Items are dealt to the CTAs in a snake (round r goes left to
// right when r is even, right to left when odd) over a balanced order: every
// stream's full-length splits first, then the streams' last (shorter) splits
// by decreasing length.  The heavy items spread evenly and the light ones fill
// the gaps, so the last CTA to finish carries about the average load.
__device__ __forceinline__ int ws_snake(int k, int bid, int grid) {
    return k * grid + ((k & 1) ? grid - 1 - bid : bid);
}

// Keys of stream s's split length, and the number of TK-key tiles its last
// split takes (0 if the stream has no splits).
template <bool RING>
__device__ __forceinline__ int ws_split_len(const WsParams &p, int s) {
    if constexpr (RING) {
        return p.split_keys;
    } else {
        const int per = p.split_keys;
        return per > 0 ? per : even_split(p.segs[s].n_keys, p.n_splits_max, p.log2_page);
    }
}

template <bool RING>
__device__ __forceinline__ WsItem ws_resolve(const WsParams &p, const int *prefix, const int *prefix_full,
                                             const int *tail_order, int n_full, int idx) {
    int lo, g, c;
    if (idx < n_full) {
        // a full-length split: the stream is the last prefix_full entry <= idx
        lo = 0;
        int hi = p.n_segs;  // prefix_full[lo] <= idx < prefix_full[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix_full[mid] <= idx)
                lo = mid;
            else
                hi = mid;
        }
        const int n_f = (prefix[lo + 1] - prefix[lo]) / p.hkv - 1;  // full splits per kv-head
        const int r = idx - prefix_full[lo];
        g = r / n_f;
        c = r - g * n_f;
    } else {
        // a last split, in the tail order
        const int t = idx - n_full;
        lo = tail_order[t / p.hkv];
        g = t % p.hkv;
        c = (prefix[lo + 1] - prefix[lo]) / p.hkv - 1;
    }
    WsItem it;
    it.s = lo;
    it.g = g;
    it.c = c;
    if constexpr (RING) {
        const tf_ring_seg e = p.rsegs[lo];
        it.q_row = e.q_row;
        it.n_rows = 1;
        it.n_keys = e.n_valid;
        it.base = e.base;
        it.size = e.size;
        it.start = e.head - e.n_valid;
        if (it.start < 0) it.start += e.size;
        it.wrap_at = e.size - it.start;  // keys at or past this index wrapped to slot 0
        it.key_lo = it.c * p.split_keys;
        it.key_hi = min(it.n_keys, it.key_lo + p.split_keys);
        it.pt_base = 0;
        it.n_pg = 0;
    } else {
        const tf_seg e = p.segs[lo];
        it.q_row = e.q_row;
        it.n_rows = e.n_rows;
        it.n_keys = e.n_keys;
        it.pt_base = e.pt_base;
        it.n_pg = e.n_pages;
        int per = p.split_keys;
        if (per <= 0) per = even_split(e.n_keys, p.n_splits_max, p.log2_page);
        it.key_lo = it.c * per;
        it.key_hi = split_end(it.n_keys, it.key_lo, per);
        it.base = 0;
        it.size = it.start = 0;
        it.wrap_at = 0x7fffffff;
    }
    // keys every row sees: [0, causal0); row i sees [0, causal0 + i) (with
    // the full flag every row sees all n_keys)
    it.causal0 = p.full ? it.n_keys : it.n_keys - it.n_rows + 1;
    it.full_hi = min(it.key_hi, it.causal0);
    return it;
}

// Next tile [j0, j0 + rows) of an item: TK keys, cut at the ring's wrap point.
template <int TK>
__device__ __forceinline__ int ws_tile_rows(const WsItem &it, int j0) {
    int j1 = min(j0 + TK, it.key_hi);
    if (j0 < it.wrap_at && j1 > it.wrap_at) j1 = it.wrap_at;
    return j1 - j0;
}

// The order of a call's items, built by one warp in shared memory: the prefix
// sums of the streams' items and full-length items, and the streams by
// decreasing length of their last split.  Reports bad entries.
template <bool RING, int TK>
__device__ __forceinline__ void ws_build_order(const WsParams &p, int lane, int *prefix, int *prefix_full,
                                               int *tail_order, int *bucket, int *total, int *n_full) {
    // per stream: its items (splits x Hkv), its full-length ones, and the
    // tile count of its last split, bucketed for the tail order
    uint32_t bits = 0;
    int running = 0, running_full = 0;
    bucket[lane] = 0;
    bucket[lane + 32] = 0;
    __syncwarp();
    for (int b0 = 0; b0 < p.n_segs; b0 += 32) {
        const int s = b0 + lane;
        const int n_sp = s < p.n_segs ? ws_stream_splits<RING>(p, s, bits) : 0;
        const int units = n_sp * p.hkv, full = n_sp > 0 ? (n_sp - 1) * p.hkv : 0;
        if (n_sp > 0) {
            const int n_keys = RING ? p.rsegs[s].n_valid : p.segs[s].n_keys;
            const int tail = n_keys - (n_sp - 1) * ws_split_len<RING>(p, s);
            atomicAdd(&bucket[min(kWsBuckets, (tail + TK - 1) / TK) - 1], 1);
        }
        int incl = units, incl_f = full;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o), vf = __shfl_up_sync(0xffffffffu, incl_f, o);
            if (lane >= o) {
                incl += v;
                incl_f += vf;
            }
        }
        if (s < p.n_segs) {
            prefix[s] = running + incl - units;
            prefix_full[s] = running_full + incl_f - full;
        }
        running += __shfl_sync(0xffffffffu, incl, 31);
        running_full += __shfl_sync(0xffffffffu, incl_f, 31);
    }
    __syncwarp();
    if (lane == 0) {
        prefix[p.n_segs] = running;
        prefix_full[p.n_segs] = running_full;
        *total = running;
        *n_full = running_full;
    }
    {
        // bucket starts in the tail order, longest tails first: lane l
        // holds buckets 63 - 2l and 62 - 2l, and an exclusive scan over
        // the lanes gives each bucket the count of the longer ones
        const int hi = kWsBuckets - 1 - 2 * lane, lo = hi - 1;
        const int n_hi = bucket[hi], n_lo = bucket[lo];
        int incl = n_hi + n_lo;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int before = incl - n_hi - n_lo;
        __syncwarp();
        bucket[hi] = before;
        bucket[lo] = before + n_hi;
    }
    __syncwarp();
    // each stream with splits takes the next place of its bucket, streams
    // in index order within a bucket
    for (int b0 = 0; b0 < p.n_segs; b0 += 32) {
        const int s = b0 + lane;
        int bk = -1;
        if (s < p.n_segs) {
            const int units = prefix[s + 1] - prefix[s];
            if (units > 0) {
                const int n_sp = units / p.hkv;
                const int n_keys = RING ? p.rsegs[s].n_valid : p.segs[s].n_keys;
                const int tail = n_keys - (n_sp - 1) * ws_split_len<RING>(p, s);
                bk = min(kWsBuckets, (tail + TK - 1) / TK) - 1;
            }
        }
        const uint32_t same = __match_any_sync(0xffffffffu, bk);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (bk >= 0) tail_order[bucket[bk] + rank] = s;
        __syncwarp();
        if (bk >= 0 && rank == 0) bucket[bk] += __popc(same);
        __syncwarp();
    }
    bits |= __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0 && bits && blockIdx.x == 0) atomicOr(p.status, bits);
}

}  // namespace tfp
