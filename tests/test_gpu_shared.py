"""Attention over shared prefixes on the GPU, against float64 over the prefix's
and the stream's own keys put end to end."""
import numpy as np
import pytest
import torch

import paged_kv_cache_segment_b200 as tf
from paged_kv_cache_segment_b200 import workloads as wl

import _serving as sv
from _gpu import DEV, dev, status_word

pytestmark = pytest.mark.gpu


def batch(seed, pre, groups, rows, keys, hq, hkv, d, psz):
    """groups[s]: the prefix of stream s (None: no prefix; such streams come last).  The prefixes' pages come first
    in the page table."""
    b = wl.make_paged_batch(seed, rows=[0] * len(pre) + rows, keys=pre + keys, n_q_heads=hq, n_kv_heads=hkv,
                            head_dim=d, page_size=psz, unused="nan", extra_pages=2)
    prefixes, segs = b.segs[: len(pre)].copy(), b.segs[len(pre) :].copy()
    for p in range(len(pre)):
        mine = [s for s, x in enumerate(groups) if x == p]
        prefixes[p, 0] = segs[mine[0], 0] if mine else 0
        prefixes[p, 1] = sum(rows[s] for s in mine)
    return b, prefixes, segs


def reference(b, prefixes, segs, groups):
    rows, hq, d = b.q.shape
    ref, fl, vmax = np.full((rows, hq, d), np.nan), np.ones((rows, hq), np.uint8), 0.0
    kp, vp = sv.bf16(b.k_pool), sv.bf16(b.v_pool)
    q = sv.bf16(b.q)
    for s, (q_row, r, n, base, _) in enumerate(segs):
        k, v = (sv.keys_of(x, b.page_table, base, n) for x in (kp, vp))
        ahead = 0
        if groups[s] is not None:
            _, _, ahead, pbase, _ = prefixes[groups[s]]
            k, v = (np.concatenate([sv.keys_of(x, b.page_table, pbase, ahead), y]) for x, y in ((kp, k), (vp, v)))
        vmax = max(vmax, float(np.nanmax(np.abs(np.where(np.isfinite(v), v, 0)))))
        ref[q_row : q_row + r], fl[q_row : q_row + r] = sv.attend(
            q[q_row : q_row + r], k, v, [ahead + n - r + i + 1 for i in range(r)], b.scale)
    return ref, fl, vmax


def shared(b, prefixes, segs, *, split=0, n_pre=16, n_own=16, host=True, out_dtype=torch.float32, stream=None,
           pages_host=True):
    rows, hq, d = b.q.shape
    out = torch.full((rows, hq, d), 5.0, dtype=out_dtype, device=DEV)
    flags = torch.full((rows, hq), 9, dtype=torch.uint8, device=DEV)
    ws = torch.full((tf.tf_paged_attn_shared_workspace_bytes(rows, hq, d, n_pre, n_own),), 255, dtype=torch.uint8,
                    device=DEV)
    st = status_word()
    prefixes, segs = np.ascontiguousarray(prefixes), np.ascontiguousarray(segs)
    tf.tf_paged_attn_shared(dev(b.q), dev(b.k_pool).view(torch.bfloat16), dev(b.v_pool).view(torch.bfloat16),
                            dev(b.page_table), dev(prefixes.reshape(-1, 5)), dev(segs), scale=b.scale,
                            split_keys=split, n_prefix_splits=n_pre, n_splits_max=n_own, workspace=ws, out=out,
                            flags=flags, status=st, prefixes_host=prefixes if host in (True, "prefixes") else None,
                            segs_host=segs if host in (True, "segs") else None,
                            page_table_host=b.page_table if host is True and pages_host else None, stream=stream)
    return out.float().cpu().numpy(), flags.cpu().numpy(), int(st.item())


CASES = [  # prefix lengths, stream -> prefix, rows, keys, hq, hkv, d, psz
    ([300], [0, 0, 0, 0], [1, 1, 1, 1], [1, 40, 64, 129], 8, 2, 64, 16),
    ([1, 777], [0, 0, 1, 1, 1], [1, 2, 1, 1, 1], [2, 5, 90, 1, 33], 16, 2, 256, 32),
    ([513], [0] * 20 + [None] * 2, [1] * 22, [7 * i + 1 for i in range(22)], 32, 8, 128, 32),
    ([64, 100, 2000], [0, 1, 1, 2, None], [5, 3, 4, 16, 6], [5, 30, 4, 300, 70], 8, 4, 128, 8),
    ([150], [0, 0], [30, 40], [35, 41], 12, 1, 64, 64),  # a group of 12: the general kernel
    ([260], [0], [1], [3], 4, 4, 128, 256),  # one row behind its prefix
    ([], [None, None], [1, 3], [20, 30], 8, 2, 128, 16),  # no prefix at all
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_float64_over_both_key_lists(case):
    pre, groups, rows, keys, hq, hkv, d, psz = CASES[case]
    b, prefixes, segs = batch(100 + case, pre, groups, rows, keys, hq, hkv, d, psz)
    ref, fl, vmax = reference(b, prefixes, segs, groups)
    for split, n_pre, n_own, host, dt in ((0, 16, 16, True, torch.float32), (0, 5, 3, False, torch.bfloat16),
                                          (64, 32, 8, True, torch.bfloat16), (128, 16, 8, False, torch.float32),
                                          (80, 25, 8, True, torch.float32)):
        out, flags, st = shared(b, prefixes, segs, split=split, n_pre=n_pre, n_own=n_own, host=host, out_dtype=dt)
        assert st == 0
        sv.check_attention(out, flags, ref, fl, vmax, dt == torch.bfloat16, f"{split} {host} {dt}")


@pytest.mark.parametrize("host", ["prefixes", "segs"])
@pytest.mark.parametrize("case", [1, 2, 3, 4])
def test_one_host_table_without_the_other(case, host):
    pre, groups, rows, keys, hq, hkv, d, psz = CASES[case]
    b, prefixes, segs = batch(200 + case, pre, groups, rows, keys, hq, hkv, d, psz)
    ref, fl, vmax = reference(b, prefixes, segs, groups)
    out, flags, st = shared(b, prefixes, segs, n_pre=5, n_own=3, host=host)
    assert st == 0
    sv.check_attention(out, flags, ref, fl, vmax, False)


def test_equals_one_paged_call_over_the_joined_pages():
    """A prefix that ends on a page's end: the same pages as one list per stream give the same attention."""
    b, prefixes, segs = batch(7, [256], [0, 0, 0], [2, 1, 1], [50, 17, 130], 16, 4, 128, 32)
    out, flags, st = shared(b, prefixes, segs)
    pt, joined = [], []
    for q_row, r, n, base, np_ in segs:
        ids = np.r_[b.page_table[:8], b.page_table[base : base + np_]]
        joined.append([q_row, r, 256 + n, len(pt), len(ids)])
        pt += list(ids)
    rows, hq, d = b.q.shape
    po, pm = torch.empty((rows, hq, 4, d), device=DEV), torch.empty((rows, hq, 4), device=DEV)
    pl, pf = torch.empty_like(pm), torch.empty((rows, hq, 4), dtype=torch.uint8, device=DEV)
    joined = np.array(joined, np.int32)
    word = status_word()
    tf.tf_paged_attn_decode(dev(b.q), dev(b.k_pool), dev(b.v_pool), dev(np.array(pt, np.int32)), dev(joined),
                            scale=b.scale, split_keys=128, n_splits_max=4, part_o=po, part_m=pm, part_l=pl,
                            part_flag=pf, status=word, segs_host=joined)
    one, fl = torch.empty((rows, hq, d), device=DEV), torch.empty((rows, hq), dtype=torch.uint8, device=DEV)
    tf.tf_attn_merge(po, pm, pl, pf, one, fl)
    assert st == 0 and int(word.item()) == 0 and (flags == 0).all() and (fl.cpu().numpy() == 0).all()
    vmax = np.abs(sv.bf16(np.where(b.v_pool == 0x7FC0, 0, b.v_pool).astype(np.uint16))).max()
    assert np.abs(out - one.cpu().numpy()).max() <= 2 * 2.0**-14 * vmax


def test_nonfinite_prefix_and_own_keys():
    b, prefixes, segs = batch(8, [100, 90], [0, 0, 1, 1], [1, 2, 1, 1], [10, 20, 30, 5], 8, 2, 64, 16)
    groups = [0, 0, 1, 1]
    b.k_pool[b.page_table[prefixes[0, 3] + 2], 1, 3, 7] = 0x7F80  # the first prefix, kv-head 1
    b.v_pool[b.page_table[segs[1, 3] + 1], 0, 3, 0] = 0xFF80  # key 19 of stream 1: only its last row sees it
    b.q[4, 5, 0] = 0x7FC0
    ref, fl, vmax = reference(b, prefixes, segs, groups)
    assert fl.any() and not fl.all()
    for host in (True, False):
        out, flags, st = shared(b, prefixes, segs, host=host)
        assert st == 0
        sv.check_attention(out, flags, ref, fl, vmax, False, str(host))


def test_bad_tables_on_the_device_and_rows_left_alone():
    groups = [0, 0, None]
    b, prefixes, segs = batch(9, [100], groups, [1, 1, 1], [10, 20, 30], 8, 2, 64, 16)
    ref, fl, vmax = reference(b, prefixes, segs, groups)
    bad = prefixes.copy()
    bad[0, 4] = 3  # 100 keys on three pages of 16
    out, flags, st = shared(b, bad, segs, host=False)
    assert st == 2 and np.isnan(out[:2]).all() and (flags[:2] == 1).all()
    sv.check_attention(out[2:], flags[2:], ref[2:], fl[2:], vmax, False)
    idle = segs.copy()
    idle[1, 1] = 0  # a stream of the group with no row this step
    for host in (True, False):
        out, flags, st = shared(b, prefixes, idle, host=host)
        assert st == 0 and (out[1] == 5.0).all() and (flags[1] == 9).all()
        keep = np.r_[0, 2]
        sv.check_attention(out[keep], flags[keep], ref[keep], fl[keep], vmax, False)


@pytest.mark.parametrize("rows", [1, 3])
def test_captured_replayed_and_on_another_stream(rows):
    groups = [0] * 9
    b, prefixes, segs = batch(11, [700], groups, [rows] * 9, [20 + 31 * i for i in range(9)], 32, 8, 128, 32)
    eager = shared(b, prefixes, segs)
    side = torch.cuda.Stream()
    n, hq, d = b.q.shape
    ws = torch.empty(tf.tf_paged_attn_shared_workspace_bytes(n, hq, d, 16, 16), dtype=torch.uint8, device=DEV)
    out, flags = torch.zeros((n, hq, d), device=DEV), torch.zeros((n, hq), dtype=torch.uint8, device=DEV)
    st = status_word()
    args = (dev(b.q), dev(b.k_pool), dev(b.v_pool), dev(b.page_table), dev(prefixes), dev(segs))
    kw = dict(scale=b.scale, n_prefix_splits=16, n_splits_max=16, workspace=ws, out=out, flags=flags, status=st,
              prefixes_host=prefixes, segs_host=segs, page_table_host=b.page_table)
    side.wait_stream(torch.cuda.current_stream())
    tf.tf_paged_attn_shared(*args, **kw, stream=side)
    side.synchronize()
    assert (out.cpu().numpy() == eager[0]).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tf.tf_paged_attn_shared(*args, **kw)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert (out.cpu().numpy() == eager[0]).all() and (flags.cpu().numpy() == eager[1]).all()
    assert int(st.item()) == 0
