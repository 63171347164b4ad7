"""Edges of the serving calls on the GPU: waits that run out, more streams than
the decode kernels take, caches and logits past 32-bit offsets, calls on two
streams at once, workspaces of the smallest size."""
import numpy as np
import pytest
import torch

import paged_kv_cache_segment_b200 as tf
from paged_kv_cache_segment_b200 import binding
from paged_kv_cache_segment_b200 import workloads as wl

import _serving as sv
from _gpu import DEV, dev, status_word
from test_gpu_q8 import attn, cache_of, q8_batch, reference
from test_gpu_shared import batch, shared
from test_gpu_shared import reference as shared_reference

pytestmark = pytest.mark.gpu


def with_hook(fn):
    tf.tf_wait_limit_test(True)
    try:
        return fn()
    finally:
        tf.tf_wait_limit_test(False)


@pytest.mark.parametrize("rows,keys,hq,hkv,d", [([1, 1], [700, 1500], 32, 8, 128),  # decode, partials and merge
                                                ([1, 1, 1], [60, 100, 7], 8, 2, 64),  # decode, one split: no merge
                                                ([5, 14], [900, 2100], 16, 2, 256),  # the tensor-core kernel
                                                ([5, 20], [90, 130], 16, 2, 128)])  # the same, one split
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_q8_wait_runs_out_flags_every_row_then_recovers(rows, keys, hq, hkv, d, dt):
    b, sides, c = q8_batch("e4m3", 3, rows=rows, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32)
    out, flags, st = with_hook(lambda: attn(c, b, "e4m3", out_dtype=dt))
    assert st & binding.TF_DEV_TIMEOUT
    assert (flags == 1).all() and np.isnan(out).all()
    out, flags, st = attn(c, b, "e4m3", out_dtype=dt)
    assert st == 0
    ref, fl, vmax = reference(b, sides, "e4m3")
    sv.check_attention(out, flags, ref, fl, vmax, dt == torch.bfloat16)


@pytest.mark.parametrize("rows,hq,hkv,d", [(1, 32, 8, 128), (4, 16, 2, 256)])
def test_shared_wait_runs_out_flags_every_row_then_recovers(rows, hq, hkv, d):
    groups = [0, 0, 0]
    b, prefixes, segs = batch(4, [500], groups, [rows] * 3, [20, 130, 300], hq, hkv, d, 32)
    out, flags, st = with_hook(lambda: shared(b, prefixes, segs))
    assert st & binding.TF_DEV_TIMEOUT
    assert (flags == 1).all() and np.isnan(out).all()
    out, flags, st = shared(b, prefixes, segs)
    assert st == 0
    ref, fl, vmax = shared_reference(b, prefixes, segs, groups)
    sv.check_attention(out, flags, ref, fl, vmax, False)


def test_three_hundred_streams():
    rng = np.random.default_rng(0)
    n = 300  # past the decode kernels' tables
    keys = [int(k) for k in rng.integers(1, 90, n)]
    b, sides, c = q8_batch("int8", 5, rows=[1] * n, keys=keys, n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16)
    ref, fl, vmax = reference(b, sides, "int8")
    out, flags, st = attn(c, b, "int8")
    assert st == 0
    sv.check_attention(out, flags, ref, fl, vmax, False)
    groups = [s % 2 for s in sorted(range(n), key=lambda s: s % 2)]
    b, prefixes, segs = batch(6, [70, 33], groups, [1] * n, keys, 4, 2, 64, 16)
    ref, fl, vmax = shared_reference(b, prefixes, segs, groups)
    out, flags, st = shared(b, prefixes, segs)
    assert st == 0
    sv.check_attention(out, flags, ref, fl, vmax, False)


@pytest.mark.parametrize("rows", [1, 12])
def test_a_cache_past_32_bit_offsets(rows):
    """70,000 pages of 64 x 2 x 256 codes (2.3e9 of them) with a stream in the last pages: written, read back, attended."""
    n_pages, hkv, psz, d, hq, n = 70000, 2, 64, 256, 4, 150
    c = tf.Q8Cache(*(torch.empty((n_pages, hkv, psz, d), dtype=torch.int8, device=DEV) for _ in "kv"),
                   *(torch.empty((n_pages, hkv, psz), dtype=torch.uint8, device=DEV) for _ in "kv"))
    pt = np.array([n_pages - 1, 35000, n_pages - 2], np.int32)
    fill = np.array([[0, n, n, 0, 3]], np.int32)
    segs = np.array([[0, rows, n, 0, 3]], np.int32)
    rng = np.random.default_rng(1)
    kr, vr = wl.normal_bf16(rng, (n, hkv, d)), wl.normal_bf16(rng, (n, hkv, d))
    st = status_word()
    tf.tf_kv_append_q8(dev(kr), dev(vr), c, dev(pt), dev(fill), status=st, segs_host=fill, page_table_host=pt)
    vals = [sv.values(*sv.quantise(x, "int8"), "int8") for x in (kr, vr)]
    small = [torch.zeros((3, hkv, psz, d), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    tf.tf_kv_read_q8(c, dev(pt), dev(fill), small[0], small[1], dev(np.arange(3, dtype=np.int32)), status=st)
    for got, want in zip(small, vals):
        rows_of = got.double().cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:n]
        assert (rows_of == want).all()
    q = wl.normal_bf16(rng, (rows, hq, d))
    out, fl = torch.empty((rows, hq, d), device=DEV), torch.empty((rows, hq), dtype=torch.uint8, device=DEV)
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(rows, hq, d, 4), dtype=torch.uint8, device=DEV)
    for host in (segs, None):
        tf.tf_paged_attn_q8(dev(q), c, dev(pt), dev(segs), scale=1 / 16, n_splits_max=4, workspace=ws, out=out, flags=fl,
                            status=st, segs_host=host)
        ref, rf = sv.attend(sv.bf16(q), vals[0], vals[1], [n - rows + i + 1 for i in range(rows)], 1 / 16)
        sv.check_attention(out.cpu().numpy(), fl.cpu().numpy(), ref, rf, np.abs(vals[1]).max(), False)
    assert int(st.item()) == 0


def test_logits_past_32_bit_offsets():
    rows, cols = 17000, 128000  # 2.2e9 elements; the last row is checked
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[:-1].zero_()
    rng = np.random.default_rng(2)
    x[-1] = torch.from_numpy(rng.normal(0, 3, cols).astype(np.float32)).to(DEV)
    tok = torch.zeros((rows, 1), dtype=torch.int32, device=DEV)
    tok[-1] = 77
    tl, fl, st = torch.empty((rows, 1), device=DEV), torch.empty(rows, dtype=torch.uint8, device=DEV), status_word()
    ids, tops = torch.empty((rows, 3), dtype=torch.int32, device=DEV), torch.empty((rows, 3), device=DEV)
    tf.tf_logprob_rows(x, tok, token_logprobs=tl, top_ids=ids, top_logprobs=tops, flags=fl, status=st)
    want = sv.logprobs(x[-1:].double().cpu().numpy(), 1.0, np.array([[77]]), 3)
    assert (ids[-1].cpu().numpy() == want[3][0]).all() and abs(tl[-1].item() - want[0][0, 0]) < 1e-4
    # a row of equal columns: the first ones, each log(1 / n)
    assert (ids[:-1] == torch.arange(3, device=DEV)).all()
    assert (tl[:-1] + np.log(cols)).abs().max().item() < 1e-4 and int(fl.sum()) == 0


def test_two_streams_at_once_with_their_own_workspaces():
    jobs = []
    for seed, kind in ((7, "e4m3"), (8, "int8")):
        b, sides, c = q8_batch(kind, seed, rows=[1] * 8, keys=[900] * 8, n_q_heads=32, n_kv_heads=8, head_dim=128,
                               page_size=32)
        n, hq, d = b.q.shape
        jobs.append(dict(args=(dev(b.q), c, dev(b.page_table), dev(b.segs)), host=b.segs, scale=b.scale,
                         ws=torch.empty(tf.tf_paged_attn_q8_workspace_bytes(n, hq, d, 8), dtype=torch.uint8, device=DEV),
                         out=torch.zeros((n, hq, d), device=DEV), fl=torch.zeros((n, hq), dtype=torch.uint8, device=DEV),
                         st=status_word(), stream=torch.cuda.Stream(), ref=reference(b, sides, kind)))
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            tf.tf_paged_attn_q8(*j["args"], scale=j["scale"], n_splits_max=8, workspace=j["ws"], out=j["out"],
                                flags=j["fl"], status=j["st"], segs_host=j["host"], stream=j["stream"])
    torch.cuda.synchronize()
    for j in jobs:
        ref, fl, vmax = j["ref"]
        sv.check_attention(j["out"].cpu().numpy(), j["fl"].cpu().numpy(), ref, fl, vmax, False)


@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("rows", [1, 6])
def test_a_captured_step_follows_streams_that_grow(rows, split):
    """A call captured with a host table of the largest lengths serves every shorter table written to the device."""
    b, sides, c = q8_batch("e4m3", 9, rows=[rows] * 2, keys=[900, 300], n_q_heads=8, n_kv_heads=2, head_dim=128,
                           page_size=32)
    n, hq, d = b.q.shape
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(n, hq, d, 8), dtype=torch.uint8, device=DEV)
    out, fl, st = torch.zeros((n, hq, d), device=DEV), torch.zeros((n, hq), dtype=torch.uint8, device=DEV), status_word()
    short = b.segs.copy()
    short[:, 2] = [100, 6]
    sg = dev(short)
    args = (dev(b.q), c, dev(b.page_table), sg)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tf.tf_paged_attn_q8(*args, scale=b.scale, split_keys=split, n_splits_max=8, workspace=ws, out=out, flags=fl,
                            status=st, segs_host=b.segs)
    for keys in ([100, 6], [128, 129], [900, 300]):
        s = b.segs.copy()
        s[:, 2] = keys
        sg.copy_(dev(s))
        g.replay()
        torch.cuda.synchronize()
        ref, rf, vmax = reference(b, sides, "e4m3", segs=s)
        assert int(st.item()) == 0
        sv.check_attention(out.cpu().numpy(), fl.cpu().numpy(), ref, rf, vmax, False, str(keys))


@pytest.mark.parametrize("rows,hq,keys", [([1, 1], 8, [100, 5]), ([1, 1], 8, [1200, 300]), ([20, 3], 16, [100, 30])])
def test_a_replay_past_its_partials_is_flagged(rows, hq, keys):
    """A chosen split holds the streams it was captured with: one that outgrows its partials is reported and flagged,
    with one split (no merge) and with several."""
    b, sides, c = q8_batch("e4m3", 10, rows=rows, keys=[3000, 300], n_q_heads=hq, n_kv_heads=2, head_dim=128,
                           page_size=32)
    n, _, d = b.q.shape
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(n, hq, d, 64), dtype=torch.uint8, device=DEV)
    out, fl, st = torch.zeros((n, hq, d), device=DEV), torch.zeros((n, hq), dtype=torch.uint8, device=DEV), status_word()
    s = b.segs.copy()
    s[:, 2] = keys
    sg = dev(s)
    args = (dev(b.q), c, dev(b.page_table), sg)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tf.tf_paged_attn_q8(*args, scale=b.scale, n_splits_max=64, workspace=ws, out=out, flags=fl, status=st, segs_host=s)
    s[0, 2] = 3000
    sg.copy_(dev(s))
    g.replay()
    torch.cuda.synchronize()
    ref, rf, vmax = reference(b, sides, "e4m3", segs=s)
    assert int(st.item()) == binding.TF_DEV_SPLITS
    r = rows[0]
    assert torch.isnan(out[:r]).all() and (fl[:r] == 1).all()
    sv.check_attention(out[r:].cpu().numpy(), fl[r:].cpu().numpy(), ref[r:], rf[r:], vmax, False)


@pytest.mark.parametrize("hq,hkv,keys", [(8, 2, [60, 20]), (8, 2, [2000, 300]), (16, 2, [900, 90]), (16, 2, [100, 9]),
                                         (12, 1, [300, 40])])
def test_a_replay_with_more_rows_than_its_launch_is_flagged(hq, hkv, keys):
    """A host table of one or two rows a stream and nine on the device: reported, what the launch holds flagged, the
    rest and the other stream as they were or as they should be (decode and the tensor-core kernel with and
    without a merge, the general kernel)."""
    few = [1, 1] if hq == 8 else [2, 1]
    b, sides, c = q8_batch("int8", 11, rows=[9, 1], keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=128,
                           page_size=32)
    n, _, d = b.q.shape
    held = b.segs.copy()
    held[:, 1] = few
    ws = torch.full((tf.tf_paged_attn_q8_workspace_bytes(n, hq, d, 64),), 255, dtype=torch.uint8, device=DEV)
    out, fl = torch.full((n, hq, d), 5.0, device=DEV), torch.full((n, hq), 9, dtype=torch.uint8, device=DEV)
    st = status_word()
    tf.tf_paged_attn_q8(dev(b.q), c, dev(b.page_table), dev(b.segs), scale=b.scale, n_splits_max=64, workspace=ws,
                        out=out, flags=fl, status=st, segs_host=held)
    ref, rf, vmax = reference(b, sides, "int8")
    got, flags = out.cpu().numpy(), fl.cpu().numpy()
    assert int(st.item()) == binding.TF_DEV_BAD_SEG
    sv.check_attention(got[9:], flags[9:], ref[9:], rf[9:], vmax, False)
    assert np.isnan(got[: few[0]]).all() and (flags[: few[0]] == 1).all()
    rest = flags[few[0] : 9]
    assert ((rest == 9) | (rest == 1)).all() and (got[few[0] : 9][rest == 9] == 5.0).all()
    assert np.isnan(got[few[0] : 9][rest == 1]).all()


def test_a_prefix_with_more_rows_than_its_launch_is_flagged():
    b, prefixes, segs = batch(12, [300], [0] * 40, [1] * 40, [9 + i for i in range(40)], 16, 2, 128, 32)
    few = prefixes.copy()
    few[0, 1] = 3
    n, hq, d = b.q.shape
    ws = torch.full((tf.tf_paged_attn_shared_workspace_bytes(n, hq, d, 8, 8),), 255, dtype=torch.uint8, device=DEV)
    out, fl = torch.full((n, hq, d), 5.0, device=DEV), torch.full((n, hq), 9, dtype=torch.uint8, device=DEV)
    st = status_word()
    tf.tf_paged_attn_shared(dev(b.q), dev(b.k_pool), dev(b.v_pool), dev(b.page_table), dev(prefixes), dev(segs),
                            scale=b.scale, n_prefix_splits=8, n_splits_max=8, workspace=ws, out=out, flags=fl,
                            status=st, prefixes_host=few, segs_host=segs)
    assert int(st.item()) == binding.TF_DEV_BAD_SEG
    assert torch.isnan(out).all() and (fl == 1).all()


@pytest.mark.parametrize("read", [False, True])
def test_cache_rows_past_the_launch_are_reported(read):
    b, sides, c = q8_batch("int8", 13, rows=[40, 2], keys=[50, 30], n_q_heads=2, n_kv_heads=2, head_dim=128,
                           page_size=16)
    held = b.segs.copy()
    held[0, 1] = 3
    st, pt, sg = status_word(), dev(b.page_table), dev(b.segs)
    before = [t.view(torch.uint8).clone() for t in c.tensors]
    if read:
        pools = [torch.full(c.tensors[0].shape, 7.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        tf.tf_kv_read_q8(c, pt, sg, *pools, pt, status=st, segs_host=held)
        changed = [(p != 7.0).flatten(1).any(1) for p in pools]
    else:
        kr = torch.full((42, 2, 128), 3.0, dtype=torch.bfloat16, device=DEV)
        tf.tf_kv_append_q8(kr, kr, c, pt, sg, status=st, segs_host=held)
        changed = [(t.view(torch.uint8) != o).flatten(1).any(1) for t, o in zip(c.tensors[:2], before)]
    assert int(st.item()) == binding.TF_DEV_BAD_SEG
    mine = set(b.page_table[b.segs[1, 3] : b.segs[1, 3] + 2].tolist())
    for x in changed:  # the first stream is skipped, the second one's last two keys are in its second page
        assert set(torch.nonzero(x).flatten().tolist()) == {int(b.page_table[b.segs[1, 3] + 1])} <= mine


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,held,keys", [(8, 2, 1, 60), (8, 2, 1, 1500),  # decode: one split, partials
                                              (16, 2, 12, 60), (16, 2, 12, 1500),  # the tensor-core kernel
                                              (12, 1, 3, 300)])  # the general kernel
def test_a_damaged_entry_touches_its_own_rows_only(hq, hkv, held, keys, dt):
    """Whatever the form of the call, of a bad device entry the rows the launch holds are flagged and reported, no
    others are written, and the streams beside it come out as they should."""
    b, sides, c = q8_batch("int8", 14, rows=[held, 2 * held, held, 2 * held], keys=[keys + 60, keys, keys // 2 + 30, 40],
                           n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=32)
    n, _, d = b.q.shape
    good = b.segs.copy()
    good[[1, 3], 1] = held  # the second half of streams 1 and 3's rows belongs to no one
    ref, rf, vmax = reference(b, sides, "int8", segs=good)
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(n, hq, d, 32), dtype=torch.uint8, device=DEV)

    def case(change, flagged, bit=binding.TF_DEV_BAD_SEG):
        segs = good.copy()
        change(segs)
        out, fl = torch.full((n, hq, d), 5.0, dtype=dt, device=DEV), torch.full((n, hq), 9, dtype=torch.uint8, device=DEV)
        st = status_word()
        tf.tf_paged_attn_q8(dev(b.q), c, dev(b.page_table), dev(segs), scale=b.scale, n_splits_max=32, workspace=ws,
                            out=out, flags=fl, status=st, segs_host=good)
        assert int(st.item()) == bit
        out, fl = out.float().cpu().numpy(), fl.cpu().numpy()
        named = np.zeros(n, bool)
        for s, (q_row, r, *_) in enumerate(good):
            if (segs[s] == good[s]).all():
                named[q_row : q_row + r] = True
        sv.check_attention(out[named], fl[named], ref[named], rf[named], vmax, dt == torch.bfloat16)
        gone = np.zeros(n, bool)
        gone[flagged] = True
        assert np.isnan(out[gone]).all() and (fl[gone] == 1).all()
        rest = ~named & ~gone
        assert (out[rest] == 5.0).all() and (fl[rest] == 9).all()

    q1, q3 = good[1, 0], good[3, 0]

    def put(s, at, x):
        def change(segs):
            segs[s, at] = x

        return change

    case(put(1, 1, 2 * held), slice(q1, q1 + held))  # more rows than the launch holds
    case(put(1, 1, held + 1), slice(q1, q1 + held))
    case(put(1, 0, -held), slice(0, 0))  # before the first row: nothing of it is written
    if held > 1:
        case(put(3, 0, n - 1), slice(n - 1, n))  # past the last one
    case(put(1, 4, 0), slice(q1, q1 + held), binding.TF_DEV_PAST_PAGES)
    case(put(3, 3, -1), slice(q3, q3 + held))


@pytest.mark.parametrize("hq,hkv,rows,keys,host", [(8, 2, 1, 60, True), (8, 2, 1, 1500, True), (16, 2, 12, 60, True),
                                                   (16, 2, 12, 1500, True), (12, 1, 3, 300, True), (8, 2, 1, 60, False)])
def test_a_device_entry_of_two_billion_keys_is_refused(hq, hkv, rows, keys, host):
    """A page table of 2^21 entries, all of one page of 1,024 keys, and an entry on the device that names all of its
    2^31 - 1 keys: past what a call takes, reported and flagged, the other stream as it should be."""
    b, sides, c = q8_batch("int8", 16, rows=[rows, rows], keys=[keys, keys // 2], n_q_heads=hq, n_kv_heads=hkv,
                           head_dim=128, page_size=1024)
    n, _, d = b.q.shape
    pt = torch.full((1 << 21,), int(b.page_table[0]), dtype=torch.int32, device=DEV)
    pt[: len(b.page_table)] = dev(b.page_table)
    segs = b.segs.copy()
    segs[1] = [rows, rows, 2**31 - 1, 0, 1 << 21]
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(n, hq, d, 64), dtype=torch.uint8, device=DEV)
    for split in (0, 1 << 30):
        out, fl = torch.full((n, hq, d), 5.0, device=DEV), torch.full((n, hq), 9, dtype=torch.uint8, device=DEV)
        st = status_word()
        tf.tf_paged_attn_q8(dev(b.q), c, pt, dev(segs), scale=b.scale, n_splits_max=64, split_keys=split, workspace=ws,
                            out=out, flags=fl, status=st, segs_host=b.segs if host else None)
        ref, rf, vmax = reference(b, sides, "int8")
        assert int(st.item()) == binding.TF_DEV_BAD_SEG
        out, fl = out.cpu().numpy(), fl.cpu().numpy()
        sv.check_attention(out[:rows], fl[:rows], ref[:rows], rf[:rows], vmax, False)
        assert np.isnan(out[rows:]).all() and (fl[rows:] == 1).all()


@pytest.mark.parametrize("rows,hq,hkv", [(1, 8, 2), (12, 16, 2), (3, 12, 1)])
@pytest.mark.parametrize("prefix", [False, True])
def test_a_shared_device_entry_of_two_billion_keys_is_refused(rows, hq, hkv, prefix):
    b, prefixes, segs = batch(19, [300], [0, 0], [rows] * 2, [200, 100], hq, hkv, 128, 1024)
    n, _, d = b.q.shape
    pt = torch.full((1 << 21,), int(b.page_table[0]), dtype=torch.int32, device=DEV)
    pt[: len(b.page_table)] = dev(b.page_table)
    dpre, dsegs = prefixes.copy(), segs.copy()
    if prefix:
        dpre[0, 2:] = [2**31 - 1, 0, 1 << 21]
    else:
        dsegs[1, 2:] = [2**31 - 1, 0, 1 << 21]
    ws = torch.empty(tf.tf_paged_attn_shared_workspace_bytes(n, hq, d, 8, 8), dtype=torch.uint8, device=DEV)
    out, fl = torch.full((n, hq, d), 5.0, device=DEV), torch.full((n, hq), 9, dtype=torch.uint8, device=DEV)
    st = status_word()
    tf.tf_paged_attn_shared(dev(b.q), dev(b.k_pool), dev(b.v_pool), pt, dev(dpre), dev(dsegs), scale=b.scale,
                            n_prefix_splits=8, n_splits_max=8, workspace=ws, out=out, flags=fl, status=st,
                            prefixes_host=prefixes, segs_host=segs)
    assert int(st.item()) & binding.TF_DEV_BAD_SEG
    gone = slice(0, n) if prefix else slice(rows, n)
    out, fl = out.cpu().numpy(), fl.cpu().numpy()
    assert np.isnan(out[gone]).all() and (fl[gone] == 1).all()
    if not prefix:
        ref, rf, vmax = shared_reference(b, prefixes, segs, [0, 0])
        sv.check_attention(out[:rows], fl[:rows], ref[:rows], rf[:rows], vmax, False)


@pytest.mark.parametrize("rows,keys,hq,hkv,d", [([12, 0, 3], [300, 2000, 90], 4, 2, 64),  # tcgen05, partials and merge
                                                ([9, 0], [60, 1500], 8, 1, 128),  # tcgen05, one split
                                                ([1, 0, 1], [300, 2000, 90], 8, 2, 128), ([0, 1], [1500, 60], 8, 2, 64),  # decode
                                                ([5, 0], [300, 2000], 24, 2, 128)])  # the general kernel
def test_a_stream_without_rows_may_have_any_keys(rows, keys, hq, hkv, d):
    """The launch holds the partials of the streams with rows; a longer stream without rows needs none."""
    b, sides, c = q8_batch("int8", 31, rows=rows, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32)
    ref, fl, vmax = reference(b, sides, "int8")
    out, flags, st = attn(c, b, "int8", n_splits_max=2)
    assert st == 0
    sv.check_attention(out, flags, ref, fl, vmax, False)


@pytest.mark.parametrize("rows,own,hq,hkv", [([5, 0, 2], [40, 900, 70], 16, 2), ([1, 0, 1], [40, 900, 70], 8, 2)])
def test_prefixes_and_streams_without_rows_may_have_any_keys(rows, own, hq, hkv):
    """The third prefix has no rows, as every stream of it has none."""
    b, prefixes, segs = batch(32, [90, 33, 1000], [0, 0, 1], rows, own, hq, hkv, 128, 16)
    assert prefixes[2, 1] == 0 and segs[1, 1] == 0
    ref, fl, vmax = shared_reference(b, prefixes, segs, [0, 0, 1])
    for host in (True, "segs", "prefixes"):
        out, flags, st = shared(b, prefixes, segs, host=host, split=64, n_pre=2, n_own=2)
        assert st == 0
        sv.check_attention(out, flags, ref, fl, vmax, False)


@pytest.mark.parametrize("fn", [tf.tf_paged_attn_decode, tf.tf_paged_attn_block])
def test_bf16_partials_of_a_stream_without_rows(fn):
    b = wl.make_paged_batch(33, rows=[12, 0], keys=[100, 1000], n_q_heads=16, n_kv_heads=2, head_dim=128, page_size=16,
                            split_keys=64, n_splits_max=2)
    n, f = b.q.shape[0], dict(device=DEV, dtype=torch.float32)
    po, pm, pl = torch.zeros((n, 16, 2, 128), **f), torch.zeros((n, 16, 2), **f), torch.zeros((n, 16, 2), **f)
    pf, st = torch.zeros((n, 16, 2), dtype=torch.uint8, device=DEV), status_word()
    fn(dev(b.q), dev(b.k_pool), dev(b.v_pool), dev(b.page_table), dev(b.segs), scale=b.scale, split_keys=64,
       n_splits_max=2, part_o=po, part_m=pm, part_l=pl, part_flag=pf, status=st, segs_host=b.segs)
    assert int(st.item()) == 0


HELD = [(12, 1, 128), (4, 1, 128), (16, 1, 64), (1, 1, 128), (2, 2, 256), (32, 2, 256)]  # general, decode, tcgen05


@pytest.mark.parametrize("hq,hkv,d", HELD)
@pytest.mark.parametrize("n_splits", [1, 8])
@pytest.mark.parametrize("more", [2, 5])
def test_an_entry_with_more_rows_than_the_launch_leaves_its_neighbours(hq, hkv, d, n_splits, more):
    """Five one-row streams; on the device the first entry has grown over the rows of the next ones: its one row that
    the launch holds is flagged, the others' are right."""
    b, sides, c = q8_batch("e4m3", 41, rows=[1] * 5, keys=[300, 90, 64, 500, 40], n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                           page_size=16)
    ref, fl, vmax = reference(b, sides, "e4m3")
    segs = b.segs.copy()
    segs[0, 1] = more
    q, pt = dev(b.q), dev(b.page_table)
    out, flags, st = torch.full(b.q.shape, 5.0, device=DEV), torch.full((5, hq), 9, dtype=torch.uint8, device=DEV), status_word()
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(5, hq, d, n_splits), dtype=torch.uint8, device=DEV)
    for _ in range(5):
        tf.tf_paged_attn_q8(q, c, pt, dev(segs), scale=b.scale, n_splits_max=n_splits, workspace=ws, out=out, flags=flags,
                            status=st, segs_host=b.segs)
        assert int(st.item()) == binding.TF_DEV_BAD_SEG
        o, f = out.cpu().numpy(), flags.cpu().numpy()
        assert (f[0] == 1).all() and np.isnan(o[0]).all()
        sv.check_attention(o[1:], f[1:], ref[1:], fl[1:], vmax, False)


@pytest.mark.parametrize("hq,hkv,d", HELD)
@pytest.mark.parametrize("which", ["segs", "prefixes"])
def test_a_shared_entry_with_more_rows_than_the_launch_leaves_its_neighbours(hq, hkv, d, which):
    """The same behind two prefixes: a stream that has grown over the next ones' rows, or the first prefix over the
    second's."""
    groups = [0, 0, 1, 1, 1] if which == "segs" else [0, 1, 1, 1, 1]
    b, prefixes, segs = batch(42, [90, 200], groups, [1] * 5, [300, 90, 64, 500, 40], hq, hkv, d, 16)
    ref, fl, vmax = shared_reference(b, prefixes, segs, groups)
    bad_segs, bad_prefixes = segs.copy(), prefixes.copy()
    if which == "segs":
        bad_segs[0, 1] = 3
        wrong = [0]
    else:
        bad_prefixes[0, 1] = 5  # more than the four that the launch holds
        wrong = [0, 1, 2, 3, 4]
    n = b.q.shape[0]
    out, flags, st = torch.full(b.q.shape, 5.0, device=DEV), torch.full((n, hq), 9, dtype=torch.uint8, device=DEV), status_word()
    ws = torch.empty(tf.tf_paged_attn_shared_workspace_bytes(n, hq, d, 8, 8), dtype=torch.uint8, device=DEV)
    tf.tf_paged_attn_shared(dev(b.q), dev(b.k_pool).view(torch.bfloat16), dev(b.v_pool).view(torch.bfloat16),
                            dev(b.page_table), dev(bad_prefixes), dev(bad_segs), scale=b.scale, n_prefix_splits=8,
                            n_splits_max=8, workspace=ws, out=out, flags=flags, status=st, prefixes_host=prefixes,
                            segs_host=segs)
    assert int(st.item()) == binding.TF_DEV_BAD_SEG
    o, f = out.cpu().numpy(), flags.cpu().numpy()
    right = [r for r in range(n) if r not in wrong]
    assert (f[wrong] == 1).all() and np.isnan(o[wrong]).all()
    sv.check_attention(o[right], f[right], ref[right], fl[right], vmax, False)
