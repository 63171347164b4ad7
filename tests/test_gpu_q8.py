"""The 8-bit cache on the GPU: append bit for bit against the format's
definition, read-back exact, attention against float64 on the dequantised keys."""
import numpy as np
import pytest
import torch

import paged_kv_cache_segment_b200 as tf
from paged_kv_cache_segment_b200 import workloads as wl

import _serving as sv
from _gpu import DEV, dev, status_word

pytestmark = pytest.mark.gpu
KINDS = ("e4m3", "int8")


def cache_of(kc, vc, ks, vs, kind):
    code = torch.float8_e4m3fn if kind == "e4m3" else torch.int8
    t = [torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in (kc, vc, ks, vs)]
    return tf.Q8Cache(t[0].view(code), t[1].view(code), t[2], t[3])


def cache_bytes(c):
    return [t.view(torch.uint8).cpu().numpy() for t in c.tensors]


def rows_of(rng, shape):
    """bf16 rows whose sizes span the format: usual ones, tiny, huge, zero, a tie, signed zeros."""
    x = rng.standard_normal(shape).astype(np.float32) * np.exp(rng.normal(0, 1, shape[:-1]))[..., None].astype(np.float32)
    flat = x.reshape(-1, shape[-1])
    n = len(flat)
    flat[0 % n] = 0.0
    if n > 1:
        flat[1] *= np.float32(2.0**-120)
    if n > 2:
        flat[2] *= np.float32(2.0**110)
    if n > 3:  # codes that sit on a rounding border: 448 sets the scale to 1
        flat[3, :] = np.float32(-0.0)
        flat[3, :6] = [448, 17, 19, 1.0625, 0.5 * 2.0**-9, -1.5 * 2.0**-9]
    if n > 4:
        flat[4, :] = 0
        flat[4, :6] = [127, 0.5, 1.5, -2.5, 126.5, -0.25]
    bits = wl.f32_to_bf16_bits(x)
    return bits


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,hkv,psz", [(64, 2, 8), (128, 8, 32), (256, 3, 64), (128, 1, 1024)])
def test_append_is_the_format(kind, d, hkv, psz):
    rows, keys = [3, 0, 1, 17, 9], [10, 0, psz, psz + 17, 2 * psz + 5]
    b = wl.make_paged_batch(3, rows=[max(r, 0) for r in rows], keys=[max(k, r) for k, r in zip(keys, rows)],
                            n_q_heads=hkv, n_kv_heads=hkv, head_dim=64, page_size=psz, extra_pages=2)
    rng = np.random.default_rng(5)
    kr, vr = rows_of(rng, (sum(rows), hkv, d)), rows_of(rng, (sum(rows), hkv, d))
    kr[6, 0, 5] = 0x7F80  # +inf, NaN: the whole row is marked
    vr[9, hkv - 1, 0] = 0x7FC1
    pools = [rng.integers(0, 256, (b.n_pages, hkv, psz, d)).astype(np.uint8) for _ in "kv"]
    scales = [rng.integers(0, 256, (b.n_pages, hkv, psz)).astype(np.uint8) for _ in "kv"]
    c = cache_of(pools[0], pools[1], scales[0], scales[1], kind)
    want = [p.copy() for p in pools + scales]
    for n, bits in enumerate((kr, vr)):
        codes, sc = sv.quantise(bits, kind)
        for q_row, r, nk, base, _ in b.segs:
            for i in range(r):
                j = nk - r + i
                page = b.page_table[base + j // psz]
                want[n][page, :, j % psz] = codes[q_row + i]
                want[2 + n][page, :, j % psz] = sc[q_row + i]
    st = status_word()
    tf.tf_kv_append_q8(dev(kr), dev(vr), c, dev(b.page_table), dev(b.segs), status=st, segs_host=b.segs,
                       page_table_host=b.page_table)
    for got, exp in zip(cache_bytes(c), want):
        assert (got == exp).all()
    assert int(st.item()) == 0
    # without host tables, and written again: the same bytes
    tf.tf_kv_append_q8(dev(kr), dev(vr), c, dev(b.page_table), dev(b.segs), status=st)
    for got, exp in zip(cache_bytes(c), want):
        assert (got == exp).all()


@pytest.mark.parametrize("kind", KINDS)
def test_every_code_reads_back_exactly_and_appends_back(kind):
    """All 256 codes under scales over the whole range: read-back is exact in bf16, and appending what was read gives
    the same values again."""
    psz, hkv, d = 8, 2, 256
    n = 40
    n_pages = n // psz
    codes = np.broadcast_to(np.arange(256, dtype=np.uint8), (n_pages, hkv, psz, d)).copy()
    if kind == "e4m3":
        codes[(codes & 127) == 127] = 0  # NaN codes are never written
    else:
        codes[codes == 128] = 0  # nor is -128
    rng = np.random.default_rng(1)
    scale = rng.integers(27, 238, (n_pages, hkv, psz)).astype(np.uint8)
    scale[0, 0, 3] = 255
    c = cache_of(codes, codes, scale, scale, kind)
    pt = rng.permutation(n_pages).astype(np.int32)
    dst = np.arange(n_pages, dtype=np.int32)[::-1].copy() + 1
    segs = np.array([[0, n, n, 0, n_pages]], np.int32)
    kp = torch.full((n_pages + 1, hkv, psz, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    st = status_word()
    tf.tf_kv_read_q8(c, dev(pt), dev(segs), kp, vp, dev(dst), status=st, segs_host=segs, page_table_host=pt,
                     dst_page_table_host=dst)
    want = np.full(tuple(kp.shape), 7.0)
    vals = sv.values(codes, scale, kind)
    for i in range(n_pages):
        want[dst[i]] = vals[pt[i]]
    for got in (kp, vp):
        got = got.double().cpu().numpy()
        assert ((got == want) | (np.isnan(got) & np.isnan(want))).all()
    rows = np.ascontiguousarray(np.concatenate([want[dst[i]].transpose(1, 0, 2) for i in range(n_pages)]))
    c2 = cache_of(np.zeros_like(codes), np.zeros_like(codes), scale * 0, scale * 0, kind)
    kr = torch.from_numpy(rows).to(DEV).to(torch.bfloat16)
    tf.tf_kv_append_q8(kr, kr, c2, dev(pt), dev(segs), status=st, segs_host=segs)
    kc, _, ks, _ = cache_bytes(c2)
    again = sv.values(kc, ks, kind)
    for i in range(n_pages):
        w = vals[pt[i]]
        assert ((again[pt[i]] == w) | np.isnan(w)).all() and (np.isnan(again[pt[i]]) == np.isnan(w)).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,hkv,psz", [(64, 2, 16), (128, 4, 8), (256, 1, 128)])
def test_read_takes_the_last_rows_of_each_stream(kind, d, hkv, psz):
    rows, keys = [5, 0, 1, 33], [2 * psz + 3, psz, 1, 33]
    b = wl.make_paged_batch(4, rows=rows, keys=keys, n_q_heads=hkv, n_kv_heads=hkv, head_dim=64, page_size=psz,
                            extra_pages=1)
    rng = np.random.default_rng(6)
    sides = [sv.quantise(rows_of(rng, (b.n_pages, hkv, psz, d)), kind) for _ in "kv"]
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    dst = rng.permutation(len(b.page_table) + 2)[: len(b.page_table)].astype(np.int32)
    segs = b.segs.copy()
    segs[:, 0] = -7  # q_row is not used
    for host in (True, False):
        pools = [torch.full((len(dst) + 2, hkv, psz, d), 3.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        st = status_word()
        tf.tf_kv_read_q8(c, dev(b.page_table), dev(segs), pools[0], pools[1], dev(dst), status=st,
                         segs_host=segs if host else None)
        assert int(st.item()) == 0
        for got, (codes, sc) in zip(pools, sides):
            want = np.full(tuple(got.shape), 3.0)
            vals = sv.values(codes, sc, kind)
            for _, r, nk, base, _ in segs:
                for j in range(nk - r, nk):
                    want[dst[base + j // psz], :, j % psz] = vals[b.page_table[base + j // psz], :, j % psz]
            assert (got.double().cpu().numpy() == want).all()


def test_bad_device_tables_are_reported_and_skipped():
    kind, d, hkv, psz = "e4m3", 64, 2, 8
    pt = np.array([0, 9, 1, -1], np.int32)
    good = np.array([0, 1, 2, 3], np.int32)
    zero = np.zeros((4, hkv, psz, d), np.uint8)
    kr = dev(wl.normal_bf16(np.random.default_rng(0), (16, hkv, d)))
    for segs, bit in ([[0, 16, 16, 0, 2]], 4), ([[0, 16, 17, 0, 2]], 2), ([[9, 8, 8, 0, 1]], 1), ([[0, 8, 4, 0, 1]], 1), \
            ([[0, 8, 8, 3, 2]], 1):
        segs = np.array(segs, np.int32)
        c = cache_of(zero, zero, zero[..., 0], zero[..., 0], kind)
        st = status_word()
        tf.tf_kv_append_q8(kr, kr, c, dev(pt), dev(segs), status=st)
        assert int(st.item()) == bit, (segs, int(st.item()))
        kc, _, ks, _ = cache_bytes(c)
        assert (kc[1:] == 0).all() and (ks[1:] == 0).all()
        assert (kc[0] != 0).any() == (bit == 4)  # only the row range on the good page was written
        if bit == 1 and segs[0, 0] == 9:
            continue  # a read does not use q_row
        pools = [torch.zeros((4, hkv, psz, d), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        st = status_word()
        tf.tf_kv_read_q8(c, dev(good), dev(segs), pools[0], pools[1], dev(pt), status=st)
        assert int(st.item()) == bit
        assert (pools[0][1:] == 0).all()


def attn(c, b, kind, *, split=0, n_splits_max=16, full=False, host=True, out_dtype=torch.float32, segs=None, out=None,
         flags=None, stream=None, ws=None):
    segs = b.segs if segs is None else segs
    rows, hq, d = b.q.shape
    out = torch.full((rows, hq, d), 5.0, dtype=out_dtype, device=DEV) if out is None else out
    flags = torch.full((rows, hq), 9, dtype=torch.uint8, device=DEV) if flags is None else flags
    n = tf.tf_paged_attn_q8_workspace_bytes(rows, hq, d, n_splits_max)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if ws is None else ws
    st = status_word()
    tf.tf_paged_attn_q8(dev(b.q), c, dev(b.page_table), dev(np.ascontiguousarray(segs, np.int32)), scale=b.scale,
                        split_keys=split, n_splits_max=n_splits_max, full=full, workspace=ws, out=out, flags=flags,
                        status=st, segs_host=segs if host else None, page_table_host=b.page_table if host else None,
                        stream=stream)
    return out.float().cpu().numpy(), flags.cpu().numpy(), int(st.item())


def q8_batch(kind, seed, poison=True, **kw):
    """A paged batch whose pool is quantised; slots past a stream's keys and pages no stream owns hold NaN rows."""
    b = wl.make_paged_batch(seed, unused="nan" if poison else "normal", **kw)
    sides = [sv.quantise(p, kind) for p in (b.k_pool, b.v_pool)]
    if poison and kind == "e4m3":
        for codes, sc in sides:
            codes[sc == 255] = 0x7F
    return b, sides, cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)


def reference(b, sides, kind, full=False, segs=None):
    rows, hq, d = b.q.shape
    ref, fl = np.full((rows, hq, d), np.nan), np.ones((rows, hq), np.uint8)
    q = sv.bf16(b.q)
    vmax = 0.0
    for q_row, r, n, base, _ in (b.segs if segs is None else segs):
        k, v = (sv.values(sv.keys_of(c, b.page_table, base, n), sv.keys_of(s, b.page_table, base, n), kind)
                for c, s in sides)
        vmax = max(vmax, float(np.nanmax(np.abs(v))) if v.size else 0.0)
        lims = [n if full else n - r + i + 1 for i in range(r)]
        ref[q_row : q_row + r], fl[q_row : q_row + r] = sv.attend(q[q_row : q_row + r], k, v, lims, b.scale)
    return ref, fl, vmax


SHAPES = [  # rows, keys, hq, hkv, d, psz: decode-shaped, odd lengths
    ([1, 1], [37, 70], 8, 2, 64, 16),
    ([1, 1, 1, 1, 1], [1, 2, 63, 64, 65], 4, 4, 128, 8),
    ([1, 1, 1], [1000, 129, 513], 32, 8, 128, 32),
    ([2, 1, 2], [300, 64, 2], 8, 2, 256, 32),
    ([1, 1], [700, 1025], 8, 1, 256, 1024),
    ([8, 3], [200, 77], 2, 2, 64, 64),
    ([1], [4111], 7, 1, 128, 256),
    # more than 8 queries a kv-head: verify rounds and blocks
    ([5, 16, 1], [400, 1000, 65], 16, 2, 256, 32),
    ([9, 2], [700, 130], 32, 8, 128, 32),
    ([40, 3], [90, 5], 4, 4, 64, 8),
    ([3, 5], [200, 333], 24, 2, 128, 16),  # a group of 12: the general kernel
    ([130], [150], 3, 1, 64, 16),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention_matches_float64(kind, shape):
    rows, keys, hq, hkv, d, psz = SHAPES[shape]
    b, sides, c = q8_batch(kind, 10 + shape, rows=rows, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                           page_size=psz, extra_pages=2)
    for full in (False, True):
        ref, fl, vmax = reference(b, sides, kind, full)
        for split, nsm, host, dt in ((0, 16, True, torch.float32), (0, 3, False, torch.bfloat16),
                                     (256, 32, True, torch.bfloat16), (64, 65, False, torch.float32),
                                     (48, 87, True, torch.float32)):
            out, flags, st = attn(c, b, kind, split=split, n_splits_max=nsm, full=full, host=host, out_dtype=dt)
            assert st == 0
            sv.check_attention(out, flags, ref, fl, vmax, dt == torch.bfloat16, f"{full} {split} {host}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,hq,hkv,d", [([1, 1], 8, 2, 128), ([3, 2], 4, 2, 64), ([6, 9], 16, 2, 256),
                                           ([4, 7], 12, 1, 128)])
def test_nonfinite_rows_flag_the_queries_that_see_them(kind, rows, hq, hkv, d):
    b, sides, _ = q8_batch(kind, 21, rows=rows, keys=[150, 170], n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                           page_size=16)
    psz = 16

    def mark(side, s, j, g):
        page = b.page_table[b.segs[s][3] + j // psz]
        sides[side][1][page, g, j % psz] = 255
        sides[side][0][page, g, j % psz] = 0

    mark(0, 0, 149, 0)  # the last key: only the last row sees it (causal)
    mark(1, 1, 169, hkv - 1)
    if rows[1] > 1:
        mark(1, 1, 168, 0)
    b.q[-1, hq - 1, 3] = 0x7F80
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    for full in (False, True):
        ref, fl, vmax = reference(b, sides, kind, full)
        for host in (True, False):
            out, flags, st = attn(c, b, kind, full=full, host=host)
            assert st == 0
            sv.check_attention(out, flags, ref, fl, vmax, False, f"{full} {host}")
    mark(1, 0, 5, 0)  # and a value row everybody sees
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    ref, fl, vmax = reference(b, sides, kind)
    out, flags, _ = attn(c, b, kind)
    sv.check_attention(out, flags, ref, fl, vmax, False)


@pytest.mark.parametrize("rows,hq,hkv", [([1, 1], 8, 2), ([4, 3], 16, 2)])
def test_value_and_key_scales_far_apart(rows, hq, hkv):
    """Value rows 2^60 apart and key rows 2^20 apart: each keeps its own scale, none is lost next to another."""
    b, sides, _ = q8_batch("int8", 31, rows=rows, keys=[300, 200], n_q_heads=hq, n_kv_heads=hkv, head_dim=128,
                           page_size=32, poison=False)
    rng = np.random.default_rng(3)
    sides[1][1][:] = rng.integers(60, 121, sides[1][1].shape)
    sides[0][1][:] = rng.integers(100, 121, sides[0][1].shape)
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], "int8")
    ref, fl, _ = reference(b, sides, "int8")
    out, flags, st = attn(c, b, "int8")
    assert st == 0 and (flags == fl).all()
    # a head's error is bounded by its own largest weighted value, so each head is held to its own size
    err = np.linalg.norm(out - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert err.max() <= 2.0**-14


def test_only_named_rows_are_written_and_bad_entries_are_flagged():
    b, sides, c = q8_batch("e4m3", 41, rows=[1, 2, 1, 1], keys=[50, 60, 70, 20], n_q_heads=4, n_kv_heads=2,
                           head_dim=64, page_size=16)
    ref, fl, vmax = reference(b, sides, "e4m3")
    segs = b.segs.copy()
    segs[2, 1] = 0  # a stream with nothing to do this step: its row stays as it was
    out, flags, st = attn(c, b, "e4m3", segs=segs)
    row = b.segs[2][0]
    assert st == 0 and (out[row] == 5.0).all() and (flags[row] == 9).all()
    keep = np.arange(5) != row
    sv.check_attention(out[keep], flags[keep], ref[keep], fl[keep], vmax, False)
    segs = b.segs.copy()
    segs[1, 4] = 1  # 60 keys on one page of 16
    out, flags, st = attn(c, b, "e4m3", segs=segs, host=False)
    assert st == 2
    rows = slice(b.segs[1][0], b.segs[1][0] + 2)
    assert np.isnan(out[rows]).all() and (flags[rows] == 1).all()
    keep = np.r_[0, 3, 4]
    sv.check_attention(out[keep], flags[keep], ref[keep], fl[keep], vmax, False)
    segs = b.segs.copy()
    out, flags, st = attn(c, b, "e4m3", segs=segs, host=False, split=16, n_splits_max=4)  # 70 keys need 5
    assert st == 8 and (flags[b.segs[2][0]] == 1).all() and np.isnan(out[b.segs[2][0]]).all()
    pt = b.page_table.copy()
    pt[b.segs[0][3] + 1] = b.n_pages
    b.page_table = pt
    out, flags, st = attn(c, b, "e4m3", host=False)
    assert st == 4 and (flags[0] == 1).all() and (flags[1:] == 0).all()


def test_attention_over_the_cache_is_attention_over_its_read_back():
    b, sides, c = q8_batch("int8", 51, rows=[4, 2], keys=[333, 90], n_q_heads=16, n_kv_heads=4, head_dim=128,
                           page_size=32)
    n = len(b.page_table)
    dst = np.arange(n, dtype=np.int32)
    pools = [torch.full((n, 4, 32, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    segs = b.segs.copy()
    segs[:, 1] = segs[:, 2]
    st = status_word()
    tf.tf_kv_read_q8(c, dev(b.page_table), dev(segs), pools[0], pools[1], dev(dst), status=st, segs_host=segs)
    rows, hq, d = b.q.shape
    full = torch.empty((rows, hq, d), device=DEV)
    for s in range(2):  # each stream's rows as a prompt chunk
        tf.tf_paged_attn_prompt(dev(b.q), pools[0], pools[1], dev(dst), b.segs[s], scale=b.scale, out=full, status=st)
    out, flags, _ = attn(c, b, "int8")
    assert int(st.item()) == 0
    ref, fl, vmax = reference(b, sides, "int8")
    sv.check_attention(out, flags, ref, fl, vmax, False)
    sv.check_attention(full.cpu().numpy(), flags, ref, fl, vmax, False)


@pytest.mark.parametrize("rows,hq,hkv,d", [([1, 1], 8, 2, 64), ([1] * 16, 32, 8, 128), ([7, 3], 16, 2, 256)])
def test_captured_replayed_and_on_another_stream(rows, hq, hkv, d):
    """The same bits from eager calls, a graph's replays and another stream; the tables may change between replays
    (they are device memory) as long as the host copies' sizes hold."""
    rng = np.random.default_rng(8)
    keys = [int(k) for k in rng.integers(300, 900, len(rows))]
    b, sides, c = q8_batch("e4m3", 61, rows=rows, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32)
    n_rows = b.q.shape[0]
    eager = attn(c, b, "e4m3")
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(n_rows, hq, d, 16), dtype=torch.uint8, device=DEV)
    out = torch.zeros((n_rows, hq, d), device=DEV)
    flags = torch.zeros((n_rows, hq), dtype=torch.uint8, device=DEV)
    st = status_word()
    args = (dev(b.q), c, dev(b.page_table), dev(b.segs))
    kw = dict(scale=b.scale, n_splits_max=16, workspace=ws, out=out, flags=flags, status=st, segs_host=b.segs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tf.tf_paged_attn_q8(*args, **kw, stream=side)
    side.synchronize()
    assert (out.cpu().numpy() == eager[0]).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tf.tf_paged_attn_q8(*args, **kw)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert (out.cpu().numpy() == eager[0]).all() and (flags.cpu().numpy() == eager[1]).all()


def test_a_decode_step_over_the_8_bit_cache():
    """A step as a server runs it: the new rows appended, every stream's row attended, the logits scored."""
    kind, hq, hkv, d, psz = "e4m3", 8, 2, 128, 16
    b, sides, c = q8_batch(kind, 71, rows=[1, 1, 2], keys=[40, 16, 33], n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                           page_size=psz)
    rng = np.random.default_rng(2)
    kr, vr = wl.normal_bf16(rng, (4, hkv, d)), wl.normal_bf16(rng, (4, hkv, d))
    st = status_word()
    tf.tf_kv_append_q8(dev(kr), dev(vr), c, dev(b.page_table), dev(b.segs), status=st, segs_host=b.segs)
    for n, bits in enumerate((kr, vr)):
        codes, sc = sv.quantise(bits, kind)
        for q_row, r, nk, base, _ in b.segs:
            for i in range(r):
                j = nk - r + i
                page = b.page_table[base + j // psz]
                sides[n][0][page, :, j % psz], sides[n][1][page, :, j % psz] = codes[q_row + i], sc[q_row + i]
    ref, fl, vmax = reference(b, sides, kind)
    out, flags, bits = attn(c, b, kind, out_dtype=torch.bfloat16)
    assert bits == 0 and int(st.item()) == 0
    sv.check_attention(out, flags, ref, fl, vmax, True)
    x = out.reshape(4, -1) @ rng.standard_normal((hq * d, 501)).astype(np.float32)
    logits = torch.from_numpy(x).to(DEV).to(torch.bfloat16)
    tok = torch.from_numpy(rng.integers(0, 501, (4, 2)).astype(np.int32)).to(DEV)
    tl, ids, tops = torch.empty((4, 2), device=DEV), torch.empty((4, 3), dtype=torch.int32, device=DEV), \
        torch.empty((4, 3), device=DEV)
    fl8 = torch.empty(4, dtype=torch.uint8, device=DEV)
    tf.tf_logprob_rows(logits, tok, token_logprobs=tl, top_ids=ids, top_logprobs=tops, flags=fl8, status=st)
    r = sv.logprobs(logits.double().cpu().numpy(), 1.0, tok.cpu().numpy(), 3)
    assert (ids.cpu().numpy() == r[3]).all() and (fl8.cpu().numpy() == 0).all()
    assert np.abs(tl.cpu().numpy() - r[0]).max() <= 1e-4 and np.abs(tops.cpu().numpy() - r[4]).max() <= 1e-4
    am = torch.empty(4, dtype=torch.int32, device=DEV)
    tf.tf_argmax_rows(logits, am, fl8)
    assert (am.cpu().numpy() == r[3][:, 0]).all()


def test_shapes_and_devices_the_binding_refuses():
    b, sides, c = q8_batch("e4m3", 81, rows=[1, 1], keys=[40, 16], n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16)
    st, pt, sg = status_word(), dev(b.page_table), dev(b.segs)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="shapes disagree"):
        tf.tf_kv_append_q8(k[:, :1].contiguous(), k[:, :1].contiguous(), c, pt, sg, status=st)
    with pytest.raises(ValueError, match="contiguous"):
        tf.tf_kv_append_q8(k.transpose(0, 1), k, c, pt, sg, status=st)
    with pytest.raises(TypeError, match="dtype"):
        tf.tf_kv_append_q8(k.float(), k.float(), c, pt, sg, status=st)
    with pytest.raises(ValueError, match="differ in length"):
        tf.tf_kv_append_q8(k, k, c, pt, sg, status=st, segs_host=b.segs[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        tf.tf_kv_append_q8(k, k.cpu(), c, pt, sg, status=st)
    with pytest.raises(ValueError, match="five numbers"):
        tf.tf_kv_append_q8(k, k, c, pt, sg.reshape(-1)[:9].contiguous(), status=st)
    out, fl = torch.zeros((2, 8, 64), device=DEV), torch.zeros((2, 8), dtype=torch.uint8, device=DEV)
    ws = torch.zeros(tf.tf_paged_attn_q8_workspace_bytes(2, 8, 64, 2), dtype=torch.uint8, device=DEV)
    kw = dict(scale=0.125, n_splits_max=2, workspace=ws, status=st)
    with pytest.raises(ValueError, match="shapes disagree"):
        tf.tf_paged_attn_q8(dev(b.q), c, pt, sg, out=out[:1], flags=fl, **kw)
    with pytest.raises(tf.TfError, match="TF_ERR_WORKSPACE|workspace"):
        tf.tf_paged_attn_q8(dev(b.q), c, pt, sg, out=out, flags=fl, **dict(kw, workspace=ws[:-1]))
    # tables as lists and as int64 are converted; the same call still stands
    tf.tf_paged_attn_q8(dev(b.q), c, pt, sg, out=out, flags=fl, segs_host=b.segs.tolist(),
                        page_table_host=b.page_table.astype(np.int64), **kw)
    ref, rf, vmax = reference(b, sides, "e4m3")
    sv.check_attention(out.cpu().numpy(), fl.cpu().numpy(), ref, rf, vmax, False)
