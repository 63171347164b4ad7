"""What the serving calls' outputs hold beyond the common bounds: bf16 rows that are the f32 rows rounded, weights far
below the largest."""
import numpy as np
import pytest
import torch

from paged_kv_cache_segment_b200 import workloads as wl

import _serving as sv
from test_gpu_q8 import attn, cache_of, q8_batch, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,keys,hq,hkv,d", [([1, 1], [700, 2000], 8, 2, 128),  # decode, partials and merge
                                                ([1, 1, 1], [37, 70, 120], 8, 2, 64),  # decode, one split
                                                ([5, 16], [900, 2100], 16, 2, 256),  # tcgen05, partials and merge
                                                ([9, 2], [700, 130], 32, 8, 128),
                                                ([5, 20], [90, 128], 16, 2, 256),  # tcgen05, one split
                                                ([40, 3], [90, 60], 4, 4, 64),
                                                ([3, 5], [200, 333], 24, 2, 128)])  # the general kernel
def test_bf16_rows_are_the_f32_rows_rounded_once(kind, rows, keys, hq, hkv, d):
    """One computation whatever the output's type: the bf16 rows equal the f32 rows rounded to nearest, bit for bit,
    and a call repeats itself."""
    b, _, c = q8_batch(kind, 15, rows=rows, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32)
    wide, flags, st = attn(c, b, kind)
    assert st == 0 and (flags == 0).all()
    want = torch.from_numpy(wide).to(torch.bfloat16).float().numpy()
    for _ in range(3):
        got, _, st = attn(c, b, kind, out_dtype=torch.bfloat16)
        assert st == 0
        assert (got == want).all(), f"{np.mean(got != want):.1%} of the elements differ"
        again, _, _ = attn(c, b, kind)
        assert (again == wide).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hq,hkv,d", [(1, 4, 1, 64), (1, 8, 2, 128), (1, 2, 1, 256),  # decode
                                           (12, 1, 1, 64), (5, 8, 2, 128), (9, 2, 1, 256)])  # tcgen05
@pytest.mark.parametrize("n,split", [(32000, 32000), (32000, 4096), (4000, 4032)])
def test_keys_far_below_one_dominant_key_keep_their_weight(kind, rows, hq, hkv, d, n, split):
    """One key of score 1.625 sqrt(D) and all others of score 0, their values in columns where its own is 0.  In base
    2 the others lie 18.8 (D 64), 26.5 and 37.5 below it; their sum is that column's output.  A weight may be off by
    2^-32 of the largest, so the n of them by n 2^-32, and a weight is else held to 2^-14 of itself.  The matrix
    units' fp32 sums of a column take two additions (hi, lo) every 16 keys, each off by at most a step, 2^-23 of a sum
    that grows evenly from 0 (half of the final one on average): n / 16 * 2 * 2^-23 / 2 = n 2^-27 of it."""
    psz = 64
    b = wl.make_paged_batch(17, rows=[rows], keys=[n], n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=psz,
                            unused="normal")
    k, v = np.zeros(b.k_pool.shape, np.float32), np.zeros(b.v_pool.shape, np.float32)
    v[..., 1], v[..., 2] = 1.0, -0.375
    at = n // 3
    page = b.page_table[b.segs[0][3] + at // psz]
    k[page, :, at % psz] = 1.625
    v[page, :, at % psz] = 0
    v[page, :, at % psz, 0] = 1.0
    sides = [sv.quantise(wl.f32_to_bf16_bits(x), kind) for x in (k, v)]
    b.q = wl.f32_to_bf16_bits(np.ones((rows, hq, d), np.float32))
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    out, flags, st = attn(c, b, kind, split=split, n_splits_max=-(-n // split))
    assert st == 0 and (flags == 0).all()
    small = np.exp(-1.625 * d * b.scale)
    for i in range(rows):
        seen = n - rows + i  # keys the row sees beside the dominant one
        want = np.zeros(d)
        want[:3] = np.array([1.0, seen * small, -0.375 * seen * small]) / (1 + seen * small)
        err = np.abs(out[i].astype(np.float64) - want)
        assert (err <= n * 2.0**-32 + (2.0**-14 + n * 2.0**-27) * np.abs(want)).all(), err.max()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 8, 2), (4, 16, 2)])
def test_value_scales_and_scores_far_from_one(kind, rows, hq, hkv):
    """Values of size 2^-90 and scores near 100: a weight's exponent is a small difference of the two, and carries no
    rounding of their sum.  A score of 100 (in base 2) is itself rounded twice (100 * 2^-23 ln 2 = 2^-16.9 of a
    weight), a weight kept to 22 bits: each head is held to 2^-15 of its own size."""
    b = wl.make_paged_batch(18, rows=[rows], keys=[700], n_q_heads=hq, n_kv_heads=hkv, head_dim=128, page_size=32,
                            unused="normal")
    x = wl.bf16_bits_to_f32(b.v_pool) * np.float32(2.0**-90)
    kk = wl.bf16_bits_to_f32(b.k_pool)
    kk[..., 0] = 24.0
    q = wl.bf16_bits_to_f32(b.q)
    q[..., 0] = 32.0  # 768 / sqrt(128) = 68 nats, 98 in base 2, for every key
    b.q = wl.f32_to_bf16_bits(q)
    sides = [sv.quantise(wl.f32_to_bf16_bits(y), kind) for y in (kk, x)]
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    out, flags, st = attn(c, b, kind)
    assert st == 0 and (flags == 0).all()
    n, base = b.segs[0][2], b.segs[0][3]
    k, v = (sv.values(sv.keys_of(cc, b.page_table, base, n), sv.keys_of(s, b.page_table, base, n), kind) for cc, s in sides)
    ref, _ = sv.attend(sv.bf16(b.q), k, v, [n - rows + i + 1 for i in range(rows)], b.scale)
    err = np.linalg.norm(out - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert err.max() <= 2.0**-15, err.max()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hq,hkv,d,n,split", [(1, 8, 2, 64, 300, 0), (1, 8, 2, 128, 120, 128), (2, 4, 1, 256, 700, 256),  # decode
                                                   (12, 4, 2, 64, 300, 64), (5, 8, 2, 128, 120, 128),  # tcgen05
                                                   (9, 2, 1, 256, 700, 256), (9, 2, 1, 256, 700, 704),
                                                   (3, 24, 2, 64, 300, 64), (3, 24, 2, 256, 300, 320)])  # the general kernel
@pytest.mark.parametrize("size", [2.0**18, 2.0**23, 2.0**26, 2.0**27, 2.0**28, 2.0**31, 2.0**40, 2.0**90, -(2.0**28), -(2.0**35)])
def test_scores_of_any_size(kind, rows, hq, hkv, d, n, split, size):
    """Scores of up to 2^90: two keys share the largest, `size` (or the smallest magnitude of the negative ones), all
    others are 7/8 of it or less (for a negative one, 9/8 of it), 2^15 below even at 2^18, so the two weigh 1/2 each and
    nothing else weighs anything.  Every score is the exact sum of two products (of 20 bits, so that the scale's product
    with it is rounded), the two keys' are the same float, and their value rows differ in scale by 2^12 in columns of
    their own.  So each column is one weight (22 bits, half of a step off, and the floats' ex2, good to 2^-22, twice)
    times one value, over a sum of two: 2^-20 of it."""
    psz = 32
    b = wl.make_paged_batch(19, rows=[rows], keys=[n], n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=psz,
                            unused="normal")
    rng = np.random.default_rng(20)
    sign, mag = np.sign(size), abs(size)
    steps = rng.choice([0.25, 0.5, 0.75, 0.875] if sign > 0 else [1.125, 1.25, 1.5, 1.75], size=n)
    one, two = n // 2 - n // 2 % 64 + 11, n // 2 - n // 2 % 64 + 43  # the two halves of a tile
    steps[[one, two]] = 1.0
    k, v = np.zeros(b.k_pool.shape, np.float32), np.zeros(b.v_pool.shape, np.float32)
    for j in range(n):
        page = b.page_table[b.segs[0][3] + j // psz]
        k[page, :, j % psz, 3:5] = sign * steps[j], sign * 0.8125
        v[page, :, j % psz] = 3.0
    for j, col, x in ((one, 1, 1.75), (two, 2, 1.5 * 2.0**-12)):
        page = b.page_table[b.segs[0][3] + j // psz]
        v[page, :, j % psz] = 0.0
        v[page, :, j % psz, col] = x
    sides = [sv.quantise(wl.f32_to_bf16_bits(x), kind) for x in (k, v)]
    q = np.zeros((rows, hq, d), np.float32)
    q[..., 3] = mag * 2.0 ** -np.floor(np.log2(b.scale))
    q[..., 4] = q[..., 3] * 2.0**-9 * 175 / 128
    b.q = wl.f32_to_bf16_bits(q)
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    out, flags, st = attn(c, b, kind, split=split, n_splits_max=-(-n // split) if split else 16)
    assert st == 0 and (flags == 0).all()
    want = np.zeros(d)
    want[1], want[2] = 1.75 / 2, 1.5 * 2.0**-12 / 2
    assert (np.abs(out.astype(np.float64) - want) <= 2.0**-20 * want).all(), out[0, 0, :4]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 2, 128), (4, 4, 256)])
def test_a_long_decode_sum_is_rounded_not_truncated(kind, hq, hkv, d):
    """All values 1.75 and scores of all sizes: the output is 1.75, from 4,096 weights summed twice (with the values and
    without).  A tile's 16 keys a warp are summed by the matrix unit, which truncates, twice: 2^-22 of them and of the
    whole.  The 64 tiles' sums are rounded, by half a step each way: 8 of 64 roundings' size, 2^-25 sqrt(64) / 2 for
    sums that grow evenly, over four warps' sums halved again, 2^-24 each; six such are 2^-22 with room.  (Truncated,
    64 tiles would lose half a step of the sum so far twice each: 64 2^-24, 2^-18.)"""
    n = 4096
    b = wl.make_paged_batch(21, rows=[1], keys=[n], n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=64,
                            unused="normal")
    sides = [sv.quantise(b.k_pool, kind), sv.quantise(wl.f32_to_bf16_bits(np.full(b.v_pool.shape, 1.75, np.float32)), kind)]
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    out, flags, st = attn(c, b, kind, split=n, n_splits_max=1)
    assert st == 0 and (flags == 0).all()
    err = np.abs(out.astype(np.float64) / 1.75 - 1)
    assert err.max() <= 2.0**-21, err.max()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("scale", [1e-3, 2.0**-29, 2.0**-40, 2.0**-100, 2.0**-126])
@pytest.mark.parametrize("rows,hq,hkv,d,n,split", [(1, 8, 2, 64, 300, 0), (2, 4, 1, 128, 90, 128),  # decode
                                                   (12, 4, 2, 64, 300, 64), (5, 8, 2, 128, 90, 128), (9, 2, 1, 256, 700, 0),
                                                   (70, 4, 2, 128, 300, 0),  # tcgen05
                                                   (3, 24, 2, 128, 300, 320)])  # the general kernel
@pytest.mark.parametrize("size", [0.0, 2.0**-100, 1.0, 2.0**100])
def test_rows_of_zeros_and_small_scales(kind, scale, rows, hq, hkv, d, n, split, size):
    """Every positive scale is taken: scores next to 0 weigh all keys alike, and so does a query of zeros."""
    if size * scale > 1:
        size = 1 / scale  # scores of the usual size
    b, sides, c = q8_batch(kind, 3, rows=[rows], keys=[n], n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32)
    q = wl.bf16_bits_to_f32(b.q) * np.float32(size)
    q[0, 0] = 0
    b.q, b.scale = wl.f32_to_bf16_bits(q), scale
    out, flags, st = attn(c, b, kind, split=split)
    assert st == 0
    ref, fl, vmax = reference(b, sides, kind)
    sv.check_attention(out, flags, ref, fl, vmax, False)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hq,hkv,d,split", [(12, 4, 2, 64, 20032), (9, 8, 2, 128, 4096), (40, 4, 1, 256, 1024),
                                                 (19300, 1, 1, 64, 0)])  # more query tiles than SMs: one wave is one split
def test_what_a_long_partial_loses(kind, rows, hq, hkv, d, split):
    """All values 1.75, scores of all sizes: the output is 1.75.  The tensor unit truncates its sums, twice every 16 keys,
    each time by less than a step, 2^-23, of a sum that grows evenly: n / 16 * 2 * 2^-23 / 2 = n 2^-27 of it for a partial
    of n keys.  Chosen splits have up to 8,192 keys.  The rest is rounded: with room 2^-20."""
    n = 20000
    b = wl.make_paged_batch(22, rows=[rows], keys=[n], n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=64,
                            unused="normal")
    sides = [sv.quantise(b.k_pool, kind), sv.quantise(wl.f32_to_bf16_bits(np.full(b.v_pool.shape, 1.75, np.float32)), kind)]
    c = cache_of(sides[0][0], sides[1][0], sides[0][1], sides[1][1], kind)
    out, flags, st = attn(c, b, kind, split=split, n_splits_max=-(-n // split) if split else 16)
    assert st == 0 and (flags == 0).all()
    err = np.abs(out.astype(np.float64) / 1.75 - 1)
    assert err.max() <= (split or 8192) * 2.0**-27 + 2.0**-20, err.max()
