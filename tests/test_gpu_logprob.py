"""Log probabilities, entropy and alternatives of logit rows on the GPU, against float64."""
import numpy as np
import pytest
import torch

import paged_kv_cache_segment_b200 as tf

import _serving as sv
from _gpu import DEV, status_word

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LOWEST = {"bf16": -3.3895313892515355e38, "f32": -3.4028234663852886e38}


def run(x, tokens, top_k, *, scale=1.0, n_cols=None, stats=True, stream=None):
    n = x.shape[0]
    f = dict(device=DEV, dtype=torch.float32)
    tl = torch.full(tuple(tokens.shape), 3.0, **f)
    ent, lse = torch.full((n,), 3.0, **f), torch.full((n,), 3.0, **f)
    ids = torch.full((n, top_k), -9, device=DEV, dtype=torch.int32)
    tops = torch.full((n, top_k), 3.0, **f)
    fl = torch.full((n,), 9, device=DEV, dtype=torch.uint8)
    st = status_word()
    tf.tf_logprob_rows(x, torch.from_numpy(np.ascontiguousarray(tokens, np.int32)).to(DEV), token_logprobs=tl,
                       entropy=ent if stats else None, lse=lse if stats else None,
                       top_ids=ids if top_k else None, top_logprobs=tops if top_k else None, flags=fl, status=st,
                       scale=scale, n_cols=n_cols, stream=stream)
    return [t.cpu().numpy() for t in (tl, ent, lse, ids, tops, fl)], int(st.item())


def check(got, want, scale, biggest):
    """Ids and flags exactly.  Values: a column's distance from the row's largest is rounded once (2^-24 of it), ex2
    and the scaling by a few 2^-23 of the exponent, fp32 sums of n terms over 512 threads by some 2^-18; against a
    log p of that size the error stays below 2^-20 of (1 + |scale * x| over the row)."""
    names = ("token_logprobs", "entropy", "lse", "top_ids", "top_logprobs", "flags")
    for name, g, w in zip(names, got, want):
        if name in ("top_ids", "flags"):
            assert (g == w).all(), f"{name}: {np.argwhere(g != w)[:4]}"
            continue
        assert (np.isnan(g) == np.isnan(w)).all(), name
        assert ((g == -np.inf) == (w == -np.inf)).all(), name
        ok = np.isfinite(w)
        err = np.abs(g[ok].astype(np.float64) - w[ok])
        # |log p| of a finite column is part of its own bound; the row's size bounds the rest
        assert (err <= 2.0**-18 * (1 + np.abs(w[ok])) + 2.0**-22 * abs(scale) * biggest).all(), \
            f"{name}: {err.max():.3e}"


def check_rows(x, tokens, top_k, scale=1.0, n_cols=None, **kw):
    xs = x[:, :n_cols].double().cpu().numpy()
    fin = np.abs(xs[np.isfinite(xs) & (np.abs(xs) < 1e30)])
    got, st = run(x, tokens, top_k, scale=scale, n_cols=n_cols, **kw)
    check(got, sv.logprobs(xs, scale, tokens, top_k), scale, fin.max() if fin.size else 0.0)
    return got, st


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols,top_k,n_tok", [(1, 1, 1, 1), (3, 2, 32, 2), (5, 7, 3, 1), (2, 31, 31, 0),
                                                   (4, 33, 32, 3), (2, 1000, 0, 1), (7, 4097, 20, 2),
                                                   (1, 50257, 20, 1), (33, 16385, 5, 1), (3, 128000, 20, 4),
                                                   (301, 2500, 1, 1), (700, 300, 8, 1), (3, 9000, 4, 70), (700, 200, 2, 33),
                                                   (700, 700, 32, 1), (800, 3500, 32, 1), (600, 45, 17, 1)])
def test_rows_match_float64(dtype, rows, cols, top_k, n_tok):
    rng = np.random.default_rng(rows * 7 + cols)
    x = torch.from_numpy(rng.normal(0, 3, (rows, cols)).astype(np.float32)).to(DEV).to(DT[dtype])
    tok = rng.integers(0, cols, (rows, n_tok))
    _, st = check_rows(x, tok, top_k)
    assert st == 0
    got, _ = run(x, tok, top_k, stats=False)  # without entropy and lse
    assert (got[1] == 3.0).all() and (got[5] == 0).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shift", range(9))
def test_rows_of_any_alignment_and_stride(dtype, shift):
    """Rows that start anywhere in 16 bytes, strided, with other data around them that must not be read."""
    rng = np.random.default_rng(shift)
    rows, cols, ld = 6, 5003 + shift, 5030 + shift
    wide = torch.full((rows + 1, ld), float("nan"), device=DEV, dtype=DT[dtype])
    wide[:rows, shift : shift + cols] = torch.from_numpy(rng.normal(0, 2, (rows, cols)).astype(np.float32)).to(DEV)
    x = wide[:rows, shift : shift + cols]
    assert x.stride(0) == ld
    check_rows(x, rng.integers(0, cols, (rows, 2)), 7)
    wide[:, :] = float("inf")
    wide[:rows, shift : shift + cols - 3] = torch.from_numpy(rng.normal(0, 2, (rows, cols - 3)).astype(np.float32)).to(DEV)
    check_rows(x, rng.integers(0, cols - 3, (rows, 1)), 3, n_cols=cols - 3)


def test_more_rows_than_the_grid_and_one_column_rows():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.normal(0, 3, (5000, 77)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    check_rows(x, rng.integers(0, 77, (5000, 1)), 4)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("cols,top_k", [(40, 8), (20000, 32), (130000, 20)])
def test_masks_ties_and_nonfinite_rows(dtype, cols, top_k):
    rng = np.random.default_rng(cols)
    inf = float("inf")
    x = torch.from_numpy(rng.normal(0, 2, (13, cols)).astype(np.float32)).to(DEV).to(DT[dtype])
    x[0] = 0.25  # every column the same
    x[1] = torch.arange(cols, device=DEV).to(torch.float32) / 64  # ascending
    x[2] = -torch.arange(cols, device=DEV).to(torch.float32) / 64
    x[3] = -inf  # all masked
    x[4] = -inf
    x[4, cols - 2] = 1.5  # one column left
    x[5, 5:] = -inf  # fewer left than alternatives asked for
    x[6, 3:] = LOWEST[dtype]  # the type's lowest value as a mask
    x[7, cols // 2] = float("nan")
    x[8, cols - 1] = inf
    x[9] = -inf
    x[9, cols // 3] = float("nan")  # a NaN among masked columns only
    x[10, torch.from_numpy(rng.random(cols) < 0.9).to(DEV)] = -inf
    x[11] = torch.where(torch.arange(cols, device=DEV) % 2 == 0, 0.0, -0.0)  # -0 equals +0
    x[12] = torch.from_numpy(rng.integers(0, 3, cols).astype(np.float32)).to(DEV)
    tok = rng.integers(0, cols, (13, 3))
    tok[4] = [cols - 2, 0, cols - 1]
    tok[5] = [0, 4, cols - 1]
    _, st = check_rows(x, tok, top_k)
    assert st == 0


@pytest.mark.parametrize("dtype", DT)
def test_masks_that_leave_whole_half_warps_empty(dtype):
    """Columns left only where a few threads of one warp look, so the other half-warps never see a logit and the
    candidates overflow their list: the exact search takes over."""
    rng = np.random.default_rng(4)
    per = 8 if dtype == "bf16" else 4
    cols = 130000
    x = torch.from_numpy(rng.normal(0, 2, (3, cols)).astype(np.float32)).to(DEV).to(DT[dtype])
    lane = (torch.arange(cols, device=DEV) // per) % 512
    x[0, lane >= 40] = -float("inf")
    x[1, lane >= 300] = -float("inf")
    x[1] = torch.where(torch.isinf(x[1]), x[1], torch.arange(cols, device=DEV).to(x.dtype))
    x[2, lane < 500] = -float("inf")
    check_rows(x, rng.integers(0, cols, (3, 1)), 32)


@pytest.mark.parametrize("scale", [2.0**-64, 0.01, 0.7, 5.0, 2.0**20])
def test_temperatures(scale):
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(0, 3, (4, 3001)).astype(np.float32)).to(DEV)
    x[1, 7:] = -float("inf")
    x[2] *= 1000
    check_rows(x, rng.integers(0, 7, (4, 2)), 5, scale=scale)


def test_tokens_out_of_range_and_the_same_token_twice():
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.normal(0, 3, (3, 500)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    got, st = check_rows(x, np.array([[0, -1], [500, 499], [3, 3]]), 2)
    assert st == 32
    assert np.isnan(got[0][0, 1]) and np.isnan(got[0][1, 0]) and got[0][2, 0] == got[0][2, 1]


def test_captured_replayed_another_stream_and_repeated():
    rng = np.random.default_rng(3)
    for rows in (1, 40, 400):
        x = torch.from_numpy(rng.normal(0, 3, (rows, 40001)).astype(np.float32)).to(DEV).to(torch.bfloat16)
        tok = rng.integers(0, 40001, (rows, 1))
        first, _ = run(x, tok, 20)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other, _ = run(x, tok, 20)
        for a, b in zip(first, other):
            assert (a == b).all()
        dtok = torch.from_numpy(tok.astype(np.int32)).to(DEV)
        tl, ids = torch.zeros((rows, 1), device=DEV), torch.zeros((rows, 20), device=DEV, dtype=torch.int32)
        tops, fl, st = torch.zeros((rows, 20), device=DEV), torch.zeros(rows, device=DEV, dtype=torch.uint8), status_word()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tf.tf_logprob_rows(x, dtok, token_logprobs=tl, top_ids=ids, top_logprobs=tops, flags=fl, status=st)
        for _ in range(3):
            tl.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert (tl.cpu().numpy() == first[0]).all() and (ids.cpu().numpy() == first[3]).all()


def test_the_first_alternative_is_the_argmax():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.normal(0, 3, (62, 128000)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    got, _ = run(x, np.zeros((62, 0)), 1)
    ids, fl = torch.empty(62, device=DEV, dtype=torch.int32), torch.empty(62, device=DEV, dtype=torch.uint8)
    tf.tf_argmax_rows(x, ids, fl)
    assert (ids.cpu().numpy() == got[3][:, 0]).all()


HIGHEST = {k: -v for k, v in LOWEST.items()}


def of_large_logits(x, tok, top_k):
    """sv.logprobs (scale 1) where logits are as large as the type's ends: log p from x - m, since log n is lost next
    to 2^127; the order from x itself, since ordinary logits are lost in x - m; in the outputs' type, since lowest -
    highest, -2^129 (1 - 2^-8) or less, is below its floats: -infinity."""
    xs = x.double().cpu().numpy()
    m = xs.max(1)
    m = np.where(np.isfinite(m), m, 0.0)
    want = list(sv.logprobs(xs - m[:, None], 1.0, tok, top_k))
    want[2] = want[2] + m
    want[3] = sv.logprobs(xs, 1.0, tok, top_k)[3]
    with np.errstate(over="ignore"):
        return [w.astype(np.float32) if w.dtype == np.float64 else w for w in want]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols,top_k", [(8, 40, 8), (8, 3001, 0), (8, 20000, 5), (8, 130000, 20),  # a CTA, a cluster
                                             (640, 300, 4), (640, 3500, 32)])  # a warp a row
def test_rows_whose_largest_logit_is_the_types_highest(dtype, rows, cols, top_k):
    """A token forced with the type's highest value: the others weigh nothing, so the entropy is 0 and not NaN,
    whatever they are (masked, the lowest value, ordinary) and wherever the row's own padding lies."""
    rng = np.random.default_rng(cols)
    hi, lo, inf = HIGHEST[dtype], LOWEST[dtype], float("inf")
    x = torch.from_numpy(rng.normal(0, 2, (rows, cols)).astype(np.float32)).to(DEV).to(DT[dtype])
    at = rng.integers(0, cols, rows)
    for r in range(0, rows, 8):
        x[r + 1] = -inf
        x[r + 2] = lo
        x[r + 3, cols // 2 :] = -inf
        x[r + 4, ::3] = lo
    x[torch.arange(rows, device=DEV), torch.from_numpy(at).to(DEV)] = hi
    x[5::8, 0] = hi  # twice (unless it is the same column)
    x[6::8] = hi / 4 * 3  # below the border of the plain form's own rule, every column the same
    x[7::8] = -inf
    x[7::8, cols - 1] = 2.0**127
    tok = np.stack([at, rng.integers(0, cols, rows)], 1)
    got, st = run(x, tok, top_k)
    check(got, of_large_logits(x, tok, top_k), 1.0, 8.0)
    assert st == 0 and (got[5] == 0).all() and np.isfinite(got[1]).all()
    assert (got[1][0::8] == 0).all() and (got[1][1::8] == 0).all() and (got[1][2::8] == 0).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("cols", [300, 512, 700, 3500])
@pytest.mark.parametrize("top_k", [8, 24, 25, 32])
def test_short_rows_with_masks_and_ties(dtype, cols, top_k):
    """Many short rows, a warp each: masks that leave a few lanes, equal columns, the lowest value as a mask, rows of
    few distinct values; their lists overflow, and the search by ties and the one key by key take over."""
    rng = np.random.default_rng(cols + top_k)
    per, inf = (8 if dtype == "bf16" else 4), float("inf")
    x = torch.from_numpy(rng.normal(0, 2, (640, cols)).astype(np.float32)).to(DEV).to(DT[dtype])
    col = torch.arange(cols, device=DEV)
    lane = (col // per) % 32
    x[0::16] = 0.25
    x[1::16, lane >= 3] = -inf
    x[2::16, lane >= 20] = -inf
    x[3::16, lane >= 31] = LOWEST[dtype]
    x[4::16] = LOWEST[dtype]
    x[5::16] = col.to(x.dtype)  # ascending (ties where bf16 cannot tell columns apart)
    x[6::16] = -inf
    x[7::16, 5:] = LOWEST[dtype]
    x[8::16] = torch.from_numpy(rng.integers(0, 3, (40, cols)).astype(np.float32)).to(DEV).to(x.dtype)
    x[9::16] = torch.where(lane == 7, 3.0, -1.0).to(x.dtype)
    x[10::16, : cols // 2] = -inf
    x[11::16, cols // 2 :] = 1.0
    x[12::16, cols // 3] = float("nan")
    tok = rng.integers(0, cols, (640, 2))
    got, st = run(x, tok, top_k)
    check(got, of_large_logits(x, tok, top_k), 1.0, 8.0)
    assert st == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", [(2, 40), (2, 130000), (640, 700)])
def test_a_cold_row_of_logits_from_end_to_end(dtype, rows, cols):
    """Logits over the type's whole range under a scale of 2^-10 or 2^-64: the distance from the largest is past the
    floats, the log p is not.  A scaled distance is rounded twice: 2^-23 of the log p."""
    hi, lo = HIGHEST[dtype], LOWEST[dtype]
    x = torch.full((rows, cols), lo, device=DEV, dtype=DT[dtype])
    x[:, 1], x[:, 3], x[:, 5], x[:, 7] = hi, hi / 2, 0.0, -float("inf")
    tok = np.tile(np.array([[0, 1, 3, 5, 7]]), (rows, 1))
    xs = x[0].double().cpu().numpy()
    for scale in (2.0**-10, 2.0**-64):
        got, st = run(x, tok, 4, scale=scale)
        want = (xs[[0, 1, 3, 5, 7]] - xs[1]) * scale
        assert st == 0 and (got[5] == 0).all() and (got[1] == 0).all()
        assert (got[3] == [1, 3, 5, 0]).all()
        for g, w in ((got[0], want), (got[4], want[[1, 2, 3, 0]])):
            assert (np.isneginf(g) == np.isneginf(w)).all()
            ok = np.isfinite(w)
            assert (np.abs(g[:, ok] - w[ok]) <= 2.0**-23 * np.abs(w[ok])).all()


def test_alternatives_need_both_of_their_outputs():
    x = torch.zeros((2, 10), device=DEV)
    tok = torch.zeros((2, 1), device=DEV, dtype=torch.int32)
    kw = dict(token_logprobs=torch.empty((2, 1), device=DEV), flags=torch.empty(2, device=DEV, dtype=torch.uint8),
              status=status_word())
    with pytest.raises(ValueError, match="both or neither"):
        tf.tf_logprob_rows(x, tok, top_logprobs=torch.empty((2, 3), device=DEV), **kw)
    with pytest.raises(ValueError, match="both or neither"):
        tf.tf_logprob_rows(x, tok, top_ids=torch.empty((2, 3), device=DEV, dtype=torch.int32), **kw)
