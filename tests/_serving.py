"""Plain float64 forms of the serving operators for the tests: the 8-bit
format, attention over given keys, log probabilities of logit rows."""
from __future__ import annotations

import numpy as np

from paged_kv_cache_segment_b200 import workloads as wl

Q_MAX = {"e4m3": 448.0, "int8": 127.0}


def bf16(bits) -> np.ndarray:
    return wl.bf16_bits_to_f32(np.asarray(bits, np.uint16)).astype(np.float64)


def e4m3_values() -> np.ndarray:
    """The value of each e4m3 byte (NaN for 0x7f, 0xff)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0**-6, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b > 127, -v, v)


def code_values(codes: np.ndarray, kind: str) -> np.ndarray:
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else e4m3_values()[codes]


def quantise(bits: np.ndarray, kind: str):
    """(codes, scale bytes) of bf16 rows [..., D] from the format's definition."""
    x = bf16(bits)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(-1)
    with np.errstate(divide="ignore"):
        k = np.ceil(np.log2(amax / Q_MAX[kind]))  # to be put right by a step where log2 rounds
    k = np.maximum(np.where(np.isfinite(k), k, -100), -100).astype(np.int64)
    k = np.where(amax > Q_MAX[kind] * 2.0**k, k + 1, k)
    k = np.where((k > -100) & (amax <= Q_MAX[kind] * 2.0 ** (k - 1)), k - 1, k)
    y = x * (2.0 ** -k.astype(np.float64))[..., None]
    if kind == "int8":
        codes = np.rint(y).astype(np.int64).astype(np.int8).view(np.uint8)
    else:  # eight steps a binade; below 2^-6 the subnormals' step
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0**-6))) - 3)
        val = np.rint(y / step) * step
        table = e4m3_values()[:127]
        codes = np.searchsorted(table, np.abs(val)).astype(np.uint8)
        assert (table[codes] == np.abs(val)).all()
        codes = np.where(np.signbit(x), codes | 128, codes).astype(np.uint8)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes, np.where(bad, 255, k + 127).astype(np.uint8)


def values(codes: np.ndarray, scale: np.ndarray, kind: str) -> np.ndarray:
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return code_values(codes, kind) * s[..., None]


def keys_of(pool: np.ndarray, page_table, pt_base: int, n: int) -> np.ndarray:
    """Keys [n][Hkv][D] of a stream from pages [pages][Hkv][P][D]."""
    p = pool.shape[2]
    j = np.arange(n)
    return pool[np.asarray(page_table)[pt_base + j // p], :, j % p]


def attend(q, k, v, lims, scale):
    """(out, flags) of rows q [T][Hq][D] over k, v [N][Hkv][D], row i seeing the first lims[i] keys: float64."""
    t, hq, d = q.shape
    g = hq // k.shape[1]
    out = np.full((t, hq, d), np.nan)
    flags = np.ones((t, hq), np.uint8)
    for i in range(t):
        for h in range(hq):
            kk, vv = k[: lims[i], h // g], v[: lims[i], h // g]
            if not (np.isfinite(q[i, h]).all() and np.isfinite(kk).all() and np.isfinite(vv).all()) or lims[i] == 0:
                continue
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            out[i, h] = p @ vv / p.sum()
            flags[i, h] = 0
    return out, flags


def check_attention(out, flags, ref, ref_flags, vmax, is_bf16, what=""):
    """fp32 output: a weight is fed to the value product with at least 16 bits (2^-17 of it, the weights sum to 1),
    a score of up to 40 in base 2 is rounded a few times (4 * 40 * 2^-24 = 2^-16.7 of a weight) and ex2 is good to
    2^-22: |error| <= 2^-14 max |V| with room for the fp32 sums.  bf16 output: a weight may be fed as one f16 (half a
    step, 2^-11 of it, so 2^-11 max |V| over weights that sum to 1), and the output is rounded: 2^-8 of the value."""
    assert (flags == ref_flags).all(), f"{what}: flags differ at {np.argwhere(flags != ref_flags)[:4]}"
    ok = ref_flags == 0
    assert np.isnan(out[~ok]).all(), f"{what}: a flagged head is not NaN"
    err = np.abs(out[ok].astype(np.float64) - ref[ok])
    bound = 2.0**-14 * vmax + (2.0**-11 * vmax + 2.0**-8 * np.abs(ref[ok]) if is_bf16 else 0.0)
    assert (err <= bound).all(), f"{what}: off by {(err - bound).max():.3e} more than the bound"


def logprobs(x: np.ndarray, scale: float, tokens: np.ndarray, top_k: int):
    """(token log p, entropy, lse, top ids, top log p, flags) of rows x (float64, -inf masked)."""
    n, c = x.shape
    tl, ent, lse = np.full(tokens.shape, np.nan), np.full(n, np.nan), np.full(n, np.nan)
    ids, tops, flags = np.full((n, top_k), -1, np.int32), np.full((n, top_k), np.nan), np.ones(n, np.uint8)
    for r in range(n):
        if np.isnan(x[r]).any() or (x[r] == np.inf).any() or (x[r] == -np.inf).all():
            continue
        flags[r] = 0
        y = x[r] * scale
        m = y.max()
        e = np.exp(y - m)
        lse[r] = m + np.log(e.sum())
        lp = y - lse[r]
        p = e / e.sum()
        live = p > 0
        ent[r] = -(p[live] * lp[live]).sum()
        for i, tok in enumerate(tokens[r]):
            if 0 <= tok < c:
                tl[r, i] = lp[tok]
        order = np.lexsort((np.arange(c), -x[r]))[:top_k]
        order = order[x[r][order] > -np.inf]
        ids[r, : len(order)] = order
        tops[r] = -np.inf
        tops[r, : len(order)] = lp[order]
    return tl, ent, lse, ids, tops, flags
