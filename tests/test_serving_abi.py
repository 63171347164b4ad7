"""include/tfserve.h on the CPU: every declared call is exported and bound,
host tensors are refused, and bad arguments are answered without a GPU."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_cache_segment_b200 as tf
from paged_kv_cache_segment_b200 import serving

import _serving as sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every case below fails a host check first
ODD = 0x10008


def host(a):
    return a.ctypes.data


def test_header_library_and_binding_agree():
    src = open(os.path.join(ROOT, "include", "tfserve.h")).read()
    names = set(re.findall(r"TFS_API\s+[\w\s\*]+?\b(tf_\w+)\s*\(", src))
    assert names == set(tf.SERVE_EXPORTS)
    lib = serving.load()
    for n in names:
        assert hasattr(lib, n) and hasattr(tf, n)


def cache(**kw):
    a = dict(k_codes=FAKE, v_codes=FAKE, k_scale=FAKE, v_scale=FAKE, kv_type=1, n_pages=16, page_size=16,
             n_kv_heads=2, head_dim=64)
    a.update(kw)
    s = serving._CacheStruct(*a.values())
    s._keep = s
    return s


def call(name, defaults, **kw):
    c = kw.pop("cache", None)
    a = dict(defaults, **kw)
    if "cache" in a and a["cache"] is not None:
        c = c or cache(**kw.pop("cache_kw", {}))
        a["cache"] = ctypes.addressof(c)
    a.pop("cache_kw", None)
    return getattr(serving.load(), name)(*a.values())


SEGS = np.array([[0, 1, 37, 0, 3], [1, 1, 70, 3, 5]], np.int32)
APPEND = dict(k=FAKE, v=FAKE, rows=2, cache=1, pt=FAKE, pt_len=8, segs=FAKE, n_segs=2, segs_host=None, pt_host=None,
              st=FAKE, stream=None)
READ = dict(cache=1, pt=FAKE, pt_len=8, segs=FAKE, n_segs=2, segs_host=None, pt_host=None, k=FAKE, v=FAKE, n_dst=8,
            dst=FAKE, dst_host=None, st=FAKE, stream=None)
ATTN = dict(q=FAKE, rows=2, hq=8, cache=1, pt=FAKE, pt_len=8, segs=FAKE, n_segs=2, segs_host=None, pt_host=None,
            scale=0.125, full=0, split=0, nsm=4, ws=FAKE, ws_bytes=1 << 30, out=FAKE, dt=0, flags=FAKE, st=FAKE,
            stream=None)
SHARED = dict(q=FAKE, rows=2, hq=8, k=FAKE, v=FAKE, n_pages=16, psz=16, hkv=2, d=64, pt=FAKE, pt_len=8, pre=FAKE,
              n_pre=1, pre_host=None, segs=FAKE, n_segs=2, segs_host=None, pt_host=None, scale=0.125, split=0, npre=4,
              nsm=4, ws=FAKE, ws_bytes=1 << 30, out=FAKE, dt=0, flags=FAKE, st=FAKE, stream=None)
LOGPROB = dict(x=FAKE, dt=1, rows=4, cols=100, ld=100, scale=1.0, tok=FAKE, n_tok=1, tl=FAKE, ent=None, lse=None, k=2,
               ids=FAKE, tops=FAKE, flags=FAKE, st=FAKE, stream=None)


def append(**kw):
    return call("tf_kv_append_q8", APPEND, **kw)


def read(**kw):
    return call("tf_kv_read_q8", READ, **kw)


def attn(**kw):
    return call("tf_paged_attn_q8", ATTN, **kw)


def shared(**kw):
    return call("tf_paged_attn_shared", SHARED, **kw)


def logprob(**kw):
    return call("tf_logprob_rows", LOGPROB, **kw)


@pytest.mark.parametrize("f", [append, read, attn])
def test_cache_checks(f):
    for kw, want in ((dict(kv_type=0), 1), (dict(kv_type=3), 1), (dict(head_dim=96), 4), (dict(page_size=24), 4),
                     (dict(page_size=4), 4), (dict(page_size=2048), 4), (dict(n_kv_heads=0), 1), (dict(n_pages=-1), 1),
                     (dict(k_codes=None), 1), (dict(v_scale=None), 1), (dict(v_codes=ODD), 6), (dict(k_scale=ODD), 6)):
        assert f(cache=cache(**kw)) == want, kw
    assert f(n_segs=0) == 0
    assert f(segs=None) == 1 and f(pt=None) == 1 and f(st=None) == 1
    assert f(n_segs=-1) == 1 and f(pt_len=-1) == 1 and f(n_segs=65536) == 4


@pytest.mark.parametrize("f", [append, read, attn, shared])
def test_host_table_checks(f):
    def seg(*rows):
        return np.array(rows, np.int32)

    past, page = SEGS.copy(), np.arange(8, dtype=np.int32)
    past[0, 2] = 49  # three pages of 16 hold 48 keys
    assert f(segs_host=host(past)) == 2
    page[4] = 16
    assert f(segs_host=host(SEGS), pt_host=host(page)) == 3
    page[4] = -1
    assert f(segs_host=host(SEGS), pt_host=host(page)) == 3
    for bad in (seg([0, 3, 2, 0, 3], [1, 1, 70, 3, 5]), seg([0, 1, 37, 6, 3], [1, 1, 70, 3, 5]),
                seg([0, 1, 37, -1, 3], [1, 1, 70, 3, 5]), seg([0, -1, 37, 0, 3], [1, 1, 70, 3, 5])):
        assert f(segs_host=host(bad)) == 1
    none = SEGS.copy()
    none[:, 1] = 0
    assert f(segs_host=host(none)) == 0  # no rows: nothing to do
    if f is not read:  # a read does not use q_row
        assert f(segs_host=host(seg([2, 1, 37, 0, 3], [1, 1, 70, 3, 5]))) == 1
    else:
        dst = np.arange(8, dtype=np.int32)
        dst[2] = 8
        assert f(segs_host=host(SEGS), dst_host=host(dst)) == 3


def test_attention_checks():
    for f in (attn, shared):
        assert f(hq=7) == 4 and f(scale=float("nan")) == 1 and f(nsm=0) == 1 and f(split=-1) == 1 and f(split=8) == 4
        assert f(q=ODD) == 6 and f(out=ODD) == 6 and f(ws=ODD) == 6 and f(ws_bytes=1000) == 7 and f(dt=2) == 1
        assert f(q=None) == 1 and f(flags=None) == 1 and f(ws=None) == 1 and f(out=None) == 1
        assert f(segs_host=host(SEGS), split=16, nsm=4) == 1  # 70 keys need five partials
        assert f(rows=0) == 0
    n = tf.tf_paged_attn_q8_workspace_bytes(2, 8, 64, 4)
    assert n >= 2 * 8 * 4 * (64 * 4 + 9) and attn(ws_bytes=n - 1) == 7
    assert tf.tf_paged_attn_q8_workspace_bytes(2, 8, 64, 0) == 0
    n = tf.tf_paged_attn_shared_workspace_bytes(2, 8, 64, 3, 4)
    assert n >= 2 * 8 * 7 * (64 * 4 + 9) and shared(ws_bytes=n - 1, npre=3) == 7
    assert tf.tf_paged_attn_shared_workspace_bytes(2, 8, 64, 0, 4) == 0
    assert attn(full=1, segs_host=host(np.array([[0, 2, 0, 0, 3], [1, 0, 0, 3, 5]], np.int32))) == 1


def test_lengths_and_workspaces_past_their_limits():
    """2^30 keys a stream or prefix; sizes whose products pass 64 bits."""
    long = np.array([[0, 1, 37, 0, 3], [1, 1, 2**31 - 1, 3, 1 << 21]], np.int32)
    over = np.array([[0, 1, 37, 0, 3], [1, 1, 2**30 + 1, 3, 1 << 21]], np.int32)
    big = dict(pt_len=(1 << 21) + 3)
    for table in (long, over):
        for split, nsm in ((0, 4), (1 << 30, 4), (0, 1)):
            kw = dict(big, split=split, nsm=nsm)
            assert attn(segs_host=host(table), cache_kw=dict(page_size=1024), **kw) == 4
            assert shared(segs_host=host(table), psz=1024, **kw) == 4
            assert shared(pre_host=host(table), n_pre=2, segs_host=host(SEGS), psz=1024, **kw) == 4
    most = 2**31 - 1
    for n in (most, 1 << 24):
        assert tf.tf_paged_attn_q8_workspace_bytes(most, 1 << 20, 256, n) == 0
        assert tf.tf_paged_attn_shared_workspace_bytes(most, 1 << 20, 256, n, 1) == 0
        assert tf.tf_paged_attn_shared_workspace_bytes(most, 1 << 20, 256, 1, n) == 0
    assert tf.tf_paged_attn_q8_workspace_bytes(1 << 20, 64, 256, 64) == (1 << 32) * (256 * 4 + 9)
    # 2^16 rows x 2^20 heads x 2^24 partials: 2^60 partials, whose bytes were taken modulo 2^64
    assert attn(rows=1 << 16, hq=1 << 20, nsm=1 << 24, cache_kw=dict(head_dim=256)) == 7
    assert shared(rows=1 << 16, hq=1 << 20, nsm=1 << 24, d=256) == 7


def test_shared_prefix_checks():
    pre = np.array([[0, 2, 40, 0, 3]], np.int32)
    ok = dict(segs_host=host(SEGS))
    for bad, want in (([[0, 2, 0, 0, 3]], 1), ([[0, 2, 49, 0, 3]], 2), ([[0, 3, 40, 0, 3]], 1), ([[-1, 2, 40, 0, 3]], 1)):
        b = np.array(bad, np.int32)
        assert shared(pre_host=host(b), **ok) == want
    two = np.array([[0, 2, 40, 0, 3], [1, 1, 8, 3, 1]], np.int32)  # row 1 behind two prefixes
    assert shared(pre_host=host(two), n_pre=2, **ok) == 1
    assert shared(pre=None) == 1 and shared(npre=0) == 1 and shared(n_pre=-1) == 1 and shared(n_pre=65536) == 4
    assert shared(pre_host=host(pre), split=16, npre=2, **ok) == 1  # 40 keys need three partials
    assert shared(d=96) == 4 and shared(psz=24) == 4 and shared(k=ODD) == 6


def test_prefixes_in_any_order_must_not_share_a_row():
    none = SEGS.copy()
    none[:, 1] = 0  # no stream has rows: a table that is taken launches nothing
    for runs, want in (([(3, 2), (0, 3), (5, 1)], 0), ([(3, 2), (0, 4), (5, 1)], 1), ([(0, 6), (2, 0)], 0),
                       ([(5, 1), (2, 2), (0, 6)], 1), ([(4, 1), (4, 1)], 1), ([(0, 0), (0, 0)], 0)):
        pre = np.array([[q, r, 40, 0, 3] for q, r in runs], np.int32)
        assert shared(rows=6, pre_host=host(pre), n_pre=len(runs), segs_host=host(none)) == want, runs


def test_logprob_checks():
    assert logprob(rows=0) == 0
    assert logprob(rows=-1) == 1 and logprob(cols=0) == 1 and logprob(ld=99) == 1 and logprob(dt=2) == 1
    assert logprob(scale=0.0) == 1 and logprob(scale=-1.0) == 1 and logprob(scale=float("nan")) == 1
    assert logprob(scale=float("inf")) == 1 and logprob(scale=1e-30) == 1 and logprob(scale=1e30) == 1
    assert logprob(k=33) == 4 and logprob(k=-1) == 1 and logprob(cols=(1 << 24) + 1, ld=1 << 25) == 4
    assert logprob(x=None) == 1 and logprob(tok=None) == 1 and logprob(tl=None) == 1 and logprob(flags=None) == 1
    assert logprob(ids=None) == 1 and logprob(tops=None) == 1 and logprob(st=None) == 1
    assert logprob(x=0x10001) == 6 and logprob(x=0x10002, dt=0) == 6


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def fake_cache():
    """A cache object whose struct is never read: the calls refuse the host tensors beside it."""
    c = object.__new__(tf.Q8Cache)
    c.n_pages, c.n_kv_heads, c.page_size, c.head_dim, c.kv_type = 2, 2, 16, 64, 1
    c.struct = cache()
    c.address, c.device = ctypes.addressof(c.struct), 0
    c.here = lambda: c.address
    return c


OUTS = dict(scale=0.125, workspace=u8(4096), out=torch.zeros(1, 8, 64), flags=u8(1, 8), status=i32(1))
CALLS = {
    "Q8Cache": lambda: tf.Q8Cache(torch.zeros(2, 2, 16, 64, dtype=torch.int8), torch.zeros(2, 2, 16, 64, dtype=torch.int8),
                                  u8(2, 2, 16), u8(2, 2, 16)),
    "tf_kv_append_q8": lambda: tf.tf_kv_append_q8(bf(1, 2, 64), bf(1, 2, 64), fake_cache(), i32(2), i32(1, 5),
                                                  status=i32(1)),
    "tf_kv_read_q8": lambda: tf.tf_kv_read_q8(fake_cache(), i32(2), i32(1, 5), bf(2, 2, 16, 64), bf(2, 2, 16, 64),
                                              i32(2), status=i32(1)),
    "tf_paged_attn_q8": lambda: tf.tf_paged_attn_q8(bf(1, 8, 64), fake_cache(), i32(2), i32(1, 5), n_splits_max=1,
                                                    **OUTS),
    "tf_paged_attn_shared": lambda: tf.tf_paged_attn_shared(bf(1, 8, 64), bf(2, 2, 16, 64), bf(2, 2, 16, 64), i32(2),
                                                            i32(1, 5), i32(1, 5), n_prefix_splits=1, n_splits_max=1,
                                                            **OUTS),
    "tf_logprob_rows": lambda: tf.tf_logprob_rows(bf(2, 100), i32(2, 1), token_logprobs=torch.zeros(2, 1), flags=u8(2),
                                                  status=i32(1)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="CUDA device"):
        CALLS[name]()


def test_every_compute_call_is_covered():
    assert {n for n in tf.SERVE_EXPORTS if not n.endswith("_bytes")} == set(CALLS) - {"Q8Cache"}


def test_shapes_the_binding_refuses():
    c8 = torch.zeros(2, 2, 16, 64, dtype=torch.int8)
    with pytest.raises(TypeError):
        tf.Q8Cache(c8.view(torch.uint8), c8.view(torch.uint8), u8(2, 2, 16), u8(2, 2, 16))
    with pytest.raises(ValueError):
        tf.Q8Cache(c8, c8, u8(2, 2, 8), u8(2, 2, 16))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_the_formats_definition_against_torch(kind):
    """The tests' own quantiser against torch's conversions, over random rows and every code."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((500, 64)) * np.exp(rng.normal(0, 8, (500, 1)))).astype(np.float32)
    t = torch.from_numpy(x).to(torch.bfloat16)
    codes, scale = sv.quantise(t.view(torch.int16).numpy().view(np.uint16), kind)
    y = t.double() * torch.from_numpy(2.0 ** (127 - scale.astype(np.float64)))[:, None]
    want = (y.float().to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3"
            else torch.round(y).to(torch.int8).view(torch.uint8)).numpy()
    assert (codes == want).all()
    top = sv.Q_MAX[kind]
    amax = y.abs().amax(1)
    assert (amax <= top).all() and (amax > top / 2).all()
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert ((sv.e4m3_values() == every) | np.isnan(every)).all()
