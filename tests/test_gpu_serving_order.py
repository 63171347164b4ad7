"""The order of calls on one stream: what a call reads and writes is done with before later work changes or reads it,
also across a prompt chunk, which may start while the call before it finishes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_segment_b200 as tf
from paged_kv_cache_segment_b200 import workloads as wl

from _gpu import DEV, dev, status_word
from test_gpu_q8 import q8_batch

pytestmark = pytest.mark.gpu


class Chunk:
    """One row over a few keys of a pool of its own: the shortest prompt chunk."""

    def __init__(self, d=128):
        b = wl.make_paged_batch(3, rows=[1], keys=[5], n_q_heads=2, n_kv_heads=1, head_dim=d, page_size=16)
        self.args = tuple(dev(x) for x in (b.q, b.k_pool, b.v_pool, b.page_table))
        self.seg, self.scale = b.segs[0], b.scale
        self.out, self.st = torch.empty(b.q.shape, device=DEV), status_word()

    def __call__(self):
        tf.tf_paged_attn_prompt(*self.args, self.seg, scale=self.scale, out=self.out, status=self.st)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,hq,hkv,d", [(1, 8, 2, 128), (1, 4, 1, 64), (12, 16, 2, 256), (40, 4, 4, 64)])
@pytest.mark.parametrize("graph", [False, True])
def test_a_prompt_chunk_behind_a_one_split_call(kind, rows, hq, hkv, d, graph):
    """Attention in one split (rows written without a merge), a prompt chunk, then the cache's rows overwritten and the
    outputs copied: the copy holds the attention of the cache as it was."""
    keys = [3000, 1700, 2900]
    b, _, c = q8_batch(kind, 5, rows=[rows] * 3, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32)
    n = b.q.shape[0]
    ws = torch.empty(tf.tf_paged_attn_q8_workspace_bytes(n, hq, d, 1), dtype=torch.uint8, device=DEV)
    out, fl, st = torch.empty((n, hq, d), device=DEV), torch.empty((n, hq), dtype=torch.uint8, device=DEV), status_word()
    q, pt, sg = dev(b.q), dev(b.page_table), dev(b.segs)
    keep = [t.view(torch.uint8).clone() for t in c.tensors]
    chunk, copy = Chunk(), torch.empty_like(out)

    def attend():
        tf.tf_paged_attn_q8(q, c, pt, sg, scale=b.scale, n_splits_max=1, workspace=ws, out=out, flags=fl, status=st,
                            segs_host=b.segs)

    def round_():
        for t, was in zip(c.tensors, keep):
            t.view(torch.uint8).copy_(was)
        out.zero_()
        attend()
        chunk()
        copy.copy_(out)
        for t in c.tensors:
            t.view(torch.uint8).zero_()

    attend()
    torch.cuda.synchronize()
    want, first = out.clone(), None
    assert int(st.item()) == 0 and int(fl.sum()) == 0
    run = round_
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            round_()
        run = g.replay
    for _ in range(10):
        run()
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
        first = chunk.out.clone() if first is None else first
        assert torch.equal(chunk.out, first)
    assert int(st.item()) == 0 and int(chunk.st.item()) == 0


@pytest.mark.parametrize("rows,hq,hkv,d,keys", [(1, 32, 8, 128, [6000, 1000]), (12, 16, 2, 256, [3000, 2000]),
                                                (3, 6, 1, 64, [900, 300])])
def test_a_prompt_chunk_between_partials_and_their_merge(rows, hq, hkv, d, keys):
    """Decode partials, a prompt chunk, the merge, two more chunks, then the pools overwritten and the outputs copied:
    the merge and the copy see what they would see without the chunks."""
    b = wl.make_paged_batch(6, rows=[rows] * 2, keys=keys, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=32,
                            split_keys=512, n_splits_max=12)
    n, c = b.q.shape[0], 12
    f = dict(device=DEV, dtype=torch.float32)
    po, pm, pl = torch.empty((n, hq, c, d), **f), torch.empty((n, hq, c), **f), torch.empty((n, hq, c), **f)
    pf = torch.empty((n, hq, c), dtype=torch.uint8, device=DEV)
    out, fl, st = torch.empty((n, hq, d), **f), torch.empty((n, hq), dtype=torch.uint8, device=DEV), status_word()
    q, pt, sg, pools = dev(b.q), dev(b.page_table), dev(b.segs), [dev(b.k_pool), dev(b.v_pool)]
    keep = [x.clone() for x in pools]
    chunk, copy = Chunk(d), torch.empty_like(out)

    def partials():
        tf.tf_paged_attn_decode(q, pools[0], pools[1], pt, sg, scale=b.scale, split_keys=512, n_splits_max=c,
                                part_o=po, part_m=pm, part_l=pl, part_flag=pf, status=st, segs_host=b.segs)

    partials()
    tf.tf_attn_merge(po, pm, pl, pf, out, fl)
    torch.cuda.synchronize()
    want = out.clone()
    assert int(st.item()) == 0 and int(fl.sum()) == 0
    for _ in range(10):
        for x, was in zip(pools, keep):
            x.copy_(was)
        po.fill_(float("nan"))
        pl.zero_()
        out.zero_()
        partials()
        chunk()
        tf.tf_attn_merge(po, pm, pl, pf, out, fl)
        chunk()
        chunk()
        copy.copy_(out)
        for x in pools:
            x.zero_()
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
    assert int(st.item()) == 0 and int(chunk.st.item()) == 0


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_a_prompt_chunk_sees_the_rows_written_just_before_it(quantised, graph):
    """Rows appended (or read back from an 8-bit cache) and a prompt chunk over them, the next call on the stream."""
    n, hq, hkv, d, psz = 4000, 8, 2, 128, 32
    b = wl.make_paged_batch(7, rows=[n], keys=[n], n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=psz)
    rng = np.random.default_rng(7)
    kr, vr = (dev(wl.normal_bf16(rng, (n, hkv, d))) for _ in "kv")
    q, pt, sg, st = dev(b.q), dev(b.page_table), dev(b.segs), status_word()
    pools = [torch.zeros((b.n_pages, hkv, psz, d), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    out = torch.empty((n, hq, d), device=DEV)
    c = tf.Q8Cache(*(torch.zeros((b.n_pages, hkv, psz, d), dtype=torch.int8, device=DEV) for _ in "kv"),
                   *(torch.zeros((b.n_pages, hkv, psz), dtype=torch.uint8, device=DEV) for _ in "kv"))
    tf.tf_kv_append_q8(kr, vr, c, pt, sg, status=st, segs_host=b.segs)

    def write():
        if quantised:
            tf.tf_kv_read_q8(c, pt, sg, *pools, pt, status=st, segs_host=b.segs)
        else:
            tf.tf_kv_append(kr, vr, *pools, pt, sg, status=st, segs_host=b.segs)

    def attend():
        tf.tf_paged_attn_prompt(q, *pools, pt, b.segs[0], scale=b.scale, out=out, status=st)

    write()
    torch.cuda.synchronize()
    attend()
    torch.cuda.synchronize()
    want = out.clone()

    def round_():
        for x in pools:
            x.fill_(float("nan"))
        write()
        attend()

    run = round_
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            round_()
        run = g.replay
    for _ in range(10):
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert int(st.item()) == 0
