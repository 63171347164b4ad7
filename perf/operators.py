"""Cases of the quantised-cache, shared-prefix and log-probability operators, and their plain forms.

Five operators of a serving round over a paged KV cache:

* ``append``   new K/V rows quantised to 8 bits as they are written into their pages
* ``read``     cached keys read back from 8 bits into bf16 pages
* ``attn``     attention over the 8-bit cache: decode, verify and block rows
* ``shared``   attention of many streams over one or more shared prefixes and their own keys
* ``logprob``  log probabilities of given tokens, the rows' entropy and their top alternatives

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits; with ``own`` true it makes
the library's calls.  ``exact`` computes the same outputs in 64 bits from the definitions.

The 8-bit format: every (key, kv-head) row of K and of V has one scale byte e, standing for 2^(e - 127), and D codes
(e4m3 or int8); an element is code * 2^(e - 127).  The exponent is the smallest k >= -100 with amax <= Q * 2^k, where
Q is 448 (e4m3) or 127 (int8), so quantising is exact but for one rounding (to nearest, ties to even) an element.
"""
import math
import random

import torch

own = False

PAGES_SPARE = 3  # pages of the pool that no stream owns


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step's new rows of 16 streams into an e4m3 cache: latency
        dict(name="append decode round e4m3", kind="append", type="e4m3", streams=16, rows_lo=1, rows_hi=1,
             keys_lo=1024, keys_hi=8192, kv_heads=8, dim=128, page=32, tables=2),
        # a whole 15,000-token prompt's rows into an int8 cache: bandwidth
        dict(name="append long prompt int8", kind="append", type="int8", streams=1, rows_lo=15000, rows_hi=15000,
             keys_lo=15000, keys_hi=15000, kv_heads=4, dim=256, page=32, tables=4),
        # a cached prefix of 12,288 keys read back for a prompt chunk in bf16
        dict(name="read cached prefix e4m3", kind="read", type="e4m3", streams=1, rows_lo=12288, rows_hi=12288,
             keys_lo=12288, keys_hi=12288, kv_heads=4, dim=256, page=32, tables=4),
        # the last keys of a few short streams read back: ragged, small pages
        dict(name="read ragged streams int8", kind="read", type="int8", streams=5, rows_lo=1, rows_hi=700,
             keys_lo=700, keys_hi=1500, kv_heads=2, dim=64, page=16, tables=6),
        # two short streams of one row: the smallest decode step
        dict(name="attn tiny decode e4m3", kind="attn", type="e4m3", streams=2, rows_lo=1, rows_hi=1, keys_lo=37,
             keys_hi=70, q_heads=8, kv_heads=2, dim=64, page=16, out="f32", tables=1),
        # the multi-stream decode step over an e4m3 cache
        dict(name="attn decode step e4m3", kind="attn", type="e4m3", streams=16, rows_lo=1, rows_hi=1, keys_lo=1024,
             keys_hi=8192, q_heads=32, kv_heads=8, dim=128, page=32, out="f32", tables=2),
        # a verify round of 1-16 rows a stream over an int8 cache
        dict(name="attn verify round int8", kind="attn", type="int8", streams=8, rows_lo=1, rows_hi=16, keys_lo=2048,
             keys_hi=16384, q_heads=16, kv_heads=2, dim=256, page=32, out="bf16", tables=3),
        # 64 streams decoding behind one system prompt of 8,192 keys
        dict(name="shared prompt decode", kind="shared", prefixes=1, prefix_lo=8192, prefix_hi=8192, streams=64,
             rows_lo=1, rows_hi=1, keys_lo=16, keys_hi=1024, q_heads=32, kv_heads=8, dim=128, page=32, out="bf16",
             tables=2),
        # small ragged groups behind two short prefixes, 1-5 rows a stream
        dict(name="shared ragged groups", kind="shared", prefixes=2, prefix_lo=500, prefix_hi=1300, streams=7,
             rows_lo=1, rows_hi=5, keys_lo=5, keys_hi=200, q_heads=16, kv_heads=2, dim=256, page=32, out="bf16",
             tables=5),
        # the rows of a verify round over a 128,000-token vocabulary, 20 alternatives
        dict(name="logprob verify rows bf16", kind="logprob", dtype="bf16", rows=62, cols=128000, tokens=1, top=20,
             masked=False),
        # one row in f32 with a third of the vocabulary masked: latency
        dict(name="logprob one masked row f32", kind="logprob", dtype="f32", rows=1, cols=128000, tokens=4, top=5,
             masked=True),
        # the rows of a prompt scored against its next tokens
        dict(name="logprob prompt rows bf16", kind="logprob", dtype="bf16", rows=1024, cols=128000, tokens=1, top=5,
             masked=False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("append", "read", "attn", "shared", "logprob"))
    tables = rng.randrange(1 << 20)
    if kind == "logprob":
        cols = _log(rng, 700, 152000)
        return dict(kind=kind, dtype=rng.choice(("bf16", "f32")), rows=_log(rng, 1, max(1, 60_000_000 // cols)),
                    cols=cols, tokens=rng.randint(1, 4), top=rng.randint(0, 32), masked=rng.random() < 0.4)
    dim = rng.choice((64, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    page = rng.choice((8, 16, 32, 64, 256))
    if kind in ("append", "read"):
        streams = _log(rng, 1, 48)
        most = max(2, 15_000_000 // (kv * dim * streams))
        rows = _log(rng, 1, most)
        lo = rng.randint(1, rows)
        keys = rows + rng.randint(0, max(1, most - rows))
        return dict(kind=kind, type=rng.choice(("e4m3", "int8")), streams=streams, rows_lo=lo, rows_hi=rows,
                    keys_lo=rows, keys_hi=keys, kv_heads=kv, dim=dim, page=page, tables=tables)
    group = rng.choice((1, 2, 4, 8))
    out = rng.choice(("f32", "bf16")) if kind == "attn" else "bf16"
    rows = rng.choice((1, 1, 1, 2, 5, 16))
    streams = _log(rng, 1, 32)
    most = min(30000, 60_000_000 // (kv * dim * streams))
    hi = _log(rng, rows + 1, max(rows + 2, most))
    lo = rng.randint(rows, hi)
    case = dict(kind=kind, streams=streams, rows_lo=rng.randint(1, rows), rows_hi=rows, keys_lo=lo, keys_hi=hi,
                q_heads=kv * group, kv_heads=kv, dim=dim, page=page, out=out, tables=tables)
    if kind == "attn":
        case["type"] = rng.choice(("e4m3", "int8"))
        return case
    prefixes = rng.randint(1, min(4, streams))
    case["keys_hi"] = max(rows, min(hi, 2000))
    case["keys_lo"] = min(lo, case["keys_hi"])
    plo = _log(rng, 1, max(2, min(16384, 20_000_000 // (kv * dim * prefixes))))
    return dict(case, prefixes=prefixes, prefix_lo=max(1, plo // rng.choice((1, 2))), prefix_hi=plo)


def _sizes(case):
    """Rows, keys and (shared) prefix lengths of a case's streams: the case's own, whatever the inputs' seed."""
    rng = random.Random(case["tables"])
    rows = [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["streams"])]
    keys = [max(r, rng.randint(case["keys_lo"], case["keys_hi"])) for r in rows]
    pre = [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case.get("prefixes", 0))]
    return rows, keys, pre


def work(case):
    if case["kind"] == "logprob":
        r, c = case["rows"], case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": r * (c * size + 8 * case["tokens"] + 8 * case["top"] + 9), "flops": 6 * r * c}
    rows, keys, pre = _sizes(case)
    hkv, d = case["kv_heads"], case["dim"]
    if case["kind"] in ("append", "read"):
        # D values of 16 bits on one side, D codes and a scale byte on the other, for K and for V
        return {"bytes": sum(rows) * hkv * 2 * (2 * d + d + 1), "flops": 4 * sum(rows) * hkv * d}
    hq = case["q_heads"]
    row_bytes = d + 1 if case["kind"] == "attn" else 2 * d
    once = sum(keys) + sum(pre)
    seen = sum(r * (n - r) + r * (r + 1) // 2 for r, n in zip(rows, keys))
    if pre:
        seen += sum(r * pre[_prefix_of(s, case)] for s, r in enumerate(rows))
    io = sum(rows) * hq * d * (2 + (4 if case["out"] == "f32" else 2))
    return {"bytes": once * hkv * 2 * row_bytes + io, "flops": 4 * d * hq * seen}


def _prefix_of(s, case):
    """The prefix of stream s: the streams in order, spread evenly over the prefixes."""
    return s * case["prefixes"] // case["streams"]


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(shape, g):
    """Rows of keys or values as a cache meets them: normal elements, some channels larger, row sizes that differ."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    channel = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    size = torch.exp(0.3 * torch.randn(shape[:-1], generator=g, device="cuda"))
    return x.mul_(channel / channel.square().mean().sqrt()).mul_(size[..., None]).to(torch.bfloat16)


def _tables(sizes, page, seed, spare=PAGES_SPARE):
    """(page ids of each stream in turn, first entry of each stream, page counts, pages of the pool)."""
    n_pages = [-(-n // page) for n in sizes]
    total = sum(n_pages) + spare
    ids = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    base = [sum(n_pages[:i]) for i in range(len(sizes))]
    return ids[: max(1, sum(n_pages))].contiguous(), base, n_pages, total


def _segs(rows, keys, base, n_pages):
    q_row, out = 0, []
    for r, n, b, p in zip(rows, keys, base, n_pages):
        out.append([q_row, r, n, b, p])
        q_row += r
    return torch.tensor(out, dtype=torch.int32)


def _last_keys(segs, table, page):
    """(page, slot) of every stream's last n_rows keys, stream by stream."""
    pages, slots = [], []
    for _, r, n, b, _ in segs.tolist():
        j = torch.arange(n - r, n)
        pages.append(table[b + j // page].long())
        slots.append(j % page)
    return torch.cat(pages).cuda(), torch.cat(slots).cuda()


def _grid(segs, table, page):
    """(page, slot) of every stream's keys [streams, longest], streams padded with their first key."""
    n_max = int(segs[:, 2].max())
    j = torch.arange(n_max)[None].expand(len(segs), -1)
    j = torch.where(j < segs[:, 2:3], j, torch.zeros_like(j))
    return table[segs[:, 3:4] + j // page].long().cuda(), (j % page).cuda()


def _row_grid(segs):
    """Rows of each stream [streams, most rows] (padded with its first row), which of them are real."""
    t_max = max(1, int(segs[:, 1].max()))
    i = torch.arange(t_max)[None].expand(len(segs), -1)
    real = i < segs[:, 1:2]
    return (segs[:, 0:1] + torch.where(real, i, torch.zeros_like(i))).long().cuda(), real.cuda()


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    st = {"case": dict(case), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if kind == "logprob":
        r, c = case["rows"], case["cols"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = torch.empty((r, c), device="cuda", dtype=dt)
        for a in range(0, r, 128):
            x[a : a + 128] = (3 * torch.randn((min(r, a + 128) - a, c), generator=g, device="cuda")).to(dt)
        tokens = torch.randint(0, c, (r, case["tokens"]), generator=g, device="cuda", dtype=torch.int32)
        if case["masked"]:  # a grammar's or a filter's banned tokens, the given ones allowed
            gone = torch.rand((r, c), generator=g, device="cuda") < 0.34
            x.masked_fill_(gone.scatter_(1, tokens.long(), False), -math.inf)
        k = case["top"]
        f, i = dict(device="cuda", dtype=torch.float32), dict(device="cuda", dtype=torch.int32)
        return dict(st, logits=x, tokens=tokens, token_logprobs=torch.empty((r, case["tokens"]), **f),
                    entropy=torch.empty(r, **f), lse=torch.empty(r, **f), top_ids=torch.empty((r, k), **i),
                    top_logprobs=torch.empty((r, k), **f), flags=torch.empty(r, device="cuda", dtype=torch.uint8))
    rows, keys, pre = _sizes(case)
    page, hkv, d = case["page"], case["kv_heads"], case["dim"]
    table, base, n_pages, total = _tables(pre + keys, page, seed)
    n_pre = len(pre)
    segs = _segs(rows, keys, base[n_pre:], n_pages[n_pre:])
    st.update(page_table=table.cuda(), page_table_host=table.numpy(), segs=segs.cuda(), segs_host=segs.numpy())
    pool = (total, hkv, page, d)
    if kind != "append":
        k, v = _rows(pool, g), _rows(pool, g)
    if kind == "append":
        code = torch.float8_e4m3fn if case["type"] == "e4m3" else torch.int8
        st.update(k_rows=_rows((sum(rows), hkv, d), g), v_rows=_rows((sum(rows), hkv, d), g))
        for n in "kv":
            st[n + "_codes"] = torch.zeros(pool, dtype=torch.uint8, device="cuda").view(code)
            st[n + "_scale"] = torch.full(pool[:3], 27, dtype=torch.uint8, device="cuda")
        st["at"] = _last_keys(segs, table, page)
        return st
    if kind in ("read", "attn"):
        st["k_codes"], st["k_scale"] = _quantise(k, case["type"])
        st["v_codes"], st["v_scale"] = _quantise(v, case["type"])
    if kind == "read":  # into bf16 pages of their own, in order
        dst = torch.arange(len(table), dtype=torch.int32)
        st.update(dst_page_table=dst.cuda(), dst_page_table_host=dst.numpy())
        for n in "kv":
            st[n + "_pool"] = torch.zeros((len(dst),) + pool[1:], dtype=torch.bfloat16, device="cuda")
        st["at"], st["to"] = _last_keys(segs, table, page), _last_keys(segs, dst, page)
        return st
    hq = case["q_heads"]
    st["q"] = torch.randn((sum(rows), hq, d), generator=g, device="cuda").to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(d)
    st["out"] = torch.empty((sum(rows), hq, d), device="cuda",
                            dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    st["flags"] = torch.empty((sum(rows), hq), device="cuda", dtype=torch.uint8)
    st["grid"], st["rows"] = _grid(segs, table, page), _row_grid(segs)
    if kind == "shared":
        groups = [[s for s in range(len(rows)) if _prefix_of(s, case) == p] for p in range(n_pre)]
        pr = [sum(rows[s] for s in grp) for grp in groups]
        prefixes = _segs(pr, pre, base[:n_pre], n_pages[:n_pre])
        st.update(k_pool=k, v_pool=v, prefixes=prefixes.cuda(), prefixes_host=prefixes.numpy(),
                  prefix_grid=_grid(prefixes, table, page), prefix_rows=_row_grid(prefixes))
    return st


# ------------------------------------------------------------------ plain forms


def _quantise(x, kind):
    """(codes, scale bytes) of the rows x [..., D]."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    top, bits = (0.875, 9) if kind == "e4m3" else (0.9921875, 7)  # 448 = 0.875 * 2^9, 127 = 0.9921875 * 2^7
    k = torch.clamp(e - bits + (m > top), min=-100)
    x = x * torch.exp2(-k.float())[..., None]
    codes = x.to(torch.float8_e4m3fn) if kind == "e4m3" else torch.round(x).to(torch.int8)
    return codes, (k + 127).to(torch.uint8)


def _values(codes, scale, kind):
    """What the codes (as bytes) and scale bytes stand for, in 32 bits."""
    v = codes.view(torch.float8_e4m3fn if kind == "e4m3" else torch.int8).float()
    return v * torch.exp2(scale.float() - 127.0)[..., None]


def _attend(q, k, v, mask, scale):
    """(m, l, o) of q [B, T, Hq, D] over k, v [B, N, Hkv, D] where mask [B, T, N] holds, in 32 bits."""
    b, t, hq, d = q.shape
    hkv = k.shape[2]
    qh = q.float().view(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    s = torch.matmul(qh, k.permute(0, 2, 3, 1)) * scale  # [B, Hkv, G * T, N]
    s = s.view(b, hkv, hq // hkv, t, -1).masked_fill(~mask[:, None, None], -math.inf)
    m = s.amax(-1)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m)[..., None])
    o = torch.matmul(p.view(b, hkv, (hq // hkv) * t, -1), v.permute(0, 2, 1, 3)).view(b, hkv, hq // hkv, t, d)
    return m, p.sum(-1), o


def _to_rows(x, rows, real, like):
    """[B, Hkv, G, T, ...] to [rows, Hq, ...]."""
    x = x.permute(0, 3, 1, 2, *range(4, x.dim())).flatten(2, 3)[real]
    out = torch.zeros((like.shape[0], like.shape[1]) + tuple(x.shape[2:]), device=x.device, dtype=x.dtype)
    out[rows[real]] = x
    return out


def _seen(st):
    """Keys that each row of each stream sees [streams, rows, keys]: the causal count."""
    segs, n = st["segs"].long(), st["grid"][0].shape[1]
    i = torch.arange(st["rows"][0].shape[1], device="cuda")
    lim = segs[:, 2:3] - segs[:, 1:2] + i[None] + 1
    return torch.arange(n, device="cuda")[None, None] < lim[:, :, None]


def _finish(m, l, o, dtype):
    out = o / l[..., None]
    return {"out": out.to(dtype), "flags": (~torch.isfinite(out).all(-1)).to(torch.uint8)}


def _plain(st):
    case, kind = st["case"], st["case"]["kind"]
    if kind == "append":
        page, slot = st["at"]
        for n in "kv":
            codes, scale = _quantise(st[n + "_rows"], case["type"])
            st[n + "_codes"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            st[n + "_scale"][page, :, slot] = scale
        return {n: st[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale")}
    if kind == "read":
        (page, slot), (to, at) = st["at"], st["to"]
        for n in "kv":
            codes = st[n + "_codes"].view(torch.uint8)[page, :, slot]
            st[n + "_pool"][to, :, at] = _values(codes, st[n + "_scale"][page, :, slot], case["type"]).bfloat16()
        return {"k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if kind == "attn":
        page, slot = st["grid"]
        k, v = (_values(st[n + "_codes"].view(torch.uint8)[page, :, slot], st[n + "_scale"][page, :, slot],
                        case["type"]) for n in "kv")
        rows, real = st["rows"]
        m, l, o = (_to_rows(x, rows, real, st["q"]) for x in _attend(st["q"][rows], k, v, _seen(st), st["scale"]))
        return _finish(m, l, o, st["out"].dtype)
    if kind == "shared":
        page, slot = st["grid"]
        rows, real = st["rows"]
        k, v = (st[n + "_pool"][page, :, slot].float() for n in "kv")
        m, l, o = (_to_rows(x, rows, real, st["q"]) for x in _attend(st["q"][rows], k, v, _seen(st), st["scale"]))
        page, slot = st["prefix_grid"]
        rows, real = st["prefix_rows"]
        k, v = (st[n + "_pool"][page, :, slot].float() for n in "kv")
        mask = torch.arange(page.shape[1], device="cuda")[None] < st["prefixes"][:, 2:3]
        mask = mask[:, None].expand(-1, rows.shape[1], -1)
        pm, pl, po = (_to_rows(x, rows, real, st["q"]) for x in _attend(st["q"][rows], k, v, mask, st["scale"]))
        top = torch.maximum(m, pm)
        a, b = torch.exp(m - top), torch.exp(pm - top)
        return _finish(top, l * a + pl * b, o * a[..., None] + po * b[..., None], st["out"].dtype)
    x = st["logits"].float()
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    l = e.sum(1, dtype=torch.float64).float()  # 128,000 terms: the sum is held wider than its terms
    t = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, dtype=torch.float64).float()
    log_l = torch.log(l)
    out = {"token_logprobs": d.gather(1, st["tokens"].long()) - log_l[:, None], "entropy": log_l - t / l,
           "lse": m[:, 0] + log_l, "flags": (~torch.isfinite(m[:, 0] + l)).to(torch.uint8)}
    if case["top"]:
        ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, : case["top"]]
        out.update(top_ids=ids.to(torch.int32), top_logprobs=d.gather(1, ids) - log_l[:, None])
    return out


# ------------------------------------------------------------------ the library's calls


def _own(st):
    import paged_kv_cache_segment_b200 as tf

    case, kind = st["case"], st["case"]["kind"]
    if kind == "logprob":
        top = case["top"] > 0
        tf.tf_logprob_rows(st["logits"], st["tokens"], token_logprobs=st["token_logprobs"], entropy=st["entropy"],
                           lse=st["lse"], top_ids=st["top_ids"] if top else None,
                           top_logprobs=st["top_logprobs"] if top else None, flags=st["flags"], status=st["status"])
        names = ("token_logprobs", "entropy", "lse", "flags") + (("top_ids", "top_logprobs") if top else ())
        return {n: st[n] for n in names}
    tables = dict(segs_host=st["segs_host"], page_table_host=st["page_table_host"], status=st["status"])
    if kind in ("append", "read", "attn") and "cache" not in st:
        st["cache"] = tf.Q8Cache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
    if kind == "append":
        tf.tf_kv_append_q8(st["k_rows"], st["v_rows"], st["cache"], st["page_table"], st["segs"], **tables)
        return {n: st[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale")}
    if kind == "read":
        tf.tf_kv_read_q8(st["cache"], st["page_table"], st["segs"], st["k_pool"], st["v_pool"], st["dst_page_table"],
                         dst_page_table_host=st["dst_page_table_host"], **tables)
        return {"k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    rows, hq, d = st["q"].shape
    if "workspace" not in st:
        n = (tf.tf_paged_attn_q8_workspace_bytes(rows, hq, d, 128) if kind == "attn" else
             tf.tf_paged_attn_shared_workspace_bytes(rows, hq, d, 64, 64))
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = dict(scale=st["scale"], workspace=st["workspace"], out=st["out"], flags=st["flags"])
    if kind == "attn":
        tf.tf_paged_attn_q8(st["q"], st["cache"], st["page_table"], st["segs"], n_splits_max=128, **outs, **tables)
    else:
        tf.tf_paged_attn_shared(st["q"], st["k_pool"], st["v_pool"], st["page_table"], st["prefixes"], st["segs"],
                                n_prefix_splits=64, n_splits_max=64, prefixes_host=st["prefixes_host"], **outs,
                                **tables)
    return {"out": st["out"], "flags": st["flags"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_attention(q, keys, values, scale):
    """One row's heads q [Hq, D] over keys, values [N, Hkv, D], in 64 bits, for rows stacked: q [T, Hq, D], lim [T]."""
    hkv, group = keys.shape[1], q.shape[1] // keys.shape[1]
    out = torch.empty_like(q)
    for h in range(hkv):
        s = torch.einsum("thd,nd->thn", q[:, h * group : (h + 1) * group], keys[:, h]) * scale[0]
        n = torch.arange(keys.shape[0], device="cuda")
        s = torch.where(n[None, None] < scale[1][:, None, None], s, torch.full_like(s, -math.inf))
        out[:, h * group : (h + 1) * group] = torch.softmax(s, -1) @ values[:, h]
    return out


def _exact_rows(x, kind):
    """(codes as the numbers they are, scale bytes) of rows x, from the format's definition in 64 bits."""
    x = x.double()
    amax = x.abs().amax(-1)
    q = 448.0 if kind == "e4m3" else 127.0
    k = torch.full_like(amax, -100.0)
    for e in range(-100, 121):
        k = torch.where(amax > q * 2.0**e, torch.full_like(k, e + 1.0), k)
    y = x * torch.exp2(-k)[..., None]
    if kind == "int8":
        step = torch.ones_like(y)
    else:  # e4m3: eight steps a binade, the subnormals' step below 2^-6
        b = torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0**-6)))
        step = torch.exp2(b - 3)
    return torch.round(y / step) * step, k + 127


def _exact_values(codes, scale, kind):
    raw = codes.view(torch.uint8).long()
    if kind == "int8":
        v = torch.where(raw > 127, raw - 256, raw).double()
    else:
        e, f = (raw >> 3) & 15, (raw & 7).double()
        v = torch.where(e == 0, f / 8 * 2.0**-6, (1 + f / 8) * torch.exp2((e - 7).double()))
        v = torch.where(raw > 127, -v, v)
    return v * torch.exp2(scale.double() - 127)[..., None]


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "logprob":
        tp = torch.empty(st["token_logprobs"].shape, dtype=torch.float64, device="cuda")
        ent = torch.empty(case["rows"], dtype=torch.float64, device="cuda")
        lse, top = torch.empty_like(ent), torch.empty((case["rows"], case["top"]), dtype=torch.float64, device="cuda")
        for a in range(0, case["rows"], 64):
            x = st["logits"][a : a + 64].double()
            lse[a : a + 64] = torch.logsumexp(x, 1)
            lp = x - lse[a : a + 64, None]
            ent[a : a + 64] = torch.special.entr(torch.exp(lp)).sum(1)
            tp[a : a + 64] = lp.gather(1, st["tokens"][a : a + 64].long())
            if case["top"]:
                top[a : a + 64] = torch.topk(lp, case["top"], dim=1)[0]
        out = {"token_logprobs": tp, "entropy": ent, "lse": lse, "flags": None}
        return dict(out, top_ids=None, top_logprobs=top) if case["top"] else out
    if kind == "append":
        page, slot = st["at"]
        out = {}
        for n in "kv":
            codes, scale = _exact_rows(st[n + "_rows"], case["type"])
            pool = torch.zeros(st[n + "_codes"].shape, dtype=torch.float32, device="cuda")
            pool[page, :, slot] = codes.float()
            out[n + "_codes"] = pool.double()
            out[n + "_scale"] = None
        return out
    if kind == "read":
        (page, slot), (to, at) = st["at"], st["to"]
        out = {}
        for n in "kv":
            v = _exact_values(st[n + "_codes"].view(torch.uint8)[page, :, slot], st[n + "_scale"][page, :, slot],
                              case["type"])
            out[n + "_pool"] = torch.zeros(st[n + "_pool"].shape, dtype=torch.float64, device="cuda")
            out[n + "_pool"][to, :, at] = v
        return out
    page = case["page"]
    table = st["page_table"].long()

    def gather(base, n):
        j = torch.arange(n, device="cuda")
        ids, slot = table[base + j // page], j % page
        if kind == "attn":
            return [_exact_values(st[c + "_codes"].view(torch.uint8)[ids, :, slot], st[c + "_scale"][ids, :, slot],
                                  case["type"]) for c in "kv"]
        return [st[c + "_pool"][ids, :, slot].double() for c in "kv"]

    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, (r0, r, n, base, _) in enumerate(st["segs_host"].tolist()):
        k, v = gather(base, n)
        ahead = 0
        if kind == "shared":
            _, _, ahead, pbase, _ = st["prefixes_host"].tolist()[_prefix_of(s, case)]
            pk, pv = gather(pbase, ahead)
            k, v = torch.cat([pk, k]), torch.cat([pv, v])
        lim = ahead + n - r + 1 + torch.arange(r, device="cuda")
        out[r0 : r0 + r] = _exact_attention(st["q"][r0 : r0 + r].double(), k, v, (st["scale"], lim))
    return {"out": out, "flags": None}
