"""Timed cases of the paged KV-cache operators: per-head norms of queries and keys with the
rotation, written straight into the cache's pages; attention of new tokens over the pages; and
copying, forking, resizing and compacting the pages themselves.

`listed()` names the cases, `draw(rng)` makes more of the same ranges, `prepare` makes what a
program holds before the call, `run` is one pass (the plain torch form, or the framework's
kernels where `own` is set), `work` counts what the pass has to move and compute, and `exact`
evaluates the definitions in float64.

A cache here is k, v bf16 [layers][pages][kv heads][page size][head dim], a table int32
[sequences][max pages] of page ids (-1 where a sequence has none), len int32 [sequences] and a
use count per page, ref int32 [pages].
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 1e7


def listed():
    return [
        # one decoded token of the 0.8B-shaped model: the latency of a single call
        dict(name="qk_one_token", op="qk", n=1, new_lo=1, new_hi=1, ctx_lo=700, ctx_hi=700, hq=8, hkv=2, d=256, ps=64,
             rot=256, f32=True, norm=True, dense=False, mix=1),
        # speculative verify of some sessions of the 27B-shaped model: a few tokens each
        dict(name="qk_verify_batch", op="qk", n=48, new_lo=1, new_hi=6, ctx_lo=0, ctx_hi=5000, hq=24, hkv=4, d=256, ps=16,
             rot=256, f32=True, norm=True, dense=False, mix=2),
        # prompts of the 27B-shaped model written into pages, fp32 projections
        dict(name="qk_prompts", op="qk", n=3, new_lo=900, new_hi=2100, ctx_lo=0, ctx_hi=700, hq=24, hkv=4, d=256, ps=64,
             rot=256, f32=True, norm=True, dense=False, mix=3),
        # no cache: bf16 heads of 128 at given positions, a quarter of each head rotated
        dict(name="qk_dense_partial", op="qk", n=1, new_lo=1777, new_hi=1777, ctx_lo=90000, ctx_hi=90000, hq=16, hkv=8, d=128,
             ps=16, rot=32, f32=False, norm=True, dense=True, mix=4),
        # decode of one session with a long context (0.8B-shaped heads)
        dict(name="attn_decode_long", op="attn", n=1, new_lo=1, new_hi=1, ctx_lo=32768, ctx_hi=32768, hq=8, hkv=2, d=256, ps=64, mix=5),
        # decode of many sessions of the 27B-shaped model, ragged contexts, small pages
        dict(name="attn_decode_batch", op="attn", n=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=8192, hq=24, hkv=4, d=256, ps=16, mix=6),
        # a chunk of a prompt over its history next to short ones, heads of 128, pages of 48
        dict(name="attn_chunks", op="attn", n=5, new_lo=1, new_hi=700, ctx_lo=50, ctx_hi=9000, hq=16, hkv=4, d=128, ps=48, mix=7),
        # a whole 4096-token prompt of the 0.8B-shaped model
        dict(name="attn_prompt", op="attn", n=1, new_lo=4096, new_hi=4096, ctx_lo=0, ctx_hi=0, hq=8, hkv=2, d=256, ps=64, mix=8),
        # eight continuations of one prompt, every attention layer of the 27B-shaped model
        dict(name="fork_continuations", op="fork", n=8, parents=1, layers=16, hkv=4, d=256, ps=16, pages=512, seqs=16, len_lo=1001, len_hi=1001, mix=9),
        # sessions that end and are replaced by new prompts: page accounting only
        dict(name="turn_over", op="turn", n=61, layers=1, hkv=1, d=64, ps=16, pages=16384, seqs=128, len_lo=1, len_hi=3000, mix=10),
        # a half-empty pool of the 0.8B-shaped model's six attention layers moved together
        dict(name="compact_pool", op="compact", layers=6, hkv=2, d=256, ps=64, pages=1024, seqs=48, len_lo=100, len_hi=1500, mix=11),
        # a prefilled prompt taken from a contiguous cache [layers][heads][positions][d] into pages
        dict(name="copy_from_contiguous", op="copy", layers=6, hkv=2, d=256, ps=64, pages=200, n=63, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng: random.Random):
    op = rng.choice(["qk", "qk", "attn", "attn", "attn", "fork", "turn", "compact", "copy"])
    mix = rng.randrange(1 << 30)
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    ps = rng.choice([8, 16, 24, 32, 48, 64, 128])
    if op == "qk":
        n = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 5000 // n))
        ctx = rng.choice([0, _log(rng, 1, 8000 // n + 1), _log(rng, 1, 8000 // n + 1)])
        return dict(op=op, n=n, new_lo=1, new_hi=new, ctx_lo=0, ctx_hi=ctx, hq=hkv * rng.randint(1, 3), hkv=hkv, d=d, ps=ps,
                    rot=rng.choice([d, d // 2, d // 4]), f32=rng.random() < 0.5, norm=rng.random() < 0.8,
                    dense=rng.random() < 0.3, mix=mix)
    if op == "attn":
        hkv = rng.choice([1, 2, 4])
        hq = hkv * rng.randint(1, 8)
        ctx = _log(rng, 1, 16000)
        n = _log(rng, 1, max(1, min(64, 400000 // ctx)))
        # queries bounded so that queries x keys stays below the 4096-token prompt's
        new = _log(rng, 1, max(1, min(1500, 60_000_000 // (n * hq * (ctx + 1500)))))
        return dict(op=op, n=n, new_lo=rng.choice([1, new]), new_hi=new, ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx, hq=hq, hkv=hkv,
                    d=d, ps=ps, mix=mix)
    layers = rng.choice([1, 2, 6])
    row = layers * hkv * ps * d * 4
    if op == "fork":
        hi = _log(rng, 1, 2000)
        seqs = _log(rng, 4, 100)
        n = rng.randint(1, seqs - 2)
        need = seqs * (hi // ps + 2)
        layers = max(1, min(layers, 400_000_000 // (need * hkv * ps * d * 4)))
        return dict(op=op, n=n, parents=rng.randint(1, seqs - 1 - n), layers=layers, hkv=hkv, d=d, ps=ps, pages=need, seqs=seqs,
                    len_lo=0, len_hi=hi, mix=mix)
    if op == "turn":
        seqs = _log(rng, 2, 200)
        hi = _log(rng, 1, 3000)
        return dict(op=op, n=rng.randint(1, seqs), layers=1, hkv=1, d=64, ps=ps, pages=seqs * (hi // ps + 2), seqs=seqs, len_lo=0,
                    len_hi=hi, mix=mix)
    if op == "compact":
        pages = _log(rng, 8, max(8, min(4000, 800_000_000 // row)))
        seqs = _log(rng, 1, max(1, min(64, pages // 4)))
        return dict(op=op, layers=layers, hkv=hkv, d=d, ps=ps, pages=pages, seqs=seqs, len_lo=1, len_hi=max(1, pages // 2 // seqs * ps),
                    mix=mix)
    pages = _log(rng, 4, max(4, min(2000, 400_000_000 // row)))
    return dict(op=op, layers=layers, hkv=hkv, d=d, ps=ps, pages=pages, n=rng.randint(1, max(1, pages // 3)), mix=mix)


# ------------------------------------------------------------------ sizes that a case stands for
def _ragged(c):
    """New tokens and context of each of the case's sequences."""
    r = random.Random(c["mix"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["n"])]
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["n"])]
    return new, ctx


def _lengths(c):
    r = random.Random(c["mix"])
    return [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["seqs"])]


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs
def _pool(g, layers, pages, c):
    shape = (layers, pages, c["hkv"], c["ps"], c["d"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)]


def _tables(seed, lens, ps, n_pages, max_pages):
    """Pages dealt out at random to sequences of these lengths: table and use counts."""
    pages = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((len(lens), max_pages), -1, np.int32)
    ref = np.zeros(n_pages, np.int32)
    at = 0
    for i, n in enumerate(lens):
        m = _ceil(n, ps)
        table[i, :m] = pages[at:at + m]
        at += m
    ref[pages[:at]] = 1
    return table, ref


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c, cache=None)
    if c["op"] in ("qk", "attn"):
        new, ctx = _ragged(c)
        n, rows = c["n"], sum(new)
        lens = [a + b for a, b in zip(new, ctx)]
        slots = np.random.default_rng(seed + 1).permutation(n + 2)[:n].astype(np.int32)   # the cache has other sequences too
        all_lens = [0] * (n + 2)
        for i, x in zip(slots, lens):
            all_lens[i] = x
        s.update(max_new=max(new), max_len=max(lens), rows=rows, host_len=lens, host_new=new, host_slots=slots,
                 seq_start=_gpu(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), seqs=_gpu(slots))
        if not c.get("dense"):
            max_pages = max(1, _ceil(max(lens), c["ps"]))
            n_pages = sum(_ceil(x, c["ps"]) for x in lens) + 3
            table, ref = _tables(seed, all_lens, c["ps"], n_pages, max_pages)
            s["k"], s["v"] = _pool(g, 1, n_pages, c)
            s.update(table=_gpu(table), ref=_gpu(ref), len=_gpu(np.array(all_lens, np.int32)))
        if c["op"] == "qk":
            dt = torch.float32 if c["f32"] else torch.bfloat16
            hq, hkv, d = c["hq"], c["hkv"], c["d"]
            x = torch.randn((rows, hq + 2 * hkv, d), generator=g, device="cuda", dtype=torch.float32).to(dt)   # one fused projection
            s.update(q_in=x[:, :hq], k_in=x[:, hq:hq + hkv], v_in=x[:, hq + hkv:])
            gain = [(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2)]
            s["gains"] = gain if c["norm"] else [None, None]
            s["positions"] = _gpu((np.arange(rows) + ctx[0]).astype(np.int32))
        else:
            s["q_in"] = torch.randn((rows, c["hq"], c["d"]), generator=g, device="cuda", dtype=torch.bfloat16)
        return s
    s["k"], s["v"] = _pool(g, c["layers"], c["pages"], c)
    rs = np.random.default_rng(seed + 1)
    if c["op"] == "copy":
        shape = (c["layers"], c["hkv"], c["pages"], c["ps"], c["d"])   # pages of a contiguous cache, seen page first
        s["k0"], s["v0"] = [torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).transpose(1, 2) for _ in range(2)]
        s.update(src=_gpu(np.arange(c["n"], dtype=np.int32)), dst=_gpu(rs.permutation(c["pages"])[:c["n"]].astype(np.int32)))
        s.update(table=torch.full((1, 1), -1, dtype=torch.int32, device="cuda"), len=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 ref=torch.zeros(c["pages"], dtype=torch.int32, device="cuda"))
        return s
    lens = _lengths(c)
    max_pages = max(1, _ceil(c["len_hi"], c["ps"]))
    order = rs.permutation(c["seqs"])
    if c["op"] == "fork":
        parents, children = order[:c["parents"]], order[c["parents"]:c["parents"] + c["n"]]
        for i in children:
            lens[i] = 0
        s.update(src=_gpu(rs.choice(parents, c["n"]).astype(np.int32)), dst=_gpu(children.astype(np.int32)))
    if c["op"] == "turn":
        s.update(seqs=_gpu(order[:c["n"]].astype(np.int32)),
                 lens=_gpu(rs.integers(c["len_lo"], c["len_hi"] + 1, c["n"]).astype(np.int32)))
    table, ref = _tables(seed, lens, c["ps"], c["pages"], max_pages)
    s.update(table=_gpu(table), ref=_gpu(ref), len=_gpu(np.array(lens, np.int32)))
    if c["op"] == "compact":
        s.update(table0=s["table"].clone(), ref0=s["ref"].clone())
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _cache(s):
    """The handle that a program makes once for its cache and keeps."""
    if s["cache"] is None:
        from hybrid_deltanet_attention_b200 import PagedCache
        s["cache"] = PagedCache(s["k"], s["v"], s["table"], s["len"], s["ref"])
    return s["cache"]


def _state(s):
    return {n: s[n] for n in ("k", "v", "table", "len", "ref")}


def _own_qk(s):
    c, (gq, gk) = s["case"], s["gains"]
    if c["dense"]:
        from hybrid_deltanet_attention_b200 import qk_norm_rope
        q, k = qk_norm_rope(s["q_in"], s["k_in"], s["positions"], q_gain=gq, k_gain=gk, eps=EPS, theta=THETA, rot_dim=c["rot"])
        return {"q": q, "k": k}
    q = _cache(s).append(0, s["q_in"], s["k_in"], s["v_in"], s["seq_start"], s["seqs"], q_gain=gq, k_gain=gk, eps=EPS, theta=THETA,
                         rot_dim=c["rot"])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _own_attn(s):
    return _cache(s).attention(0, s["q_in"], s["seq_start"], s["seqs"])


def _own_fork(s):
    _cache(s).fork(s["src"], s["dst"])
    return _state(s)


def _own_turn(s):
    c = _cache(s)
    c.free(s["seqs"])
    c.resize(s["seqs"], s["lens"])
    return {n: s[n] for n in ("table", "len", "ref")}


def _own_compact(s):
    s["table"].copy_(s["table0"])   # put back first, so that each pass has the same pages to move
    s["ref"].copy_(s["ref0"])
    _cache(s).compact()
    return _state(s)


def _own_copy(s):
    from hybrid_deltanet_attention_b200 import PagedCache
    if "cache0" not in s:
        s["cache0"] = PagedCache(s["k0"], s["v0"], s["table"], s["len"], s["ref"])
    _cache(s).copy_pages(s["src"], s["dst"], source=s["cache0"])
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ plain forms
def _plain_rotate(x, gain, positions, c):
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
    half = c["rot"] // 2
    freq = THETA ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / c["rot"])
    angle = torch.remainder(positions.double()[:, None] * freq, 2 * math.pi)[:, None, :]   # far positions: 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1).bfloat16()


def _row_positions(s):
    """Slot and position of each new row."""
    rows = torch.arange(s["rows"], device="cuda")
    i = torch.searchsorted(s["seq_start"][1:].long(), rows, right=True)
    slot = s["seqs"][i].long()
    return slot, s["len"][slot].long() - s["seq_start"][i + 1] + rows


def _plain_qk(s):
    c, (gq, gk) = s["case"], s["gains"]
    if c["dense"]:
        return {"q": _plain_rotate(s["q_in"], gq, s["positions"], c), "k": _plain_rotate(s["k_in"], gk, s["positions"], c)}
    slot, pos = _row_positions(s)
    page = s["table"][slot, pos // c["ps"]].long()
    s["k"][0, page, :, pos % c["ps"]] = _plain_rotate(s["k_in"], gk, pos, c)
    s["v"][0, page, :, pos % c["ps"]] = s["v_in"].bfloat16()
    return {"q": _plain_rotate(s["q_in"], gq, pos, c), "k": s["k"], "v": s["v"]}


def _plain_attn(s):
    c = s["case"]
    n, nq, nk, hkv, d = c["n"], s["max_new"], s["max_len"], c["hkv"], c["d"]
    at = torch.arange(nk, device="cuda")
    slots = s["seqs"].long()
    lens = s["len"][slots].long()
    page = s["table"][slots][:, at // c["ps"]].clamp(min=0).long()
    seen = at < lens[:, None]
    k = s["k"][0][page, :, at % c["ps"]].float()                                   # [n][nk][hkv][d]
    v = torch.where(seen[..., None, None], s["v"][0][page, :, at % c["ps"]].float(), 0.0)
    start = s["seq_start"].long()
    new = start[1:] - start[:-1]
    t = torch.arange(nq, device="cuda")
    row = (start[:-1, None] + t).clamp(max=s["rows"] - 1)
    q = s["q_in"][row].float().view(n, nq, hkv, -1, d)
    pos = lens[:, None] - new[:, None] + t
    z = torch.einsum("nqhgd,nkhd->nhgqk", q, k) / math.sqrt(d)
    mask = (at <= pos[..., None]) & seen[:, None]
    z = z.masked_fill(~mask[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(z - m)
    o = torch.einsum("nhgqk,nkhd->nqhgd", p, v)
    l = p.sum(-1).permute(0, 3, 1, 2)[..., None]                                   # noqa: E741
    o = torch.where(l > 0, o / l, 0.0).reshape(n, nq, -1, d)
    return o[t < new[:, None]].bfloat16()


def _pages_of(lens, ps):
    return (lens + ps - 1) // ps


def _plain_take(s, wanted):
    """The lowest free pages for the marked entries of a matrix, in row order."""
    free = (s["ref"] == 0).nonzero().flatten()
    n = int(wanted.sum())
    s["ref"][free[:n]] = 1
    return free[:n].to(torch.int32)


def _plain_copy_rows(s, src, dst, rows):
    keep = (torch.arange(s["case"]["ps"], device="cuda") < rows[:, None])[None, :, None, :, None]
    s["k"][:, dst] = torch.where(keep, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(keep, s["v"][:, src], s["v"][:, dst])


def _plain_fork(s):
    ps, src, dst, table, ref = s["case"]["ps"], s["src"].long(), s["dst"].long(), s["table"], s["ref"]
    col = torch.arange(table.shape[1], device="cuda")
    minus = torch.tensor(-1, dtype=torch.int32, device="cuda")
    old = table[dst]
    had = old[col < _pages_of(s["len"][dst], ps)[:, None]].long()
    ref.index_add_(0, had, minus.expand(had.shape))
    n, rows = s["len"][src], table[src]
    full = (n // ps)[:, None]
    kept = rows[col < full].long()
    ref.index_add_(0, kept, -minus.expand(kept.shape))
    part = (col == full) & (n % ps > 0)[:, None]
    pages = _plain_take(s, part)
    _plain_copy_rows(s, rows[part].long(), pages.long(), (n % ps)[n % ps > 0])
    rows[part] = pages
    table[dst] = torch.where(col < _pages_of(n, ps)[:, None], rows, minus)
    s["len"][dst] = n
    return _state(s)


def _plain_resize(s, seqs, new):
    ps, table, ref = s["case"]["ps"], s["table"], s["ref"]
    col = torch.arange(table.shape[1], device="cuda")
    minus = torch.tensor(-1, dtype=torch.int32, device="cuda")
    rows, n = table[seqs], s["len"][seqs]
    low = torch.minimum(n, new)
    gone = rows[(col >= _pages_of(new, ps)[:, None]) & (col < _pages_of(n, ps)[:, None])].long()
    ref.index_add_(0, gone, minus.expand(gone.shape))
    edge = (col == (low // ps)[:, None]) & (low % ps > 0)[:, None]
    shared = edge & (ref[rows.clamp(min=0).long()] > 1)   # a partly filled page that others use: its own copy
    wanted = shared | ((col >= _pages_of(low, ps)[:, None]) & (col < _pages_of(new, ps)[:, None]))
    was = rows[shared].long()
    pages = torch.full_like(rows, -1)
    pages[wanted] = _plain_take(s, wanted)
    ref.index_add_(0, was, minus.expand(was.shape))
    _plain_copy_rows(s, was, pages[shared].long(), (low % ps)[shared.any(1)])
    rows = torch.where(wanted, pages, rows)
    table[seqs] = torch.where(col < _pages_of(new, ps)[:, None], rows, minus)
    s["len"][seqs] = new


def _plain_turn(s):
    seqs = s["seqs"].long()
    _plain_resize(s, seqs, torch.zeros_like(s["lens"]))
    _plain_resize(s, seqs, s["lens"])
    return {n: s[n] for n in ("table", "len", "ref")}


def _plain_compact(s):
    s["table"].copy_(s["table0"])   # put back first, so that each pass has the same pages to move
    s["ref"].copy_(s["ref0"])
    ps, table, ref = s["case"]["ps"], s["table"], s["ref"]
    at = torch.arange(ref.shape[0], device="cuda")
    live = ref > 0
    total = live.sum()
    src = (live & (at >= total)).nonzero().flatten()
    dst = (~live & (at < total)).nonzero().flatten()
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    to = at.to(torch.int32)
    to[src] = dst.to(torch.int32)
    used = torch.arange(table.shape[1], device="cuda") < _pages_of(s["len"], ps)[:, None]
    table.copy_(torch.where(used, to[table.clamp(min=0).long()], table))
    ref[dst] = ref[src]
    ref[src] = 0
    return _state(s)


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["k"][:, dst] = s["k0"][:, src]
    s["v"][:, dst] = s["v0"][:, src]
    return {"k": s["k"], "v": s["v"]}


_plain = dict(qk=_plain_qk, attn=_plain_attn, fork=_plain_fork, turn=_plain_turn, compact=_plain_compact, copy=_plain_copy)
_own = dict(qk=_own_qk, attn=_own_attn, fork=_own_fork, turn=_own_turn, compact=_own_compact, copy=_own_copy)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "qk":
        rows = sum(_ragged(c)[0])
        size = 4 if c["f32"] else 2
        heads_in, heads_out = c["hq"] + (1 if c["dense"] else 2) * c["hkv"], c["hq"] + (1 if c["dense"] else 2) * c["hkv"]
        return dict(bytes=rows * c["d"] * (heads_in * size + heads_out * 2) + 4 * rows + 4 * c["d"],
                    flops=rows * (c["hq"] + c["hkv"]) * (4 * c["d"] + 3 * c["rot"]))
    if c["op"] == "attn":
        new, ctx = _ragged(c)
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, ctx))
        keys = sum(a + b for a, b in zip(new, ctx))
        return dict(bytes=4 * keys * c["hkv"] * c["d"] + 4 * sum(new) * c["hq"] * c["d"] + 4 * _ceil(keys, c["ps"]),
                    flops=4 * pairs * c["hq"] * c["d"])
    slot = 4 * c["layers"] * c["hkv"] * c["d"]   # K and V of one position
    if c["op"] == "copy":
        return dict(bytes=2 * c["n"] * c["ps"] * slot + 8 * c["n"], flops=0)
    lens = _lengths(c)
    if c["op"] == "turn":
        pages = sum(_ceil(x, c["ps"]) for x in lens) * c["n"] // c["seqs"]
        return dict(bytes=4 * (2 * c["pages"] + 4 * pages + 4 * c["n"]), flops=0)
    if c["op"] == "compact":
        live = sum(_ceil(x, c["ps"]) for x in lens)
        moved = live * (c["pages"] - live) // c["pages"]   # pages are dealt out at random
        return dict(bytes=2 * moved * c["ps"] * slot + 8 * c["pages"] + 8 * live, flops=0)
    mean = sum(lens) / len(lens)
    rows = (mean % c["ps"]) if c["len_lo"] == c["len_hi"] else min(mean, c["ps"] / 2)
    return dict(bytes=2 * c["n"] * (rows * slot + 4 * mean / c["ps"]) + 4 * c["pages"], flops=0)


# ------------------------------------------------------------------ the definitions in float64
def exact(case, seed):
    s = prepare(case, seed)
    return dict(qk=_exact_qk, attn=_exact_attn).get(case["op"], _exact_pages)(s)


def _exact_heads(x, gain, pos, c):
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * gain.double()
    y = x.clone()
    half = c["rot"] // 2
    for i in range(half):
        w = pos.double() * math.pow(THETA, -2.0 * i / c["rot"])
        cs, sn = torch.cos(w)[:, None], torch.sin(w)[:, None]
        y[..., i] = x[..., i] * cs - x[..., i + half] * sn
        y[..., i + half] = x[..., i + half] * cs + x[..., i] * sn
    return y


def _exact_qk(s):
    c, (gq, gk) = s["case"], s["gains"]
    if c["dense"]:
        pos = s["positions"]
        return {"q": _exact_heads(s["q_in"], gq, pos, c), "k": _exact_heads(s["k_in"], gk, pos, c)}
    pos, page = [], []
    table = s["table"].cpu().numpy()
    for slot, n, new in zip(s["host_slots"], s["host_len"], s["host_new"]):
        pos += range(n - new, n)
        page += [int(table[slot, p // c["ps"]]) for p in range(n - new, n)]
    pos, page = torch.tensor(pos, device="cuda"), torch.tensor(page, device="cuda")
    k, v = s["k"].double(), s["v"].double()
    k[0, page, :, pos % c["ps"]] = _exact_heads(s["k_in"], gk, pos, c)
    v[0, page, :, pos % c["ps"]] = s["v_in"].double()
    return {"q": _exact_heads(s["q_in"], gq, pos, c), "k": k, "v": v}


def _exact_attn(s):
    c = s["case"]
    d, group = c["d"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q_in"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for slot, n, new in zip(s["host_slots"], s["host_len"], s["host_new"]):
        pages = s["table"][int(slot), :_ceil(n, c["ps"])].long()
        k = s["k"][0][pages].double().transpose(0, 1).reshape(c["hkv"], -1, d)[:, :n]
        v = s["v"][0][pages].double().transpose(0, 1).reshape(c["hkv"], -1, d)[:, :n]
        hidden = torch.arange(n, device="cuda") > torch.arange(n - new, n, device="cuda")[:, None]
        for h in range(c["hq"]):
            z = s["q_in"][at:at + new, h].double() @ k[h // group].T * d ** -0.5
            z[hidden] = -math.inf
            out[at:at + new, h] = torch.softmax(z, -1) @ v[h // group]
        at += new
    return out


def _exact_pages(s):
    c = s["case"]
    ps, op = c["ps"], c["op"]
    k, v = s["k"].clone(), s["v"].clone()
    if op == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            k[:, b], v[:, b] = s["k0"][:, a], s["v0"][:, a]
        return {"k": k, "v": v}
    table, lens, ref = (s[n].cpu().numpy().copy() for n in ("table", "len", "ref"))
    if op == "fork":
        # every child gives up what it had, then takes its parent's pages
        for b in s["dst"].tolist():
            for p in table[b, :_ceil(int(lens[b]), ps)]:
                ref[p] -= 1
        free = [p for p in range(c["pages"]) if ref[p] == 0]
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            n = int(lens[a])
            table[b], lens[b] = -1, n
            for j in range(_ceil(n, ps)):
                p = int(table[a, j])
                if (j + 1) * ps <= n:
                    ref[p] += 1
                else:
                    to = free.pop(0)
                    k[:, to, :, :n % ps], v[:, to, :, :n % ps] = k[:, p, :, :n % ps], v[:, p, :, :n % ps]
                    p, ref[to] = to, 1
                table[b, j] = p
    elif op == "turn":
        seqs = s["seqs"].tolist()
        for i in seqs:
            for p in table[i, :_ceil(int(lens[i]), ps)]:
                ref[p] -= 1
            table[i], lens[i] = -1, 0
        free = [p for p in range(c["pages"]) if ref[p] == 0]
        for i, n in zip(seqs, s["lens"].tolist()):
            lens[i] = n
            for j in range(_ceil(n, ps)):
                table[i, j] = free.pop(0)
                ref[table[i, j]] = 1
        k = v = None
    else:
        live = [p for p in range(c["pages"]) if ref[p] > 0]
        holes = [p for p in range(len(live)) if ref[p] == 0]
        to = {a: b for a, b in zip([p for p in live if p >= len(live)], holes)}
        for a, b in to.items():
            k[:, b], v[:, b] = k[:, a], v[:, a]
            ref[b], ref[a] = ref[a], 0
        for i in range(c["seqs"]):
            for j in range(_ceil(int(lens[i]), ps)):
                table[i, j] = to.get(int(table[i, j]), table[i, j])
    whole = {"table": _gpu(table), "len": _gpu(lens), "ref": _gpu(ref)}
    return whole if k is None else {"k": k, "v": v, **whole}
