"""Paged-cache operators on the GPU against plain float64 and loop implementations."""
import random

import numpy as np
import pytest

import paged_ref as ref
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16_HALF_STEP = 2.0 ** -8


def hda():
    import hybrid_deltanet_attention_b200 as m
    return m


def ints(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def make_cache(rng, lens, ps, hkv, d, layers=1, spare=3, max_pages=None, fill=True):
    """A cache whose sequences hold `lens` positions in shuffled pages, the memory full of random entries."""
    need = sum(ref.pages_of(n, ps) for n in lens)
    n_pages = need + spare
    mp = max_pages or max([1] + [ref.pages_of(n, ps) for n in lens])
    c = hda().PagedCache.empty(layers, n_pages, hkv, ps, d, len(lens), mp)
    if fill:
        c.k.normal_()
        c.v.normal_()
    pages = rng.permutation(n_pages)
    table, at = np.full((len(lens), mp), -1, np.int32), 0
    for i, n in enumerate(lens):
        m = ref.pages_of(n, ps)
        table[i, :m] = pages[at:at + m]
        at += m
    c.table.copy_(torch.from_numpy(table))
    c.len.copy_(ints(lens))
    c.ref[torch.from_numpy(pages[:at]).cuda()] = 1
    return c, table


def gather(t, layer, row, n, ps):
    """Positions 0..n-1 of a sequence as float64 [n][hkv][d]."""
    if n == 0:
        return np.zeros((0, t.shape[2], t.shape[4]))
    pages = torch.from_numpy(row[:ref.pages_of(n, ps)]).long().cuda()
    x = t[layer][pages].transpose(1, 2).reshape(-1, t.shape[2], t.shape[4])[:n]
    return f64(x)


# ------------------------------------------------------------------ norm, rotation, append
def check_rope(got, x, gain, pos, rot, eps, theta):
    want, mag = ref.rope(x, gain, pos, rot, eps, theta)
    # one bf16 rounding, and fp32 arithmetic on terms of size mag: the norm's sum of at most 256 squares over a warp
    # tree (16 steps, halved by the square root), rsqrt, sine and cosine of an angle rounded
    # to fp32 in [-pi, pi] (2^-23), five products and a sum stay below 2^-19 of it
    bound = BF16_HALF_STEP * np.abs(want) + 2.0 ** -19 * mag * (1 + BF16_HALF_STEP) + 1e-38
    bad = np.abs(got - want) > bound
    assert not bad.any(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("d,rot,dtype,norm,ps", [(256, 256, "float32", True, 64), (256, 64, "bfloat16", True, 16),
                                                 (128, 128, "bfloat16", False, 24), (128, 32, "float32", True, 8),
                                                 (64, 64, "float32", False, 48), (64, 16, "bfloat16", True, 128),
                                                 (64, 0, "float32", True, 8), (128, 8, "float32", True, 16)])
def test_append_norms_rotates_and_stores(d, rot, dtype, norm, ps):
    rng = np.random.default_rng(d + rot + ps)
    hq, hkv, dt = 6, 2, getattr(torch, dtype)
    new = [1, 0, 7, ps, 2 * ps + 3, 0, 1]
    lens = [1, 5, 7 + ps - 1, ps, 3 * ps + 3, 0, 4000]
    c, table = make_cache(rng, lens + [9], ps, hkv, d, layers=2)
    order = [3, 0, 6, 1, 4, 5, 2]                       # the call's order of sequences
    start = np.concatenate([[0], np.cumsum([new[i] for i in order])]).astype(np.int32)
    rows = int(start[-1])
    x = torch.randn(rows + 2, hq + 2 * hkv + 1, d, device="cuda").to(dt)   # two more rows behind the last sequence
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    gains = [(1 + 0.2 * torch.randn(d, device="cuda")).bfloat16() for _ in range(2)] if norm else [None, None]
    out = torch.full((rows + 2, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    c.append(1, q, k, v, ints(start), ints(order), q_gain=gains[0], k_gain=gains[1], eps=1e-5, theta=1e6, rot_dim=rot, out=out)
    c.sync()
    pos = np.concatenate([np.arange(lens[i] - new[i], lens[i]) for i in order]).astype(np.int64)
    slot = np.concatenate([np.full(new[i], i) for i in order])
    g = [f64(t) if t is not None else None for t in gains]
    check_rope(f64(out)[:rows], f64(q)[:rows], g[0], pos, rot, 1e-5, 1e6)
    assert (out[rows:] == 7.0).all()
    page, at = torch.from_numpy(table[slot, pos // ps]).long().cuda(), torch.from_numpy(pos % ps).cuda()
    check_rope(f64(c.k[1, page, :, at]), f64(k)[:rows], g[1], pos, rot, 1e-5, 1e6)
    assert torch.equal(c.v[1, page, :, at], v[:rows].bfloat16())
    k0[1, page, :, at], v0[1, page, :, at] = c.k[1, page, :, at], c.v[1, page, :, at]
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)   # nothing else written


@pytest.mark.parametrize("d,dtype", [(64, "float32"), (128, "bfloat16"), (256, "float32")])
def test_dense_rope_far_and_negative_positions(d, dtype):
    rows = 9
    q = torch.randn(rows, 3, d, device="cuda").to(getattr(torch, dtype))
    k = torch.randn(rows, 1, d, device="cuda").to(getattr(torch, dtype))
    pos = np.array([0, 1, -1, 1000003, 2 ** 31 - 1, -2 ** 31, 262144, 77, 5], np.int64)
    qo, ko = hda().qk_norm_rope(q, k, ints(pos), theta=1e4)
    # at 2^31 an angle in float64 is off by about 2^31 * 2^-52 times a small factor: below 2^-19
    check_rope(f64(qo), f64(q), None, pos, d, 1e-6, 1e4)
    check_rope(f64(ko), f64(k), None, pos, d, 1e-6, 1e4)


def test_dense_rope_in_place_and_zero_rows():
    x = torch.randn(33, 5, 128, device="cuda").bfloat16()
    q, k = x[:, :4], x[:, 4:]
    pos = ints(range(33))
    want = hda().qk_norm_rope(q, k, pos)
    got = hda().qk_norm_rope(q, k, pos, q_out=q, k_out=k)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    a, b = hda().qk_norm_rope(q[:0], k[:0], pos[:0])
    assert a.shape == (0, 4, 128) and b.shape == (0, 1, 128)


def test_norm_of_zeros_large_values_and_nan_stay_in_their_head():
    q = torch.zeros(4, 2, 64, device="cuda")
    q[1] = 1e18
    q[2, 0] = float("nan")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    qo, _ = hda().qk_norm_rope(q, q[:, :1], ints([0, 0, 0, 0]), q_gain=g, k_gain=g)
    assert (qo[0] == 0).all() and (qo[3] == 0).all() and (qo[2, 1] == 0).all()
    assert torch.equal(qo[1], torch.ones_like(qo[1])) and qo[2, 0].isnan().all()


def test_append_beyond_the_table_or_a_bad_page_stores_nothing():
    rng = np.random.default_rng(0)
    c, _ = make_cache(rng, [4, 20, 9], 8, 1, 64)
    c.table[1, 0] = 10 ** 6                       # positions 0..7 of sequence 1
    k0, v0 = c.k.clone(), c.v.clone()
    x = torch.randn(30, 3, 64, device="cuda")
    # six new rows where only four positions exist; twenty over a bad page; and a sequence id that does not exist
    out = c.append(0, x[:, :1], x[:, 1:2], x[:, 2:], ints([0, 6, 26, 30]), ints([0, 1, 3]))
    assert int(c.err.item()) == hda().MK_DEVERR_BAD_PAGE
    with pytest.raises(hda().MkError):
        c.sync()
    assert (out[:2] == 0).all() and (out[6:14] == 0).all() and (out[26:] == 0).all() and (out[2:6] != 0).any() and (out[14:26] != 0).any()
    c.sync()                                      # the word was cleared
    changed = (c.k != k0).any(-1).sum().item()
    assert changed == 4 + 12 and (c.v != v0).any(-1).sum().item() == 4 + 12


# ------------------------------------------------------------------ attention
def run_attention(seed, lens, new, hq, hkv, d, ps, scale=None, poison=True, layer=0, layers=1, q_scale=1.0, pad=0):
    rng = np.random.default_rng(seed)
    torch.manual_seed(seed)
    c, table = make_cache(rng, lens, ps, hkv, d, layers=layers)
    order = list(rng.permutation(len(lens)))
    start = np.concatenate([[0], np.cumsum([new[i] for i in order])]).astype(np.int32)
    rows = int(start[-1])
    q = (torch.randn(rows + 1, hq + pad, d, device="cuda") * q_scale).bfloat16()[:, :hq]
    keys = {i: (gather(c.k, layer, table[i], lens[i], ps), gather(c.v, layer, table[i], lens[i], ps)) for i in order}
    if poison:                                    # whatever is not a sequence's position is NaN
        keep = torch.zeros(c.k.shape[1], ps, dtype=torch.bool, device="cuda")
        for i, n in enumerate(lens):
            for j in range(ref.pages_of(n, ps)):
                keep[int(table[i, j]), :max(0, min(ps, n - j * ps))] = True
        mask = ~keep[None, :, None, :, None].expand_as(c.k)
        c.k[mask] = float("nan")
        c.v[mask] = float("nan")
    out = torch.full((rows + 1, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    c.attention(layer, q, ints(start), ints(order), scale=scale, out=out)
    c.sync()
    assert (out[rows:] == 3.0).all()              # the row behind the last sequence
    sc = scale if scale is not None else d ** -0.5
    for a, i in enumerate(order):
        if not new[i]:
            continue
        k, v = keys[i]
        pos = np.arange(lens[i] - new[i], lens[i])
        o, mag, big = ref.attention(f64(q[start[a]:start[a + 1]]), k, v, pos, sc)
        got = f64(out[start[a]:start[a + 1]])
        bound = ref.attention_bound(o, mag, big, sc, d)
        err = np.abs(got - o)
        assert np.all(err <= bound), (i, lens[i], new[i], float((err / bound).max()), np.argwhere(~(err <= bound))[:3])
        assert (got[pos < 0] == 0).all()          # rows that see nothing
    return out[:rows], c


@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 256, 64), (24, 4, 256, 16), (4, 1, 64, 8), (16, 4, 128, 48), (3, 3, 64, 128), (7, 1, 128, 24),
                                         (8, 1, 256, 256), (5, 1, 256, 32), (128, 1, 64, 16), (100, 1, 128, 32),
                                         (130, 2, 64, 64)])
def test_attention_ragged_lengths(hq, hkv, d, ps):
    lens = [1, 0, 64, 127, 128, 129, 300, 5, ps, 2 * ps + 1, 77]
    new = [1, 0, 1, 3, 128, 129, 44, 5, 1, 2 * ps, 0]
    run_attention(hq * d + ps, lens, new, hq, hkv, d, ps)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_decode_of_many_sequences(d):
    rng = random.Random(d)
    lens = [rng.randint(1, 700) for _ in range(100)]
    run_attention(d, lens, [1] * 100, 12, 2, d, 16)


@pytest.mark.parametrize("d,hq,hkv", [(256, 8, 2), (128, 6, 1), (64, 2, 2)])
def test_attention_long_context_few_rows(d, hq, hkv):
    """One sequence: its keys are split over the whole GPU and joined."""
    run_attention(d, [20011], [1], hq, hkv, d, 64)
    run_attention(d + 1, [9001, 3], [6, 2], hq, hkv, d, 32)


@pytest.mark.parametrize("d,hq,hkv", [(256, 8, 2), (128, 16, 4), (64, 4, 4)])
def test_attention_prompt(d, hq, hkv):
    run_attention(d, [1100], [1100], hq, hkv, d, 64)
    run_attention(d, [700, 1500], [333, 1], hq, hkv, d, 16, layer=1, layers=3, pad=3)


# prompts whose row tiles stay whole (one to seven for each of 148 CTAs), that are cut, and that are either way
# beside sequences without rows, without positions and with rows before the first position
@pytest.mark.parametrize("hq,hkv,d,lens,new", [(32, 4, 64, [900, 2100, 1500], [900, 2000, 700]), (8, 2, 256, [2600], [2600]),
                                               (16, 4, 128, [1900, 0, 1300, 40], [1700, 3, 0, 700]), (12, 2, 256, [70, 9000], [70, 400]),
                                               (64, 8, 64, [1700] * 2, [1650] * 2), (3, 1, 128, [1030] * 31 + [1], [128] * 31 + [1]),
                                               (128, 1, 64, [140, 1200], [140, 300]), (4, 4, 128, [513, 1, 2000], [300, 1, 1999])])
def test_attention_of_whole_row_tiles(hq, hkv, d, lens, new):
    run_attention(71, lens, new, hq, hkv, d, 16)


@pytest.mark.parametrize("d", [64, 256])
def test_attention_large_scores_and_scales(d):
    """Scores spanning hundreds of units, in both signs of the scale, and a scale of zero (the mean)."""
    for scale in (1.0, -0.7, 0.0):
        run_attention(3, [500, 200], [17, 200], 4, 2, d, 16, scale=scale, q_scale=4.0)


def test_attention_rows_that_see_nothing():
    """More new rows than positions: the first ones lie before position 0."""
    run_attention(9, [5, 0, 130], [9, 4, 200], 4, 2, 128, 16)


def test_attention_bad_pages_and_sequences():
    rng = np.random.default_rng(1)
    c, table = make_cache(rng, [300, 40], 16, 2, 128)
    c.table[0, 3] = -5
    c.table[0, 4] = c.k.shape[1]
    q = torch.randn(3, 4, 128, device="cuda").bfloat16()
    out = c.attention(0, q, ints([0, 1, 2, 3]), ints([0, 1, 2]))
    assert int(c.err.item()) == hda().MK_DEVERR_BAD_PAGE
    with pytest.raises(hda().MkError):
        c.sync()
    assert (out[2] == 0).all() and torch.isfinite(out.float()).all()
    k, v = gather(c.k, 0, table[1], 40, 16), gather(c.v, 0, table[1], 40, 16)
    o, mag, big = ref.attention(f64(q[1:2]), k, v, np.array([39]), 128 ** -0.5)
    assert np.all(np.abs(f64(out[1:2]) - o) <= ref.attention_bound(o, mag, big, 128 ** -0.5, 128))
    k, v = gather(c.k, 0, np.where(np.isin(np.arange(19), [3, 4]), 0, table[0]), 300, 16), gather(c.v, 0, np.where(np.isin(np.arange(19), [3, 4]), 0, table[0]), 300, 16)
    k[48:80], v[48:80] = 0, 0                     # bad pages read as zeros
    o, mag, big = ref.attention(f64(q[:1]), k, v, np.array([299]), 128 ** -0.5)
    assert np.all(np.abs(f64(out[:1]) - o) <= ref.attention_bound(o, mag, big, 128 ** -0.5, 128))


def test_attention_of_many_short_sequences():
    """More sequences than one round of the kernel's lookup takes."""
    rng = random.Random(4)
    lens = [rng.randint(0, 40) for _ in range(1300)]
    run_attention(11, lens, [min(n, rng.choice([0, 1, 1, 2])) for n in lens], 2, 1, 64, 8)


def test_rows_before_and_between_sequences():
    """The first sequence need not start at row 0; rows outside stay as they are."""
    rng = np.random.default_rng(3)
    c, table = make_cache(rng, [40, 70], 16, 2, 128)
    x = torch.randn(20, 8, 128, device="cuda")
    out = torch.full((20, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    c.append(0, x[:, :4], x[:, 4:6], x[:, 6:], ints([7, 7, 12]), ints([0, 1]), out=out)
    q = out.clone()
    o = torch.full_like(out, 5.0)
    c.attention(0, q, ints([7, 7, 12]), ints([0, 1]), out=o)
    c.sync()
    for t in (out, o):
        assert (t[:7] == 5.0).all() and (t[12:] == 5.0).all() and (t[7:12] != 5.0).any()
    k, v = gather(c.k, 0, table[1], 70, 16), gather(c.v, 0, table[1], 70, 16)
    want, mag, big = ref.attention(f64(q[7:12]), k, v, np.arange(65, 70), 128 ** -0.5)
    assert np.all(np.abs(f64(o[7:12]) - want) <= ref.attention_bound(want, mag, big, 128 ** -0.5, 128))


def test_pages_further_apart_than_32_bits():
    """Pages, layers and heads 2^31 entries and more from each other."""
    m, far = hda(), (1 << 30) + 4096
    big = [torch.empty(2 * far + far // 2 + 65536, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv = [t.as_strided((2, 3, 1, 16, 128), (far // 2, far, 16 * 128, 128, 1)) for t in big]   # [layers][pages][heads][slots][d]
    c = m.PagedCache(kv[0], kv[1], torch.full((3, 3), -1, dtype=torch.int32, device="cuda"), ints([0, 0, 0]), ints([0, 0, 0]))
    c.resize(ints([0]), ints([8]))
    c.resize(ints([1]), ints([8]))
    c.free(ints([0]))
    c.resize(ints([1]), ints([40]))                # pages 1, 0, 2
    assert c.table[1].tolist() == [1, 0, 2]
    for layer in range(2):
        x = torch.randn(40, 6, 128, device="cuda")
        q = c.append(layer, x[:, :4], x[:, 4:5], x[:, 5:], ints([0, 40]), ints([1]))
        o = c.attention(layer, q, ints([0, 40]), ints([1]))
        c.sync()
        row = c.table[1].cpu().numpy()
        k, v = gather(c.k, layer, row, 40, 16), gather(c.v, layer, row, 40, 16)
        assert np.array_equal(v[:, 0], f64(x[:, 5].bfloat16()))
        want, mag, s = ref.attention(f64(q), k, v, np.arange(40), 128 ** -0.5)
        assert np.all(np.abs(f64(o) - want) <= ref.attention_bound(want, mag, s, 128 ** -0.5, 128))
    c.copy_pages(ints([2]), ints([0]))
    c.sync()
    assert torch.equal(c.k[:, 0], c.k[:, 2]) and torch.equal(c.v[:, 0], c.v[:, 2])


def test_two_calls_at_once():
    """Two caches worked on in two streams at the same time, eager and captured."""
    rng = np.random.default_rng(5)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work, want = [], []
    for i in range(2):
        c, table = make_cache(rng, [3000 + i, 77], 16, 2, 128)
        q = torch.randn(90, 8, 128, device="cuda").bfloat16()
        start = ints([0, 60, 90])
        work.append((c, q, start))
        want.append(c.attention(0, q, start))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (c, q, start) in enumerate(work):
            got[i].append(c.attention(0, q, start, stream=streams[i]))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, q, start in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.attention(0, q, start))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for i, g in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            got[i].append(outs[i].clone())
    for i in range(2):
        work[i][0].sync()
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_attention_is_the_same_every_time():
    lens, new = [3000, 17, 900, 1, 250], [1, 17, 33, 1, 250]
    a, _ = run_attention(4, lens, new, 8, 2, 256, 32)
    b, _ = run_attention(4, lens, new, 8, 2, 256, 32)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ pages
def signature(cache, pages):
    """Page contents that stand for `pages.slot`: every entry of a slot is its number."""
    x = torch.from_numpy(pages.slot.astype(np.float32)).cuda()
    for t in (cache.k, cache.v):
        t.copy_(x[None, :, None, :, None].expand_as(t).bfloat16())


def same(cache, pages):
    assert np.array_equal(cache.table.cpu().numpy(), pages.table)
    assert np.array_equal(cache.len.cpu().numpy(), pages.len)
    assert np.array_equal(cache.ref.cpu().numpy(), pages.ref)
    for s, n in enumerate(pages.len):             # what each sequence holds
        for j in range(ref.pages_of(int(n), pages.ps)):
            m = min(pages.ps, int(n) - j * pages.ps)
            want = torch.from_numpy(pages.slot[pages.table[s, j], :m].astype(np.float32)).cuda()
            for t in (cache.k, cache.v):
                got = t[:, int(pages.table[s, j]), :, :m].float()
                assert torch.equal(got, want[None, None, :, None].expand_as(got))


@pytest.mark.parametrize("ps,n_pages,n_seqs,d,seed", [(8, 40, 6, 64, 0), (16, 300, 40, 128, 1), (24, 9000, 70, 64, 2), (64, 30, 3, 256, 3)])
def test_random_page_operations(ps, n_pages, n_seqs, d, seed):
    rng = random.Random(seed)
    mp = 9
    c = hda().PagedCache.empty(2, n_pages, 2, ps, d, n_seqs, mp)
    p = ref.Pages(n_pages, n_seqs, mp, ps)
    mark = 0
    for step in range(60):
        ids = rng.sample(range(n_seqs), rng.randint(1, n_seqs))
        op = rng.choice("rrrfffc")
        ok = True
        if op == "r":
            lens = [rng.choice([0, rng.randint(0, ps * mp), rng.randint(0, ps), rng.randint(0, mp) * ps, int(p.len[i])]) for i in ids]
            c.resize(ints(ids), ints(lens))
            ok = p.resize(ids, lens)
        elif op == "f" and len(ids) > 1:
            cut = rng.randint(1, len(ids) - 1)
            src = [rng.choice(ids[:cut]) for _ in ids[cut:]]
            c.fork(ints(src), ints(ids[cut:]))
            ok = p.fork(src, ids[cut:])
        elif op == "c":
            c.compact()
            p.compact()
        assert int(c.err.item()) == (0 if ok else hda().MK_DEVERR_NO_PAGES)
        c.err.zero_()
        same(c, p)
        # new contents in every used page (values that bf16 holds exactly)
        for q in range(n_pages):
            if p.ref[q]:
                mark += 1
                p.slot[q] = (np.arange(ps) + mark * 7) % 251
        signature(c, p)
    assert p.len.sum() > 0


def test_large_tables():
    """More sequences in a call than a plan keeps in shared memory (1024) and more pages than it counts there
    (49152): tables, lengths and counts against the loops."""
    rng = random.Random(8)
    c = hda().PagedCache.empty(1, 60001, 1, 8, 64, 1500, 40)
    p = ref.Pages(60001, 1500, 40, 8)

    def check(ok):
        assert int(c.err.item()) == (0 if ok else hda().MK_DEVERR_NO_PAGES)
        c.err.zero_()
        for t, w in ((c.table, p.table), (c.len, p.len), (c.ref, p.ref)):
            assert np.array_equal(t.cpu().numpy(), w)

    def resize(ids, lens):
        c.resize(ints(ids), ints(lens))
        check(p.resize(ids, lens))

    resize(list(range(1500)), [rng.randint(200, 320) for _ in range(1500)])   # past the 49152nd page
    resize(list(range(1500)), [320] * 1500)
    ids = rng.sample(range(1500), 1200)
    resize(ids, [rng.randint(0, 320) for _ in ids])
    dst = rng.sample(range(1500), 1100)
    src = [rng.choice([i for i in range(1500) if i not in set(dst)]) for _ in range(3)]
    src = [rng.choice(src) for _ in dst]
    c.fork(ints(src), ints(dst))
    check(p.fork(src, dst))
    resize(dst[:1050], [rng.randint(0, 320) for _ in dst[:1050]])             # shared pages cut in the middle
    c.compact()
    p.compact()
    check(True)


def test_free_and_zero_lengths():
    c = hda().PagedCache.empty(1, 20, 1, 8, 64, 5, 4)
    c.resize(ints([4, 0, 2]), ints([32, 0, 9]))
    c.sync()
    assert c.table[4].tolist() == [0, 1, 2, 3] and c.table[2].tolist() == [4, 5, -1, -1] and c.len.tolist() == [0, 0, 9, 0, 32]
    c.free(ints([4, 1]))
    c.resize(ints([]), ints([]))
    c.fork(ints([]), ints([]))
    c.free(ints([]))
    c.sync()
    assert c.table[4].tolist() == [-1] * 4 and c.ref.tolist() == [0] * 4 + [1, 1] + [0] * 14 and c.len.tolist() == [0, 0, 9, 0, 0]


def test_a_truncated_shared_page_gets_its_own_copy():
    c = hda().PagedCache.empty(1, 12, 1, 8, 64, 3, 4)
    c.resize(ints([0]), ints([24]))
    c.k.normal_()
    c.v.normal_()
    c.fork(ints([0, 0]), ints([1, 2]))
    k0 = c.k.clone()
    c.resize(ints([1, 2]), ints([12, 17]))        # ends inside the shared pages 1 and 2
    c.sync()
    t = c.table.tolist()
    assert t == [[0, 1, 2, -1], [0, 3, -1, -1], [0, 1, 4, -1]] and c.ref.tolist() == [3, 2, 1, 1, 1] + [0] * 7
    assert torch.equal(c.k[0, 3, 0, :4], k0[0, 1, 0, :4]) and torch.equal(c.k[0, 4, 0, :1], k0[0, 2, 0, :1])
    assert torch.equal(c.k[0, 3, 0, 4:], k0[0, 3, 0, 4:]) and torch.equal(c.k[0, :3], k0[0, :3])   # only used slots move


def test_calls_that_fail_change_nothing():
    m = hda()
    c = m.PagedCache.empty(1, 6, 1, 8, 64, 4, 5)
    c.resize(ints([0, 1]), ints([20, 9]))
    c.sync()
    snap = [t.clone() for t in (c.table, c.len, c.ref)]

    def unchanged(bit):
        assert int(c.err.item()) == bit
        c.err.zero_()
        for t, s in zip((c.table, c.len, c.ref), snap):
            assert torch.equal(t, s)

    c.resize(ints([0, 2]), ints([8, 33]))          # gives two back, wants five of three
    unchanged(m.MK_DEVERR_NO_PAGES)
    for seqs, lens in (([0, 0], [1, 2]), ([4], [1]), ([-1], [1]), ([2], [41]), ([2], [-1])):
        c.resize(ints(seqs), ints(lens))
        unchanged(m.MK_DEVERR_BAD_PAGE)
    for a, b in (([0], [0]), ([0, 1], [2, 2]), ([0, 2], [2, 3]), ([5], [2]), ([0], [-1])):
        c.fork(ints(a), ints(b))
        unchanged(m.MK_DEVERR_BAD_PAGE)
    c.resize(ints([2]), ints([8]))                 # one page left
    c.sync()
    c.table[1, 1] = 6
    snap = [t.clone() for t in (c.table, c.len, c.ref)]
    c.fork(ints([1]), ints([3]))                   # a page that does not exist
    unchanged(m.MK_DEVERR_BAD_PAGE)
    c.free(ints([1]))
    unchanged(m.MK_DEVERR_BAD_PAGE)


def test_copy_between_caches_of_other_strides_and_bad_ids():
    m = hda()
    a = m.PagedCache.empty(3, 7, 2, 16, 128, 1, 1)
    kv = [torch.randn(3, 2, 9, 16, 128, device="cuda").bfloat16().transpose(1, 2) for _ in range(2)]
    b = m.PagedCache(kv[0], kv[1], ints([0]).view(1, 1), ints([0]), ints([0] * 9))
    k0 = a.k.clone()
    a.copy_pages(ints([8, 0, 3, 9, -1, 2]), ints([1, 6, 0, 2, 3, 7]), source=b)   # the last three name no page
    with pytest.raises(m.MkError):
        a.sync()
    for t, s in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(t[:, 1], s[:, 8]) and torch.equal(t[:, 6], s[:, 0]) and torch.equal(t[:, 0], s[:, 3])
    assert torch.equal(a.k[:, 2:6], k0[:, 2:6])
    a.copy_pages(ints([0, 1]), ints([2, 3]))
    a.sync()
    assert torch.equal(a.k[:, 2:4], a.k[:, 0:2]) and torch.equal(a.v[:, 2:4], a.v[:, 0:2])


# ------------------------------------------------------------------ together
def test_continuations_of_a_prompt():
    """A prompt in two chunks, three continuations forked from it, steps of one and of several tokens with a compaction
    and a truncation between: every step's attention against float64 over the tokens' own history."""
    torch.manual_seed(0)
    rng = random.Random(0)
    hq, hkv, d, ps, layers = 8, 2, 256, 16, 2
    c = hda().PagedCache.empty(layers, 120, hkv, ps, d, 6, 40)
    gains = [(1 + 0.1 * torch.randn(d, device="cuda")).bfloat16() for _ in range(2)]
    c.resize(ints([0, 5]), ints([100, 200]))       # an older session whose end leaves holes
    hist = {0: [], 1: [], 2: [], 3: []}            # per sequence: rotated keys and values of both layers

    def step(seqs, news):
        lens = [len(hist[s]) + n for s, n in zip(seqs, news)]
        c.resize(ints(seqs), ints(lens))
        start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        for layer in range(layers):
            x = torch.randn(int(start[-1]), hq + 2 * hkv, d, device="cuda")
            q = c.append(layer, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], ints(start), ints(seqs), q_gain=gains[0], k_gain=gains[1])
            o = c.attention(layer, q, ints(start), ints(seqs))
            for a, (s, n) in enumerate(zip(seqs, news)):
                r = slice(int(start[a]), int(start[a + 1]))
                pos = np.arange(lens[a] - n, lens[a])
                want, mag = ref.rope(f64(x[r, hq:hq + hkv]), f64(gains[1]), pos, d, 1e-6, 1e7)
                pages = c.table[s].cpu().numpy()
                k, v = gather(c.k, layer, pages, lens[a], ps), gather(c.v, layer, pages, lens[a], ps)
                assert np.all(np.abs(k[-n:] - want) <= BF16_HALF_STEP * np.abs(want) + 2.0 ** -18 * mag)
                for t in range(n):                 # the history is what was appended, through forks and moves
                    if layer == 0:
                        hist[s].append([None, None])
                    hist[s][lens[a] - n + t][layer] = (k[lens[a] - n + t], v[lens[a] - n + t])
                hk, hv = (np.stack([h[layer][i] for h in hist[s]]) for i in (0, 1))
                assert np.array_equal(hk, k) and np.array_equal(hv, v)
                oo, m2, big = ref.attention(f64(q[r]), hk, hv, pos, d ** -0.5)
                assert np.all(np.abs(f64(o[r]) - oo) <= ref.attention_bound(oo, m2, big, d ** -0.5, d))
        c.sync()

    c.free(ints([0]))
    step([0], [150])
    step([0], [33])
    c.fork(ints([0, 0, 0]), ints([1, 2, 3]))
    for s in (1, 2, 3):
        hist[s] = [list(h) for h in hist[0]]
    step([2, 0, 3, 1], [1, 1, 1, 1])
    c.free(ints([5]))
    c.compact()
    step([1, 3], [6, 2])
    c.resize(ints([1]), ints([len(hist[1]) - 4]))  # drafts that were not accepted
    hist[1] = hist[1][:-4]
    step([0, 1, 2, 3], [rng.randint(1, 5) for _ in range(4)])
    used = [p for row, n in zip(c.table.tolist(), c.len.tolist()) for p in row[:ref.pages_of(n, ps)]]
    assert np.array_equal(np.bincount(used, minlength=120), c.ref.cpu().numpy())


def test_model_cache_as_pages():
    """A tiny model's prompt: attention over its own cache, and its pages kept in a pool and put back."""
    m = hda()
    cfg = synth.TINY
    model = m.Model(cfg, m.weights_to_device(synth.make_weights(cfg)), max_ctx=128)
    prompt = torch.from_numpy(synth.make_prompt(cfg, 70)).cuda()
    model.prefill(prompt)
    pages = model.kv_pages(16)
    assert pages.len.item() == 70
    for call in (lambda: pages.resize(ints([0]), ints([1])), lambda: pages.free(ints([0])), lambda: pages.fork(ints([0]), ints([0])),
                 pages.compact):
        with pytest.raises(ValueError):
            call()
    q = torch.randn(3, cfg.at_q_heads, cfg.at_head_dim, device="cuda").bfloat16()
    o = pages.attention(0, q, ints([0, 3]))
    k, v = (f64(t[0].transpose(0, 1)[:70]) for t in (model.k_cache, model.v_cache))
    sc = cfg.at_head_dim ** -0.5
    want, mag, big = ref.attention(f64(q), k, v, np.arange(67, 70), sc)
    assert np.all(np.abs(f64(o) - want) <= ref.attention_bound(want, mag, big, sc, cfg.at_head_dim))
    pool = m.PagedCache.empty(cfg.n_at, 12, cfg.at_kv_heads, 16, cfg.at_head_dim, 1, 8)
    pool.resize(ints([0]), ints([70]))
    pool.copy_pages(ints(range(5)), pool.table[0, :5].contiguous(), source=pages)
    pool.sync()
    k0, S, conv = model.k_cache.clone(), model.S.clone(), model.conv_history.clone()
    tok, nxt, l1, l2 = ints([5]), ints([0]), torch.empty(cfg.vocab, device="cuda"), torch.empty(cfg.vocab, device="cuda")
    model.decode(tok, nxt, l1)
    model.sync()
    model.reset()                                  # another prompt, then the kept one again
    model.prefill(prompt[:9])
    pages.copy_pages(pool.table[0, :5].contiguous(), ints(range(5)), source=pool)
    model.S.copy_(S)
    model.conv_history.copy_(conv)
    model.set_position(70)
    assert torch.equal(model.k_cache[:, :, :70], k0[:, :, :70])
    model.decode(tok, nxt, l2)
    model.sync()
    # the same state; the decode kernel adds its residual parts with fp32 reductions whose order
    # differs from launch to launch, so its logits agree to the parity tests' bound, not to the bit
    assert float((l1 - l2).abs().max()) <= 3e-2


def test_captured_calls_follow_lengths_and_tables():
    """One captured step replayed on new lengths, tables and inputs, on a stream of its own."""
    torch.manual_seed(3)
    c = hda().PagedCache.empty(1, 64, 2, 16, 128, 3, 20)
    seqs, lens, start = ints([0, 2]), ints([10, 33]), ints([0, 1, 2])
    x = torch.randn(2, 10, 128, device="cuda")

    def step():
        c.resize(seqs, lens)
        q = c.append(0, x[:, :6], x[:, 6:8], x[:, 8:], start, seqs)
        return q, c.attention(0, q, start, seqs)

    c.k.normal_()
    c.v.normal_()
    step()                                         # loads the kernels before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq, go = step()
    side = torch.cuda.Stream()
    for a, b in ((11, 34), (12, 300), (1, 301), (320, 16)):
        lens.copy_(ints([a, b]))
        x.normal_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        assert int(c.err.item()) == 0
        for i, (s, n) in enumerate(((0, a), (2, b))):
            row = c.table[s].cpu().numpy()
            k, v = gather(c.k, 0, row, n, 16), gather(c.v, 0, row, n, 16)
            want, mag, big = ref.attention(f64(gq[i:i + 1]), k, v, np.array([n - 1]), 128 ** -0.5)
            assert np.all(np.abs(f64(go[i:i + 1]) - want) <= ref.attention_bound(want, mag, big, 128 ** -0.5, 128))


def test_captured_prompts_whole_and_cut():
    """One captured call replayed on lengths whose row tiles stay whole, are cut, and stay whole again."""
    torch.manual_seed(4)
    c = hda().PagedCache.empty(1, 500, 2, 16, 64, 2, 400)
    rows = 700
    seqs, lens, start = ints([1, 0]), ints([350, 350]), ints([0, 350, rows])
    q = torch.randn(rows, 8, 64, device="cuda").bfloat16()
    c.k.normal_()
    c.v.normal_()
    c.resize(seqs, lens)
    c.attention(0, q, start, seqs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.resize(seqs, lens)
        out = c.attention(0, q, start, seqs)
    for a, b, cut in ((400, 360, 350), (2, 6300, 2), (1200, 330, 300)):
        lens.copy_(ints([a, b]))
        start.copy_(ints([0, cut, rows]))
        out.fill_(7.0)
        g.replay()
        assert int(c.err.item()) == 0
        for s, n, lo, hi in ((1, a, 0, cut), (0, b, cut, rows)):
            row = c.table[s].cpu().numpy()
            k, v = gather(c.k, 0, row, n, 16), gather(c.v, 0, row, n, 16)
            pos = np.arange(n - (hi - lo), n)
            want, mag, big = ref.attention(f64(q[lo:hi]), k, v, pos, 64 ** -0.5)
            assert np.all(np.abs(f64(out[lo:hi]) - want) <= ref.attention_bound(want, mag, big, 64 ** -0.5, 64))
            assert (out[lo:hi][torch.from_numpy(pos < 0).cuda()] == 0).all()


def test_captured_page_calls():
    """Fork, resize and compaction captured once and replayed on changed lists."""
    c = hda().PagedCache.empty(2, 60, 2, 8, 64, 6, 8)
    p = ref.Pages(60, 6, 8, 8)
    src, dst, seqs, lens = ints([0]), ints([1]), ints([0, 2]), ints([0, 0])
    c.fork(src, dst)                               # loads the kernels before the capture
    c.resize(seqs, lens)
    c.compact()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.resize(seqs, lens)
        c.fork(src, dst)
        c.compact()
    rng = random.Random(3)
    for step in range(12):
        ids = rng.sample(range(6), 2)
        new = [rng.randint(0, 40), rng.randint(0, 40)]
        a, b = rng.sample(range(6), 2)
        for t, v in ((seqs, ids), (lens, new), (src, [a]), (dst, [b])):
            t.copy_(ints(v))
        for q in range(60):
            p.slot[q] = (np.arange(8) + 8 * q + step) % 251
        signature(c, p)
        g.replay()
        c.sync()
        assert p.resize(ids, new) and p.fork([a], [b])
        p.compact()
        same(c, p)


def test_calls_on_another_stream():
    s = torch.cuda.Stream()
    rng = np.random.default_rng(2)
    c, table = make_cache(rng, [400], 16, 1, 64)
    q = torch.randn(1, 2, 64, device="cuda").bfloat16()
    torch.cuda.synchronize()
    o = c.attention(0, q, ints([0, 1]), stream=s)
    c.sync(s)
    assert torch.equal(o, c.attention(0, q, ints([0, 1])))


def test_binding_refusals():
    m = hda()
    c = m.PagedCache.empty(1, 4, 2, 8, 64, 2, 2)
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    start = ints([0, 2])
    for bad in (lambda: c.attention(0, q.float(), start), lambda: c.attention(0, q[:, :, :32], start), lambda: c.attention(0, q.cpu(), start),
                lambda: c.attention(0, q, start.long()), lambda: c.attention(0, q, start, ints([0, 1])),
                lambda: c.attention(0, q.transpose(0, 1), start), lambda: c.attention(0, q, ints([0, 1, 1, 2])),
                lambda: c.append(0, q, q[:, :1], q[:, :1], start), lambda: c.append(0, q, q[:, :2], q[:, :2].float(), start),
                lambda: c.resize(start, ints([0])), lambda: c.fork(ints([0]), ints([])), lambda: c.copy_pages(ints([0]), ints([1, 2])),
                lambda: m.qk_norm_rope(q, q[:1], ints([0, 1])), lambda: m.qk_norm_rope(q, q, ints([0])),
                lambda: m.PagedCache(c.k, c.v.float(), c.table, c.len, c.ref), lambda: m.PagedCache(c.k, c.v, c.table, c.len[:1], c.ref),
                lambda: m.PagedCache(c.k[..., ::2], c.v[..., ::2], c.table, c.len, c.ref)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: c.attention(1, q, start), lambda: c.attention(0, q[:, :3], start), lambda: c.append(0, q, q[:, :2], q[:, :2], start, rot_dim=10),
                lambda: c.copy_pages(ints([0]), ints([1]), source=m.PagedCache.empty(2, 4, 2, 8, 64, 1, 1))):
        with pytest.raises(m.MkError):
            bad()
