"""Attention over values that name their key tile, so that a result shows which tiles it was made of: with random values the
sum over a long context is about as small as what its roundings may add up to."""
import numpy as np
import pytest

import paged_ref as ref

TILE = 128


def named_values(n, d):
    """Entry e of a position's value is 1 for its tile of 128 (columns in turn), 0 otherwise."""
    return (np.arange(n)[:, None] // TILE % d == np.arange(d)[None, :]).astype(np.float64)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [9001, 20011])
def test_a_lost_or_mistaken_tile_is_far_outside_the_bound(n, d):
    rng = np.random.default_rng(d)
    q, k, v = rng.standard_normal((1, 1, d)), rng.standard_normal((n, 1, d)), named_values(n, d)[:, None]
    pos, sc = np.array([n - 1]), d ** -0.5
    o, mag, big = ref.attention(q, k, v, pos, sc)
    bound = ref.attention_bound(o, mag, big, sc, d)
    w = np.exp(q[0, 0] @ k[:, 0].T * sc)
    tiles = -(-n // TILE)
    for t in range(tiles):
        rest = np.ones(n)
        rest[t * TILE:(t + 1) * TILE] = 0
        lost = (w * rest) @ v[:, 0] / (w * rest).sum()
        at = np.arange(n)
        at[t * TILE:(t + 1) * TILE] = (at[t * TILE:(t + 1) * TILE] + TILE) % (n // TILE * TILE)
        other = w[at] @ v[at, 0] / w[at].sum()
        for got in (lost, other):
            assert (np.abs(got - o[0, 0]) / bound[0, 0]).max() >= 10, t


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(256, 8, 2), (128, 16, 4), (64, 4, 4)])
@pytest.mark.parametrize("lens,new", [([20011], [1]), ([9001, 5], [6, 5]), ([9001], [80]), ([900, 6000], [1, 700]), ([2600], [2600])])
def test_attention_takes_every_tile_once(d, hq, hkv, lens, new):
    """A decoded token, drafts, a chunk and prompts over keys that are cut over the whole GPU, and row tiles that stay whole."""
    import test_gpu_paged as base
    torch = base.torch
    torch.manual_seed(2)
    c, table = base.make_cache(np.random.default_rng(1), lens, 16, hkv, d)
    for i, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        page = torch.from_numpy(table[i]).long().cuda()[at // 16]
        c.v[0, page, :, at % 16] = torch.from_numpy(named_values(n, d)).cuda().bfloat16()[:, None].expand(n, hkv, d)
    start = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn(int(start[-1]), hq, d, device="cuda").bfloat16()
    out = c.attention(0, q, base.ints(start))
    c.sync()
    for i, n in enumerate(lens):
        rows = slice(int(start[i]), int(start[i + 1]))
        k, v = base.gather(c.k, 0, table[i], n, 16), base.gather(c.v, 0, table[i], n, 16)
        want, mag, big = ref.attention(base.f64(q[rows]), k, v, np.arange(n - new[i], n), d ** -0.5)
        err = np.abs(base.f64(out[rows]) - want)
        assert np.all(err <= ref.attention_bound(want, mag, big, d ** -0.5, d)), (i, n)
