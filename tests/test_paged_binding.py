"""The paged binding's own state, on the CPU: a cache whose library and streams are stand-ins."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


class Library:
    """Scratch of 1000 bytes a row; notes whether the tensors' device was current when it was asked."""

    def __init__(self):
        self.inside, self.asked, self.calls = 0, [], []

    def mk_paged_attention_scratch(self, cache, rows, heads):
        self.asked.append(self.inside)
        return 1000 * rows + heads

    def mk_paged_attention(self, cache, layer, q, ldq, rows, heads, start, seqs, n, scale, out, ldo, scratch, size, stream):
        self.calls.append((rows, heads, size))
        return 0


@pytest.fixture
def cache(monkeypatch):
    from hybrid_deltanet_attention_b200 import paged
    c, lib = object.__new__(paged.PagedCache), Library()
    c.lib, c._attention, c._p = lib, lib.mk_paged_attention, None
    c.device, c._index, c._d, c._n_seqs, c._kv_heads, c._scale = torch.device("cpu"), -1, 64, 4, 1, 0.125
    c._scratch = (0, 0, 0)
    c._bytes = torch.empty(0, dtype=torch.uint8)
    c.between = lambda: None                       # what another thread does while this one is inside the call

    @contextlib.contextmanager
    def on(device, stream):
        lib.inside += 1
        c.between()
        yield 0
        lib.inside -= 1

    monkeypatch.setattr(paged, "_on", on)
    monkeypatch.setattr(paged.PagedCache, "_first_use", lambda self, stream: None, raising=False)
    return c


def attention(c, rows, heads=2):
    return c.attention(0, torch.zeros(rows, heads, 64, dtype=torch.bfloat16), torch.tensor([0, rows], dtype=torch.int32))


def test_scratch_is_asked_for_on_the_tensors_device(cache):
    for rows in (3, 3, 5, 3):
        attention(cache, rows)
    assert cache.lib.asked == [1, 1, 1]            # once per change of shape, inside
    assert cache.lib.calls == [(3, 2, 3002), (3, 2, 3002), (5, 2, 5002), (3, 2, 3002)]


def test_scratch_is_of_the_calls_own_shape_whatever_other_threads_call(cache):
    attention(cache, 3)

    def other():
        cache.between = lambda: None
        attention(cache, 7, 1)

    cache.between = other
    attention(cache, 3)
    assert cache.lib.calls == [(3, 2, 3002), (7, 1, 7001), (3, 2, 3002)]
