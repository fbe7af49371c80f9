"""Order inside and between paged-cache calls: roles of the attention kernel that run late, streams, devices and threads."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

import test_gpu_paged as base

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def late_build(d, ns):
    """mk_paged_attention of a build in which one softmax group waits `ns` before it reads a row tile's results."""
    from hybrid_deltanet_attention_b200 import _abi, build
    obj, so = str(d / "paged_attn.o"), str(d / f"libmk_late_{ns}.so")
    flags = [f for f in build.FLAGS if f != "-shared"]
    src = os.path.join(build.CSRC, "paged_attn.cu")
    subprocess.check_call([build.nvcc(), *build.ARCH, *flags, f"-DMK_TEST_SLOW_EPILOGUE_NS={ns}ull", "-c", src, "-o", obj])
    subprocess.check_call([build.nvcc(), *build.ARCH, "-shared", "-Xcompiler", "-fPIC", obj, build.LIB, "-o", so])
    fn = C.CDLL(so).mk_paged_attention
    own = _abi.load_library().mk_paged_attention
    fn.argtypes, fn.restype = own.argtypes, own.restype
    assert C.cast(fn, C.c_void_p).value != C.cast(own, C.c_void_p).value
    return fn


@pytest.fixture(scope="module")
def late_reader(tmp_path_factory):
    return late_build(tmp_path_factory.mktemp("late_reader"), 20000)


# CTAs with several row tiles: cut ones with partial results, whole ones, and both kinds beside empty sequences
@pytest.mark.parametrize("hq,hkv,d,lens,new", [(8, 2, 256, [2600], [2600]), (8, 2, 256, [70, 9000, 0, 300], [70, 400, 2, 300]),
                                               (16, 4, 128, [1900, 1300, 40], [1700, 3, 40]), (16, 4, 128, [200] * 150, [3] * 150),
                                               (32, 4, 64, [900, 2100, 1500], [900, 2000, 700]), (12, 2, 64, [500, 77] * 60, [1] * 120)])
def test_a_row_tile_read_late_keeps_its_results(late_reader, monkeypatch, hq, hkv, d, lens, new):
    """The next row tile's first product must not overwrite O while a softmax group still reads the one before."""
    want, _ = base.run_attention(31, lens, new, hq, hkv, d, 16)
    cls = base.hda().PagedCache
    init = cls.__init__

    def late(self, *a, **kw):
        init(self, *a, **kw)
        self._attention = late_reader

    monkeypatch.setattr(cls, "__init__", late)
    got, c = base.run_attention(31, lens, new, hq, hkv, d, 16)   # against float64 too
    assert c._attention is late_reader and torch.equal(got, want)


def test_a_wait_that_gives_up_ends_the_call_with_an_error(tmp_path):
    """A group that reads 1.3 s late outlasts the kernel's waits of one second: every role gives up, what is in flight ends,
    the call reports it, and the next call is right again."""
    m = base.hda()
    rng = np.random.default_rng(1)
    c, table = base.make_cache(rng, [2600], 16, 2, 128)
    q, start = torch.randn(2600, 8, 128, device="cuda").bfloat16(), base.ints([0, 2600])
    want, own = c.attention(0, q, start), c._attention
    c.sync()
    c._attention = late_build(tmp_path, 1300000000)
    c.attention(0, q, start)
    with pytest.raises(m.MkError, match="gave up"):
        c.sync()
    c._attention = own
    got = c.attention(0, q, start)
    c.sync()
    assert torch.equal(got, want)


# ------------------------------------------------------------------ streams
BUSY = 200_000_000                                 # clocks that a stream is kept busy, about 0.1 s


def test_a_cache_dropped_after_a_call_on_a_given_stream():
    """Its table and its own arrays are not given to anything else while the call still waits on that stream."""
    m = base.hda()
    torch.manual_seed(0)
    c, table = base.make_cache(np.random.default_rng(0), [900, 700], 16, 2, 64)
    q, start, s = torch.randn(60, 4, 64, device="cuda").bfloat16(), base.ints([0, 20, 60]), torch.cuda.Stream()
    want = c.attention(0, q, start)
    c.sync()
    other = torch.flip(c.table, (0,)).contiguous()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    got = m.PagedCache(c.k, c.v, c.table.clone(), c.len.clone(), c.ref.clone()).attention(0, q, start, stream=s)
    keep = [torch.full_like(c.len, 3) for _ in range(64)] + [other.clone() for _ in range(64)] + [torch.ones_like(c.err) for _ in range(64)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(keep) == 192


def test_a_source_cache_dropped_after_a_copy_on_a_given_stream():
    m = base.hda()
    to, s = m.PagedCache.empty(1, 4, 2, 16, 64, 1, 1), torch.cuda.Stream()
    fr = m.PagedCache.empty(1, 4, 2, 16, 64, 1, 1)
    fr.k.normal_()
    fr.v.normal_()
    k, v, ids = fr.k.clone(), fr.v.clone(), base.ints(range(4))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    to.copy_pages(ids, ids, source=fr, stream=s)
    del fr
    keep = [torch.zeros_like(k) for _ in range(64)]
    torch.cuda.synchronize()
    assert torch.equal(to.k, k) and torch.equal(to.v, v) and len(keep) == 64


def test_the_error_word_is_in_order_with_the_calls_of_a_stream():
    """It is cleared before the first call on any stream, and sync(stream) reads and clears it between that stream's calls."""
    m = base.hda()
    s, seqs, lens = torch.cuda.Stream(), base.ints([9]), base.ints([1])       # a sequence that does not exist
    t = m.PagedCache.empty(1, 4, 1, 8, 64, 2, 2)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)                        # the current stream is busy: a new cache's arrays are cleared after that
    c = m.PagedCache(t.k, t.v, t.table, t.len, t.ref)
    c.resize(seqs, lens, stream=s)
    with pytest.raises(m.MkError):
        c.sync(s)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    c.resize(seqs, lens, stream=s)
    with pytest.raises(m.MkError):
        c.sync(s)
    c.resize(seqs, lens, stream=s)                 # a second error, while the current stream is still busy
    torch.cuda.synchronize()
    with pytest.raises(m.MkError):
        c.sync(s)
    c.sync(s)
    c.sync()


def test_a_call_on_a_stream_of_another_device_is_refused():
    m = base.hda()
    c = m.PagedCache.empty(1, 4, 1, 8, 64, 2, 2)

    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 7), 12345

    for call in (lambda: c.compact(stream=Elsewhere()), lambda: c.sync(Elsewhere())):
        with pytest.raises(ValueError, match="the stream is on"):
            call()
