"""The paged-cache entry points refuse bad arguments on the host, before any device call (fake
addresses are never touched), and the plain page accounting keeps its own invariants."""
import ctypes as C
import os
import random
import subprocess

import numpy as np
import pytest

from paged_ref import Pages, pages_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000   # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from hybrid_deltanet_attention_b200 import _abi, build
    build.build()
    return _abi.load_library()


def cache(**kw):
    from hybrid_deltanet_attention_b200 import _abi
    c = _abi.MkPagedCache()
    v = dict(k=A, v=A, layer_stride=1 << 20, page_stride=64 * 128, head_stride=64 * 128 // 2, slot_stride=128, n_layers=2, n_pages=10,
             kv_heads=2, page_size=32, head_dim=128, n_seqs=4, max_pages=5, table=A, len=A, ref=A, work=A, err=A)
    v.update(kw)
    for n, x in v.items():
        setattr(c, n, x)
    return c


BAD_CACHES = [dict(k=0), dict(table=0), dict(err=0), dict(v=A + 8), dict(head_dim=96), dict(page_size=12), dict(page_size=0),
              dict(page_size=65544), dict(n_pages=0), dict(kv_heads=0), dict(n_seqs=0), dict(max_pages=0), dict(slot_stride=120),
              dict(page_stride=12), dict(head_stride=-64), dict(layer_stride=-8), dict(max_pages=1 << 26)]


def test_struct_sizes_match_c(tmp_path):
    from hybrid_deltanet_attention_b200 import _abi
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mk.h"\nint main(){printf("%zu %zu %zu %zu", sizeof(mk_paged_cache),'
                   ' offsetof(mk_paged_cache, err), sizeof(mk_qk_rope), offsetof(mk_qk_rope, seqs));}\n')
    exe = tmp_path / "s"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    out = [int(x) for x in subprocess.check_output([str(exe)]).decode().split()]
    assert out == [C.sizeof(_abi.MkPagedCache), _abi.MkPagedCache.err.offset, C.sizeof(_abi.MkQkRope), _abi.MkQkRope.seqs.offset]


@pytest.mark.parametrize("kw", BAD_CACHES, ids=lambda k: "-".join(f"{a}={b}" for a, b in k.items()))
def test_bad_caches_are_refused_by_every_call(lib, kw):
    from hybrid_deltanet_attention_b200 import _abi
    bad, ok = C.byref(cache(**kw)), C.byref(cache())
    for rc in (lib.mk_pages_resize(bad, A, A, 1, None), lib.mk_pages_fork(bad, A, A, 1, None), lib.mk_pages_compact(bad, None),
               lib.mk_pages_copy(bad, ok, A, A, 1, None), lib.mk_pages_copy(ok, bad, A, A, 1, None),
               lib.mk_paged_attention(bad, 0, A, 1024, 1, 8, A, None, 1, 0.1, A, 1024, A, 1 << 40, None)):
        assert rc == _abi.MK_ERR_ARG and lib.mk_last_error()
    assert lib.mk_paged_attention_scratch(bad, 1, 8) == 0


def test_page_calls_refuse_bad_counts(lib):
    from hybrid_deltanet_attention_b200 import _abi
    c = C.byref(cache())
    E = _abi.MK_ERR_ARG
    assert lib.mk_pages_resize(c, A, A, 5, None) == E        # more sequences than the cache has
    assert lib.mk_pages_resize(c, A, A, -1, None) == E
    assert lib.mk_pages_resize(c, None, A, 1, None) == E
    assert lib.mk_pages_fork(c, A, None, 1, None) == E
    assert lib.mk_pages_fork(c, A, A, 5, None) == E
    assert lib.mk_pages_copy(c, c, A, None, 1, None) == E
    assert lib.mk_pages_copy(c, c, A, A, -2, None) == E
    assert lib.mk_pages_copy(c, C.byref(cache(page_size=16)), A, A, 1, None) == E
    assert lib.mk_pages_copy(c, C.byref(cache(n_layers=1)), A, A, 1, None) == E
    assert lib.mk_pages_copy(None, c, A, A, 1, None) == E
    assert lib.mk_pages_resize(None, A, A, 1, None) == E
    for rc in (lib.mk_pages_resize(c, A, A, 0, None), lib.mk_pages_fork(c, A, A, 0, None), lib.mk_pages_copy(c, c, A, A, 0, None)):
        assert rc == _abi.MK_OK                              # nothing to do, nothing launched
    assert lib.mk_pages_work_ints(None) == 0 and lib.mk_pages_work_ints(c) >= 10 + 4


def rope_args(**kw):
    from hybrid_deltanet_attention_b200 import _abi
    a = _abi.MkQkRope()
    v = dict(dtype=_abi.MK_DT_F32, rows=3, q_heads=4, kv_heads=2, head_dim=128, rot_dim=128, theta=1e6, eps=1e-6, q=A, ldq=512, k=A,
             ldk=256, v=A, ldv=256, q_out=A, ldq_out=512, k_out=A, ldk_out=256, positions=A)
    v.update(kw)
    for n, x in v.items():
        setattr(a, n, x)
    return C.byref(a), a


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(rows=-1), dict(q_heads=0), dict(kv_heads=0), dict(head_dim=192), dict(rot_dim=-8),
                                dict(rot_dim=136), dict(rot_dim=12), dict(theta=0.0), dict(theta=float("nan")), dict(eps=-1.0),
                                dict(q=0), dict(k_out=0), dict(positions=0), dict(q=A + 4), dict(q_gain=A + 2), dict(ldq=504),
                                dict(ldk=260), dict(ldq_out=0), dict(ldk_out=128)],
                         ids=lambda k: "-".join(f"{a}={b}" for a, b in k.items()))
def test_rope_refuses(lib, kw):
    from hybrid_deltanet_attention_b200 import _abi
    assert lib.mk_qk_norm_rope(rope_args(**kw)[0], None) == _abi.MK_ERR_ARG


def test_rope_with_a_cache_refuses(lib):
    from hybrid_deltanet_attention_b200 import _abi
    good = cache()
    base = dict(cache=C.addressof(good), layer=0, n=1, seq_start=A)
    for kw in (dict(layer=2), dict(layer=-1), dict(kv_heads=1), dict(n=-1), dict(seq_start=0), dict(v=0), dict(ldv=8), dict(v=A + 8)):
        p, keep = rope_args(**dict(base, **kw))
        assert lib.mk_qk_norm_rope(p, None) == _abi.MK_ERR_ARG, kw
    assert lib.mk_qk_norm_rope(rope_args(rows=0)[0], None) == _abi.MK_OK
    assert lib.mk_qk_norm_rope(rope_args(**dict(base, n=0))[0], None) == _abi.MK_OK
    assert lib.mk_qk_norm_rope(None, None) == _abi.MK_ERR_ARG


def test_attention_refuses(lib):
    from hybrid_deltanet_attention_b200 import _abi
    c = cache()

    def call(**kw):
        v = dict(layer=0, q=A, ldq=1024, rows=3, hq=8, start=A, seqs=None, n=1, scale=0.1, out=A, ldo=1024, scr=A, size=1 << 40)
        v.update(kw)
        return lib.mk_paged_attention(C.byref(c), v["layer"], v["q"], v["ldq"], v["rows"], v["hq"], v["start"], v["seqs"], v["n"],
                                      v["scale"], v["out"], v["ldo"], v["scr"], v["size"], None)

    for kw in (dict(layer=2), dict(layer=-1), dict(q=None), dict(q=A + 8), dict(out=None), dict(out=A + 2), dict(ldq=1016),
               dict(ldq=1028), dict(ldo=8), dict(rows=-1), dict(hq=0), dict(hq=7), dict(hq=258, ldq=1 << 16, ldo=1 << 16), dict(start=None), dict(n=-1), dict(n=65537),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(scr=None), dict(scr=A + 4), dict(size=0)):
        assert call(**kw) == _abi.MK_ERR_ARG, kw
    assert call(rows=0) == _abi.MK_OK and call(n=0) == _abi.MK_OK
    assert lib.mk_paged_attention_scratch(C.byref(c), 3, 7) == 0
    assert lib.mk_paged_attention_scratch(C.byref(c), -1, 8) == 0


def test_plain_page_accounting_invariants():
    """Counts equal the table's entries, no partly filled page is shared, and failing calls change nothing."""
    rng = random.Random(5)
    p = Pages(40, 6, 9, 8)
    for _ in range(400):
        before = p.copy()
        k = rng.randint(1, 4)
        ids = rng.sample(range(6), k)
        op = rng.choice("rrfc")
        ok = True
        if op == "r":
            ok = p.resize(ids, [rng.randint(0, 72) for _ in ids])
        elif op == "f" and k > 1:
            ok = p.fork([ids[0]] * (k - 1), ids[1:])
        elif op == "c":
            p.compact()
        if not ok:
            assert (p.table == before.table).all() and (p.len == before.len).all() and (p.ref == before.ref).all()
        used = p.table[p.table >= 0]
        assert (np.bincount(used, minlength=40) == p.ref).all()
        for s in range(6):
            n = int(p.len[s])
            assert (p.table[s, :pages_of(n, 8)] >= 0).all() and (p.table[s, pages_of(n, 8):] == -1).all()
            if n % 8:
                assert p.ref[p.table[s, n // 8]] == 1
