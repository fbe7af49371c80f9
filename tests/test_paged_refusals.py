"""Arguments at the ends of their ranges that the paged-cache entry points refuse on the host."""
import ctypes as C

import pytest

from test_paged_abi import A, cache, lib, rope_args  # noqa: F401


@pytest.mark.parametrize("scale", [2.1e38, -3.4e38, float("inf"), float("nan")])
def test_attention_refuses_scales_past_its_log2_units(lib, scale):  # noqa: F811
    """scale * log2 e is a factor in fp32: past 2.36e38 it would be infinite and every score of zero NaN."""
    from hybrid_deltanet_attention_b200 import _abi
    c = cache()
    rc = lib.mk_paged_attention(C.byref(c), 0, A, 1024, 3, 8, A, None, 1, scale, A, 1024, A, 0, None)
    assert rc == _abi.MK_ERR_ARG and b"scale" in lib.mk_last_error()


def test_rotation_refuses_an_infinite_theta(lib):  # noqa: F811
    """Its first angle would be position * inf^0 = position, but 0 * log2(inf) is NaN."""
    from hybrid_deltanet_attention_b200 import _abi
    assert lib.mk_qk_norm_rope(rope_args(theta=float("inf"), q=0)[0], None) == _abi.MK_ERR_ARG and b"theta" in lib.mk_last_error()
