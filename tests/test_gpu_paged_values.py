"""Values and table states of the paged-cache operators that random entries do not reach."""
import numpy as np
import pytest

import paged_ref as ref
import test_gpu_paged as base

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1.5e-36, -1.5e-36, 0.0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_small_scales_of_large_scores(d, scale):
    """Scores near fp32's end, so that a scale far below 2^-100 gives ordinary weights, and one of zero the mean."""
    base.run_attention(5, [300, 40, 1], [40, 40, 1], 4, 2, d, 16, scale=scale, q_scale=1e35)
