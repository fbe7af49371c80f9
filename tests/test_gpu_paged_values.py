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


@pytest.mark.parametrize("n_pages", [20, 4099, 60001])
def test_compaction_leaves_an_uncounted_page_alone(n_pages):
    """An entry whose page has no count stays as it is, whatever an earlier compaction did with that page."""
    m = base.hda()
    c = m.PagedCache.empty(1, n_pages, 1, 8, 64, 3, 2)

    def put(s, pages, counted=True):
        c.table[s, :len(pages)] = base.ints(pages)
        c.len[s] = 8 * len(pages)
        if counted:
            c.ref[base.ints(pages).long()] += 1

    a, b = n_pages - 10, n_pages - 8
    put(0, [0, a])
    c.compact()                                    # a moves to page 1
    c.sync()
    assert c.table[0].tolist() == [0, 1]
    put(1, [b])
    put(2, [a], counted=False)
    c.compact()                                    # b moves to page 2
    c.sync()
    assert c.table.tolist() == [[0, 1], [2, -1], [a, -1]] and c.ref[:4].tolist() == [1, 1, 1, 0]
