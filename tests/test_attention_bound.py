"""CPU: the bound that the GPU tests hold attention to is sharp enough: a stretch of 64 positions that goes missing, wherever it lies, and
a part of a split that does, exceed it in every long case."""
import math

import numpy as np
import pytest

from tests import attention_model as A

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.mark.parametrize("lens,heads,kv,dim,page,sd,qt,window,sinks", A.LONG)
def test_lost_positions_exceed_the_bound(lens, heads, kv, dim, page, sd, qt, window, sinks):
    cache = A.make(lens, kv, dim, page, sd, seed=heads + dim)
    q = np.random.RandomState(7).randn(len(lens), heads, dim)
    scale = 1 / math.sqrt(dim)
    ref, bound = A.reference(q, cache, lens, None, None, scale, window, sinks)
    norm = np.linalg.norm(ref, axis=-1)
    assert (bound[0] < 0.01 * norm[0]).all(), "the bound is no longer small beside the result"
    # the right result, rounded once, is within it
    assert not A.off(ref * (1 + 0.99 * HALF[qt]), ref, bound, HALF[qt]).any()
    n = lens[0]
    first = n - window if window else 0
    starts = sorted({first // 64 * 64 + 64, (first + n) // 2 // 64 * 64, (n - 1) // 64 * 64 - 64, max(first, n - 64)})
    for at in starts:
        lost, _ = A.reference(q[:1], cache, lens[:1], None, None, scale, window, sinks, hidden=range(at, at + 64))
        assert A.off(lost, ref[:1], bound[:1], HALF[qt]).all(), f"64 positions from {at} may go missing"
