"""Edges of the attention side on the GPU: values, lengths, masks and handles
that the ordinary sizes do not reach.  Tolerances as in test_gpu_attn.py."""
import numpy as np
import pytest

import attn_plain as ap
from gpu_util import torch
from test_gpu_attn import KINDS, Batch, check, dev, half_ulp, qg  # noqa: F401  (qg: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Ts,Ls", [([9, 1, 5], [3, 1, 300]), ([60, 45, 20], [20, 2, 130])])
def test_attn_widest_window(qg, kind, causal, Ts, Ls):
    """The largest window hides nothing, for requests with more new tokens than
    context too: the bits of a call without a window."""
    b = Batch(qg, kind, 64, 16, 2, 1, Ts, Ls, seed=21)
    want = b.check(causal, 0)
    for window in (2 ** 31 - 1, 2 ** 30, 400):
        got = b.run(causal, window)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
