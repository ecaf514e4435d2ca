"""Scaled frequencies against their formulas, pair by pair (no GPU)."""
import math

import pytest


@pytest.fixture(scope="module")
def q():
    from skinny_gemm_q4_gb300 import build, qgemv
    build.build()
    qgemv.load()
    return qgemv


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("base", [1e4, 5e5, 1e6])
@pytest.mark.parametrize("factor,length,low,high", [(4.0, 8192.0, 0.0, 0.0), (32.0, 32768.0, 0.0, 0.0),
                                                    (8.0, 4096.0, 2.0, 20.0), (1.5, 100.0, 0.0, 0.0)])
def test_every_frequency(q, rot, base, factor, length, low, high):
    """A pair i turns n(i) = length base^(-2 i / rot) / (2 pi) times in the
    trained length.  Yarn: the ramp runs over the pair index from the (floored)
    index of `high` turns to the (ceiled) one of `low`; bands: over the turns."""
    d = dict(base=base, factor=factor, original_len=length, low=low, high=high)
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    turns = [length * f / (2 * math.pi) for f in plain]

    lo_n, hi_n = low or 1.0, high or 32.0
    # n(i) = n  <=>  i = rot / 2 * log_base(length / (2 pi n))
    first = max(0, math.floor(rot / 2 * math.log(length / (2 * math.pi * hi_n), base)))
    last = min(rot - 1, math.ceil(rot / 2 * math.log(length / (2 * math.pi * lo_n), base)))
    got, ms = q.qgemv_rope_freqs(q.rope_desc(128, rot, scaling=q.ROPE_SCALE_YARN, **d))
    for i, (g, f) in enumerate(zip(got, plain)):
        part = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
        assert g == pytest.approx(f * ((1 - part) + part / factor), rel=1e-13), i
    assert ms == pytest.approx(1 + math.log(factor) / 10, rel=1e-15)

    hi_n = high or 4.0
    got, ms = q.qgemv_rope_freqs(q.rope_desc(128, rot, scaling=q.ROPE_SCALE_BANDS, **d))
    for i, (g, f, n) in enumerate(zip(got, plain, turns)):
        keep = 1.0 if n >= hi_n else 0.0 if n <= lo_n else (n - lo_n) / (hi_n - lo_n)
        assert g == pytest.approx(f * (keep + (1 - keep) / factor), rel=1e-13), i
    assert ms == 1.0

    got, ms = q.qgemv_rope_freqs(q.rope_desc(128, rot, scaling=q.ROPE_SCALE_LINEAR, **d))
    assert ms == 1.0 and all(g == pytest.approx(f / factor, rel=1e-15) for g, f in zip(got, plain))
