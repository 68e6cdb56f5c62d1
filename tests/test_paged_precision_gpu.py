"""How exact the paged decode's weights are, seen where the output's own
rounding is small: columns whose values nearly cancel."""
import numpy as np
import pytest

import paged_reference as ref
from test_paged_decode_gpu import Case, _built  # noqa: F401  (the fixture builds)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("splits", [1, 4, 12])
@pytest.mark.parametrize("kw", [dict(), dict(d=64, P=16), dict(Hq=16), dict(Hq=2)], ids=str)
def test_bf16_pages_lose_no_bits_of_a_weight(kw, splits, tsf):
    """|o - exact| against half a step of o and 2^-16 of the mass for a weight
    (two bf16 parts: the first is off by half a step, 2^-8 of the weight at most,
    the second by half a step of that rest, 2^-8 of 2^-8), besides the scores' and
    sums' errors that decode_tolerance derives. Weights rounded to bf16 alone, off
    by up to 2^-8 each, are far outside where an output is small."""
    c = Case([700, 0, 1, 65, 333, 64], splits=splits, tsf=tsf, **kw)
    got = c.check()
    want = ref.decode(c.q, c.k, c.v, c.table, c.lens, c.scale, c.tsf, splits, tiles=got["tile_state"])
    ds = want["size"] * 2.0 ** -19 + 2.0 ** -20
    chain = (700 / 64 + 64) * 2.0 ** -24
    tol = (2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(want["o"]) +
           (2.0 ** -16 + 2 * ds[..., None] + chain) * want["mass"] + 1e-30)
    d = np.abs(got["o"] - want["o"])
    assert np.all(d <= tol), float((d / tol).max())


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("tsf", [0.0, 4.0])
def test_a_call_repeats_itself_to_the_bit(tsf, fmt):
    c = Case([4000, 0, 1, 65, 333, 2049], fmt=fmt, tsf=tsf, splits=12, Hq=16, Hkv=4)
    first = c.run()
    for _ in range(5):
        again = c.run()
        for n in ("o", "lse", "tile_state"):
            assert np.array_equal(first[n], again[n]), n
