"""The formats' definitions in numpy against closed forms, so that the GPU's codes are
compared with something that was checked itself."""
import numpy as np
import pytest

from tests import mx_ref as ref


@pytest.mark.parametrize("kind, mags, top", [("fp4", ref.E2M1, 6), ("fp8", ref.E4M3, 448)])
def test_magnitudes(kind, mags, top):
    assert len(mags) == (8 if kind == "fp4" else 127) and mags[-1] == top
    assert np.all(np.diff(mags) > 0)
    # idempotent: the values a block stands for are their own rounding
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 96)) * np.exp2(rng.integers(-20, 20, (5, 96)))
    c, e = ref.encode(x, kind)
    v = ref.decode(c, e, kind)
    c2, e2 = ref.encode(v, kind)
    assert np.array_equal(ref.decode(c2, e2, kind), v)


def test_fp4_rounding_and_exponent():
    x = np.zeros((1, 32))
    x[0, :12] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -5, .2500001, 7.9]
    c, e = ref.encode(x, "fp4")
    assert e[0, 0] == 0
    want = [6, 0, 1, 1, 2, 2, 4, 4, 0, -4, .5, 6]
    assert ref.decode(c, e, "fp4")[0, :12].tolist() == want
    assert c[0, 8] == 8                            # -0
    for amax, exp in ((8, 1), (7.99, 0), (4, 0), (3.99, -1), (2.0 ** -149, -127), (0, 0)):
        assert ref.encode(np.full((1, 32), float(amax)), "fp4")[1][0, 0] == exp


def test_fp8_exponent_never_saturates():
    for amax, exp in ((448, 0), (448.0001, 1), (224, -1), (224.0001, 0), (1, -8), (0, 0)):
        c, e = ref.encode(np.full((1, 3), float(amax)), "fp8")
        assert e[0, 0] == exp
        if amax:
            assert abs(ref.decode(c, e, "fp8")[0, 0] / amax - 1) <= 2.0 ** -4


def test_exponents_order():
    e = np.arange(40).reshape(4, 10)
    s = ref.pack_exponents(e)
    assert s.shape == (2, 16, 8)
    assert np.array_equal(ref.unpack_exponents(s, 4, 10), e)
    assert s[0, 2].tolist() == [127 + e[2, b] for b in (0, 4, 1, 5, 2, 6, 3, 7)]
    assert np.all(s[1, :, [1, 3, 4, 5, 6, 7]] == 127) and np.all(s[:, 4:] == 127)
