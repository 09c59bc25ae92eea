"""The precision checks of the fp32 products, on a model of them: all six products pass, five do not."""
import numpy as np
import pytest

import linear_precision as P


def test_parts_add_up():
    x = np.random.default_rng(0).standard_normal(10000).astype(np.float32)
    p = P.parts(x)
    assert np.array_equal(sum(p), x.astype(np.float64))
    assert np.all(np.abs(p[1]) <= 2.0 ** -8 * np.abs(x)) and np.all(np.abs(p[2]) <= 2.0 ** -16 * np.abs(x))


@pytest.mark.parametrize("k", [17, 64, 300, 588, 2100])
@pytest.mark.parametrize("missing", [None, *P.PAIRS])
def test_frobenius_bound_tells_a_missing_product(k, missing):
    rng = np.random.default_rng(k)
    a, b = rng.standard_normal((70, k)).astype(np.float32), rng.standard_normal((60, k)).astype(np.float32)
    got = P.products(a, b, [p for p in P.PAIRS if p != missing])
    want = a.astype(np.float64) @ b.astype(np.float64).T
    assert (P.relative(got, want) <= P.FROBENIUS / 10) if missing is None else (P.relative(got, want) > 2 * P.FROBENIUS)


@pytest.mark.parametrize("kind", P.KINDS)
@pytest.mark.parametrize("missing", [None, *P.PAIRS])
def test_cancelling_operands_need_each_product(kind, missing):
    a, b = P.cancelling(kind, 40, 30, 20)
    got = P.products(a, b, [p for p in P.PAIRS if p != missing])
    want = a.astype(np.float64) @ b.astype(np.float64).T
    off = np.abs(got - want) > P.cancelling_tolerance(a, b)
    if missing is None:
        assert not off.any()
    elif missing == P.NEEDS[kind]:
        assert off.all()
