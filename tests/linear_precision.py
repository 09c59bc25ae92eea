"""What the fp32 products of the Linear layer owe to each part of their operands.

A product goes through three bf16 parts a value and six products of parts: a0 b0, a0 b1, a1 b0, a0 b2, a1 b1, a2 b0.  The
checks here fail where one of the six is missing (tests/test_linear_precision_host.py drops each in turn) and hold for
all six (tests/test_gpu_linear_precision.py).  u = 2^-24."""
import numpy as np
import torch

U = 2.0 ** -24
PAIRS = ((0, 0), (0, 1), (1, 0), (0, 2), (1, 1), (2, 0))


def parts(x):
    """The three bf16 parts of fp32 values, in fp64."""
    x, out = torch.as_tensor(np.asarray(x, dtype=np.float32)), []
    for _ in range(3):
        out.append(x.bfloat16().float())
        x = x - out[-1]
    return [p.double().numpy() for p in out]


def products(a, b, pairs=PAIRS):
    """a b^T from the given products of parts, summed exactly (in fp64)."""
    pa, pb = parts(a), parts(b)
    return sum(pa[i] @ pb[j].T for i, j in pairs)


# Frobenius norm of the error over that of the result, for operands of random signs.  A tensor-core addition drops at most
# 2 u of its sum, one u on average, always towards zero; 16 additions of partial sums that grow as the root of their number
# lose 16 x 2/3 u, after which fp32 additions take over (one u between them, over the K of the tests).  The three products
# left out are 2 u of the largest terms, and below one u together.  13 u; a missing product is 40 u.
FROBENIUS = 13 * U


# Each element, S being the sum of its terms' magnitudes: 16 additions on the tensor core drop at most 2 u of the sum so
# far, and the alignment of each one's sixteen terms 2 u of those: 34 u S (and 2^-8 of that in the smaller products'
# columns).  The products left out are 2 u S.  The fp32 additions of K / 256 sums, of eight ranks and of three columns
# round by one u each.
def element_tolerance(a, b):
    a, b = np.abs(np.asarray(a, dtype=np.float64)), np.abs(np.asarray(b, dtype=np.float64))
    return (34 + 1 + 2 + a.shape[1] / 256 + 11) * U * (a @ b.T)


def relative(got, want):
    return np.linalg.norm(np.asarray(got, dtype=np.float64) - want) / np.linalg.norm(want)


def cancelling(kind, groups, rows, cols, seed=0):
    """Operands a [rows, 4 groups], b [cols, 4 groups] whose leading products cancel within each four terms, so that the
    sum is what is left of low parts: of a1, a2, b1, b2, or of a1 b1."""
    rng = np.random.default_rng(seed)

    def value(n):  # three parts of one sign: bf16 values, the last one of fp32's own last bits
        part = lambda low, high: torch.from_numpy(rng.uniform(low, high, (n, groups)).astype(np.float32)).bfloat16().double().numpy()  # noqa: E731
        return part(1.01, 1.9), part(0.6 * 2.0 ** -8, 0.9 * 2.0 ** -8), rng.integers(38, 58, (n, groups)) * 2.0 ** -23

    zero = np.zeros_like
    (a0, a1, a2), (b0, b1, b2) = value(rows), value(cols)
    if kind == "a1 b1":  # (a0 + a1)(b0 + b1) - (a0 + a1) b0 - a0 (b0 + b1) + a0 b0
        a, b = (a0 + a1, -(a0 + a1), -a0, a0), (b0 + b1, b0, b0 + b1, b0)
    elif kind == "a1":
        a, b = (a0 + a1, -a0, zero(a0), zero(a0)), (b0, b0, b0, b0)
    elif kind == "a2":
        a, b = (a0 + a1 + a2, -(a0 + a1), zero(a0), zero(a0)), (b0, b0, b0, b0)
    elif kind == "b1":
        a, b = (a0, a0, a0, a0), (b0 + b1, -b0, zero(b0), zero(b0))
    else:
        a, b = (a0, a0, a0, a0), (b0 + b1 + b2, -(b0 + b1), zero(b0), zero(b0))
    stack = lambda t: np.stack(t, 2).reshape(t[0].shape[0], -1)  # noqa: E731
    a, b = stack(a), stack(b)
    for x in (a, b):
        assert np.array_equal(x, x.astype(np.float32))  # fp32 holds them
    return a.astype(np.float32), b.astype(np.float32)


KINDS = ("a1", "a2", "b1", "b2", "a1 b1")
NEEDS = {"a1": (1, 0), "a2": (2, 0), "b1": (0, 1), "b2": (0, 2), "a1 b1": (1, 1)}


def cancelling_tolerance(a, b):
    """Sixteen terms meet in a tensor-core addition, which drops at most 2 u of them and of the sum so far; here that sum
    is small beside the terms.  2 u of all terms' magnitudes, and as much again for the fp32 additions and roundings."""
    return 4 * U * (np.abs(a.astype(np.float64)) @ np.abs(b.astype(np.float64)).T)
