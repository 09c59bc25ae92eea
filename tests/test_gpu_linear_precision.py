"""The fp32 Linear layer keeps fp32's precision over fp32's range: the bounds of linear_precision.py."""
import linear_precision as P
import numpy as np
import pytest
import torch

from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu


def np64(t):
    return t.detach().double().cpu().numpy()


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda()


def forward(x, w):
    (rows, k), n = x.shape, w.shape[0]
    y = torch.empty(rows, n, device="cuda")
    A.dsv4v_linear_forward(A.make_linear(rows, k, n, dtype=A.DSV4V_F32), x, w, None, None, None, y)
    assert A.dsv4v_device_error() == 0
    return np64(y), np64(x) @ np64(w).T


def backward(x, w, d_y):
    (rows, k), n = x.shape, w.shape[0]
    layer = A.make_linear(rows, k, n, dtype=A.DSV4V_F32)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
    A.dsv4v_linear_backward(layer, x, w, None, d_y, dx, dw, None, ws)
    assert A.dsv4v_device_error() == 0
    return (np64(dx), np64(d_y) @ np64(w)), (np64(dw), np64(d_y).T @ np64(x))


# One row of an operand at each scale, against an operand of about 2^`other`: each row's own error, from values whose low
# parts bf16 cannot hold (below 2^-110) and subnormal ones to values whose bf16 parts overflow.
SCALES = [0, -60, -95, -108, -115, -125, -133, -140, 30, 60, 100, 113, 126]


def scaled(k, seed):
    rows = torch.tensor([2.0 ** s for s in SCALES], dtype=torch.float64)[:, None]
    return (normal((len(SCALES), k), seed).cpu().double().clamp(-1.9, 1.9) * rows).float().cuda()


@pytest.mark.parametrize("k,n", [(100, 70), (588, 201), (4600, 40)])
@pytest.mark.parametrize("other", [-8, 20])
def test_forward_rows_of_every_scale(k, n, other):
    # the results stay between 2^-125 and the end of fp32's range for the rows that are looked at
    x = scaled(k, 1)
    use = [i for i, s in enumerate(SCALES) if -120 <= s + other <= 115]
    keep = torch.zeros(len(SCALES), 1, device="cuda")
    keep[use] = 1
    y, want = forward(x * keep, normal((n, k), 2) * 2.0 ** other)
    for i in use:
        assert P.relative(y[i], want[i]) <= P.FROBENIUS, (SCALES[i], P.relative(y[i], want[i]))


@pytest.mark.parametrize("k,n", [(100, 70), (588, 201)])
def test_tiny_operands_meet_large_ones(k, n):
    # 2^-140 to 2^-95 against 2^100
    low = [i for i, s in enumerate(SCALES) if s <= -95]
    x = scaled(k, 1)[low].contiguous()
    w = normal((n, k), 2) * 2.0 ** 100
    y, want = forward(x, w)
    for i in range(len(low)):
        assert P.relative(y[i], want[i]) <= P.FROBENIUS, (SCALES[low[i]], P.relative(y[i], want[i]))


@pytest.mark.parametrize("rows,k,n", [(50, 100, 13), (300, 130, 13)])
def test_gradients_of_tiny_operands(rows, k, n):
    # d_y's columns at 2^-140 to 1 (dw's rows), then its rows (dx's)
    cols = torch.tensor([2.0 ** s for s in np.linspace(-140, 0, n)], dtype=torch.float64)
    x, w = normal((rows, k), 1) * 2.0 ** 60, normal((n, k), 2) * 2.0 ** 60
    d_y = (normal((rows, n), 3).cpu().double() * cols).float().cuda()
    _, (dw, want) = backward(x, w, d_y)
    assert max(P.relative(dw[i], want[i]) for i in range(n)) <= P.FROBENIUS
    down = torch.tensor([2.0 ** s for s in np.linspace(-140, 0, rows)], dtype=torch.float64)
    d_y = (normal((rows, n), 3).cpu().double() * down[:, None]).float().cuda()
    (dx, want), _ = backward(x, w, d_y)
    assert max(P.relative(dx[i], want[i]) for i in range(rows)) <= P.FROBENIUS


# ---------------------------------------------------------------------------------------------- all six products
@pytest.mark.parametrize("rows,k,n", [(5, 257, 1000), (63, 17, 65), (130, 588, 97), (777, 588, 201), (300, 300, 130), (129, 256, 64),
                                      (70, 1100, 60), (777, 588, 1001), (40, 4000, 72), (2, 4608, 40)])
def test_forward_is_as_near_as_all_products_make_it(rows, k, n):
    x, w = normal((rows, k), 1), normal((n, k), 2)
    y, want = forward(x, w)
    assert P.relative(y, want) <= P.FROBENIUS
    assert np.all(np.abs(y - want) <= P.element_tolerance(np64(x), np64(w)))


@pytest.mark.parametrize("rows,k,n", [(63, 17, 65), (130, 588, 97), (777, 588, 201), (257, 64, 1000), (300, 130, 300), (777, 588, 1001),
                                      (2100, 400, 1001), (4000, 64, 72)])
def test_gradients_are_as_near_as_all_products_make_them(rows, k, n):
    x, w, d_y = normal((rows, k), 1), normal((n, k), 2), normal((rows, n), 3)
    operands = ((np64(d_y), np64(w).T), (np64(d_y).T, np64(x).T))
    for (got, want), (a, b) in zip(backward(x, w, d_y), operands):
        assert P.relative(got, want) <= P.FROBENIUS
        assert np.all(np.abs(got - want) <= P.element_tolerance(a, b))


@pytest.mark.parametrize("kind", P.KINDS)
@pytest.mark.parametrize("groups", [9, 150, 1000])
@pytest.mark.parametrize("where", ["forward", "dx", "dw"])
def test_sums_that_are_left_of_low_parts(kind, groups, where):
    # rows 90, columns 70, a contraction of 4 groups: the forward's over features, dx's over outputs, dw's over rows
    a, b = P.cancelling(kind, groups, 90, 70)
    want = a.astype(np.float64) @ b.astype(np.float64).T
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    if where == "forward":
        got = forward(dev(a), dev(b))[0]
    elif where == "dx":  # d_y . w
        got = backward(normal((90, 70), 1), dev(b.T), dev(a))[0][0]
    else:  # d_y^T . x
        got = backward(dev(b.T), normal((90, 70), 1), dev(a.T))[1][0]
    assert np.all(np.abs(got - want) <= P.cancelling_tolerance(a, b))


# ---------------------------------------------------------------------------------------------- what is not finite
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38, 1e34])
@pytest.mark.parametrize("rows,k,n", [(40, 100, 70), (300, 300, 130), (777, 588, 201), (60, 2100, 40)])
def test_a_value_that_bf16_cannot_hold_changes_its_own_sums_alone(rows, k, n, bad):
    # the other sums of its tiles keep their bits
    x, w, d_y = normal((rows, k), 1), normal((n, k), 2), normal((rows, n), 3)
    b, r = normal((n,), 4), normal((rows, n), 5)
    layer = A.make_linear(rows, k, n, A.ACT_GELU, A.DSV4V_F32)

    def forward_all(x):
        y, z = torch.empty(rows, n, device="cuda"), torch.empty(rows, n, device="cuda")
        A.dsv4v_linear_forward(layer, x, w, b, r, z, y)
        return y, z

    def backward_all(x, d_y):
        plain = A.make_linear(rows, k, n, dtype=A.DSV4V_F32)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws = torch.empty(A.dsv4v_linear_backward_workspace_size(plain), dtype=torch.uint8, device="cuda")
        A.dsv4v_linear_backward(plain, x, w, None, d_y, dx, dw, None, ws)
        return dx, dw

    i, c, f = rows // 2, k // 3, n // 2
    clean_y, clean_z = forward_all(x)
    clean_dx, clean_dw = backward_all(x, d_y)
    x1, d1 = x.clone(), d_y.clone()
    x1[i, c], d1[i, f] = bad, bad
    others = torch.arange(rows, device="cuda") != i
    for got, want in zip(forward_all(x1), (clean_y, clean_z)):
        assert torch.equal(got[others], want[others])
    z = forward_all(x1)[1][i].double().cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        want = np64(x1[i]) @ np64(w).T + np64(b)
    fits = np.abs(want) <= np.finfo(np.float32).max
    assert np.array_equal(np.isnan(z), np.isnan(want))
    assert np.all(np.abs(z[fits] - want[fits]) <= 2.0 ** -20 * np.abs(want[fits]))
    # a gradient of one output: its row of dx and its row of dw; a value of x: its column of dw
    dx, _ = backward_all(x, d1)
    assert torch.equal(dx[others], clean_dx[others])
    _, dw = backward_all(x, d1)
    rest = torch.arange(n, device="cuda") != f
    assert torch.equal(dw[rest], clean_dw[rest])
    _, dw = backward_all(x1, d_y)
    rest = torch.arange(k, device="cuda") != c
    assert torch.equal(dw[:, rest], clean_dw[:, rest])
