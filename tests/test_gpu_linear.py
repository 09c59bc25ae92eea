"""The Linear layer and its gradient against the fp64 oracle (oracle/dsv4v_linear.py), through the C ABI.

Tolerances, element by element, S = the sum of the product's absolute terms:
  * bf16 products: the tensor core adds 16 terms at a time to an fp32 accumulator; an addition loses at
    most 2^-23 of what is summed so far: (K / 16 + 8) 2^-23 S.
  * fp32 products: sums of 128 terms, and of K / 128 such sums: (128 + K / 128 + 4) 2^-24 S.
  * Activations: their slope is at most 1.13; their own error is the formula's 1.5e-7 and a few
    2^-23 roundings (MUFU exponential and reciprocal): 4e-7 (1 + |z|).  fp32: 8 roundings, 2^-21 |y|.
  * One rounding of each output: 2^-8 (bf16) or 2^-24 (fp32) of it.
  * Backward: dz is rounded once as an operand (not without an activation): 2^-8 (2^-24) of |dz|, weighed
    by the other operand; the derivative's own error is at most 1e-6 (1 + |z|) |dy|.  db sums unrounded
    values: (rows + 16) 2^-24 of their absolute sum.
Beside these, bf16 results stay within 2^-8 of the oracle's in the Frobenius norm (twice that where dz
is rounded)."""
import numpy as np
import pytest
import torch

from oracle import dsv4v_linear as O
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu

ACT = {"none": A.ACT_NONE, "gelu": A.ACT_GELU, "silu": A.ACT_SILU}
TYPES = {"bf16": (torch.bfloat16, A.DSV4V_BF16, 2.0 ** -8), "f32": (torch.float32, A.DSV4V_F32, 2.0 ** -24)}


def np64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A [rows, cols] matrix with row stride ld inside a buffer of sentinels, to see that only the matrix is written."""

    def __init__(self, rows, cols, ld, dtype, offset=0, fill=None):
        self.shape, self.ld, self.offset = (rows, cols), ld, 64 + offset
        self.buf = torch.full((64 + offset + max(1, rows) * ld + 64,), 7.0, device="cuda").to(dtype)
        self.t = self.buf[self.offset:self.offset + max(1, rows) * ld].as_strided((rows, cols), (ld, 1))
        if fill is not None:
            self.t.copy_(fill)

    def untouched(self):
        around = self.buf.clone()
        around[self.offset:self.offset + max(1, self.shape[0]) * self.ld].as_strided(self.shape, (self.ld, 1)).fill_(7.0)
        return bool((around == 7.0).all())


def normal(shape, scale, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale).to(dtype).cuda()


def pad8(n):
    return (n + 7) // 8 * 8


def abs_products(a, b):
    return np.abs(a) @ np.abs(b).T


def accumulate(kind, k, s):
    return (k / 16 + 8) * 2.0 ** -23 * s if kind == "bf16" else (128 + k / 128 + 4) * 2.0 ** -24 * s


def own_error(kind, z, y):
    return 4e-7 * (1 + np.abs(z)) if kind == "bf16" else 2.0 ** -21 * np.abs(y)


def close(got, want, tol, what):
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) - tol)}"


def run_forward(kind, rows, k, n, act, bias=True, residual=True, save_z=True, in_place=False, ld_x=None, ld_w=None, ld_y=None,
                y_offset=0, seed=0):
    dtype, code, half = TYPES[kind]
    pad = pad8 if kind == "bf16" else (lambda v: v)
    ld_x, ld_w, ld_y = ld_x or pad(k), ld_w or pad(k), ld_y or n
    x = Guarded(rows, k, ld_x, dtype, fill=normal((rows, k), 1.0, dtype, seed))
    w = Guarded(n, k, ld_w, dtype, fill=normal((n, k), k ** -0.5, dtype, seed + 1))
    b = normal((n,), 0.5, torch.float32, seed + 2) if bias else None
    r0 = normal((rows, n), 1.0, dtype, seed + 3)
    y = Guarded(rows, n, ld_y, dtype, y_offset, fill=r0 if in_place else None)
    r = y if in_place else (Guarded(rows, n, ld_y, dtype, y_offset, fill=r0) if residual else None)
    z = Guarded(rows, n, ld_y, dtype, y_offset) if save_z else None
    layer = A.make_linear(rows, k, n, ACT[act], code, ld_x=ld_x, ld_w=ld_w, ld_residual=ld_y, ld_z=ld_y, ld_y=ld_y)
    A.dsv4v_linear_forward(layer, x.t, w.t, b, r.t if r else None, z.t if z else None, y.t)
    assert A.dsv4v_device_error() == 0
    want_y, want_z = O.forward(np64(x.t), np64(w.t), None if b is None else np64(b), np64(r0) if r else None, act)
    acc = accumulate(kind, k, abs_products(np64(x.t), np64(w.t)) + (0 if b is None else np.abs(np64(b))))
    tol = half * np.abs(want_y) + 1.13 * acc + (own_error(kind, want_z, want_y) if act != "none" else 0)
    if r:  # the sum with the residual is rounded in fp32 once more
        tol = tol + 2.0 ** -23 * np.abs(np64(r0))
    close(np64(y.t), want_y, tol, "y")
    assert y.untouched()
    if z:
        close(np64(z.t), want_z, half * np.abs(want_z) + acc, "z")
        assert z.untouched()
    if kind == "bf16" and rows * n >= 64:
        assert np.linalg.norm(np64(y.t) - want_y) <= 2.0 ** -8 * np.linalg.norm(want_y)


# Every tile and split the plans know is met: small tiles split over clusters of 2, 4 and 8 (few tiles, long
# sums), whole tiles, pairs; extents on, before and behind a tile's edge.
SHAPES = [(1, 1, 1), (1, 8, 3), (1, 4608, 4608), (2, 64, 7), (3, 2816, 64), (5, 9, 1000), (8, 1024, 2816), (17, 63, 129),
          (64, 4096, 512), (127, 65, 255), (128, 64, 64), (129, 128, 257), (200, 588, 1001), (255, 1000, 96), (784, 1024, 1024),
          (777, 588, 1001), (784, 1024, 2816), (1025, 200, 2100), (2500, 72, 1155), (4100, 130, 2100),
          (1144, 72, 2055), (1355, 264, 1861), (2858, 1864, 1872)]


@pytest.mark.parametrize("rows,k,n", SHAPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_forward(rows, k, n, act):
    run_forward("bf16", rows, k, n, act)


@pytest.mark.parametrize("rows,k,n", [(1, 1, 1), (1, 300, 5), (63, 17, 65), (64, 16, 64), (130, 588, 97), (777, 588, 201), (6, 1100, 60),
                                      (300, 300, 130), (129, 256, 64), (5, 257, 1000)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_forward_fp32(rows, k, n, act):
    run_forward("f32", rows, k, n, act)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("k,n", [(1, 1), (7, 300), (200, 9), (1033, 77), (2048, 130), (4608, 64), (13000, 33)])
def test_linear_forward_of_a_few_rows(kind, rows, k, n):
    # the weight-streaming kernels: extents that leave lanes, warps and pieces without work, and lengths behind their limit
    run_forward(kind, rows, k, n, "gelu")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n", [(1, 520, 40), (33, 4100, 72), (300, 100, 264), (3000, 72, 1160)])
@pytest.mark.parametrize("bias,residual,save_z", [(False, False, False), (True, False, False), (False, True, False), (False, False, True)])
def test_linear_forward_without_each_part(kind, rows, k, n, bias, residual, save_z):
    run_forward(kind, rows, k, n, "silu", bias, residual, save_z)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n,ld_y,offset", [(40, 72, 64, 64, 0), (40, 72, 64, 72, 0), (40, 72, 64, 67, 0), (40, 72, 64, 72, 1),
                                                  (40, 72, 61, 61, 3), (2, 4608, 61, 64, 0), (2, 4608, 61, 65, 1),
                                                  (3000, 72, 1153, 1160, 0), (3000, 72, 1160, 1161, 5)])
def test_linear_forward_strides(kind, rows, k, n, ld_y, offset):
    run_forward(kind, rows, k, n, "gelu", ld_x=pad8(k) + 16, ld_w=pad8(k) + 8, ld_y=ld_y, y_offset=offset)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("rows", [5, 16, 17, 32, 33])
@pytest.mark.parametrize("k,n,ld_y,offset", [(9, 40, 40, 0), (72, 264, 264, 0), (72, 264, 272, 1), (130, 1153, 1160, 0), (130, 1160, 1161, 5),
                                             (1100, 2600, 2600, 0), (4608, 4600, 4600, 0), (200, 18901, 18904, 0), (200, 19001, 19008, 0)])
def test_linear_forward_of_rows_that_share_a_weight_tile(rows, k, n, ld_y, offset, act):
    # a few dozen rows: the weights' features take the place of the rows in the MMAs, split or not
    run_forward("bf16", rows, k, n, act, ld_y=ld_y, y_offset=offset)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n", [(16, 72, 264), (40, 1100, 2600), (1, 4608, 200), (300, 72, 264), (3000, 72, 1160), (3000, 72, 1161)])
def test_linear_forward_adds_in_place(kind, rows, k, n):
    run_forward(kind, rows, k, n, "none", in_place=True, save_z=False)


def test_linear_forward_matches_the_residual_gemm():
    # the same product as the block's own output projection
    cfg = A.make_config(1024, 16, 2816, 2, 4096, 1)
    a, w, x = normal((784, 1024), 1.0, torch.bfloat16, 1), normal((1024, 1024), 0.02, torch.bfloat16, 2), normal((784, 1024), 1.0, torch.bfloat16, 3)
    ws = torch.empty(A.dsv4v_workspace_size(cfg, A.BatchRef([(28, 28)])), dtype=torch.uint8, device="cuda")
    want = x.clone()
    A.dsv4v_linear_residual(cfg, 784, 1024, a, w, want, ws)
    y = torch.empty_like(x)
    A.dsv4v_linear_forward(A.make_linear(784, 1024, 1024), a, w, None, x, None, y)
    assert (y.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    assert torch.linalg.norm(y.float() - want.float()) <= 2.0 ** -8 * torch.linalg.norm(want.float())


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_linear_activations_over_their_range(act, kind):
    # one weight of 1 hands chosen values to the activation: far tails, zero, what is not finite
    dtype, code, half = TYPES[kind]
    v = torch.cat([torch.linspace(-40, 40, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e4, -3e4, 1e38, -1e38])]).to(dtype).cuda()
    n = v.numel()
    x = torch.zeros(n, 8, dtype=dtype, device="cuda")
    x[:, 0] = v
    w = torch.zeros(1, 8, dtype=dtype, device="cuda")
    w[0, 0] = 1
    y, z = torch.empty(n, 1, dtype=dtype, device="cuda"), torch.empty(n, 1, dtype=dtype, device="cuda")
    layer = A.make_linear(n, 8, 1, ACT[act], code)
    A.dsv4v_linear_forward(layer, x, w, None, None, z, y)
    assert torch.equal(z[:, 0], v)
    want = O.activation(np64(v), act)
    close(np64(y)[:, 0], want, half * np.abs(want) + own_error("bf16", np.minimum(np.abs(np64(v)), 40), want), "y")
    dz = torch.empty(1, 8, dtype=dtype, device="cuda")
    ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
    dx = torch.empty(n, 8, dtype=dtype, device="cuda")
    A.dsv4v_linear_backward(layer, x, w, z, torch.ones_like(y), dx, None, None, ws)
    want = O.derivative(np64(v), act)
    close(np64(dx)[:, 0], want, half * np.abs(want) + 1e-6 * (1 + np.minimum(np.abs(np64(v)), 40)), "dx")
    # what is not finite stays in its own row
    x[5, 0], x[9, 0], x[11, 1] = float("nan"), float("inf"), float("inf")
    A.dsv4v_linear_forward(layer, x, w, None, None, z, y)
    got = np64(y)[:, 0]
    ok = np.ones(n, bool)
    ok[[5, 9, 11]] = False
    assert np.isnan(got[5]) and got[9] == np.inf and np.isnan(got[11]) and np.isfinite(got[ok]).all()


# ---------------------------------------------------------------------------------------------- backward
def run_backward(kind, rows, k, n, act, want=("dx", "dw", "db"), ld_x=None, ld_w=None, ld_y=None, offset=0, seed=0):
    dtype, code, half = TYPES[kind]
    pad = pad8 if kind == "bf16" else (lambda v: v)
    ld_x, ld_w, ld_y = ld_x or pad(k), ld_w or pad(k), ld_y or n
    x = Guarded(rows, k, ld_x, dtype, fill=normal((rows, k), 1.0, dtype, seed))
    w = Guarded(n, k, ld_w, dtype, fill=normal((n, k), n ** -0.5, dtype, seed + 1))
    z = Guarded(rows, n, ld_y, dtype, offset, fill=normal((rows, n), 1.5, dtype, seed + 2)) if act != "none" else None
    dy = Guarded(rows, n, ld_y, dtype, offset, fill=normal((rows, n), 1.0, dtype, seed + 3))
    out = {"dx": Guarded(rows, k, ld_x, dtype), "dw": Guarded(n, k, ld_w, dtype), "db": Guarded(1, n, n, torch.float32)}
    give = lambda key: None if key not in want else (out[key].t.reshape(-1) if key == "db" else out[key].t)  # noqa: E731
    layer = A.make_linear(rows, k, n, ACT[act], code, ld_x=ld_x, ld_w=ld_w, ld_z=ld_y, ld_y=ld_y)
    ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda").fill_(255)
    A.dsv4v_linear_backward(layer, x.t if "dw" in want else None, w.t if "dx" in want else None, z.t if z else None, dy.t,
                            give("dx"), give("dw"), give("db"), ws)
    assert A.dsv4v_device_error() == 0
    xs, wsd, zs, dys = np64(x.t), np64(w.t), (np64(z.t) if z else np.zeros((rows, n))), np64(dy.t)
    dx, dw, db, dz = O.backward(xs, wsd, zs, dys, act)
    off = (half * np.abs(dz) + 1e-6 * (1 + np.abs(zs)) * np.abs(dys)) if act != "none" else np.zeros_like(dz)
    if "dx" in want:
        tol = half * np.abs(dx) + off @ np.abs(wsd) + accumulate(kind, n, np.abs(dz) @ np.abs(wsd))
        close(np64(out["dx"].t), dx, tol, "dx")
        if kind == "bf16" and rows * k >= 64:
            assert np.linalg.norm(np64(out["dx"].t) - dx) <= 2.0 ** -7 * np.linalg.norm(dx)
    if "dw" in want:
        tol = half * np.abs(dw) + off.T @ np.abs(xs) + accumulate(kind, rows, np.abs(dz).T @ np.abs(xs))
        close(np64(out["dw"].t), dw, tol, "dw")
        if kind == "bf16" and k * n >= 64:
            assert np.linalg.norm(np64(out["dw"].t) - dw) <= 2.0 ** -7 * np.linalg.norm(dw)
    if "db" in want:
        tol = (rows + 16) * 2.0 ** -24 * np.abs(dz).sum(0) + (1e-6 * ((1 + np.abs(zs)) * np.abs(dys)).sum(0) if act != "none" else 0)
        close(np64(out["db"].t)[0], db, tol + 2.0 ** -24 * np.abs(db), "db")
    for key in out:
        if key in want:
            assert out[key].untouched(), key
        else:
            assert bool((out[key].buf == 7.0).all()), key


@pytest.mark.parametrize("rows,k,n", SHAPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_backward(rows, k, n, act):
    run_backward("bf16", rows, k, n, act)


@pytest.mark.parametrize("rows,k,n", [(1, 1, 1), (1, 300, 5), (63, 17, 65), (64, 16, 64), (130, 588, 97), (777, 588, 201), (1100, 60, 6),
                                      (300, 130, 300), (257, 64, 1000), (5, 60, 1100), (2100, 400, 1001)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_backward_fp32(rows, k, n, act):
    run_backward("f32", rows, k, n, act)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dx", "dw"), ()])
def test_linear_backward_each_gradient_alone(kind, act, want):
    run_backward(kind, 140, 72, 200, act, want)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("rows,k,n,ld_y,offset", [(40, 72, 64, 72, 0), (40, 72, 64, 67, 0), (40, 72, 64, 72, 1), (40, 70, 61, 61, 3),
                                                  (3000, 72, 1153, 1160, 0), (3000, 71, 1160, 1161, 5)])
def test_linear_backward_strides(kind, act, rows, k, n, ld_y, offset):
    run_backward(kind, rows, k, n, act, ld_x=pad8(k) + 16, ld_w=pad8(k) + 8, ld_y=ld_y, offset=offset)


def test_linear_fp32_values_that_bf16_cannot_hold():
    # the fp32 products go through bf16 parts: the largest finite values, infinities and NaN come out as in fp32
    rows, k, n = 40, 100, 70
    x, w = normal((rows, k), 1.0, torch.float32, 1), normal((n, k), 1.0, torch.float32, 2)
    big = torch.finfo(torch.float32).max
    x[3], w[5] = 0.0, 0.0
    x[3, 7], w[5, 9] = big, -big           # rounds to a bf16 infinity
    x[8, 1], x[9, 2], x[10, 4] = float("inf"), float("nan"), -float("inf")
    w[20, 1] = 0.0                          # infinity times zero
    x[11], x[12] = 1e-30, 1e30
    with np.errstate(invalid="ignore"):
        want = np64(x) @ np64(w).T
    y = torch.empty(rows, n, device="cuda")
    A.dsv4v_linear_forward(A.make_linear(rows, k, n, dtype=A.DSV4V_F32), x, w, None, None, None, y)
    got = np64(y)
    over = np.isfinite(want) & (np.abs(want) > big)
    want[over] = np.sign(want[over]) * np.inf
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    ok = np.isfinite(want)
    terms = np.abs(np.nan_to_num(np64(x), posinf=0, neginf=0)) @ np.abs(np64(w)).T
    close(got[ok], want[ok], (accumulate("f32", k, terms) + 2.0 ** -24 * np.abs(np.nan_to_num(want)))[ok], "y")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_linear_without_rows(kind):
    dtype, code, _ = TYPES[kind]
    layer = A.make_linear(0, 72, 33, A.ACT_SILU, code)
    x, y = torch.empty(0, 72, dtype=dtype, device="cuda"), torch.empty(0, 33, dtype=dtype, device="cuda")
    w = normal((33, 72), 1.0, dtype, 0)
    A.dsv4v_linear_forward(layer, x, w, None, None, None, y)
    dw, db = torch.full((33, 72), 7.0, device="cuda").to(dtype), torch.full((33,), 7.0, device="cuda")
    ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
    A.dsv4v_linear_backward(layer, x, w, y, y, torch.empty_like(x), dw, db, ws)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_gradient_against_differences(act):
    # d(sum of y * g) along random directions, from differences of the fp64 forward, against the fp32 kernels' gradients
    rows, k, n, step = 50, 37, 29, 1e-5
    x, w, b, g = (normal(s, 1.0, torch.float32, i) for i, s in enumerate([(rows, k), (n, k), (n,), (rows, n)]))
    layer = A.make_linear(rows, k, n, ACT[act], A.DSV4V_F32)
    y, z = torch.empty(rows, n, device="cuda"), torch.empty(rows, n, device="cuda")
    A.dsv4v_linear_forward(layer, x, w, b, None, z, y)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
    A.dsv4v_linear_backward(layer, x, w, z, g, dx, dw, db, ws)
    rng = np.random.default_rng(1)
    value = lambda X, W, B: float((O.forward(X, W, B, None, act)[0] * np64(g)).sum())  # noqa: E731
    at = [np64(x), np64(w), np64(b)]
    for i, d in enumerate((dx, dw, db)):
        u = rng.standard_normal(at[i].shape)
        hi, lo = [a.copy() for a in at], [a.copy() for a in at]
        hi[i] += step * u
        lo[i] -= step * u
        want = (value(*hi) - value(*lo)) / (2 * step)
        got = float((np64(d) * u).sum())
        assert abs(got - want) <= 1e-4 * float(np.abs(np64(d) * u).sum())


def test_linear_calls_are_repeatable():
    # the same bits each time, the split paths among them
    for rows, k, n in ((1, 4608, 512), (784, 1024, 2816), (3000, 200, 1160)):
        x, w, dy = normal((rows, k), 1.0, torch.bfloat16, 1), normal((n, k), 0.02, torch.bfloat16, 2), normal((rows, n), 1.0, torch.bfloat16, 3)
        layer = A.make_linear(rows, k, n, A.ACT_GELU)
        ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
        seen = []
        for _ in range(3):
            y, z = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
            dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
            A.dsv4v_linear_forward(layer, x, w, None, None, z, y)
            A.dsv4v_linear_backward(layer, x, w, z, dy, dx, dw, db, ws)
            seen.append((y, z, dx, dw, db))
        for other in seen[1:]:
            assert all(torch.equal(a, b) for a, b in zip(seen[0], other))


def test_linear_on_another_stream_and_two_at_once():
    # two streams, each with its own buffers, at the same time
    rows, k, n = 300, 1024, 520
    layer = A.make_linear(rows, k, n, A.ACT_SILU)
    want, got, streams, sets = [], [], [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(2):
        x, w, dy = normal((rows, k), 1.0, torch.bfloat16, 10 * i), normal((n, k), 0.02, torch.bfloat16, 10 * i + 1), normal((rows, n), 1.0, torch.bfloat16, 10 * i + 2)
        sets.append((x, w, dy))

    def run(i, stream=None):
        x, w, dy = sets[i]
        y, z = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
        ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
        A.dsv4v_linear_forward(layer, x, w, None, None, z, y, stream=stream)
        A.dsv4v_linear_backward(layer, x, w, z, dy, dx, dw, db, ws, stream=stream)
        return y, z, dx, dw, db, ws

    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(i, streams[i].cuda_stream) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a[:5], b[:5]))


def test_linear_beyond_32_bit_offsets():
    # outputs of over 2^31 elements: the last rows are those of a layer of their own
    rows, k, n, last = 70001, 16, 32776, 300
    x, w = normal((rows, k), 1.0, torch.bfloat16, 1), normal((n, k), 0.25, torch.bfloat16, 2)
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    A.dsv4v_linear_forward(A.make_linear(rows, k, n, A.ACT_SILU), x, w, None, None, None, y)
    want = O.forward(np64(x[-last:]), np64(w), act="silu")[0]
    assert np.linalg.norm(np64(y[-last:]) - want) <= 2.0 ** -8 * np.linalg.norm(want)
    layer = A.make_linear(rows, k, n)
    ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
    y[:-last] = 0  # d_y: only the last rows count
    A.dsv4v_linear_backward(layer, x, w, None, y, dx, dw, db, ws)
    dy = np64(y[-last:])
    want_dx, want_dw, want_db, _ = O.backward(np64(x[-last:]), np64(w), None, dy)
    for got, want in ((dx[-last:], want_dx), (dw, want_dw)):
        assert np.linalg.norm(np64(got) - want) <= 2.0 ** -8 * np.linalg.norm(want)
    assert np.abs(np64(db) - want_db).max() <= (last + 16) * 2.0 ** -24 * np.abs(dy).sum(0).max()
    assert not dx[:-last].any() and A.dsv4v_device_error() == 0


FIRST_CALL = """
import torch
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A
x, w = torch.randn(300, 256, device="cuda").bfloat16(), torch.randn(304, 256, device="cuda").bfloat16()
y, z = torch.empty(300, 304, device="cuda").bfloat16(), torch.empty(300, 304, device="cuda").bfloat16()
dx, dw, db, norm = torch.empty_like(x), torch.empty_like(w), torch.empty(304, device="cuda"), torch.empty((), device="cuda")
m, v = torch.zeros(w.numel(), device="cuda"), torch.zeros(w.numel(), device="cuda")
layer = A.make_linear(300, 256, 304, A.ACT_GELU)
ws = torch.empty(A.dsv4v_linear_backward_workspace_size(layer), dtype=torch.uint8, device="cuda")
grads, table = A.GradTable([dw, db]), A.AdamwTable([dict(param=w, grad=dw, exp_avg=m, exp_avg_sq=v)])
nws = torch.empty(A.dsv4v_grad_norm_workspace_size(grads), dtype=torch.uint8, device="cuda")
def step():
    A.dsv4v_linear_forward(layer, x, w, None, None, z, y)
    A.dsv4v_linear_backward(layer, x, w, z, y, dx, dw, db, ws)
    A.dsv4v_grad_norm(grads, norm, nws)
    A.dsv4v_adamw_step(A.make_adamw(1e-3), table, grad_norm=norm)
w0 = w.clone()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, dx, dw, db, norm, w)]
w.copy_(w0), m.zero_(), v.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw, db, norm, w))) and not torch.equal(w, w0)
print("first call captured")
"""


def test_a_programs_first_calls_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, cwd=root, timeout=240)
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stderr[-2000:]
