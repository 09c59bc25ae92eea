"""The Linear layer without a GPU: pins of its oracle, workspace sizes, and the refusals of bad arguments, which
come before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dsv4v_linear as O
from vision_transformer_encoder_dsv4v_b200 import build
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A


@pytest.fixture(scope="module")
def lib():
    build.build()
    return A.lib()


# ---------------------------------------------------------------------------------------------- oracle
def test_activations_closed_forms():
    v = np.array([0.0, 1.0, -1.0, 50.0, -50.0])
    np.testing.assert_allclose(O.activation(v, "gelu"), [0, 0.8413447460685429, -0.15865525393145707, 50, 0], atol=1e-15)
    np.testing.assert_allclose(O.activation(v, "silu"), [0, 0.7310585786300049, -0.2689414213699951, 50, 0], atol=1e-15)
    assert np.array_equal(O.activation(v, "none"), v)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_oracle_gradients_against_differences(act):
    rng = np.random.default_rng(0)
    x, w, b, g = rng.standard_normal((5, 4)), rng.standard_normal((3, 4)), rng.standard_normal(3), rng.standard_normal((5, 3))
    z = O.forward(x, w, b, None, act)[1]
    dx, dw, db, _ = O.backward(x, w, z, g, act)
    at, h = [x, w, b], 1e-6
    for i, d in enumerate((dx, dw, db)):
        for idx in np.ndindex(at[i].shape):
            hi, lo = [a.copy() for a in at], [a.copy() for a in at]
            hi[i][idx] += h
            lo[i][idx] -= h
            diff = sum(s * (O.forward(*p, None, act)[0] * g).sum() for s, p in ((1, hi), (-1, lo))) / (2 * h)
            assert abs(diff - d[idx]) < 1e-7 * max(1, abs(diff))


def test_oracle_matches_torchs_layers():
    rng = np.random.default_rng(1)
    x, w, b, r = (torch.from_numpy(rng.standard_normal(s)) for s in ((6, 5), (4, 5), (4,), (6, 4)))
    for act, f in (("gelu", torch.nn.functional.gelu), ("silu", torch.nn.functional.silu), ("none", lambda v: v)):
        want = f(torch.nn.functional.linear(x, w, b)) + r
        np.testing.assert_allclose(O.forward(x.numpy(), w.numpy(), b.numpy(), r.numpy(), act)[0], want.numpy(), rtol=1e-12)


# ---------------------------------------------------------------------------------------------- refusals
AL = 4096  # an aligned address that nothing dereferences
DX, DW, Z, Y, R = (AL * (i + 10) for i in range(5))


def forward(lib, layer, x=AL, w=2 * AL, bias=None, residual=None, z=None, y=Y):
    return lib.dsv4v_linear_forward(ctypes.byref(layer) if layer is not None else None, x, w, bias, residual, z, y, None)


def backward(lib, layer, x=AL, w=2 * AL, z=Z, d_y=Y, dx=DX, dw=DW, db=AL, ws=AL, ws_bytes=1 << 40):
    return lib.dsv4v_linear_backward(ctypes.byref(layer) if layer is not None else None, x, w, z, d_y, dx, dw, db, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), 1), (dict(rows=(1 << 30) + 1), 1), (dict(in_features=0), 1), (dict(out_features=0), 1),
    (dict(in_features=-5), 1), (dict(activation=3), 1), (dict(activation=-1), 1), (dict(dtype=2), 1),
    (dict(in_features=(1 << 20) + 8), 2), (dict(out_features=(1 << 20) + 1), 2),
    (dict(ld_x=56), 1), (dict(ld_w=56), 1), (dict(ld_y=7), 1), (dict(ld_z=7), 1), (dict(ld_residual=7), 1), (dict(ld_y=-8), 1),
    (dict(ld_x=68), 2), (dict(ld_w=66), 2), (dict(in_features=60), 2), (dict(ld_y=1 << 33), 2)])
def test_linear_refuses_layers(lib, bad, status):
    layer = A.make_linear(**dict(dict(rows=4, in_features=64, out_features=8, dtype=A.DSV4V_BF16), **bad))
    assert forward(lib, layer) == status
    assert backward(lib, layer) == status
    assert A.dsv4v_linear_backward_workspace_size(layer) == 0


def test_linear_forward_refuses_pointers(lib):
    layer = A.make_linear(4, 64, 8, A.ACT_GELU)
    assert forward(lib, None) == 1
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(x=AL + 8), dict(w=AL + 2), dict(y=Y + 1), dict(bias=AL + 8),
                dict(residual=R + 1), dict(z=Z + 1), dict(y=AL), dict(z=AL), dict(z=Y), dict(z=R, residual=R)):
        assert forward(lib, layer, **bad) == 1, bad
    strided = A.make_linear(4, 64, 8, ld_residual=16)
    assert forward(lib, strided, residual=Y) == 1  # in place with other strides
    f32 = A.make_linear(4, 63, 8, dtype=A.DSV4V_F32)
    for bad in (dict(x=AL + 2), dict(w=AL + 1), dict(y=Y + 2), dict(z=Z + 2)):
        assert forward(lib, f32, **bad) == 1, bad
    assert forward(lib, A.make_linear(0, 64, 8), x=None, w=None, y=None) == 0  # nothing to do


def test_linear_backward_refuses_pointers(lib):
    layer = A.make_linear(4, 64, 8, A.ACT_SILU)
    assert backward(lib, None) == 1
    for bad in (dict(d_y=None), dict(z=None), dict(w=None), dict(x=None), dict(d_y=Y + 1), dict(z=Z + 1), dict(x=AL + 8),
                dict(w=AL + 8), dict(dx=DX + 1), dict(dw=DW + 1), dict(db=AL + 2), dict(dx=Y), dict(dx=2 * AL), dict(dx=Z),
                dict(dw=AL), dict(dw=2 * AL), dict(dw=Y), dict(dw=Z), dict(dw=DX)):
        assert backward(lib, layer, **bad) == 1, bad


def test_linear_backward_workspace_size(lib):
    one = A.dsv4v_linear_backward_workspace_size(A.make_linear(1, 64, 8))
    assert 256 <= one < A.dsv4v_linear_backward_workspace_size(A.make_linear(784, 1024, 2816))
    # dz and, per strip of rows, the column sums
    assert A.dsv4v_linear_backward_workspace_size(A.make_linear(784, 1024, 2816)) >= 784 * 2816 * 2 + 2816 * 4
    assert A.dsv4v_linear_backward_workspace_size(A.make_linear(0, 64, 8)) >= 256


def test_binding_refuses_shapes_and_types():
    layer, bf16 = A.make_linear(4, 64, 8), torch.bfloat16
    good = lambda r, c: torch.zeros(r, c, dtype=bf16)  # noqa: E731
    if not torch.cuda.is_available():  # host tensors, and no device to be the current one
        assert A._device_index() == -1
    matrix = lambda t: A._matrix(t, "x", 4, 64, 0, bf16, -1)  # noqa: E731  (host tensors are on "device" -1)
    assert matrix(good(4, 64)) and matrix(None) is None
    for bad, match in [(torch.zeros(4, 64), "float32"), (good(4, 63), "shape"), (good(64, 4).t(), "strides"),
                       (good(4, 72)[:, :64], "strides")]:
        with pytest.raises(ValueError, match=match):
            matrix(bad)
    with pytest.raises(ValueError, match="on cpu"):
        A._matrix(good(4, 64), "x", 4, 64, 0, bf16, 0)
    assert layer.out_features == 8
