"""Written matrices of the Linear layer that are another argument: refused before any CUDA call."""
import ctypes

import pytest

from vision_transformer_encoder_dsv4v_b200 import build
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

X, W, R, Z, Y, DX, DW = (4096 * (i + 1) for i in range(7))  # aligned addresses that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return A.lib()


@pytest.mark.parametrize("dtype", [A.DSV4V_BF16, A.DSV4V_F32])
@pytest.mark.parametrize("bad", [dict(y=X), dict(y=W), dict(z=X), dict(z=W), dict(z=Y), dict(z=R)])
def test_forward_refuses_an_output_that_is_an_input(lib, dtype, bad):
    p = dict(dict(x=X, w=W, residual=R, z=Z, y=Y), **bad)
    layer = A.make_linear(4, 64, 64, dtype=dtype)
    assert lib.dsv4v_linear_forward(ctypes.byref(layer), p["x"], p["w"], None, p["residual"], p["z"], p["y"], None) == 1


@pytest.mark.parametrize("rows", [0, 4])
def test_backward_refuses_a_gradient_in_the_weights_place(lib, rows):
    layer = A.make_linear(rows, 64, 64)
    assert lib.dsv4v_linear_backward(ctypes.byref(layer), X, W, None, Y, DX, W, None, 4096 * 20, 1 << 40, None) == 1
