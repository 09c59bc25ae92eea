"""The optimizer step without a GPU: pins of its oracle, workspace sizes, and the refusals of bad arguments,
which come before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dsv4v_optim as O
from vision_transformer_encoder_dsv4v_b200 import build
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A


@pytest.fixture(scope="module")
def lib():
    build.build()
    return A.lib()


# ---------------------------------------------------------------------------------------------- oracle
def test_e4m3_values_are_the_types():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = O.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(codes))
    assert np.array_equal(got[~np.isnan(got)], codes[~np.isnan(codes)])


def test_block_scale_closed_forms():
    assert O.block_scale(0.0) == 0.0
    assert O.block_scale(448.0) == 1.0 and O.block_scale(448.5) == 2.0 and O.block_scale(224.0) == 0.5
    assert O.block_scale(1e-45) == 2.0 ** -126


def test_adamw_first_step_is_the_sign():
    # from zero moments the corrected ratio is g / |g|, whatever the betas
    g = np.array([3.0, -0.25, 1e-3])
    p, m, v = O.adamw(np.zeros(3), g, np.zeros(3), np.zeros(3), 1, 0.01, 0.9, 0.999, 1e-12)
    np.testing.assert_allclose(p, -0.01 * np.sign(g), rtol=1e-8)
    np.testing.assert_allclose(m, 0.1 * g)
    np.testing.assert_allclose(v, 0.001 * g * g)


def test_adamw_matches_torchs_optimizer():
    rng = np.random.default_rng(0)
    w = torch.nn.Parameter(torch.from_numpy(rng.standard_normal(50)))
    opt = torch.optim.AdamW([w], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.2)
    p, m, v = w.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        w.grad = torch.from_numpy(g.copy())
        norm = O.grad_norm([g])
        torch.nn.utils.clip_grad_norm_([w], 2.0)
        opt.step()
        p, m, v = O.adamw(p, g, m, v, step, 3e-3, 0.8, 0.95, 1e-6, 0.2, norm, 2.0)
        np.testing.assert_allclose(p, w.detach().numpy(), rtol=1e-6)


def test_grad_norm_closed_form():
    assert O.grad_norm([np.full(9, 2.0), np.array([8.0])]) == 10.0
    assert O.grad_norm([]) == 0.0


# ---------------------------------------------------------------------------------------------- refusals
AL = 4096  # an aligned address that nothing dereferences


def grad(**kw):
    return A.Grad(**dict(dict(data=AL, n=10, dtype=A.DSV4V_BF16), **kw))


def call_norm(lib, g, n=1, out=AL, ws=AL, ws_bytes=1 << 30):
    return lib.dsv4v_grad_norm(ctypes.byref(g) if g is not None else None, n, out, ws, ws_bytes, None)


def test_grad_norm_workspace_size(lib):
    assert A.dsv4v_grad_norm_workspace_size(-1) == 0
    one = A.dsv4v_grad_norm_workspace_size(0)
    assert one == A.dsv4v_grad_norm_workspace_size(1) > 0 and one % 256 == 0
    assert A.dsv4v_grad_norm_workspace_size(10000) > one


def test_grad_norm_refusals(lib):
    assert call_norm(lib, grad(), n=-1) == 1
    assert call_norm(lib, None) == 1
    assert call_norm(lib, grad(n=-1)) == 1
    assert call_norm(lib, grad(data=None)) == 1
    assert call_norm(lib, grad(dtype=7)) == 1
    assert call_norm(lib, grad(data=AL + 1)) == 1  # not aligned to bf16
    assert call_norm(lib, grad(data=AL + 2, dtype=A.DSV4V_F32)) == 1
    assert call_norm(lib, grad(), out=None) == 1
    assert call_norm(lib, grad(), out=AL + 2) == 1
    assert call_norm(lib, grad(n=(1 << 40) + 1)) == 2
    assert call_norm(lib, grad(), ws=None) == 3
    assert call_norm(lib, grad(), ws=AL + 16) == 3
    assert call_norm(lib, grad(), ws_bytes=100) == 3


def tensor(**kw):
    d = dict(param=AL, grad=AL, master=None, exp_avg=AL, exp_avg_sq=AL, exp_avg_scale=None, exp_avg_sq_scale=None, n=10,
             param_dtype=A.DSV4V_BF16, grad_dtype=A.DSV4V_BF16, state_bits=32, weight_decay=0.0)
    return A.AdamwTensor(**dict(d, **kw))


def call_step(lib, t=None, cfg=None, n=1, norm=None, lr=None, step=None):
    t = tensor() if t is None else t
    cfg = A.make_adamw(1e-3) if cfg is None else cfg
    return lib.dsv4v_adamw_step(ctypes.byref(cfg), ctypes.byref(t), n, norm, lr, step, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param_dtype=2),
    dict(grad_dtype=-1), dict(state_bits=16), dict(weight_decay=-0.1), dict(weight_decay=float("nan")),
    dict(weight_decay=float("inf")), dict(param=AL + 1), dict(grad=AL + 1), dict(param=AL + 2, param_dtype=A.DSV4V_F32),
    dict(master=AL, param_dtype=A.DSV4V_F32), dict(master=AL + 2), dict(exp_avg=AL + 2), dict(exp_avg_sq=AL + 2),
    dict(exp_avg_scale=AL), dict(state_bits=8), dict(state_bits=8, exp_avg_scale=AL),
    dict(state_bits=8, exp_avg_scale=AL, exp_avg_sq_scale=AL + 2)])
def test_adamw_refuses_tensors(lib, bad):
    assert call_step(lib, tensor(**bad)) == 1


@pytest.mark.parametrize("bad", [
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-60),
    dict(eps=float("inf")), dict(lr=float("inf")), dict(lr=float("nan")), dict(step=0), dict(max_grad_norm=-1.0),
    dict(max_grad_norm=float("inf")), dict(max_grad_norm=1.0)])  # the last: clipping without a norm
def test_adamw_refuses_hyperparameters(lib, bad):
    assert call_step(lib, cfg=A.make_adamw(**dict(dict(lr=1e-3), **bad))) == 1


def test_adamw_refuses_calls(lib):
    cfg = A.make_adamw(1e-3)
    t = tensor()
    assert lib.dsv4v_adamw_step(None, ctypes.byref(t), 1, None, None, None, None) == 1
    assert lib.dsv4v_adamw_step(ctypes.byref(cfg), None, 1, None, None, None, None) == 1
    assert call_step(lib, n=-1) == 1
    assert call_step(lib, norm=AL + 2) == 1
    assert call_step(lib, lr=AL + 1) == 1
    assert call_step(lib, step=AL + 4) == 1
    assert call_step(lib, tensor(n=(1 << 40) + 1)) == 2


def test_tables_refuse_host_tensors():
    with pytest.raises(ValueError, match="on cpu"):
        A.GradTable([torch.zeros(3)])
    x = torch.zeros(3)
    with pytest.raises(ValueError, match="on cpu"):
        A.AdamwTable([dict(param=x, grad=x, exp_avg=x, exp_avg_sq=x)])
