"""A call's status is its own: an error that an earlier call of the thread returned does not come back from a later one."""
import ctypes

import pytest
import torch

from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu

DSV4V_ERR_CUDA = 4


def leave_an_error():
    # waiting for a stream that is being captured is refused by the runtime, on the host, and ends the capture
    from cuda.bindings import runtime as rt
    err, stream = rt.cudaStreamCreate()
    assert err == rt.cudaError_t.cudaSuccess
    assert rt.cudaStreamBeginCapture(stream, rt.cudaStreamCaptureMode.cudaStreamCaptureModeRelaxed)[0] == rt.cudaError_t.cudaSuccess
    status = A.lib().dsv4v_device_error(ctypes.c_void_p(int(stream)))
    rt.cudaStreamEndCapture(stream)
    rt.cudaStreamDestroy(stream)
    assert status == DSV4V_ERR_CUDA


def test_an_optimizer_step_that_was_taken_is_not_reported_as_failed():
    w, g = torch.ones(10, device="cuda"), torch.ones(10, device="cuda")
    table = A.AdamwTable([dict(param=w, grad=g, exp_avg=torch.zeros(10, device="cuda"), exp_avg_sq=torch.zeros(10, device="cuda"))])
    leave_an_error()
    A.dsv4v_adamw_step(A.make_adamw(0.5), table)
    torch.cuda.synchronize()
    assert torch.allclose(w, torch.full_like(w, 0.5))


def test_an_fp32_norm_that_ran_is_not_reported_as_failed():
    x, w = torch.ones(4, 128, device="cuda"), torch.full((128,), 2.0, device="cuda")
    y = torch.empty_like(x)
    leave_an_error()
    A.dsv4v_rmsnorm(A.make_config(128, 2, 256, 2, 256, 1, dtype=A.DSV4V_F32), 4, x, w, y)
    assert torch.allclose(y, torch.full_like(y, 2.0), rtol=1e-5)
