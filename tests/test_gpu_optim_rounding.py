"""What the optimizer's operators lose to rounding, on inputs that are made to show it.

u = 2^-24 is half a step of fp32."""
import numpy as np
import pytest
import torch

from oracle import dsv4v_optim as O
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def np64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def norm_of(grads):
    table = A.GradTable(grads)
    out = torch.full((), -1.0, device="cuda")
    ws = torch.empty(A.dsv4v_grad_norm_workspace_size(table), dtype=torch.uint8, device="cuda")
    A.dsv4v_grad_norm(table, out, ws)
    return out


# ---------------------------------------------------------------------------------------------- norm
# One value of 1 and squares just below u behind it: an fp32 sum that holds the 1 loses each of them.  Eight squares take
# eight roundings, at most 8 u of their sum: 4 u of the norm, and u for its own rounding.  Sums of sixteen would lose 15 u
# here, 7.4 u of the norm.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def ones_among_small(n, piece, runs, dtype):
    # pieces of `piece` elements, 256 of them side by side; of each `runs` such rows the first has the ones
    i = torch.arange(n)
    one = (i % piece == 0) & (i // (256 * piece) % runs == 0)
    return torch.where(one, 1.0, 2.0 ** -12 * (1 - 2.0 ** -8)).to(dtype)


def at_offset(g, offset):
    buf = torch.zeros(g.numel() + offset, dtype=g.dtype, device="cuda")
    buf[offset:] = g
    return buf[offset:]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("piece,runs", [(8, 1), (8, 2), (4, 2), (4, 4), (16, 1)])
@pytest.mark.parametrize("offset", [0, 1])
def test_grad_norm_keeps_what_a_large_neighbour_hides(dtype, piece, runs, offset):
    g = at_offset(ones_among_small(8 * 8192, piece, runs, dtype), offset)
    want = O.grad_norm([np64(g)])
    assert abs(float(norm_of([g])) - want) <= 5 * U * want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("piece,runs", [(8, 2), (4, 4)])
@pytest.mark.parametrize("n", [8192, 8193, 50000])
def test_grad_norm_does_not_depend_on_the_address(dtype, piece, runs, n):
    g = ones_among_small(n, piece, runs, dtype)
    got = [norm_of([at_offset(g, offset)]) for offset in range(8)]
    assert all(torch.equal(got[0], x) for x in got[1:])


# ---------------------------------------------------------------------------------------------- AdamW
@pytest.mark.parametrize("decay", [1e-8, 3e-8, 1e-7, 1e-6])
@pytest.mark.parametrize("on_device", [False, True])
def test_adamw_takes_a_small_decay_on_average(decay, on_device):
    # weights from 1 to 2, whose step (2 u) is above lr weight_decay, and updates of a few such steps: each result's
    # rounding is even over a step, so the mean over n weights is off by 2 u / sqrt(12 n) times a few, beside 20 u of
    # the update and of the decay
    n, lr, step = 1 << 20, 2.0 ** -20, 1000
    gen = torch.Generator().manual_seed(0)
    uniform = lambda lo, hi: (lo + (hi - lo) * torch.rand(n, generator=gen)).cuda()  # noqa: E731
    p, m, v = uniform(1, 2), uniform(-0.1, 0.1), uniform(1e-3, 1e-2)
    g = torch.randn(n, generator=gen).cuda()
    want, _, _ = O.adamw(np64(p), np64(g), np64(m), np64(v), step, lr, decay=decay / lr)
    size = np.abs(want - np64(p)).max()
    table = A.AdamwTable([dict(param=p, grad=g, exp_avg=m, exp_avg_sq=v, weight_decay=decay / lr)])
    if on_device:
        count, rate = torch.tensor(step - 1, device="cuda"), torch.tensor(lr, device="cuda")
        A.dsv4v_adamw_step(A.make_adamw(1.0), table, lr_dev=rate, step_dev=count)
    else:
        A.dsv4v_adamw_step(A.make_adamw(lr, step=step), table)
    mean = (np64(p) - want).mean()
    assert abs(mean) <= 6 * 2 * U / np.sqrt(12 * n) + 20 * U * size
