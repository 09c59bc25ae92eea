"""A few rows of the bf16 Linear layer on both sides of the widths where its kernels change, against fp64."""
import numpy as np
import pytest
import torch

from oracle import dsv4v_linear as O
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
@pytest.mark.parametrize("k", [72, 2048, 2056])
@pytest.mark.parametrize("side", [-1, 0, 1, 3000])
def test_linear_forward_of_a_few_rows_at_the_widths_limit(rows, k, side):
    n = 32 * torch.cuda.get_device_properties(0).multi_processor_count + side
    gen = torch.Generator().manual_seed(rows)
    normal = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, w = normal(rows, k).bfloat16().cuda(), (normal(n, k) * k ** -0.5).bfloat16().cuda()
    b, r = normal(n).cuda(), normal(rows, n).bfloat16().cuda()
    y, z = torch.full((rows, n), 7.0, device="cuda").bfloat16(), torch.full((rows, n), 7.0, device="cuda").bfloat16()
    A.dsv4v_linear_forward(A.make_linear(rows, k, n, A.ACT_SILU), x, w, b, r, z, y)
    assert A.dsv4v_device_error() == 0
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    want_y, want_z = O.forward(f(x), f(w), f(b), f(r), "silu")
    # a rounding to bf16 (2^-8), the activation's slope (1.1) times the sums' error ((K / 16 + 8) 2^-23 of their terms), its own 4e-7
    acc = (k / 16 + 8) * 2.0 ** -23 * (np.abs(f(x)) @ np.abs(f(w)).T + np.abs(f(b)))
    assert np.all(np.abs(f(z) - want_z) <= 2.0 ** -8 * np.abs(want_z) + acc)
    assert np.all(np.abs(f(y) - want_y) <= 2.0 ** -8 * np.abs(want_y) + 1.1 * acc + 4e-7 * (1 + np.abs(want_z)) + 2.0 ** -23 * np.abs(f(r)))
