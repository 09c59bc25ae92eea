"""Stochastic rounding of 8-bit optimizer states without a GPU: its oracle, the table's layout, the refusals."""
import ctypes

import numpy as np
import pytest

from oracle import dsv4v_optim as O
from vision_transformer_encoder_dsv4v_b200 import build
from vision_transformer_encoder_dsv4v_b200 import dsv4v as A


@pytest.fixture(scope="module")
def lib():
    build.build()
    return A.lib()


def test_philox_known_answers():
    # the published answers of ten rounds, for zeros and for all ones
    words = lambda c, k: [int(x) for x in O.philox(c, k, 10)]  # noqa: E731
    assert words((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert words((ones,) * 4, (ones, ones)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_draws_differ_by_step_tensor_and_element():
    m, v = O.draws(5000, 7, 3)
    every = [m, v, *O.draws(5000, 8, 3), *O.draws(5000, 7, 4), *O.draws(5000, 7 + (1 << 32), 3)]
    assert len(np.unique(np.concatenate(every))) > 40000 * 0.99
    for u in every:
        assert 0 <= u.min() and u.max() < 1
        assert abs(u.mean() - 0.5) < 5 * (1 / 12 / 5000) ** 0.5
    for i, a in enumerate(every):
        for b in every[i + 1:]:
            assert abs(np.corrcoef(a, b)[0, 1]) < 5 / 5000 ** 0.5
    again = O.draws(17, 7, 3)
    assert np.array_equal(again[0], m[:17]) and np.array_equal(again[1], v[:17])


def test_neighbours():
    lo, hi = O.code_neighbours(np.array([0.0, 2.0 ** -10, 2.0 ** -9, 1.0, 1.06, 447.0, 448.0]))
    assert np.array_equal(lo, [0, 0, 2.0 ** -9, 1, 1, 416, 448])
    assert np.array_equal(hi, [2.0 ** -9, 2.0 ** -9, 2.0 ** -8, 1.125, 1.125, 448, 480])


def test_expectations_are_kept():
    # the mean over many steps' draws, within five of its deviations (a draw's is at most half the gap, 1/8 of the value
    # for the first moment and 17/64 for the second)
    m = np.array([448.0, 1.03, -1.1, 3e-3, -200.0, 0.0])
    v = np.array([448.0, 1.03, 1.2, 3e-3, 200.0, 0.0]) ** 2
    n, sm, sv = 4000, np.zeros(6), np.zeros(6)
    for step in range(1, n + 1):
        qm, qr, em, er = O.stochastic_codes(m, v, step, 0)
        assert em[0] == 1 and er[0] == 1
        sm, sv = sm + qm, sv + qr ** 2
    assert np.all(np.abs(sm / n - m) <= 5 * (np.abs(m) / 16 + 2.0 ** -10) / n ** 0.5)
    assert np.all(np.abs(sv / n - v) <= 5 * (v * 17 / 128 + 2.0 ** -19) / n ** 0.5)


def test_a_small_root_is_raised_to_the_smallest_code():
    for step in range(1, 20):
        _, qr, _, _ = O.stochastic_codes(np.zeros(3), np.array([448.0 ** 2, 1e-12, 0.0]), step, 0)
        assert np.array_equal(qr, [448.0, 2.0 ** -9, 0.0])


# ---------------------------------------------------------------------------------------------- the interface
def test_the_tables_layout_is_as_it_was_before_the_field():
    # state_rounding lies in what was padding
    assert ctypes.sizeof(A.AdamwTensor) == 88
    assert A.AdamwTensor.state_bits.offset == 72 and A.AdamwTensor.state_rounding.offset == 76
    assert A.AdamwTensor.weight_decay.offset == 80


@pytest.mark.parametrize("bits,rounding,ok", [(8, 0, True), (8, 1, True), (8, 2, False), (8, -1, False), (32, 0, True), (32, 1, False)])
def test_roundings_that_are_refused(lib, bits, rounding, ok):
    at = 4096
    scale = at if bits == 8 else None
    # with an n that the library does not take, an accepted tensor gives the status behind the check
    t = A.AdamwTensor(at, at, None, at, at, scale, scale, (1 << 40) + 1, A.DSV4V_BF16, A.DSV4V_BF16, bits, rounding, 0.0)
    status = lib.dsv4v_adamw_step(ctypes.byref(A.make_adamw(1e-3)), ctypes.byref(t), 1, None, None, None, None)
    assert status == (2 if ok else 1)
