"""Sines and cosines of the rotation in binary32, where the angle's last bits count."""
import numpy as np
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_angles_next_to_half_a_turn(layout):
    """Positions next to odd multiples of pi, frequency 1: the sine is 0.1 to 1e-6 and has its own 24 bits.  The angle
    in binary64 is off by 2^-52 of itself at most (the constant 1 / (2 pi) by 2^-54, the product by 2^-53), the sine of
    the rounded angle by 2 units in its last place, what rounding left out by 2^-22 of it, their sum and the product
    with 1 by a half each: 2^-21 in all.  An angle rounded to binary32 would be off by up to 2^-26 of a turn, 9e-8."""
    q4 = lib()
    at = [3, 22, 355, 355 * 3, 355 * 5, 103993, 104348, 208341, 312689 * 3, 22 * 41]
    pos = torch.tensor(at + [-p for p in at], dtype=torch.int32, device="cuda")
    x = torch.zeros(len(pos), 1, 2, device="cuda")
    x[:, 0, 0] = 1.0
    got = q4.q4_rope(x, pos, torch.ones(1, dtype=torch.float64, device="cuda"), layout)[:, 0].double().cpu().numpy()
    p = pos.cpu().numpy().astype(np.float64)
    for column, want in ((0, np.cos(p)), (1, np.sin(p))):
        assert (np.abs(got[:, column] - want) <= 2.0 ** -21 * np.abs(want) + 2.0 ** -52 * np.abs(p)).all(), (got[:, column], want)
