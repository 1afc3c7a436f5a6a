"""The rotation's angles at far positions, against angles reduced exactly as rational numbers.

Every pair is (1, 0) and eps is 1/2, so that a head is normed to itself and its pairs become (cos, sin).  What is off: the reduced angle's
rounding to FP32, at most 2^-26 quarter turns; the sine's and cosine's own error, 2 steps of 2^-24; the norm's reciprocal root and the
product with it, a step each.  A product of FP64 alone is off by up to 2^-22 radians at an angle of 2^31, four steps more, and
angles of five times that are among these.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
from gpu_util import DEV, require_gpu, say

pytestmark = pytest.mark.gpu
PI = Fraction("3.141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067")
TOL = 2.0 ** -26 * np.pi / 2 + 4 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def exact(positions, freq):
    """cos and sin [T, P] of the angles, whose turns are reduced before anything is rounded."""
    angle = np.empty((len(positions), len(freq)))
    for j, f in enumerate(freq):
        turn = Fraction(float(f)) / (2 * PI)
        for i, p in enumerate(positions):
            t = int(p) * turn
            angle[i, j] = 2 * np.pi * float(t - round(t))
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("start", [0, 10 ** 6, 2 ** 27 + 1, 2 ** 31 - 300, -(2 ** 31)])
@pytest.mark.parametrize("neighbours", [False, True])
def test_angles(start, neighbours):
    say(f"qk angles from {start} neighbours={neighbours}")
    T, d = 300, 64
    freq = np.float32(1e4 ** (-np.arange(0, d, 2) / d))
    freq[1:3] = 0.7, 5.3
    pos = start + np.arange(T)
    x = torch.zeros(T, 1, d, device=DEV)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if neighbours else (slice(0, d // 2), slice(d // 2, None))
    x[..., first] = 1.0
    one = torch.ones(d, device=DEV)
    y, _ = gdn.gdn_qk_norm_rope(x, x, one, one, torch.from_numpy(pos).to(torch.int32).to(DEV), torch.from_numpy(freq).to(DEV), eps=0.5,
                                neighbours=neighbours)
    c, s = exact(pos, freq)
    y = y[:, 0].double().cpu().numpy()
    for got, want in ((y[:, first], c), (y[:, second], s)):
        err = np.abs(got - want).max()
        say(f"largest error {err:.2e} of {TOL:.2e}")
        assert err <= TOL
