"""The norm and rotation of more tokens than a launch has turns for, and of values whose squares are large."""
import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
import test_gpu_qk as base
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_more_turns_than_workgroups():
    """One head of 16 takes 16 tokens a turn, and the forward launch has 2^20 workgroups: those in front take a second turn.  Rows do not
    depend on one another, so two calls of half the tokens give the same bits."""
    n = 2 ** 24 + 16 * 700 + 5
    g = torch.Generator(device=DEV).manual_seed(9)
    q, k = (torch.randn((n, 1, 16), generator=g, device=DEV).bfloat16() for _ in range(2))
    w, pos = torch.rand(16, generator=g, device=DEV) + 0.5, torch.arange(n, dtype=torch.int32, device=DEV)
    f = torch.tensor([1.0, 0.3, 0.1, 0.03, 0.01, 0.003, 0.001, 0.0003], device=DEV)
    whole = gdn.gdn_qk_norm_rope(q, k, w, w, pos, f)
    half = n // 2
    for at in (slice(0, half), slice(half, n)):
        part = gdn.gdn_qk_norm_rope(q[at], k[at], w, w, pos[at], f)
        assert all(torch.equal(a[at], b) for a, b in zip(whole, part))
    rows = slice(n - 40, n)
    assert not whole[0][rows].isnan().any() and whole[0][rows].float().abs().mean() > 0.1


def test_values_whose_squares_are_large():
    """Rows of 1e18, whose squares are 2^119, and of zeros: results and gradients are finite."""
    v = base.make(4, 2, 2, 64, 64, "f32")
    v["q"][0], v["k"][1], v["q"][2] = 0.0, 0.0, 1e18
    v["dq"][2] = 0.0
    args = (v["q"], v["k"], v["qw"], v["kw"], v["pos"], v["freq"])
    for t in (*gdn.gdn_qk_norm_rope(*args), *gdn.gdn_qk_norm_rope_backward(v["dq"], v["dk"], *args)):
        assert t.isfinite().all()
