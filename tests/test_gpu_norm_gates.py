"""Gates of the norm over the whole range of a sigmoid, forward and backward, against the float64 oracle.

The bounds are those of test_gpu_norm.  Below -87 a sigmoid is among FP32's smallest numbers, where its rounding is a step of
2^-149 whatever its size: times |z| <= 130 and the values that it multiplies (|v| and |dy w h| stay below 8 here) that is less
than 2^-138, which every output may be off besides the half step of its own type's smallest numbers (bf16 2^-134).
"""
import pytest

import test_gpu_norm as base
from gpu_util import DEV, require_gpu, torch_dtype

pytestmark = pytest.mark.gpu
TINY = {"f32": 2.0 ** -138, "bf16": 2.0 ** -134 + 2.0 ** -138, "f16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gates(dt):
    """Every value of a 16-bit type up to 130 in size; in FP32 an even sweep of [-110, -80] and one of [-130, 130]."""
    import torch
    if dt == "f32":
        return torch.cat([torch.linspace(-110, -80, 30_001), torch.linspace(-130, 130, 30_000)])
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch_dtype(dt))
    return v[v.float().abs() <= 130]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gate", ["before", "after"])
@pytest.mark.parametrize("width,groups,rms", [(256, 2, True), (1000, 1, False)])
def test_every_gate(dt, gate, width, groups, rms, monkeypatch):
    import torch
    z = gates(dt)
    z = z[torch.randperm(z.numel(), generator=torch.Generator().manual_seed(3))]
    rows = z.numel() // width
    plain = base.make

    def make(*a, **kw):
        d, r = plain(*a, **kw)
        d["z"] = z[:rows * width].view(rows, width).to(DEV)
        r["z"] = d["z"].double().cpu().numpy()
        return d, r
    monkeypatch.setattr(base, "make", make)
    monkeypatch.setattr(base, "TINY", TINY)
    base.check(rows, width, groups, dt, rms, False, gate)


@pytest.mark.parametrize("after", [False, True])
def test_far_and_nonfinite_gates(after):
    """A gate far below zero closes: what it multiplies is zero.  NaN and infinities stay in their own slice."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    x, z, w = torch.ones((4, 256), device=DEV), torch.ones((4, 256), device=DEV), torch.ones(256, device=DEV)
    z[0, 3], z[0, 7] = -1e30, -torch.finfo(torch.float32).max
    z[1, 5], z[2, 5], z[3, 5] = float("nan"), float("inf"), -float("inf")
    y, mean, rstd = gdn.gdn_layer_norm(x, w, gate=z, groups=2, rms=True, gate_after=after, save_stats=True)
    g = gdn.gdn_layer_norm_backward(torch.ones_like(x), x, w, mean, rstd, gate=z, groups=2, rms=True, gate_after=after)
    assert (y[0, [3, 7]] == 0).all() and y[0].isfinite().all() and g.dx[0].isfinite().all()
    assert (g.dgate[0, [3, 7]] == 0).all() and (after or (g.dx[0, [3, 7]] == 0).all())
    assert y[:, 128:].isfinite().all() and g.dx[:, 128:].isfinite().all() and g.dgate[:, 128:].isfinite().all()
    for row in (1, 2, 3):
        assert not y[row, 5].isfinite()
