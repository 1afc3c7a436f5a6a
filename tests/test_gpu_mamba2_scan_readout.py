"""What the scan reads from its recurrence, without the skip's D x in front of it: D is 0, B and C are of size 1, as a short
convolution leaves them.  Against the float64 oracle, forward and backward.

In bf16 the state and the decay-weighted products meet y and dx in two bf16 terms each, half a step of the second being 2^-16 of
the value; all else is FP32, K of test_gpu_mamba2_scan.  So an element of y or dx is off by (K + 2^-16) of its terms' sizes
before it is rounded, as a bound.  As a rule it is off by a few times 2^-17 of itself, and is the rounding of the exact value
unless that lies so close to the middle between two bf16 numbers, 2^-7 to 2^-8 apart: in about one of 100 elements.  A single
bf16 term would be off by 2^-9 and more, in every other element.
"""
import numpy as np
import pytest
import torch

import oracle as O
import test_gpu_mamba2_scan as base
from gpu_util import DEV, require_gpu, say, torch_dtype

pytestmark = pytest.mark.gpu
LOW = 1.02 * 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def as_rounded(got, ref, what):
    want = torch.from_numpy(ref).to(got.dtype)
    same = (got.cpu() == want).double().mean().item()
    say(f"{what}: {100 * same:.2f}% of the elements are the exact value's rounding")
    assert same >= 0.95, what


def check(lens, H, G, d, n, dt, sdt="f32", resets=0, seed=1, only=None):
    import gated_deltanet_state_gdn_amd as gdn
    say(f"scan readout lens={lens} H={H} G={G} d={d} n={n} {dt} state={sdt} resets={resets}")
    v, r = base.make(lens, H, G, d, n, dt, sdt, seed)
    for k in ("Bm", "Cm"):
        v[k] = (v[k].float() * n ** 0.5).to(v[k].dtype)
    v["D"].zero_()
    if resets:  # every so many tokens a step of 2^14 and nothing to write clears the state
        v["dt"][resets // 2::resets] = 16384.0
        v["x"][resets // 2::resets] = 0.0
    r.update((k, v[k].double().cpu().numpy()) for k in base.NAMES)
    pool = v["pool"].clone()
    y = gdn.gdn_mamba2_scan(*(v[k] for k in base.NAMES), v["cu"], pool=pool, slot_map=v["slots"])
    g = gdn.gdn_mamba2_scan_backward(v["dy"], *(v[k] for k in base.NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"], dfinal=v["dfinal"])
    torch.cuda.synchronize()
    ins, form = [r[k] for k in base.NAMES], dict(cu=r["cu"], init=r["pool"], slot_map=r["slots"])
    (y_r, f_r), (y_s, f_s) = O.mamba2_scan(*ins, **form), O.mamba2_scan(*ins, **form, sizes=True)
    low = LOW if dt == "bf16" else 0.0
    base.close(y, y_r, (base.K + low) * y_s, dt, "y")
    used = [s for s, k in enumerate(lens) if k > 0]
    base.close(pool[torch.as_tensor(r["slots"][used]).long().to(DEV)], f_r[used], base.K * f_s[used], sdt, "final states")
    form["dfinal"] = r["dfinal"]
    ref, size = O.mamba2_scan_backward(r["dy"], *ins, **form), O.mamba2_scan_backward(r["dy"], *ins, **form, sizes=True)
    slack = dict(dx=base.K + low, dBm=base.K + low, dCm=base.K + low)
    for name, p, q, s in zip(g._fields, g, ref, size):
        if only is not None and name not in only:
            continue
        base.close(p, q, slack.get(name, base.K) * s, dt if name in ("dx", "dBm", "dCm", "ddt") else "f32", name)
    if dt == "bf16":
        as_rounded(y, y_r, "y")
        as_rounded(g.dx, ref[0], "dx")


@pytest.mark.parametrize("n", [16, 64, 128])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_every_size(d, n):
    check([70, 0, 129, 1, 64], 6, 2, d, n, "bf16")


def test_two_heads_a_workgroup():
    """d = 64 with walks enough for two heads a workgroup, the last one half empty."""
    check([40 + i % 60 for i in range(90)], 11, 1, 64, 64, "bf16")


def test_segments():
    check([900, 40, 0, 1300], 2, 1, 64, 128, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d,n", [(16, 64), (64, 128)])
def test_decays_that_clear_the_state(d, n, dt):
    """Steps of 2^14: the log-decays summed in a chunk pass 2^17, and differences behind them still have to hold."""
    check([200, 33], 4, 2, d, n, dt, resets=23)
