"""The scan with d = 64 where there are walks enough (512 sequences x pairs of heads) for two heads a workgroup, against the float64
oracle with the tolerances of test_gpu_mamba2_scan."""
import pytest
import torch

import oracle as O
import test_gpu_mamba2_scan as base
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# 90 sequences: mostly short, some empty, a few past one and two chunks
SHORT = [i * 7 % 12 for i in range(86)] + [65, 64, 130, 1]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [16, 64, 128])
@pytest.mark.parametrize("H,G", [(12, 1), (22, 2)])
def test_two_heads_a_workgroup(H, G, n, dt):
    """Six workgroups a sequence; with 11 heads a group the last workgroup of a group has one head."""
    base.check_scan(SHORT, H, G, 64, n, dt, "f32")
    base.check_backward(SHORT, H, G, 64, n, dt, "f32", dfinal=True)


def test_f16_and_no_states():
    base.check_scan(SHORT, 11, 1, 64, 64, "f16", "f16")
    base.check_scan(SHORT, 11, 1, 64, 128, "bf16")
    base.check_backward(SHORT, 11, 1, 64, 128, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_padded_sequences(dt):
    """Every third sequence is padded: zero outputs, gradients and dinit; the others as the oracle has them."""
    import gated_deltanet_state_gdn_amd as gdn
    v, r = base.make(SHORT, 11, 1, 64, 64, dt, "f32")
    v["slots"][::3] = -1
    r["slots"] = v["slots"].cpu().numpy()
    before = v["pool"].clone()
    y = gdn.gdn_mamba2_scan(*(v[k] for k in base.NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"])
    g = gdn.gdn_mamba2_scan_backward(v["dy"], *(v[k] for k in base.NAMES), v["cu"], pool=before, slot_map=v["slots"], dfinal=v["dfinal"])
    torch.cuda.synchronize()
    ins, form = [r[k] for k in base.NAMES], dict(cu=r["cu"], init=r["pool"], slot_map=r["slots"])
    (y_r, f_r), (y_s, f_s) = O.mamba2_scan(*ins, **form), O.mamba2_scan(*ins, **form, sizes=True)
    low = base.HALF["bf16"] * 1.02 if dt == "bf16" else 0.0
    base.close(y, y_r, (base.K + low) * y_s, dt, "y")
    used = [s for s, k in enumerate(SHORT) if k > 0 and s % 3]
    base.close(v["pool"][torch.as_tensor(r["slots"][used]).long().to(DEV)], f_r[used], base.K * f_s[used], "f32", "final states")
    ref = O.mamba2_scan_backward(r["dy"], *ins, **form, dfinal=r["dfinal"])
    size = O.mamba2_scan_backward(r["dy"], *ins, **form, dfinal=r["dfinal"], sizes=True)
    slack = dict(dx=base.K + low, dBm=base.K + low * 2.0 ** -8, dCm=base.K + low * 2.0 ** -8)
    for name, p, q, s in zip(g._fields, g, ref, size):
        base.close(p, q, slack.get(name, base.K) * s, dt if name in ("dx", "dBm", "dCm", "ddt") else "f32", name)
    assert not g.dinit[::3].any()


def test_long_sequences_among_short_ones():
    lens = [700, 0, 600] + [170 + i for i in range(17)]
    base.check_scan(lens, 63, 1, 64, 16, "bf16", "f32")
    base.check_backward(lens, 63, 1, 64, 16, "bf16", "f32", dfinal=True)
