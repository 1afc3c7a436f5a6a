"""Where the norm and rotation's gradients go: into given tensors, in place of what they come from, and into slices of wider rows."""
import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
import test_gpu_qk as base
from gpu_util import DEV, require_gpu, say

pytestmark = pytest.mark.gpu
T, Hq, Hk, d = 1100, 3, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def joint(a, b):
    """Two tensors as slices of one tensor of rows, with room behind them."""
    rows = torch.cat([a.reshape(T, -1), b.reshape(T, -1), torch.full((T, 16), 5.0, dtype=a.dtype, device=DEV)], 1)
    return rows, rows[:, :Hq * d].unflatten(1, (Hq, d)), rows[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
def test_gradients_in_given_tensors(dt, neighbours):
    say(f"qk gradients in given tensors {dt} neighbours={neighbours}")
    v = base.make(T, Hq, Hk, d, 48, dt)
    params = (v["qw"], v["kw"], v["pos"], v["freq"])
    want = gdn.gdn_qk_norm_rope_backward(v["dq"], v["dk"], v["q"], v["k"], *params, neighbours=neighbours)

    def check(got, rows=None):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert rows is None or (rows[:, -16:] == 5).all()

    def call(dy, x, **outs):
        return gdn.gdn_qk_norm_rope_backward(*dy, *x, *params, neighbours=neighbours, **outs)

    dy, x = (v["dq"], v["dk"]), (v["q"], v["k"])
    rows, a, b = joint(torch.zeros_like(v["q"]), torch.zeros_like(v["k"]))
    got = call(dy, x, dq=a, dk=b)
    assert got.dq is a and got.dk is b
    check(got, rows)
    own = [t.clone() for t in dy]
    check(call(own, x, dq=own[0], dk=own[1]))
    own = [t.clone() for t in x]
    check(call(dy, own, dq=own[0], dk=own[1]))
    rows, a, b = joint(*dy)
    check(call((a, b), x, dq=a, dk=b), rows)
    rows, a, b = joint(*x)
    check(call(dy, (a, b), dq=a, dk=b), rows)
