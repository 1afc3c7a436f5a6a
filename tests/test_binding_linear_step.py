"""The calls of linear attention on the host: what the one-token form says where a gradient is asked for, and scales beyond FP32."""
import warnings

import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn

z = torch.zeros


def args():
    return dict(q=z(2, 2, 16), k=z(2, 1, 16), v=z(2, 4, 16), log_decay=z(4), pool=z(3, 4, 16, 16), slot_map=z(2, dtype=torch.int32))


@pytest.mark.parametrize("name", ["q", "k", "v", "log_decay", "pool"])
def test_no_graph(name):
    a = args()
    a[name].requires_grad_()
    with pytest.warns(UserWarning, match="gdn_linear_scan_backward"), pytest.raises(ValueError, match="must lie on a GPU"):
        gdn.gdn_linear_decode_step(**a)
    with warnings.catch_warnings(), torch.no_grad():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="must lie on a GPU"):
            gdn.gdn_linear_decode_step(**a)


@pytest.mark.parametrize("scale", [1e-50, 1e39, 0.0, -0.5, float("nan")])
def test_scales_that_float32_does_not_hold(scale):
    """The library takes 0 for the default, so a scale that rounds to it would be another one."""
    a = args()
    scan = {k: v for k, v in a.items() if k not in ("pool", "slot_map")} | dict(cu_seqlens=torch.tensor([0, 2], dtype=torch.int32))
    for call in (lambda: gdn.gdn_linear_decode_step(**a, scale=scale), lambda: gdn.gdn_linear_scan(**scan, scale=scale),
                 lambda: gdn.gdn_linear_scan_backward(z(2, 4, 16), **scan, scale=scale)):
        with pytest.raises(ValueError, match="scale must be positive"):
            call()
    with pytest.raises(ValueError, match="must lie on a GPU"):
        gdn.gdn_linear_decode_step(**a, scale=1e-40)
