"""The one-token call of linear attention on the host: what it says where a gradient is asked for."""
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
