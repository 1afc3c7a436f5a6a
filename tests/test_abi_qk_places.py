"""Refusals of the tensors given for the norm and rotation's gradients, on the host."""
import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn

z = torch.zeros
T, d = 6, 32


@pytest.mark.parametrize("bad", [dict(dq=z(T, 3, 40)), dict(dk=z(T + 1, 1, d)), dict(dk=z(T, 1, d).half()), dict(dq=z(1, 3, d).expand(T, 3, d)),
                                 dict(dq=z(T, d, 3).transpose(1, 2))])
def test_refusals(bad):
    args = dict(q=z(T, 3, d), k=z(T, 1, d), q_weight=z(d), k_weight=z(d), positions=z(T, dtype=torch.int32), inv_freq=z(8),
                dq_out=z(T, 3, d), dk_out=z(T, 1, d))
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope_backward(**args | bad)
    with pytest.raises(ValueError, match="must lie on a GPU"):
        gdn.gdn_qk_norm_rope_backward(**args | dict(dq=z(T, 3, d), dk=z(T, 1, d)))
