"""The norm's and the scan's calls have no graph, and say so where an input requires grad.  (The tensors lie on the host, so every
call ends in a refusal behind the warning.)"""
import warnings

import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
from test_binding_devices import norm_args, scan_args


def calls(which):
    ins, states = scan_args("cpu")
    norm = norm_args("cpu")
    for k in which:
        for args in (ins, states, norm):
            if k in args:
                args[k].requires_grad_()
    return (lambda: gdn.gdn_mamba2_scan(**ins, **states)), (lambda: gdn.gdn_layer_norm(**norm))


@pytest.mark.parametrize("k", ["x", "Bm", "Cm", "dt", "A_log", "dt_bias", "D", "pool"])
def test_scan_warns(k):
    with pytest.warns(UserWarning, match="gdn_mamba2_scan_backward"), pytest.raises(ValueError):
        calls([k])[0]()


@pytest.mark.parametrize("k", ["x", "weight", "bias", "gate"])
def test_norm_warns(k):
    with pytest.warns(UserWarning, match="gdn_layer_norm_backward"), pytest.raises(ValueError):
        calls([k])[1]()


def test_silent_without_gradients():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for call in calls([]):
            with pytest.raises(ValueError):
                call()
        with torch.no_grad():
            for call in calls(["x", "weight", "D"]):
                with pytest.raises(ValueError):
                    call()
