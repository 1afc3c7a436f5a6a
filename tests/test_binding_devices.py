"""Tensors that do not lie on the launch's GPU are refused on the host by the norm's and the scan's calls."""
import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn

T, H, G, d, n, N = 6, 4, 2, 16, 16, 2


def scan_args(device):
    z = lambda *s, **k: torch.zeros(*s, device=device, **k)  # noqa: E731
    ins = dict(x=z(T, H, d), Bm=z(T, G, n), Cm=z(T, G, n), dt=z(T, H), A_log=z(H), dt_bias=z(H), D=z(H),
               cu_seqlens=torch.tensor([0, 2, T], dtype=torch.int32, device=device))
    return ins, dict(pool=z(3, H, d, n), slot_map=torch.tensor([2, 0], dtype=torch.int32, device=device))


def norm_args(device):
    z = lambda *s: torch.ones(*s, device=device)  # noqa: E731
    return dict(x=z(4, 8), weight=z(8), bias=z(8), gate=z(4, 8))


def test_host_tensors_are_refused():
    ins, states = scan_args("cpu")
    for call in (lambda: gdn.gdn_mamba2_scan(**ins), lambda: gdn.gdn_mamba2_scan(**ins, **states),
                 lambda: gdn.gdn_mamba2_scan_backward(dy=ins["x"], **ins), lambda: gdn.gdn_layer_norm(**norm_args("cpu")),
                 lambda: gdn.gdn_layer_norm_backward(dy=torch.ones(4, 8), mean=torch.zeros(4, 1), rstd=torch.ones(4, 1), **norm_args("cpu"))):
        with pytest.raises(ValueError, match="must lie on a GPU"):
            call()


@pytest.mark.gpu
def test_one_host_tensor_is_refused():
    ins, states = scan_args("cuda")
    gdn.gdn_mamba2_scan(**ins, **states)
    for k in (*ins, *states):
        if k == "x":
            continue
        a, b = dict(ins), dict(states)
        (a if k in a else b)[k] = (a if k in a else b)[k].cpu()
        for call in (lambda: gdn.gdn_mamba2_scan(**a, **b), lambda: gdn.gdn_mamba2_scan_backward(dy=ins["x"], **a, **b)):
            with pytest.raises(ValueError, match="must lie on cuda"):
                call()
    for kw in (dict(out=torch.zeros(T, H, d)), dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="must lie on cuda"):
            gdn.gdn_mamba2_scan(**ins, **kw)
    for kw in (dict(dy=torch.zeros(T, H, d)), dict(dy=ins["x"], dfinal=torch.zeros(N, H, d, n))):
        with pytest.raises(ValueError, match="must lie on cuda"):
            gdn.gdn_mamba2_scan_backward(**ins, **kw)
    good = norm_args("cuda")
    y, mean, rstd = gdn.gdn_layer_norm(**good, save_stats=True)
    back = dict(good, dy=y, mean=mean, rstd=rstd)
    gdn.gdn_layer_norm_backward(**back)
    for k in ("weight", "bias", "gate"):
        with pytest.raises(ValueError, match="must lie on cuda"):
            gdn.gdn_layer_norm(**dict(good, **{k: good[k].cpu()}))
    for k in ("weight", "bias", "gate", "dy", "mean", "rstd"):
        with pytest.raises(ValueError, match="must lie on cuda"):
            gdn.gdn_layer_norm_backward(**dict(back, **{k: back[k].cpu()}))
    with pytest.raises(ValueError, match="must lie on cuda"):
        gdn.gdn_layer_norm(**good, out=torch.zeros(4, 8))
    torch.cuda.synchronize()
