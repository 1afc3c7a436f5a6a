"""Calls whose tensors lie on a GPU that is not the current one: that GPU is current while the library launches, and its own current stream
is the one taken.  On the host, with the library and the devices stood in for."""
import contextlib

import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
from gated_deltanet_state_gdn_amd import _binding as bd

z = torch.zeros
T, H, d = 6, 2, 16


def calls():
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    tok, seqs, head = z(T, H, d), ints(0, 2, T), z(H)
    states, slots, one = z(9, H, d, d), ints(2, 0), z(2, H, d)
    m2 = dict(x=tok, Bm=tok, Cm=tok, dt=z(T, H), A_log=head, dt_bias=head, D=head, cu_seqlens=seqs)
    x, w = z(4, 8), z(8)
    qk = dict(q=tok, k=tok, q_weight=z(d), k_weight=z(d), positions=z(T, dtype=torch.int32), inv_freq=z(8))
    return {
        "gdn_mamba2_scan": lambda: gdn.gdn_mamba2_scan(**m2),
        "gdn_mamba2_scan_backward": lambda: gdn.gdn_mamba2_scan_backward(tok, **m2),
        "gdn_layer_norm": lambda: gdn.gdn_layer_norm(x, w),
        "gdn_layer_norm_backward": lambda: gdn.gdn_layer_norm_backward(x, x, w, z(4, 1), z(4, 1)),
        "gdn_linear_decode_step": lambda: gdn.gdn_linear_decode_step(one, one, one, head, states, slots),
        "gdn_linear_scan": lambda: gdn.gdn_linear_scan(tok, tok, tok, head, seqs),
        "gdn_linear_scan_backward": lambda: gdn.gdn_linear_scan_backward(tok, tok, tok, tok, head, seqs),
        "gdn_qk_norm_rope": lambda: gdn.gdn_qk_norm_rope(**qk),
        "gdn_qk_norm_rope_backward": lambda: gdn.gdn_qk_norm_rope_backward(tok, tok, **qk),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_launch_on_the_tensors_gpu(monkeypatch, name):
    call, now, launches = calls()[name], [0], []

    @contextlib.contextmanager
    def device(gpu):
        before, now[0] = now[0], gpu
        yield
        now[0] = before

    class Library:
        def __getattr__(self, f):
            if f.endswith("workspace_bytes"):
                return lambda *a: 0
            return lambda *a: launches.append((f, now[0], a[-1])) or 0

    monkeypatch.setattr(bd, "lib", lambda: Library())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda gpu: 100 + gpu, raising=False)
    for f in (bd._scan_workspace, bd._linear_workspace):
        f.cache_clear()
    call()
    for f in (bd._scan_workspace, bd._linear_workspace):
        f.cache_clear()
    assert launches == [(name, 1, 101)] and now == [0]
