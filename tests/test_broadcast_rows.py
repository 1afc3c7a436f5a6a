"""Tensors whose rows are one row expanded (stride 0, which the library's C interface reads as dense): inputs are copied, outputs
refused.  The norm's and the scan's calls."""
import ctypes

import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
from gated_deltanet_state_gdn_amd import _binding as bd


def test_expanded_inputs_are_copied():
    def read(row):  # 100 rows as the library would read them
        ptr, stride = row
        return torch.frombuffer((ctypes.c_float * 800).from_address(ptr), dtype=torch.float32).view(100, 8) if stride == 0 else None
    copies = []
    row, tok = torch.randn(1, 8).expand(100, 8), torch.randn(1, 2, 4).expand(100, 2, 4)
    assert torch.equal(read(bd._rows(row, row.shape, row.dtype, "x", copies)), row)
    assert torch.equal(read(bd._token_rows(tok, (2, 4), tok.dtype, "x", copies)), tok.reshape(100, 8))
    ones = torch.ones(()).expand(100, 8)  # the gradient of a sum over everything
    assert torch.equal(read(bd._rows(ones, ones.shape, ones.dtype, "dy", copies)), ones)
    assert len(copies) == 3
    for t in (torch.randn(100, 8), torch.randn(100, 12)[:, 2:10]):
        assert bd._rows(t, t.shape, t.dtype, "x", copies)[0] == t.data_ptr()
    assert len(copies) == 3


def test_no_stride_of_zero_reaches_the_library():
    row, tok = torch.ones(1, 64), torch.ones(1, 4, 16)
    with pytest.raises(ValueError, match="share"):
        bd._rows(row.expand(100, 64), (100, 64), row.dtype, "out")
    with pytest.raises(ValueError, match="share"):
        bd._token_rows(tok.expand(100, 4, 16), (4, 16), tok.dtype, "x")
    assert bd._rows(torch.ones(3, 70)[:, :64], (3, 64), row.dtype, "x")[1] == 70
    assert bd._rows(torch.ones(3, 70)[1:2, :64], (1, 64), row.dtype, "x")[1] == 0


def test_expanded_output_is_refused():
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError, match="share"):
        gdn.gdn_layer_norm(x, w, out=torch.zeros(1, 8).expand(4, 8))


def _same(got, want):
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert (g is None and w is None) or torch.equal(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("own_stream", [False, True])
def test_norm(own_stream):
    stream = torch.cuda.Stream() if own_stream else None
    w = torch.randn(200, device="cuda")
    x, z, dy = (torch.randn(1, 200, device="cuda").bfloat16() for _ in range(3))
    full = lambda t: t.repeat(300, 1)  # noqa: E731
    wide = lambda t: t.expand(300, 200)  # noqa: E731
    some = torch.randn(300, 200, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for a, g, d in ((x, z, dy), (some, z, dy), (some, z, some), (x, some, some)):
        each = [(full(t), wide(t)) if t.shape[0] == 1 else (t, t) for t in (a, g, d)]
        torch.cuda.synchronize()
        want, got = ([*gdn.gdn_layer_norm(v[0][k], w, gate=v[1][k], rms=True, save_stats=True, stream=stream)] for k, v in ((0, each), (1, each)))
        _same(got, want)
        want, got = ([*gdn.gdn_layer_norm_backward(v[2][k], v[0][k], w, *want[1:], gate=v[1][k], rms=True, stream=stream)] for k, v in ((0, each), (1, each)))
        _same(got, want)


@pytest.mark.gpu
def test_gradient_behind_a_sum():
    """What autograd hands on behind a sum over rows has strides (0, 1)."""
    x, w = torch.randn(50, 64, device="cuda"), torch.randn(64, device="cuda")
    y, mean, rstd = gdn.gdn_layer_norm(x, w, save_stats=True)
    seen = []
    y.requires_grad_().register_hook(seen.append)
    y.sum(0).square().sum().backward()
    assert seen[0].stride() == (0, 1)
    _same(gdn.gdn_layer_norm_backward(seen[0], x, w, mean, rstd), gdn.gdn_layer_norm_backward(seen[0].contiguous(), x, w, mean, rstd))


@pytest.mark.gpu
@pytest.mark.parametrize("own_stream", [False, True])
def test_scan(own_stream):
    stream = torch.cuda.Stream() if own_stream else None
    T, H, G, d, n = 150, 4, 2, 64, 128
    r = lambda *s: (torch.randn(*s, device="cuda") * 0.3).bfloat16()  # noqa: E731
    P = [torch.randn(H, device="cuda") for _ in range(3)]
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    one = [r(1, H, d), r(1, G, n), r(1, G, n), r(1, H), r(1, H, d)]
    wide, full = [t.expand(T, *t.shape[1:]) for t in one], [t.repeat(T, *[1] * (t.dim() - 1)) for t in one]
    torch.cuda.synchronize()
    _same([gdn.gdn_mamba2_scan(*wide[:4], *P, cu, stream=stream)], [gdn.gdn_mamba2_scan(*full[:4], *P, cu, stream=stream)])
    _same(gdn.gdn_mamba2_scan_backward(wide[4], *wide[:4], *P, cu, stream=stream),
          gdn.gdn_mamba2_scan_backward(full[4], *full[:4], *P, cu, stream=stream))
