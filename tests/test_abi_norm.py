"""Refusals of the norm's entry points, on the host (no kernel is launched: every call fails its checks or has no rows to do)."""
import ctypes
import os

import pytest

import gated_deltanet_state_gdn_amd as gdn
from gated_deltanet_state_gdn_amd import _binding as bd

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bd.LIB_PATH):
        from gated_deltanet_state_gdn_amd import build
        build.build()
    return gdn.lib()


def _fwd(L, rows=4, width=64, groups=1, gate=0, x=FAKE, xs=0, z=None, zs=0, dt=gdn.GDN_BF16, w=FAKE, b=None, eps=1e-5, y=FAKE,
         ys=0, out_dt=gdn.GDN_BF16, mean=None, rstd=None, dims=True):
    q = bd.gdn_norm_dims(rows, width, groups, 0, gate)
    return L.gdn_layer_norm(ctypes.byref(q) if dims else None, x, xs, z, zs, dt, w, b, eps, y, ys, out_dt, mean, rstd, None)


BAD_DIMS = [
    (dict(rows=-1), gdn.GDN_EINVAL),
    (dict(width=0), gdn.GDN_EINVAL),
    (dict(groups=0), gdn.GDN_EINVAL),
    (dict(groups=3), gdn.GDN_EINVAL),                       # does not divide the width
    (dict(gate=3), gdn.GDN_EINVAL),
    (dict(width=16385), gdn.GDN_EUNSUPPORTED),
    (dict(width=65536, groups=65536), gdn.GDN_EUNSUPPORTED),
    (dict(dt=5), gdn.GDN_EINVAL),
    (dict(x=None), gdn.GDN_EINVAL),
    (dict(x=FAKE + 1), gdn.GDN_EINVAL),
    (dict(xs=63), gdn.GDN_EINVAL),                          # rows would overlap
    (dict(xs=-64), gdn.GDN_EINVAL),
    (dict(z=FAKE), gdn.GDN_EINVAL),                         # a gate tensor and no gate
    (dict(gate=1), gdn.GDN_EINVAL),                         # a gate and no tensor
    (dict(gate=2, z=FAKE, zs=1), gdn.GDN_EINVAL),
    (dict(w=None), gdn.GDN_EINVAL),
    (dict(b=FAKE + 2), gdn.GDN_EINVAL),
]


@pytest.mark.parametrize("case,expect", BAD_DIMS + [
    (dict(dims=False), gdn.GDN_EINVAL),
    (dict(eps=-1.0), gdn.GDN_EINVAL),
    (dict(eps=float("nan")), gdn.GDN_EINVAL),
    (dict(out_dt=-1), gdn.GDN_EINVAL),
    (dict(y=None), gdn.GDN_EINVAL),
    (dict(y=FAKE + 2, out_dt=gdn.GDN_F32), gdn.GDN_EINVAL),
    (dict(ys=10), gdn.GDN_EINVAL),
    (dict(mean=FAKE), gdn.GDN_EINVAL),                      # one statistic without the other
    (dict(rows=0, x=None, y=None, w=None), gdn.GDN_OK),     # no rows: nothing is read or written
])
def test_forward_refusals(L, case, expect):
    st = _fwd(L, **case)
    assert st == expect, gdn.gdn_last_error()
    assert (gdn.gdn_last_error() == "") == (expect == gdn.GDN_OK)


def _bwd(L, rows=4, width=64, groups=1, gate=0, dy=FAKE, x=FAKE, xs=0, z=None, zs=0, dt=gdn.GDN_BF16, w=FAKE, b=None, mean=FAKE,
         rstd=FAKE, dx=FAKE, dxs=0, dz=None, dw=FAKE, db=None, ws=FAKE, wsb=1 << 30):
    q = bd.gdn_norm_dims(rows, width, groups, 0, gate)
    return L.gdn_layer_norm_backward(ctypes.byref(q), dy, 0, x, xs, z, zs, dt, w, b, mean, rstd, dx, dxs, dz, 0, dw, db, ws, wsb, None)


@pytest.mark.parametrize("case,expect", BAD_DIMS + [
    (dict(dy=None), gdn.GDN_EINVAL),
    (dict(dx=None), gdn.GDN_EINVAL),
    (dict(dxs=5), gdn.GDN_EINVAL),
    (dict(dz=FAKE), gdn.GDN_EINVAL),
    (dict(gate=1, z=FAKE), gdn.GDN_EINVAL),                 # the gate's gradient has no place
    (dict(mean=None), gdn.GDN_EINVAL),
    (dict(rstd=FAKE + 1), gdn.GDN_EINVAL),
    (dict(dw=None), gdn.GDN_EINVAL),
    (dict(ws=None), gdn.GDN_EINVAL),
    (dict(ws=FAKE + 16), gdn.GDN_EINVAL),
    (dict(wsb=4), gdn.GDN_EINVAL),
])
def test_backward_refusals(L, case, expect):
    st = _bwd(L, **case)
    assert st == expect, gdn.gdn_last_error()
    assert gdn.gdn_last_error() != ""


def test_workspace_size(L):
    size = lambda *a: L.gdn_layer_norm_backward_workspace_bytes(ctypes.byref(bd.gdn_norm_dims(*a)))  # noqa: E731
    assert size(0, 64, 1, 0, 0) == 0
    assert size(4, 63, 2, 0, 0) == 0                        # refused sizes need nothing
    assert size(1, 4096, 1, 0, 0) == 2 * 4096 * 4           # one workgroup's row of dw and db
    assert size(1 << 40, 4096, 1, 0, 0) == size(1 << 20, 4096, 1, 0, 0)


def test_binding_refuses_shapes_and_layouts():
    import torch
    x, w = torch.zeros(4, 6), torch.ones(6)
    for call in (lambda: gdn.gdn_layer_norm(x[0], w), lambda: gdn.gdn_layer_norm(x, w[:5]), lambda: gdn.gdn_layer_norm(x, w.double()),
                 lambda: gdn.gdn_layer_norm(x.t(), torch.ones(4)), lambda: gdn.gdn_layer_norm(x, w, gate=x[:3]),
                 lambda: gdn.gdn_layer_norm(x, w, gate=x.bfloat16()), lambda: gdn.gdn_layer_norm(x, w, out=x[:, :5]),
                 lambda: gdn.gdn_layer_norm_backward(x.bfloat16(), x, w, x[:, :1], x[:, :1])):
        with pytest.raises((ValueError, gdn.GdnError)):
            call()


@pytest.mark.parametrize("width,groups,fits", [(16 * 3 * 23 * 89 * 683, 16 * 3 * 89, True), (1 << 26, 4096, False), (65535 * 16384, 65535, False)])
def test_backward_width_past_a_launch(L, width, groups, fits):
    """The kernel that adds dw and db has 64 threads a column: widths at which they pass 2^32 are refused before any launch."""
    dims = bd.gdn_norm_dims(2, width, groups, 0, 0)
    assert (L.gdn_layer_norm_backward_workspace_bytes(ctypes.byref(dims)) > 0) == fits
    assert _bwd(L, rows=2, width=width, groups=groups, ws=None, wsb=0) == (gdn.GDN_EINVAL if fits else gdn.GDN_EUNSUPPORTED)
    assert _fwd(L, rows=2, width=width, groups=groups, y=None) == gdn.GDN_EINVAL  # the forward pass takes any width
