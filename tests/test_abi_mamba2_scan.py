"""Refusals of the sequence scan's entry points, on the host (no kernel is launched in any case here)."""
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


DIMS = dict(H=8, G=2, d=64, n=128)


def _common(N, T, dims, cu, x, Bm, Cm, dt, st, p, pool, sm):
    q = bd.gdn_m2_dims(*(dict(DIMS, **dims)[k] for k in ("H", "G", "d", "n"))) if dims is not None else None
    return [ctypes.byref(q) if q else None, N, cu, T, x, Bm, Cm, dt, ctypes.byref(st) if st else None, ctypes.byref(p) if p else None,
            ctypes.byref(pool) if pool else None, sm]


P = bd.gdn_m2_params(FAKE, FAKE, FAKE, FAKE)
POOL = bd.gdn_pool(FAKE, gdn.GDN_F32, 4)


def _fwd(L, N=2, T=100, dims={}, cu=FAKE, x=FAKE, Bm=FAKE, Cm=FAKE, dt=gdn.GDN_BF16, st=None, p=P, pool=POOL, sm=FAKE, y=FAKE,
         out_dt=gdn.GDN_BF16, ws=FAKE, wsb=1 << 40):
    return L.gdn_mamba2_scan(*_common(N, T, dims, cu, x, Bm, Cm, dt, st, p, pool, sm), y, out_dt, ws, wsb, None)


BAD = [
    (dict(dims=None), gdn.GDN_EINVAL),
    (dict(dims=dict(G=3)), gdn.GDN_EINVAL),
    (dict(dims=dict(d=32)), gdn.GDN_EUNSUPPORTED),
    (dict(dims=dict(n=256)), gdn.GDN_EUNSUPPORTED),
    (dict(dims=dict(H=65536, G=1)), gdn.GDN_EUNSUPPORTED),
    (dict(N=-1), gdn.GDN_EINVAL),
    (dict(T=-1), gdn.GDN_EINVAL),
    (dict(T=1 << 31), gdn.GDN_EINVAL),
    (dict(N=0), gdn.GDN_EINVAL),                                  # tokens and no sequence
    (dict(N=1, T=2147483647, dims=dict(H=128, G=1)), gdn.GDN_EUNSUPPORTED),  # past the grid
    (dict(dt=9), gdn.GDN_EINVAL),
    (dict(cu=None), gdn.GDN_EINVAL),
    (dict(x=None), gdn.GDN_EINVAL),
    (dict(x=FAKE + 8), gdn.GDN_EINVAL),
    (dict(Bm=FAKE + 2), gdn.GDN_EINVAL),
    (dict(Cm=None), gdn.GDN_EINVAL),
    (dict(p=None), gdn.GDN_EINVAL),
    (dict(p=bd.gdn_m2_params(FAKE, None, FAKE, FAKE)), gdn.GDN_EINVAL),
    (dict(p=bd.gdn_m2_params(None, FAKE, FAKE, FAKE)), gdn.GDN_EINVAL),
    (dict(st=bd.gdn_m2_strides(8 * 64 - 8, 0, 0, 0)), gdn.GDN_EINVAL),
    (dict(st=bd.gdn_m2_strides(8 * 64 + 4, 0, 0, 0)), gdn.GDN_EINVAL),
    (dict(st=bd.gdn_m2_strides(0, 0, 2 * 128 - 8, 0)), gdn.GDN_EINVAL),
    (dict(st=bd.gdn_m2_strides(0, 0, 0, 7)), gdn.GDN_EINVAL),
    (dict(st=bd.gdn_m2_strides((1 << 22) + 8, 0, 0, 0)), gdn.GDN_EUNSUPPORTED),   # past 32-bit offsets in a block
    (dict(dims=dict(H=40000, G=1, d=128)), gdn.GDN_EUNSUPPORTED),
    (dict(st=bd.gdn_m2_strides(0, -256, 0, 0)), gdn.GDN_EINVAL),
    (dict(pool=None), gdn.GDN_EINVAL),                            # slots and no pool
    (dict(sm=None), gdn.GDN_EINVAL),
    (dict(pool=bd.gdn_pool(FAKE + 8, gdn.GDN_F32, 4)), gdn.GDN_EINVAL),
    (dict(ws=None), gdn.GDN_EINVAL),
    (dict(ws=FAKE + 128), gdn.GDN_EINVAL),
    (dict(wsb=1000), gdn.GDN_EINVAL),
]


@pytest.mark.parametrize("case,expect", BAD + [
    (dict(out_dt=3), gdn.GDN_EINVAL),
    (dict(y=None), gdn.GDN_EINVAL),
    (dict(y=FAKE + 2, out_dt=gdn.GDN_F32), gdn.GDN_EINVAL),
    (dict(T=0, ws=None, wsb=0, y=None), gdn.GDN_OK),
    (dict(N=0, T=0, cu=None), gdn.GDN_OK),
])
def test_forward_refusals(L, case, expect):
    st = _fwd(L, **case)
    assert st == expect, gdn.gdn_last_error()
    assert (gdn.gdn_last_error() == "") == (expect == gdn.GDN_OK)


def _bwd(L, N=2, T=100, dims={}, cu=FAKE, x=FAKE, Bm=FAKE, Cm=FAKE, dt=gdn.GDN_BF16, st=None, p=P, pool=POOL, sm=FAKE, dy=FAKE,
         dfinal=None, dx=FAKE, dB=FAKE, dC=FAKE, ddt=FAKE, dA=FAKE, db=FAKE, dD=FAKE, dinit=None, ws=FAKE, wsb=1 << 40):
    return L.gdn_mamba2_scan_backward(*_common(N, T, dims, cu, x, Bm, Cm, dt, st, p, pool, sm), dy, dfinal, dx, dB, dC, ddt, dA, db, dD,
                                      dinit, ws, wsb, None)


@pytest.mark.parametrize("case,expect", BAD + [
    (dict(dy=None), gdn.GDN_EINVAL),
    (dict(dy=FAKE + 8), gdn.GDN_EINVAL),
    (dict(dfinal=FAKE + 4), gdn.GDN_EINVAL),
    (dict(dinit=FAKE + 8), gdn.GDN_EINVAL),
    (dict(dx=None), gdn.GDN_EINVAL),
    (dict(dB=FAKE + 1), gdn.GDN_EINVAL),
    (dict(ddt=None), gdn.GDN_EINVAL),
    (dict(dA=None), gdn.GDN_EINVAL),
    (dict(dD=FAKE + 2), gdn.GDN_EINVAL),
])
def test_backward_refusals(L, case, expect):
    st = _bwd(L, **case)
    assert st == expect, gdn.gdn_last_error()
    assert gdn.gdn_last_error() != ""


def test_workspace_sizes(L):
    f = lambda N, T, **d: L.gdn_mamba2_scan_workspace_bytes(ctypes.byref(bd.gdn_m2_dims(*dict(DIMS, **d).values())), N, T)  # noqa: E731
    b = lambda N, T, **d: L.gdn_mamba2_scan_backward_workspace_bytes(ctypes.byref(bd.gdn_m2_dims(*dict(DIMS, **d).values())), N, T)  # noqa: E731
    assert f(0, 0) == b(0, 0) == 0
    assert f(2, 100, d=32) == 0
    assert 0 < f(2, 100) < b(2, 100)
    # two FP32 states a head and block of 128 tokens
    assert b(1, 1 << 16, H=64, G=8) - b(1, 1 << 15, H=64, G=8) > 2 * 256 * 64 * 64 * 128 * 4


def test_binding_refuses_shapes_and_types():
    import torch
    T, H, G, d, n, N = 6, 4, 2, 16, 16, 2
    z = torch.zeros
    good = dict(x=z(T, H, d), Bm=z(T, G, n), Cm=z(T, G, n), dt=z(T, H), A_log=z(H), dt_bias=z(H), D=z(H), cu_seqlens=z(N + 1, dtype=torch.int32))
    pool, slots = z(3, H, d, n), z(N, dtype=torch.int32)
    for bad in (dict(x=z(T, H * d)), dict(Cm=z(T, G, n + 16)), dict(Cm=z(T, G, n).bfloat16()), dict(Bm=z(T - 1, G, n)), dict(dt=z(T, H + 1)),
                dict(x=z(H, T, d).transpose(0, 1)), dict(A_log=z(H).double()), dict(D=z(H + 1)), dict(cu_seqlens=z(N + 1, dtype=torch.int64)),
                dict(pool=pool), dict(slot_map=slots), dict(pool=z(3, H, n, d + 1), slot_map=slots), dict(pool=pool, slot_map=slots.long()),
                dict(pool=pool, slot_map=slots[:1]), dict(out=z(T, H, d + 1))):
        with pytest.raises(ValueError):
            gdn.gdn_mamba2_scan(**dict(good, **bad))
    for bad in (dict(dy=z(T, H, d + 1)), dict(dy=z(T, H, d).bfloat16()), dict(dfinal=z(N, H, d, n).bfloat16()), dict(dfinal=z(N + 1, H, d, n))):
        with pytest.raises(ValueError):
            gdn.gdn_mamba2_scan_backward(**dict(good, **dict(dict(dy=z(T, H, d)), **bad)))


# Sizes at which a kernel's launch would have 2^32 threads: (N, T, dims, forward is refused, backward is refused).
LAUNCHES = [
    (300_000, 300_000, dict(H=128, G=8), True, True),                   # walks of two heads
    (1 << 24, 1 << 24, dict(H=1, G=1), True, True),                     # chunks, one token each
    ((1 << 24) - 1, 64, dict(H=1, G=1), True, True),
    (1 << 23, 64, dict(H=1, G=1), False, True),                         # the gradient kernel has 512 threads a workgroup
    (70_000, 70_000, dict(H=128, G=8), False, False),
    (1_100_000, 1_100_000, dict(H=8, G=8, d=16, n=16), False, True),
    (1_100_000, 1_100_000, dict(H=16, G=16, d=16, n=16), True, True),
    ((1 << 31) - 1, 0, dict(H=1, G=1), False, None),                    # no token: nothing to launch
]


@pytest.mark.parametrize("N,T,dims,fwd,bwd", LAUNCHES)
def test_launches_past_2_32_threads(L, N, T, dims, fwd, bwd):
    q = ctypes.byref(bd.gdn_m2_dims(*dict(DIMS, **dims).values()))
    for refused, size, call in ((fwd, L.gdn_mamba2_scan_workspace_bytes, _fwd), (bwd, L.gdn_mamba2_scan_backward_workspace_bytes, _bwd)):
        if refused is None:
            continue
        assert (size(q, N, T) == 0) == refused
        # without a workspace nothing is launched either way; only the reason differs
        st = call(L, N=N, T=T, dims=dims, ws=None)
        assert st == (gdn.GDN_EUNSUPPORTED if refused else gdn.GDN_OK if T == 0 else gdn.GDN_EINVAL), gdn.gdn_last_error()
        assert not refused or "threads" in gdn.gdn_last_error()
