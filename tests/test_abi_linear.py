"""Refusals of linear attention's entry points and of the norm and rotation of queries and keys, on the host (no kernel is launched:
every call fails its checks or has nothing to do)."""
import ctypes
import os
import warnings

import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
from gated_deltanet_state_gdn_amd import _binding as bd

FAKE = 0x7F0000000000
DIMS = dict(H=8, Hq=4, Hk=2, Hv=8, dk=64, dv=64, scale=0.0)
POOL = bd.gdn_pool(FAKE, gdn.GDN_F32, 4)
E, U, OK = gdn.GDN_EINVAL, gdn.GDN_EUNSUPPORTED, gdn.GDN_OK


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bd.LIB_PATH):
        from gated_deltanet_state_gdn_amd import build
        build.build()
    return gdn.lib()


def ref(x):
    return ctypes.byref(x) if x is not None else None


def head(dims):
    return ref(bd.gdn_linear_dims(*dict(DIMS, **dims).values()) if dims is not None else None)


def tail(q, k, v, dt, st, g, pool, sm):
    return q, k, v, dt, ref(bd.gdn_linear_strides(*st) if st is not None else None), g, ref(pool), sm


def step(L, B=3, dims={}, q=FAKE, k=FAKE, v=FAKE, dt=gdn.GDN_BF16, st=None, g=FAKE, pool=POOL, sm=FAKE, out=FAKE, out_dt=gdn.GDN_F32):
    return L.gdn_linear_decode_step(head(dims), B, *tail(q, k, v, dt, st, g, pool, sm), out, out_dt, None)


# enough tokens that the call needs a workspace
def scan(L, N=2, T=20000, dims={}, cu=FAKE, q=FAKE, k=FAKE, v=FAKE, dt=gdn.GDN_BF16, st=None, g=FAKE, pool=POOL, sm=FAKE, out=FAKE,
         out_dt=gdn.GDN_BF16, ws=FAKE, wsb=1 << 44):
    return L.gdn_linear_scan(head(dims), N, cu, T, *tail(q, k, v, dt, st, g, pool, sm), out, out_dt, ws, wsb, None)


def back(L, N=2, T=20000, dims={}, cu=FAKE, q=FAKE, k=FAKE, v=FAKE, dt=gdn.GDN_BF16, st=None, g=FAKE, pool=POOL, sm=FAKE, do=FAKE,
         dfinal=None, dq=FAKE, dk=FAKE, dv=FAKE, dinit=None, ws=FAKE, wsb=1 << 44):
    return L.gdn_linear_scan_backward(head(dims), N, cu, T, *tail(q, k, v, dt, st, g, pool, sm), do, dfinal, dq, dk, dv, dinit, ws, wsb, None)


BAD = [
    (dict(dims=None), E),
    (dict(dims=dict(H=0)), E),
    (dict(dims=dict(Hq=3)), E),                    # does not divide the states
    (dict(dims=dict(Hk=0)), E),
    (dict(dims=dict(Hv=16)), E),
    (dict(dims=dict(dk=0, dv=0)), E),
    (dict(dims=dict(dk=64, dv=128)), U),
    (dict(dims=dict(dk=96, dv=96)), U),
    (dict(dims=dict(scale=float("inf"))), E),
    (dict(dims=dict(scale=float("nan"))), E),
    (dict(dims=dict(H=1 << 16, Hq=1, Hk=1, Hv=1, dk=128, dv=128)), U),
    (dict(dt=7), E),
    (dict(q=None), E),
    (dict(k=FAKE + 8), E),
    (dict(v=FAKE + 2), E),
    (dict(st=(4 * 64 - 8, 0, 0)), E),              # tokens would overlap
    (dict(st=(0, 2 * 64 + 4, 0)), E),              # not whole vectors
    (dict(st=(0, 0, -512)), E),
    (dict(st=(0, 0, (1 << 22) + 8)), U),
    (dict(g=None), E),
    (dict(g=FAKE + 2), E),
    (dict(pool=None), E),
    (dict(sm=None), E),
    (dict(sm=FAKE + 1), E),
    (dict(pool=bd.gdn_pool(FAKE + 8, gdn.GDN_F32, 4)), E),
    (dict(pool=bd.gdn_pool(FAKE, 9, 4)), E),
    (dict(pool=bd.gdn_pool(FAKE, gdn.GDN_F32, 0)), E),
]


@pytest.mark.parametrize("case,expect", BAD + [
    (dict(B=-1), E), (dict(B=1 << 21), U), (dict(out=None), E), (dict(out=FAKE + 2), E), (dict(out_dt=-1), E),
    (dict(B=0, q=None, out=None, pool=None, sm=None), OK),
])
def test_step_refusals(L, case, expect):
    assert step(L, **case) == expect, gdn.gdn_last_error()
    assert (gdn.gdn_last_error() == "") == (expect == OK)


SIZES = [(dict(N=-1), E), (dict(T=-1), E), (dict(T=1 << 31), E), (dict(N=0, T=4), E), (dict(cu=None), E), (dict(cu=FAKE + 2), E),
         (dict(ws=None), E), (dict(ws=FAKE + 128), E), (dict(wsb=1000), E), (dict(N=1 << 24, T=1 << 24), U)]


@pytest.mark.parametrize("case,expect", BAD + SIZES + [
    (dict(out=None), E), (dict(out=FAKE + 8), E), (dict(out_dt=3), E),
    (dict(T=0, ws=None, out=None), OK), (dict(N=0, T=0, cu=None, ws=None), OK), (dict(N=(1 << 31) - 1, T=0, ws=None), OK),
])
def test_scan_refusals(L, case, expect):
    assert scan(L, **case) == expect, gdn.gdn_last_error()
    assert (gdn.gdn_last_error() == "") == (expect == OK)


@pytest.mark.parametrize("case,expect", BAD + SIZES + [
    (dict(do=None), E), (dict(do=FAKE + 8), E), (dict(dfinal=FAKE + 4), E), (dict(dinit=FAKE + 8), E), (dict(dq=None), E), (dict(dk=FAKE + 2), E),
    (dict(dv=None), E), (dict(N=(1 << 31) - 1, T=0), U), (dict(T=(1 << 31) - 1, dims=dict(H=64, Hq=1, Hk=1, Hv=1)), U), (dict(N=0, T=0, cu=None, ws=None), OK),
])
def test_backward_refusals(L, case, expect):
    assert back(L, **case) == expect, gdn.gdn_last_error()
    assert (gdn.gdn_last_error() == "") == (expect == OK)


def test_workspace_sizes(L):
    f = lambda N, T, **d: L.gdn_linear_scan_workspace_bytes(head(d), N, T)  # noqa: E731
    b = lambda N, T, **d: L.gdn_linear_scan_backward_workspace_bytes(head(d), N, T)  # noqa: E731
    assert f(0, 0) == b(0, 0) == 0
    assert f(1, 500) == 0                                     # one walk over eight chunks: nothing to keep
    assert f(2, 100, dk=96, dv=96) == 0
    same = dict(Hq=8, Hk=8, Hv=8)
    assert b(1, 500, **same) == 0
    assert b(1, 500, Hq=8, Hk=4, Hv=8) == 500 * 8 * 64 * 4    # every state's own dk
    assert f(1, 1 << 16, **same) > 0 and b(1, 1 << 16, **same) > 0  # segments' states


# ------------------------------------------------------------------ norm and rotation of q and k
def qk_head(tokens=5, Hq=4, Hk=2, d=64, rot=32, nb=0, axes=1, pair=None):
    return ref(bd.gdn_qk_dims(tokens, Hq, Hk, d, rot, nb, axes, pair))


def qk(L, dims={}, q=FAKE, qs=0, k=FAKE, ks=0, dt=gdn.GDN_BF16, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, f=FAKE, yq=FAKE, yqs=0, yk=FAKE, yks=0):
    return L.gdn_qk_norm_rope(qk_head(**dims) if dims is not None else None, q, qs, k, ks, dt, qw, kw, eps, pos, f, yq, yqs, yk, yks, None)


def qk_back(L, dims={}, gq=FAKE, gqs=0, gk=FAKE, gks=0, q=FAKE, qs=0, k=FAKE, ks=0, dt=gdn.GDN_BF16, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE,
            f=FAKE, yq=FAKE, yqs=0, yk=FAKE, yks=0, dqw=FAKE, dkw=FAKE, ws=FAKE, wsb=1 << 40):
    return L.gdn_qk_norm_rope_backward(qk_head(**dims) if dims is not None else None, gq, gqs, gk, gks, q, qs, k, ks, dt, qw, kw, eps, pos, f,
                                       yq, yqs, yk, yks, dqw, dkw, ws, wsb, None)


QK = [
    (dict(dims=None), E), (dict(dims=dict(tokens=-1)), E), (dict(dims=dict(tokens=1 << 31)), U), (dict(dims=dict(Hq=0)), E),
    (dict(dims=dict(Hk=-2)), E), (dict(dims=dict(d=8, rot=8)), U), (dict(dims=dict(d=100)), U), (dict(dims=dict(d=264)), U),
    (dict(dims=dict(rot=0)), E), (dict(dims=dict(rot=72)), E), (dict(dims=dict(rot=15)), E), (dict(dims=dict(rot=12)), U),
    (dict(dims=dict(axes=0)), E), (dict(dims=dict(axes=5)), U), (dict(dims=dict(axes=2, pair=bytes([0, 1] * 7 + [0, 2]))), E),
    (dict(dims=dict(Hq=1 << 17)), U), (dict(dt=3), E), (dict(q=None), E), (dict(k=FAKE + 8), E), (dict(qs=4 * 64 - 8), E), (dict(ks=130), E),
    (dict(qs=-256), E), (dict(ks=(1 << 22) + 8), U), (dict(qw=None), E), (dict(kw=FAKE + 2), E), (dict(eps=-1.0), E), (dict(eps=float("nan")), E),
    (dict(pos=None), E), (dict(f=FAKE + 1), E), (dict(yq=None), E), (dict(yk=FAKE + 4), E), (dict(yqs=64), E),
]


@pytest.mark.parametrize("case,expect", QK + [(dict(dims=dict(tokens=0), q=None, pos=None, yq=None), OK)])
def test_qk_refusals(L, case, expect):
    assert qk(L, **case) == expect, gdn.gdn_last_error()
    assert (gdn.gdn_last_error() == "") == (expect == OK)


@pytest.mark.parametrize("case,expect", QK + [(dict(gq=None), E), (dict(gk=FAKE + 8), E), (dict(gqs=8), E), (dict(dqw=None), E), (dict(dkw=FAKE + 1), E),
                                              (dict(ws=None), E), (dict(ws=FAKE + 64), E), (dict(wsb=16), E)])
def test_qk_backward_refusals(L, case, expect):
    assert qk_back(L, **case) == expect, gdn.gdn_last_error()
    assert gdn.gdn_last_error() != ""


# ------------------------------------------------------------------ the binding
T, H, d, N = 6, 4, 16, 2
z = torch.zeros


def linear(device="cpu"):
    w = lambda *s, **k: z(*s, device=device, **k)  # noqa: E731
    return (dict(q=w(T, 2, d), k=w(T, 1, d), v=w(T, H, d), log_decay=w(H)), dict(cu_seqlens=torch.tensor([0, 2, T], dtype=torch.int32, device=device)),
            dict(pool=w(9, H, d, d), slot_map=torch.tensor([2, 0], dtype=torch.int32, device=device)))


def rotation(device="cpu"):
    w = lambda *s, **k: z(*s, device=device, **k)  # noqa: E731
    return dict(q=w(T, 3, 32), k=w(T, 1, 32), q_weight=w(32), k_weight=w(32), positions=w(T, dtype=torch.int32), inv_freq=w(8))


def test_binding_refuses_shapes_and_types():
    ins, cu, states = linear()
    for bad in (dict(q=z(T, 2 * d)), dict(q=z(T - 1, 2, d)), dict(k=z(T, 1, d + 1)), dict(k=z(T, 1, d).bfloat16()), dict(v=z(H, T, d).transpose(0, 1)),
                dict(log_decay=z(H).double()), dict(log_decay=z(1, H)), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf"))):
        with pytest.raises(ValueError):
            gdn.gdn_linear_scan(**dict(ins, **cu, **states) | bad)
        with pytest.raises(ValueError):
            gdn.gdn_linear_scan_backward(z(T, H, d), **dict(ins, **cu, **states) | bad)
        with pytest.raises(ValueError):
            gdn.gdn_linear_decode_step(**dict(ins, pool=states["pool"], slot_map=z(T, dtype=torch.int32)) | bad)
    for bad in (dict(cu_seqlens=z(3, dtype=torch.int64)), dict(pool=states["pool"]), dict(slot_map=states["slot_map"]),
                dict(pool=z(9, H, d), slot_map=states["slot_map"]), dict(pool=z(9, H, d, d + 1), slot_map=states["slot_map"]),
                dict(pool=states["pool"], slot_map=states["slot_map"].long()), dict(pool=states["pool"], slot_map=states["slot_map"][:1]),
                dict(out=z(T, H, d + 1))):
        with pytest.raises(ValueError):
            gdn.gdn_linear_scan(**dict(ins, **cu) | bad)
    for bad in (dict(do=z(T, H, d + 1)), dict(do=z(T, H, d).bfloat16()), dict(dfinal=z(N, H, d, d).bfloat16()), dict(dfinal=z(N + 1, H, d, d))):
        with pytest.raises(ValueError):
            gdn.gdn_linear_scan_backward(**dict(ins, **cu, do=z(T, H, d)) | bad)
    rot = rotation()
    grads = dict(dq_out=z(T, 3, 32), dk_out=z(T, 1, 32))
    for bad in (dict(q=z(T, 96)), dict(k=z(T + 1, 1, 32)), dict(k=z(T, 1, 40)), dict(k=z(T, 1, 32).half()), dict(q_weight=z(16)), dict(k_weight=z(32).half()),
                dict(positions=z(T)), dict(positions=z(T + 1, dtype=torch.int32)), dict(positions=z(2, T, dtype=torch.int32)),
                dict(positions=z(2, T, dtype=torch.int32), axes=[0, 1]), dict(axes=[4] * 8), dict(axes=[-1] * 8), dict(inv_freq=z(8).double()),
                dict(inv_freq=z(1, 8))):
        with pytest.raises(ValueError):
            gdn.gdn_qk_norm_rope(**rot | bad)
        with pytest.raises(ValueError):
            gdn.gdn_qk_norm_rope_backward(**rot | grads | bad)
    for bad in (dict(q_out=z(T, 3, 40)), dict(k_out=z(T + 1, 1, 32)), dict(k_out=z(T, 1, 32).half()), dict(q_out=z(1, 3, 32).expand(T, 3, 32))):
        with pytest.raises(ValueError):
            gdn.gdn_qk_norm_rope(**rot | bad)
    for bad in (dict(dq_out=z(T, 3, 40)), dict(dk_out=z(T, 1, 32).bfloat16())):
        with pytest.raises(ValueError):
            gdn.gdn_qk_norm_rope_backward(**rot | grads | bad)


def test_host_tensors_are_refused():
    ins, cu, states = linear()
    rot = rotation()
    for call in (lambda: gdn.gdn_linear_scan(**ins, **cu), lambda: gdn.gdn_linear_scan(**ins, **cu, **states),
                 lambda: gdn.gdn_linear_scan_backward(z(T, H, d), **ins, **cu),
                 lambda: gdn.gdn_linear_decode_step(**ins, pool=states["pool"], slot_map=z(T, dtype=torch.int32)),
                 lambda: gdn.gdn_qk_norm_rope(**rot), lambda: gdn.gdn_qk_norm_rope_backward(rot["q"], rot["k"], **rot)):
        with pytest.raises(ValueError, match="must lie on a GPU"):
            call()


def test_calls_without_a_graph_say_so():
    for k in ("q", "k", "v", "pool", "log_decay"):
        ins, cu, states = linear()
        next(a for a in (ins, states) if k in a)[k].requires_grad_()
        with pytest.warns(UserWarning, match="constant" if k == "log_decay" else "gdn_linear_scan_backward"), pytest.raises(ValueError):
            gdn.gdn_linear_scan(**ins, **cu, **states)
    for k in ("q", "k", "q_weight", "k_weight"):
        rot = rotation()
        rot[k].requires_grad_()
        with pytest.warns(UserWarning, match="gdn_qk_norm_rope_backward"), pytest.raises(ValueError):
            gdn.gdn_qk_norm_rope(**rot)
    with warnings.catch_warnings(), torch.no_grad():
        warnings.simplefilter("error")
        with pytest.raises(ValueError):
            gdn.gdn_qk_norm_rope(**rot)


@pytest.mark.gpu
def test_one_host_tensor_is_refused():
    ins, cu, states = linear("cuda")
    rot = rotation("cuda")
    whole = dict(ins, **cu, **states)
    gdn.gdn_linear_scan(**whole)
    for k in whole:
        if k != "q":
            for call in (lambda a: gdn.gdn_linear_scan(**a), lambda a: gdn.gdn_linear_scan_backward(z(T, H, d, device="cuda"), **a)):
                with pytest.raises(ValueError, match="must lie on cuda"):
                    call(whole | {k: whole[k].cpu()})
    for bad in (dict(out=z(T, H, d)), dict(workspace=z(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="must lie on cuda"):
            gdn.gdn_linear_scan(**whole, **bad)
    for bad in (dict(do=z(T, H, d)), dict(do=z(T, H, d, device="cuda"), dfinal=z(N, H, d, d))):
        with pytest.raises(ValueError, match="must lie on cuda"):
            gdn.gdn_linear_scan_backward(**whole | bad)
    one = dict(ins, pool=states["pool"], slot_map=torch.arange(T, dtype=torch.int32, device="cuda"))
    gdn.gdn_linear_decode_step(**one)
    for k in one:
        if k != "q":
            with pytest.raises(ValueError, match="must lie on cuda"):
                gdn.gdn_linear_decode_step(**one | {k: one[k].cpu()})
    gdn.gdn_qk_norm_rope(**rot)
    for k in rot:
        if k != "q":
            with pytest.raises(ValueError, match="must lie on cuda"):
                gdn.gdn_qk_norm_rope(**rot | {k: rot[k].cpu()})
            with pytest.raises(ValueError, match="must lie on cuda"):
                gdn.gdn_qk_norm_rope_backward(rot["q"], rot["k"], **rot | {k: rot[k].cpu()})
    torch.cuda.synchronize()
