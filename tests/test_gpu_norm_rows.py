"""The norm's backward pass where every workgroup walks several rows (more than twice as many rows as workgroups, not a multiple),
and its outputs in the place of its inputs."""
import ctypes

import pytest
import torch

import test_gpu_norm as base
from gpu_util import DEV, require_gpu, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("rows,width", [(4200, 1000), (4200, 513), (1101, 4096), (1101, 2049), (603, 4097), (603, 8192), (603, 8193), (603, 16384)])
@pytest.mark.parametrize("dt,rms,bias,gate", [("bf16", False, True, "none"), ("bf16", False, True, "before"), ("bf16", False, True, "after"),
                                              ("f32", True, False, "before"), ("f16", True, True, "after")])
def test_rows_of_a_workgroup(rows, width, dt, rms, bias, gate):
    base.check(rows, width, 1, dt, rms, bias, gate)


def test_groups_share_the_workgroups():
    base.check(1301, 8192, 8, "bf16", True, False, "before")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "before", "after"])
@pytest.mark.parametrize("rows,width", [(40_000, 7), (33_001, 127), (9001, 511), (4200, 999), (2101, 2047), (1101, 4095), (603, 8191), (603, 9001)])
def test_outputs_in_place(rows, width, gate, dt):
    """dx over dy, dx over x, dz over z: the same bits as in tensors of their own."""
    import gated_deltanet_state_gdn_amd as gdn
    from gated_deltanet_state_gdn_amd import _binding as bd
    d, _ = base.make(rows, width, dt, True, gate, 3)
    z = d["z"]
    kw = dict(gate=z, gate_after=gate == "after")
    _, mean, rstd = gdn.gdn_layer_norm(d["x"], d["w"], d["b"], save_stats=True, **kw)
    want = gdn.gdn_layer_norm_backward(d["dy"], d["x"], d["w"], mean, rstd, bias=d["b"], **kw)
    dims = bd.gdn_norm_dims(rows, width, 1, 0, dict(none=0, before=1, after=2)[gate])
    L = gdn.lib()
    ws = torch.empty(L.gdn_layer_norm_backward_workspace_bytes(ctypes.byref(dims)), dtype=torch.uint8, device=DEV)
    for over in ("dy", "x"):
        t = {k: d[k].clone() for k in ("dy", "x")}
        zz = z.clone() if z is not None else None
        dw, db = torch.empty(width, device=DEV), torch.empty(width, device=DEV)
        pz = zz.data_ptr() if zz is not None else None
        st = L.gdn_layer_norm_backward(ctypes.byref(dims), t["dy"].data_ptr(), 0, t["x"].data_ptr(), 0, pz, 0, bd.dtype_code(torch_dtype(dt)),
                                       d["w"].data_ptr(), d["b"].data_ptr(), mean.data_ptr(), rstd.data_ptr(), t[over].data_ptr(), 0, pz, 0,
                                       dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == gdn.GDN_OK, gdn.gdn_last_error()
        assert torch.equal(t[over], want.dx) and torch.equal(dw, want.dweight) and torch.equal(db, want.dbias)
        assert zz is None or torch.equal(zz, want.dgate)
