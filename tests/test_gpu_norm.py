"""GPU parity of gdn_layer_norm and gdn_layer_norm_backward against the float64 oracle.

Tolerances count roundings.  An output in type t is off by half a step of it, eps(t) / 2 relative.  In FP32, a slice's sum
takes at most 16 additions a lane and 14 across lanes and waves, so means and variances are within 32 x 2^-24 of the mean of
what they add; with the few products before and after, a normalised value is within K = 64 x 2^-24 of (|h| + 1), and the
same holds for each term of a gradient.  The weight's gradient adds its rows in at most rows / 16 + 64 further steps.
"""
import numpy as np
import pytest

import oracle as O

from gpu_util import DEV, host, require_gpu, say, torch_dtype, widen

pytestmark = pytest.mark.gpu
EPS = 1e-5
K = 64 * 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}  # half a step among the smallest f16 numbers


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(rows, width, dt, bias, gate, seed, offset=0.0, gap=0):
    """Device tensors (rows `gap` elements further apart than the width) and their values in float64."""
    import torch
    g = torch.Generator().manual_seed(seed)

    def rowed(scale, shift=0.0):
        t = (torch.randn((rows, width + gap), generator=g) * scale + shift).to(torch_dtype(dt)).to(DEV)
        return t[:, :width] if gap == 0 else t[:, gap // 2:gap // 2 + width]
    d = dict(x=rowed(1.0, offset), dy=rowed(0.05), z=rowed(1.5) if gate != "none" else None,
             w=(torch.randn(width, generator=g) * 0.2 + 1).to(DEV), b=torch.randn(width, generator=g).to(DEV) if bias else None)
    return d, {k: None if v is None else v.double().cpu().numpy() for k, v in d.items()}


def close(got, ref, slack, dt, what):
    got = got.double().cpu().numpy() if not isinstance(got, np.ndarray) else got
    err, bound = np.abs(got - ref), HALF[dt] * np.abs(ref) + slack + TINY[dt]
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    assert (err <= bound).all(), f"{what}: {np.argwhere(err > bound)[:4].tolist()} off by up to {(err / bound).max():.2f} bounds"


def check(rows, width, groups, dt, rms, bias, gate, seed=1, out_dt=None, **kw):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    say(f"norm rows={rows} width={width} groups={groups} {dt} rms={rms} bias={bias} gate={gate} {kw}")
    d, r = make(rows, width, dt, bias, gate, seed, **kw)
    form = dict(groups=groups, rms=rms, gate_after=gate == "after")
    y, mean, rstd = gdn.gdn_layer_norm(d["x"], d["w"], d["b"], gate=d["z"], eps=EPS, save_stats=True, out_dtype=torch_dtype(out_dt or dt), **form)
    g = gdn.gdn_layer_norm_backward(d["dy"], d["x"], d["w"], mean, rstd, bias=d["b"], gate=d["z"], **form)
    torch.cuda.synchronize()
    ref = {k: r[k] for k in ("x", "w", "b", "z")}
    y_r, m_r, r_r = O.layer_norm(**ref, **form, eps=EPS)
    dx_r, dw_r, db_r, dz_r = O.layer_norm_backward(r["dy"], **ref, **form, eps=EPS)
    # the sizes of what is added
    silu, slope = O.norm_oracle._silu(r["z"]) if gate != "none" else (1.0, 0.0)
    u = (r["x"] * silu if gate == "before" else r["x"]).reshape(rows, groups, -1)
    big = np.abs(u).mean(-1, keepdims=True)
    rs = r_r[..., None]
    h = ((u - m_r[..., None]) * rs).reshape(rows, width)
    away = (big * rs * np.ones(u.shape)).reshape(rows, width)  # |mean| r: what a mean far from zero costs
    sh = K * (np.abs(h) + 1 + away)
    sv = sh * np.abs(r["w"]) + 4 * HALF["f32"] * np.abs(0.0 if r["b"] is None else r["b"])
    close(mean, m_r, K * big[..., 0], "f32", "mean")
    close(rstd, r_r, K * r_r * (1 + (big * rs)[..., 0]), "f32", "rstd")
    after = silu if gate == "after" else 1.0
    close(y, y_r, sv * np.abs(after) + K * np.abs(y_r), out_dt or dt, "y")
    e = (r["dy"] * after * r["w"]).reshape(u.shape)
    hg, shg = np.abs(h).reshape(u.shape), sh.reshape(u.shape)
    eh = np.abs(e * hg).mean(-1, keepdims=True)
    se = (np.abs(e) * shg).mean(-1, keepdims=True)
    sdu = (rs * (K * (1 + away.reshape(u.shape)) * (np.abs(e) + np.abs(e).mean(-1, keepdims=True) + hg * eh) + shg * eh + hg * se)).reshape(rows, width)
    close(g.dx, dx_r, sdu * np.abs(silu if gate == "before" else 1.0) + K * np.abs(dx_r), dt, "dx")
    if gate == "before":
        close(g.dgate, dz_r, sdu * np.abs(r["x"] * slope) + K * np.abs(dz_r) + K * np.abs(sdu / K * r["x"]), dt, "dgate")
    elif gate == "after":
        close(g.dgate, dz_r, np.abs(r["dy"]) * (sv * np.abs(slope) + K * np.abs(y_r if r["z"] is None else r["w"] * h)) + K * np.abs(r["dy"]) * np.abs(0.0 if r["b"] is None else r["b"]), dt, "dgate")
    else:
        assert g.dgate is None
    dv = np.abs(r["dy"] * after)
    steps = (rows / 16 + 64) * 2.0 ** -24
    close(g.dweight, dw_r, (dv * (sh + (steps + K) * np.abs(h))).sum(0), "f32", "dweight")
    if bias:
        close(g.dbias, db_r, ((steps + K) * dv).sum(0), "f32", "dbias")
    else:
        assert g.dbias is None


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rms,bias,gate", [(False, True, "none"), (True, False, "before"), (True, True, "after"), (False, True, "before")])
def test_forms(dt, rms, bias, gate):
    """Every form on slices of 128 (16 lanes), 200 (one wave) and 2048 (four waves)."""
    for width, groups in ((256, 2), (200, 1), (2048, 1)):
        check(19, width, groups, dt, rms, bias, gate)


@pytest.mark.parametrize("width,groups", [(1, 1), (7, 1), (8, 1), (129, 1), (513, 1), (999, 3), (1025, 1), (2049, 1), (4097, 1), (8193, 1), (16384, 1), (8192, 8)])
def test_widths(width, groups):
    """Both sides of every change of lanes, odd widths (rows then start at any 2-byte element), one element."""
    check(5, width, groups, "bf16", False, True, "none")
    check(3, width, groups, "f32", True, False, "after")


@pytest.mark.parametrize("rows", [1, 2, 16, 17, 4099])
def test_rows(rows):
    check(rows, 96, 1, "bf16", True, False, "after")
    check(rows, 1200, 1, "f16", False, True, "none")


@pytest.mark.parametrize("gap", [6, 64])
def test_rows_apart(gap):
    """Rows that are slices of wider rows: any stride, starts that are not 16-byte aligned."""
    check(33, 320, 1, "bf16", False, True, "before", gap=gap)
    check(33, 320, 1, "f32", True, False, "after", gap=gap)


def test_mean_far_from_zero_and_other_output_type():
    """A mean 200 deviations from zero: the variance comes from the deviations, so only the mean's own rounding shows."""
    check(9, 1000, 1, "f32", False, True, "none", offset=200.0)
    check(9, 1000, 1, "bf16", False, True, "none", out_dt="f32")
    check(9, 1000, 1, "f32", False, True, "none", out_dt="bf16")


def test_constant_zero_and_nonfinite_rows():
    """A constant row normalises to the bias, a zero row too; NaN and infinities stay in their own slice."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    x = torch.zeros((4, 256), device=DEV)
    x[1] = 3.0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    w, b = torch.ones(256, device=DEV), torch.full((256,), 0.25, device=DEV)
    y = gdn.gdn_layer_norm(x, w, b, groups=2)
    assert (y[:2] == 0.25).all()
    assert y[2, :128].isnan().all() and (y[2, 128:] == 0.25).all()
    assert (y[3, :128] == 0.25).all() and not y[3, 128:].isfinite().any()


def test_no_rows():
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    x, w = torch.empty((0, 64), device=DEV), torch.ones(64, device=DEV)
    y, mean, rstd = gdn.gdn_layer_norm(x, w, save_stats=True)
    assert y.shape == (0, 64) and mean.shape == (0, 1)
    g = gdn.gdn_layer_norm_backward(x, x, w, mean, rstd, bias=w)
    assert (g.dweight == 0).all() and (g.dbias == 0).all() and g.dx.shape == (0, 64)


def test_equal_calls_equal_bits_streams_and_graph():
    """Sums have one order: the same bits on another stream and from replays of a captured graph with other work between."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    d, _ = make(3001, 1536, "bf16", True, "before", 5)
    form = dict(gate=d["z"])
    y, mean, rstd = gdn.gdn_layer_norm(d["x"], d["w"], d["b"], save_stats=True, **form)
    ref = gdn.gdn_layer_norm_backward(d["dy"], d["x"], d["w"], mean, rstd, bias=d["b"], **form)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    on = gdn.gdn_layer_norm_backward(d["dy"], d["x"], d["w"], mean, rstd, bias=d["b"], stream=s, **form)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, on))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, m2, r2 = gdn.gdn_layer_norm(d["x"], d["w"], d["b"], save_stats=True, **form)
        got = gdn.gdn_layer_norm_backward(d["dy"], d["x"], d["w"], m2, r2, bias=d["b"], **form)
    for _ in range(3):
        got.dweight.fill_(7.0), got.dx.zero_(), y2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(ref, got))
