"""GPU parity of gdn_qk_norm_rope and its backward against the float64 oracle.

Tolerances count FP32 roundings.  Forward: the sum of squares, all of one sign, takes 13 additions and 8 products on its way, half
of whose relative errors reach r; with r's own, the two products, and a cosine and sine off by at most 2^-22 (the angle's last
eighth of a turn is rounded once, and the functions are good to 2 steps), a value is within KF = 48 steps of 2^-24 of |a| + |b|,
the sizes of its normed pair.  Backward: the same for the turned gradient, the second sum has 13 additions of terms of either
sign, so dx is within KB = 96 steps of r (|dh| + |xh| mean |dh xh|) with the pair's sizes in |dh|.  The weights' gradients are
sums in chains of at most 400 here: KW = 512 steps of the sum of sizes.  Outputs are off by half a step of their type.
"""
import numpy as np
import pytest

import oracle as O

from gpu_util import DEV, require_gpu, say, torch_dtype

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24
KF, KB, KW = 48 * STEP, 96 * STEP, 512 * STEP
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(T, Hq, Hk, d, rot, dt, axes=None, far=0, seed=1, wide=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)

    def tensor(h, scale):
        x = (torch.randn((T, h, d), generator=g) * scale).to(torch_dtype(dt)).to(DEV)
        if wide:
            row = torch.full((T, h * d + wide), float("nan"), dtype=x.dtype, device=DEV)
            row[:, :-wide] = x.reshape(T, -1)
            x = row[:, :-wide].unflatten(1, (h, d))
        return x

    v = dict(q=tensor(Hq, 2.0), k=tensor(Hk, 0.5), dq=tensor(Hq, 0.1), dk=tensor(Hk, 0.1))
    v["qw"], v["kw"] = (torch.randn(d, generator=g).to(DEV) for _ in range(2))
    n = max(axes) + 1 if axes else 1
    pos = r.integers(0, 200, size=(n, T)) + far
    v["pos"] = torch.from_numpy(pos if axes else pos[0]).to(torch.int32).to(DEV)
    v["freq"] = (1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV)
    return v


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, slack, dt, what):
    got = f64(got)
    err, bound = np.abs(got - ref), HALF[dt] * np.abs(ref) + slack + TINY[dt]
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    worst = (err / bound).max() if err.size else 0.0
    assert worst <= 1.0, f"{what}: {np.argwhere(err > bound)[:4].tolist()} off by up to {worst:.2f} bounds"


def pair_sizes(n, P, neighbours):
    """|a| + |b| of each value's pair."""
    i = np.arange(P)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + P)
    s = np.abs(n).copy()
    s[..., a] = s[..., b] = np.abs(n[..., a]) + np.abs(n[..., b])
    return s


def check(v, dt, eps, neighbours, axes, **how):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    form = dict(eps=eps, neighbours=neighbours, axes=axes)
    args = (v["q"], v["k"], v["qw"], v["kw"], v["pos"], v["freq"])
    out = gdn.gdn_qk_norm_rope(*args, **form, **how)
    g = gdn.gdn_qk_norm_rope_backward(v["dq"], v["dk"], *args, **form)
    torch.cuda.synchronize()
    pos, freq, P = f64(v["pos"]), f64(v["freq"]), v["freq"].shape[0]
    for i, name in enumerate("qk"):
        x, w, dy = f64(v[name]), f64(v[name + "w"]), f64(v["d" + name])
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        close(out[i], O.qk_norm_rope(x, w, pos, freq, **form), KF * pair_sizes(x * r * w, P, neighbours), dt, name)
        dx, dw = O.qk_norm_rope_backward(dy, x, w, pos, freq, **form)
        dn, xh = pair_sizes(dy, P, neighbours), np.abs(x * r)
        dh = dn * np.abs(w)
        close(g[i], dx, KB * r * (dh + xh * (dh * xh).mean(-1, keepdims=True)), dt, "d" + name)
        close(g[2 + i], dw, KW * (dn * xh).sum((0, 1)), "f32", f"d{name}_weight")


@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(1, 1, 1, 16, 8), (3, 32, 8, 128, 128), (7, 4, 2, 64, 32), (130, 6, 1, 80, 40), (33, 5, 5, 24, 24),
                                           (65, 3, 2, 256, 256), (17, 2, 70, 192, 64), (2, 2, 2, 96, 8), (600, 2, 1, 32, 32), (2500, 3, 2, 128, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
def test_qk(T, Hq, Hk, d, rot, dt, neighbours):
    say(f"qk T={T} heads={Hq}, {Hk} d={d} rot={rot} {dt} neighbours={neighbours}")
    check(make(T, Hq, Hk, d, rot, dt), dt, 1e-6, neighbours, None)


@pytest.mark.parametrize("axes", [[0, 1, 2] * 5 + [3], [0] * 6 + [1] * 5 + [2] * 5, [1] * 16])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
def test_several_axes(axes, dt, neighbours):
    check(make(50, 3, 2, 40, 32, dt, axes), dt, 1e-5, neighbours, axes)


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 300, -(2 ** 31)])
def test_far_positions(far):
    """In FP32 such angles would be off by whole turns; in FP64 by 2^-53 of 2^31, far below a step of a sine."""
    check(make(20, 2, 2, 64, 64, "f32", far=far), "f32", 1e-6, False, None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slices_of_wider_rows(dt):
    check(make(70, 3, 2, 64, 64, dt, wide=16), dt, 1e-6, False, None)


def test_rows_of_zeros_and_of_large_values():
    """A row of zeros is normed by eps alone; squares up to 2^124 stay finite."""
    import torch
    v = make(4, 2, 2, 64, 64, "f32")
    v["q"][0], v["k"][1], v["q"][2] = 0.0, 0.0, 1e18
    v["dq"][2] = 0.0
    check(v, "f32", 1e-6, False, None)
    assert torch.isfinite(v["q"]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("neighbours", [False, True])
def test_results_in_place_of_the_inputs(dt, neighbours):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v = make(45, 3, 2, 64, 48, dt)
    args = (v["qw"], v["kw"], v["pos"], v["freq"])
    want = gdn.gdn_qk_norm_rope(v["q"], v["k"], *args, neighbours=neighbours)
    rows = torch.cat([v["q"].reshape(45, -1), v["k"].reshape(45, -1)], 1)  # one projection's output
    q, k = rows[:, :192].unflatten(1, (3, 64)), rows[:, 192:].unflatten(1, (2, 64))
    got = gdn.gdn_qk_norm_rope(q, k, *args, neighbours=neighbours, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_without_tokens():
    import gated_deltanet_state_gdn_amd as gdn
    v = make(0, 2, 1, 32, 32, "bf16")
    args = (v["q"], v["k"], v["qw"], v["kw"], v["pos"], v["freq"])
    q, k = gdn.gdn_qk_norm_rope(*args)
    assert q.shape == (0, 2, 32) and k.shape == (0, 1, 32)
    g = gdn.gdn_qk_norm_rope_backward(v["dq"], v["dk"], *args)
    assert g.dq.shape == (0, 2, 32) and not g.dq_weight.any() and not g.dk_weight.any()


def test_captured_calls_and_another_stream():
    """Every replay as the eager call, with eager work between."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v = make(3000, 4, 2, 64, 64, "bf16")
    args = (v["q"], v["k"], v["qw"], v["kw"], v["pos"], v["freq"])

    def work(**how):
        return [*gdn.gdn_qk_norm_rope(*args, **how), *gdn.gdn_qk_norm_rope_backward(v["dq"], v["dk"], *args, **how)]

    want = [t.clone() for t in work()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        got = work(stream=handle)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for turn in range(4):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), turn
        again = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want)), turn
