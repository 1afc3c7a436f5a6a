"""GPU parity of gdn_mamba2_scan and gdn_mamba2_scan_backward against the float64 oracle.

Tolerances count roundings, as multiples of the sum of the terms' absolute values ("sizes", from the oracle).  In FP32 a term
passes a dozen roundings (products, exponentials of differences, the gates, whose errors reach the decay e^{c} as |c| e^{c} <= 0.4
of them), sums add at most 128 values a chunk or block in any order, and a state takes two more roundings a chunk: K = 512 steps
of 2^-24 cover sequences of up to some 100 chunks.  With bf16 inputs and a 16-bit output the state and the decay-weighted
products are rounded to bf16 once each, half a step (2^-8) of each term; the sums over heads behind dB and dC are kept to 2^-16.
The output itself is off by half a step of its type.
"""
import numpy as np
import pytest

import oracle as O
from workloads import gen

from gpu_util import DEV, require_gpu, say, torch_dtype

pytestmark = pytest.mark.gpu
K = 512 * 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# half a step among the smallest numbers: an f16 output's own; in FP32 that of every decay (2^-150), in sums of up to 2^10 units
TINY = {"f32": 2.0 ** -140, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}
NAMES = ("x", "Bm", "Cm", "dt", "A_log", "dt_bias", "D")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(lens, H, G, d, n, dt, sdt=None, seed=1, wide=0):
    """Device tensors and their float64 values; wide: x, Bm, Cm and dt are slices of wider rows (by that many elements)."""
    import torch
    T, N = sum(lens), len(lens)
    A_log, dt_bias, Dk = gen.m2_params(seed, H)
    raw = gen.m2_inputs(seed, 0, (T,), H, G, d, n, dt)
    dev = {k: gen.to_torch(raw[k], DEV) for k in ("x", "Bm", "Cm", "dt")}
    for k, v in zip(("A_log", "dt_bias", "D"), (A_log, dt_bias, Dk)):
        dev[k] = torch.from_numpy(v).to(DEV)
    dev = {k: v.reshape((T, H, d) if k == "x" else (T, G, n) if k in ("Bm", "Cm") else v.shape) for k, v in dev.items()}
    if wide:
        for k in ("x", "Bm", "Cm", "dt"):
            row = torch.full((T, dev[k][0].numel() + wide), float("nan"), dtype=dev[k].dtype, device=DEV)
            row[:, :-wide] = dev[k].reshape(T, -1)
            dev[k] = row[:, :-wide].unflatten(1, dev[k].shape[1:]) if dev[k].dim() == 3 else row[:, :-wide]
    g = torch.Generator().manual_seed(seed)
    dev["dy"] = (torch.randn((T, H, d), generator=g) * 0.1).to(torch_dtype(dt)).to(DEV)
    dev["dfinal"] = torch.randn((N, H, d, n), generator=g).mul(0.1).to(DEV)
    dev["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    if sdt is not None:
        dev["pool"] = (torch.randn((N + 2, H, d, n), generator=g) * 0.1).to(torch_dtype(sdt)).to(DEV)
        dev["slots"] = torch.randperm(N + 2, generator=g)[:N].to(torch.int32).to(DEV)
    ref = {k: v.double().cpu().numpy() for k, v in dev.items() if k not in ("cu", "slots")}
    ref["cu"] = dev["cu"].cpu().numpy()
    ref["slots"] = dev["slots"].cpu().numpy() if sdt is not None else None
    return dev, ref


def close(got, ref, slack, dt, what):
    got = got.double().cpu().numpy()
    err, bound = np.abs(got - ref), HALF[dt] * np.abs(ref) + slack + TINY[dt]
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    worst = (err / np.maximum(bound, 1e-300)).max() if err.size else 0.0
    assert worst <= 1.0, f"{what}: {np.argwhere(err > bound)[:4].tolist()} off by up to {worst:.2f} bounds"


def check_scan(lens, H, G, d, n, dt, sdt=None, out_dt=None, seed=1, wide=0):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    say(f"scan lens={lens} H={H} G={G} d={d} n={n} {dt} state={sdt} out={out_dt} wide={wide}")
    v, r = make(lens, H, G, d, n, dt, sdt, seed, wide)
    before = v["pool"].clone() if sdt else None
    y = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=v.get("pool"), slot_map=v.get("slots"), out_dtype=torch_dtype(out_dt or dt))
    torch.cuda.synchronize()
    ins = [r[k] for k in NAMES]
    form = dict(cu=r["cu"], init=r.get("pool"), slot_map=r["slots"])
    y_r, f_r = O.mamba2_scan(*ins, **form)
    y_s, f_s = O.mamba2_scan(*ins, **form, sizes=True)
    low = HALF["bf16"] * 1.02 if dt == "bf16" and (out_dt or dt) != "f32" else 0.0
    close(y, y_r, (K + low) * y_s, out_dt or dt, "y")
    if sdt:
        used = [s for s, k in enumerate(lens) if k > 0]
        slots = r["slots"][used]
        close(v["pool"][torch.as_tensor(slots).long().to(DEV)], f_r[used], K * f_s[used], sdt, "final states")
        rest = [i for i in range(before.shape[0]) if i not in slots]
        assert torch.equal(v["pool"][rest], before[rest]), "slots that no token reached"


def check_backward(lens, H, G, d, n, dt, sdt=None, dfinal=False, seed=1, wide=0):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    say(f"scan backward lens={lens} H={H} G={G} d={d} n={n} {dt} state={sdt} dfinal={dfinal} wide={wide}")
    v, r = make(lens, H, G, d, n, dt, sdt, seed, wide)
    before = v["pool"].clone() if sdt else None
    got = gdn.gdn_mamba2_scan_backward(v["dy"], *(v[k] for k in NAMES), v["cu"], pool=v.get("pool"), slot_map=v.get("slots"),
                                       dfinal=v["dfinal"] if dfinal else None)
    torch.cuda.synchronize()
    ins = [r["dy"]] + [r[k] for k in NAMES]
    form = dict(cu=r["cu"], init=r.get("pool"), slot_map=r["slots"], dfinal=r["dfinal"] if dfinal else None)
    ref, size = O.mamba2_scan_backward(*ins, **form), O.mamba2_scan_backward(*ins, **form, sizes=True)
    low = HALF["bf16"] * 1.02 if dt == "bf16" else 0.0
    slack = dict(dx=K + low, dBm=K + low * 2.0 ** -8, dCm=K + low * 2.0 ** -8)
    for name, p, q, s in zip(got._fields, got, ref, size):
        if p is None:
            assert name == "dinit" and sdt is None
            continue
        close(p, q, slack.get(name, K) * s, dt if name in ("dx", "dBm", "dCm", "ddt") else "f32", name)
    if sdt:
        assert torch.equal(before, v["pool"]), "the initial states are read only"


RAGGED = [1, 0, 63, 64, 65, 130, 2, 200]


@pytest.mark.parametrize("dt", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("n", [16, 64, 128])
def test_scan_shapes(d, n, dt):
    """Every compiled pair of d and n, ragged lengths around the chunk, three heads a group (a workgroup's heads do not divide it)."""
    check_scan(RAGGED, 6, 2, d, n, dt, "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("n", [16, 64, 128])
def test_backward_shapes(d, n, dt):
    check_backward(RAGGED, 6, 2, d, n, dt, "f32", dfinal=True)


@pytest.mark.parametrize("sdt,out_dt", [("bf16", "bf16"), ("f16", "bf16"), ("f32", "f32"), ("bf16", "f32"), (None, "bf16"), ("f32", "f16")])
def test_scan_types(sdt, out_dt):
    check_scan([70, 1, 129], 4, 1, 64, 128, "bf16", sdt, out_dt)


@pytest.mark.parametrize("G,H", [(1, 1), (1, 5), (4, 4), (8, 40)])
def test_heads_and_groups(G, H):
    check_scan([100, 33], H, G, 64, 64, "bf16", "f32")
    check_backward([100, 33], H, G, 64, 64, "bf16")


@pytest.mark.parametrize("lens", [[1], [2], [64], [128], [129], [1] * 70, [0, 0, 5, 0]])
def test_lengths(lens):
    check_scan(lens, 2, 1, 64, 128, "bf16", "f32")
    check_backward(lens, 2, 1, 64, 128, "bf16", "f32", dfinal=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_segments(dt):
    """Few heads and a long sequence among short ones: sequences cut into segments, forward and in reverse, with states and without."""
    check_scan([2300, 5, 0, 700], 2, 1, 64, 128, dt, "f32")
    check_backward([2300, 5, 0, 700], 2, 1, 64, 128, dt, "f32", dfinal=True)
    check_scan([1500], 3, 3, 16, 16, dt)
    check_backward([1500], 3, 3, 16, 16, dt)


def test_ragged_batch_in_segments():
    """Walks enough, of uneven lengths: the two longest sequences are cut, the others (of two segments too) are not."""
    lens = [1300, 1, 0, 200, 700, 512, 129]
    check_scan(lens, 64, 2, 64, 16, "bf16", "f32")
    check_backward(lens, 64, 2, 64, 16, "bf16", "f32", dfinal=True)
    check_scan(lens, 64, 2, 64, 16, "f32")


def test_more_sequences_than_a_grid_side():
    """70,000 sequences of one token: y and dx against the formula of one token."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    N, H, d, n = 70_000, 4, 16, 16
    gen = torch.Generator().manual_seed(5)
    x, Bm, Cm, dt = (torch.randn(*s, generator=gen).to(DEV) for s in ((N, H, d), (N, 1, n), (N, 1, n), (N, H)))
    A_log, dt_bias, D = (torch.randn(H, generator=gen).to(DEV) for _ in range(3))
    cu = torch.arange(N + 1, dtype=torch.int32, device=DEV)
    y = gdn.gdn_mamba2_scan(x, Bm, Cm, dt, A_log, dt_bias, D, cu)
    g = gdn.gdn_mamba2_scan_backward(torch.ones_like(x), x, Bm, Cm, dt, A_log, dt_bias, D, cu)
    torch.cuda.synchronize()
    x, Bm, Cm, dt, dt_bias, D = (t.double() for t in (x, Bm, Cm, dt, dt_bias, D))
    step = torch.nn.functional.softplus(dt + dt_bias)
    scale = step * (Bm * Cm).sum(-1)
    size = step * (Bm * Cm).abs().sum(-1) + D.abs()
    # n products, their sum, dt' (a logarithm and an exponential, 8 units), two products and a sum: under 32 roundings of the terms' sizes
    assert ((y - (scale + D)[..., None] * x).abs() <= 32 * 2.0 ** -24 * size[..., None] * x.abs()).all()
    assert ((g.dx - (scale + D)[..., None]).abs() <= 32 * 2.0 ** -24 * size[..., None]).all()


def test_tokens_apart():
    """Inputs that are slices of wider rows (the gaps hold NaN)."""
    check_scan([70, 61], 4, 2, 64, 128, "bf16", "f32", wide=24)
    check_backward([70, 61], 4, 2, 64, 128, "bf16", wide=24)
    check_scan([70, 61], 4, 2, 16, 64, "f32", "f32", wide=8)
    check_backward([70, 61], 4, 2, 16, 64, "f32", wide=8)


def test_padded_sequences():
    """Slots outside the pool: zero outputs and gradients, nothing touched; the other sequences as alone."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, r = make([80, 40, 150], 4, 2, 64, 128, "bf16", "f32")
    v["slots"] = torch.tensor([-1, 2, v["pool"].shape[0]], dtype=torch.int32, device=DEV)
    before = v["pool"].clone()
    y = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"])
    g = gdn.gdn_mamba2_scan_backward(v["dy"], *(v[k] for k in NAMES), v["cu"], pool=before, slot_map=v["slots"], dfinal=v["dfinal"])
    torch.cuda.synchronize()
    for t in (y, g.dx, g.dBm, g.dCm, g.ddt):
        assert not t[:80].any() and not t[120:].any() and t[80:120].any()
    assert not g.dinit[0].any() and not g.dinit[2].any() and g.dinit[1].any()
    keep = [i for i in range(before.shape[0]) if i != 2]
    assert torch.equal(before[keep], v["pool"][keep])
    ins = [r["dy"]] + [r[k] for k in NAMES]
    ref = O.mamba2_scan_backward(*ins, cu=r["cu"], init=r["pool"], slot_map=[-1, 2, 99], dfinal=r["dfinal"])
    size = O.mamba2_scan_backward(*ins, cu=r["cu"], init=r["pool"], slot_map=[-1, 2, 99], dfinal=r["dfinal"], sizes=True)
    for name, p, q, s in list(zip(g._fields, g, ref, size))[4:]:
        close(p, q, K * s, "f32", name)


def test_nonfinite_values_stay_in_their_sequence():
    """NaN and infinities reach nothing of the sequences beside theirs, nor earlier chunks of their own."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([64, 130, 64], 4, 2, 64, 128, "bf16", "f32")
    clean = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=v["pool"].clone(), slot_map=v["slots"])
    v["x"][64 + 70, 1, 3] = float("nan")
    v["Bm"][64 + 100, 0, 5] = float("inf")
    y = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"])
    assert torch.equal(y[:128], clean[:128]) and torch.equal(y[194:], clean[194:])
    assert y[64 + 128:194, 1, 3].isnan().all()


def test_strong_and_absent_decay():
    """Decays that underflow within a token or two, and steps so small that nothing decays or is written."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    for bias in (8.0, -30.0):
        v, r = make([150], 4, 2, 64, 64, "f32", "f32")
        v["dt_bias"].fill_(bias)
        r["dt_bias"] = np.full(4, bias)
        y = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=v["pool"].clone(), slot_map=v["slots"])
        g = gdn.gdn_mamba2_scan_backward(v["dy"], *(v[k] for k in NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"])
        ins, form = [r[k] for k in NAMES], dict(cu=r["cu"], init=r["pool"], slot_map=r["slots"])
        close(y, O.mamba2_scan(*ins, **form)[0], K * O.mamba2_scan(*ins, **form, sizes=True)[0], "f32", f"y at bias {bias}")
        ref = O.mamba2_scan_backward(r["dy"], *ins, **form)
        size = O.mamba2_scan_backward(r["dy"], *ins, **form, sizes=True)
        for name, p, q, s in zip(g._fields, g, ref, size):
            close(p, q, K * s, "f32", f"{name} at bias {bias}")


def test_split_call_and_decode_go_on():
    """Two calls over a split sequence, and a decode step after them, against one call: f32 states carry exactly."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([300], 4, 2, 64, 128, "f32", "f32")
    P = [v[k] for k in ("A_log", "dt_bias", "D")]
    cut = lambda a, b: [v[k][a:b].contiguous() for k in ("x", "Bm", "Cm", "dt")]  # noqa: E731
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    one = v["pool"].clone()
    y = gdn.gdn_mamba2_scan(*cut(0, 300), *P, cu(300), pool=one, slot_map=v["slots"])
    two = v["pool"].clone()
    ya = gdn.gdn_mamba2_scan(*cut(0, 173), *P, cu(173), pool=two, slot_map=v["slots"])
    yb = gdn.gdn_mamba2_scan(*cut(173, 299), *P, cu(126), pool=two, slot_map=v["slots"])
    yc = gdn.gdn_mamba2_decode_step(*cut(299, 300), *P, two, v["slots"])
    torch.testing.assert_close(torch.cat([ya, yb, yc]), y, rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(two, one, rtol=1e-4, atol=1e-4)


def test_far_slot():
    """A state that begins past 2^32 bytes of its pool."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([70], 128, 8, 64, 128, "bf16", "bf16")
    far = torch.empty((2300, 128, 64, 128), dtype=torch.bfloat16, device=DEV)  # 2 MiB a slot
    far[2299] = v["pool"][int(v["slots"][0])]
    y0 = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"])
    y1 = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=far, slot_map=torch.tensor([2299], dtype=torch.int32, device=DEV))
    assert torch.equal(y0, y1) and torch.equal(far[2299], v["pool"][int(v["slots"][0])])


def test_nothing_to_do():
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([0, 0], 2, 1, 16, 16, "f32", "f32")
    before = v["pool"].clone()
    y = gdn.gdn_mamba2_scan(*(v[k] for k in NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"])
    g = gdn.gdn_mamba2_scan_backward(v["dy"], *(v[k] for k in NAMES), v["cu"], pool=v["pool"], slot_map=v["slots"], dfinal=v["dfinal"])
    assert y.shape == (0, 2, 16) and torch.equal(before, v["pool"])
    assert torch.equal(g.dinit, v["dfinal"]) and not g.dA_log.any() and not g.ddt_bias.any() and not g.dD.any()
    none = v["cu"][:1]
    g = gdn.gdn_mamba2_scan_backward(v["dy"], *(v[k] for k in NAMES), none)
    assert not g.dA_log.any()


def test_equal_bits_streams_and_graph():
    """Equal calls give equal bits: again, on another stream, and from replays of a captured graph with other work between them."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([1300, 64, 9], 4, 2, 64, 128, "bf16", "f32")
    ins, first = [v[k] for k in NAMES] + [v["cu"]], v["pool"].clone()
    form = dict(pool=first, slot_map=v["slots"], dfinal=v["dfinal"])

    def fwd(pool, **kw):
        pool.copy_(first)
        return gdn.gdn_mamba2_scan(*ins, pool=pool, slot_map=v["slots"], **kw)
    y, ref = fwd(v["pool"]), gdn.gdn_mamba2_scan_backward(v["dy"], *ins, **form)
    end = v["pool"].clone()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, gdn.gdn_mamba2_scan_backward(v["dy"], *ins, **form)))
    s = torch.cuda.Stream()
    on = gdn.gdn_mamba2_scan_backward(v["dy"], *ins, **form, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, on))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = fwd(v["pool"])
        got = gdn.gdn_mamba2_scan_backward(v["dy"], *ins, **form)
    for _ in range(3):
        y2.zero_(), got.dx.zero_(), got.dA_log.fill_(3.0), v["pool"].fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(end, v["pool"]) and all(torch.equal(p, q) for p, q in zip(ref, got))
