"""GPU parity of gdn_linear_scan, gdn_linear_scan_backward and gdn_linear_decode_step against the float64 oracle.

Tolerances count roundings, as multiples of the sum of the terms' absolute values ("sizes", from the oracle).  In FP32 a term
passes a dozen roundings (products, a decay from a table rounded once, the scale), sums add at most 128 values a chunk in any
order, and a state takes two more roundings a chunk: K = 512 steps of 2^-24 cover sequences of up to some 100 chunks.  With bf16
inputs and outputs the state and the weighted products enter the output in two bf16 terms, whose rest is at most 2^-16 of each.
The output itself is off by half a step of its type.  Decays below 2^-126 may count as zero, so a term is off by up to that times
its factors, which stay below 2^10.
"""
import numpy as np
import pytest

import oracle as O

from gpu_util import DEV, require_gpu, say, torch_dtype

pytestmark = pytest.mark.gpu
K = 512 * 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -116, "bf16": 2.0 ** -116, "f16": 2.0 ** -25}
TWO_TERMS = 1.02 * 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def slopes(H):
    return -np.exp2(-8.0 * np.arange(1, H + 1) / H).astype(np.float32)


def make(lens, heads, d, dt, sdt=None, seed=1, wide=0, decay=None):
    """Device tensors and their float64 values; wide: q, k and v are slices of wider rows (by that many elements, NaN)."""
    import torch
    H, Hq, Hk, Hv = heads
    T, N = sum(lens), len(lens)
    g = torch.Generator().manual_seed(seed)
    dev = {}
    for name, h in (("q", Hq), ("k", Hk), ("v", Hv)):
        x = torch.randn((T, h, d), generator=g).to(torch_dtype(dt)).to(DEV)
        if wide:
            row = torch.full((T, h * d + wide), float("nan"), dtype=x.dtype, device=DEV)
            row[:, :-wide] = x.reshape(T, -1)
            x = row[:, :-wide].unflatten(1, (h, d))
        dev[name] = x
    dev["g"] = torch.from_numpy(np.asarray(slopes(H) if decay is None else decay, np.float32)).to(DEV)
    dev["do"] = torch.randn((T, H, d), generator=g).mul(0.1).to(torch_dtype(dt)).to(DEV)
    dev["dfinal"] = torch.randn((N, H, d, d), generator=g).mul(0.1).to(DEV)
    dev["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    if sdt is not None:
        dev["pool"] = torch.randn((N + 2, H, d, d), generator=g).to(torch_dtype(sdt)).to(DEV)
        dev["slots"] = torch.randperm(N + 2, generator=g)[:N].to(torch.int32).to(DEV)
    ref = {k: v.double().cpu().numpy() for k, v in dev.items() if k not in ("cu", "slots")}
    ref["cu"] = dev["cu"].cpu().numpy()
    ref["slots"] = dev["slots"].cpu().numpy() if sdt is not None else None
    return dev, ref


def close(got, ref, slack, dt, what):
    got = got.double().cpu().numpy()
    err, bound = np.abs(got - ref), HALF[dt] * np.abs(ref) + slack + TINY[dt]
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    worst = (err / bound).max() if err.size else 0.0
    assert worst <= 1.0, f"{what}: {np.argwhere(err > bound)[:4].tolist()} off by up to {worst:.2f} bounds"


def ins(r):
    return [r[k] for k in ("q", "k", "v", "g")]


def check_scan(lens, heads, d, dt, sdt=None, out_dt=None, scale=None, **how):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    say(f"linear scan lens={lens} heads={heads} d={d} {dt} state={sdt} out={out_dt} scale={scale} {how}")
    v, r = make(lens, heads, d, dt, sdt, **how)
    before = v["pool"].clone() if sdt else None
    o = gdn.gdn_linear_scan(v["q"], v["k"], v["v"], v["g"], v["cu"], pool=v.get("pool"), slot_map=v.get("slots"), scale=scale,
                            out_dtype=torch_dtype(out_dt or dt))
    torch.cuda.synchronize()
    form = dict(cu=r["cu"], init=r.get("pool"), slot_map=r["slots"], scale=scale)
    o_r, f_r = O.linear_scan(*ins(r), **form)
    o_s, f_s = O.linear_scan(*ins(r), **form, sizes=True)
    low = TWO_TERMS if dt == "bf16" and (out_dt or dt) == "bf16" else 0.0
    close(o, o_r, (K + low) * o_s, out_dt or dt, "o")
    if sdt:
        used = [s for s, n in enumerate(lens) if n > 0]
        slots = r["slots"][used]
        close(v["pool"][torch.as_tensor(slots).long().to(DEV)], f_r[used], K * f_s[used], sdt, "final states")
        rest = [i for i in range(before.shape[0]) if i not in slots]
        assert torch.equal(v["pool"][rest], before[rest]), "slots that no token reached"


def check_backward(lens, heads, d, dt, sdt=None, dfinal=False, scale=None, **how):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    say(f"linear scan backward lens={lens} heads={heads} d={d} {dt} state={sdt} dfinal={dfinal} scale={scale} {how}")
    v, r = make(lens, heads, d, dt, sdt, **how)
    before = v["pool"].clone() if sdt else None
    got = gdn.gdn_linear_scan_backward(v["do"], v["q"], v["k"], v["v"], v["g"], v["cu"], pool=v.get("pool"), slot_map=v.get("slots"),
                                       dfinal=v["dfinal"] if dfinal else None, scale=scale)
    torch.cuda.synchronize()
    form = dict(cu=r["cu"], init=r.get("pool"), slot_map=r["slots"], dfinal=r["dfinal"] if dfinal else None, scale=scale)
    ref, size = O.linear_scan_backward(r["do"], *ins(r), **form), O.linear_scan_backward(r["do"], *ins(r), **form, sizes=True)
    low = TWO_TERMS if dt == "bf16" else 0.0
    for name, p, q, s in zip(got._fields, got, ref, size):
        if p is None:
            assert name == "dinit" and sdt is None
            continue
        close(p, q, (K + (0.0 if name == "dinit" else low)) * s, "f32" if name == "dinit" else dt, name)
    if sdt:
        assert torch.equal(before, v["pool"]), "the initial states are read only"


SCANS = [
    # lens, (H, Hq, Hk, Hv), d, dtype, state
    ([1], (1, 1, 1, 1), 16, "bf16", None),
    ([64], (2, 2, 2, 2), 32, "bf16", "f32"),
    ([65, 63, 1, 0, 130], (2, 2, 2, 2), 64, "bf16", "f32"),
    ([37, 64, 129], (4, 2, 2, 4), 128, "bf16", "bf16"),
    ([200, 5], (8, 8, 2, 4), 64, "bf16", "f16"),
    ([0, 70, 0], (6, 1, 3, 6), 32, "bf16", "bf16"),
    ([700], (2, 2, 2, 2), 128, "bf16", "f32"),       # cut into segments
    ([1300, 3, 900, 0, 64], (3, 3, 1, 1), 64, "bf16", "f32"),
    ([1000, 1, 257], (2, 1, 2, 2), 16, "bf16", None),
    ([1], (2, 2, 2, 2), 128, "f32", "f32"),
    ([65, 63, 1, 0, 130], (2, 1, 2, 2), 64, "f32", "f32"),
    ([700, 90], (2, 2, 2, 2), 32, "f32", "f32"),
    ([130, 64], (4, 4, 1, 1), 128, "f32", "bf16"),
    ([75, 600], (2, 2, 1, 2), 16, "f32", None),
    ([65, 129, 31], (2, 2, 2, 2), 64, "f16", "f16"),
    ([640, 17], (2, 1, 1, 2), 128, "f16", "f32"),
]


@pytest.mark.parametrize("lens,heads,d,dt,sdt", SCANS)
def test_scan(lens, heads, d, dt, sdt):
    check_scan(lens, heads, d, dt, sdt)


@pytest.mark.parametrize("lens,heads,d,dt,sdt", SCANS)
@pytest.mark.parametrize("dfinal", [False, True])
def test_backward(lens, heads, d, dt, sdt, dfinal):
    check_backward(lens, heads, d, dt, sdt, dfinal)


@pytest.mark.parametrize("dt,out_dt", [("bf16", "f32"), ("f16", "bf16"), ("f32", "f16")])
def test_scan_output_types(dt, out_dt):
    check_scan([100, 33], (2, 2, 1, 2), 64, dt, "f32", out_dt, scale=0.37)


@pytest.mark.parametrize("d", [16, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_of_slices_of_wider_rows(d, dt):
    """What lies between the tokens is NaN, and is not read."""
    check_scan([70, 0, 129], (2, 2, 1, 2), d, dt, "f32", wide=8)
    check_backward([70, 0, 129], (2, 2, 1, 2), d, dt, "f32", True, scale=1.25, wide=24)


@pytest.mark.parametrize("decay", [[0.0, 0.0], [-float("inf"), -1e30], [-30.0, -88.0], [-1e-6, 0.003]])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_at_the_ends_of_the_decays(decay, dt):
    """No decay, none of the past kept, underflow inside a chunk, hardly any decay and a little growth."""
    check_scan([200, 66], (2, 2, 2, 2), 32, dt, "f32", decay=decay)
    check_backward([200, 66], (2, 2, 2, 2), 32, dt, "f32", True, decay=decay)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_padded_sequences(dt):
    """Slots outside the pool: zero outputs and gradients, no slot touched; the sequences beside them as ever."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    lens = [66, 700, 0, 40]
    for bad in ([-1, None, 99, None], [None, 6, None, -5]):
        v, r = make(lens, (2, 2, 1, 2), 64, dt, "f32", seed=4)
        slots = v["slots"].clone()
        for i, b in enumerate(bad):
            if b is not None:
                slots[i] = b
        r["slots"] = slots.cpu().numpy()
        before = v["pool"].clone()
        o = gdn.gdn_linear_scan(v["q"], v["k"], v["v"], v["g"], v["cu"], pool=v["pool"], slot_map=slots)
        form = dict(cu=r["cu"], init=r["pool"], slot_map=r["slots"])
        low = TWO_TERMS if dt == "bf16" else 0.0
        close(o, O.linear_scan(*ins(r), **form)[0], (K + low) * O.linear_scan(*ins(r), **form, sizes=True)[0], dt, "o")
        got = gdn.gdn_linear_scan_backward(v["do"], v["q"], v["k"], v["v"], v["g"], v["cu"], pool=before, slot_map=slots, dfinal=v["dfinal"])
        ref = O.linear_scan_backward(r["do"], *ins(r), **form, dfinal=r["dfinal"])
        size = O.linear_scan_backward(r["do"], *ins(r), **form, dfinal=r["dfinal"], sizes=True)
        for name, p, q, s in zip(got._fields, got, ref, size):
            close(p, q, (K + low) * s, "f32" if name == "dinit" else dt, name)
        for i, b in enumerate(bad):
            if b is not None:
                at = slice(int(r["cu"][i]), int(r["cu"][i + 1]))
                assert not o[at].any() and not got.dq[at].any() and not got.dv[at].any() and not got.dinit[i].any()
        rest = [i for i in range(before.shape[0]) if i not in [s for s, n in zip(r["slots"], lens) if n]]
        assert torch.equal(v["pool"][rest], before[rest])


def test_scan_without_tokens():
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, r = make([0, 0], (2, 2, 2, 2), 32, "bf16", "f32")
    before = v["pool"].clone()
    o = gdn.gdn_linear_scan(v["q"], v["k"], v["v"], v["g"], v["cu"], pool=v["pool"], slot_map=v["slots"])
    assert o.shape == (0, 2, 32) and torch.equal(before, v["pool"])
    g = gdn.gdn_linear_scan_backward(v["do"], v["q"], v["k"], v["v"], v["g"], v["cu"], pool=v["pool"], slot_map=v["slots"], dfinal=v["dfinal"])
    assert torch.equal(g.dinit, v["dfinal"]) and g.dq.shape == (0, 2, 32)
    g = gdn.gdn_linear_scan_backward(v["do"], v["q"], v["k"], v["v"], v["g"], v["cu"][:1], pool=v["pool"], slot_map=v["slots"][:0])
    assert g.dinit.shape == (0, 2, 32, 32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_sequence_does_not_see_its_neighbours(dt):
    """A NaN in one sequence stays there, in its state too."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([70, 30, 90], (2, 2, 2, 2), 64, dt, "f32")
    clean = v["pool"].clone()
    want = gdn.gdn_linear_scan(v["q"], v["k"], v["v"], v["g"], v["cu"], pool=clean, slot_map=v["slots"])
    for name in ("q", "k", "v"):
        pool, x = v["pool"].clone(), dict(v)
        x[name] = v[name].clone()
        x[name][70:100] = float("nan")
        o = gdn.gdn_linear_scan(x["q"], x["k"], x["v"], v["g"], v["cu"], pool=pool, slot_map=v["slots"])
        assert torch.equal(o[:70], want[:70]) and torch.equal(o[100:], want[100:]) and o[70:100].isnan().all()
        for s in (0, 2):
            slot = int(v["slots"][s])
            assert torch.equal(pool[slot], clean[slot])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_goes_on_from_its_state(dt):
    """Two calls over halves of a prompt, and single tokens behind them, are one call: the same terms, in other chunks."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    lens, cut = [300, 77], [100, 64]
    v, r = make(lens, (4, 2, 4, 2), 64, dt, "f32", seed=9)
    pool = v["pool"].clone()
    cu = r["cu"]
    one = torch.cat([torch.arange(cu[s], cu[s] + cut[s]) for s in range(2)]).to(DEV)
    two = torch.cat([torch.arange(cu[s] + cut[s], cu[s + 1] - 1) for s in range(2)]).to(DEV)
    last = torch.tensor([cu[1] - 1, cu[2] - 1], device=DEV)
    outs = torch.zeros((377, 4, 64), dtype=v["q"].dtype, device=DEV)
    for at, sizes in ((one, cut), (two, [n - c - 1 for n, c in zip(lens, cut)])):
        c = torch.tensor([0, sizes[0], sum(sizes)], dtype=torch.int32, device=DEV)
        outs[at] = gdn.gdn_linear_scan(v["q"][at], v["k"][at], v["v"][at], v["g"], c, pool=pool, slot_map=v["slots"])
    outs[last] = gdn.gdn_linear_decode_step(v["q"][last], v["k"][last], v["v"][last], v["g"], pool, v["slots"], out_dtype=outs.dtype)
    form = dict(cu=cu, init=r["pool"], slot_map=r["slots"])
    (o, f), (os, fs) = O.linear_scan(*ins(r), **form), O.linear_scan(*ins(r), **form, sizes=True)
    close(outs, o, (K + (TWO_TERMS if dt == "bf16" else 0)) * os, dt, "o")
    close(pool[v["slots"].long()], f, K * fs, "f32", "states")


# ------------------------------------------------------------------ single tokens
@pytest.mark.parametrize("B,heads,d,dt,sdt", [
    (1, (1, 1, 1, 1), 16, "bf16", "f32"), (3, (4, 2, 2, 4), 128, "bf16", "f32"), (5, (6, 3, 1, 2), 64, "bf16", "bf16"),
    (2, (2, 2, 2, 2), 32, "f32", "f16"), (40, (16, 16, 4, 4), 128, "bf16", "f32"), (40, (16, 16, 16, 16), 128, "f16", "bf16"),
    (33, (17, 17, 17, 17), 64, "f32", "f16"), (17, (32, 1, 32, 8), 32, "f16", "f32"), (70, (8, 8, 8, 8), 16, "bf16", "bf16"),
    (64, (16, 16, 16, 16), 128, "f32", "f32"),
])
def test_step(B, heads, d, dt, sdt):
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    say(f"linear step B={B} heads={heads} d={d} {dt} state={sdt}")
    for out_dt, wide in ((None, 0), (dt, 8)):
        v, r = make([1] * B, heads, d, dt, sdt, seed=2, wide=wide)
        slots = v["slots"].clone()
        if B > 2:
            slots[1], slots[B - 1] = -1, B + 2
        live = [b for b in range(B) if 0 <= int(slots[b]) < B + 2]
        before = v["pool"].clone()
        o = gdn.gdn_linear_decode_step(v["q"], v["k"], v["v"], v["g"], v["pool"], slots, scale=0.3,
                                       out_dtype=torch_dtype(out_dt) if out_dt else None)
        assert o.dtype == (torch_dtype(out_dt) if out_dt else torch.float32)
        torch.cuda.synchronize()
        states = r["pool"][slots.cpu().numpy()[live]]
        q, k, x, g = (r[n] if n == "g" else r[n][live] for n in ("q", "k", "v", "g"))
        o_r, s_r = O.linear_step(q, k, x, g, states, 0.3)
        o_s, s_s = O.linear_step(np.abs(q), np.abs(k), np.abs(x), g, np.abs(states), 0.3)
        close(o[live], o_r, K * o_s, out_dt or "f32", "o")
        close(v["pool"][slots[live].long()], s_r, K * s_s, sdt, "states")
        rest = [i for i in range(B + 2) if i not in slots[live].tolist()]
        assert torch.equal(v["pool"][rest], before[rest])
        assert not o[[b for b in range(B) if b not in live]].any()


# ------------------------------------------------------------------ streams and graphs
def test_equal_calls_give_equal_bits_and_captured_ones_too():
    """Scan, its backward and single tokens, replayed from a graph with eager work between: every replay as the eager call.  Two
    captured calls share one workspace, as they run one after the other."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([900, 130, 0, 64], (4, 4, 2, 1), 64, "bf16", "f32")
    start = v["pool"].clone()
    one = {k: v[k][:4].contiguous() for k in ("q", "k", "v")}
    size = max(gdn._binding._linear_workspace(b, 4, 4, 2, 1, 64, 4, 1094) for b in (False, True))
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def work():
        v["pool"].copy_(start)
        g = gdn.gdn_linear_scan_backward(v["do"], v["q"], v["k"], v["v"], v["g"], v["cu"], pool=v["pool"], slot_map=v["slots"],
                                         dfinal=v["dfinal"], workspace=ws)
        o = gdn.gdn_linear_scan(v["q"], v["k"], v["v"], v["g"], v["cu"], pool=v["pool"], slot_map=v["slots"], workspace=ws)
        y = gdn.gdn_linear_decode_step(one["q"], one["k"], one["v"], v["g"], v["pool"], v["slots"])
        return [*g, o, y]

    want = [t.clone() for t in work()] + [v["pool"].clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for turn in range(4):
        for t in outs:
            t.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs + [v["pool"]], want):
            assert torch.equal(a, b), turn
        again = work()
        torch.cuda.synchronize()
        for a, b in zip(again, want):
            assert torch.equal(a, b), turn


def test_on_another_stream():
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([700, 130], (2, 2, 1, 2), 64, "bf16", "f32")
    pool = v["pool"].clone()
    want = gdn.gdn_linear_scan(v["q"], v["k"], v["v"], v["g"], v["cu"], pool=pool, slot_map=v["slots"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        p = v["pool"].clone()
        torch.cuda.synchronize()
        o = gdn.gdn_linear_scan(v["q"], v["k"], v["v"], v["g"], v["cu"], pool=p, slot_map=v["slots"], stream=handle)
        s.synchronize()
        assert torch.equal(o, want) and torch.equal(p, pool)


def test_expanded_inputs_are_copied():
    """A gradient behind a sum over tokens is one row for all of them."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    v, _ = make([66, 65], (2, 2, 2, 2), 64, "bf16")
    do, q = v["do"][:1].expand(131, 2, 64), v["q"][:1].expand(131, 2, 64)
    a = gdn.gdn_linear_scan_backward(do, q, v["k"], v["v"], v["g"], v["cu"])
    b = gdn.gdn_linear_scan_backward(do.contiguous(), q.contiguous(), v["k"], v["v"], v["g"], v["cu"])
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
