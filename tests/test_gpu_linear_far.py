"""Linear attention and the norm and rotation of queries and keys where offsets pass 32 bits, and with rows behind the last
sequence."""
import pytest

from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def slopes(H):
    import torch
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H)


def test_slots_past_32_bits():
    """A pool of 5.4 GB: states in the last slots as in a pool of three."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    H, d, slots = 32, 128, 2600
    g = torch.Generator(device=DEV).manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    far, near = torch.zeros(slots, H, d, d, device=DEV), randn(3, H, d, d)
    assert far.numel() * 4 > 2 ** 32 and far.numel() > 2 ** 30
    far[slots - 3:] = near
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    q, k, v = (randn(130, H, d).bfloat16() for _ in range(3))
    one = lambda p, s: gdn.gdn_linear_decode_step(q[:2], k[:2], v[:2], slopes(H), p, ints(s))  # noqa: E731
    assert torch.equal(one(far, [slots - 1, slots - 3]), one(near, [2, 0]))
    many = lambda p, s: gdn.gdn_linear_scan(q, k, v, slopes(H), ints([0, 70, 130]), pool=p, slot_map=ints(s))  # noqa: E731
    assert torch.equal(many(far, [slots - 2, slots - 1]), many(near, [1, 2]))
    assert torch.equal(far[slots - 3:], near) and not far[:slots - 3].any()


def test_tokens_past_32_bits():
    """2^31 elements lie in front of the last sequence, which comes out as it does by itself (in other segments: what differs is
    the order of FP32 sums, so at most some values' last bit)."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    H, d, T, last = 128, 128, 131072 + 700, 700
    g = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn((T, H, d), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    assert (T - last) * H * d == 2 ** 31
    cu = torch.tensor([0, T - last, T], dtype=torch.int32, device=DEV)
    alone = torch.tensor([0, last], dtype=torch.int32, device=DEV)
    ends = lambda t: t[T - last:].contiguous()  # noqa: E731

    def close(a, b, what):
        off = (a.float() - b.float()).abs()
        assert (off <= 2.0 ** -7 * b.float().abs() + 1e-3 * b.float().abs().mean()).all(), what
        assert (off > 0).float().mean() < 0.01, what

    o = gdn.gdn_linear_scan(q, k, v, slopes(H), cu)
    close(o[T - last:], gdn.gdn_linear_scan(ends(q), ends(k), ends(v), slopes(H), alone), "o")
    got = gdn.gdn_linear_scan_backward(o, q, k, v, slopes(H), cu)
    want = gdn.gdn_linear_scan_backward(ends(o), ends(q), ends(k), ends(v), slopes(H), alone)
    for name, a, b in zip(got._fields, got, want):
        if a is not None:
            close(a[T - last:], b, name)


def test_rotation_past_32_bits():
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    T, H, d = 270000, 64, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k = (torch.randn((T, h, d), generator=g, device=DEV, dtype=torch.bfloat16) for h in (H, 1))
    assert (T - 50) * H * d > 2 ** 31
    w, pos = torch.ones(d, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    f = (1e4 ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)).float()
    y, yk = gdn.gdn_qk_norm_rope(q, k, w, w, pos, f)
    e, ek = gdn.gdn_qk_norm_rope(q[-50:].contiguous(), k[-50:].contiguous(), w, w, pos[-50:].contiguous(), f)
    assert torch.equal(y[-50:], e) and torch.equal(yk[-50:], ek)
    back = gdn.gdn_qk_norm_rope_backward(y, yk, q, k, w, w, pos, f)
    end = gdn.gdn_qk_norm_rope_backward(e, ek, q[-50:].contiguous(), k[-50:].contiguous(), w, w, pos[-50:].contiguous(), f)
    assert torch.equal(back.dq[-50:], end.dq) and torch.equal(back.dk[-50:], end.dk)


@pytest.mark.parametrize("front", [0, 200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_no_sequence(dt, front):
    """A batch with room behind its last sequence and in front of its first: those rows are not read (they are NaN) and outputs
    not written."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    T, used = 900 + front, 730 + front
    g = torch.Generator(device=DEV).manual_seed(4)
    q, k, v, do = (torch.randn((T, h, 64), generator=g, device=DEV).to(t) for h in (4, 2, 1, 4))
    for x in (q, k, v, do):
        x[:front] = x[used:] = float("nan")
    cu = torch.tensor([front, 700 + front, used], dtype=torch.int32, device=DEV)
    out = torch.full((T, 4, 64), 7.0, device=DEV, dtype=t)
    gdn.gdn_linear_scan(q, k, v, slopes(4), cu, out=out)
    assert (out[:front] == 7).all() and (out[used:] == 7).all()
    # the host counts with all rows, so the cuts differ: only the order of FP32 sums
    cut = lambda x: x[front:used].contiguous()  # noqa: E731
    want = gdn.gdn_linear_scan(cut(q), cut(k), cut(v), slopes(4), cu - front)
    got = gdn.gdn_linear_scan_backward(do, q, k, v, slopes(4), cu)
    ref = gdn.gdn_linear_scan_backward(cut(do), cut(q), cut(k), cut(v), slopes(4), cu - front)
    step = 2.0 ** -7 if dt == "bf16" else 2.0 ** -14
    for a, b in ((out, want), (got.dq, ref.dq), (got.dk, ref.dk), (got.dv, ref.dv)):
        a, b = a[front:used].float(), b.float()
        assert ((a - b).abs() <= step * (b.abs() + b.abs().mean())).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,lens,cuts", [(40, [1500] + [20] * 9 + [0, 700], (1, 1)), (300, [64, 900, 1, 65, 130], (1, 0)),
                                         (40, [6000] + [20] * 20 + [0, 700], (1, 0)), (32, [6000] + [33] * 7, (1, 1))])
def test_ragged_batches_in_segments(H, lens, cuts, dt):
    """Batches whose long sequences alone are cut, against one sequence a call."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator(device=DEV).manual_seed(5)
    T, d = sum(lens), 32
    q, k, v, do = (torch.randn((T, H, d), generator=g, device=DEV).to(t) for _ in range(4))
    start = torch.randn((len(lens), H, d, d), generator=g, device=DEV)
    dfinal = torch.randn((len(lens), H, d, d), generator=g, device=DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    pool, slots = start.clone(), ints(list(range(len(lens))))
    assert tuple(int(gdn._binding._linear_workspace(back, H, H, H, H, d, len(lens), T) > 0) for back in (False, True)) == cuts
    grads = gdn.gdn_linear_scan_backward(do, q, k, v, slopes(H), ints(cu), pool=start, slot_map=slots, dfinal=dfinal)
    o = gdn.gdn_linear_scan(q, k, v, slopes(H), ints(cu), pool=pool, slot_map=slots)
    step = {"bf16": 2.0 ** -7, "f32": 2.0 ** -14}

    def close(a, b, kind, what):
        a, b = a.float(), b.float()
        assert ((a - b).abs() <= step[kind] * (b.abs() + (b.abs().mean() if b.numel() else 0))).all(), what

    for s, n in enumerate(lens):
        at = slice(cu[s], cu[s + 1])
        one, p = ints([0, n]), start[s:s + 1].clone()
        x = [y[at].contiguous() for y in (do, q, k, v)]
        b = gdn.gdn_linear_scan_backward(*x, slopes(H), one, pool=p, slot_map=ints([0]), dfinal=dfinal[s:s + 1].contiguous())
        y = gdn.gdn_linear_scan(*x[1:], slopes(H), one, pool=p, slot_map=ints([0]))
        close(o[at], y, dt, f"o of {n}")
        close(pool[s], p[0], "f32", f"state of {n}")
        for name, u, w in zip(grads._fields, grads, b):
            close(u[s] if name == "dinit" else u[at], w[0] if name == "dinit" else w, "f32" if name == "dinit" else dt, f"{name} of {n}")


def test_two_graphs_of_one_workspace():
    """A forward and a backward call captured apart, with one workspace, replayed in turn and each twice in a row."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    g = torch.Generator(device=DEV).manual_seed(6)
    T, cu = 2100, torch.tensor([0, 1500, 1600, 2100], dtype=torch.int32, device=DEV)
    q, k, v, do = (torch.randn((T, h, 64), generator=g, device=DEV).bfloat16() for h in (4, 2, 1, 4))
    need = [gdn._binding._linear_workspace(back, 4, 4, 2, 1, 64, 3, T) for back in (False, True)]
    assert all(need)
    ws = torch.empty(max(need), dtype=torch.uint8, device=DEV)
    calls = [lambda: [gdn.gdn_linear_scan(q, k, v, slopes(4), cu, workspace=ws)],
             lambda: list(gdn.gdn_linear_scan_backward(do, q, k, v, slopes(4), cu, workspace=ws)[:3])]
    want = [[t.clone() for t in f()] for f in calls]
    graphs, outs = [], []
    for f in calls:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f()
        torch.cuda.current_stream().wait_stream(s)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(f())
    for turn, i in enumerate((0, 1, 0, 1, 1, 0, 0)):
        for t in outs[i]:
            t.fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), turn
        assert all(torch.equal(a, b) for f, w in zip(calls, want) for a, b in zip(f(), w)), turn


def test_expanded_inputs_on_another_stream():
    """Copies and outputs that the call makes belong to the stream it runs on, also when memory is used again at once."""
    import torch
    import gated_deltanet_state_gdn_amd as gdn
    g = torch.Generator(device=DEV).manual_seed(7)
    T, cu = 1400, torch.tensor([0, 900, 1400], dtype=torch.int32, device=DEV)
    row = torch.randn((1, 4, 64), generator=g, device=DEV).bfloat16()
    q, k, v = (torch.randn((T, 4, 64), generator=g, device=DEV).bfloat16() for _ in range(3))
    want = gdn.gdn_linear_scan_backward(row.expand(T, 4, 64).contiguous(), q, k, v, slopes(4), cu)
    decay = slopes(4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(4):
        got = gdn.gdn_linear_scan_backward(row.expand(T, 4, 64), q, k, v, decay, cu, stream=s)
        junk = [torch.full((T, 4, 64), 3.0, device=DEV, dtype=torch.bfloat16) for _ in range(4)]
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
        del junk
