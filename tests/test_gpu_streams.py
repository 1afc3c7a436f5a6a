"""Calls on a stream that is not the current one, beside work queued on the current stream that still uses memory it has given up."""
import pytest
import torch

import gated_deltanet_state_gdn_amd as gdn
from gpu_util import DEV, require_gpu, say

pytestmark = pytest.mark.gpu
T, H, d = 1500, 4, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def calls():
    g = torch.Generator(device=DEV).manual_seed(8)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    tok = lambda h=H: randn(T, h, d).bfloat16()  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    cu, decay = ints([0, 900, T]), -torch.exp2(-2.0 * torch.arange(1, H + 1, device=DEV))
    q, k, v, do, rows = tok(), tok(), tok(), tok(), randn(T, H * d).bfloat16()
    w, head, wide = randn(d), randn(H), randn(H * d)
    pos, freq = torch.arange(T, dtype=torch.int32, device=DEV), (1e4 ** (-torch.arange(0, d, 2, device=DEV) / d)).float()
    stat = gdn.gdn_layer_norm(rows, wide, save_stats=True)[1:]
    pool, slots = randn(T, H, d, d), torch.arange(T, dtype=torch.int32, device=DEV)
    states, two = randn(2, H, d, d), ints([0, 1])
    dt = randn(T, H).bfloat16()
    m2 = (q, k, v, dt, head * 0.1, head * 0.1, head)
    return {
        "linear_scan": lambda **s: gdn.gdn_linear_scan(q, k, v, decay, cu, **s),
        "linear_scan_backward": lambda **s: gdn.gdn_linear_scan_backward(do, q, k, v, decay, cu, pool=states, slot_map=two, **s),
        "linear_step": lambda **s: gdn.gdn_linear_decode_step(q, k, v, decay, pool.clone() if not s else pool, slots, **s),
        "qk": lambda **s: gdn.gdn_qk_norm_rope(q, k, w, w, pos, freq, **s),
        "qk_backward": lambda **s: gdn.gdn_qk_norm_rope_backward(do, v, q, k, w, w, pos, freq, **s),
        "norm": lambda **s: gdn.gdn_layer_norm(rows, wide, **s),
        "norm_backward": lambda **s: gdn.gdn_layer_norm_backward(rows, rows, wide, *stat, **s),
        "mamba2_scan": lambda **s: gdn.gdn_mamba2_scan(*m2, cu, **s),
        "mamba2_scan_backward": lambda **s: gdn.gdn_mamba2_scan_backward(do, *m2, cu, **s),
    }


def tensors(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


class Delay:
    """Some ten milliseconds of products on the current stream, into memory of their own."""

    def __init__(self):
        self.a, self.b = torch.randn(4096, 4096, device=DEV).bfloat16(), torch.empty(4096, 4096, device=DEV, dtype=torch.bfloat16)

    def __call__(self):
        for _ in range(60):
            torch.mm(self.a, self.a, out=self.b)


@pytest.mark.parametrize("name", ["linear_scan", "linear_scan_backward", "linear_step", "qk", "qk_backward", "norm", "norm_backward",
                                  "mamba2_scan", "mamba2_scan_backward"])
def test_beside_queued_work(name):
    say(f"beside queued work: {name}")
    call, delay = calls()[name], Delay()
    want = [t.clone() for t in tensors(call())]
    sizes = [t.nbytes for t in want] + [1 << 20, 1 << 22, 1 << 23, 1 << 24, 1 << 25]  # results and workspaces
    delay()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    # blocks that are given up while work on them is still in the current stream's queue
    temporary = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes]
    after = [torch.empty_like(t) for t in temporary]
    delay()
    for t, y in zip(temporary, after):
        torch.add(t, 1, out=y)
    del temporary, t
    got = call(stream=s)
    s.synchronize()
    first = [t.clone() for t in tensors(got)]
    torch.cuda.synchronize()
    assert all((y == 8).all() for y in after), "memory in use was written"
    assert all(torch.equal(a, b) for a, b in zip(first, want))

    if name == "linear_step":  # its states have gone on
        return
    # results that are given up while work on the current stream still reads them
    kept = [torch.empty_like(t) for t in want]
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    delay()
    for t, y in zip(tensors(got), kept):
        y.copy_(t)
    del got, t
    for _ in range(3):
        with torch.cuda.stream(s):
            junk = [torch.full((t.nbytes,), 99, dtype=torch.uint8, device=DEV) for t in want]
        call(stream=s)
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want)), "a result in use was written"


@pytest.mark.parametrize("name", ["linear_scan", "linear_scan_backward", "qk", "qk_backward", "norm_backward", "mamba2_scan_backward"])
def test_captured_on_a_second_stream(name):
    """A graph whose call runs on a stream beside the capturing one, and joins it: every replay as the eager call."""
    say(f"captured on a second stream: {name}")
    call = calls()[name]
    want = [t.clone() for t in tensors(call())]
    side = torch.cuda.Stream()
    call(stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        outs = tensors(call(stream=side))
        torch.cuda.current_stream().wait_stream(side)
    for turn in range(4):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), turn
        assert all(torch.equal(a, b) for a, b in zip(tensors(call()), want)), turn
