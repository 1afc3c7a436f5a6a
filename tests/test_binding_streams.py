"""Where the binding takes its own buffers from, when a call is given a stream that is not the current one: from that stream's memory,
never from the current stream's, whose freed blocks may still be in use by work queued there.  On the host, with the library and
torch's streams stood in for."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import gated_deltanet_state_gdn_amd as gdn
from gated_deltanet_state_gdn_amd import _binding as bd

T, H, d = 6, 2, 16
NEW = ("aten.empty.memory_format", "aten.new_empty.default", "aten.clone.default", "aten._to_copy.default")


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Library:
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("workspace_bytes") else 0


class Allocations(TorchDispatchMode):
    def __init__(self, where):
        super().__init__()
        self.where, self.seen = where, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if str(func) in NEW:
            self.seen.append((str(func), self.where["now"]))
        return func(*args, **(kwargs or {}))


def calls():
    z = torch.zeros
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    tok, seqs = z(T, H, d), ints(0, 2, T)
    head, states, slots = z(H), z(9, H, d, d), ints(2, 0)
    one = z(2, H, d)
    gates = (z(2, H), z(2, H), head, head)
    ring, m2 = gdn.new_ring(9, H, H, 4, d, d, torch.bfloat16, "cpu"), gdn.new_m2_ring(9, H, H, 4, d, d, torch.bfloat16, "cpu")
    m2_in = dict(x=tok, Bm=tok, Cm=tok, dt=z(T, H), A_log=head, dt_bias=head, D=head, cu_seqlens=seqs)
    x, w = z(4, 8), z(8)
    qk = dict(q=tok, k=tok, q_weight=z(d), k_weight=z(d), positions=z(T, dtype=torch.int32), inv_freq=z(8))
    per_window = lambda t: t[:, None].expand(2, 1, *t.shape[1:]).contiguous()  # noqa: E731
    wone, wgates = per_window(one), (per_window(gates[0]), per_window(gates[1]), head, head)
    row = z(1, H, d).expand(T, H, d)
    return {
        "decode": lambda **s: gdn.gdn_decode_step(one, one, one, *gates, states, slots, **s),
        "spec": lambda **s: gdn.gdn_spec_decode(wone, wone, wone, *wgates, states, slots, slots[:, None].contiguous(), **s),
        "copy": lambda **s: gdn.gdn_copy_state_blocks([states], slots, slots, **s),
        "prefill": lambda **s: gdn.gdn_chunk_prefill(tok, tok, tok, z(T, H), z(T, H), head, head, states, slots, seqs, **s),
        "replay": lambda **s: gdn.gdn_replay_decode(wone, wone, wone, *wgates, states, slots, ring, **s),
        "mamba2": lambda **s: gdn.gdn_mamba2_decode_step(one, one, one, z(2, H), head, head, head, states, slots, **s),
        "mamba2_replay": lambda **s: gdn.gdn_mamba2_replay_decode(wone, wone, wone, z(2, 1, H), head, head, head, states, slots, m2, **s),
        "mamba2_scan": lambda **s: gdn.gdn_mamba2_scan(**m2_in, **s),
        "mamba2_scan_expanded": lambda **s: gdn.gdn_mamba2_scan(**dict(m2_in, x=row), **s),
        "mamba2_scan_backward": lambda **s: gdn.gdn_mamba2_scan_backward(tok, **m2_in, pool=states, slot_map=slots, **s),
        "norm": lambda **s: gdn.gdn_layer_norm(x, w, save_stats=True, **s),
        "norm_backward": lambda **s: gdn.gdn_layer_norm_backward(x, x, w, z(4, 1), z(4, 1), bias=w, gate=x, **s),
        "linear_step": lambda **s: gdn.gdn_linear_decode_step(one, one, one, head, states, slots, **s),
        "linear_scan": lambda **s: gdn.gdn_linear_scan(tok, tok, tok, head, seqs, **s),
        "linear_scan_backward": lambda **s: gdn.gdn_linear_scan_backward(row, tok, tok, tok, head, seqs, pool=states, slot_map=slots, **s),
        "qk": lambda **s: gdn.gdn_qk_norm_rope(**qk, **s),
        "qk_backward": lambda **s: gdn.gdn_qk_norm_rope_backward(tok, tok, **qk, **s),
    }


@pytest.fixture
def streams(monkeypatch):
    """What stands in for streams; `now` is the one whose memory is taken, `used` the streams that tensors were marked for."""
    state = {"now": 0, "used": [], "tables": []}  # a host table's upload is no allocation here

    @contextlib.contextmanager
    def inside(s):
        before, state["now"] = state["now"], s.cuda_stream
        yield
        state["now"] = before

    @contextlib.contextmanager
    def launch(stream, *tensors):
        yield bd._stream(stream)

    table = bd.make_state_table
    monkeypatch.setattr(bd, "make_state_table", lambda *a: (state["tables"].append(("table", state["now"])), table(*a))[1])
    monkeypatch.setattr(bd, "lib", lambda: Library())
    monkeypatch.setattr(bd, "_on_gpu", lambda stream, *t: bd._stream(stream), raising=False)
    monkeypatch.setattr(bd, "_launch_on", launch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(state["now"]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda *a: state["now"], raising=False)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, **k: Stream(handle))
    monkeypatch.setattr(torch.cuda, "stream", inside)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state["used"].append((t.untyped_storage().data_ptr(), s.cuda_stream)))
    for f in (bd._scan_workspace, bd._linear_workspace):
        f.cache_clear()
    yield state
    for f in (bd._scan_workspace, bd._linear_workspace):
        f.cache_clear()


def results(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("current,given", [(0, 77), (5, 77), (5, 0)])
def test_buffers_come_from_the_call_s_stream(streams, name, current, given):
    call = calls()[name]
    streams["now"] = current
    with Allocations(streams) as log:
        out = call(stream=given)
    seen = log.seen + streams["tables"]
    assert seen and all(where == given for _, where in seen), seen
    assert streams["now"] == current
    marked = {p for p, s in streams["used"] if s == current}
    assert all(t.untyped_storage().data_ptr() in marked for t in results(out)), "results are used on the current stream"


@pytest.mark.parametrize("name", list(calls()))
def test_the_current_stream_needs_nothing(streams, name):
    call = calls()[name]
    for given in (None, 5):
        streams["now"] = 5
        with Allocations(streams) as log:
            call(stream=given)
        assert all(where == 5 for _, where in log.seen + streams["tables"]) and not streams["used"]
