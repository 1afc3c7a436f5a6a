"""The example block: the norm, the scan, their gradients and the decode step
together, against the same block written out token by token in 64 bits."""
import pytest
import torch
import torch.nn.functional as F

from examples.mamba2_block import Mamba2Block

pytestmark = pytest.mark.gpu

# Everything is FP32 here.  An output passes five stages (norm, product, scan,
# norm, product) and a gradient those and their mirrors, ten roundings of sums
# of up to 256 terms each: 10 * sqrt(256) * 2^-24 of the whole, times 3 for the
# factors between them (the norms divide by about 1, decays are below 1).
TOL = 10 * 16 * 3 * 2.0 ** -24


def reference(p, b, x, cu):
    u = F.layer_norm(x, x.shape[1:], p["norm_w"], p["norm_b"], 1e-5)
    rows = u @ p["w_in"].T
    z, xs, Bm, Cm, dt = torch.split(rows[:, :sum(b.parts)], b.parts, dim=1)
    H, d, G, n = b.H, b.d, b.G, b.n
    xs, Bm, Cm = xs.unflatten(1, (H, d)), Bm.unflatten(1, (G, n)), Cm.unflatten(1, (G, n))
    dts = F.softplus(dt + p["dt_bias"])
    ys = []
    for lo, hi in zip(cu[:-1], cu[1:]):
        S = x.new_zeros(H, d, n)
        for t in range(lo, hi):
            Bh, Ch = (v[t].repeat_interleave(H // G, 0) for v in (Bm, Cm))
            S = torch.exp(-torch.exp(p["A_log"]) * dts[t])[:, None, None] * S
            S = S + dts[t][:, None, None] * xs[t][:, :, None] * Bh[:, None, :]
            ys.append((S * Ch[:, None, :]).sum(-1) + p["D"][:, None] * xs[t])
    y = (torch.stack(ys).flatten(1) * F.silu(z)).unflatten(1, (G, -1))
    y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-5)
    return x + (y.flatten(1) * p["gate_w"]) @ p["w_out"].T


def close(name, a, b):
    err = (a.detach().double().cpu() - b).norm() / b.norm()
    assert err <= TOL, f"{name}: {err:.2e} > {TOL:.2e}"


def make():
    torch.manual_seed(7)
    b = Mamba2Block(64, heads=4, headdim=16, groups=2, dstate=64, dtype=torch.float32)
    with torch.no_grad():
        for q in (b.norm_w, b.gate_w, b.norm_b, b.dt_bias):
            q += 0.3 * torch.randn_like(q)
    return b, {k: v.detach().double().cpu().requires_grad_() for k, v in b.named_parameters()}


def test_block_trains():
    b, p = make()
    cu = [0, 70, 71, 71, 140]
    x = torch.randn(140, 64, device="cuda", requires_grad=True)
    dy = torch.randn(140, 64, device="cuda")
    x64 = x.detach().double().cpu().requires_grad_()
    y = b(x, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    y.backward(dy)
    want = reference(p, b, x64, cu)
    want.backward(dy.double().cpu())
    close("y", y, want.detach())
    close("dx", x.grad, x64.grad)
    for k, v in b.named_parameters():
        close(k, v.grad, p[k].grad)


def test_block_serves():
    b, p = make()
    x = torch.randn(75, 64, device="cuda")
    want = reference(p, b, x.double().cpu(), [0, 75]).detach()
    states, slot = b.new_states(3), torch.tensor([1], dtype=torch.int32, device="cuda")
    out = [b.prefill(x[:70], torch.tensor([0, 70], dtype=torch.int32, device="cuda"), states, slot)]
    for t in range(70, 75):
        out.append(b.decode(x[t:t + 1], states, slot))
    close("y", torch.cat(out), want)
    assert not states[0].any() and not states[2].any()


# In bf16, the block's own type, sums are FP32 and each of the ten stages rounds what it hands on by at most 2^-8 of it, with the
# same 3 for the factors between them; a head's sums over tokens of either sign (A_log, dt_bias, D) keep a third or less of what
# they add.
TOL_BF16 = 10 * 3 * 2.0 ** -8


def test_block_in_bf16():
    torch.manual_seed(8)
    b = Mamba2Block(64, heads=4, headdim=16, groups=2, dstate=64)
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in b.named_parameters()}
    cu = [0, 70, 71, 71, 140]
    x = torch.randn(140, 64, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(140, 64, device="cuda").bfloat16()
    x64 = x.detach().double().cpu().requires_grad_()
    y = b(x, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    y.backward(dy)
    want = reference(p, b, x64, cu)
    want.backward(dy.double().cpu())
    grads = [("y", y.detach(), want.detach()), ("dx", x.grad, x64.grad)] + [(k, v.grad, p[k].grad) for k, v in b.named_parameters()]
    for name, got, ref in grads:
        err = ((got.double().cpu() - ref).norm() / ref.norm()).item()
        print(f"{name}: {err:.2e}", flush=True)
        assert err <= TOL_BF16 * (3 if name in ("A_log", "dt_bias", "D") else 1), name
    # serving: a prompt, then single tokens
    states, slot = b.new_states(3), torch.tensor([1], dtype=torch.int32, device="cuda")
    x = x.detach()
    out = [b.prefill(x[:70], torch.tensor([0, 70], dtype=torch.int32, device="cuda"), states, slot)]
    out += [b.decode(x[t:t + 1], states, slot) for t in range(70, 75)]
    want = reference(p, b, x64[:75], [0, 75]).detach()
    err = ((torch.cat(out).double().cpu() - want).norm() / want.norm()).item()
    assert err <= TOL_BF16
