"""The example block: the norm and rotation of queries and keys, the scan, the block's norms, their gradients and the decode step
together, against the same block written out token by token in 64 bits."""
import pytest
import torch
import torch.nn.functional as F

from examples.linear_block import LinearBlock

pytestmark = pytest.mark.gpu

# In FP32 an output passes six stages (norm, product, norm and rotation, scan, norm, product) and a gradient those and their
# mirrors, twelve roundings of sums of up to 256 terms each: 12 * sqrt(256) * 2^-24 of the whole, times 3 for the factors between
# them (the norms divide by about 1, decays are below 1).
TOL = 12 * 16 * 3 * 2.0 ** -24
# In bf16 sums are FP32 and each of the twelve stages rounds what it hands on by at most 2^-8 of it, with the same 3.
TOL_BF16 = 12 * 3 * 2.0 ** -8
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def reference(p, b, x, pos, cu):
    H, G = b.H, b.G
    u = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-5) * p["norm_w"]
    q, k, v, gate = torch.split(u @ p["w_in"].T, b.parts, dim=1)
    q, k, v = q.unflatten(1, (H, -1)), k.unflatten(1, (G, -1)), v.unflatten(1, (G, -1))
    angle = torch.tensor(pos, dtype=torch.float64)[:, None] * b.inv_freq.double().cpu()
    c, s, n = angle.cos()[:, None], angle.sin()[:, None], angle.shape[1]

    def turned(t, w):
        t = t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6) * w
        lo, hi, rest = t[..., :n], t[..., n:2 * n], t[..., 2 * n:]
        return torch.cat([lo * c - hi * s, hi * c + lo * s, rest], -1)

    q, k = turned(q, p["q_w"]), turned(k, p["k_w"])
    k, v = k.repeat_interleave(H // G, 1), v.repeat_interleave(H // G, 1)
    lam = torch.exp(b.log_decay.double().cpu())[:, None, None]
    os = []
    for lo, hi in zip(cu[:-1], cu[1:]):
        S = x.new_zeros(H, b.d, b.d)
        for t in range(lo, hi):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            os.append((q[t][:, :, None] * S).sum(1) * b.d ** -0.5)
    o = torch.stack(os)
    o = (o * torch.rsqrt(o.pow(2).mean(-1, keepdim=True) + 1e-5)).flatten(1) * p["out_w"] * F.silu(gate)
    return x + o @ p["w_out"].T


def close(name, a, b, tol):
    err = ((a.detach().double().cpu() - b).norm() / b.norm()).item()
    print(f"{name}: {err:.2e}", flush=True)
    assert err <= tol, f"{name}: {err:.2e} > {tol:.2e}"


def make(dtype):
    torch.manual_seed(7)
    b = LinearBlock(64, heads=4, kv_heads=2, dim=32, rotary=16, dtype=dtype)
    with torch.no_grad():
        for q in (b.norm_w, b.out_w, b.q_w, b.k_w):
            q += 0.3 * torch.randn_like(q)
    return b, {k: v.detach().double().cpu().requires_grad_() for k, v in b.named_parameters()}


@pytest.mark.parametrize("dtype,tol", [(torch.float32, TOL), (torch.bfloat16, TOL_BF16)])
def test_block_trains(dtype, tol):
    b, p = make(dtype)
    cu = [0, 70, 71, 71, 140]
    pos = [i for lo, hi in zip(cu[:-1], cu[1:]) for i in range(hi - lo)]
    x = torch.randn(140, 64, device="cuda").to(dtype).requires_grad_()
    dy = torch.randn(140, 64, device="cuda").to(dtype)
    x64 = x.detach().double().cpu().requires_grad_()
    y = b(x, ints(pos), ints(cu))
    y.backward(dy)
    want = reference(p, b, x64, pos, cu)
    want.backward(dy.double().cpu())
    close("y", y, want.detach(), tol)
    close("dx", x.grad, x64.grad, tol)
    for k, v in b.named_parameters():
        close(k, v.grad, p[k].grad, tol)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, TOL), (torch.bfloat16, TOL_BF16)])
def test_block_serves(dtype, tol):
    b, p = make(dtype)
    x = torch.randn(75, 64, device="cuda").to(dtype)
    want = reference(p, b, x.double().cpu(), list(range(75)), [0, 75]).detach()
    states, slot = b.new_states(3), ints([1])
    out = [b.prefill(x[:70], ints(list(range(70))), ints([0, 70]), states, slot)]
    for t in range(70, 75):
        out.append(b.decode(x[t:t + 1], ints([t]), states, slot))
    close("y", torch.cat(out), want, tol)
    assert not states[0].any() and not states[2].any()


def test_example_runs(capsys):
    from examples import linear_block
    linear_block.main()
    assert "training step 9" in capsys.readouterr().out
