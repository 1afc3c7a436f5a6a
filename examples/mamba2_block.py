"""A Mamba2 block on this library: training steps, then a prompt and single tokens.

    python -m examples.mamba2_block

The block is  x + W_out norm(scan(W_in norm(x)))  over packed sequences: a layer
norm, one product giving the gate z, the scan's x, B, C and dt, the recurrence,
an RMS norm by groups with the gate before it, and a product back.  (The short
convolution that such blocks put in front of the scan is left out.)  Training
runs both directions of the norm and of the scan; serving takes a prompt through
the scan, which leaves its final state in the sequence's slot, and goes on from
there with gdn_mamba2_decode_step.  The two products are torch's.
"""
import torch

from gated_deltanet_state_gdn_amd import (
    gdn_layer_norm, gdn_layer_norm_backward, gdn_mamba2_decode_step, gdn_mamba2_scan, gdn_mamba2_scan_backward,
)


class Norm(torch.autograd.Function):
    """gdn_layer_norm with its gradient."""

    @staticmethod
    def forward(ctx, x, weight, bias, gate, kw):
        y, mean, rstd = gdn_layer_norm(x, weight, bias, gate=gate, save_stats=True, **kw)
        ctx.save_for_backward(x, weight, bias, gate, mean, rstd)
        ctx.kw = {k: v for k, v in kw.items() if k != "eps"}
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, gate, mean, rstd = ctx.saved_tensors
        g = gdn_layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, bias=bias, gate=gate, **ctx.kw)
        return g.dx, g.dweight, g.dbias, g.dgate, None


class Scan(torch.autograd.Function):
    """gdn_mamba2_scan from zero states with its gradient."""

    @staticmethod
    def forward(ctx, x, Bm, Cm, dt, A_log, dt_bias, D, cu_seqlens):
        ctx.save_for_backward(x, Bm, Cm, dt, A_log, dt_bias, D, cu_seqlens)
        return gdn_mamba2_scan(x, Bm, Cm, dt, A_log, dt_bias, D, cu_seqlens)

    @staticmethod
    def backward(ctx, dy):
        g = gdn_mamba2_scan_backward(dy.contiguous(), *ctx.saved_tensors)
        return g.dx, g.dBm, g.dCm, g.ddt, g.dA_log, g.ddt_bias, g.dD, None


class Mamba2Block(torch.nn.Module):
    def __init__(self, width, heads, headdim, groups, dstate, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.H, self.d, self.G, self.n = heads, headdim, groups, dstate
        inner = heads * headdim
        # dt's columns come last, so that x, B and C start at multiples of 16 bytes; rows are padded to one
        self.parts = [inner, inner, groups * dstate, groups * dstate, heads]
        rows = -(-sum(self.parts) // 8) * 8
        make = lambda *s: torch.randn(*s, device=device) * s[-1] ** -0.5  # noqa: E731
        P = torch.nn.Parameter
        self.w_in, self.w_out = P(make(rows, width).to(dtype)), P(make(width, inner).to(dtype))
        self.norm_w, self.norm_b = P(torch.ones(width, device=device)), P(torch.zeros(width, device=device))
        self.gate_w = P(torch.ones(inner, device=device))
        self.A_log = P(torch.rand(heads, device=device))
        self.dt_bias, self.D = P(torch.zeros(heads, device=device)), P(torch.ones(heads, device=device))

    def new_states(self, slots):
        return torch.zeros(slots, self.H, self.d, self.n, device=self.w_in.device)

    def _split(self, rows):
        z, x, Bm, Cm, dt = torch.split(rows[:, :sum(self.parts)], self.parts, dim=1)
        heads = lambda t, h: t.unflatten(1, (h, -1))  # noqa: E731
        return z, heads(x, self.H), heads(Bm, self.G), heads(Cm, self.G), dt

    def forward(self, x, cu_seqlens):
        """x [tokens, width] of packed sequences; differentiable."""
        u = Norm.apply(x, self.norm_w, self.norm_b, None, {})
        z, *ins = self._split(u @ self.w_in.T)
        y = Scan.apply(*ins, self.A_log, self.dt_bias, self.D, cu_seqlens).flatten(1)
        y = Norm.apply(y, self.gate_w, None, z, {"groups": self.G, "rms": True})
        return x + y @ self.w_out.T

    @torch.no_grad()
    def _serve(self, x, scan):
        u = gdn_layer_norm(x, self.norm_w, self.norm_b)
        z, *ins = self._split(u @ self.w_in.T)
        y = scan(*ins, self.A_log, self.dt_bias, self.D).flatten(1)
        return x + gdn_layer_norm(y, self.gate_w, gate=z, groups=self.G, rms=True) @ self.w_out.T

    def prefill(self, x, cu_seqlens, states, slot_map):
        """The same over prompts, from and to the sequences' slots of `states`."""
        return self._serve(x, lambda *a: gdn_mamba2_scan(*a, cu_seqlens, pool=states, slot_map=slot_map))

    def decode(self, x, states, slot_map):
        """One token of each sequence; x [sequences, width]."""
        return self._serve(x, lambda x, Bm, Cm, dt, *p: gdn_mamba2_decode_step(
            x.contiguous(), Bm.contiguous(), Cm.contiguous(), dt.contiguous(), *p, states, slot_map, out_dtype=x.dtype))


def main():
    torch.manual_seed(0)
    block = Mamba2Block(256, heads=8, headdim=64, groups=2, dstate=128)
    lengths = [300, 1, 211]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = ints([0, 300, 301, 512])
    x, target = (torch.randn(512, 256, device="cuda").bfloat16() for _ in range(2))
    opt = torch.optim.SGD(block.parameters(), lr=0.5)
    for step in range(10):
        loss = (block(x, cu) - target).float().pow(2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print(f"training step {step}: loss {loss.item():.4f}")

    states, slots = block.new_states(4), ints([2, 0, 3])
    block.prefill(x, cu, states, slots)
    after = block.decode(x[:3], states, slots)
    # the same tokens behind their prompts, in one scan
    pieces = [torch.cat([p, x[i:i + 1]]) for i, p in enumerate(torch.split(x, lengths))]
    whole = block(torch.cat(pieces), ints([0, 301, 303, 515]))[[300, 302, 514]]
    print(f"a token by decode against the scan: largest difference {(after - whole).abs().max().item():.4f}, "
          f"largest value {whole.abs().max().item():.2f}")


if __name__ == "__main__":
    main()
