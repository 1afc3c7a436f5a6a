"""A linear-attention block on this library: training steps, then a prompt and single tokens.

    python -m examples.linear_block

The block is  x + W_out norm(attention(W_in norm(x)))  over packed sequences: an
RMS norm, one product giving queries, keys, values and the output's gate, the
norm and rotation of queries and keys, linear attention with a fixed decay a
head, an RMS norm by heads with the gate behind it, and a product back.  Training
runs both directions of all four; serving takes a prompt through the scan, which
leaves its final state in the sequence's slot, and goes on from there with
gdn_linear_decode_step.  The two products are torch's.
"""
import torch

from gated_deltanet_state_gdn_amd import (
    gdn_layer_norm, gdn_linear_decode_step, gdn_linear_scan, gdn_linear_scan_backward, gdn_qk_norm_rope, gdn_qk_norm_rope_backward,
)

from .mamba2_block import Norm


class QkNormRope(torch.autograd.Function):
    """gdn_qk_norm_rope with its gradient."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        return gdn_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)

    @staticmethod
    def backward(ctx, dq, dk):
        g = gdn_qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors)
        return g.dq, g.dk, g.dq_weight, g.dk_weight, None, None


class Attention(torch.autograd.Function):
    """gdn_linear_scan from zero states with its gradient."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, cu_seqlens):
        ctx.save_for_backward(q, k, v, log_decay, cu_seqlens)
        return gdn_linear_scan(q, k, v, log_decay, cu_seqlens)

    @staticmethod
    def backward(ctx, do):
        g = gdn_linear_scan_backward(do.contiguous(), *ctx.saved_tensors)
        return g.dq, g.dk, g.dv, None, None


class LinearBlock(torch.nn.Module):
    def __init__(self, width, heads, kv_heads, dim, rotary=None, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.H, self.G, self.d = heads, kv_heads, dim
        inner = heads * dim
        self.parts = [inner, kv_heads * dim, kv_heads * dim, inner]  # q, k, v and the gate
        make = lambda *s: torch.randn(*s, device=device) * s[-1] ** -0.5  # noqa: E731
        P = torch.nn.Parameter
        self.w_in, self.w_out = P(make(sum(self.parts), width).to(dtype)), P(make(width, inner).to(dtype))
        self.norm_w, self.out_w = P(torch.ones(width, device=device)), P(torch.ones(inner, device=device))
        self.q_w, self.k_w = (P(torch.ones(dim, device=device)) for _ in range(2))
        rotary = rotary or dim
        h, i = torch.arange(1, heads + 1, device=device), torch.arange(0, rotary, 2, device=device)
        self.register_buffer("log_decay", -torch.exp2(-8.0 * h / heads))
        self.register_buffer("inv_freq", (1e4 ** (-i.double() / rotary)).float())

    def new_states(self, slots):
        return torch.zeros(slots, self.H, self.d, self.d, device=self.w_in.device)

    def _split(self, rows):
        q, k, v, gate = torch.split(rows, self.parts, dim=1)
        return q.unflatten(1, (self.H, -1)), k.unflatten(1, (self.G, -1)), v.unflatten(1, (self.G, -1)), gate

    def forward(self, x, positions, cu_seqlens):
        """x [tokens, width] of packed sequences and their tokens' positions; differentiable."""
        u = Norm.apply(x, self.norm_w, None, None, {"rms": True})
        q, k, v, gate = self._split(u @ self.w_in.T)
        q, k = QkNormRope.apply(q, k, self.q_w, self.k_w, positions, self.inv_freq)
        o = Attention.apply(q, k, v, self.log_decay, cu_seqlens).flatten(1)
        o = Norm.apply(o, self.out_w, None, gate, {"groups": self.H, "rms": True, "gate_after": True})
        return x + o @ self.w_out.T

    @torch.no_grad()
    def _serve(self, x, positions, attention):
        q, k, v, gate = self._split(gdn_layer_norm(x, self.norm_w, rms=True) @ self.w_in.T)
        gdn_qk_norm_rope(q, k, self.q_w, self.k_w, positions, self.inv_freq, q_out=q, k_out=k)
        o = attention(q, k, v, self.log_decay).flatten(1)
        return x + gdn_layer_norm(o, self.out_w, gate=gate, groups=self.H, rms=True, gate_after=True) @ self.w_out.T

    def prefill(self, x, positions, cu_seqlens, states, slot_map):
        """The same over prompts, from and to the sequences' slots of `states`."""
        return self._serve(x, positions, lambda *a: gdn_linear_scan(*a, cu_seqlens, pool=states, slot_map=slot_map))

    def decode(self, x, positions, states, slot_map):
        """One token of each sequence; x [sequences, width]."""
        return self._serve(x, positions, lambda *a: gdn_linear_decode_step(*a, states, slot_map, out_dtype=x.dtype))


def main():
    torch.manual_seed(0)
    block = LinearBlock(256, heads=8, kv_heads=4, dim=64)
    lengths = [300, 1, 211]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    places = lambda *lens: ints([i for n in lens for i in range(n)])  # noqa: E731
    cu = ints([0, 300, 301, 512])
    x, target = (torch.randn(512, 256, device="cuda").bfloat16() for _ in range(2))
    opt = torch.optim.SGD(block.parameters(), lr=0.5)
    for step in range(10):
        loss = (block(x, places(*lengths), cu) - target).float().pow(2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print(f"training step {step}: loss {loss.item():.4f}")

    states, slots = block.new_states(4), ints([2, 0, 3])
    block.prefill(x, places(*lengths), cu, states, slots)
    after = block.decode(x[:3], ints(lengths), states, slots)
    # the same tokens behind their prompts, in one scan
    pieces = [torch.cat([p, x[i:i + 1]]) for i, p in enumerate(torch.split(x, lengths))]
    whole = block(torch.cat(pieces), places(301, 2, 212), ints([0, 301, 303, 515]))[[300, 302, 514]]
    print(f"a token by decode against the scan: largest difference {(after - whole).abs().max().item():.4f}, "
          f"largest value {whole.abs().max().item():.2f}")


if __name__ == "__main__":
    main()
