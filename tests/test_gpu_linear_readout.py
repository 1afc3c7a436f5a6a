"""What the bf16 linear scan reads from its state and from its weighted products, to the last of FP32's 24 bits, in both directions.

Decays are 1, the scale is 1, and the vectors are such that each output is a single FP32 value, or a sum that FP32 holds exactly.  So
no step but the output's own rounding may lose anything, and the results have to equal the rounded values.  Those lie 2^-12 of a bf16
step or less beside the middle between two bf16 numbers, where 16 bits of them would be the middle itself and go to the even neighbour.
"""
import pytest
import torch

from gpu_util import DEV, require_gpu, say

pytestmark = pytest.mark.gpu
T = 150  # two whole chunks and a part


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def near_ties(shape):
    """FP32 values right beside the middle between two bf16 numbers: above the middle behind an even number, below it behind an odd one."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(shape, generator=g).bfloat16()
    x = torch.where(x == 0, torch.ones_like(x), x)
    bits = x.view(torch.int16).to(torch.int32) << 16
    odd = (bits >> 16 & 1).bool()
    return (bits + torch.where(odd, 0x8000 - 4, 0x8000 + 4).to(torch.int32)).view(torch.float32)


def rows(d, heads, values):
    """[T, heads, d] bf16 whose token t holds values(t), for every head."""
    x = torch.zeros(T, heads, d)
    for t in range(T):
        x[t] = values(t)
    return x.bfloat16().to(DEV)


def unit(d, t):
    return torch.eye(d)[t % d]


def call(d, heads, backward, q=None, k=None, v=None, do=None, init=None, dfinal=None):
    import gated_deltanet_state_gdn_amd as gdn
    H, Hq, Hk, Hv = heads
    zero = lambda x, h: rows(d, h, lambda t: torch.zeros(d)) if x is None else rows(d, h, x)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    ins = (zero(q, Hq), zero(k, Hk), zero(v, Hv), torch.zeros(H, device=DEV), ints([0, T]))
    states = dict(pool=init.to(DEV), slot_map=ints([0])) if init is not None else {}
    if not backward:
        return gdn.gdn_linear_scan(*ins, **states, scale=1.0)
    return gdn.gdn_linear_scan_backward(zero(do, H), *ins, **states, dfinal=dfinal.to(DEV) if dfinal is not None else None, scale=1.0)


def same(got, want, what):
    want = want.to(got.dtype)
    wrong = (got.cpu() != want).sum().item()
    assert wrong == 0, f"{what}: {wrong} of {want.numel()} elements are not the exact value's rounding"


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_state(d):
    """One-hot vectors read a row or a column of the state; nothing is written to it."""
    say(f"linear readout state d={d}")
    S, one = near_ties((1, 2, d, d)), lambda t: unit(d, t)
    pick = torch.arange(T) % d
    row, column = S[0][:, pick].transpose(0, 1), S[0][:, :, pick].permute(2, 0, 1)  # [T, H, d]
    assert (row.bfloat16().float() != row).all()
    full = (2, 2, 2, 2)
    same(call(d, full, False, q=one, init=S), row, "o")
    same(call(d, full, True, do=one, init=S).dq, column, "dq")
    same(call(d, full, True, k=one, dfinal=S).dv, row, "dv")
    same(call(d, full, True, v=one, dfinal=S).dk, column, "dk")


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("H", [1, 2])
def test_products(d, H):
    """1 + 2^-8 + 2^-20 as the product of two vectors, times a one-hot one: from the token with that on, or in reverse up to it.  With
    two states to a head its gradient is the sum of two such values."""
    say(f"linear readout products d={d} H={H}")
    u, ones = torch.zeros(d), torch.ones(d)
    u[:3] = torch.tensor([1.0, 2.0 ** -8, 2.0 ** -20])
    value = 1 + 2.0 ** -8 + 2.0 ** -20
    t, c = torch.arange(T)[:, None], torch.arange(d)[None]
    heads, all_u, all_ones = (H, 1, 1, 1), lambda t: u, lambda t: ones
    early = lambda t: unit(d, t) if t < d else torch.zeros(d)  # noqa: E731
    late = lambda t: unit(d, t) if t >= T - d else torch.zeros(d)  # noqa: E731
    last = T - 1 - (T - 1 - c) % d  # the token that holds column c behind T - d
    forward, reverse = ((t >= c) * value)[:, None], ((t <= last) * value)[:, None]
    same(call(d, heads, False, q=all_u, k=all_ones, v=early), forward.expand(T, H, d), "o")
    same(call(d, heads, True, do=all_u, v=all_ones, k=early).dq, H * forward, "dq")
    same(call(d, heads, True, k=all_u, q=all_ones, do=late).dv, H * reverse, "dv")
    same(call(d, heads, True, v=all_u, do=all_ones, q=late).dk, H * reverse, "dk")
