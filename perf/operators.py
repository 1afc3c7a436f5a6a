"""The Mamba2 sequence scan and the block's normalisation, forward and backward: cases, inputs and plain forms.

Four operators, named by a case's "op":

  scan       y_t = S_t C_t + D x_t over packed sequences, S_t = e^{g_t} S_{t-1} + dt'_t x_t B_t^T, from and to slots of a state pool
  scan_bwd   the gradients of that scan with respect to every input, from dy and, where a case has it, the final states' gradient
  norm       layer or RMS norm of slices of a row, with a weight, an optional bias and an optional SiLU gate before or after it
  norm_bwd   its gradients, the weight's and bias's summed over all rows

`own` False computes them in elementary torch operations, True by the library's kernels.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
Q = 64  # tokens a chunk of the plain scan
EPS = 1e-5


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


# ------------------------------------------------------------------ cases
def _scan(op, lens, H, G, d, n, dtype, state, **name):
    return dict(name, op=op, lens=lens, H=H, G=G, d=d, n=n, dtype=dtype, state=state)


def _norm(op, rows, N, groups, dtype, rms, bias, gate, **name):
    return dict(name, op=op, rows=rows, N=N, groups=groups, dtype=dtype, rms=rms, bias=bias, gate=gate)


def listed():
    return [
        # a chat turn's few new tokens appended to one session on a small layer: latency
        _scan("scan", "37", 8, 1, 64, 128, "bf16", "f32", name="scan_turn"),
        # the prefill of four prompts through a full layer (128 heads of 64 x 128 in 8 groups)
        _scan("scan", "1024,3000,8192,8192", 128, 8, 64, 128, "bf16", "f32", name="scan_prefill"),
        # a serving step's mix of short and empty continuations, 16-bit states
        _scan("scan", "1,0,63,64,65,500,2,129,333,7,1024,1,90,255,0,611,1,48,200,1500", 32, 2, 64, 128, "bf16", "bf16", name="scan_mix"),
        # one document in full precision on a narrow state
        _scan("scan", "4099", 24, 1, 64, 64, "f32", "f32", name="scan_f32"),
        # a training step's batch of four sequences through the full layer
        _scan("scan_bwd", "4096,4096,4096,4096", 128, 8, 64, 128, "bf16", "none", name="scan_bwd_train"),
        # one long document whose state came from an earlier part and goes on into a later one (truncated backpropagation)
        _scan("scan_bwd", "16385", 32, 1, 64, 128, "bf16", "f32", name="scan_bwd_long"),
        # a small model's packed documents in full precision
        _scan("scan_bwd", "1,130,0,511,77,300", 6, 2, 16, 64, "f32", "f32", name="scan_bwd_f32"),
        # the gated group norm after three sequences' decode step: latency
        _norm("norm", 3, 8192, 8, "bf16", True, False, "before", name="norm_token"),
        # the layer norm in front of a block over a prefill
        _norm("norm", 20408, 4096, 1, "bf16", False, True, "none", name="norm_prefill"),
        # its backward pass in a training step
        _norm("norm_bwd", 16384, 4096, 1, "bf16", False, True, "none", name="norm_bwd_train"),
        # the backward pass of the gated group norm behind the scan
        _norm("norm_bwd", 16384, 8192, 8, "bf16", True, False, "before", name="norm_bwd_gated"),
        # per-head norm of a read-out with its gate behind, full precision, an odd number of rows
        _norm("norm_bwd", 40001, 128, 1, "f32", True, False, "after", name="norm_bwd_heads"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan_bwd", "norm", "norm_bwd"])
    if op.startswith("scan"):
        d, n = rng.choice([16, 64, 64, 64, 128]), rng.choice([16, 64, 128, 128])
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.randint(1, 16)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32", "f16"])
        most = 16384 * 128 * 64 * 128 // (4 if op == "scan_bwd" else 2) // (1 if dtype == "bf16" else 8)
        tokens = _log(rng, 1, max(2, min(20000, most // (H * d * n))))
        cuts = sorted(rng.randint(0, tokens) for _ in range(rng.choice([0, 0, 1, 3, rng.randint(4, 24)])))
        ends = cuts + [tokens]
        lens = ",".join(str(b - a) for a, b in zip([0] + cuts, ends))
        state = rng.choice(["f32", "f32", dtype]) if op == "scan" else rng.choice(["none", "f32", dtype])
        return _scan(op, lens, H, G, d, n, dtype, state)
    groups = rng.choice([1, 1, 1, 2, 8])
    size = rng.choice([_log(rng, 16, 16384 // groups), 8 * _log(rng, 2, 2048 // groups)])
    N = groups * size
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    rows = _log(rng, 1, max(2, min(200000, (16384 * 8192 // (2 if dtype == "f32" else 1)) // N)))
    return _norm(op, rows, N, groups, dtype, rng.random() < 0.5, rng.random() < 0.4,
                 rng.choice(["none", "none", "before", "after"]))


# ------------------------------------------------------------------ inputs
def _randn(gen, shape, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32) * scale + shift


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]
    if case["op"].startswith("scan"):
        lens, H, G, d, n = _lens(case), case["H"], case["G"], case["d"], case["n"]
        T, N = sum(lens), len(lens)
        u = torch.rand((3, H), generator=gen, device="cuda")
        step = torch.exp(math.log(1e-3) + u[1] * math.log(1e2))
        cu = torch.zeros(N + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
        s = dict(op=case["op"], lens=lens, cu=cu.cuda(),
                 x=_randn(gen, (T, H, d)).to(dt), Bm=_randn(gen, (T, G, n), n ** -0.5).to(dt), Cm=_randn(gen, (T, G, n), n ** -0.5).to(dt),
                 dt=_randn(gen, (T, H), 0.5).to(dt), A_log=torch.log(1 + 15 * u[0]), dt_bias=torch.log(torch.expm1(step)), D=0.5 + u[2],
                 pool=None, slots=None, dfinal=None)
        if case["state"] != "none":
            s["pool"] = _randn(gen, (N + 2, H, d, n), 0.1).to(DT[case["state"]])
            s["slots"] = torch.randperm(N + 2, generator=gen, device="cuda")[:N].to(torch.int32)
        if case["op"] == "scan_bwd":
            s["dy"] = _randn(gen, (T, H, d), 0.05).to(dt)
            if case["state"] != "none":
                s["dfinal"] = _randn(gen, (N, H, d, n), 0.05)
        return s
    rows, N, groups = case["rows"], case["N"], case["groups"]
    s = dict(op=case["op"], groups=groups, rms=case["rms"], after=case["gate"] == "after",
             x=_randn(gen, (rows, N), 1.0, 0.1).to(dt), w=_randn(gen, (N,), 0.1, 1.0),
             b=_randn(gen, (N,), 0.1) if case["bias"] else None, z=_randn(gen, (rows, N)).to(dt) if case["gate"] != "none" else None)
    if case["op"] == "norm_bwd":
        s["dy"] = _randn(gen, (rows, N), 0.05).to(dt)
        u = s["x"].double()
        if case["gate"] == "before":
            z = s["z"].double()
            u = u * z * torch.sigmoid(z)
        u = u.view(rows, groups, N // groups)
        s["mean"] = torch.zeros((rows, groups), device="cuda") if case["rms"] else u.mean(-1).float()
        s["rstd"] = torch.rsqrt((u - s["mean"].double()[..., None]).square().mean(-1) + EPS).float()
    return s


# ------------------------------------------------------------------ plain forms
def _scan_plain(lens, cu, x, Bm, Cm, dt, A_log, dt_bias, D, S0):
    """The scan in chunks of Q tokens: products inside a chunk, and the states between chunks by one product with the matrix of the
    decays from chunk to chunk.  Log-decays are summed in 64 bits: their sums grow with the sequence and only differences matter.
    Arguments in 32 bits; S0 [sequences, H, d, n].  Returns y and the final states."""
    T, H, d = x.shape
    G, n = Bm.shape[1:]
    dev = x.device
    N = len(lens)
    nc = sum(-(-v // Q) for v in lens)
    if nc == 0:
        return x * D[:, None], S0
    count = (cu[1:] - cu[:-1] + Q - 1).div(Q, rounding_mode="floor").long()
    first = count.cumsum(0) - count
    seq = torch.repeat_interleave(torch.arange(N, device=dev), count, output_size=nc)
    tok = cu[seq].long()[:, None] + (torch.arange(nc, device=dev) - first[seq])[:, None] * Q + torch.arange(Q, device=dev)
    live = tok < cu[seq + 1].long()[:, None]
    at = tok.clamp(max=T - 1)
    dtp = torch.nn.functional.softplus(dt + dt_bias, threshold=60.0)
    g = -torch.exp(A_log.double()) * dtp.double()
    dtc = torch.where(live[..., None], dtp[at], 0.0)                       # [nc, Q, H]
    cum = torch.where(live[..., None], g[at], 0.0).cumsum(1)              # [nc, Q, H] in 64 bits
    X = (torch.where(live[..., None, None], x[at], 0.0)).transpose(1, 2)   # [nc, H, Q, d]
    Bc = torch.where(live[..., None, None], Bm[at], 0.0).transpose(1, 2)   # [nc, G, Q, n]
    Cc = torch.where(live[..., None, None], Cm[at], 0.0).transpose(1, 2)
    c = cum.transpose(1, 2)                                                # [nc, H, Q]
    low = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    L = torch.exp(torch.where(low, c[..., :, None] - c[..., None, :], -math.inf)).float()
    CB = torch.matmul(Cc, Bc.transpose(2, 3).contiguous()).repeat_interleave(H // G, 1)
    xd = X * dtc.transpose(1, 2)[..., None]
    y = torch.matmul(CB * L, xd)
    w = torch.exp(c[..., -1:] - c).float()
    Z = torch.matmul((xd * w[..., None]).transpose(2, 3).contiguous(), Bc.repeat_interleave(H // G, 1))  # [nc, H, d, n]
    total = c[..., -1].cumsum(0)                                           # [nc, H] in 64 bits
    before = total - c[..., -1]
    order = torch.arange(nc, device=dev)
    earlier = (order[:, None] > order[None, :]) & (seq[:, None] == seq[None, :])
    M = torch.exp(torch.where(earlier, before.t()[:, :, None] - total.t()[:, None, :], -math.inf)).float()
    S = torch.matmul(M, Z.permute(1, 0, 2, 3).reshape(H, nc, d * n)).view(H, nc, d, n).transpose(0, 1)
    S = S + torch.exp(before - before[first.clamp(max=nc - 1)][seq]).float()[..., None, None] * S0[seq]
    y = y + torch.exp(c).float()[..., None] * torch.matmul(Cc.repeat_interleave(H // G, 1), S.transpose(2, 3).contiguous())
    out = torch.zeros((T, H, d), device=dev).index_put((tok[live],), y.transpose(1, 2)[live]) + x * D[:, None]
    last = (first + count - 1).clamp(min=0)
    end = torch.exp(c[..., -1]).float()[..., None, None] * S + Z
    return out, torch.where((count > 0)[:, None, None, None], end[last], S0)


def _silu(z):
    return z * torch.sigmoid(z)


def _run_plain(s):
    op = s["op"]
    if op in ("scan", "scan_bwd"):
        pool, slots = s["pool"], s["slots"]
        lens, names = s["lens"], ("x", "Bm", "Cm", "dt", "A_log", "dt_bias", "D")
        H, d, n = s["x"].shape[1], s["x"].shape[2], s["Bm"].shape[2]
        S0 = pool[slots.long()].float() if pool is not None else torch.zeros((len(lens), H, d, n), device="cuda")
        if op == "scan":
            y, end = _scan_plain(lens, s["cu"], *(s[k].float() for k in names), S0)
            pool[slots.long()] = end.to(pool.dtype)
            return {"y": y.to(s["x"].dtype), "state": pool}
        leaves = [s[k].float().detach().requires_grad_() for k in names] + [S0.requires_grad_()]
        with torch.enable_grad():
            y, end = _scan_plain(lens, s["cu"], *leaves)
        outs, grads = ([y], [s["dy"].float()]) if s["dfinal"] is None else ([y, end], [s["dy"].float(), s["dfinal"]])
        got = torch.autograd.grad(outs, leaves, grads)
        r = {"d" + k: v.to(s[k].dtype) for k, v in zip(names, got)}
        if pool is not None:
            r["dinit"] = got[-1]
        return r
    x, z = s["x"].float(), s["z"].float() if s["z"] is not None else None
    w, b = s["w"], s["b"]
    rows, N = x.shape
    u = (x * _silu(z) if z is not None and not s["after"] else x).view(rows, s["groups"], N // s["groups"])
    if op == "norm":
        mean = torch.zeros(u.shape[:2], device="cuda") if s["rms"] else u.mean(-1)
        rstd = torch.rsqrt((u - mean[..., None]).square().mean(-1) + EPS)
        y = ((u - mean[..., None]) * rstd[..., None]).view(rows, N) * w
        y = y + b if b is not None else y
        y = y * _silu(z) if s["after"] else y
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    dy, mean, rstd = s["dy"].float(), s["mean"], s["rstd"]
    xh = ((u - mean[..., None]) * rstd[..., None]).view(rows, N)
    r, dv = {}, dy
    if z is not None:
        sg = torch.sigmoid(z)
        slope = sg * (1 + z * (1 - sg))
    if s["after"]:
        v = xh * w
        v = v + b if b is not None else v
        r["dz"] = (dy * v * slope).to(s["x"].dtype)
        dv = dy * _silu(z)
    r["dw"] = (dv * xh).sum(0)
    if b is not None:
        r["db"] = dv.sum(0)
    dxh, xg = (dv * w).view(u.shape), xh.view(u.shape)
    du = dxh - xg * (dxh * xg).mean(-1, keepdim=True)
    if not s["rms"]:
        du = du - dxh.mean(-1, keepdim=True)
    du = (du * rstd[..., None]).view(rows, N)
    if z is not None and not s["after"]:
        r["dz"] = (du * x * slope).to(s["x"].dtype)
        du = du * _silu(z)
    r["dx"] = du.to(s["x"].dtype)
    return r


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import gated_deltanet_state_gdn_amd as gdn
    op = s["op"]
    if op in ("scan", "scan_bwd"):
        ins = [s[k] for k in ("x", "Bm", "Cm", "dt", "A_log", "dt_bias", "D", "cu")]
        if op == "scan":
            y = gdn.gdn_mamba2_scan(*ins, pool=s["pool"], slot_map=s["slots"])
            return {"y": y, "state": s["pool"]}
        g = gdn.gdn_mamba2_scan_backward(s["dy"], *ins, pool=s["pool"], slot_map=s["slots"], dfinal=s["dfinal"])
        r = {"dx": g.dx, "dBm": g.dBm, "dCm": g.dCm, "ddt": g.ddt, "dA_log": g.dA_log, "ddt_bias": g.ddt_bias, "dD": g.dD}
        if s["pool"] is not None:
            r["dinit"] = g.dinit
        return r
    form = dict(gate=s["z"], groups=s["groups"], rms=s["rms"], gate_after=s["after"])
    if op == "norm":
        y, mean, rstd = gdn.gdn_layer_norm(s["x"], s["w"], s["b"], eps=EPS, save_stats=True, **form)
        return {"y": y, "mean": mean, "rstd": rstd}
    g = gdn.gdn_layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], bias=s["b"], **form)
    r = {"dx": g.dx, "dw": g.dweight}
    if s["b"] is not None:
        r["db"] = g.dbias
    if s["z"] is not None:
        r["dz"] = g.dgate
    return r


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b = SIZE[case["dtype"]]
    if case["op"].startswith("scan"):
        lens, H, G, d, n = _lens(case), case["H"], case["G"], case["d"], case["n"]
        T, N = sum(lens), sum(v > 0 for v in lens)
        states = N * H * d * n
        tokens = T * (H * d + 2 * G * n + H) * b
        if case["op"] == "scan":  # x, B, C, dt in, y out, states both ways; per token and head a rank-one update and a read-out
            return {"bytes": tokens + T * H * d * b + 2 * states * SIZE[case["state"]], "flops": 4.0 * T * H * d * n}
        # inputs and dy in, four gradients out; per token and head both states' updates and the three products with them
        extra = 0 if case["state"] == "none" else states * (SIZE[case["state"]] + 8)
        return {"bytes": 2 * tokens + T * H * d * b + extra, "flops": 10.0 * T * H * d * n}
    rows, N = case["rows"], case["N"]
    each = (1 if case["gate"] == "none" else 2) * rows * N * b  # x and z
    stats = 8 * rows * case["groups"]
    if case["op"] == "norm":
        return {"bytes": each + rows * N * b + stats, "flops": 8.0 * rows * N}
    return {"bytes": 2 * each + rows * N * b + stats, "flops": 16.0 * rows * N}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    def scan(s):
        """Token by token, all sequences of the case side by side, in float64; the backward pass walks the same steps in reverse from
        states kept every K steps."""
        lens, dev, f = s["lens"], "cuda", torch.float64
        N, (T, H, d), (G, n) = len(lens), s["x"].shape, s["Bm"].shape[1:]
        x, Bm, Cm = s["x"].to(f), s["Bm"].to(f), s["Cm"].to(f)
        raw = s["dt"].to(f) + s["dt_bias"].to(f)
        dtp = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
        A, D = -torch.exp(s["A_log"].to(f)), s["D"].to(f)
        start = s["cu"][:-1].long()
        length = torch.tensor(lens, device=dev)
        S = s["pool"][s["slots"].long()].to(f) if s["pool"] is not None else torch.zeros((N, H, d, n), dtype=f, device=dev)
        most, heads = max(lens), torch.arange(H, device=dev) // (H // G)
        order = sorted(range(N), key=lambda i: -lens[i])  # the sequences still running at a step are the first ones
        perm = torch.tensor(order, device=dev)
        start, S = start[perm], S[perm].contiguous()
        running = [sum(v > t for v in lens) for t in range(most)]

        def token(t):
            k = running[t]
            i = start[:k] + t
            return k, i, dtp[i], torch.exp(A * dtp[i]), x[i], Bm[i][:, heads], Cm[i][:, heads]

        y = torch.zeros((T, H, d), dtype=f, device=dev)
        K = max(1, int(math.isqrt(max(1, most))))
        kept = {}
        for t in range(most):
            if s["op"] == "scan_bwd" and t % K == 0:
                kept[t] = S.clone()
            k, i, dp, e, xt, B, C = token(t)
            S[:k] *= e[..., None, None]
            S[:k] += (dp[..., None] * xt)[..., None] * B[:, :, None, :]
            if s["op"] == "scan":
                y[i] = torch.matmul(S[:k], C[..., None])[..., 0] + D[:, None] * xt
        back = torch.empty_like(perm)
        back[perm] = torch.arange(N, device=dev)
        if s["op"] == "scan":
            pool = s["pool"].to(f)
            used = length > 0
            pool[s["slots"].long()[used]] = S[back][used]
            return {"y": y, "state": pool}
        dy = s["dy"].to(f)
        dx, ddt = torch.zeros_like(x), torch.zeros((T, H), dtype=f, device=dev)
        dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
        dA = torch.zeros(H, dtype=f, device=dev)
        dS = s["dfinal"].to(f)[perm].clone() if s["dfinal"] is not None else torch.zeros_like(S)
        for t0 in range((most - 1) // K * K, -1, -K):
            S = kept.pop(t0)
            states = [S]
            for t in range(t0, min(t0 + K, most)):
                k, i, dp, e, xt, B, C = token(t)
                S = S.clone()
                S[:k] = S[:k] * e[..., None, None] + (dp[..., None] * xt)[..., None] * B[:, :, None, :]
                states.append(S)
            for t in range(min(t0 + K, most) - 1, t0 - 1, -1):
                k, i, dp, e, xt, B, C = token(t)
                g, old, new = dy[i], states[t - t0], states[t - t0 + 1]
                dS[:k] += g[..., None] * C[:, :, None, :]
                dC[i] = torch.matmul(g[:, :, None, :], new[:k])[:, :, 0].view(k, G, H // G, n).sum(2)
                xB = torch.matmul(dS[:k], B[..., None])[..., 0]
                dx[i] = dp[..., None] * xB + D[:, None] * g
                dB[i] = (dp[..., None] * torch.matmul(xt[:, :, None, :], dS[:k])[:, :, 0]).view(k, G, H // G, n).sum(2)
                dg = e * (dS[:k] * old[:k]).sum((2, 3))
                ddt[i] = (xt * xB).sum(-1) + A * dg
                dA += (A * dp * dg).sum(0)
                dS[:k] *= e[..., None, None]
        ddt = ddt * torch.sigmoid(raw)
        r = {"dx": dx, "dBm": dB, "dCm": dC, "ddt": ddt, "dA_log": dA, "ddt_bias": ddt.sum(0), "dD": (dy * x).sum((0, 2))}
        if s["pool"] is not None:
            r["dinit"] = dS[back]
        return r

    def norm(s):
        f = torch.float64
        leaves = {k: s[k].to(f).requires_grad_(s["op"] == "norm_bwd") for k in ("x", "w", "b", "z") if s[k] is not None}
        x, w, b, z = (leaves.get(k) for k in ("x", "w", "b", "z"))
        gate = z / (1 + torch.exp(-z)) if z is not None else None
        u = x * gate if z is not None and not s["after"] else x
        u = u.reshape(u.shape[0], s["groups"], -1)
        if s["op"] == "norm":
            mean = u.mean(-1) * (0.0 if s["rms"] else 1.0)
            rstd = 1 / torch.sqrt(((u - mean[..., None]) ** 2).mean(-1) + EPS)
        else:  # the backward pass is that of the norm at the statistics it is given, which follow u
            mean = s["mean"].to(f) + (0.0 if s["rms"] else (u - u.detach()).mean(-1))
            var = s["rstd"].to(f) ** -2 + (((u - mean[..., None]) ** 2).mean(-1) - ((u - mean[..., None]) ** 2).mean(-1).detach())
            rstd = var ** -0.5
        y = ((u - mean[..., None]) * rstd[..., None]).reshape(x.shape) * w
        y = y + b if b is not None else y
        y = y * gate if s["after"] else y
        if s["op"] == "norm":
            return {"y": y, "mean": mean, "rstd": rstd}
        names = [k for k in ("x", "w", "b", "z") if k in leaves]
        return dict(zip(["d" + k for k in names], torch.autograd.grad(y, [leaves[k] for k in names], s["dy"].to(f))))

    s = prepare(case, seed)
    return scan(s) if case["op"].startswith("scan") else norm(s)
