"""Linear attention with a fixed decay a head, its one-token form, and the norm and rotation of queries and keys in front of
it: cases, inputs and plain forms.

Five operators, named by a case's "op":

  scan      o_t = scale S_t^T q_t over packed sequences, S_t = e^g S_{t-1} + k_t v_t^T with one g a head, from and to slots of
            a state pool; q, k and v may have fewer heads than there are states
  scan_bwd  the gradients of that scan with respect to q, k, v and, where a case has states, the initial states
  step      one token for each sequence of a batch, states updated in their slots
  qk        RMS norm of every query and key head, with a weight, and the rotation by the token's position behind it, whose
            pairs are halves of the head or neighbours and follow one of several position axes
  qk_bwd    its gradients, the weights' summed over all tokens and heads

`own` False computes them in elementary torch operations, True by the library's kernels.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
Q = 64  # tokens a chunk of the plain scan
EPS = 1e-6


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


# ------------------------------------------------------------------ cases
def _scan(op, lens, H, Hq, Hk, Hv, d, dtype, state, **name):
    return dict(name, op=op, lens=lens, H=H, Hq=Hq, Hk=Hk, Hv=Hv, d=d, dtype=dtype, state=state)


def _step(B, H, Hq, Hk, Hv, d, dtype, state, **name):
    return dict(name, op="step", B=B, H=H, Hq=Hq, Hk=Hk, Hv=Hv, d=d, dtype=dtype, state=state)


def _qk(op, T, Hq, Hk, d, rot, pairs, axes, far, dtype, **name):
    return dict(name, op=op, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, pairs=pairs, axes=axes, far=far, dtype=dtype)


def listed():
    return [
        # a chat turn's few new tokens appended to one session: latency
        _scan("scan", "37", 16, 16, 16, 16, 64, "bf16", "f32", name="scan_turn"),
        # the prefill of four prompts through a layer of 32 heads of 128, two heads to a query and key
        _scan("scan", "1024,3000,8192,8192", 32, 16, 16, 32, 128, "bf16", "f32", name="scan_prefill"),
        # a serving step's mix of short and empty continuations, four query heads to a key and value, 16-bit states
        _scan("scan", "1,0,63,64,65,500,2,129,333,7,1024,1,90,255,0,611,1,48,200,1500", 32, 32, 8, 8, 64, "bf16", "bf16", name="scan_mix"),
        # one document in full precision
        _scan("scan", "4099", 24, 24, 24, 24, 64, "f32", "f32", name="scan_f32"),
        # a training step's batch of four sequences
        _scan("scan_bwd", "4096,4096,4096,4096", 32, 32, 32, 32, 128, "bf16", "none", name="scan_bwd_train"),
        # one long document whose state came from an earlier part and goes on into a later one, shared keys and values
        _scan("scan_bwd", "16385", 16, 16, 4, 4, 128, "bf16", "f32", name="scan_bwd_long"),
        # one session's next token: latency
        _step(1, 32, 16, 16, 32, 128, "bf16", "f32", name="step_one"),
        # a decode step of a full batch
        _step(256, 32, 16, 16, 32, 128, "bf16", "f32", name="step_batch"),
        # queries and keys of three sequences' next tokens, far into their contexts: latency
        _qk("qk", 3, 32, 8, 128, 128, "halves", 1, True, "bf16", name="qk_token"),
        # those of a prefill, half of each head rotated
        _qk("qk", 20408, 32, 16, 128, 64, "halves", 1, False, "bf16", name="qk_prefill"),
        # the backward pass of a training step
        _qk("qk_bwd", 16384, 32, 32, 128, 128, "halves", 1, False, "bf16", name="qk_bwd_train"),
        # a video's patches with time, height and width, full precision, neighbouring pairs, heads of 80
        _qk("qk_bwd", 4001, 16, 16, 80, 80, "neighbours", 3, False, "f32", name="qk_bwd_video"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    H = rng.choice([1, 2, 4, 6, 8, 12, 16, 24, 32, 40, 64])
    share = lambda: H // rng.choice([v for v in (1, 1, 1, 2, 4, H) if H % v == 0])  # noqa: E731
    return H, share(), share(), share()


def draw(rng):
    op = rng.choice(["scan", "scan_bwd", "step", "qk", "qk_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32", "f16"])
    if op == "step":
        H, Hq, Hk, Hv = _heads(rng)
        d = rng.choice([16, 32, 64, 128, 128])
        return _step(_log(rng, 1, max(2, min(1024, 256 * 32 * 128 * 128 // (H * d * d)))), H, Hq, Hk, Hv, d, dtype, rng.choice(["f32", "f32", "bf16", "f16"]))
    if op.startswith("scan"):
        H, Hq, Hk, Hv = _heads(rng)
        d = rng.choice([16, 32, 64, 64, 128, 128])
        most = 16384 * 32 * 128 * 128 // (1 if dtype == "bf16" else 8)
        tokens = _log(rng, 1, max(2, min(20000, most // (H * d * d))))
        cuts = sorted(rng.randint(0, tokens) for _ in range(rng.choice([0, 0, 1, 3, rng.randint(4, 24)])))
        ends = cuts + [tokens]
        lens = ",".join(str(b - a) for a, b in zip([0] + cuts, ends))
        return _scan(op, lens, H, Hq, Hk, Hv, d, dtype, rng.choice(["f32", "f32", dtype]) if op == "scan" else rng.choice(["none", "f32", dtype]))
    Hk = rng.choice([1, 2, 4, 8, 16, 32])
    Hq = Hk * rng.choice([1, 1, 2, 4, 8])
    d = rng.choice([32, 64, 80, 96, 128, 128, 128, 192, 256])
    rot = rng.choice([d, d, d // 16 * 8, 16])
    T = _log(rng, 1, max(2, min(50000, 16384 * 64 * 128 // (2 if dtype == "f32" else 1) // ((Hq + Hk) * d))))
    return _qk(op, T, Hq, Hk, d, rot, rng.choice(["halves", "halves", "neighbours"]), rng.choice([1, 1, 3]), rng.random() < 0.3, dtype)


# ------------------------------------------------------------------ inputs
def _randn(gen, shape, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32) * scale + shift


def _log_decay(H):
    """Slopes that halve over the heads in equal ratios, from a memory of about one token to one of about 256."""
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H).float().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DT[case["dtype"]], case["op"]
    if op in ("scan", "scan_bwd", "step"):
        H, Hq, Hk, Hv, d = (case[k] for k in ("H", "Hq", "Hk", "Hv", "d"))
        lens = _lens(case) if op != "step" else [1] * case["B"]
        T, N = sum(lens), len(lens)
        # values come out of a projection together with the output's gate, so their rows are apart, but for the single tokens
        wide = _randn(gen, (T, (1 if op == "step" else 2) * Hv * d)).to(dt)
        s = dict(op=op, lens=lens, q=_randn(gen, (T, Hq, d)).to(dt), k=_randn(gen, (T, Hk, d)).to(dt), wide=wide, Hv=Hv, d=d, H=H,
                 g=_log_decay(H), pool=None, slots=None, dfinal=None)
        if op != "step":
            cu = torch.zeros(N + 1, dtype=torch.int32)
            cu[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
            s["cu"] = cu.cuda()
        if case["state"] != "none":
            s["pool"] = _randn(gen, (N + 2, H, d, d), 2.0).to(DT[case["state"]])
            s["slots"] = torch.randperm(N + 2, generator=gen, device="cuda")[:N].to(torch.int32)
        if op == "scan_bwd":
            s["do"] = _randn(gen, (T, H, d), 0.05).to(dt)
            if case["state"] != "none":
                s["dfinal"] = _randn(gen, (N, H, d, d), 0.05)
        return s
    T, Hq, Hk, d, rot = (case[k] for k in ("T", "Hq", "Hk", "d", "rot"))
    # queries, keys and values come out of one projection
    s = dict(op=op, rows=_randn(gen, (T, (Hq + 2 * Hk) * d), 1.5).to(dt), Hq=Hq, Hk=Hk, d=d, rot=rot, neighbours=case["pairs"] == "neighbours",
             qw=_randn(gen, (d,), 0.1, 1.0), kw=_randn(gen, (d,), 0.1, 1.0), axes=None,
             freq=(1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda())
    start = torch.randint(0, 1000000 if case["far"] else 2, (1,), generator=gen, device="cuda")
    pos = torch.arange(T, device="cuda") % 8192 + start
    if case["axes"] > 1:  # a third of the pairs for time, then height and width in turn; frames of 26 x 34 patches
        P = rot // 2
        s["axes"] = [0 if i < P // 3 else 1 + (i - P // 3) % 2 for i in range(P)]
        i = torch.arange(T, device="cuda")
        pos = torch.stack([start + i // 884, start + i // 34 % 26, start + i % 34])
    s["pos"] = pos.to(torch.int32)
    if op == "qk_bwd":
        s["dq"], s["dk"] = _randn(gen, (T, Hq, d), 0.05).to(dt), _randn(gen, (T, Hk, d), 0.05).to(dt)
    return s


def _values(s):
    return s["wide"][:, : s["Hv"] * s["d"]].unflatten(1, (s["Hv"], s["d"]))


def _queries_keys(s):
    a, b, d = s["Hq"] * s["d"], (s["Hq"] + s["Hk"]) * s["d"], s["d"]
    return s["rows"][:, :a].unflatten(1, (s["Hq"], d)), s["rows"][:, a:b].unflatten(1, (s["Hk"], d))


# ------------------------------------------------------------------ plain forms
def _scan_plain(lens, cu, q, k, v, g, S0):
    """The scan in chunks of Q tokens: products inside a chunk, and the states between chunks by one product with the matrix of the
    decays from chunk to chunk.  q, k, v [T, own heads, d] in 32 bits, S0 [sequences, H, d, d].  Returns o and the final states."""
    (T, _, d), H, N, dev = q.shape, g.shape[0], len(lens), q.device
    scale = d ** -0.5
    nc = sum(-(-n // Q) for n in lens)
    if nc == 0:
        return torch.zeros((T, H, d), device=dev), S0
    count = (cu[1:] - cu[:-1] + Q - 1).div(Q, rounding_mode="floor").long()
    first = count.cumsum(0) - count
    seq = torch.repeat_interleave(torch.arange(N, device=dev), count, output_size=nc)
    tok = cu[seq].long()[:, None] + (torch.arange(nc, device=dev) - first[seq])[:, None] * Q + torch.arange(Q, device=dev)
    end = cu[seq + 1].long()
    live = tok < end[:, None]
    at = tok.clamp(max=T - 1)
    size = live.sum(1)                                                      # tokens of each chunk
    g = g.double()

    def chunks(x):                                                          # [nc, H, Q, d]
        return torch.where(live[..., None, None], x[at], 0.0).transpose(1, 2).repeat_interleave(H // x.shape[1], 1)

    Qc, Kc, Vc = chunks(q), chunks(k), chunks(v)
    i = torch.arange(Q, device=dev)
    L = torch.exp(torch.where(i[:, None] >= i, g[:, None, None] * (i[:, None] - i), -math.inf)).float()
    o = torch.matmul(torch.matmul(Qc, Kc.transpose(2, 3).contiguous()) * L, Vc)
    left = (size[:, None] - 1 - i).clamp(min=0)                             # tokens behind, in the chunk
    w = torch.exp(g[:, None] * left[:, None]).float()                       # [nc, H, Q]
    Z = torch.matmul((Kc * w[..., None]).transpose(2, 3).contiguous(), Vc)  # [nc, H, d, d]
    total = size.cumsum(0)
    before = total - size
    order = torch.arange(nc, device=dev)
    earlier = (order[:, None] > order[None, :]) & (seq[:, None] == seq[None, :])
    M = torch.exp(torch.where(earlier, g[:, None, None] * (before[:, None] - total[None, :]), -math.inf)).float()
    S = torch.matmul(M, Z.transpose(0, 1).reshape(H, nc, d * d)).view(H, nc, d, d).transpose(0, 1)
    gone = (before - before[first.clamp(max=nc - 1)][seq])[:, None] * g     # [nc, H]
    S = S + torch.exp(gone).float()[..., None, None] * S0[seq]
    o = o + torch.exp(g[:, None] * (i + 1)).float()[..., None] * torch.matmul(Qc, S)
    out = torch.zeros((T, H, d), device=dev).index_put((tok[live],), o.transpose(1, 2)[live])
    last = (first + count - 1).clamp(min=0)
    behind = torch.exp(size[:, None] * g).float()[..., None, None] * S + Z
    return out * scale, torch.where((count > 0)[:, None, None, None], behind[last], S0)


def _rotate(x, s, back):
    """x [T, heads, d] in 32 bits, rotated by the tokens' positions (or back); angles in 64 bits."""
    rot, pos = s["rot"], s["pos"].double()
    angle = (pos[s["axes"]].t() if s["axes"] is not None else pos[:, None]) * s["freq"].double()
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    sn = -sn if back else sn
    if s["neighbours"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_plain(s):
    op = s["op"]
    if op in ("scan", "scan_bwd"):
        pool, slots, lens, H, d = s["pool"], s["slots"], s["lens"], s["H"], s["d"]
        S0 = pool[slots.long()].float() if pool is not None else torch.zeros((len(lens), H, d, d), device="cuda")
        if op == "scan":
            o, end = _scan_plain(lens, s["cu"], s["q"].float(), s["k"].float(), _values(s).float(), s["g"], S0)
            pool[slots.long()] = end.to(pool.dtype)
            return {"o": o.to(s["q"].dtype), "state": pool}
        leaves = [t.float().detach().requires_grad_() for t in (s["q"], s["k"], _values(s))] + [S0.requires_grad_()]
        with torch.enable_grad():
            o, end = _scan_plain(lens, s["cu"], *leaves[:3], s["g"], leaves[3])
        outs, grads = ([o], [s["do"].float()]) if s["dfinal"] is None else ([o, end], [s["do"].float(), s["dfinal"]])
        got = torch.autograd.grad(outs, leaves, grads)
        r = {n: t.to(s["q"].dtype) for n, t in zip(("dq", "dk", "dv"), got)}
        if pool is not None:
            r["dinit"] = got[-1]
        return r
    if op == "step":
        pool, slots, H, d = s["pool"], s["slots"].long(), s["H"], s["d"]
        q, k, v = (t.float().repeat_interleave(H // t.shape[1], 1) for t in (s["q"], s["k"], _values(s)))
        S = pool[slots].float() * torch.exp(s["g"])[:, None, None] + k[..., :, None] * v[..., None, :]
        pool[slots] = S.to(pool.dtype)
        return {"o": (q[..., :, None] * S).sum(-2) * d ** -0.5, "state": pool}
    r = {}
    for name, x, w in zip("qk", _queries_keys(s), (s["qw"], s["kw"])):
        u = x.float()
        rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
        if op == "qk":
            r[name] = _rotate(u * rstd * w, s, False).to(x.dtype)
            continue
        dn = _rotate(s["d" + name].float(), s, True)
        xh = u * rstd
        r["dw" + name] = (dn * xh).sum((0, 1))
        dh = dn * w
        r["d" + name] = ((dh - xh * (dh * xh).mean(-1, keepdim=True)) * rstd).to(x.dtype)
    return r


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import gated_deltanet_state_gdn_amd as gdn
    op = s["op"]
    if op == "scan":
        o = gdn.gdn_linear_scan(s["q"], s["k"], _values(s), s["g"], s["cu"], pool=s["pool"], slot_map=s["slots"])
        return {"o": o, "state": s["pool"]}
    if op == "scan_bwd":
        g = gdn.gdn_linear_scan_backward(s["do"], s["q"], s["k"], _values(s), s["g"], s["cu"], pool=s["pool"], slot_map=s["slots"], dfinal=s["dfinal"])
        r = {"dq": g.dq, "dk": g.dk, "dv": g.dv}
        if s["pool"] is not None:
            r["dinit"] = g.dinit
        return r
    if op == "step":
        return {"o": gdn.gdn_linear_decode_step(s["q"], s["k"], _values(s), s["g"], s["pool"], s["slots"]), "state": s["pool"]}
    q, k = _queries_keys(s)
    form = dict(eps=EPS, neighbours=s["neighbours"], axes=s["axes"])
    if op == "qk":
        q, k = gdn.gdn_qk_norm_rope(q, k, s["qw"], s["kw"], s["pos"], s["freq"], **form)
        return {"q": q, "k": k}
    g = gdn.gdn_qk_norm_rope_backward(s["dq"], s["dk"], q, k, s["qw"], s["kw"], s["pos"], s["freq"], **form)
    return {"dwq": g.dq_weight, "dq": g.dq, "dwk": g.dk_weight, "dk": g.dk}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b, op = SIZE[case["dtype"]], case["op"]
    if op in ("scan", "scan_bwd", "step"):
        lens = _lens(case) if op != "step" else [1] * case["B"]
        H, d = case["H"], case["d"]
        T, N = sum(lens), sum(v > 0 for v in lens)
        states = N * H * d * d
        ins = T * (case["Hq"] + case["Hk"] + case["Hv"]) * d * b
        if op != "scan_bwd":  # q, k, v in, o out, states both ways; per token and head a rank-one update and a read-out
            out = T * H * d * (b if op == "scan" else 4)
            return {"bytes": ins + out + 2 * states * SIZE[case["state"]], "flops": 4.0 * T * H * d * d}
        # inputs and do in, three gradients out; per token and head both states' updates and the three products with them
        extra = 0 if case["state"] == "none" else states * (SIZE[case["state"]] + 8)
        return {"bytes": 2 * ins + T * H * d * b + extra, "flops": 10.0 * T * H * d * d}
    n = case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
    pos = 4 * case["T"] * case["axes"]
    return {"bytes": (2 if op == "qk" else 3) * n * b + pos, "flops": (8.0 if op == "qk" else 16.0) * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    f = torch.float64

    def scan(s):
        """Every pair of tokens, a block of rows at a time: o_i = scale (sum_{j<=i} e^{g (i-j)} (q_i.k_j) v_j + e^{g (i+1)} S0^T q_i)."""
        H, d, dev = s["H"], s["d"], "cuda"
        heads = lambda t: t.to(f).transpose(0, 1).repeat_interleave(H // t.shape[1], 0)  # [H, T, d]  # noqa: E731
        back = s["op"] == "scan_bwd"
        q, k, v, g = heads(s["q"]), heads(s["k"]), heads(_values(s)), s["g"].to(f)
        do = heads(s["do"]) if back else None
        scale = 1 / math.sqrt(d)
        out = {n: torch.zeros_like(q) for n in (("dq", "dk", "dv") if back else ("o",))}
        pool = s["pool"].to(f) if s["pool"] is not None else None
        ends = torch.zeros((len(s["lens"]), H, d, d), dtype=f, device=dev)
        a = 0
        for n, T in enumerate(s["lens"]):
            at = slice(a, a + T)
            t = torch.arange(T, device=dev, dtype=f)
            S0 = pool[int(s["slots"][n])] if pool is not None else torch.zeros((H, d, d), dtype=f, device=dev)
            since = torch.exp(g[:, None] * (t + 1))[..., None]                 # [H, T, 1]
            until = torch.exp(g[:, None] * (T - 1 - t))[..., None]
            clear = torch.exp(g * T)[:, None, None]
            for r in range(0, T, 256):
                e = min(r + 256, T)
                rows, cols = slice(a + r, a + e), slice(a, a + e)
                diff = t[r:e, None] - t[None, :e]
                W = torch.where(diff >= 0, torch.exp(g[:, None, None] * diff.clamp(min=0)), 0.0)
                A = torch.bmm(q[:, rows], k[:, cols].transpose(1, 2).contiguous()) * W
                if not back:
                    out["o"][:, rows] = torch.bmm(A, v[:, cols].contiguous())
                    continue
                B = torch.bmm(do[:, rows].contiguous(), v[:, cols].transpose(1, 2).contiguous()) * W
                out["dq"][:, rows] = torch.bmm(B, k[:, cols].contiguous())
                out["dk"][:, cols] += torch.bmm(B.transpose(1, 2).contiguous(), q[:, rows].contiguous())
                out["dv"][:, cols] += torch.bmm(A.transpose(1, 2).contiguous(), do[:, rows].contiguous())
            if not back:
                out["o"][:, at] += since * torch.bmm(q[:, at].contiguous(), S0)
                ends[n] = clear * S0 + torch.bmm((k[:, at] * until).transpose(1, 2).contiguous(), v[:, at].contiguous())
            else:
                F = s["dfinal"][n].to(f) if s["dfinal"] is not None else torch.zeros_like(S0)
                out["dq"][:, at] += since * torch.bmm(do[:, at].contiguous(), S0.transpose(1, 2).contiguous())
                out["dk"][:, at] += until * torch.bmm(v[:, at].contiguous(), F.transpose(1, 2).contiguous()) / scale
                out["dv"][:, at] += until * torch.bmm(k[:, at].contiguous(), F) / scale
                ends[n] = clear * F + scale * torch.bmm((q[:, at] * since).transpose(1, 2).contiguous(), do[:, at].contiguous())
            a += T
        if not back:
            pool[s["slots"].long()] = ends
            return {"o": out["o"].transpose(0, 1) * scale, "state": pool}
        r = {}
        for name, like in zip(("dq", "dk", "dv"), (s["q"], s["k"], _values(s))):
            r[name] = scale * out[name].transpose(0, 1).reshape(-1, like.shape[1], H // like.shape[1], d).sum(2)
        if pool is not None:
            r["dinit"] = ends
        return r

    def step(s):
        H, d, slots = s["H"], s["d"], s["slots"].long()
        q, k, v = (t.to(f).repeat_interleave(H // t.shape[1], 1) for t in (s["q"], s["k"], _values(s)))
        pool = s["pool"].to(f)
        S = torch.exp(s["g"].to(f))[None, :, None, None] * pool[slots]
        S += torch.matmul(k[..., None], v[:, :, None, :])
        pool[slots] = S
        return {"o": torch.matmul(q[:, :, None, :], S)[:, :, 0] / math.sqrt(d), "state": pool}

    def qk(s):
        """Pairs as complex numbers, turned by e^{i angle}."""
        rot, d = s["rot"], s["d"]
        where = torch.tensor(s["axes"] if s["axes"] is not None else [0] * (rot // 2), device="cuda")
        pos = s["pos"].to(f) if s["axes"] is not None else s["pos"].to(f)[None]
        turn = torch.polar(torch.ones((), dtype=f, device="cuda"), pos[where].transpose(0, 1) * s["freq"].to(f))[:, None]
        i = torch.arange(rot // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if s["neighbours"] else (i, i + rot // 2)
        r = {}
        for name, x, w in zip("qk", _queries_keys(s), (s["qw"], s["kw"])):
            x, w = x.to(f).requires_grad_(), w.to(f).requires_grad_()
            with torch.enable_grad():
                n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
                z = torch.complex(n[..., first], n[..., second]) * turn
                y = n.index_copy(2, first, z.real).index_copy(2, second, z.imag)
            if s["op"] == "qk":
                r[name] = y.detach()
            else:
                r["d" + name], r["dw" + name] = torch.autograd.grad(y, (x, w), s["d" + name].to(f))
        return r if s["op"] == "qk" else {k: r[k] for k in ("dwq", "dq", "dwk", "dk")}

    s = prepare(case, seed)
    return {"scan": scan, "scan_bwd": scan, "step": step}.get(case["op"], qk)(s)
