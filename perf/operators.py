"""Cases of the token-mixer operators beside the KDA scan: linear attention with a decay per head (whole
sequences, their gradients, single tokens), rotary positions over (t, h, w), and layer norm with its gradients.

``run`` computes a case in elementary torch operations (fp32, angles in fp64) where ``own`` is false, and through
``linear_attention_video_b200`` where it is true; ``exact`` computes it in fp64 from the definition.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
CHUNK = 256   # chunk of the plain form of linear attention
BASE = 10000.0


def listed():
    return [
        # one token of every running sequence: latency and the states' bandwidth
        dict(name="step_b1_f32", op="step", B=1, H=16, d=64, dtype="f32"),
        dict(name="step_b256_bf16", op="step", B=256, H=16, d=128, dtype="bf16"),
        # prompts of different lengths in one padded batch, entering with a state
        dict(name="linear_fwd_prompts_bf16", op="linear_fwd", B=8, H=16, d=128, N=2000, dtype="bf16", ragged=True, state=True),
        # a short odd sequence in fp32
        dict(name="linear_fwd_odd_f32", op="linear_fwd", B=2, H=6, d=64, N=1237, dtype="f32", ragged=False, state=False),
        # the token streams of a 5 s and a 30 s clip at 480x832 (512 text tokens + 21 or 121 frames of 30 x 52)
        dict(name="linear_fwd_video_30s_bf16", op="linear_fwd", B=1, H=16, d=128, N=189272, dtype="bf16", ragged=False, state=False),
        dict(name="linear_bwd_video_5s_bf16", op="linear_bwd", B=1, H=16, d=128, N=33272, dtype="bf16", ragged=False, state=False),
        # training on a padded batch of fp32 sequences that enter with a state
        dict(name="linear_bwd_ragged_f32", op="linear_bwd", B=3, H=8, d=64, N=777, dtype="f32", ragged=True, state=True),
        # the queries and keys of one decoded token per sequence, at far positions
        dict(name="rope_token_bf16", op="rope_fwd", B=64, H=16, d=128, text=1, T=0, Hg=0, Wg=0, dtype="bf16", given=True, interleaved=False),
        # the 5 s clip's queries and keys, positions from the grid
        dict(name="rope_video_5s_bf16", op="rope_fwd", B=1, H=16, d=128, text=512, T=21, Hg=30, Wg=52, dtype="bf16", given=False, interleaved=False),
        # gradients of fp32 queries and keys over small odd grids
        dict(name="rope_bwd_odd_f32", op="rope_bwd", B=2, H=6, d=64, text=77, T=5, Hg=13, Wg=17, dtype="f32", given=False, interleaved=True),
        # the norm before the mixer of the 5 s clip, width 16 heads x 128
        dict(name="norm_fwd_video_5s_bf16", op="norm_fwd", rows=33272, cols=2048, dtype="bf16"),
        # its gradients, the weight's and the bias's sums among them
        dict(name="norm_bwd_video_5s_bf16", op="norm_bwd", rows=33272, cols=2048, dtype="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "linear_fwd", "linear_bwd", "rope_fwd", "rope_bwd", "norm_fwd", "norm_bwd"])
    dtype, d, H = rng.choice(["bf16", "f32"]), rng.choice([64, 128]), rng.randint(1, 24)
    if op == "step":
        return dict(op=op, B=_between(rng, 1, 256), H=H, d=d, dtype=dtype)
    if op in ("linear_fwd", "linear_bwd"):
        B = _between(rng, 1, 16)
        return dict(op=op, B=B, H=H, d=d, N=_between(rng, 1, (40000 if op == "linear_fwd" else 20000) // B), dtype=dtype, ragged=rng.random() < 0.5, state=rng.random() < 0.5)
    if op in ("rope_fwd", "rope_bwd"):
        grid = (0, 0, 0) if rng.random() < 0.25 else (_between(rng, 1, 24), _between(rng, 1, 32), _between(rng, 1, 52))
        text = _between(rng, 1, 2000) if grid[0] == 0 else rng.choice([0, _between(rng, 1, 600)])
        return dict(op=op, B=_between(rng, 1, 4), H=H, d=d, text=text, T=grid[0], Hg=grid[1], Wg=grid[2], dtype=dtype,
                    given=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    cols = _between(rng, 32, 8192)
    return dict(op=op, rows=_between(rng, 1, min(100000, 100_000_000 // cols)), cols=cols, dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _decays(H):
    """log decays from quickly to slowly forgetting heads: halves of a nat down to 2^-8."""
    return torch.tensor([-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)], dtype=torch.float32, device="cuda")


def _pairs(d):
    """Rotated pairs of the t, h and w axes: a quarter for time, the rest split between height and width."""
    t = d // 8
    h = (d // 2 - t) // 2
    return t, h, d // 2 - t - h


def _inv_freq(d):
    """Each axis has a ladder of frequencies of its own."""
    parts = [torch.tensor([BASE ** (-j / n) for j in range(n)], dtype=torch.float64) for n in _pairs(d)]
    return torch.cat(parts).to(torch.float32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(case=case)
    op = case["op"]
    if op == "step":
        B, H, d = case["B"], case["H"], case["d"]
        s.update(q=normal(B, 1, H, d, scale=d ** -0.5), k=normal(B, 1, H, d), v=normal(B, 1, H, d), log_decay=_decays(H),
                 state=normal(B, H, d, d, scale=4.0, dtype=torch.float32))
    elif op in ("linear_fwd", "linear_bwd"):
        B, H, d, N = case["B"], case["H"], case["d"], case["N"]
        s.update(q=normal(B, N, H, d, scale=d ** -0.5), k=normal(B, N, H, d), v=normal(B, N, H, d), log_decay=_decays(H))
        s["lengths"] = None
        if case["ragged"]:   # one item fills the batch, the others are shorter
            n = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            n[0] = N
            s["lengths"] = n
        s["state"] = normal(B, H, d, d, dtype=torch.float32) if case["state"] else None
        if op == "linear_bwd":
            s["d_o"] = normal(B, N, H, d)
            s["d_final"] = normal(B, H, d, d, scale=0.1, dtype=torch.float32) if case["state"] else None
    elif op in ("rope_fwd", "rope_bwd"):
        B, H, d = case["B"], case["H"], case["d"]
        N = case["text"] + case["T"] * case["Hg"] * case["Wg"]
        s.update(q=normal(B, N, H, d), k=normal(B, N, H, d), inv_freq=_inv_freq(d))
        s["positions"] = None
        if case["given"]:   # far along in a long stream
            start = torch.randint(0, 250000, (B, 1, 1), generator=g, device="cuda")
            step = torch.randint(0, 2, (B, N, 3), generator=g, device="cuda").cumsum(1)
            s["positions"] = (start + step).to(torch.int32)
    else:
        R, D = case["rows"], case["cols"]
        x = torch.randn(R, D, generator=g, device="cuda")
        x = (x * torch.rand(R, 1, generator=g, device="cuda").add_(0.5) + torch.randn(R, 1, generator=g, device="cuda")).to(dt)
        s.update(x=x, weight=normal(D, scale=0.2, dtype=torch.float32).add_(1.0), bias=normal(D, scale=0.2, dtype=torch.float32))
        if op == "norm_bwd":
            s["dy"] = normal(R, D)
            x64 = x.double()
            mean = x64.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (x64.var(1, unbiased=False) + EPS).rsqrt().float()
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import linear_attention_video_b200 as kda
    c, op = s["case"], s["case"]["op"]
    dt = DT[c["dtype"]]
    new = torch.empty_like
    if op in ("norm_fwd", "norm_bwd"):
        x = s["x"]
        if op == "norm_fwd":
            y, mean, rstd = new(x), x.new_empty(x.shape[0], dtype=torch.float32), x.new_empty(x.shape[0], dtype=torch.float32)
            kda.kda_layernorm_fwd(x, y, s["weight"], s["bias"], EPS, mean, rstd)
            return y, mean, rstd
        if "ws" not in s:
            s["ws"] = kda.alloc_layernorm_bwd_workspace(x.shape[0], x.shape[1])
        dx, dw, db = new(x), new(s["weight"]), new(s["bias"])
        kda.kda_layernorm_bwd(s["dy"], x, s["mean"], s["rstd"], dx, s["ws"], s["weight"], dw, db)
        return dx, dw, db
    if "p" not in s:   # what a user's program keeps: the problem, and the workspace where there is one
        text, grid = (c["text"], (c["T"], c["Hg"], c["Wg"])) if op.startswith("rope") else (c.get("N", 1), (0, 0, 0))
        s["p"] = kda.problem(c["B"], c["H"], c["d"], text, grid)
        if op == "linear_fwd":
            s["ws"] = kda.alloc_linear_workspace(s["p"], dt)
        elif op == "linear_bwd":
            s["ws"] = kda.alloc_linear_bwd_workspace(s["p"], dt)
        elif op.startswith("rope"):
            s["rope"] = kda.rope(_pairs(c["d"]), interleaved=c["interleaved"])
    p = s["p"]
    if op == "step":
        o, out = new(s["v"]), new(s["state"])
        kda.kda_linear_step(p, s["q"], s["k"], s["v"], s["log_decay"], s["state"], o, out)
        return o, out
    if op == "linear_fwd":
        o, final = new(s["v"]), s["q"].new_empty(c["B"], c["H"], c["d"], c["d"], dtype=torch.float32)
        kda.kda_linear_fwd(p, s["q"], s["k"], s["v"], s["log_decay"], o, s["ws"], lengths=s["lengths"],
                           initial_state=s["state"], final_state=final)
        return o, final
    if op == "linear_bwd":
        dq, dk, dv = new(s["q"]), new(s["k"]), new(s["v"])
        d_initial = s["q"].new_empty(c["B"], c["H"], c["d"], c["d"], dtype=torch.float32)
        kda.kda_linear_bwd(p, s["q"], s["k"], s["v"], s["log_decay"], s["d_o"], dq, dk, dv, s["ws"], lengths=s["lengths"],
                           initial_state=s["state"], d_final_state=s["d_final"], d_initial_state=d_initial)
        return dq, dk, dv, d_initial
    q, k = new(s["q"]), new(s["k"])
    call = kda.kda_rope_fwd if op == "rope_fwd" else kda.kda_rope_bwd
    call(p, s["rope"], s["q"], s["k"], s["inv_freq"], q, k, positions=s["positions"])
    return q, k


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _powers(log_decay, n):
    """lam^n for whole numbers n >= 0 (any shape), per head: [H, *n.shape] fp32, computed in 64 bits."""
    shape = (-1,) + (1,) * n.dim()
    return torch.exp(log_decay.double().view(shape) * n.double().unsqueeze(0)).float()


def _chunks(x, C):
    """[B, N, H, d] (zero rows behind) -> [B, H, n, C, d] fp32."""
    B, N, H, d = x.shape
    n = -(-N // C)
    y = torch.zeros(B, n * C, H, d, dtype=torch.float32, device=x.device)
    y[:, :N] = x
    return y.view(B, n, C, H, d).permute(0, 3, 1, 2, 4)


def _flat(y, N):
    B, H, n, C, d = y.shape
    return y.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, d)[:, :N]


def _until(x, lengths):
    if lengths is None:
        return x
    keep = torch.arange(x.shape[1], device=x.device).view(1, -1, 1, 1) < lengths.view(-1, 1, 1, 1)
    return torch.where(keep, x, torch.zeros((), dtype=x.dtype, device=x.device))


def _lengths(s):
    c = s["case"]
    return torch.full((c["B"],), c["N"], device="cuda") if s["lengths"] is None else s["lengths"].long()


def _carried(local, log_decay, C, reverse):
    """What enters each chunk of what the chunks before it (behind it, if reverse) left, decayed: local [B, H, n, d, d]."""
    B, H, n, d, _ = local.shape
    i = torch.arange(n, device=local.device)
    gap = (i.view(-1, 1) - i.view(1, -1) - 1) if not reverse else (i.view(1, -1) - i.view(-1, 1) - 1)
    w = torch.where(gap >= 0, _powers(log_decay, gap.clamp(min=0) * C), torch.zeros((), device=local.device))
    return (w.unsqueeze(0) @ local.reshape(B, H, n, d * d)).view(B, H, n, d, d)


def _plain_linear(s):
    c, ld, N, n = s["case"], s["log_decay"], s["case"]["N"], _lengths(s)
    C = min(CHUNK, N)
    dev = ld.device
    q, k, v = (_chunks(_until(s[x], s["lengths"]), C) for x in "qkv")
    i = torch.arange(C, device=dev)
    gap = i.view(-1, 1) - i.view(1, -1)
    D = torch.where(gap >= 0, _powers(ld, gap.clamp(min=0)), torch.zeros((), device=dev)).unsqueeze(1)   # [H, 1, C, C]
    into = _powers(ld, i + 1).view(1, -1, 1, C, 1)        # lam^(i+1): from the state that enters
    outof = _powers(ld, C - 1 - i).view(1, -1, 1, C, 1)   # lam^(C-1-j): to the state that leaves
    S = _carried(k.transpose(-1, -2) @ (v * outof), ld, C, False)
    chunk = torch.arange(q.shape[2], device=dev)
    if s["state"] is not None:
        S = S + _powers(ld, chunk * C).view(1, -1, q.shape[2], 1, 1) * s["state"].unsqueeze(2)
    token = torch.arange(q.shape[2] * C, device=dev)
    left = (n.view(-1, 1) - 1 - token.view(1, -1))        # tokens between this one and the last
    end = torch.where(left >= 0, _powers(ld, left.clamp(min=0)), torch.zeros((), device=dev))   # [H, B, tokens]
    end = end.transpose(0, 1).reshape(c["B"], c["H"], q.shape[2], C, 1)
    whole = _powers(ld, n).t().view(c["B"], c["H"], 1, 1)
    if c["op"] == "linear_fwd":
        o = (D * (q @ k.transpose(-1, -2))) @ v + into * (q @ S)
        final = (k.transpose(-1, -2) @ (v * end)).sum(2)
        if s["state"] is not None:
            final = final + whole * s["state"]
        return _until(_flat(o, N), s["lengths"]).to(s["v"].dtype), final
    g = _chunks(_until(s["d_o"], s["lengths"]), C)
    local = (q * into).transpose(-1, -2) @ g              # [B, H, n, d, d]: reaches the state before the chunk
    G = _carried(local, ld, C, True)
    dq = (D * (g @ v.transpose(-1, -2))) @ k + into * (g @ S.transpose(-1, -2))
    dk = (D * (g @ v.transpose(-1, -2))).transpose(-1, -2) @ q + outof * (v @ G.transpose(-1, -2))
    dv = (D * (q @ k.transpose(-1, -2))).transpose(-1, -2) @ g + outof * (k @ G)
    first = (_powers(ld, chunk * C).view(1, -1, q.shape[2], 1, 1) * local).sum(2)
    if s["d_final"] is not None:
        F = s["d_final"].unsqueeze(2)
        dk = dk + end * (v @ F.transpose(-1, -2))
        dv = dv + end * (k @ F)
        first = first + whole * s["d_final"]
    dt = s["q"].dtype
    return tuple(_until(_flat(x, N), s["lengths"]).to(dt) for x in (dq, dk, dv)) + (first,)


def _grid_positions(c, dev):
    """Text token i at (i, i, i); the grid starts at text on every axis."""
    text, T, Hg, Wg = c["text"], c["T"], c["Hg"], c["Wg"]
    a = torch.arange(text, device=dev).view(-1, 1).expand(-1, 3)
    m = torch.arange(T * Hg * Wg, device=dev)
    hw = max(1, Hg * Wg)
    b = torch.stack([m // hw, m % hw // max(1, Wg), m % max(1, Wg)], 1) + text
    return torch.cat([a, b]).unsqueeze(0)


def _axis_of_pair(d, dev):
    return torch.repeat_interleave(torch.arange(3, device=dev), torch.tensor(_pairs(d), device=dev))


def _plain_rope(s):
    c = s["case"]
    d, dev = c["d"], s["q"].device
    pos = _grid_positions(c, dev) if s["positions"] is None else s["positions"]
    angle = pos.double()[:, :, _axis_of_pair(d, dev)] * s["inv_freq"].double()
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    if c["op"] == "rope_bwd":
        sin = -sin
    out = []
    for x in (s["q"], s["k"]):
        y = x.float()
        a, b = (y[..., 0::2], y[..., 1::2]) if c["interleaved"] else (y[..., : d // 2], y[..., d // 2:])
        z = (a * cos - b * sin, a * sin + b * cos)
        y = torch.stack(z, -1).flatten(-2) if c["interleaved"] else torch.cat(z, -1)
        out.append(y.to(x.dtype))
    return tuple(out)


def _plain_norm(s):
    x = s["x"].float()
    if s["case"]["op"] == "norm_fwd":
        mean = x.mean(1)
        r = x - mean.unsqueeze(1)
        rstd = 1 / torch.sqrt((r * r).mean(1) + EPS)
        return (r * rstd.unsqueeze(1) * s["weight"] + s["bias"]).to(s["x"].dtype), mean, rstd
    dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
    h = (x - s["mean"].unsqueeze(1)) * rstd
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * h).sum(0), dy.sum(0)


def _plain_step(s):
    lam = torch.exp(s["log_decay"].double()).float().view(1, -1, 1, 1)
    q, k, v = (s[x][:, 0].float() for x in "qkv")
    state = lam * s["state"] + k.unsqueeze(-1) * v.unsqueeze(-2)
    o = (state * q.unsqueeze(-1)).sum(-2)
    return o.unsqueeze(1).to(s["v"].dtype), state


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "step":
        return _plain_step(state)
    if op.startswith("linear"):
        return _plain_linear(state)
    return _plain_rope(state) if op.startswith("rope") else _plain_norm(state)


# ---------------------------------------------------------------------------
# work and the definitions in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        n = case["rows"] * case["cols"]
        return {"bytes": n * e * (2 if op == "norm_fwd" else 3) + 8 * case["rows"] + 8 * case["cols"],
                "flops": n * (8 if op == "norm_fwd" else 14)}
    B, H, d = case["B"], case["H"], case["d"]
    if op == "step":
        return {"bytes": B * H * (8 * d * d + 4 * d * e), "flops": 5 * B * H * d * d}
    if op.startswith("rope"):
        N = case["text"] + case["T"] * case["Hg"] * case["Wg"]
        return {"bytes": 4 * B * N * H * d * e + (12 * B * N if case["given"] else 0), "flops": 6 * B * N * H * d}
    rows, states = B * case["N"] * H, B * H * d * d * 4   # the recurrent form: 4 d^2 a token forward, 10 d^2 backward
    if op == "linear_fwd":
        return {"bytes": 4 * rows * d * e + states * (2 if case["state"] else 1), "flops": 4 * rows * d * d}
    return {"bytes": 7 * rows * d * e + states * (3 if case["state"] else 1), "flops": 10 * rows * d * d}


def _exact_linear(s):
    """Token by token, as the recurrence is written."""
    c = s["case"]
    B, H, d, N = c["B"], c["H"], c["d"], c["N"]
    lam = s["log_decay"].double().exp().view(1, H, 1, 1)
    n = _lengths(s).view(B, 1, 1, 1)
    q, k, v = (s[x].double().permute(1, 0, 2, 3).contiguous() for x in "qkv")
    ragged = s["lengths"] is not None
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    back = c["op"] == "linear_bwd"
    do = s["d_o"].double().permute(1, 0, 2, 3).contiguous() if back else None
    read = torch.zeros_like(q)   # o, or dq
    for t in range(N):
        new = torch.addcmul(lam * S, k[t].unsqueeze(-1), v[t].unsqueeze(-2))
        S = torch.where(t < n, new, S) if ragged else new
        if back:
            read[t] = torch.matmul(S, do[t].unsqueeze(-1)).squeeze(-1)
        else:
            read[t] = torch.matmul(q[t].unsqueeze(-2), S).squeeze(-2)
    live = (torch.arange(N, device="cuda").view(-1, 1, 1, 1) < n.view(1, B, 1, 1)) if ragged else torch.ones((), dtype=torch.bool, device="cuda")
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    tidy = lambda x: torch.where(live, x, zero).permute(1, 0, 2, 3)   # noqa: E731
    if not back:
        return tidy(read), S
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    G = torch.zeros_like(S) if s["d_final"] is None else s["d_final"].double()   # gradient of S_t
    for t in range(N - 1, -1, -1):
        at = torch.addcmul(G, q[t].unsqueeze(-1), do[t].unsqueeze(-2))
        dk[t] = torch.matmul(at, v[t].unsqueeze(-1)).squeeze(-1)
        dv[t] = torch.matmul(k[t].unsqueeze(-2), at).squeeze(-2)
        G = torch.where(t < n, lam * at, G) if ragged else lam * at
    return tidy(read), tidy(dk), tidy(dv), G


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("linear"):
        return _exact_linear(s)
    if op == "step":
        lam = s["log_decay"].double().exp()
        q, k, v = (s[x].double().squeeze(1) for x in "qkv")
        state = torch.einsum("h,bhij->bhij", lam, s["state"].double()) + torch.einsum("bhi,bhj->bhij", k, v)
        return torch.einsum("bhi,bhij->bhj", q, state).unsqueeze(1), state
    if op.startswith("rope"):   # a rotation is a product of complex numbers
        d = case["d"]
        pos = (_grid_positions(case, s["q"].device) if s["positions"] is None else s["positions"]).double()
        parts = torch.split(s["inv_freq"].double(), _pairs(d))
        angle = torch.cat([pos[..., a:a + 1] * f for a, f in enumerate(parts)], -1).unsqueeze(2)
        turn = torch.polar(torch.ones_like(angle), angle if op == "rope_fwd" else -angle)
        out = []
        for x in (s["q"].double(), s["k"].double()):
            z = torch.complex(x[..., 0::2], x[..., 1::2]) if case["interleaved"] else torch.complex(x[..., : d // 2], x[..., d // 2:])
            z = torch.view_as_real(z * turn)
            out.append(z.flatten(-2) if case["interleaved"] else torch.cat([z[..., 0], z[..., 1]], -1))
        return tuple(out)
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    if op == "norm_fwd":
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + EPS).rsqrt()
        return (x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd
    dy, rstd = s["dy"].double(), s["rstd"].double()
    h = (x - s["mean"].double()[:, None]) * rstd[:, None]
    g, D = dy * w, x.shape[1]
    dx = (g - (g.sum(1, keepdim=True) + h * (g * h).sum(1, keepdim=True)) / D) * rstd[:, None]
    return dx, torch.einsum("rc,rc->c", dy, h), dy.sum(0)
