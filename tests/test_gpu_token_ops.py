"""Rotary positions, layer norm and linear attention with a decay per head against the fp64 reference (B200).

Element-wise tolerances, from the roundings on the way: u |ref| for the output's own rounding (u = eps / 2), and c M
with M the same sum over absolute values.  fp32 work: c = 2^-16, the operand splits' 6 x 2^-22 and at most 200 additions
in sequence of 2^-24 each.  bf16 linear attention may round each decayed score (and the scaled rows beside a state) once
to bf16 before its second product: 2^-8 more.  Beside them the relative L2 bounds of the other parity tests.
"""
import itertools

import pytest
import torch

from oracle import token_ops as ops
from tests._util import TOL_BF16_REL_L2, TOL_F32_REL_L2

pytestmark = pytest.mark.gpu

C32 = 2.0 ** -16
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    import linear_attention_video_b200 as kda
    assert torch.cuda.is_available()
    return kda


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def close(got, ref, M, c, what=""):
    """|got - ref| <= u |ref| + c M, element by element, and the relative L2 bound of the type."""
    u = torch.finfo(got.dtype).eps / 2
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    err = (got.double() - ref).abs()
    bad = err > u * ref.abs() + c * M + 1e-37
    assert not bad.any(), (what, int(bad.sum()), float(err.max()))
    den = float(ref.norm())
    rel = float((got.double() - ref).norm()) / den if den else 0.0
    assert rel <= (TOL_BF16_REL_L2 if got.dtype == torch.bfloat16 else TOL_F32_REL_L2), (what, rel)


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def lin_inputs(seed, B, N, H, d, dtype, decays=None):
    g = gen(seed)
    x = {"q": randn(g, B, N, H, d, dtype=dtype, scale=d ** -0.5)}
    x.update({n: randn(g, B, N, H, d, dtype=dtype) for n in ("k", "v", "d_o")})
    ld = [-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)] if decays is None else decays
    x["ld"] = torch.tensor(ld, dtype=torch.float32, device="cuda")
    x["S0"], x["dSN"] = randn(g, B, H, d, d), randn(g, B, H, d, d)
    return x


def run_fwd(kda, x, lengths=None, state=True, final=True, ws=None, stream=None):
    B, N, H, d = x["q"].shape
    p = kda.problem(B, H, d, N, (0, 0, 0))
    o = torch.full_like(x["v"], float("nan"))
    SN = torch.full((B, H, d, d), float("nan"), device="cuda") if final else None
    ws = kda.alloc_linear_workspace(p, x["q"].dtype) if ws is None else ws
    kda.kda_linear_fwd(p, x["q"], x["k"], x["v"], x["ld"], o, ws, lengths=lengths,
                       initial_state=x["S0"] if state else None, final_state=SN, stream=stream)
    return o, SN, ws


def run_bwd(kda, x, lengths=None, state=True, first=True):
    B, N, H, d = x["q"].shape
    p = kda.problem(B, H, d, N, (0, 0, 0))
    dq, dk, dv = (torch.full_like(x[n], float("nan")) for n in "qkv")
    dS0 = torch.full((B, H, d, d), float("nan"), device="cuda") if first else None
    ws = kda.alloc_linear_bwd_workspace(p, x["q"].dtype)
    kda.kda_linear_bwd(p, x["q"], x["k"], x["v"], x["ld"], x["d_o"], dq, dk, dv, ws, lengths=lengths,
                       initial_state=x["S0"] if state else None, d_final_state=x["dSN"] if state else None,
                       d_initial_state=dS0)
    assert kda.kda_read_status(ws) == kda.KDA_OK
    return dq, dk, dv, dS0


def check_fwd(kda, x, lengths=None, state=True):
    o, SN, ws = run_fwd(kda, x, lengths, state)
    assert kda.kda_read_status(ws) == kda.KDA_OK
    S0 = x["S0"] if state else None
    ref = ops.linear_fwd(x["q"], x["k"], x["v"], x["ld"], lengths, S0)
    M = ops.linear_fwd(*(x[n].abs() for n in "qkv"), x["ld"], lengths, None if S0 is None else S0.abs())
    bf16 = x["q"].dtype == torch.bfloat16
    close(o, ref[0], M[0], C32 + (2.0 ** -8 if bf16 else 0.0), "o")
    close(SN, ref[1], M[1], C32, "final state")
    # without the states' arguments the rest is the same
    assert torch.equal(run_fwd(kda, x, lengths, state, final=False)[0], o)


def check_bwd(kda, x, lengths=None, state=True):
    got = run_bwd(kda, x, lengths, state)
    S0, dSN = (x["S0"], x["dSN"]) if state else (None, None)
    ref = ops.linear_bwd(x["q"], x["k"], x["v"], x["ld"], x["d_o"], lengths, S0, dSN)
    a = lambda t: None if t is None else t.abs()   # noqa: E731
    M = ops.linear_bwd(*(x[n].abs() for n in "qkv"), x["ld"], x["d_o"].abs(), lengths, a(S0), a(dSN))
    bf16 = x["q"].dtype == torch.bfloat16
    for name, g, r, m in zip(("dq", "dk", "dv", "dS0"), got, ref, M):
        close(g, r, m, C32 + (2.0 ** -8 if bf16 and name != "dS0" else 0.0), name)


# one token, inside a tile, at and across the borders of tiles and segments
SHAPES = [(1, 1, 1, 64), (2, 1, 3, 128), (1, 31, 2, 64), (2, 64, 2, 128), (1, 65, 3, 64), (1, 129, 2, 128),
          (2, 257, 2, 128), (1, 511, 1, 64), (1, 513, 2, 128), (2, 1000, 2, 64), (1, 2049, 2, 128), (1, 2500, 1, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,H,d", SHAPES)
def test_linear_fwd(kda, B, N, H, d, dtype):
    x = lin_inputs(N + d, B, N, H, d, DT[dtype])
    check_fwd(kda, x)
    check_fwd(kda, x, state=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,H,d", SHAPES)
def test_linear_bwd(kda, B, N, H, d, dtype):
    x = lin_inputs(N + d + 1, B, N, H, d, DT[dtype])
    check_bwd(kda, x)
    check_bwd(kda, x, state=False)


@pytest.mark.parametrize("dtype,d", list(itertools.product(["f32", "bf16"], [64, 128])))
def test_linear_ragged_batches_ignore_what_stands_behind(kda, dtype, d):
    """Lengths of 0, 1, around tile and segment borders, N and out of range; NaN and infinities behind the ends."""
    N = 1100
    n = [0, 1, 63, 64, 65, 127, 128, 129, 512, 513, 1024, 1099, 1100, 5000, -3]
    x = lin_inputs(5, len(n), N, 2, d, DT[dtype])
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    for b, m in enumerate(n):
        for i, name in enumerate(("q", "k", "v", "d_o")):
            x[name][b, max(0, min(m, N)):] = (float("nan"), float("inf"), -float("inf"), float("nan"))[(b + i) % 4]
    clean = {k: v.clone() for k, v in x.items()}
    for name in ("q", "k", "v", "d_o"):
        clean[name] = ops._until(x[name], lengths).to(x[name].dtype)
    bf16 = x["q"].dtype == torch.bfloat16
    ref = ops.linear_fwd(clean["q"], clean["k"], clean["v"], x["ld"], lengths, x["S0"])
    M = ops.linear_fwd(*(clean[i].abs() for i in "qkv"), x["ld"], lengths, x["S0"].abs())
    o, SN, _ = run_fwd(kda, x, lengths)
    close(o, ref[0], M[0], C32 + (2.0 ** -8 if bf16 else 0.0), "o")
    close(SN, ref[1], M[1], C32, "final state")
    assert torch.equal(SN[0], x["S0"][0]) and torch.equal(SN[-1], x["S0"][-1])
    ref = ops.linear_bwd(clean["q"], clean["k"], clean["v"], x["ld"], clean["d_o"], lengths, x["S0"], x["dSN"])
    M = ops.linear_bwd(*(clean[i].abs() for i in "qkv"), x["ld"], clean["d_o"].abs(), lengths, x["S0"].abs(), x["dSN"].abs())
    for name, g, r, m in zip(("dq", "dk", "dv", "dS0"), run_bwd(kda, x, lengths), ref, M):
        close(g, r, m, C32 + (2.0 ** -8 if bf16 and name != "dS0" else 0.0), name)
    for g in run_bwd(kda, x, lengths)[:3]:
        for b, m in enumerate(n):
            assert not g[b, max(0, min(m, N)):].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_extreme_decays(kda, dtype):
    """No decay, slow ones, ones that leave a token alone, minus infinity."""
    decays = [0.0, -1e-6, -1e-3, -3.0, -90.0, -1e4, -float("inf")]
    x = lin_inputs(6, 1, 700, len(decays), 64, DT[dtype], decays)
    check_fwd(kda, x)
    check_bwd(kda, x)


@pytest.mark.parametrize("dtype,d", list(itertools.product(["f32", "bf16"], [64, 128])))
def test_linear_magnitudes(kda, dtype, d):
    """Inputs far from 1: products stay in range of the type's exponent, whatever the scale of one operand."""
    for sq, sk, sv in ((1e4, 1e4, 1e-8), (1e-12, 1e15, 1.0), (1.0, 1e-15, 1e18)):
        x = lin_inputs(7, 1, 300, 2, d, torch.float32)
        x["q"], x["k"], x["v"] = x["q"] * sq, x["k"] * sk, x["v"] * sv
        x["d_o"] = x["d_o"] / sv
        x = {n: t.to(DT[dtype]) if n in ("q", "k", "v", "d_o") else t for n, t in x.items()}
        x["S0"] *= sk * sv
        x["dSN"] *= sq / sv
        check_fwd(kda, x)
        check_bwd(kda, x)


def test_linear_many_heads_and_items(kda):
    check_fwd(kda, lin_inputs(8, 19, 70, 13, 64, torch.bfloat16))
    check_bwd(kda, lin_inputs(9, 19, 70, 13, 128, torch.bfloat16))


def test_linear_empty_sequence_passes_the_states(kda):
    x = lin_inputs(10, 2, 1, 2, 64, torch.float32)
    p = kda.problem(2, 2, 64, 0, (0, 0, 0))
    ws, wb = kda.alloc_linear_workspace(p, torch.float32), kda.alloc_linear_bwd_workspace(p, torch.float32)
    e, SN = torch.empty(8, device="cuda"), torch.empty_like(x["S0"])
    e2, e3, e4 = (torch.empty(8, device="cuda") for _ in range(3))
    kda.kda_linear_fwd(p, e, e, e, x["ld"], e2, ws, initial_state=x["S0"], final_state=SN)
    assert torch.equal(SN, x["S0"])
    kda.kda_linear_bwd(p, e, e, e, x["ld"], e, e2, e3, e4, wb, d_final_state=x["dSN"], d_initial_state=SN)
    assert torch.equal(SN, x["dSN"])
    kda.kda_linear_fwd(p, e, e, e, x["ld"], e2, ws, final_state=SN)
    assert not SN.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_backward_against_differences(kda, dtype):
    """The gradients against differences of the GPU's own fp32 forward pass along random directions: with |o| known to
    2^-16 M and steps of 2^-4 of the inputs' scale (the loss is multilinear, so central differences are exact in it)."""
    x = lin_inputs(11, 2, 600, 2, 64, torch.float32)
    lengths = torch.tensor([600, 333], dtype=torch.int32, device="cuda")
    x = {n: t.to(DT[dtype]).float() if n in ("q", "k", "v", "d_o") else t for n, t in x.items()}
    keep = torch.arange(600, device="cuda").view(1, -1, 1, 1) < lengths.view(-1, 1, 1, 1)

    def loss(y):
        o, SN, _ = run_fwd(kda, y, lengths)
        return float((o.double() * x["d_o"].double() * keep).sum() + (SN.double() * x["dSN"].double()).sum())

    typed = {n: t.to(DT[dtype]) if n in ("q", "k", "v", "d_o") else t for n, t in x.items()}
    grads = dict(zip(("q", "k", "v", "S0"), run_bwd(kda, typed, lengths)))
    g, h = gen(12), 2.0 ** -4
    for name in ("q", "k", "v", "S0"):
        way = randn(g, *x[name].shape)
        at = lambda s: dict(x, **{name: x[name] + s * h * way})   # noqa: E731
        diff = (loss(at(1)) - loss(at(-1))) / (2 * h)
        mine = float((grads[name].double() * way.double()).sum())
        # a sum of n gradients along independent signs: rounding of each by u and of the sums by 2^-16 of their size
        scale = float((grads[name].double() * way.double()).norm())
        u = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -12
        assert abs(diff - mine) <= 8 * u * scale + 1e-4 * abs(mine), (name, diff, mine, scale)


@pytest.mark.parametrize("dtype,d", list(itertools.product(["f32", "bf16"], [64, 128])))
def test_linear_step(kda, dtype, d):
    for B, H in ((1, 1), (3, 5), (40, 16)):
        x = lin_inputs(13 + B, B, 1, H, d, DT[dtype])
        p = kda.problem(B, H, d, 1, (0, 0, 0))
        o, S = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
        kda.kda_linear_step(p, x["q"], x["k"], x["v"], x["ld"], x["S0"], o, S)
        ref = ops.linear_fwd(x["q"], x["k"], x["v"], x["ld"], None, x["S0"])
        M = ops.linear_fwd(*(x[n].abs() for n in "qkv"), x["ld"], None, x["S0"].abs())
        close(o, ref[0], M[0], C32, "o")
        close(S, ref[1], M[1], C32, "state")
        again, o2 = x["S0"].clone(), torch.empty_like(o)
        kda.kda_linear_step(p, x["q"], x["k"], x["v"], x["ld"], again, o2, again)   # in place
        assert torch.equal(again, S) and torch.equal(o2, o)


def test_prompt_then_tokens_equal_the_whole_sequence(kda):
    """Prompts of different lengths, then one token at a time from the states they left, against the whole sequences."""
    B, N, H, d, more = 3, 200, 4, 128, 5
    x = lin_inputs(14, B, N + more, H, d, torch.bfloat16)
    n = torch.tensor([200, 17, 128], dtype=torch.int32, device="cuda")
    prompt = {k: v[:, :N].contiguous() if k in ("q", "k", "v") else v for k, v in x.items()}
    _, S, _ = run_fwd(kda, prompt, n)
    p, outs = kda.problem(B, H, d, 1, (0, 0, 0)), []
    rows = torch.arange(B, device="cuda")
    for t in range(more):
        tok = {i: x[i][rows, n.long() + t].unsqueeze(1).contiguous() for i in "qkv"}
        o = torch.empty_like(tok["v"])
        kda.kda_linear_step(p, tok["q"], tok["k"], tok["v"], x["ld"], S, o, S)
        outs.append(o)
    ref, refS = ops.linear_fwd(x["q"], x["k"], x["v"], x["ld"], n + more, x["S0"])
    M, MS = ops.linear_fwd(*(x[i].abs() for i in "qkv"), x["ld"], n + more, x["S0"].abs())
    for t, o in enumerate(outs):
        at = (rows, n.long() + t)
        close(o[:, 0], ref[at], M[at], C32, f"token {t}")
    close(S, refS, MS, C32, "state")


def test_linear_side_stream_graph_and_shared_workspace(kda):
    """Captured once and replayed on new inputs; two graphs on one stream may share a workspace; a side stream."""
    x = lin_inputs(15, 1, 1500, 2, 128, torch.bfloat16)
    p = kda.problem(1, 2, 128, 1500, (0, 0, 0))
    ws, wb = kda.alloc_linear_workspace(p, torch.bfloat16), kda.alloc_linear_bwd_workspace(p, torch.bfloat16)
    o, SN = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    grads = [torch.empty_like(x[n]) for n in "qkv"]

    def fwd():
        kda.kda_linear_fwd(p, x["q"], x["k"], x["v"], x["ld"], o, ws, initial_state=x["S0"], final_state=SN)

    def bwd():
        kda.kda_linear_bwd(p, x["q"], x["k"], x["v"], x["ld"], x["d_o"], *grads, wb, initial_state=x["S0"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd()
        bwd()
    torch.cuda.current_stream().wait_stream(side)
    first = [t.clone() for t in (o, SN, *grads)]
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        fwd()
    with torch.cuda.graph(g2):
        fwd()
        bwd()
    for t in (o, SN, *grads):
        t.fill_(float("nan"))
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (o, SN, *grads)))
    y = lin_inputs(16, 1, 1500, 2, 128, torch.bfloat16)
    for n in ("q", "k", "v", "d_o", "S0"):
        x[n].copy_(y[n])
    g2.replay()
    torch.cuda.synchronize()
    want = run_fwd(kda, y)
    assert torch.equal(o, want[0]) and torch.equal(SN, want[1])
    assert all(torch.equal(a, b) for a, b in zip(grads, run_bwd(kda, dict(y, dSN=torch.zeros_like(y["dSN"])), first=False)))


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def pairs_of(d):
    return (d // 8, d // 8 + 3, d // 4 - 3)


@pytest.mark.parametrize("dtype,d,inter", list(itertools.product(["f32", "bf16"], [64, 128], [False, True])))
@pytest.mark.parametrize("B,H,text,grid", [(1, 1, 1, (0, 0, 0)), (2, 3, 5, (2, 3, 7)), (3, 16, 0, (1, 9, 11)), (1, 24, 40, (5, 1, 13)),
                                           (9, 2, 3, (0, 0, 0))])
def test_rope(kda, B, H, text, grid, dtype, d, inter):
    g = gen(B * 100 + d)
    N = text + grid[0] * grid[1] * grid[2]
    p, r = kda.problem(B, H, d, text, grid), kda.rope(pairs_of(d), interleaved=inter)
    q, k = randn(g, B, N, H, d, dtype=DT[dtype]), randn(g, B, N, H, d, dtype=DT[dtype])
    f = torch.rand(d // 2, generator=g, device="cuda")
    far = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, N, 3), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    for pos in (None, far):
        at = ops.grid_positions(B, text, grid) if pos is None else pos
        for call, inverse in ((kda.kda_rope_fwd, False), (kda.kda_rope_bwd, True)):
            qo, ko = torch.empty_like(q), torch.empty_like(k)
            call(p, r, q, k, f, qo, ko, positions=pos)
            for x, y in ((q, qo), (k, ko)):
                ref = ops.rope(x, f, at, pairs_of(d), inter, inverse)
                M = x.double().abs()
                pair = M.view(*M.shape[:-1], d // 2, 2).flip(-1).flatten(-2) if inter else M.roll(d // 2, -1)
                # the angle: half a step of a fraction of a turn in fp32, 2 pi 2^-26; cos, sin and products: 4 x 2^-24.
                # An angle w in fp64 is itself off by 2^-53 |w| here (a 31-bit position times a 24-bit frequency), and
                # by 2 x 2^-53 |w| in the kernel (1 / (2 pi) and the product): 12 x 2^-24 at |w| = 2^31
                w = float(at.abs().max()) * float(f.max())
                close(y, ref, M + pair, 6 * 2.0 ** -24 + 3 * 2.0 ** -53 * w)
            one = torch.empty_like(q)
            call(p, r, q, None, f, one, None, positions=pos)      # one tensor
            assert torch.equal(one, qo)
            qi, ki = q.clone(), k.clone()
            call(p, r, qi, ki, f, qi, ki, positions=pos)          # in place
            assert torch.equal(qi, qo) and torch.equal(ki, ko)


def test_rope_backward_is_the_forward_passes_transpose(kda):
    g = gen(3)
    p, r = kda.problem(2, 3, 64, 7, (2, 3, 5)), kda.rope(pairs_of(64))
    x, dy = randn(g, 2, 37, 3, 64), randn(g, 2, 37, 3, 64)
    f = torch.rand(32, generator=g, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    kda.kda_rope_fwd(p, r, x, None, f, y, None)
    kda.kda_rope_bwd(p, r, dy, None, f, dx, None)
    a, b = float((y.double() * dy.double()).sum()), float((x.double() * dx.double()).sum())
    # both sides round every element by at most 8 x 2^-24 of its pair
    assert abs(a - b) <= 16 * 2.0 ** -24 * 2 * float((x.double().abs() * dy.double().abs().max()).sum())


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
COLS = [1, 2, 7, 8, 31, 64, 100, 128, 257, 520, 1000, 1024, 1028, 2048, 4100, 5001, 8192, 16383, 16384]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_layernorm(kda, cols, dtype):
    for rows, offset in ((1, 0.0), (5, 3.0), (700, -20.0)):
        g = gen(cols + rows)
        x = (randn(g, rows, cols) * (0.2 + torch.rand(rows, 1, generator=g, device="cuda")) + offset).to(DT[dtype])
        dy = randn(g, rows, cols, dtype=DT[dtype])
        w, b = randn(g, cols) + 1, randn(g, cols)
        for weight, bias in ((w, b), (None, None)):
            y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            kda.kda_layernorm_fwd(x, y, weight, bias, 1e-5, mean, rstd)
            ref = ops.layernorm_fwd(x, weight, bias, 1e-5)
            aw = 1.0 if weight is None else weight.double().abs()
            # statistics: at most 48 additions in sequence (32 of a thread, 5 of a warp, the warps, the mean)
            c = 64 * 2.0 ** -24
            size = x.double().abs().mean(1) + x.double().abs().amax(1)
            err = (mean.double() - ref[1]).abs()
            assert (err <= c * size + 1e-37).all()
            # var is off by 2 |d mean| sqrt(var) + c var; against eps beside it
            dv = 2 * c * size / (1 / ref[2]) + c
            assert ((rstd.double() - ref[2]).abs() <= ref[2] * (dv + c)).all()
            h = (x.double() - ref[1][:, None]).abs() * ref[2][:, None]
            M = aw * (h * (1 + dv / c)[:, None] + (size * ref[2])[:, None]) + (0.0 if bias is None else bias.double().abs())
            u = torch.finfo(y.dtype).eps / 2
            assert ((y.double() - ref[0]).abs() <= u * ref[0].abs() + 2 * c * M + 1e-37).all()
            # gradients at the statistics the forward pass gave
            dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            ws = kda.alloc_layernorm_bwd_workspace(rows, cols)
            kda.kda_layernorm_bwd(dy, x, mean, rstd, dx, ws, weight, dw, db)
            rx, rw, rb = ops.layernorm_bwd(dy, x, mean, rstd, weight)
            R = rstd.double()[:, None]
            hs = (x.double().abs() + mean.double().abs()[:, None]) * R      # h with its subtraction's own rounding
            G = dy.double().abs() * aw
            Mx = R * (G + G.mean(1, keepdim=True) + hs * (G * hs).mean(1, keepdim=True))
            u = torch.finfo(dx.dtype).eps / 2
            assert ((dx.double() - rx).abs() <= u * rx.abs() + c * Mx + 1e-37).all()
            assert ((dw.double() - rw).abs() <= c * (dy.double().abs() * hs).sum(0) + 1e-37).all()
            assert ((db.double() - rb).abs() <= c * dy.double().abs().sum(0) + 1e-37).all()
            # either sum alone, none of them, and the same bits again
            dx2, dw2, db2 = torch.empty_like(x), torch.empty_like(dw), torch.empty_like(db)
            kda.kda_layernorm_bwd(dy, x, mean, rstd, dx2, ws, weight, dw2, None)
            kda.kda_layernorm_bwd(dy, x, mean, rstd, dx2, ws, weight, None, db2)
            assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
            kda.kda_layernorm_bwd(dy, x, mean, rstd, dx2, ws, weight)
            assert torch.equal(dx, dx2)
            y2 = torch.empty_like(y)
            kda.kda_layernorm_fwd(x, y2, weight, bias, 1e-5)
            assert torch.equal(y, y2)


def test_layernorm_constant_rows_and_no_rows(kda):
    x = torch.full((3, 257), 5.0, device="cuda")
    y = torch.empty_like(x)
    b = torch.randn(257, device="cuda")
    kda.kda_layernorm_fwd(x, y, None, b)
    assert torch.equal(y, b.expand(3, -1))
    z = torch.empty(8, device="cuda")
    dw, db = torch.full((16,), 7.0, device="cuda"), torch.full((16,), 7.0, device="cuda")
    ws = kda.alloc_layernorm_bwd_workspace(0, 16)
    lib = kda._lib
    assert lib.kda_layernorm_bwd(0, 16, 1, z.data_ptr(), z.data_ptr(), None, z.data_ptr(), z.data_ptr(), z.data_ptr(),
                                 dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(), None) == kda.KDA_OK
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_layernorm_of_tensors_without_rows(kda):
    e, s = torch.empty(2, 0, 16, device="cuda"), torch.empty(2, 0, device="cuda")
    y, w = torch.empty_like(e), torch.ones(16, device="cuda")
    kda.kda_layernorm_fwd(e, y, w, w, 1e-5, s, torch.empty_like(s))
    dw, db = torch.full((16,), 7.0, device="cuda"), torch.full((16,), 7.0, device="cuda")
    kda.kda_layernorm_bwd(e, e.clone(), s, s.clone(), y, kda.alloc_layernorm_bwd_workspace(0, 16), w, dw, db)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_layernorm_many_rows(kda):
    g = gen(77)
    x, dy = randn(g, 100003, 48, dtype=torch.bfloat16), randn(g, 100003, 48, dtype=torch.bfloat16)
    y, mean, rstd = torch.empty_like(x), torch.empty(100003, device="cuda"), torch.empty(100003, device="cuda")
    kda.kda_layernorm_fwd(x, y, None, None, 1e-5, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty(48, device="cuda"), torch.empty(48, device="cuda")
    kda.kda_layernorm_bwd(dy, x, mean, rstd, dx, kda.alloc_layernorm_bwd_workspace(100003, 48), None, dw, db)
    _, rw, rb = ops.layernorm_bwd(dy, x, mean, rstd)
    assert float((dw.double() - rw).norm() / rw.norm()) < TOL_F32_REL_L2
    assert float((db.double() - rb).norm() / rb.norm()) < TOL_F32_REL_L2


def test_layernorm_backward_workspace_has_a_status(kda):
    """Whatever stood in the workspace before."""
    x, dy = randn(gen(78), 37, 257), randn(gen(79), 37, 257)
    for sums in (None, torch.empty(257, device="cuda")):
        ws = kda.alloc_layernorm_bwd_workspace(37, 257).fill_(0xff)
        kda.kda_layernorm_bwd(dy, x, x.mean(1), x.std(1).reciprocal(), torch.empty_like(x), ws, None, sums)
        assert kda.kda_read_status(ws) == kda.KDA_OK


@pytest.mark.parametrize("d", [64, 128])
def test_linear_values_beside_the_largest(kda, d):
    """fp32 values above the largest bf16 one, 3.39e38, in the inputs and in a state: their first bf16 term may not be
    infinite.  Sums and products stay in range."""
    top = torch.finfo(torch.float32).max
    for dtype in (torch.float32, torch.bfloat16):
        x = lin_inputs(17, 1, 300, 2, d, torch.float32)
        x["S0"] = torch.where(x["S0"] > 1.0, top, x["S0"].sign() * 1e36)
        x["dSN"] *= 1e-30
        if dtype == torch.float32:
            x["v"] = torch.where(x["v"] > 1.0, top, x["v"] * 1e36)
        x["q"], x["k"], x["d_o"] = x["q"] * 1e-6, x["k"] * 1e-12, x["d_o"] * 1e-30
        x = {n: t.to(dtype) if n in ("q", "k", "v", "d_o") else t for n, t in x.items()}
        o, SN, ws = run_fwd(kda, x)
        ref = ops.linear_fwd(x["q"], x["k"], x["v"], x["ld"], None, x["S0"])
        M = ops.linear_fwd(*(x[n].abs() for n in "qkv"), x["ld"], None, x["S0"].abs())
        assert torch.isfinite(ref[0].float()).all() and torch.isfinite(ref[1].float()).all()
        c = C32 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
        close(o, ref[0], M[0], c, "o")
        close(SN, ref[1], M[1], C32, "final state")
        ref = ops.linear_bwd(x["q"], x["k"], x["v"], x["ld"], x["d_o"], None, x["S0"], x["dSN"])
        M = ops.linear_bwd(*(x[n].abs() for n in "qkv"), x["ld"], x["d_o"].abs(), None, x["S0"].abs(), x["dSN"].abs())
        for name, g, r, m in zip(("dq", "dk", "dv", "dS0"), run_bwd(kda, x), ref, M):
            if name == "dv":
                # k dSN and k (q do) are of 1e-12 x 1e-30: all of it lies below the smallest normal number, 2^-126, where
                # one step is 2^-149 (bf16: 2^-133), 1e-3 of it (all of it), and no relative bound can hold
                assert float(m.max()) < 2.0 ** -126 and ((g.double() - r).abs() <= 2.0 ** -126).all()
                continue
            close(g, r, m, C32 if name == "dS0" else c, name)
