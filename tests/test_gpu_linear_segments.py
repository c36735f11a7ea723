"""Linear attention with a decay per head where a call's result hangs on the order of copies and products inside the
map: items that end in the first tile of a segment, with a state entering it (needs a B200)."""
import pytest
import torch

from oracle import token_ops as ops
from tests.test_gpu_token_ops import C32, close, lin_inputs, run_bwd, run_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import linear_attention_video_b200 as kda
    assert torch.cuda.is_available()
    yield kda
    torch.cuda.empty_cache()


def ragged(seed, n, N, H, d, dtype=torch.bfloat16):
    """Inputs of items of n tokens each, NaN and infinities behind them, and the lengths."""
    x = lin_inputs(seed, len(n), N, H, d, dtype)
    for b, m in enumerate(n):
        for i, name in enumerate(("q", "k", "v", "d_o")):
            x[name][b, m:] = (float("nan"), float("inf"), -float("inf"), float("nan"))[(b + i) % 4]
    return x, torch.tensor(n, dtype=torch.int32, device="cuda")


# few heads: segments of 128 tokens; many: longer ones
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,H", [([1, 100, 129, 150, 385, 513, 897, 900], 3),
                                 ([1, 17, 127, 257, 260, 383, 513, 514, 530, 600, 639, 769, 770, 895, 1025, 1026, 1060, 1099, 1100], 16)])
def test_items_that_end_in_a_segments_first_tile_repeat_their_bits(kda, n, H, d):
    """Beside memory traffic on another stream, which moves the arrival of the copies against one another."""
    N = n[-1]
    x, lengths = ragged(21, n, N, H, d)
    want = run_fwd(kda, x, lengths)[:2] + run_bwd(kda, x, lengths)
    assert all(torch.isfinite(t).all() for t in want)
    busy, other = torch.cuda.Stream(), torch.empty(2, 1 << 28, dtype=torch.uint8, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        with torch.cuda.stream(busy):
            for _ in range(4):
                other[0].copy_(other[1])
        got = run_fwd(kda, x, lengths)[:2] + run_bwd(kda, x, lengths)
        for a, b in zip(got, want):
            wrong += (a != b).sum()
    torch.cuda.synchronize()
    assert int(wrong) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_items_that_end_in_a_segments_first_tile(kda, d):
    x, lengths = ragged(22, [1, 100, 129, 150, 385, 513, 897, 900], 900, 3, d)
    clean = dict(x, **{i: ops._until(x[i], lengths) for i in ("q", "k", "v", "d_o")})
    c = C32 + 2.0 ** -8   # the decayed scores and the state may be rounded once to bf16
    o, SN, _ = run_fwd(kda, x, lengths)
    ref = ops.linear_fwd(*(clean[i] for i in "qkv"), x["ld"], lengths, x["S0"])
    M = ops.linear_fwd(*(clean[i].abs() for i in "qkv"), x["ld"], lengths, x["S0"].abs())
    close(o, ref[0], M[0], c, "o")
    close(SN, ref[1], M[1], C32, "final state")
    ref = ops.linear_bwd(*(clean[i] for i in "qkv"), x["ld"], clean["d_o"], lengths, x["S0"], x["dSN"])
    M = ops.linear_bwd(*(clean[i].abs() for i in "qkv"), x["ld"], clean["d_o"].abs(), lengths, x["S0"].abs(), x["dSN"].abs())
    for name, g, r, m in zip(("dq", "dk", "dv", "dS0"), run_bwd(kda, x, lengths), ref, M):
        close(g, r, m, c if name != "dS0" else C32, name)


def rounded(ref):
    """What one rounding of the exact outputs to bf16 is off by, as a norm."""
    return float((ref.to(torch.bfloat16).double() - ref).norm())


def check_only_the_outputs_are_rounded(got, ref, M, what):
    """Scores and states enter their products as two bf16 terms, which leaves 2^-16 of each; with the additions' 2^-16
    of the sum over absolute values (C32) an element is within u |ref| + 3 x 2^-16 M.  The output's own rounding is
    the rest: the error's norm is that of rounding the exact outputs, and at most 3 x 2^-16 of M's beside it."""
    close(got, ref, M, 2 * 2.0 ** -16 + C32, what)
    err = float((got.double() - ref).norm())
    assert err <= rounded(ref) + 3 * 2.0 ** -16 * float(M.norm()), (what, err / rounded(ref))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,N,H", [(1, 384, 4), (2, 777, 3)])
def test_outputs_of_bf16_problems_are_rounded_once(kda, B, N, H, d):
    x = lin_inputs(23, B, N, H, d, torch.bfloat16)
    o, SN, _ = run_fwd(kda, x)
    ref = ops.linear_fwd(x["q"], x["k"], x["v"], x["ld"], None, x["S0"])
    M = ops.linear_fwd(*(x[i].abs() for i in "qkv"), x["ld"], None, x["S0"].abs())
    check_only_the_outputs_are_rounded(o, ref[0], M[0], "o")
    ref = ops.linear_bwd(x["q"], x["k"], x["v"], x["ld"], x["d_o"], None, x["S0"], x["dSN"])
    M = ops.linear_bwd(*(x[i].abs() for i in "qkv"), x["ld"], x["d_o"].abs(), None, x["S0"].abs(), x["dSN"].abs())
    for name, g, r, m in zip(("dq", "dk", "dv"), run_bwd(kda, x), ref, M):
        check_only_the_outputs_are_rounded(g, r, m, name)


@pytest.mark.parametrize("d", [64, 128])
def test_one_token_through_the_pass_and_through_the_step(kda, d):
    """The next token of a state through kda_linear_fwd and kda_linear_step: both from the fp32 state, each rounded once."""
    B, H = 5, 7
    x = lin_inputs(24, B, 1, H, d, torch.bfloat16)
    o, SN, _ = run_fwd(kda, x)
    p = kda.problem(B, H, d, 1, (0, 0, 0))
    o1, S1 = torch.empty_like(o), torch.empty_like(SN)
    kda.kda_linear_step(p, x["q"], x["k"], x["v"], x["ld"], x["S0"], o1, S1)
    M, MS = ops.linear_fwd(*(x[i].abs() for i in "qkv"), x["ld"], None, x["S0"].abs())
    # two roundings of values at most 4 x 2^-16 M apart: half a step each, 2^-8 of the larger
    apart = (o.double() - o1.double()).abs()
    assert (apart <= 2.0 ** -8 * (o.double().abs() + o1.double().abs()) + 4 * 2.0 ** -16 * M).all()
    assert float((apart > 4 * 2.0 ** -16 * M).double().mean()) < 0.05   # most do not straddle a border
    assert ((SN.double() - S1.double()).abs() <= 2 * C32 * MS).all()


def tokens_per_segment(kda, x, lengths):
    """The segment that a bf16 problem is cut into, from how far its pass writes into the workspace: 4 d^2 bytes per
    item, head and segment behind the first 256."""
    B, N, H, d = x["q"].shape
    ws = kda.alloc_linear_workspace(kda.problem(B, H, d, N, (0, 0, 0)), torch.bfloat16)
    marks = ws[: ws.numel() // 4 * 4].view(torch.int32)
    marks.fill_(0x5a5a5a5a)
    run_fwd(kda, x, lengths, ws=ws)
    states = -(-(int((marks != 0x5a5a5a5a).nonzero()[-1]) + 1 - 64) // (d * d))
    assert states % (B * H) == 0
    return next(s for s in (128, 256, 512, 1024) if -(-N // s) == states // (B * H))


ENDS = [0, 1, 63, 64, 65, 127, 128, 129, 191, 193, 255, 256, 257, 383, 385, 511, 513, 900, 1100]


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("d,H", [(64, 15), (128, 16)])
def test_long_segments(kda, d, H, state):
    """Segments of several tiles against the recurrence: nothing forgotten, far tokens, ragged ends in every tile, NaN
    behind them.  Enough items and heads for the longest segments, which the test asks for."""
    x, lengths = ragged(25, ENDS, 1100, H, d)
    x["ld"][:6] = torch.tensor([0.0, -1e-3, -1e-6, -0.02, -4.0, -float("inf")])
    assert tokens_per_segment(kda, x, lengths) == 256
    clean = dict(x, **{i: ops._until(x[i], lengths) for i in ("q", "k", "v", "d_o")})
    S0, dSN = (x["S0"], x["dSN"]) if state else (None, None)
    size = lambda t: None if t is None else t.abs()   # noqa: E731
    o, SN, _ = run_fwd(kda, x, lengths, state)
    ref = ops.linear_fwd(*(clean[i] for i in "qkv"), x["ld"], lengths, S0)
    M = ops.linear_fwd(*(clean[i].abs() for i in "qkv"), x["ld"], lengths, size(S0))
    check_only_the_outputs_are_rounded(o, ref[0], M[0], "o")
    close(SN, ref[1], M[1], C32, "final state")
    ref = ops.linear_bwd(*(clean[i] for i in "qkv"), x["ld"], clean["d_o"], lengths, S0, dSN)
    M = ops.linear_bwd(*(clean[i].abs() for i in "qkv"), x["ld"], clean["d_o"].abs(), lengths, size(S0), size(dSN))
    for name, g, r, m in zip(("dq", "dk", "dv", "dS0"), run_bwd(kda, x, lengths, state), ref, M):
        if name == "dS0":
            close(g, r, m, C32, name)
        else:
            check_only_the_outputs_are_rounded(g, r, m, name)
