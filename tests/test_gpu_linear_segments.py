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


# few heads: segments of 128 tokens; many: of 512 (d = 128) and 256 (d = 64)
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
