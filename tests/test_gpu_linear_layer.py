"""The linear layer of the mixer stacks (needs a B200): layer norm, rotary positions and linear attention with a
decay per head as they run together: a prompt pass, its gradients, and single tokens after it.

The layer rounds its intermediates to bf16 (u = 2^-8, half a step): h, q / k / v before and after the turn, o and y on
the way forward; dy Wo^T, dq / dk / dv before and after the turn, dh on the way back.  Against fp64 without any of
them, an output of m independent roundings of its path is off by about m u / sqrt(3) of its norm at random; forward
m = 9 (h, q, q', k, k', v, o, y and the scores), backward m = 16, doubled for what the products do not average out.
"""
import math

import pytest
import torch

from oracle import token_ops as ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
FWD, BWD = 2 * math.sqrt(9 / 3) * U, 2 * math.sqrt(16 / 3) * U
H, d, TEXT, GRID = 4, 128, 70, (3, 9, 11)
N, D = TEXT + 3 * 9 * 11, H * d
PAIRS = (16, 24, 24)


def reference(layer, x, lengths=None, positions=None, S0=None):
    """The layer in fp64 and differentiable (oracle's definitions composed; rotation and attention as matrices)."""
    B, n, _ = x.shape
    mean = x.mean(-1, keepdim=True)
    h = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + 1e-5) * layer["norm_w"] + layer["norm_b"]
    q, k, v = ((h @ layer[w]).view(B, n, H, d) for w in ("wq", "wk", "wv"))
    pos = ops.grid_positions(B, TEXT, GRID).to(x.device) if positions is None else positions
    axis = torch.tensor([0] * 16 + [1] * 24 + [2] * 24, device=x.device)
    w = (pos.double()[..., axis] * layer["inv_freq"]).unsqueeze(2)
    turn = lambda t: torch.cat([t[..., :64] * w.cos() - t[..., 64:] * w.sin(), t[..., :64] * w.sin() + t[..., 64:] * w.cos()], -1)   # noqa: E731
    q, k = turn(q), turn(k)
    i = torch.arange(n, device=x.device)
    gap = i.view(-1, 1) - i
    decay = torch.where(gap >= 0, torch.exp(layer["log_decay"].view(H, 1, 1) * gap.clamp(min=0)), torch.zeros((), device=x.device).double())
    o = torch.einsum("bihc,bjhc,hij,bjhe->bihe", q, k, decay, v)
    if lengths is not None:
        o = o * (i.view(1, -1, 1, 1) < lengths.view(-1, 1, 1, 1))
    return o.reshape(B, n, D) @ layer["wo"]


@pytest.fixture(scope="module")
def layer():
    from linear_attention_video_b200 import mixer
    return mixer.LinearLayer(2, H, d, TEXT, GRID, seed=5)


def weights(layer):
    return {n: getattr(layer, n).double() for n in ("wq", "wk", "wv", "wo", "norm_w", "norm_b", "log_decay", "inv_freq")}


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def _x(seed, B=2, n=N):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, n, D, generator=g).to("cuda", torch.bfloat16)


def test_forward_and_gradients(layer):
    x, dy = _x(1), _x(2)
    lengths = torch.tensor([N, 211], dtype=torch.int32, device="cuda")
    for n in (None, lengths):
        w = {k: t.requires_grad_(k not in ("log_decay", "inv_freq")) for k, t in weights(layer).items()}
        x64 = x.double().requires_grad_()
        y = reference(w, x64, n)
        got = layer(x, lengths=n)
        assert rel(got, y.detach()) <= FWD, rel(got, y.detach())
        if n is not None:
            assert not got[1, 211:].any()
        y.backward(dy.double())
        dx, grads = layer.backward(x, dy, lengths=n)
        assert rel(dx, x64.grad) <= BWD, rel(dx, x64.grad)
        for name, g in grads.items():
            assert rel(g, w[name].grad) <= BWD, (name, rel(g, w[name].grad))


@pytest.mark.parametrize("second", [0, 211])
def test_what_stands_behind_a_sequence_reaches_no_output(layer, second):
    """NaN and infinities there change no bit of the output and of any gradient."""
    x, dy = _x(3), _x(4)
    lengths = torch.tensor([N, second], dtype=torch.int32, device="cuda")
    junk_x, junk_dy = x.clone(), dy.clone()
    junk_x[1, second:], junk_dy[1, second:] = math.nan, math.inf
    assert torch.equal(layer(junk_x, lengths=lengths), layer(x, lengths=lengths))
    dx, grads = layer.backward(x, dy, lengths=lengths)
    got, got_grads = layer.backward(junk_x, junk_dy, lengths=lengths)
    assert torch.equal(got, dx) and not got[1, second:].any()
    for name, g in grads.items():
        assert torch.isfinite(g).all() and torch.equal(got_grads[name], g), name


def test_prompts_then_tokens(layer):
    """Prompts of different lengths, then five tokens each from the states they left, against whole sequences."""
    from linear_attention_video_b200 import mixer
    more = 5
    x = _x(3, n=N + more)
    n = torch.tensor([N, 130], dtype=torch.int32, device="cuda")
    pos = torch.arange(N + more, dtype=torch.int32, device="cuda").view(1, -1, 1).expand(2, -1, 3).contiguous()
    text = mixer.LinearLayer(2, H, d, N, (0, 0, 0), seed=5)   # text positions: (i, i, i)
    state = torch.empty(2, H, d, d, device="cuda")
    text(x[:, :N].contiguous(), lengths=n, final_state=state)
    w = weights(text)
    full = reference(w, x.double(), positions=pos)
    rows = torch.arange(2, device="cuda")
    for t in range(more):
        at = n.long() + t
        y = text.step(x[rows, at].unsqueeze(1).contiguous(), state, pos[rows, at].unsqueeze(1).contiguous())
        assert rel(y[:, 0], full[rows, at]) <= FWD, (t, rel(y[:, 0], full[rows, at]))


def test_stack_runs_end_to_end():
    from linear_attention_video_b200 import mixer
    layers = mixer.stack("linear", 1, H, d, TEXT, GRID)
    y = mixer.run_stack(layers, _x(4, B=1))
    assert y.shape == (1, N, D) and bool(torch.isfinite(y).all())


def test_layer_captured_in_a_graph(layer):
    x, dy = _x(6), _x(7)
    y = layer(x)
    dx, grads = layer.backward(x, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # warm-up on the capture's side stream
        layer(x)
        layer.backward(x, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = layer(x)
        dx2, grads2 = layer.backward(x, dy)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2)
    assert torch.equal(grads["norm_w"], grads2["norm_w"]) and torch.equal(grads["norm_b"], grads2["norm_b"])


def test_gradients_of_a_piece_between_carried_states(layer):
    """A sequence in pieces: the state that enters, the gradient that comes back through the state that leaves, and the
    gradient for the piece before, with items that end inside the piece."""
    g = torch.Generator().manual_seed(8)
    x, dy = _x(8), _x(9)
    S0, dSN = (torch.randn(2, H, d, d, generator=g).cuda() for _ in range(2))
    for n in (None, torch.tensor([N, 211], dtype=torch.int32, device="cuda")):
        w = {k: t.requires_grad_(k not in ("log_decay", "inv_freq")) for k, t in weights(layer).items()}
        x64, s64 = x.double().requires_grad_(), S0.double().requires_grad_()
        y, SN = carried_reference(w, x64, s64, n)
        final = torch.empty_like(S0)
        assert rel(layer(x, lengths=n, initial_state=S0, final_state=final), y.detach()) <= FWD
        assert rel(final, SN.detach()) <= FWD
        ((y * dy.double()).sum() + (SN * dSN.double()).sum()).backward()
        dS0 = torch.empty_like(S0)
        dx, grads = layer.backward(x, dy, lengths=n, initial_state=S0, d_final_state=dSN, d_initial_state=dS0)
        assert rel(dx, x64.grad) <= BWD, rel(dx, x64.grad)
        assert rel(dS0, s64.grad) <= BWD, rel(dS0, s64.grad)
        for name, t in grads.items():
            assert rel(t, w[name].grad) <= BWD, (name, rel(t, w[name].grad))


def carried_reference(w, x, S0, lengths=None):
    """The layer in fp64 from a state, and the state behind each item's last token; differentiable."""
    B, n, _ = x.shape
    mean = x.mean(-1, keepdim=True)
    h = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + 1e-5) * w["norm_w"] + w["norm_b"]
    q, k, v = ((h @ w[i]).view(B, n, H, d) for i in ("wq", "wk", "wv"))
    pos = ops.grid_positions(B, TEXT, GRID).to(x.device)
    a = (pos.double()[..., torch.tensor([0] * 16 + [1] * 24 + [2] * 24, device=x.device)] * w["inv_freq"]).unsqueeze(2)
    turn = lambda t: torch.cat([t[..., :64] * a.cos() - t[..., 64:] * a.sin(), t[..., :64] * a.sin() + t[..., 64:] * a.cos()], -1)   # noqa: E731
    q, k = turn(q), turn(k)
    i, ld = torch.arange(n, device=x.device), w["log_decay"].view(H, 1, 1)
    last = torch.full((B,), n, device=x.device) if lengths is None else lengths.long()
    live = (i.view(1, -1, 1, 1) < last.view(-1, 1, 1, 1)).double()
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    gap = i.view(-1, 1) - i
    decay = torch.where(gap >= 0, torch.exp(ld * gap.clamp(min=0)), zero)
    o = torch.einsum("bihc,bjhc,hij,bjhe->bihe", q, k, decay, v)
    o = o + torch.einsum("hi,bihc,bhce->bihe", torch.exp(ld[..., 0] * (i + 1)), q, S0)
    left = last.view(-1, 1, 1) - 1 - i                                            # [B, 1, n]
    end = torch.where(left >= 0, torch.exp(ld.view(1, H, 1) * left.clamp(min=0)), zero)
    SN = torch.einsum("bhj,bjhc,bjhe->bhce", end, k, v) + torch.exp(ld.view(1, H, 1, 1) * last.view(-1, 1, 1, 1)) * S0
    return (o * live).reshape(B, n, D) @ w["wo"], SN
