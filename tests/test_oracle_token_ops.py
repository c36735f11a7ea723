"""The fp64 reference of the operators beside the KDA scan, pinned on the CPU: closed forms and differences."""
import torch

from oracle import token_ops as ops


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_linear_forward_is_the_decayed_causal_product():
    B, N, H, d = 2, 7, 3, 4
    q, k, v, S0 = _rand(B, N, H, d), _rand(B, N, H, d, seed=1), _rand(B, N, H, d, seed=2), _rand(B, H, d, d, seed=3)
    ld = torch.tensor([0.0, -0.3, -2.0])
    lam = ld.double().exp()
    o, S = ops.linear_fwd(q, k, v, ld, S0=S0)
    i = torch.arange(N)
    gap = i.view(-1, 1) - i
    D = torch.where(gap >= 0, lam.view(H, 1, 1) ** gap.clamp(min=0), torch.zeros(()).double())
    ref = torch.einsum("hij,bihd,bjhd,bjhe->bihe", D, q, k, v) + torch.einsum("hi,bihd,bhde->bihe", lam.view(H, 1) ** (i + 1), q, S0)
    assert torch.allclose(o, ref, rtol=1e-12, atol=1e-12)
    refS = torch.einsum("hj,bjhd,bjhe->bhde", lam.view(H, 1) ** (N - 1 - i), k, v) + lam.view(1, H, 1, 1) ** N * S0
    assert torch.allclose(S, refS, rtol=1e-12, atol=1e-12)


def test_linear_lengths_cut_each_item():
    B, N, H, d = 3, 6, 2, 4
    q, k, v = (_rand(B, N, H, d, seed=s) for s in range(3))
    S0 = _rand(B, H, d, d, seed=9)
    ld = torch.tensor([-0.1, -0.5])
    n = torch.tensor([0, 4, 6])
    o, S = ops.linear_fwd(q, k, v, ld, n, S0)
    for b in range(B):
        m = int(n[b])
        ob, Sb = ops.linear_fwd(q[b:b + 1, :m], k[b:b + 1, :m], v[b:b + 1, :m], ld, None, S0[b:b + 1])
        assert torch.equal(o[b, :m], ob[0]) and torch.equal(S[b], Sb[0]) and not o[b, m:].any()


def test_linear_backward_against_differences():
    B, N, H, d = 2, 5, 2, 3
    ld, n = torch.tensor([-0.2, -1.0]), torch.tensor([5, 3])
    x = [_rand(B, N, H, d, seed=s) for s in range(3)] + [_rand(B, H, d, d, seed=3)]
    do, dS = _rand(B, N, H, d, seed=4), _rand(B, H, d, d, seed=5)

    def loss(q, k, v, S0):
        o, S = ops.linear_fwd(q, k, v, ld, n, S0)
        return float((ops._until(do, n) * o).sum() + (dS * S).sum())

    grads = ops.linear_bwd(x[0], x[1], x[2], ld, do, n, x[3], dS)
    for which in range(4):
        for at in range(0, x[which].numel(), 7):
            h = 1e-5
            up, down = ([y.clone() for y in x] for _ in range(2))
            up[which].view(-1)[at] += h
            down[which].view(-1)[at] -= h
            diff = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(diff - float(grads[which].reshape(-1)[at])) < 1e-7 * max(1.0, abs(diff))


def test_rope_turns_pairs_and_back():
    x = _rand(2, 5, 3, 8)
    pos = ops.grid_positions(2, 2, (1, 1, 3))
    assert pos[0].tolist() == [[0, 0, 0], [1, 1, 1], [2, 2, 2], [2, 2, 3], [2, 2, 4]]
    f = torch.tensor([1.0, 0.5, 0.25, 0.125])
    for inter in (False, True):
        y = ops.rope(x, f, pos, (1, 1, 2), inter)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
        assert torch.allclose(ops.rope(y, f, pos, (1, 1, 2), inter, inverse=True), x)
        assert torch.equal(y[:, 0], x[:, 0])   # position 0
    y = ops.rope(x, f, pos, (1, 1, 2), True)
    w = 4 * 0.125                              # last token, last pair: width position 4
    assert torch.allclose(y[0, 4, 0, 6], x[0, 4, 0, 6] * torch.cos(torch.tensor(w).double()) - x[0, 4, 0, 7] * torch.sin(torch.tensor(w).double()))


def test_layernorm_backward_against_differences():
    R, C = 3, 5
    x, w, b, dy = _rand(R, C), _rand(C, seed=1), _rand(C, seed=2), _rand(R, C, seed=3)
    y, mean, rstd = ops.layernorm_fwd(x, w, b)
    assert torch.allclose(((y - b) / w).mean(1), torch.zeros(R).double(), atol=1e-12)
    dx, dw, db = ops.layernorm_bwd(dy, x, mean, rstd, w)
    loss = lambda x, w, b: float((ops.layernorm_fwd(x, w, b)[0] * dy).sum())   # noqa: E731
    args, grads = [x, w, b], [dx, dw, db]
    for which in range(3):
        for at in range(args[which].numel()):
            h = 1e-5
            up, down = ([y.clone() for y in args] for _ in range(2))
            up[which].view(-1)[at] += h
            down[which].view(-1)[at] -= h
            diff = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(diff - float(grads[which].view(-1)[at])) < 1e-7 * max(1.0, abs(diff))
