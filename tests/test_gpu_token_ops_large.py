"""Element offsets past 32 bits, calls on several streams at once, for the operators beside the KDA scan (B200).

The large tensors (2.2 to 2.5 billion elements) are checked on their last rows, against the same call on those rows
alone: rows, tokens of a quickly forgetting head and states do not depend on what lies far before them.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import linear_attention_video_b200 as kda
    assert torch.cuda.is_available()
    yield kda
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, dtype=torch.bfloat16):
    """Uniform on [-1, 1), made in place."""
    return torch.empty(*shape, dtype=dtype, device="cuda").uniform_(-1, 1, generator=g)


def test_layernorm_past_32_bits(kda):
    R, C, last = 160_003, 16_000, 5
    assert R * C > 2 ** 31
    x, dy = rand(gen(1), R, C), rand(gen(2), R, C)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    dw, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    kda.kda_layernorm_fwd(x, y, None, None, 1e-5, mean, rstd)
    kda.kda_layernorm_bwd(dy, x, mean, rstd, dx, kda.alloc_layernorm_bwd_workspace(R, C), None, dw, db)
    xs, dys = x[-last:].clone(), dy[-last:].clone()
    ys, dxs, ms, rs = torch.empty_like(xs), torch.empty_like(xs), torch.empty(last, device="cuda"), torch.empty(last, device="cuda")
    kda.kda_layernorm_fwd(xs, ys, None, None, 1e-5, ms, rs)
    kda.kda_layernorm_bwd(dys, xs, ms, rs, dxs, kda.alloc_layernorm_bwd_workspace(last, C), None, dw, db)
    assert torch.equal(y[-last:], ys) and torch.equal(mean[-last:], ms) and torch.equal(rstd[-last:], rs)
    assert torch.equal(dx[-last:], dxs)


def test_rope_and_linear_past_32_bits(kda):
    N, H, d, last = 1_100_003, 16, 128, 1500
    assert N * H * d > 2 ** 31
    p, r = kda.problem(1, H, d, N, (0, 0, 0)), kda.rope((16, 24, 24))
    f = torch.rand(d // 2, generator=gen(3), device="cuda")
    q, k, v = (rand(gen(s), 1, N, H, d) for s in (4, 5, 6))
    tail = lambda t, n=last: t[:, -n:].clone()   # noqa: E731
    q0, k0, v0 = tail(q), tail(k), tail(v)
    kda.kda_rope_fwd(p, r, q, k, f, q, k)
    # the same tokens alone, at their positions
    ps = kda.problem(1, H, d, last, (0, 0, 0))
    pos = torch.arange(N - last, N, dtype=torch.int32, device="cuda").view(1, -1, 1).expand(1, last, 3).contiguous()
    kda.kda_rope_fwd(ps, r, q0, k0, f, q0, k0, positions=pos)
    assert torch.equal(tail(q), q0) and torch.equal(tail(k), k0)
    # heads that forget within 20 tokens (exp(-4 x 1000) is 0 in fp32): the last 500 tokens know the last 1500 only
    ld = torch.full((H,), -4.0, device="cuda")
    o, S = torch.empty_like(v), torch.empty(1, H, d, d, device="cuda")
    kda.kda_linear_fwd(p, q, k, v, ld, o, kda.alloc_linear_workspace(p, torch.bfloat16), final_state=S)
    os_, Ss = torch.empty_like(v0), torch.empty_like(S)
    kda.kda_linear_fwd(ps, q0, k0, v0, ld, os_, kda.alloc_linear_workspace(ps, torch.bfloat16), final_state=Ss)
    a, b = tail(o, 500).double(), os_[:, -500:].double()
    # both round each output and each of its few terms once: 2 x (2^-8 + 2^-8) of its size at most, far less in the norm
    assert float((a - b).norm() / b.norm()) < 5e-3
    assert float((S.double() - Ss.double()).norm() / Ss.double().norm()) < 1e-5
    # gradients
    g = rand(gen(7), 1, N, H, d)
    grads = [torch.empty_like(v) for _ in range(3)]
    kda.kda_linear_bwd(p, q, k, v, ld, g, *grads, kda.alloc_linear_bwd_workspace(p, torch.bfloat16))
    gs = [torch.empty_like(v0) for _ in range(3)]
    kda.kda_linear_bwd(ps, q0, k0, v0, ld, tail(g), *gs, kda.alloc_linear_bwd_workspace(ps, torch.bfloat16))
    for x, y in zip(grads, gs):
        a, b = tail(x, 500).double(), y[:, -500:].double()
        assert float((a - b).norm() / b.norm()) < 5e-3


def test_step_states_past_32_bits(kda):
    B, H, d, last = 8_500, 16, 128, 3
    assert B * H * d * d > 2 ** 31
    ld = -torch.rand(H, generator=gen(8), device="cuda")
    S = rand(gen(9), B, H, d, d, dtype=torch.float32)
    q, k, v = (rand(gen(s), B, 1, H, d) for s in (10, 11, 12))
    alone = [t[-last:].clone() for t in (q, k, v, S)]
    o = torch.empty_like(v)
    kda.kda_linear_step(kda.problem(B, H, d, 1, (0, 0, 0)), q, k, v, ld, S, o, S)
    os_ = torch.empty_like(alone[2])
    kda.kda_linear_step(kda.problem(last, H, d, 1, (0, 0, 0)), *alone[:3], ld, alone[3], os_, alone[3])
    assert torch.equal(S[-last:], alone[3]) and torch.equal(o[-last:], os_)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_on_several_streams_at_once(kda, dtype):
    """Forward and backward passes of three problems on three streams, each with its workspace, as on one."""
    sizes = [(1, 3, 128, 2000), (2, 5, 64, 900), (1, 8, 128, 3100)]
    data = []
    for i, (B, H, d, N) in enumerate(sizes):
        p = kda.problem(B, H, d, N, (0, 0, 0))
        x = [rand(gen(20 + 5 * i + j), B, N, H, d, dtype=dtype) for j in range(4)]
        ld = -torch.rand(H, generator=gen(40 + i), device="cuda")
        data.append((p, x, ld, kda.alloc_linear_workspace(p, dtype), kda.alloc_linear_bwd_workspace(p, dtype)))

    def run(streams):
        outs = []
        for (p, (q, k, v, g), ld, ws, wb), s in zip(data, streams):
            o, grads = torch.empty_like(v), [torch.empty_like(v) for _ in range(3)]
            n = torch.empty_like(v)
            kda.kda_linear_fwd(p, q, k, v, ld, o, ws, stream=s)
            kda.kda_linear_bwd(p, q, k, v, ld, g, *grads, wb, stream=s)
            kda.kda_layernorm_fwd(o, n, stream=s)
            outs += [o, *grads, n]
        return outs

    torch.cuda.synchronize()
    one = run([None] * 3)
    torch.cuda.synchronize()
    for _ in range(3):
        many = run([torch.cuda.Stream() for _ in range(3)])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(one, many))
    for _, _, _, ws, wb in data:
        assert kda.kda_read_status(ws) == kda.KDA_OK and kda.kda_read_status(wb) == kda.KDA_OK
