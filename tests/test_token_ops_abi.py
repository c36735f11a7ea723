"""Refusals of the operators beside the KDA scan (CPU only): every bad argument is an error of the call, before
anything reaches the GPU.  Addresses stand in for device pointers; none is ever read."""
import ctypes
import math

import pytest
import torch

import linear_attention_video_b200 as kda

A = 1 << 20          # aligned addresses far apart
BIG = 1 << 40


def _p(**kw):
    args = dict(B=2, H=3, d=64, text_len=8, grid=(1, 2, 4))
    args.update(kw)
    return kda.problem(**args)


def _linear(p, dt=1, q=A, k=2 * A, v=3 * A, ld=4 * A, n=5 * A, s0=6 * A, o=7 * A, sn=8 * A, ws=9 * A, nb=BIG):
    return kda._lib.kda_linear_fwd(ctypes.byref(p), dt, q, k, v, ld, n, s0, o, sn, ws, nb, None)


def _linear_bwd(p, dt=1, nb=BIG, **kw):
    names = ("q", "k", "v", "ld", "n", "s0", "do", "dsn", "dq", "dk", "dv", "ds0", "ws")
    a = {n: (i + 1) * A for i, n in enumerate(names)}
    a.update(kw)
    return kda._lib.kda_linear_bwd(ctypes.byref(p), dt, *(a[n] for n in names), nb, None)


def _step(p, dt=1, q=A, k=2 * A, v=3 * A, ld=4 * A, si=5 * A, o=6 * A, so=7 * A):
    return kda._lib.kda_linear_step(ctypes.byref(p), dt, q, k, v, ld, si, o, so, None)


def _rope(p, r, dt=1, q=A, k=2 * A, f=3 * A, pos=4 * A, qo=5 * A, ko=6 * A, which="kda_rope_fwd"):
    return getattr(kda._lib, which)(ctypes.byref(p), ctypes.byref(r), dt, q, k, f, pos, qo, ko, None)


def _norm(rows=4, cols=8, dt=1, x=A, w=2 * A, b=3 * A, eps=1e-5, y=4 * A, m=5 * A, r=6 * A):
    return kda._lib.kda_layernorm_fwd(rows, cols, dt, x, w, b, eps, y, m, r, None)


def _norm_bwd(rows=4, cols=8, dt=1, nb=BIG, **kw):
    names = ("dy", "x", "w", "m", "r", "dx", "dw", "db", "ws")
    a = {n: (i + 1) * A for i, n in enumerate(names)}
    a.update(kw)
    return kda._lib.kda_layernorm_bwd(rows, cols, dt, *(a[n] for n in names), nb, None)


INVALID, UNSUPPORTED = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
MISALIGNED, WORKSPACE = kda.KDA_ERR_MISALIGNED, kda.KDA_ERR_WORKSPACE


@pytest.mark.parametrize("call", [_linear, _linear_bwd])
def test_linear_refusals(call):
    p = _p()
    assert call(_p(d=96)) == UNSUPPORTED and call(_p(d=64, dv=128)) == UNSUPPORTED
    assert call(_p(B=0)) == INVALID and call(_p(text_len=-1)) == INVALID and call(_p(grid=(1, 0, 4))) == INVALID
    assert call(_p(B=65536)) == UNSUPPORTED and call(_p(H=65536)) == UNSUPPORTED
    assert call(p, dt=2) == INVALID
    assert call(_p(reuse_records=True)) == INVALID
    assert call(_p(d=128, qkv_f16=True), dt=0) == INVALID
    for name in ("q", "k", "v", "ld"):
        assert call(p, **{name: None}) == INVALID and call(p, **{name: A + 8}) == MISALIGNED, name
    for name in ("n", "s0"):
        assert call(p, **{name: 40 * A + 4}) == MISALIGNED, name
    assert call(p, ws=None) == WORKSPACE and call(p, ws=20 * A + 128) == WORKSPACE
    need = (kda.kda_linear_workspace_bytes if call is _linear else kda.kda_linear_bwd_workspace_bytes)(p, torch.float32)
    assert need > 256 and call(p, nb=need - 1) == WORKSPACE


def test_linear_outputs_must_not_alias():
    p = _p()
    bytes_ = 2 * 16 * 3 * 64 * 4
    for name in ("q", "k", "v", "ld", "n", "s0"):
        assert _linear(p, **{name: 7 * A}) == INVALID, name               # o over an input
    assert _linear(p, o=A + bytes_ - 16) == INVALID                       # o begins in q's last bytes
    assert _linear(p, sn=7 * A + 16) == INVALID                           # two outputs
    assert _linear(p, s0=30 * A, sn=30 * A) == INVALID                    # the scan does not work in place
    assert _linear(p, ws=7 * A) == INVALID
    for out in ("dq", "dk", "dv", "ds0"):
        assert _linear_bwd(p, **{out: A}) == INVALID, out
    assert _linear_bwd(p, dq=50 * A, dk=50 * A) == INVALID


def test_step_refusals():
    p = _p(text_len=1, grid=(0, 0, 0))
    assert _step(_p()) == INVALID and _step(_p(text_len=0, grid=(0, 0, 0))) == INVALID    # not one token
    for name in ("q", "k", "v", "ld", "si", "o", "so"):
        assert _step(p, **{name: None}) == INVALID and _step(p, **{name: 40 * A + 4}) == MISALIGNED, name
    assert _step(p, so=5 * A + 16) == INVALID     # neither in place nor apart
    assert _step(p, o=5 * A) == INVALID and _step(p, so=A) == INVALID
    assert _step(_p(text_len=1, grid=(0, 0, 0), d=32)) == UNSUPPORTED


@pytest.mark.parametrize("which", ["kda_rope_fwd", "kda_rope_bwd"])
def test_rope_refusals(which):
    p, r = _p(), kda.rope((4, 14, 14))
    call = lambda p=p, r=r, **kw: _rope(p, r, which=which, **kw)   # noqa: E731
    for pairs in ((4, 14, 13), (4, 14, 15), (-4, 18, 18), (0, 0, 0)):
        assert call(r=kda.rope(pairs)) == INVALID, pairs
    assert call(r=kda.kda_rope(4, 14, 14, 2)) == INVALID
    assert call(p=_p(d=80)) == UNSUPPORTED
    for name in ("q", "f", "qo"):
        assert call(**{name: None}) == INVALID, name
    assert call(k=None) == INVALID and call(ko=None) == INVALID       # both or neither
    for name in ("q", "k", "f", "pos", "qo", "ko"):
        assert call(**{name: 40 * A + 4}) == MISALIGNED, name
    assert call(qo=2 * A, ko=50 * A) == INVALID                      # q_out over k
    assert call(qo=A + 64) == INVALID                                # over q, but not in place
    assert call(ko=5 * A) == INVALID                                 # two outputs
    assert call(f=5 * A) == INVALID
    assert call(p=kda.problem(1 << 12, 1, 64, 1 << 20, (0, 0, 0))) == UNSUPPORTED


def test_layernorm_refusals():
    for call in (_norm, _norm_bwd):
        assert call(cols=0) == INVALID and call(rows=-1) == INVALID and call(dt=3) == INVALID
        assert call(cols=16385) == UNSUPPORTED and call(rows=1 << 31) == UNSUPPORTED
        assert call(x=None) == INVALID and call(x=40 * A + 4) == MISALIGNED and call(w=40 * A + 8) == MISALIGNED
    assert _norm(eps=-1.0) == INVALID and _norm(eps=math.nan) == INVALID
    assert _norm(y=A) == INVALID and _norm(y=A + 64) == INVALID and _norm(m=6 * A) == INVALID
    for name in ("dy", "m", "r", "dx"):
        assert _norm_bwd(**{name: None}) == INVALID, name
    assert _norm_bwd(dx=2 * A) == INVALID and _norm_bwd(dw=8 * A) == INVALID and _norm_bwd(ws=6 * A) == INVALID
    assert _norm_bwd(ws=None) == WORKSPACE and _norm_bwd(ws=20 * A + 16) == WORKSPACE
    assert _norm_bwd(nb=kda.kda_layernorm_bwd_workspace_bytes(4, 8) - 1) == WORKSPACE
    assert kda.kda_layernorm_bwd_workspace_bytes(4, 0) == 0
    with pytest.raises(kda.KdaError):
        kda.alloc_layernorm_bwd_workspace(4, 20000)


def test_layernorm_of_no_rows_takes_empty_tensors():
    """A tensor without elements has no address; only what the call would not read or write may lack one."""
    assert _norm(rows=0, x=None, y=None, m=None, r=None) == kda.KDA_OK and kda.kda_last_launch_count() == 0
    none = dict(rows=0, dy=None, x=None, m=None, r=None, dx=None)
    assert _norm_bwd(**none, dw=None, db=None) == kda.KDA_OK and kda.kda_last_launch_count() == 0
    assert _norm(rows=0, x=4, y=None) == MISALIGNED and _norm_bwd(**none, ws=None) == WORKSPACE


def test_a_refused_call_launches_nothing():
    assert _linear(_p(), q=None) and kda.kda_last_launch_count() == 0
    assert _norm(cols=0) and kda.kda_last_launch_count() == 0


def test_binding_checks_tensors_before_the_call():
    B, N, H, d = 2, 16, 3, 64
    p, r = _p(), kda.rope((4, 14, 14))
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)   # noqa: E731
    act, st = lambda: z(B, N, H, d), lambda: z(B, H, d, d)             # noqa: E731
    one = kda.problem(B, H, d, 1, (0, 0, 0))
    calls = {
        "linear_fwd": (lambda a: kda.kda_linear_fwd(p, a["q"], a["k"], a["v"], a["ld"], a["o"], a["ws"], a["n"], a["s0"], a["sn"]),
                       dict(q=act(), k=act(), v=act(), ld=z(H), o=act(), ws=z(1 << 16), n=z(B, dtype=torch.int32), s0=st(), sn=st())),
        "linear_bwd": (lambda a: kda.kda_linear_bwd(p, a["q"], a["k"], a["v"], a["ld"], a["do"], a["dq"], a["dk"], a["dv"], a["ws"],
                                                    a["n"], a["s0"], a["dsn"], a["ds0"]),
                       dict(q=act(), k=act(), v=act(), ld=z(H), do=act(), dq=act(), dk=act(), dv=act(), ws=z(1 << 16),
                            n=z(B, dtype=torch.int32), s0=st(), dsn=st(), ds0=st())),
        "linear_step": (lambda a: kda.kda_linear_step(one, a["q"], a["k"], a["v"], a["ld"], a["si"], a["o"], a["so"]),
                        dict(q=z(B, 1, H, d), k=z(B, 1, H, d), v=z(B, 1, H, d), ld=z(H), si=st(), o=z(B, 1, H, d), so=st())),
        "rope": (lambda a: kda.kda_rope_fwd(p, r, a["q"], a["k"], a["f"], a["qo"], a["ko"], a["pos"]),
                 dict(q=act(), k=act(), f=z(d // 2), qo=act(), ko=act(), pos=z(B, N, 3, dtype=torch.int32))),
        "norm": (lambda a: kda.kda_layernorm_fwd(z(4, 8), a["y"], a["w"], a["b"], 1e-5, a["m"], a["r"]),
                 dict(y=z(4, 8), w=z(8), b=z(8), m=z(4), r=z(4))),
        "norm_bwd": (lambda a: kda.kda_layernorm_bwd(a["dy"], z(4, 8), a["m"], a["r"], a["dx"], a["ws"], a["w"], a["dw"], a["db"]),
                     dict(dy=z(4, 8), m=z(4), r=z(4), dx=z(4, 8), ws=z(4096), w=z(8), dw=z(8), db=z(8))),
    }
    for where, (call, base) in calls.items():
        for n, t in base.items():
            if n == "ws":
                continue
            with pytest.raises(kda.KdaError, match="elements"):
                call(dict(base, **{n: t.reshape(-1)[:-1]}))
            with pytest.raises(kda.KdaError, match="dtype|unsupported"):
                call(dict(base, **{n: t.to(torch.float64)}))
        with pytest.raises(kda.KdaError, match="CUDA tensor"):
            call(base)
    call, base = calls["linear_fwd"]
    with pytest.raises(kda.KdaError, match="contiguous"):
        call(dict(base, v=z(B, H, N, d).transpose(1, 2)))
    with pytest.raises(kda.KdaError):
        kda.alloc_linear_workspace(_p(d=96), torch.float32)
    with pytest.raises(kda.KdaError):
        kda.kda_layernorm_fwd(torch.zeros(()), torch.zeros(()))


@pytest.mark.parametrize("which", ["kda_rope_fwd", "kda_rope_bwd"])
def test_rope_in_place_is_over_the_outputs_own_input_alone(which):
    """One tensor as q and k: q_out over it would turn what k is still read from."""
    p, r = _p(), kda.rope((4, 14, 14))
    call = lambda **kw: _rope(p, r, which=which, **kw)   # noqa: E731
    assert call(q=A, k=A, qo=A, ko=6 * A) == INVALID
    assert call(q=A, k=A, qo=5 * A, ko=A) == INVALID
    assert call(q=A, k=A, qo=A, ko=A) == INVALID
    assert call(q=A, k=2 * A, qo=2 * A, ko=A) == INVALID           # over each other's


def test_step_in_place_is_over_the_state_alone():
    p = _p(text_len=1, grid=(0, 0, 0))
    assert _step(p, q=5 * A, si=5 * A, so=5 * A) == INVALID        # q lies in the state


def test_linear_workspace_sizes_never_fall_as_the_problem_grows():
    """A workspace for the largest problem serves every smaller one: fewer items, heads or tokens never need more."""
    N = [1, 2, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 2048, 2500, 4096, 4608, 4609, 5000, 9216, 10000, 18944, 20000, 40000, 189272]
    pairs = [(1, 1), (1, 2), (1, 3), (1, 8), (1, 13), (1, 16), (2, 16), (3, 16), (9, 16), (10, 15), (19, 16), (37, 16), (64, 24)]
    for size in (kda.kda_linear_workspace_bytes, kda.kda_linear_bwd_workspace_bytes):
        for dtype in (torch.bfloat16, torch.float32):
            for d in (64, 128):
                at = [[size(kda.problem(B, H, d, n, (0, 0, 0)), dtype) for n in N] for B, H in pairs]
                for (B, H), row in zip(pairs, at):
                    assert row == sorted(row) and row[0] > 256, (d, dtype, B, H)
                for n, col in zip(N, zip(*at)):   # by items x heads
                    assert sorted(col) == [s for _, s in sorted((B * H, s) for (B, H), s in zip(pairs, col))], (d, dtype, n)


def test_layernorm_workspace_sizes_never_fall_as_the_problem_grows():
    rows = [0, 1, 2, 15, 16, 147, 148, 149, 295, 296, 297, 591, 592, 593, 5000, 100000]
    cols = [1, 7, 16, 127, 128, 129, 256, 257, 1024, 1025, 2047, 2048, 2049, 3000, 4095, 4096, 4097, 5001, 8192, 8193, 16384]
    at = [[kda.kda_layernorm_bwd_workspace_bytes(r, c) for c in cols] for r in rows]
    for r, row in zip(rows, at):
        assert row == sorted(row), r
    for c, col in zip(cols, zip(*at)):
        assert list(col) == sorted(col), c
