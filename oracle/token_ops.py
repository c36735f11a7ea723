"""fp64 reference of the operators beside the KDA scan: linear attention with a decay per head, rotary
positions over (time, height, width), layer norm.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``: only ``tests/`` may import it.  Plain torch in fp64 on
whatever device the inputs are, written from the definitions: the recurrence token by token, the rotation pair
by pair, the norm and its gradient row by row.
"""
from __future__ import annotations

import torch


def _until(x, lengths):
    """x [B, N, ...] in fp64 with zeros behind each item's length (whatever stood there)."""
    x = x.double()
    if lengths is None:
        return x
    n = torch.arange(x.shape[1], device=x.device).view(1, -1, *[1] * (x.dim() - 2))
    return torch.where(n < lengths.to(x.device).view(-1, 1, *[1] * (x.dim() - 2)), x, torch.zeros((), dtype=x.dtype, device=x.device))


def linear_fwd(q, k, v, log_decay, lengths=None, S0=None):
    """o [B, N, H, d] and the state behind each item's last token [B, H, d, d]."""
    q, k, v = (_until(x, lengths) for x in (q, k, v))
    B, N, H, d = q.shape
    lam = log_decay.double().exp().view(1, H, 1, 1)
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if S0 is None else S0.double().clone()
    o = torch.zeros_like(v)
    n = torch.full((B,), N, device=q.device) if lengths is None else lengths.clamp(0, N)
    for t in range(N):
        live = (t < n).view(B, 1, 1, 1)
        S = torch.where(live, lam * S + k[:, t].unsqueeze(-1) * v[:, t].unsqueeze(-2), S)
        o[:, t] = (S * q[:, t].unsqueeze(-1)).sum(-2)
    return o, S


def linear_bwd(q, k, v, log_decay, d_o, lengths=None, S0=None, dSN=None):
    """dq, dk, dv, dS0 of sum(d_o * o) + sum(dSN * S_N)."""
    q, k, v, d_o = (_until(x, lengths) for x in (q, k, v, d_o))
    B, N, H, d = q.shape
    lam = log_decay.double().exp().view(1, H, 1, 1)
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if S0 is None else S0.double().clone()
    G = torch.zeros_like(S) if dSN is None else dSN.double().clone()
    n = torch.full((B,), N, device=q.device) if lengths is None else lengths.clamp(0, N)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(N):
        live = (t < n).view(B, 1, 1, 1)
        S = torch.where(live, lam * S + k[:, t].unsqueeze(-1) * v[:, t].unsqueeze(-2), S)
        dq[:, t] = (S * d_o[:, t].unsqueeze(-2)).sum(-1)
    for t in range(N - 1, -1, -1):
        live = (t < n).view(B, 1, 1, 1)
        at = G + q[:, t].unsqueeze(-1) * d_o[:, t].unsqueeze(-2)     # the gradient of S_t
        dk[:, t] = (at * v[:, t].unsqueeze(-2)).sum(-1)
        dv[:, t] = (at * k[:, t].unsqueeze(-1)).sum(-2)
        G = torch.where(live, lam * at, G)
    return dq, dk, dv, G


def grid_positions(B, text, grid):
    """[B, N, 3]: text token i at (i, i, i), visual token (t, h, w) at text + (t, h, w)."""
    T, Hg, Wg = grid
    rows = [(i, i, i) for i in range(text)]
    rows += [(text + t, text + h, text + w) for t in range(T) for h in range(Hg) for w in range(Wg)]
    return torch.tensor(rows, dtype=torch.int64).view(1, -1, 3).expand(B, -1, -1)


def rope(x, inv_freq, positions, pairs, interleaved=False, inverse=False):
    """x [B, N, H, d] with every pair turned by positions[b, n, axis] * inv_freq[j]."""
    x = x.double()
    d = x.shape[-1]
    axis = [0] * pairs[0] + [1] * pairs[1] + [2] * pairs[2]
    out = torch.empty_like(x)
    for j in range(d // 2):
        w = positions[..., axis[j]].to(x.device).double() * inv_freq[j].to(x.device).double()
        c, s = torch.cos(w).unsqueeze(-1), torch.sin(w).unsqueeze(-1)
        if inverse:
            s = -s
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + d // 2)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def layernorm_fwd(x, weight=None, bias=None, eps=1e-5):
    """y, mean, rstd of x [rows, cols]."""
    x = x.double()
    mean = x.mean(1)
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, mean, rstd


def layernorm_bwd(dy, x, mean, rstd, weight=None):
    """dx, d_weight, d_bias at the statistics that the forward pass gave."""
    dy, x = dy.double(), x.double()
    h = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy if weight is None else dy * weight.double()
    dx = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)
