"""Token-mixer layers of the hybrid-backbone comparison, with synthetic weights, for timing a
KDA/MLA 3:1 stack against an MHA/MLA 3:1 stack as the token count grows (paper.rainbus.top,
实验结果 and Figure 18; genai-atlas, "Evidence": the hybrid runs 2.14x faster at 255k tokens).

The KDA layer's short conv and scan are this library's kernels (``kda_fwd``), and so are the norm, the
rotary positions and the linear attention of the linear layer; the linear projections are bf16 cuBLAS
GEMMs (torch.matmul), the gate activations are torch element-wise ops, and the softmax attention of the
MHA and MLA layers is PyTorch's fused scaled-dot-product attention (a library kernel, like cuBLAS),
bidirectional over all tokens.

Layer readings (the pages give no sizes for the MLA projections):
  * width D = H * d (16 heads of 128: width 2048, the largest trained model's);
  * MLA: latent c = x Wdkv of d_c = 512; per-head keys c Wuk of d_n = 96 and values c Wuv of 128;
    a key part shared by all heads, k_direct = x Wkr of d_r = 32; queries x Wq of d_n + d_r = 128 per
    head; softmax scale 1/sqrt(128);
  * MHA: q, k, v of 128 per head, softmax scale 1/sqrt(128);
  * KDA: q, k, v projections (q and k scaled to a norm of about 1 per head), log alpha =
    -softplus(x Wa - 5) per channel (alpha near 0.99), beta = sigmoid(x Wb) per head, the
    modality-aware short conv and the scan (no scale on q), output projection;
  * linear (no counterpart in the pages; the mixer with the coarsest memory, one constant decay per
    head, to compare the KDA layer's gates against): layer norm of the input, q, k, v projections,
    rotary positions over (t, h, w) on q and k, linear attention with a decay per head, output
    projection.  It trains (``backward``), takes prompts of different lengths in one padded batch, and
    goes on token by token (``step``).
"""
from __future__ import annotations

import math

import torch
import torch.nn.functional as F

from . import (alloc_layernorm_bwd_workspace, alloc_linear_bwd_workspace, alloc_linear_workspace, alloc_workspace,
               kda_fwd, kda_layernorm_bwd, kda_layernorm_fwd, kda_linear_bwd, kda_linear_fwd, kda_linear_step,
               kda_rope_bwd, kda_rope_fwd, problem, rope)

D_LATENT, D_NOPE, D_DIRECT = 512, 96, 32
GATE_BIAS = -5.0   # log alpha = -softplus(x Wa - 5): alpha near 0.99, the long-memory regime
ROPE_BASE = 10000.0


def _w(g, shape, fan_in, device, scale=1.0):
    return (torch.randn(*shape, generator=g) * (scale / math.sqrt(fan_in))).to(device=device, dtype=torch.bfloat16)


class MHALayer:
    def __init__(self, H, d, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        D = H * d
        self.H, self.d = H, d
        self.wq, self.wk, self.wv = (_w(g, (D, D), D, device) for _ in range(3))
        self.wo = _w(g, (D, D), D, device)

    def attention(self, x):
        """Per-head softmax attention output [B, N, H, d] (bf16), before the output projection."""
        B, N, _ = x.shape
        q, k, v = ((x @ w).view(B, N, self.H, self.d).transpose(1, 2) for w in (self.wq, self.wk, self.wv))
        return F.scaled_dot_product_attention(q, k, v).transpose(1, 2)

    def __call__(self, x):
        B, N, _ = x.shape
        return self.attention(x).reshape(B, N, -1) @ self.wo


class MLALayer:
    def __init__(self, H, d, device="cuda", seed=1):
        g = torch.Generator().manual_seed(seed)
        D = H * d
        self.H, self.d = H, d
        self.wdkv = _w(g, (D, D_LATENT), D, device)
        self.wuk = _w(g, (D_LATENT, H * D_NOPE), D_LATENT, device)
        self.wuv = _w(g, (D_LATENT, H * d), D_LATENT, device)
        self.wkr = _w(g, (D, D_DIRECT), D, device)
        self.wq = _w(g, (D, H * (D_NOPE + D_DIRECT)), D, device)
        self.wo = _w(g, (H * d, D), H * d, device)

    def qkv(self, x):
        """Queries, keys (latent part and the shared part) and values, [B, N, H, .] bf16."""
        B, N, _ = x.shape
        c = x @ self.wdkv
        kc = (c @ self.wuk).view(B, N, self.H, D_NOPE)
        v = (c @ self.wuv).view(B, N, self.H, self.d)
        kr = (x @ self.wkr).view(B, N, 1, D_DIRECT).expand(B, N, self.H, D_DIRECT)
        q = (x @ self.wq).view(B, N, self.H, D_NOPE + D_DIRECT)
        return q, torch.cat([kc, kr], dim=3), v

    def attention(self, x):
        q, k, v = self.qkv(x)
        return F.scaled_dot_product_attention(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2)).transpose(1, 2)

    def __call__(self, x):
        B, N, _ = x.shape
        return self.attention(x).reshape(B, N, -1) @ self.wo


class KDALayer:
    """Projections, then the modality-aware short conv and the KDA scan of this library, then the
    output projection.  Sized for one token layout (text_len + T * Hg * Wg tokens)."""

    def __init__(self, B, H, d, text_len, grid, device="cuda", seed=2, vis_causal_t=False, workspace=None):
        g = torch.Generator().manual_seed(seed)
        D = H * d
        self.B, self.H, self.d, self.text_len, self.grid = B, H, d, text_len, tuple(grid)
        # q and k of norm about 1 per head (beta |k'|^2 < 2 keeps the delta-rule update contracting)
        self.wq, self.wk = (_w(g, (D, D), D, device, 1.0 / math.sqrt(d)) for _ in range(2))
        self.wv = _w(g, (D, D), D, device)
        self.wa = _w(g, (D, D), D, device)
        self.wb = _w(g, (D, H), D, device)
        self.wo = _w(g, (D, D), D, device)
        self.w_text = (torch.randn(3, D, 4, generator=g) / 2.0).to(device)
        self.w_vis = (torch.randn(3, D, 27, generator=g) / math.sqrt(27)).to(device)
        self.p = problem(B, H, d, text_len, self.grid, vis_causal_t=vis_causal_t)
        # the workspace (conv outputs, block records) can be shared by layers that run one after another
        self.ws = alloc_workspace(self.p, torch.bfloat16, device) if workspace is None else workspace

    def inputs(self, x):
        """q, k, v (bf16), log alpha (fp32, -softplus) and beta (bf16, sigmoid) of the scan."""
        B, N, _ = x.shape
        q, k, v = ((x @ w).view(B, N, self.H, self.d).contiguous() for w in (self.wq, self.wk, self.wv))
        la = (-F.softplus((x @ self.wa).float() + GATE_BIAS)).view(B, N, self.H, self.d).contiguous()
        beta = torch.sigmoid(x @ self.wb).contiguous()
        return q, k, v, la, beta

    def mix(self, x):
        """The scan output o [B, N, H, d] (bf16), before the output projection."""
        q, k, v, la, beta = self.inputs(x)
        o = torch.empty_like(q)
        kda_fwd(self.p, q, k, v, la, beta, self.w_text, self.w_vis, o, self.ws)
        return o

    def __call__(self, x):
        B, N, _ = x.shape
        return self.mix(x).view(B, N, -1) @ self.wo


class LinearLayer:
    """Layer norm, projections, rotary positions, linear attention with a constant decay per head, output
    projection.  Sized for one token layout (text_len + T * Hg * Wg tokens); ``step`` takes any position."""

    def __init__(self, B, H, d, text_len, grid, device="cuda", seed=3, workspace=None):
        g = torch.Generator().manual_seed(seed)
        D = H * d
        self.B, self.H, self.d = B, H, d
        # q of norm about 1 and k of about sqrt(d): scores q . k of about 1
        self.wq = _w(g, (D, D), D, device, 1.0 / math.sqrt(d))
        self.wk, self.wv, self.wo = (_w(g, (D, D), D, device) for _ in range(3))
        self.norm_w = (1.0 + 0.1 * torch.randn(D, generator=g)).to(device)
        self.norm_b = (0.1 * torch.randn(D, generator=g)).to(device)
        # heads that forget from within two tokens to over some hundreds
        self.log_decay = torch.tensor([-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)], device=device)
        # a quarter of a head's pairs follow time, the rest height and width; a ladder of frequencies per axis
        n_t = d // 8
        pairs = (n_t, (d // 2 - n_t) // 2, d // 2 - n_t - (d // 2 - n_t) // 2)
        self.rope = rope(pairs)
        self.inv_freq = torch.cat([ROPE_BASE ** (-torch.arange(n, dtype=torch.float64) / n) for n in pairs]).float().to(device)
        self.p = problem(B, H, d, text_len, grid)
        self.p1 = problem(B, H, d, 1, (0, 0, 0))
        self.ws = alloc_linear_workspace(self.p, torch.bfloat16, device) if workspace is None else workspace
        self.ws_bwd = None

    def _qkv(self, p, x, positions, stats=None):
        """The normalised input and q, k (turned), v, each [B, N, H, d]."""
        B, N, D = x.shape
        h = torch.empty_like(x)
        kda_layernorm_fwd(x, h, self.norm_w, self.norm_b, 1e-5, *(stats or (None, None)))
        q, k, v = ((h @ w).view(B, N, self.H, self.d) for w in (self.wq, self.wk, self.wv))
        kda_rope_fwd(p, self.rope, q, k, self.inv_freq, q, k, positions=positions)
        return h, q, k, v

    def mix(self, x, lengths=None, initial_state=None, final_state=None, positions=None):
        """The attention output [B, N, H, d] (bf16), before the output projection."""
        _, q, k, v = self._qkv(self.p, x, positions)
        o = torch.empty_like(v)
        kda_linear_fwd(self.p, q, k, v, self.log_decay, o, self.ws, lengths=lengths, initial_state=initial_state,
                       final_state=final_state)
        return o

    def __call__(self, x, **kw):
        B, N, _ = x.shape
        return self.mix(x, **kw).view(B, N, -1) @ self.wo

    def step(self, x, state, positions):
        """One token per item: x [B, 1, D], positions [B, 1, 3] int32; advances state [B, H, d, d] in place."""
        _, q, k, v = self._qkv(self.p1, x, positions)
        o = torch.empty_like(v)
        kda_linear_step(self.p1, q, k, v, self.log_decay, state, o, state)
        return o.view(self.B, 1, -1) @ self.wo

    def backward(self, x, dy, lengths=None, positions=None, initial_state=None, d_final_state=None, d_initial_state=None):
        """Gradients of sum(dy * self(x)) + sum(d_final_state * final state): that of x, and a dict of the weights'.
        A sequence in pieces gives its piece's initial_state again and gets the gradient for the piece before in
        d_initial_state (fp32 states [B, H, d, d], or None).  The forward pass up to the attention is computed again;
        nothing of it has to be kept.  Tokens behind an item's length change nothing."""
        B, N, D = x.shape
        rows = B * N
        if lengths is not None:   # the weights' products run over all rows: 0 times what stands there has to be 0
            behind = (torch.arange(N, device=x.device) >= lengths.view(B, 1)).unsqueeze(-1)
            x, dy = x.masked_fill(behind, 0), dy.masked_fill(behind, 0)
        mean, rstd = (torch.empty(rows, dtype=torch.float32, device=x.device) for _ in range(2))
        h, q, k, v = self._qkv(self.p, x, positions, (mean, rstd))
        o = torch.empty_like(v)
        kda_linear_fwd(self.p, q, k, v, self.log_decay, o, self.ws, lengths=lengths, initial_state=initial_state)
        if self.ws_bwd is None:
            self.ws_bwd = (alloc_linear_bwd_workspace(self.p, x.dtype, x.device),
                           alloc_layernorm_bwd_workspace(rows, D, x.device))
        d_o = (dy @ self.wo.t()).view(B, N, self.H, self.d)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        kda_linear_bwd(self.p, q, k, v, self.log_decay, d_o, dq, dk, dv, self.ws_bwd[0], lengths=lengths,
                       initial_state=initial_state, d_final_state=d_final_state, d_initial_state=d_initial_state)
        kda_rope_bwd(self.p, self.rope, dq, dk, self.inv_freq, dq, dk, positions=positions)
        flat = lambda t: t.reshape(rows, D)   # noqa: E731
        grads = {"wo": flat(o).t() @ flat(dy), "wq": flat(h).t() @ flat(dq), "wk": flat(h).t() @ flat(dk),
                 "wv": flat(h).t() @ flat(dv)}
        dh = flat(dq) @ self.wq.t()
        dh.addmm_(flat(dk), self.wk.t())
        dh.addmm_(flat(dv), self.wv.t())
        dx = torch.empty_like(x)
        grads["norm_w"], grads["norm_b"] = torch.empty_like(self.norm_w), torch.empty_like(self.norm_b)
        kda_layernorm_bwd(dh, x, mean, rstd, dx, self.ws_bwd[1], self.norm_w, grads["norm_w"], grads["norm_b"])
        return dx, grads


def stack(kind: str, B, H, d, text_len, grid, device="cuda"):
    """Four token mixers: 'kda' = KDA, KDA, KDA, MLA; 'mha' = MHA, MHA, MHA, MLA (the pages' 3:1); 'linear' =
    linear, linear, linear, MLA."""
    if kind in ("kda", "linear"):
        layer = KDALayer if kind == "kda" else LinearLayer
        first = layer(B, H, d, text_len, grid, device, seed=10)
        layers = [first] + [layer(B, H, d, text_len, grid, device, seed=10 + i, workspace=first.ws) for i in (1, 2)]
    elif kind == "mha":
        layers = [MHALayer(H, d, device, seed=10 + i) for i in range(3)]
    else:
        raise ValueError(kind)
    return layers + [MLALayer(H, d, device, seed=20)]


def run_stack(layers, x):
    for layer in layers:
        x = x + layer(x)
    return x
