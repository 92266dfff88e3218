"""The gated delta rule and the norms around a block -- TEST INFRASTRUCTURE
ONLY (like the rest of oracle/): the library never imports it.

Plain float64 PyTorch CPU operations, step by step, from the definitions in
include/ssm.h; gradients by automatic differentiation of those.  Pinned in
tests/test_oracle_blocks.py (closed forms, differences).
"""
from __future__ import annotations

import torch

F64 = torch.float64


def f64(t, grad=False):
    """A float64 CPU copy (None for None)."""
    if t is None:
        return None
    t = t.detach().to("cpu", F64)
    return t.clone().requires_grad_(True) if grad else t


def gdr(q, k, v, delta, A, beta, *, delta_bias=None, delta_softplus=True, beta_sigmoid=True, qk_l2norm=True,
        scale=None, initial_state=None):
    """(out, last_state) on float64 tensors shaped as gdr_chunk_fwd's."""
    B, L, Hk, K = q.shape
    Hv, V = v.shape[-2:]
    scale = K ** -0.5 if scale is None else scale
    if qk_l2norm:
        q = q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
        k = k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    q, k = (t.repeat_interleave(Hv // max(Hk, 1), 2) for t in (q * scale, k))
    dt = delta if delta_bias is None else delta + delta_bias
    if delta_softplus:
        # beyond 100 softplus(x) - x < 4e-44 is nothing in float64; its exp(x) would overflow the derivative
        dt = torch.nn.functional.softplus(dt, threshold=100)
    b = torch.sigmoid(beta) if beta_sigmoid else beta
    S = torch.zeros(B, Hv, V, K, dtype=q.dtype) if initial_state is None else initial_state
    outs = []
    for t in range(L):
        S = torch.exp(dt[:, t] * A)[..., None, None] * S
        u = v[:, t] - (S @ k[:, t].unsqueeze(-1)).squeeze(-1)
        S = S + b[:, t, :, None, None] * u.unsqueeze(-1) * k[:, t].unsqueeze(-2)
        outs.append((S @ q[:, t].unsqueeze(-1)).squeeze(-1))
    out = torch.stack(outs, 1) if outs else torch.zeros(B, 0, Hv, V, dtype=q.dtype)
    return out, S


def gated_norm(x, weight, *, z=None, group=None, eps=1e-5, norm_before_gate=False):
    g = x.shape[-1] if group is None else group
    gate = 1.0 if z is None else z * torch.sigmoid(z)
    u = x if norm_before_gate else x * gate
    r = u.reshape(*x.shape[:-1], -1, g)
    n = (r / (r.pow(2).mean(-1, keepdim=True) + eps).sqrt()).reshape(x.shape)
    return n * weight * gate if norm_before_gate else n * weight


def residual_update(x, *, residual=None, scale=None, post_weight=None, alpha=1.0, eps=1e-5):
    t = x
    if post_weight is not None:
        t = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * post_weight
    if scale is not None:
        s = scale if scale.dim() == 2 else scale.unsqueeze(0)
        t = t.reshape(s.shape[0], -1, x.shape[-1]) * s.unsqueeze(1)
        t = t.reshape(x.shape)
    return t if residual is None else alpha * residual + t


def norm(r, weight, *, bias=None, layer_norm=False, eps=1e-5):
    c = r - r.mean(-1, keepdim=True) if layer_norm else r
    y = c / (c.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight
    return y if bias is None else y + bias
