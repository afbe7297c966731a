"""Float64 definitions of the operators around the recurrence, token by token in plain
PyTorch: short causal convolution, selective scan, gated norm, residual norm.

Every function takes tensors of any floating type, widens them, and is differentiable, so
that autograd of these definitions gives the reference gradients.  Token tensors are one
joint axis [tokens, ...]; ``bounds`` lists each sequence's start and the last one's end.
"""
from __future__ import annotations

import torch


def _d(t):
    return None if t is None else t.double()


def _silu(v):
    return v * torch.sigmoid(v)


def short_conv(x, weight, bias=None, initial_state=None, bounds=None, silu=True):
    """x [tokens, C] -> (out [tokens, C], final_state [N, W-1, C]); tokens outside every
    sequence give NaN."""
    x, weight, bias, initial_state = map(_d, (x, weight, bias, initial_state))
    C, W = weight.shape
    rows, finals = [None] * x.shape[0], []
    for n, (s, e) in enumerate(zip(bounds, bounds[1:])):
        past = [initial_state[n, j] if initial_state is not None else x.new_zeros(C) for j in range(W - 1)]
        for t in range(s, e):
            past.append(x[t])
            pre = sum(weight[:, j] * past[len(past) - W + j] for j in range(W))
            if bias is not None:
                pre = pre + bias
            rows[t] = _silu(pre) if silu else pre
        finals.append(torch.stack(past[len(past) - (W - 1):]))
    rows = [x.new_full((C,), float("nan")) if r is None else r for r in rows]
    return (torch.stack(rows) if rows else x.new_zeros(0, C)), (torch.stack(finals) if finals else x.new_zeros(0, W - 1, C))


def softplus(v):
    """log(1 + exp(v)), without overflow, and 0 at -inf."""
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def selective_scan(x, dt, A_log, Bm, Cm, D=None, dt_bias=None, z=None, h0=None, bounds=None):
    """x, dt, z [tokens, C], Bm, Cm [tokens, G, N] -> (out [tokens, C], h_final [n, C, N])."""
    x, dt, A_log, Bm, Cm, D, dt_bias, z, h0 = map(_d, (x, dt, A_log, Bm, Cm, D, dt_bias, z, h0))
    C, N = A_log.shape
    per = C // Bm.shape[1]
    A = -torch.exp(A_log)
    rows, finals = [None] * x.shape[0], []
    for n, (s, e) in enumerate(zip(bounds, bounds[1:])):
        h = h0[n] if h0 is not None else x.new_zeros(C, N)
        for t in range(s, e):
            delta = softplus(dt[t] if dt_bias is None else dt[t] + dt_bias)
            b, c = (m[t].repeat_interleave(per, dim=0) for m in (Bm, Cm))
            h = torch.exp(delta[:, None] * A) * h + (delta * x[t])[:, None] * b
            y = (h * c).sum(-1)
            if D is not None:
                y = y + D * x[t]
            rows[t] = y if z is None else y * _silu(z[t])
        finals.append(h)
    rows = [x.new_full((C,), float("nan")) if r is None else r for r in rows]
    return (torch.stack(rows) if rows else x.new_zeros(0, C)), (torch.stack(finals) if finals else x.new_zeros(0, C, N))


def _rms_norm(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated_norm(x, gate, weight, eps=1e-6):
    x, gate, weight = map(_d, (x, gate, weight))
    return _rms_norm(x, eps) * weight * _silu(gate)


def residual_norm(x, residual, weight, scale=None, post_weight=None, eps=1e-6, stored=None):
    """(out, h).  ``stored``: h as the device stored it, which the norm reads (its rounding
    counts as the identity in the gradient)."""
    x, residual, weight, scale, post_weight = map(_d, (x, residual, weight, scale, post_weight))
    u = x if post_weight is None else _rms_norm(x, eps) * post_weight
    h = residual + (u if scale is None else scale * u)
    read = h if stored is None else h + (stored.double() - h).detach()
    return _rms_norm(read, eps) * weight, h
