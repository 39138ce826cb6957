"""fp64 definitions of the scalar-gate operators, token by token (test infrastructure, CPU).

* ``gated_fwd`` / ``gated_bwd``: the gated delta rule with one decay per head on packed
  sequences, S_t = e^{g_t} (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T, o_t = S_t^T q_t, and
  its gradients by autograd of that loop.
* ``prep``: norms of the heads of q or k, weights and the rotation, written with complex
  numbers; its gradients come by autograd too.
* ``copy``: copies of states within a pool, pair by pair from a snapshot.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def _f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def bounds(cu, B=None, T=None):
    """[(first, end)] of every sequence."""
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    cu = [int(x) for x in cu]
    return list(zip(cu[:-1], cu[1:]))


def _loop(q, k, v, g, beta, S0, spans):
    """q, k [tokens, Hk, dk]; v [tokens, Hv, dv]; g, beta [tokens, Hv]; S0 [N, Hv, dk, dv] or None. Rows
    outside the sequences come back as zeros."""
    Hk, dk = q.shape[1:]
    Hv, dv = v.shape[1:]
    rep = Hv // Hk
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    rows = [None] * q.shape[0]
    states = []
    for n, (a, b) in enumerate(spans):
        S = torch.zeros(Hv, dk, dv, dtype=F64) if S0 is None else S0[n]
        for t in range(a, b):
            R = S * torch.exp(g[t])[:, None, None]
            w = v[t] - torch.einsum("hij,hi->hj", R, k[t])
            S = R + torch.einsum("hi,hj->hij", k[t], beta[t][:, None] * w)
            rows[t] = torch.einsum("hij,hi->hj", S, q[t])
        states.append(S)
    zero = torch.zeros(Hv, dv, dtype=F64)
    o = torch.stack([zero if r is None else r for r in rows]) if rows else torch.zeros(0, Hv, dv, dtype=F64)
    ST = torch.stack(states) if states else torch.zeros(0, Hv, dk, dv, dtype=F64)
    return o, ST


def _flat(t, drop):
    t = _f64(t)
    return None if t is None else t.reshape(-1, *t.shape[drop:])


def gated_fwd(q, k, v, g, beta, S0=None, cu=None):
    """Dense [B, T, ...] (cu None) or packed [tokens, ...] inputs. Returns (o, S_T) in their shape, fp64."""
    lead = 2 if cu is None else 1
    spans = bounds(cu, *(q.shape[:2] if cu is None else ()))
    o, ST = _loop(*(_flat(t, lead) for t in (q, k, v, g, beta)), _f64(S0), spans)
    return o.reshape(v.shape), ST


def gated_bwd(q, k, v, g, beta, grad_o, S0=None, grad_S_T=None, cu=None):
    """Gradients of <grad_o, o> + <grad_S_T, S_T>, fp64, in the inputs' shapes."""
    lead = 2 if cu is None else 1
    spans = bounds(cu, *(q.shape[:2] if cu is None else ()))
    x = [_flat(t, lead).requires_grad_() for t in (q, k, v, g, beta)]
    N, (Hv, dv), dk = len(spans), v.shape[-2:], q.shape[-1]
    s0 = (torch.zeros(N, Hv, dk, dv, dtype=F64) if S0 is None else _f64(S0).clone()).requires_grad_()
    o, ST = _loop(*x, s0, spans)
    loss = (o * _flat(grad_o, lead)).sum() + (0 if grad_S_T is None else (ST * _f64(grad_S_T)).sum())
    got = torch.autograd.grad(loss, x + [s0], allow_unused=True)
    names, like = ("dq", "dk", "dv", "dg", "dbeta", "dS0"), (q, k, v, g, beta, s0)
    return {n: (torch.zeros(t.shape, dtype=F64) if r is None else r.reshape(t.shape)) for n, r, t in zip(names, got, like)}


def prep(x, positions=None, inv_freq=None, norm="l2", layout="half", weight=None, eps=1e-6, scale=1.0, rope_scale=1.0):
    """x [tokens, heads, d] fp64 (may require grad), positions [tokens], inv_freq [R / 2]."""
    d = x.shape[-1]
    if norm == "l2":
        n = (x * x).sum(-1, keepdim=True).sqrt()
        x = torch.where(n > 1e-12, x / n.clamp_min(1e-12), x / 1e-12)
    elif norm == "rms":
        x = x / ((x * x).sum(-1, keepdim=True) / d + eps).sqrt()
    if weight is not None:
        x = x * weight
    x = x * scale
    if inv_freq is None or inv_freq.numel() == 0:
        return x
    r = 2 * inv_freq.numel()
    head, rest = x[..., :r], x[..., r:]
    a, b = (head[..., :r // 2], head[..., r // 2:]) if layout == "half" else (head[..., 0::2], head[..., 1::2])
    angle = positions.to(F64)[:, None, None] * inv_freq
    z = torch.complex(a, b) * torch.polar(torch.full_like(angle, rope_scale), angle)
    head = torch.cat([z.real, z.imag], -1) if layout == "half" else torch.stack([z.real, z.imag], -1).flatten(-2)
    return torch.cat([head, rest], -1)


def copy(S, src, dst):
    """S [layers, slots, ...]: pairs in order from a snapshot; indexes beyond the pool are skipped."""
    old, new = S.clone(), S.clone()
    for a, b in zip(src.tolist(), dst.tolist()):
        if b < 0 or b >= S.shape[1] or a >= S.shape[1]:
            continue
        new[:, b] = 0 if a < 0 else old[:, a]
    return new
