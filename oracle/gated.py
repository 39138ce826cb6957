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


def grad_squares(q, k, v, g, beta, grad_o, S0=None, grad_S_T=None, cu=None, chunk=64):
    """For every element of dq and dk: the sum over its products a b of their squares, counted once
    for each factor that the chunked kernels round to bf16 (states, updates, the weighted pair
    products and the pair products' own factors). Shapes of q, k; fp64. Their square root times a
    rounding's standard deviation is that of the element's error before its last rounding."""
    lead = 2 if cu is None else 1
    spans = bounds(cu, *(q.shape[:2] if cu is None else ()))
    qf, kf, vf, gf, bf, of = (_flat(t, lead) for t in (q, k, v, g, beta, grad_o))
    Hk, dk = qf.shape[1:]
    Hv, dv = vf.shape[1:]
    rep = Hv // Hk
    out_q, out_k = torch.zeros_like(qf), torch.zeros_like(kf)
    for n, (a, e) in enumerate(spans):
        for h in range(Hv):
            kk, qq, vv, gg, bb, oo = kf[a:e, h // rep], qf[a:e, h // rep], vf[a:e, h], gf[a:e, h], bf[a:e, h], of[a:e, h]
            S = torch.zeros(dk, dv, dtype=F64) if S0 is None else _f64(S0)[n, h]
            T = e - a
            starts, U, Rs = {}, torch.zeros(T, dv, dtype=F64), []
            for t in range(T):
                if t % chunk == 0:
                    starts[t] = S
                R = S * torch.exp(gg[t])
                U[t] = bb[t] * (vv[t] - R.T @ kk[t])
                S = R + torch.outer(kk[t], U[t])
            dS = torch.zeros(dk, dv, dtype=F64) if grad_S_T is None else _f64(grad_S_T)[n, h]
            ends, dV = {}, torch.zeros(T, dv, dtype=F64)
            for t in reversed(range(T)):
                if t == T - 1 or (t + 1) % chunk == 0:
                    ends[t // chunk * chunk] = dS
                dS = dS + torch.outer(qq[t], oo[t])
                dV[t] = bb[t] * (dS.T @ kk[t])
                dS = (dS - torch.outer(kk[t], dV[t])) * torch.exp(gg[t])
            for t0, S_in in starts.items():
                z = slice(t0, min(t0 + chunk, T))
                G = gg[z].clamp_min(-128.0).cumsum(0)
                D = torch.exp((G[:, None] - G[None]).clamp_max(0)).tril()
                eg, dec = torch.exp(G)[:, None], torch.exp(G[-1] - G)[:, None]
                u, do, dx, qz, kz = U[z], oo[z], dV[z], qq[z], kk[z]
                Dw, Da = D * (do @ u.T), D.tril(-1) * (dx @ u.T)
                w2 = Dw ** 2 + D ** 2 * (do ** 2 @ u.T ** 2)              # Dw itself, and u in it
                a2 = Da ** 2 + 2 * D.tril(-1) ** 2 * (dx ** 2 @ u.T ** 2)  # Da, u and dV in it
                dS2, S2 = ends[t0].T ** 2, S_in.T ** 2
                tok = slice(a + t0, a + t0 + u.shape[0])
                out_q[tok, h // rep] += eg ** 2 * (do ** 2 @ S2) + w2 @ kz ** 2
                out_k[tok, h // rep] += (2 * eg ** 2 * (dx ** 2 @ S2) + 2 * dec ** 2 * (u ** 2 @ dS2)
                                         + w2.T @ qz ** 2 + a2 @ kz ** 2 + a2.T @ kz ** 2)
    return out_q.reshape(q.shape), out_k.reshape(k.shape)


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
