"""Inputs and tolerances shared by the tests of the scalar-gate operators.

Tolerances, derived before any run. A rounding to type t is off by at most u_t = eps(t) / 2
relative to the value: bf16 2^-8, fp32 2^-24.

* bf16 outputs that are otherwise computed in fp32: u_bf16 |ref| for the stored rounding, and
  as much of the tensor's RMS for values that cancel: the tensor-core output product takes the
  state, the pairwise weights and the updates rounded once to bf16 (u_bf16 each, random over the
  d or 64 terms of a sum, so their sum is off by about sqrt(3) u_bf16 / sqrt(3) = u_bf16 of its
  RMS size at one standard deviation); four standard deviations are allowed: 4 u_bf16 RMS.
* fp32 outputs: as a norm, 1e-5 of the norm. The tensor-core kernels split every operand that is
  not a raw input into two bf16 terms: off by at most u_bf16^2 = 1.5e-5 of a value, 2.7e-6 at
  RMS (uniform rounding: u / sqrt(3) times the mean of 1/mantissa, twice), and three such
  products follow one another. CUDA-core kernels: sums of some hundred fp32 terms, 1e-6.
"""
from __future__ import annotations

import torch

U_BF16 = 2.0 ** -8
NORM_F32 = 1e-5


def unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def make(lead, Hk, Hv, dk, dv, dtype, seed, N, gate=-3.0, s0=True):
    """q, k (unit keys), v, g, beta, S0, grad_o, grad_S_T on the CPU. `lead`: the token dimensions."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k = (unit(r(*lead, Hk, dk)) * dk ** -0.5).to(dtype), unit(r(*lead, Hk, dk)).to(dtype)
    v = r(*lead, Hv, dv).to(dtype)
    g = -torch.exp(r(*lead, Hv) * 1.2 + gate)
    beta = 2 * torch.sigmoid(r(*lead, Hv))
    S0 = r(N, Hv, dk, dv) * 0.3 if s0 else None
    return q, k, v, g, beta, S0, r(*lead, Hv, dv).to(dtype), r(N, Hv, dk, dv) * 0.3


def near(name, got, want):
    """fp32: the norm of the difference; bf16: every value (see above)."""
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    assert g.shape == w.shape, (name, g.shape, w.shape)
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    if w.numel() == 0:
        return
    rms = float(w.square().mean().sqrt())
    if got.dtype == torch.bfloat16:
        over = (g - w).abs() - (U_BF16 * w.abs() + 4 * U_BF16 * rms)
        worst = float(over.max())
        assert worst <= 0, f"{name}: off by {float((g - w).abs().max()):.3e}, rms {rms:.3e}"
    else:
        err = float((g - w).norm())
        assert err <= NORM_F32 * float(w.norm()), f"{name}: norm off by {err / max(float(w.norm()), 1e-300):.3e}"
        assert float((g - w).abs().max()) <= 40 * NORM_F32 * max(rms, 1e-300) + 4 * NORM_F32 * float(w.abs().max()), name
