"""Inputs and tolerances shared by the tests of the scalar-gate operators.

Tolerances, derived before any run. A rounding to type t is off by at most u_t = eps(t) / 2
relative to the value: bf16 2^-8, fp32 2^-24.

* bf16 outputs computed to fp32 before their one rounding (o, dv): u_bf16 |ref|, and 1e-5 of the
  tensor's RMS times 40 for values that cancel (below).
* dq and dk, whose operands the tensor-core kernels round to bf16 as well: a rounding's error is
  uniform over half a step and so at most u / sqrt(3) of the value in standard deviation; the
  errors of a sum's products are independent, so its standard deviation is at most that times
  the root of the sum of the products' squares, counted once for each rounded factor
  (oracle.gated.grad_squares). Six standard deviations and the last rounding are allowed.
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


def near(name, got, want, squares=None):
    """fp32: the norm of the difference; bf16: every value (see above; `squares` for dq and dk)."""
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    assert g.shape == w.shape, (name, g.shape, w.shape)
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    if w.numel() == 0:
        return
    rms = float(w.square().mean().sqrt())
    if got.dtype == torch.bfloat16:
        tol = U_BF16 * w.abs() + 40 * NORM_F32 * rms
        if squares is not None:
            tol = tol + 6 * U_BF16 / 3 ** 0.5 * squares.sqrt()
        assert ((g - w).abs() <= tol).all(), f"{name}: off by {float((g - w).abs().max()):.3e}, rms {rms:.3e}"
    else:
        err = float((g - w).norm())
        assert err <= NORM_F32 * float(w.norm()), f"{name}: norm off by {err / max(float(w.norm()), 1e-300):.3e}"
        assert float((g - w).abs().max()) <= 40 * NORM_F32 * max(rms, 1e-300) + 4 * NORM_F32 * float(w.abs().max()), name


def near_grads(got, q, k, v, g, b, do, S0=None, dST=None, cu=None):
    """Every gradient of the gated delta rule against fp64."""
    from oracle import gated as ref
    want = ref.gated_bwd(q, k, v, g, b, do, S0, dST, cu)
    squares = dict(zip(("dq", "dk"), ref.grad_squares(q, k, v, g, b, do, S0, dST, cu)))
    for name in want:
        near(name, got[name], want[name], squares.get(name))
