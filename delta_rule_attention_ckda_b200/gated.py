"""Binding of the scalar-gate operators (argument marshalling only; every step runs in CUDA).

    gated_chunk_fwd(q, k, v, g, beta, S0=None)    -> (o, S_T)
    gated_bwd(q, k, v, g, beta, grad_o, S0=None)  -> gradients
    gated_decode_step(q, k, v, g, beta, S)        -> o   (states of a pool, in place)
    qk_norm_rope(q, k) / qk_norm_rope_bwd(...)    -> queries and keys ready for the rule
    state_copy(S, src, dst)                       -> S   (forks, moves and clears states)

The rule, per sequence and value head, with one decay e^{g_t} per token:

    S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t

q and k have Hk heads, v, g, beta and the states Hv, a multiple of Hk. Dense tensors are
[B, T, heads, d]; with cu_seqlens (int32 [N+1], device) they are packed, [total, heads, d].
q, k and v may be slices of wider rows (heads and channels contiguous, one distance from token
to token); for the tensor cores, which take bf16 heads of a multiple of 8 channels, they start
on 16 bytes and that distance is a multiple of 8 elements. The full conventions are in
include/ckda.h.
"""
from __future__ import annotations

from functools import lru_cache
from math import prod
from typing import Optional, Tuple

import torch

from ._lib import _device, _dt, _raise, load

NORMS = {"none": 0, "l2": 1, "rms": 2}          # ckda_prep_norm_t
LAYOUTS = {"half": 0, "interleaved": 1}
F32, I32 = torch.float32, torch.int32


# The checks below run in front of calls of a few microseconds, so each is a few comparisons.

def _on(t, name: str, dev) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
        raise ValueError(f"{name} is on {t.device}, the call's tensors are on {dev}")


def _check(t, name: str, shape, dtype, dev) -> None:
    """Type, device, shape, dtype and contiguity of one tensor argument."""
    _on(t, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name: str, lead: int, dtype, dev) -> int:
    """Checks a tensor of rows [..., heads, d] with `lead` leading token dimensions whose heads
    and channels are contiguous; returns the distance from token to token in elements."""
    _on(t, name, dev)
    if t.dim() != lead + 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {lead + 2} dimensions")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    heads, d = shape[-2], shape[-1]
    inner = heads * d
    if t.is_contiguous() or t.numel() == 0:
        return inner or 1
    st = t.stride()
    if (d > 1 and st[-1] != 1) or (heads > 1 and st[-2] != d):
        raise ValueError(f"{name} must have contiguous heads and channels, has strides {st}")
    row = None                                    # the distance between tokens, over every leading dimension
    step = 1
    for i in range(lead - 1, -1, -1):
        if t.shape[i] > 1:
            if row is None:
                row = st[i] // step if st[i] % step == 0 else -1
            if st[i] != row * step:
                raise ValueError(f"{name} must have one distance from token to token, has strides {st}")
        step *= t.shape[i]
    row = max(inner, 1) if row is None else row
    if row < inner:
        raise ValueError(f"{name} has overlapping tokens, strides {st}")
    return row


def _count(n: int, what: str) -> None:
    """The library counts in 32 bits; ctypes would cut a larger number to its lower half."""
    if n > 0x7fffffff:
        raise ValueError(f"more than 2**31 - 1 {what}")


def _indexes(t, name: str, n: Optional[int], dev) -> None:
    _on(t, name, dev)
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {'one dimension' if n is None else (n,)}")
    if t.dtype != I32:
        raise TypeError(f"{name} must be {I32}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _span(t):
    """[first, end) of a tensor's memory; None for no tensor or an empty one."""
    if t is None:
        return None
    n = t.numel()
    if n == 0:
        return None
    a = t.data_ptr()
    if not t.is_contiguous():
        n = sum((k - 1) * s for k, s in zip(t.shape, t.stride())) + 1
    return a, a + n * t.element_size()


def _apart(out, name: str, others) -> None:
    """An output may share memory with none of `others` ((name, tensor) pairs; None names none)."""
    mine = _span(out)
    if mine is None:
        return
    a, b = mine
    for other, t in others:
        if t is None:
            continue
        p = t.data_ptr()
        if p >= b or p == 0:
            continue
        span = _span(t)
        if span is not None and a < span[1]:
            raise ValueError(f"{name} overlaps {other}")


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle of a device, without making a stream object where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev, stream, fn, where: str, args) -> None:
    """Calls fn(*args, stream) with `dev` as the current device, which the library launches on."""
    if stream is None:
        raw = _raw_stream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the call's tensors are on {dev}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st:
        _raise(st, where)


@lru_cache(maxsize=4096)
def _bytes(which: str, device_index: int, sizes) -> int:
    """A workspace query: a function of the sizes and the device alone."""
    with torch.cuda.device(device_index):
        return int(getattr(load(), which)(*sizes))


def _empty(like, shape, stream, dtype=None):
    """New memory on like's device and (unless given) of its type, for a call on `stream`: of that
    stream, so that torch hands it out again only behind the call, whatever the current stream is."""
    if stream is None:
        return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)
    if stream.device != like.device:
        raise ValueError(f"stream is on {stream.device}, the call's tensors are on {like.device}")
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _workspace(which: str, dev, sizes, workspace, stream, like, used):
    need = _bytes(which, dev.index, sizes)
    if workspace is None:
        if need == 0:
            return None, 0
        return _empty(like, need, stream, torch.uint8), need
    _on(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _apart(workspace, "workspace", used)
    return workspace, workspace.numel() * workspace.element_size()


def _given(grads, names) -> dict:
    """The outputs given for a backward call, by name."""
    got = dict(grads or {})
    for name in got:
        if name not in names:
            raise ValueError(f"grads has no {name!r}, only {', '.join(names)}")
    return got


def _call_device(t, name: str = "q"):
    dev = _device(t, name)
    return dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())


class _Problem:
    """The checked inputs of a gated delta rule call."""

    def __init__(self, q, k, v, g, beta, S0, cu_seqlens):
        dev = self.dev = _call_device(q)
        packed = cu_seqlens is not None
        lead = 1 if packed else 2
        qs = _rows(q, "q", lead, None, dev)
        dt = q.dtype
        self.dt = _dt(q)
        ks, vs = _rows(k, "k", lead, dt, dev), _rows(v, "v", lead, dt, dev)
        tokens = tuple(q.shape[:lead])
        Hk, dk = q.shape[-2:]
        Hv, dv = v.shape[-2:]
        if k.shape != q.shape:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected {tuple(q.shape)}")
        if tuple(v.shape[:lead]) != tokens:
            raise ValueError(f"v has shape {tuple(v.shape)}, expected {tokens + (Hv, dv)}")
        if Hk < 1 or Hv < 1 or Hv % Hk != 0:
            raise ValueError(f"v has {Hv} heads, not a multiple of the {Hk} of q and k")
        _check(g, "g", tokens + (Hv,), F32, dev)
        _check(beta, "beta", tokens + (Hv,), F32, dev)
        if packed:
            _indexes(cu_seqlens, "cu_seqlens", None, dev)
            if cu_seqlens.shape[0] < 1:
                raise ValueError("cu_seqlens must hold N + 1 offsets")
            N, T, total = cu_seqlens.shape[0] - 1, 0, tokens[0]
        else:
            N, T = tokens
            total = N * T
        _count(max(total, N, T), "tokens")
        self.o_shape = tokens + (Hv, dv)
        self.g_shape = tokens + (Hv,)
        self.state_shape = (N, Hv, dk, dv)
        if S0 is not None:
            _check(S0, "S0", self.state_shape, F32, dev)
        self.spans = [("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta),
                      ("cu_seqlens", cu_seqlens)]
        self.sizes = (N, T, total, Hk, Hv, dk, dv, qs, ks, vs, self.dt)
        self.ws_sizes = (N, total, Hk, Hv, dk, dv, self.dt)


def gated_fwd_workspace_bytes(N, total, Hk, Hv, dk, dv, dtype=torch.bfloat16) -> int:
    return int(load().ckda_gated_fwd_workspace_bytes(N, total, Hk, Hv, dk, dv, _dt(torch.empty(0, dtype=dtype))))


def gated_segment_tokens(N, total, Hk, Hv, dk, dv, dtype=torch.bfloat16) -> int:
    """Tokens in a segment where gated_chunk_fwd runs long sequences as segments (0: whole)."""
    return int(load().ckda_gated_fwd_segment_tokens(N, total, Hk, Hv, dk, dv, _dt(torch.empty(0, dtype=dtype))))


def gated_bwd_segment_tokens(N, total, Hk, Hv, dk, dv, dtype=torch.bfloat16) -> int:
    """As gated_segment_tokens, of gated_bwd's own plan."""
    return int(load().ckda_gated_bwd_segment_tokens(N, total, Hk, Hv, dk, dv, _dt(torch.empty(0, dtype=dtype))))


def gated_chunk_fwd(q, k, v, g, beta, S0=None, *, cu_seqlens=None, o=None, S_T=None, want_state=True, workspace=None,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """ckda_gated_fwd. Returns (o, S_T): o in v's type and shape (rows behind the last packed
    sequence are not written), S_T [N, Hv, dk, dv] fp32, which may be S0 itself. Allocates o, S_T
    and the workspace with torch when not given."""
    p = _Problem(q, k, v, g, beta, S0, cu_seqlens)
    dev = p.dev
    spans = p.spans
    if o is None:
        o = _empty(v, p.o_shape, stream)
    else:
        _check(o, "o", p.o_shape, v.dtype, dev)
        _apart(o, "o", spans + [("S0", S0)])
    if S_T is not None:
        _check(S_T, "S_T", p.state_shape, F32, dev)
        same = S0 is not None and S_T.data_ptr() == S0.data_ptr()
        _apart(S_T, "S_T", spans + [("o", o)] + ([] if same else [("S0", S0)]))
    elif want_state:
        S_T = _empty(g, p.state_shape, stream)
    workspace, wbytes = _workspace("ckda_gated_fwd_workspace_bytes", dev, p.ws_sizes, workspace, stream, g,
                                   spans + [("S0", S0), ("o", o), ("S_T", S_T)])
    _launch(dev, stream, load().ckda_gated_fwd, "ckda_gated_fwd",
            (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T), _ptr(cu_seqlens), *p.sizes,
             _ptr(workspace), wbytes))
    return o, S_T


def gated_bwd_workspace_bytes(N, total, Hk, Hv, dk, dv, dtype=torch.bfloat16) -> int:
    return int(load().ckda_gated_bwd_workspace_bytes(N, total, Hk, Hv, dk, dv, _dt(torch.empty(0, dtype=dtype))))


def gated_bwd(q, k, v, g, beta, grad_o, S0=None, grad_S_T=None, *, cu_seqlens=None, want_dS0=True, grads=None,
              workspace=None, stream=None):
    """ckda_gated_bwd: gradients of L = <grad_o, o> + <grad_S_T, S_T> for gated_chunk_fwd. Returns a
    dict with dq, dk, dv (in q's type), dg, dbeta, dS0 (fp32; dS0 None unless want_dS0). Output
    tensors may be passed in `grads` (same keys); dS0 may be grad_S_T itself. Rows behind the last
    packed sequence are not written."""
    p = _Problem(q, k, v, g, beta, S0, cu_seqlens)
    dev = p.dev
    _check(grad_o, "grad_o", p.o_shape, v.dtype, dev)
    if grad_S_T is not None:
        _check(grad_S_T, "grad_S_T", p.state_shape, F32, dev)
    got = _given(grads, ("dq", "dk", "dv", "dg", "dbeta", "dS0"))
    shapes = {"dq": (q.shape, q.dtype), "dk": (q.shape, q.dtype), "dv": (p.o_shape, q.dtype), "dg": (p.g_shape, F32),
              "dbeta": (p.g_shape, F32), "dS0": (p.state_shape, F32)}
    given = []
    for name, (shape, dtype) in shapes.items():
        if name == "dS0" and not want_dS0:
            got[name] = None
        elif got.get(name) is None:
            got[name] = _empty(q if dtype is q.dtype else g, shape, stream)
        else:
            _check(got[name], name, shape, dtype, dev)
            given.append(name)
    for i, name in enumerate(given):
        others = p.spans + [("grad_o", grad_o), ("S0", S0)] + [(n, got[n]) for n in given[:i]]
        if not (name == "dS0" and grad_S_T is not None and got[name].data_ptr() == grad_S_T.data_ptr()):
            others.append(("grad_S_T", grad_S_T))
        _apart(got[name], name, others)
    workspace, wbytes = _workspace("ckda_gated_bwd_workspace_bytes", dev, p.ws_sizes, workspace, stream, g,
                                   p.spans + [("S0", S0), ("grad_o", grad_o), ("grad_S_T", grad_S_T), *got.items()])
    _launch(dev, stream, load().ckda_gated_bwd, "ckda_gated_bwd",
            (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(grad_o), _ptr(grad_S_T), _ptr(got["dq"]),
             _ptr(got["dk"]), _ptr(got["dv"]), _ptr(got["dg"]), _ptr(got["dbeta"]), _ptr(got["dS0"]), _ptr(cu_seqlens),
             *p.sizes, _ptr(workspace), wbytes))
    return got


def gated_decode_step(q, k, v, g, beta, S, *, slots=None, o=None, stream=None) -> torch.Tensor:
    """ckda_gated_decode_step: one token of N sequences, q, k [N, Hk, dk], v [N, Hv, dv], g, beta
    [N, Hv]. Updates states of the pool S [P, Hv, dk, dv] in place: row n's is S[slots[n]] (int32;
    None: S[n]); rows with a negative slot are padding and keep their o. Returns o [N, Hv, dv]."""
    dev = _call_device(q)
    qs = _rows(q, "q", 1, None, dev)
    dt = q.dtype
    ks, vs = _rows(k, "k", 1, dt, dev), _rows(v, "v", 1, dt, dev)
    shape = q.shape
    N, Hk, dk = shape
    rows, Hv, dv = v.shape
    if k.shape != shape:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected {tuple(shape)}")
    if rows != N:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected {(N, Hv, dv)}")
    if Hk < 1 or Hv < 1 or Hv % Hk != 0:
        raise ValueError(f"v has {Hv} heads, not a multiple of the {Hk} of q and k")
    _check(g, "g", (N, Hv), F32, dev)
    _check(beta, "beta", (N, Hv), F32, dev)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be a [pool, Hv, dk, dv] tensor")
    pool = S.shape[0]
    _count(max(N, pool), "rows or states")
    _check(S, "S", (pool, Hv, dk, dv), F32, dev)
    if slots is not None:
        _indexes(slots, "slots", N, dev)
    elif pool < N:
        raise ValueError(f"S holds {pool} states, the call has {N} rows")
    spans = [("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("slots", slots)]
    _apart(S, "S", spans)
    if o is None:
        o = _empty(v, (N, Hv, dv), stream)
    else:
        _check(o, "o", (N, Hv, dv), dt, dev)
        _apart(o, "o", spans + [("S", S)])
    _launch(dev, stream, load().ckda_gated_decode_step, "ckda_gated_decode_step",
            (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o), _ptr(slots), N, pool, Hk, Hv, dk, dv, qs, ks,
             vs, _dt(q)))
    return o


class _Prep:
    """The checked arguments that qk_norm_rope and its backward share."""

    def __init__(self, q, k, positions, inv_freq, norm, layout, q_weight, k_weight, eps, q_scale, rope_scale):
        dev = self.dev = _call_device(q)
        if q.dim() < 3:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected [..., heads, d]")
        lead = q.dim() - 2
        self.qs = _rows(q, "q", lead, None, dev)
        self.dt = _dt(q)
        shape = q.shape
        self.tokens_shape = shape[:-2]
        self.Hq, self.d = shape[-2], shape[-1]
        self.Hk, self.ks = 0, 0
        if k is not None:
            self.ks = _rows(k, "k", lead, q.dtype, dev)
            self.Hk = k.shape[-2]
            if k.shape != self.tokens_shape + (self.Hk, self.d):
                raise ValueError(f"k has shape {tuple(k.shape)}, expected {tuple(self.tokens_shape) + (self.Hk, self.d)}")
        tokens = prod(self.tokens_shape)
        _count(tokens, "tokens")
        if norm not in NORMS:
            raise ValueError(f"norm must be one of {sorted(NORMS)}, got {norm!r}")
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _check(w, name, (self.d,), F32, dev)
        rotary, pos64 = 0, 0
        if inv_freq is not None:
            if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
                raise ValueError("inv_freq must be a tensor of one dimension")
            _check(inv_freq, "inv_freq", inv_freq.shape, torch.float64, dev)
            rotary = 2 * inv_freq.numel()
            if rotary > self.d:
                raise ValueError(f"inv_freq turns {rotary} channels, a head has {self.d}")
        if positions is not None:
            if inv_freq is None:
                raise ValueError("positions without inv_freq")
            if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
                raise TypeError("positions must be an int32 or int64 tensor")
            _check(positions, "positions", self.tokens_shape, positions.dtype, dev)
            pos64 = int(positions.dtype == torch.int64)
        self.spans = [("q", q), ("k", k), ("q_weight", q_weight), ("k_weight", k_weight),
                      ("positions", positions), ("inv_freq", inv_freq)]
        self.ptrs = (_ptr(q_weight), _ptr(k_weight), _ptr(positions), pos64, _ptr(inv_freq))
        self.sizes = (tokens, max(1, self.tokens_shape[-1]), self.Hq, self.Hk, self.d, rotary, self.qs, self.ks, self.dt,
                      NORMS[norm], LAYOUTS[layout], float(eps), float(q_scale), float(rope_scale))

    def out(self, t, name, like, others, stream):
        """An output of like's shape and type, allocated or checked to share memory with none of `others`."""
        if t is None:
            return torch.empty_like(like) if stream is None and like.is_contiguous() else _empty(like, like.shape, stream)
        _check(t, name, like.shape, like.dtype, self.dev)
        _apart(t, name, others)
        return t


def qk_norm_rope(q, k=None, *, positions=None, inv_freq=None, norm="l2", layout="half", q_weight=None, k_weight=None,
                 eps=1e-6, q_scale=1.0, rope_scale=1.0, q_out=None, k_out=None, stream=None):
    """ckda_qk_prep: the norm of every head of q [..., Hq, d] and k [..., Hk, d], weights, and the
    rotation of the first 2 * len(inv_freq) channels by the tokens' positions, in one pass.
    norm: "l2", "rms" (with eps) or "none"; layout: pairs (p, p + R/2) ("half") or (2p, 2p + 1)
    ("interleaved"). inv_freq is fp64 (see rope_frequencies); positions int32 or int64 of the
    tokens' shape, None: the index along the last token dimension. Returns (q_out, k_out), which may
    be q and k themselves where those are contiguous (k_out None without k)."""
    p = _Prep(q, k, positions, inv_freq, norm, layout, q_weight, k_weight, eps, q_scale, rope_scale)

    def others(t, src, own):
        if t is None:
            return ()
        same = src.is_contiguous() and t.data_ptr() == src.data_ptr()
        return [x for x in p.spans if not (same and x[0] == own)]

    q_out = p.out(q_out, "q_out", q, others(q_out, q, "q"), stream)
    if k is None:
        k_out = None
    else:
        k_out = p.out(k_out, "k_out", k, [*others(k_out, k, "k"), ("q_out", q_out)], stream)
    _launch(p.dev, stream, load().ckda_qk_prep, "ckda_qk_prep",
            (_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), *p.ptrs, *p.sizes))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, grad_q, grad_k=None, *, positions=None, inv_freq=None, norm="l2", layout="half", q_weight=None,
                     k_weight=None, eps=1e-6, q_scale=1.0, rope_scale=1.0, grads=None, workspace=None, stream=None):
    """ckda_qk_prep_bwd: gradients of qk_norm_rope from those of its outputs. Returns a dict with dq,
    dk (contiguous, in q's type) and dq_weight, dk_weight (fp32 [d]; None without that weight).
    Output tensors may be passed in `grads` (same keys)."""
    p = _Prep(q, k, positions, inv_freq, norm, layout, q_weight, k_weight, eps, q_scale, rope_scale)
    _check(grad_q, "grad_q", p.tokens_shape + (p.Hq, p.d), q.dtype, p.dev)
    if (k is None) != (grad_k is None):
        raise ValueError("k and grad_k come together")
    if k is not None:
        _check(grad_k, "grad_k", p.tokens_shape + (p.Hk, p.d), q.dtype, p.dev)
    got = _given(grads, ("dq", "dk", "dq_weight", "dk_weight"))
    spans = p.spans + [("grad_q", grad_q), ("grad_k", grad_k)]
    got["dq"] = p.out(got.get("dq"), "dq", q, spans, stream)
    spans.append(("dq", got["dq"]))
    got["dk"] = p.out(got.get("dk"), "dk", k, spans, stream) if k is not None else None
    spans.append(("dk", got["dk"]))
    weights = False
    for name, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        if w is None:
            got[name] = None
            continue
        weights = True
        if got.get(name) is None:
            got[name] = _empty(w, (p.d,), stream)
        else:
            _check(got[name], name, (p.d,), F32, p.dev)
            _apart(got[name], name, spans)
        spans.append((name, got[name]))
    wbytes = 0
    if weights or workspace is not None:
        workspace, wbytes = _workspace("ckda_qk_prep_bwd_workspace_bytes", p.dev, (p.d,), workspace, stream, q, spans)
    _launch(p.dev, stream, load().ckda_qk_prep_bwd, "ckda_qk_prep_bwd",
            (_ptr(q), _ptr(k), _ptr(grad_q), _ptr(grad_k), _ptr(got["dq"]), _ptr(got["dk"]), _ptr(got["dq_weight"]),
             _ptr(got["dk_weight"]), *p.ptrs, *p.sizes, _ptr(workspace), wbytes))
    return got


def rope_frequencies(rotary: int, base: float = 10000.0, *, factor: float = 1.0, scaling: str = "none",
                     trained: int = 4096, slow: float = 1.0, fast: float = 32.0, device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq, rope_scale) for qk_norm_rope: fp64 [rotary / 2] frequencies base^(-2p / rotary),
    scaled for contexts `factor` times the `trained` length:
      "none":    as they are;
      "linear":  all divided by factor (positions interpolated);
      "base":    base * factor^(rotary / (rotary - 2)), which leaves the fastest pair alone and
                 divides the slowest by factor;
      "by_parts": pairs that turn more than `fast` times in the trained length are left alone,
                 those that turn less than `slow` times are divided by factor, between them a ramp
                 in the pair index (which goes past the last pair where that still turns more than
                 `slow` times); rope_scale is then 0.1 ln(factor) + 1."""
    import math
    if rotary < 2 or rotary % 2 != 0:
        raise ValueError(f"rotary must be even and at least 2, got {rotary}")
    if not (base > 1.0 and factor >= 1.0 and trained >= 1 and 0 < slow < fast):
        raise ValueError("need base > 1, factor >= 1, trained >= 1 and 0 < slow < fast")
    p = torch.arange(0, rotary, 2, dtype=torch.float64) / rotary
    scale = 1.0
    if scaling == "none":
        f = base ** -p
    elif scaling == "linear":
        f = base ** -p / factor
    elif scaling == "base":
        if rotary < 4:
            raise ValueError("scaling by the base needs two pairs at least")
        f = (base * factor ** (rotary / (rotary - 2))) ** -p
    elif scaling == "by_parts":
        def index(turns):                         # the (real) pair index that turns this often in `trained` tokens
            return rotary * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(fast)), 0), math.ceil(index(slow))
        ramp = ((torch.arange(rotary // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        if hi <= 0:                               # even the first pair turns less than `slow` times
            ramp.fill_(1)
        f = base ** -p * (1 - ramp + ramp / factor)
        scale = 0.1 * math.log(factor) + 1.0
    else:
        raise ValueError(f"scaling must be one of none, linear, base, by_parts, got {scaling!r}")
    return f.to(device) if device is not None else f, scale


def state_copy(S, src, dst, *, pool_dim=0, stream=None) -> torch.Tensor:
    """ckda_state_copy, in place on a pool of states S [P, Hv, dk, dv] (pool_dim 0), or on every
    layer's, S [L, P, Hv, dk, dv] (pool_dim 1): slot dst[i] takes the state of slot src[i] as it was
    before the call, or zeros where src[i] is negative; a negative dst[i] names nothing; of pairs
    with the same dst the last counts. src, dst: int32, at most 1024. Returns S."""
    dev = _call_device(S, "S")
    if pool_dim not in (0, 1) or S.dim() < pool_dim + 2:
        raise ValueError(f"S has shape {tuple(S.shape)}, with the pool in dimension {pool_dim}")
    _check(S, "S", S.shape, F32, dev)
    _indexes(src, "src", None, dev)
    _indexes(dst, "dst", src.shape[0], dev)
    _apart(S, "S", [("src", src), ("dst", dst)])
    layers, slots = S.shape[0] if pool_dim else 1, S.shape[pool_dim]
    if slots == 0:
        raise ValueError("S holds no states")
    _count(max(layers, slots), "layers or states")
    _launch(dev, stream, load().ckda_state_copy, "ckda_state_copy",
            (_ptr(S), _ptr(src), _ptr(dst), src.shape[0], layers, slots, prod(S.shape[pool_dim + 1:])))
    return S
