"""Host-side checks of the scalar-gate operators that need no GPU: the C entries reject bad
arguments before any launch, workspace and plan queries, the binding's checks, the frequency
helper, and the fp64 definitions the GPU tests rely on."""
import ctypes
import math

import pytest
import torch

from gated_util import make
from oracle import gated as ref

BF, F32 = 1, 0
P = ctypes.c_void_p(0x10000)              # never followed: every call below returns before a launch
ODD16, ODD4 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    from delta_rule_attention_ckda_b200 import build
    build.build()
    import delta_rule_attention_ckda_b200 as ck
    return ck.load()


def fwd(lib, q=P, k=P, v=P, g=P, beta=P, S0=None, o=P, ST=None, cu=None, N=1, T=4, total=4, Hk=1, Hv=1, dk=16, dv=16,
        qs=16, ks=16, vs=16, dt=BF, ws=P, wb=1 << 40):
    return lib.ckda_gated_fwd(q, k, v, g, beta, S0, o, ST, cu, N, T, total, Hk, Hv, dk, dv, qs, ks, vs, dt, ws, wb, None)


def test_forward_rejects(lib):
    for bad in (dict(dk=0), dict(dv=129), dict(N=-1), dict(T=-1), dict(Hk=0), dict(Hk=2, Hv=3, qs=32, ks=32, vs=48), dict(dt=7),
                dict(total=5), dict(q=None), dict(o=None), dict(g=None), dict(qs=15), dict(vs=8)):
        assert fwd(lib, **bad) == 1, bad
    for bad in (dict(q=ODD16), dict(S0=ODD16), dict(ST=ODD16), dict(g=ODD4), dict(beta=ODD4), dict(cu=ODD4), dict(ws=ODD16)):
        assert fwd(lib, **bad) == 3, bad
    assert fwd(lib, qs=20) == 3 and fwd(lib, vs=17) == 3                  # bf16 rows off 16 bytes
    assert fwd(lib, ws=None, wb=0) == 6
    assert fwd(lib, N=1 << 20, T=1 << 12, total=0x7fffffff) in (1, 2)
    assert fwd(lib, N=0, total=0) == 0                                    # nothing to do


def test_backward_rejects(lib):
    def bwd(grad_o=P, gq=P, gg=P, wb=1 << 40, dt=BF, dk=16, qs=16):
        return lib.ckda_gated_bwd(P, P, P, P, P, None, grad_o, None, gq, P, P, gg, P, None, None, 1, 4, 4, 1, 1, dk, 16, qs, 16, 16,
                                  dt, P, wb, None)
    assert bwd(grad_o=None) == 1 and bwd(gq=None) == 1 and bwd(dk=200) == 1 and bwd(dt=3) == 1 and bwd(qs=4) == 1
    assert bwd(gq=ODD16) == 3 and bwd(gg=ODD4) == 3
    assert bwd(wb=16) == 6 and bwd(wb=16, dt=F32) == 6


def test_decode_rejects(lib):
    def dec(q=P, S=P, slots=None, N=2, pool=2, Hk=1, Hv=1, dk=16, dv=16, qs=16, dt=BF):
        return lib.ckda_gated_decode_step(q, P, P, P, P, S, P, slots, N, pool, Hk, Hv, dk, dv, qs, 16, 16, dt, None)
    assert dec(pool=1) == 1 and dec(pool=0, slots=P) == 1 and dec(S=None) == 1 and dec(q=None) == 1
    assert dec(dk=0) == 1 and dec(Hk=2) == 1 and dec(qs=3) == 1 and dec(dt=9) == 1
    assert dec(S=ODD16) == 3 and dec(slots=ODD4) == 3
    assert dec(N=0) == 0


def test_prep_rejects(lib):
    def prep(q=P, out=P, w=None, pos=None, p64=0, f=P, tokens=4, period=4, Hq=1, Hk=0, d=16, rot=8, qs=16, dt=BF, norm=1, inter=0):
        return lib.ckda_qk_prep(q, None, out, None, w, None, pos, p64, f, tokens, period, Hq, Hk, d, rot, qs, 0, dt, norm, inter,
                                1e-6, 1.0, 1.0, None)
    for bad in (dict(d=0), dict(d=257, qs=257), dict(rot=3), dict(rot=18), dict(Hq=0), dict(tokens=-1), dict(dt=4), dict(norm=3),
                dict(inter=2), dict(p64=2), dict(qs=8), dict(f=None), dict(period=0), dict(q=None), dict(out=None), dict(Hk=1)):
        assert prep(**bad) == 1, bad
    assert prep(q=ODD16) == 3 and prep(out=ODD16) == 3 and prep(w=ODD16) == 3
    assert prep(pos=ctypes.c_void_p(0x10004), p64=1) == 3 and prep(f=ctypes.c_void_p(0x10004)) == 3
    assert prep(Hq=5000, qs=80000) == 2
    assert prep(tokens=0, q=None, out=None) == 0
    assert lib.ckda_qk_prep_bwd_workspace_bytes(0) == 0 and lib.ckda_qk_prep_bwd_workspace_bytes(257) == 0
    assert lib.ckda_qk_prep_bwd_workspace_bytes(128) % 256 == 0


def test_copy_rejects(lib):
    def copy(S=P, src=P, dst=P, pairs=1, layers=1, slots=2, row=64):
        return lib.ckda_state_copy(S, src, dst, pairs, layers, slots, row, None)
    assert copy(S=None) == 1 and copy(src=None) == 1 and copy(slots=0) == 1 and copy(pairs=-1) == 1 and copy(row=-4) == 1
    assert copy(S=ODD16) == 3 and copy(src=ODD4) == 3
    assert copy(pairs=1025) == 2 and copy(row=63) == 2 and copy(layers=70000) == 2
    assert copy(pairs=0, src=None) == 0 and copy(layers=0) == 0


def test_workspace_and_segments(lib):
    """bf16 with heads of a multiple of 8 channels takes workspace; a batch that fills the GPU runs
    whole, one long sequence on few heads in segments whose maps take more (148 SMs without a GPU)."""
    b = lib.ckda_gated_fwd_workspace_bytes
    assert b(1, 100, 1, 1, 128, 128, F32) == 0 and b(1, 100, 1, 1, 17, 128, BF) == 0
    assert b(0, 0, 1, 1, 128, 128, BF) == 0 and b(1, 100, 1, 1, 0, 128, BF) == 0
    assert b(8, 32768, 16, 16, 128, 128, BF) > 512 * 16 * 4 * 8192        # Z and P, two terms each, per chunk
    seg = lib.ckda_gated_fwd_segment_tokens
    assert seg(8, 32768, 16, 16, 128, 128, BF) == 0 and seg(1, 512, 16, 16, 128, 128, BF) == 0
    n = seg(1, 65536, 16, 16, 128, 128, BF)
    assert n % 64 == 0 and 1024 <= n < 65536
    assert seg(1, 65536, 16, 16, 128, 128, F32) == 0
    back = lib.ckda_gated_bwd_workspace_bytes
    assert back(8, 32768, 16, 16, 128, 128, BF) > b(8, 32768, 16, 16, 128, 128, BF)
    assert back(1, 10, 1, 1, 8, 8, F32) > 0 and back(1, 0, 1, 1, 8, 8, F32) == 0


def test_backward_plan(lib):
    """The backward pass has a plan of its own: its workspace holds what that plan takes."""
    fwd_plan, plan, need = lib.ckda_gated_fwd_segment_tokens, lib.ckda_gated_bwd_segment_tokens, lib.ckda_gated_bwd_workspace_bytes
    n = plan(1, 65536, 16, 16, 128, 128, BF)
    assert n % 64 == 0 and 1024 <= n < 65536 and n != fwd_plan(1, 65536, 16, 16, 128, 128, BF)
    assert plan(8, 32768, 16, 16, 128, 128, BF) == 0 and plan(1, 65536, 16, 16, 128, 128, F32) == 0 and plan(0, 0, 1, 1, 64, 64, BF) == 0
    assert plan(1, 2777, 2, 4, 64, 128, BF) > 0 and plan(1, 2777, 2, 4, 0, 128, BF) == 0
    whole = 65536 // 64 * 16 * (4 * 8192 + 3 * 128 * 128 * 2 + 64 * 128 * 6)        # what every chunk keeps, vectors and sums apart
    places = 65536 // n * 16 * 3 * 128 * 128 * 4                                     # states, maps and cotangents of segments
    assert need(1, 65536, 16, 16, 128, 128, BF) >= whole + places


def test_device_error_name(lib):
    assert lib.ckda_status_string(7) not in (b"unknown status", b"ok")


def test_build_checks_register_splits():
    """A chain compiled to another number of registers than its split adds up to fails the build, not the calls."""
    from delta_rule_attention_ckda_b200 import build
    said = ("ptxas info    : Compiling entry function '_ZN4ckda5gated16chain_bwd_kernelILi64EEEvv' for 'sm_100a'\n"
            "ptxas info    : Function properties for _ZN4ckda5gated16chain_bwd_kernelILi64EEEvv\n"
            "    104 bytes stack frame, 104 bytes spill stores, 108 bytes spill loads\n"
            "ptxas info    : Used {} registers, used 2 barriers, 104 bytes cumulative stack size\n"
            "ptxas info    : Compiling entry function '_ZN4ckda5gated12intra_kernelILi64EEEvv' for 'sm_100a'\n"
            "ptxas info    : Used 90 registers, used 1 barriers\n")
    build._check_registers(said.format(128))
    for n in (80, 127, 168):
        with pytest.raises(RuntimeError, match="chain_bwd_kernel.*registers"):
            build._check_registers(said.format(n))


class _Fake(torch.Tensor):
    """A host tensor that reports a CUDA device: the checks in front of a call run without a GPU."""
    @property
    def device(self):
        return getattr(self, "_dev", torch.device("cuda", 0))


def fake(*shape, dtype=torch.bfloat16, dev="cuda:0"):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(_Fake)
    t._dev = torch.device(dev)
    return t


def test_binding_checks():
    import delta_rule_attention_ckda_b200 as ck
    f32 = dict(dtype=torch.float32)
    q, k, v, g, b = fake(1, 4, 1, 16), fake(1, 4, 1, 16), fake(1, 4, 2, 16), fake(1, 4, 2, **f32), fake(1, 4, 2, **f32)
    cpu = torch.zeros(1, 4, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ck.gated_chunk_fwd(cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError, match="cuda:1"):
        ck.gated_chunk_fwd(q, fake(1, 4, 1, 16, dev="cuda:1"), v, g, b)
    with pytest.raises(TypeError):
        ck.gated_chunk_fwd(q, k, v, fake(1, 4, 2), b)
    with pytest.raises(ValueError, match="multiple"):
        ck.gated_chunk_fwd(fake(1, 4, 2, 16), fake(1, 4, 2, 16), fake(1, 4, 3, 16), fake(1, 4, 3, **f32), fake(1, 4, 3, **f32))
    with pytest.raises(ValueError, match="contiguous heads"):
        ck.gated_chunk_fwd(fake(1, 4, 1, 32)[..., ::2], k, v, g, b)
    with pytest.raises(ValueError, match="distance"):
        ck.gated_chunk_fwd(fake(4, 2, 1, 16).transpose(0, 1), fake(2, 4, 1, 16), fake(2, 4, 1, 16), fake(2, 4, 1, **f32), fake(2, 4, 1, **f32))
    with pytest.raises(ValueError, match="overlaps q"):
        ck.gated_chunk_fwd(q, k, q, fake(1, 4, 1, **f32), fake(1, 4, 1, **f32), o=q)
    with pytest.raises(TypeError):
        ck.gated_chunk_fwd(q[0], k[0], v[0], g[0], b[0], cu_seqlens=fake(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        ck.gated_chunk_fwd(q[0], k[0], v[0], g[0], b[0], cu_seqlens=[0, 4])
    grads = {"dq": fake(1, 4, 1, 16), "dv": fake(1, 4, 2, 16), "dg": fake(1, 4, 2, **f32), "dbeta": fake(1, 4, 2, **f32),
             "dS0": fake(1, 2, 16, 16, **f32)}
    grads["dk"] = grads["dq"]
    with pytest.raises(ValueError, match="no 'dS_0'"):
        ck.gated_bwd(q, k, v, g, b, fake(1, 4, 2, 16), grads={"dS_0": grads["dS0"]})
    with pytest.raises(ValueError, match="dk overlaps dq"):
        ck.gated_bwd(q, k, v, g, b, fake(1, 4, 2, 16), grads=grads)
    S = fake(3, 2, 16, 16, **f32)
    with pytest.raises(ValueError, match="rows"):
        ck.gated_decode_step(fake(4, 1, 16), fake(4, 1, 16), fake(4, 2, 16), fake(4, 2, **f32), fake(4, 2, **f32), S)
    with pytest.raises(TypeError):
        ck.gated_decode_step(q[0], k[0], v[0], g[0], b[0], S, slots=fake(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="norm"):
        ck.qk_norm_rope(q, k, norm="max")
    with pytest.raises(ValueError, match="layout"):
        ck.qk_norm_rope(q, k, layout="pairs")
    with pytest.raises(ValueError, match="without inv_freq"):
        ck.qk_norm_rope(q, k, positions=fake(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="turns"):
        ck.qk_norm_rope(q, k, inv_freq=fake(9, dtype=torch.float64))
    with pytest.raises(TypeError):
        ck.qk_norm_rope(q, k, inv_freq=fake(4, **f32))
    with pytest.raises(ValueError, match="come together"):
        ck.qk_norm_rope_bwd(q, k, fake(1, 4, 1, 16))
    with pytest.raises(ValueError, match="expected"):
        ck.state_copy(S, fake(2, dtype=torch.int32), fake(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="pool"):
        ck.state_copy(S, fake(2, dtype=torch.int32), fake(2, dtype=torch.int32), pool_dim=2)


def test_binding_counts():
    """Counts beyond 32 bits are refused: cut to their lower half, 2**32 tokens would be none. (Tensors without memory.)"""
    import delta_rule_attention_ckda_b200 as ck

    def big(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(_Fake)

    n, bf, i32 = 1 << 32, torch.bfloat16, torch.int32
    for lead in ((1, n), (n, 1), (1 << 20, 1 << 12), (1, 1 << 31)):
        x, g = big(*lead, 1, 1, dtype=bf), big(*lead, 1)
        with pytest.raises(ValueError, match="2[*][*]31"):
            ck.gated_chunk_fwd(x, x, x, g, g)
        with pytest.raises(ValueError, match="2[*][*]31"):
            ck.gated_bwd(x, x, x, g, g, x)
    x, g = big(n + 4, 1, 1, dtype=bf), big(n + 4, 1)
    with pytest.raises(ValueError, match="2[*][*]31"):
        ck.gated_chunk_fwd(x, x, x, g, g, cu_seqlens=big(2, dtype=i32))
    with pytest.raises(ValueError, match="2[*][*]31"):
        ck.gated_decode_step(x, x, x, g, g, big(n + 4, 1, 1, 1))
    x, g = big(4, 1, 1, dtype=bf), big(4, 1)
    with pytest.raises(ValueError, match="2[*][*]31"):
        ck.gated_decode_step(x, x, x, g, g, big(n + 5, 1, 1, 1), slots=big(4, dtype=i32))
    for shape in ((1, n + 8, 4), (n + 8, 1, 4)):
        with pytest.raises(ValueError, match="2[*][*]31"):
            ck.state_copy(big(*shape), big(1, dtype=i32), big(1, dtype=i32), pool_dim=1)


def test_rows_of_wider_tensors():
    """The distance between tokens of slices, over one and two leading dimensions."""
    from delta_rule_attention_ckda_b200.gated import _rows
    dev = torch.device("cuda", 0)
    wide = fake(2, 5, 12 * 8)
    assert _rows(wide[..., :32].unflatten(-1, (4, 8)), "q", 2, None, dev) == 96
    assert _rows(wide.flatten(0, 1)[:, 32:64].unflatten(-1, (4, 8)), "q", 1, None, dev) == 96
    assert _rows(fake(2, 5, 4, 8), "q", 2, None, dev) == 32
    assert _rows(fake(1, 5, 96)[..., :32].unflatten(-1, (4, 8)), "q", 2, None, dev) == 96
    assert _rows(fake(5, 1, 96)[..., :32].unflatten(-1, (4, 8)), "q", 2, None, dev) == 96
    with pytest.raises(ValueError):
        _rows(fake(1, 4, 8).expand(5, 4, 8), "q", 1, None, dev)


def test_frequencies():
    import delta_rule_attention_ckda_b200 as ck
    f, s = ck.rope_frequencies(64)
    assert f.dtype == torch.float64 and s == 1.0 and f[0] == 1.0 and math.isclose(float(f[1]), 10000 ** (-2 / 64))
    lin, _ = ck.rope_frequencies(64, factor=4.0, scaling="linear")
    assert torch.allclose(lin * 4, f, rtol=1e-15)
    base, _ = ck.rope_frequencies(64, factor=4.0, scaling="base")
    assert base[0] == 1.0 and math.isclose(float(base[-1]) * 4, float(f[-1]), rel_tol=1e-12)
    part, s = ck.rope_frequencies(64, factor=4.0, scaling="by_parts", trained=4096)
    turns = 4096 * f / (2 * math.pi)
    assert math.isclose(s, 0.1 * math.log(4.0) + 1.0)
    assert torch.equal(part[turns > 40], f[turns > 40]) and torch.allclose(part[turns < 0.7] * 4, f[turns < 0.7], rtol=1e-15)
    assert (part[1:] < part[:-1]).all()
    for bad in (dict(rotary=3), dict(rotary=0), dict(rotary=64, factor=0.5), dict(rotary=64, scaling="log"),
                dict(rotary=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            ck.rope_frequencies(bad.pop("rotary"), **bad)


@pytest.mark.parametrize("rotary,base,trained", [(64, 10000.0, 131072), (128, 10000.0, 32768), (64, 10000.0, 4096), (16, 500.0, 8192),
                                                 (128, 500000.0, 8192), (64, 10000.0, 6), (2, 10000.0, 4096)])
def test_frequencies_by_parts(rotary, base, trained):
    """What the three parts promise, also where no pair turns as little as `slow` times, or every pair does."""
    import delta_rule_attention_ckda_b200 as ck
    f, _ = ck.rope_frequencies(rotary, base)
    part, _ = ck.rope_frequencies(rotary, base, factor=8.0, scaling="by_parts", trained=trained)
    index = lambda turns: rotary * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    share = (1 - part / f) / (1 - 1 / 8)                                  # 0: left alone, 1: divided by factor
    for p in range(rotary // 2):
        if p <= math.floor(index(32.0)):
            assert abs(share[p]) < 1e-12, p
        elif p >= index(1.0):
            assert p < math.ceil(index(1.0)) or abs(share[p] - 1) < 1e-12, p
        else:                                                             # between: strictly, in steps of one size
            lo, hi = max(math.floor(index(32.0)), 0), math.ceil(index(1.0))
            assert abs(share[p] - (p - lo) / (hi - lo)) < 1e-12, p


def test_oracle_rule_is_the_per_channel_rule():
    """The scalar-gate definition against the library's per-channel oracle with the gate repeated."""
    import numpy as np
    import oracle
    q, k, v, g, b, S0, _, _ = make((2, 30), 2, 2, 8, 6, torch.float32, 1, 2)
    o, ST = ref.gated_fwd(q, k, v, g, b, S0)
    alpha = torch.exp(g.double())[..., None].expand(2, 30, 2, 8)
    o2, S2 = oracle.oracle_fwd(q, k, v, alpha, b, S0)
    assert np.abs(o.numpy() - o2).max() < 1e-12 and np.abs(ST.numpy() - S2).max() < 1e-12


def test_oracle_gradients_by_differences():
    q, k, v, g, b, S0, do, dST = make((7,), 1, 2, 5, 4, torch.float32, 2, 2)
    cu = [0, 4, 7]
    x = {n: t.double() for n, t in zip("qkvgbS", (q, k, v, g, b, S0))}

    def loss(**new):
        y = {**x, **new}
        o, ST = ref.gated_fwd(y["q"], y["k"], y["v"], y["g"], y["b"], y["S"], cu)
        return float((o * do.double()).sum() + (ST * dST.double()).sum())

    got = ref.gated_bwd(q, k, v, g, b, do, S0, dST, cu)
    gen = torch.Generator().manual_seed(0)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("b", "dbeta"), ("S", "dS0")):
        way = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        slope = (loss(**{n: x[n] + h * way}) - loss(**{n: x[n] - h * way})) / (2 * h)
        assert abs(slope - float((got[d] * way).sum())) < 1e-7 * max(1.0, abs(slope)), n


def test_oracle_rotation_and_copies():
    """A rotation keeps the length of each pair and turns it by the angle; copies read a snapshot."""
    x = torch.randn(3, 2, 8, dtype=torch.float64)
    f = torch.tensor([0.5, 0.1], dtype=torch.float64)
    for layout in ("half", "interleaved"):
        y = ref.prep(x, torch.tensor([0, 1, 7]), f, norm="none", layout=layout)
        assert torch.allclose(y[0], x[0]) and torch.equal(y[..., 4:], x[..., 4:])
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
    a, b = (0, 2), (0, 1)
    for layout, (i, j) in (("half", a), ("interleaved", b)):
        y = ref.prep(x, torch.tensor([0, 1, 7]), f, norm="none", layout=layout)
        c, s = math.cos(3.5), math.sin(3.5)
        assert torch.allclose(y[2, :, i], x[2, :, i] * c - x[2, :, j] * s)
    S = torch.arange(4.0).view(1, 4, 1)
    got = ref.copy(S, torch.tensor([0, 1, -1, 9]), torch.tensor([1, 0, 3, 2]))
    assert got.flatten().tolist() == [1.0, 0.0, 2.0, 0.0]
