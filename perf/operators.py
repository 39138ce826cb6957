"""The cases by which the library's scalar-gate operators are measured, with their plain forms.

Four operators that a linear-attention layer runs next to one another:

* ``prep``: norms of queries and keys for each head with the position rotation in the same pass
  (``qk_norm_rope`` and ``qk_norm_rope_bwd``);
* ``prefill`` and ``train``: the gated delta rule with one decay per head, in chunks
  (``gated_chunk_fwd`` and ``gated_bwd``);
* ``decode``: its single-token step on a pool of states (``gated_decode_step``);
* ``copy``: forking, moving and clearing states of that pool (``state_copy``).

``own`` false: elementary torch operations. ``own`` true: the calls a user makes.
"""
import math

import torch

own = False

DEV = "cuda"
C = 64                         # tokens in a chunk of the plain form
BF = torch.bfloat16


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # The layer step of a 1.3B-parameter model: 8 sequences of 4096 tokens, 16 heads of 128.
        dict(name="prefill layer", op="prefill", seqs=8, tokens=32768, ragged=False, hk=16, hv=16, dk=128, dv=128, s0=False),
        # Requests of different lengths packed into one batch, value heads sharing key heads, states
        # that earlier chunks of the same requests left.
        dict(name="prefill packed", op="prefill", seqs=13, tokens=9001, ragged=True, hk=8, hv=16, dk=128, dv=128, s0=True),
        # One long document: few sequences, many tokens.
        dict(name="prefill long", op="prefill", seqs=1, tokens=65536, ragged=False, hk=16, hv=16, dk=128, dv=128, s0=True),
        # The same layer's backward pass.
        dict(name="train layer", op="train", seqs=8, tokens=32768, ragged=False, hk=16, hv=16, dk=128, dv=128, s0=False),
        # Documents packed for training of a small model, with shared key heads.
        dict(name="train packed", op="train", seqs=5, tokens=2777, ragged=True, hk=2, hv=4, dk=64, dv=128, s0=True),
        # A full serving batch: 256 sequences, 268 MB of state.
        dict(name="decode 256", op="decode", seqs=256, slots=256, hk=16, hv=16, dk=128, dv=128),
        # A few users: the latency of one token.
        dict(name="decode 3", op="decode", seqs=3, slots=32, hk=8, hv=16, dk=128, dv=128),
        # The step before the layer: queries and keys read in place out of a fused projection, L2
        # norms, half of each head rotated.
        dict(name="prep layer", op="prep", tokens=32768, hq=16, hk=16, dim=128, rotary=64, norm="l2", layout="half", fused=True, back=False),
        # The same step for a handful of tokens far into their contexts, RMS norms with weights.
        dict(name="prep decode", op="prep", tokens=7, hq=16, hk=4, dim=128, rotary=128, norm="rms", layout="interleaved", fused=False, back=False),
        # Its backward pass.
        dict(name="prep train", op="prep", tokens=16383, hq=16, hk=8, dim=128, rotary=128, norm="rms", layout="half", fused=False, back=True),
        # A beam search step: states forked, some slots cleared for new requests.
        dict(name="copy fork", op="copy", layers=1, slots=288, pairs=96, heads=16, dk=128, dv=128),
        # One finished request's slot refilled from the end of a small pool, in every layer.
        dict(name="copy compact", op="copy", layers=12, slots=16, pairs=2, heads=4, dk=64, dv=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "decode", "prep", "prep", "copy"])
    if op in ("prefill", "train"):
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        hv = hk * rng.choice([1, 1, 2, 4]) if hk <= 4 else 16
        tokens = _log(rng, 1, 32768 if op == "prefill" else 16384)
        seqs = max(1, min(tokens, _log(rng, 1, 64)))
        ragged = rng.random() < 0.6
        if not ragged:
            tokens = max(1, tokens // seqs) * seqs
        return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, hk=hk, hv=hv, dk=rng.choice([64, 128]),
                    dv=rng.choice([64, 128]), s0=rng.random() < 0.5)
    if op == "decode":
        hk = rng.choice([1, 2, 4, 8, 16])
        seqs = _log(rng, 1, 256)
        return dict(op=op, seqs=seqs, slots=seqs + rng.randrange(0, 9), hk=hk, hv=hk * rng.choice([1, 2]) if hk < 16 else 16,
                    dk=rng.choice([64, 128]), dv=rng.choice([64, 128]))
    if op == "prep":
        dim = rng.choice([64, 96, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 16384), hq=rng.choice([1, 2, 4, 8, 16]), hk=rng.choice([1, 2, 4, 8]), dim=dim,
                    rotary=rng.choice([0, dim // 4, dim // 2, dim]), norm=rng.choice(["none", "l2", "rms"]),
                    layout=rng.choice(["half", "interleaved"]), fused=rng.random() < 0.5, back=rng.random() < 0.5)
    slots = _log(rng, 2, 256)
    layers = rng.choice([1, 2, 6])
    return dict(op="copy", layers=layers, slots=max(2, slots // layers), pairs=max(1, min(slots // layers, _log(rng, 1, 96))),
                heads=rng.choice([1, 4, 16]), dk=rng.choice([64, 128]), dv=rng.choice([64, 128]))


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lengths(case, seed):
    """The sequences' lengths: equal, or cut at random places (a few of one token, some long)."""
    n, total = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [total // n] * n
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=g, dtype=torch.float64).mul(2.5).exp()
    cuts = torch.floor(torch.cumsum(w / w.sum(), 0) * (total - n)).long().tolist()
    cuts[-1] = total - n
    return [b - a + 1 for a, b in zip([0] + cuts[:-1], cuts)]


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def _gates(shape, g):
    decay = -torch.exp(torch.randn(shape, device=DEV, generator=g) * 1.2 - 3.0)      # a few tokens to hundreds
    beta = 2 * torch.sigmoid(torch.randn(shape, device=DEV, generator=g))
    return decay, beta


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)

    def rand(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    if case["op"] in ("prefill", "train"):
        n, total, hk, hv, dk, dv = (case[x] for x in ("seqs", "tokens", "hk", "hv", "dk", "dv"))
        lens = _lengths(case, seed)
        lead = (total,) if case["ragged"] else (n, total // n)
        st["max_len"] = max(lens)
        st["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        st["q"] = (_unit(rand(*lead, hk, dk)) * dk ** -0.5).to(BF)
        st["k"] = _unit(rand(*lead, hk, dk)).to(BF)
        st["v"] = rand(*lead, hv, dv).to(BF)
        st["g"], st["beta"] = _gates((*lead, hv), g)
        st["S0"] = rand(n, hv, dk, dv) * 0.1 if case["s0"] else None
        if case["op"] == "train":
            st["grad_o"] = rand(*lead, hv, dv).to(BF)
            st["grad_S_T"] = rand(n, hv, dk, dv) * 0.1 if case["s0"] else None
    elif case["op"] == "decode":
        n, p, hk, hv, dk, dv = (case[x] for x in ("seqs", "slots", "hk", "hv", "dk", "dv"))
        st["q"] = (_unit(rand(n, hk, dk)) * dk ** -0.5).to(BF)
        st["k"] = _unit(rand(n, hk, dk)).to(BF)
        st["v"] = rand(n, hv, dv).to(BF)
        st["g"], st["beta"] = _gates((n, hv), g)
        st["S"] = rand(p, hv, dk, dv) * 0.3
        st["slots"] = torch.randperm(p, device=DEV, generator=g)[:n].to(torch.int32)
    elif case["op"] == "prep":
        t, hq, hk, d, r = (case[x] for x in ("tokens", "hq", "hk", "dim", "rotary"))
        if case["fused"]:          # slices of one projection's output, the values between them skipped
            both = rand(t, (hq + 2 * hk) * d).mul(2).to(BF)
            st["q"] = both[:, :hq * d].unflatten(-1, (hq, d))
            st["k"] = both[:, hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
        else:
            st["q"], st["k"] = rand(t, hq, d).mul(2).to(BF), rand(t, hk, d).mul(2).to(BF)
        st["positions"] = torch.randint(0, 1 << 20, (t,), device=DEV, generator=g, dtype=torch.int32)
        st["inv_freq"] = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / max(r, 1)) if r else None
        st["wq"] = st["wk"] = None
        if case["norm"] == "rms":
            st["wq"], st["wk"] = 1 + 0.1 * rand(d), 1 + 0.1 * rand(d)
        if case["back"]:
            st["dq"], st["dk"] = rand(t, hq, d).to(BF), rand(t, hk, d).to(BF)
    else:
        p, m = case["slots"], case["pairs"]
        st["S"] = rand(case["layers"], p, case["heads"], case["dk"], case["dv"])
        st["dst"] = torch.randperm(p, device=DEV, generator=g)[:m].to(torch.int32)
        src = torch.randint(0, p, (m,), device=DEV, generator=g, dtype=torch.int32)
        st["src"] = torch.where(torch.rand(m, device=DEV, generator=g) < 0.1, torch.full_like(src, -1), src)
    return st


# ------------------------------------------------------------------------------- plain forms

def _grid(st):
    """Where each token of the packed tensors lies in a [sequence, padded length] grid: the token of every
    place (the one past the end for padding), and the place of every token."""
    cu = st["cu"].long()
    total = st["tokens"]
    padded = max(1, -(-st["max_len"] // C)) * C
    at = cu[:-1, None] + torch.arange(padded, device=DEV)
    at = torch.where(at < cu[1:, None], at, total)
    tok = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    return at, seq * padded + tok - cu[seq]


def _chunks(x, at, heads):
    """[..., h, d] packed -> [sequence, heads, chunk, C, d] in 32 bits, zeros in the padding, shared heads repeated."""
    d = x.shape[-1]
    x = x.reshape(-1, x.shape[-2], d).float()
    x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[at]
    return x.repeat_interleave(heads // x.shape[2], 2).transpose(1, 2).unflatten(2, (-1, C))


def _packed(x, place, like):
    """The reverse of _chunks, rounded to the type of `like`."""
    x = x.flatten(2, 3).transpose(1, 2)
    return x.reshape(-1, *x.shape[2:])[place].reshape(*like.shape[:-2], x.shape[2], x.shape[3]).to(like.dtype)


def _plain_forward(st, at):
    hv = st["hv"]
    q, k, v = (_chunks(st[n], at, hv) for n in ("q", "k", "v"))
    g = _chunks(st["g"][..., None], at, hv)[..., 0].double().cumsum(-1)
    beta = _chunks(st["beta"][..., None], at, hv)
    low = torch.ones(C, C, device=DEV, dtype=torch.bool).tril()
    decay = torch.where(low, (g[..., :, None] - g[..., None, :]).clamp_max(60.0).exp().float(), 0)
    p = q @ k.mT * decay
    a = (k @ k.mT * decay).tril(-1) * beta.mT
    inv = torch.eye(C, device=DEV).expand_as(a).contiguous()                  # (1 + a)^-1 row by row
    for i in range(1, C):
        inv[..., i, :i] = -(a[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    into, out, whole = g.exp().float()[..., None], (g[..., -1:] - g).exp().float()[..., None], g[..., -1].exp().float()[..., None, None]
    S = st["S0"]
    S = q.new_zeros(q.shape[0], hv, st["dk"], st["dv"]) if S is None else S
    o, w, states = torch.empty_like(v), torch.empty_like(v), []
    for c in range(q.shape[2]):
        states.append(S)
        w[:, :, c] = inv[:, :, c] @ (v[:, :, c] - into[:, :, c] * (k[:, :, c] @ S))
        u = beta[:, :, c] * w[:, :, c]
        o[:, :, c] = into[:, :, c] * (q[:, :, c] @ S) + p[:, :, c] @ u
        S = whole[:, :, c] * S + (out[:, :, c] * k[:, :, c]).mT @ u
    return dict(q=q, k=k, v=v, beta=beta, decay=decay, p=p, a=a, inv=inv, into=into, out=out, whole=whole, o=o, w=w, states=states, S=S)


def _plain_prefill(st):
    at, place = _grid(st)
    f = _plain_forward(st, at)
    return _packed(f["o"], place, st["v"]), f["S"]


def _plain_train(st):
    at, place = _grid(st)
    f = _plain_forward(st, at)
    q, k, v, beta, decay, p, inv, into, out, whole, w = (f[n] for n in ("q", "k", "v", "beta", "decay", "p", "inv", "into", "out", "whole", "w"))
    do = _chunks(st["grad_o"], at, st["hv"])
    dS = st["grad_S_T"]
    dS = torch.zeros_like(f["S"]) if dS is None else dS
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dbeta, dgate, end = torch.empty_like(beta), torch.empty_like(beta), f["S"]
    for c in reversed(range(q.shape[2])):
        S, qc, kc, vc, dc, wc, bc = f["states"][c], q[:, :, c], k[:, :, c], v[:, :, c], do[:, :, c], w[:, :, c], beta[:, :, c]
        ic, oc, D = into[:, :, c], out[:, :, c], decay[:, :, c]
        u = bc * wc
        du = p[:, :, c].mT @ dc + oc * (kc @ dS)
        dx = inv[:, :, c].mT @ (bc * du)
        dw = D * (dc @ u.mT)
        da = -D.tril(-1) * (dx @ u.mT)
        dq[:, :, c] = ic * (dc @ S.mT) + dw @ kc
        dk[:, :, c] = -ic * (dx @ S.mT) + oc * (u @ dS.mT) + dw.mT @ qc + da @ kc + da.mT @ kc
        dv[:, :, c] = dx
        into_w = du - (D.tril(-1) * (kc @ kc.mT)).mT @ dx                     # the cotangent of beta * w
        dbeta[:, :, c] = (wc * into_w).sum(-1, keepdim=True)
        own_part = (dc * f["o"][:, :, c] - dx * vc).double().sum(-1, keepdim=True)
        after = (end.double() * dS).sum((-1, -2))[..., None, None]
        dgate[:, :, c] = (own_part.flip(-2).cumsum(-2).flip(-2) + after).float()
        end = S
        dS = whole[:, :, c] * dS + (ic * qc).mT @ dc - (ic * kc).mT @ dx
    shared = (st["hk"], st["hv"] // st["hk"])
    dq, dk = dq.unflatten(1, shared).sum(2), dk.unflatten(1, shared).sum(2)
    return {"dq": _packed(dq, place, st["q"]), "dk": _packed(dk, place, st["k"]), "dv": _packed(dv, place, st["v"]),
            "dg": _packed(dgate, place, st["g"][..., None])[..., 0], "dbeta": _packed(dbeta, place, st["beta"][..., None])[..., 0], "dS0": dS}


def _plain_decode(st):
    rep = st["hv"] // st["hk"]
    slots = st["slots"].long()
    q, k = (st[n].float().repeat_interleave(rep, 1)[..., None] for n in ("q", "k"))
    S = st["S"][slots] * st["g"].exp()[..., None, None]
    u = st["beta"][..., None, None] * (st["v"].float()[..., None, :] - (S * k).sum(-2, keepdim=True))
    S = S + k * u
    st["S"][slots] = S
    return (S * q).sum(-2).to(BF), st["S"]


def _angles(st):
    x = st["positions"].double()[:, None] * st["inv_freq"]
    return x.cos().float()[:, None], x.sin().float()[:, None]


def _pairs(x, r, layout):
    x = x[..., :r]
    return (x[..., :r // 2], x[..., r // 2:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])


def _turned(x, st, sign):
    r = st["rotary"]
    if not r:
        return x
    cos, sin = _angles(st)
    a, b = _pairs(x, r, st["layout"])
    a, b = a * cos - sign * b * sin, b * cos + sign * a * sin
    rot = torch.cat([a, b], -1) if st["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([rot, x[..., r:]], -1)


def _inverse_norm(x, norm):
    if norm == "none":
        return torch.ones_like(x[..., :1])
    if norm == "l2":
        return 1 / (x * x).sum(-1, keepdim=True).sqrt().clamp_min(1e-12)
    return 1 / ((x * x).mean(-1, keepdim=True) + 1e-6).sqrt()


def _plain_prep(st):
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        y = x.float()
        y = y * _inverse_norm(y, st["norm"])
        out.append(_turned(y if w is None else y * w, st, 1).to(BF))
    return tuple(out)


def _plain_prep_back(st):
    out = {}
    for n, x, w, dy in (("q", st["q"], st["wq"], st["dq"]), ("k", st["k"], st["wk"], st["dk"])):
        x = x.float()
        r = _inverse_norm(x, st["norm"])
        dz = _turned(dy.float(), st, -1)
        if w is not None:
            out["dw" + n] = (dz * x * r).sum((0, 1))
            dz = dz * w
        if st["norm"] != "none":
            y = x * r
            dz = dz - y * ((dz * y).sum(-1, keepdim=True) / (x.shape[-1] if st["norm"] == "rms" else 1))
        out["d" + n] = (dz * r).to(BF)
    return out


def _plain_copy(st):
    S, src, dst = st["S"], st["src"].long(), st["dst"].long()
    S[:, dst] = torch.where((src >= 0)[:, None, None, None], S[:, src.clamp_min(0)], 0)
    return S


def run(st):
    op = st["op"]
    if own:
        import delta_rule_attention_ckda_b200 as ck
        if op in ("prefill", "train"):
            cu = st["cu"] if st["ragged"] else None
            args = (st["q"], st["k"], st["v"], st["g"], st["beta"])
            if op == "prefill":
                return ck.gated_chunk_fwd(*args, st["S0"], cu_seqlens=cu)
            return ck.gated_bwd(*args, st["grad_o"], st["S0"], st["grad_S_T"], cu_seqlens=cu)
        if op == "decode":
            return ck.gated_decode_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], slots=st["slots"]), st["S"]
        if op == "prep":
            how = dict(positions=st["positions"] if st["rotary"] else None, inv_freq=st["inv_freq"], norm=st["norm"],
                       layout=st["layout"], q_weight=st["wq"], k_weight=st["wk"])
            if not st["back"]:
                return ck.qk_norm_rope(st["q"], st["k"], **how)
            got = ck.qk_norm_rope_bwd(st["q"], st["k"], st["dq"], st["dk"], **how)
            names = {"dq": "dq", "dk": "dk", "dq_weight": "dwq", "dk_weight": "dwk"}
            return {names[n]: x for n, x in got.items() if x is not None}
        return ck.state_copy(st["S"], st["src"], st["dst"], pool_dim=1)
    if op == "prefill":
        return _plain_prefill(st)
    if op == "train":
        return _plain_train(st)
    if op == "decode":
        return _plain_decode(st)
    if op == "prep":
        return _plain_prep_back(st) if st["back"] else _plain_prep(st)
    return _plain_copy(st)


# ------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("prefill", "train"):
        t, n, hk, hv, dk, dv = (case[x] for x in ("tokens", "seqs", "hk", "hv", "dk", "dv"))
        state = n * hv * dk * dv * 4
        tensors = t * (2 * hk * dk * 2 + hv * dv * 2)                         # q, k, v
        # per token and head: the state read by k and q and updated, and half of a 64-token chunk's pairs
        flops = 2 * t * hv * (3 * dk * dv + (C // 2) * (2 * dk + 2 * dv))
        if op == "prefill":
            return {"bytes": tensors + t * hv * (8 + dv * 2) + state * (2 if case["s0"] else 1), "flops": flops}
        return {"bytes": 2 * tensors + t * hv * (16 + dv * 2) + state * (3 if case["s0"] else 1), "flops": 3 * flops}
    if op == "decode":
        n, hk, hv, dk, dv = (case[x] for x in ("seqs", "hk", "hv", "dk", "dv"))
        return {"bytes": n * (hv * dk * dv * 8 + 4 * hk * dk + hv * (4 * dv + 8) + 4), "flops": n * hv * dk * dv * 7}
    if op == "prep":
        t, h, d = case["tokens"], case["hq"] + case["hk"], case["dim"]
        return {"bytes": t * (h * d * 2 * (3 if case["back"] else 2) + 4), "flops": t * h * d * (12 if case["back"] else 7)}
    row = case["layers"] * case["heads"] * case["dk"] * case["dv"] * 4
    return {"bytes": 2 * row * case["pairs"], "flops": 0}


# ------------------------------------------------------------------------------- exact values

def _exact_steps(st):
    """The rule token by token in 64 bits, every sequence at once. Yields what each step needs."""
    cu = st["cu"].long()
    n, hv, rep = st["seqs"], st["hv"], st["hv"] // st["hk"]
    length = (cu[1:] - cu[:-1])
    flat = {x: st[x].reshape(-1, *st[x].shape[-2:]) for x in ("q", "k", "v")}
    flat["g"], flat["beta"] = st["g"].reshape(-1, hv), st["beta"].reshape(-1, hv)
    if "grad_o" in st:
        flat["grad_o"] = st["grad_o"].reshape(-1, *st["grad_o"].shape[-2:])

    def token(t):
        live = (t < length).view(n, 1)
        at = (cu[:-1] + t).clamp_max(st["tokens"] - 1)
        x = {name: f[at].double() for name, f in flat.items()}
        x["q"], x["k"] = (x[m].repeat_interleave(rep, 1) for m in ("q", "k"))
        x["g"], x["beta"] = torch.where(live, x["g"], 0.0), torch.where(live, x["beta"], 0.0)
        if "grad_o" in x:
            x["grad_o"] = torch.where(live[..., None], x["grad_o"], 0.0)
        x["live"], x["at"] = live, at
        return x

    return token


def _exact_step(S, x):
    R = S * x["g"].exp()[..., None, None]
    w = x["v"] - torch.einsum("nhij,nhi->nhj", R, x["k"])
    return R, w, R + torch.einsum("nhi,nhj->nhij", x["k"], x["beta"][..., None] * w)


def _exact_prefill(st):
    token = _exact_steps(st)
    n, hv, dk, dv = (st[x] for x in ("seqs", "hv", "dk", "dv"))
    S = torch.zeros(n, hv, dk, dv, device=DEV, dtype=torch.float64) if st["S0"] is None else st["S0"].double()
    o = torch.zeros(st["tokens"] + 1, hv, dv, device=DEV, dtype=torch.float64)
    for t in range(st["max_len"]):
        x = token(t)
        _, _, S = _exact_step(S, x)
        o[torch.where(x["live"][:, 0], x["at"], st["tokens"])] = torch.einsum("nhij,nhi->nhj", S, x["q"])
    return o[:-1].reshape(*st["v"].shape), S


def _exact_train(st):
    token = _exact_steps(st)
    n, hk, hv, dk, dv, total = (st[x] for x in ("seqs", "hk", "hv", "dk", "dv", "tokens"))
    S = torch.zeros(n, hv, dk, dv, device=DEV, dtype=torch.float64) if st["S0"] is None else st["S0"].double()
    every, kept = 32, []
    for t in range(st["max_len"]):
        if t % every == 0:
            kept.append(S)
        _, _, S = _exact_step(S, token(t))
    new = lambda *s: torch.zeros(total + 1, *s, device=DEV, dtype=torch.float64)  # noqa: E731
    dq, dk_, dv_, dg, db = new(hv, dk), new(hv, dk), new(hv, dv), new(hv), new(hv)
    dS = torch.zeros_like(S) if st["grad_S_T"] is None else st["grad_S_T"].double()
    for first in reversed(range(0, st["max_len"], every)):
        S, states = kept.pop(), []
        for t in range(first, min(first + every, st["max_len"])):
            x = token(t)
            R, w, S = _exact_step(S, x)
            states.append((x, R, w, S))
        for x, R, w, S in reversed(states):
            to = torch.where(x["live"][:, 0], x["at"], total)
            dS = dS + torch.einsum("nhi,nhj->nhij", x["q"], x["grad_o"])
            dq[to] = torch.einsum("nhij,nhj->nhi", S, x["grad_o"])
            du = torch.einsum("nhij,nhi->nhj", dS, x["k"])
            b = x["beta"][..., None]
            dv_[to] = b * du
            db[to] = (du * w).sum(-1)
            dk_[to] = torch.einsum("nhij,nhj->nhi", dS, b * w) - torch.einsum("nhij,nhj->nhi", R, b * du)
            dS = dS - torch.einsum("nhi,nhj->nhij", x["k"], b * du)
            dg[to] = (dS * R).sum((-1, -2))
            dS = dS * x["g"].exp()[..., None, None]
    share = lambda x: x[:-1].reshape(*st["q"].shape[:-2], hk, hv // hk, dk).sum(-2)  # noqa: E731
    return {"dq": share(dq), "dk": share(dk_), "dv": dv_[:-1].reshape(st["v"].shape), "dg": dg[:-1].reshape(st["g"].shape),
            "dbeta": db[:-1].reshape(st["beta"].shape), "dS0": dS}


def _exact_decode(st):
    rep = st["hv"] // st["hk"]
    S = st["S"].double()
    slots = st["slots"].long()
    x = {n: st[n].double() for n in ("v", "g", "beta")}
    x["q"], x["k"] = (st[n].double().repeat_interleave(rep, 1) for n in ("q", "k"))
    new = _exact_step(S[slots], x)[2]
    S[slots] = new
    return torch.einsum("nhij,nhi->nhj", new, x["q"]), S


def _exact_prep(st):
    """Each pair of channels as a complex number, turned by exp(i angle); gradients by autograd."""
    r, half = st["rotary"], st["layout"] == "half"

    def forward(x, w):
        if st["norm"] == "l2":
            x = torch.nn.functional.normalize(x, dim=-1, eps=1e-12)
        if st["norm"] == "rms":
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        if not r:
            return x
        head = x[..., :r]
        z = head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if half else head.unflatten(-1, (r // 2, 2))
        angle = st["positions"].double()[:, None, None] * st["inv_freq"]
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(angle), angle))
        z = z.transpose(-1, -2) if half else z
        return torch.cat([z.flatten(-2), x[..., r:]], -1)

    out, got = [], {}
    for n in ("q", "k"):
        x = st[n].double().requires_grad_(st["back"])
        w = None if st["w" + n] is None else st["w" + n].double().requires_grad_(st["back"])
        y = forward(x, w)
        if not st["back"]:
            out.append(y)
            continue
        grads = torch.autograd.grad(y, [x] if w is None else [x, w], st["d" + n].double())
        got["d" + n] = grads[0]
        if w is not None:
            got["dw" + n] = grads[1]
    return got if st["back"] else tuple(out)


def _exact_copy(st):
    S = st["S"].double()
    new = S.clone()
    for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
        new[:, b] = 0.0 if a < 0 else S[:, a]
    return new


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prefill":
        return _exact_prefill(st)
    if case["op"] == "train":
        return _exact_train(st)
    if case["op"] == "decode":
        return _exact_decode(st)
    return _exact_prep(st) if case["op"] == "prep" else _exact_copy(st)
