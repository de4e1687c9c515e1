"""Calls of the norm and rotation of queries and keys (and its gradients) and of retention (whole sequences, its
gradients, a single token), to be timed.

Each head's query and key is normed, weighted, and rotated by its token's position; retention then keeps the state
S [d, dv] of a head as

    S_t = gamma_h S_{t-1} + k_t v_t^T,    y_t = S_t^T q_t.

``run`` makes one call: with ``own`` the library's, otherwise the same operator in elementary torch operations in 32
bits (the angles of the rotation and the powers of gamma in 64).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------- the cases
def _rotate(op, name, dtype, B, Hq, Hk, N, d, rotated, norm="rms", pairs="halves", layout="bnhd", start=0):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hk": Hk, "N": N, "d": d, "rotated": rotated,
            "norm": norm, "pairs": pairs, "layout": layout, "start": start}


def _retain(op, name, dtype, B, H, N, d, dv, layout="bhnd", state=True):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "H": H, "N": N, "d": d, "dv": dv, "layout": layout,
            "state": state}


def listed():
    return [
        # one layer of a training step: the projection's output, q, k and v side by side in each token
        _rotate("rotate", "rotate_b8n8192h16d128", "bf16", 8, 16, 16, 8192, 128, 128),
        # the next part of a prompt, of odd length and far on; a quarter of each head is rotated, pairs are neighbours
        _rotate("rotate", "rotate_b3n1031h12d64", "bf16", 3, 12, 4, 1031, 64, 16, pairs="adjacent", start=100000),
        # one token of a single sequence: latency
        _rotate("rotate", "rotate_token_b1h16d128", "bf16", 1, 16, 16, 0, 128, 128, start=8191),
        # the gradients of one layer of a training step
        _rotate("rotate_backward", "rotate_backward_b8n8192h16d128", "bf16", 8, 16, 16, 8192, 128, 128),
        # gradients in float32 of unit lengths, shared keys, heads before tokens
        _rotate("rotate_backward", "rotate_backward_b2h6n777d96_f32", "f32", 2, 6, 2, 777, 96, 96, norm="l2",
                layout="bhnd"),
        # one layer of a training step: whole sequences from an empty state, nothing carried out
        _retain("retention", "retention_b8h16n8192d128", "bf16", 8, 16, 8192, 128, 128, state=False),
        # the prefill of one long document that decoding goes on from
        _retain("retention", "retention_b1h32n131072d64", "bf16", 1, 32, 131072, 64, 64),
        # the next part of a prompt, of odd length, with heads inside tokens
        _retain("retention", "retention_b3h8n1031d128dv64", "bf16", 3, 8, 1031, 128, 64, layout="bnhd"),
        # the gradients of one layer of a training step
        _retain("retention_backward", "retention_backward_b8h16n8192d128", "bf16", 8, 16, 8192, 128, 128, state=False),
        # gradients in float32 through a carried state, odd length
        _retain("retention_backward", "retention_backward_b2h4n777d64_f32", "f32", 2, 4, 777, 64, 64),
        # one token of each of 256 sequences
        _retain("retention_step", "retention_step_b256h32d128", "bf16", 256, 32, 1, 128, 128),
        # one token of a single sequence: latency
        _retain("retention_step", "retention_step_b1h16d128", "bf16", 1, 16, 1, 128, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_backward", "retention", "retention", "retention_backward", "retention_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("rotate"):
        group = rng.choice([1, 1, 2, 4])
        c = _rotate(op, None, dtype, 1, 1, 1, 0, rng.choice([32, 64, 96, 128, 128, 256]), 0)
        c["Hk"] = rng.randint(1, 16 // group)
        c["Hq"] = c["Hk"] * group
        one = (c["Hq"] + c["Hk"]) * c["d"]
        if op == "rotate" and rng.random() < 0.3:   # single tokens
            c["B"] = _log(rng, 1, 512)
        else:
            c["N"] = _log(rng, 1, min(32768, (1 << 26) // one))
            c["B"] = _log(rng, 1, max(1, min(16, (1 << 26) // (one * c["N"]))))
        c["rotated"] = rng.choice([c["d"], c["d"], c["d"] // 2, c["d"] // 4])
        c["norm"] = rng.choice(["rms", "rms", "l2"])
        c["pairs"] = rng.choice(["halves", "halves", "adjacent"])
        c["layout"] = rng.choice(["bnhd", "bhnd"])
        c["start"] = rng.choice([0, 0, _log(rng, 1, 1 << 20)])
        del c["name"]
        return c
    c = _retain(op, None, dtype, 1, 1, 1, rng.choice([32, 64, 64, 128, 128]), rng.choice([32, 64, 64, 128, 128]),
                layout=rng.choice(["bhnd", "bnhd"]), state=rng.random() < 0.6)
    del c["name"]
    c["H"] = rng.randint(1, 32)
    if op == "retention_step":
        c["layout"], c["state"] = "bhnd", True
        c["B"] = _log(rng, 1, 192)
    else:
        # at most a quarter of the tokens of the largest training case
        c["N"] = _log(rng, 1, 32768 if op == "retention" else 8192)
        c["H"] = min(c["H"], max(1, (1 << 18) // c["N"]))
        c["B"] = _log(rng, 1, max(1, min(16, (1 << 18) // (c["N"] * c["H"]))))
    return c


# ---------------------------------------------------------------------------------------------------- the inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = _dt(case)

    def randn(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    st = {"case": case}
    if case["op"].startswith("rotate"):
        B, Hq, Hk, N, d, r = (case[x] for x in ("B", "Hq", "Hk", "N", "d", "rotated"))
        token = N == 0   # one token of each sequence
        # the projection's output: q, k and v of a token side by side; heads of different scale
        lead = (B,) if token else (B, N)
        x = randn(*lead, Hq + 2 * Hk, d) * (0.5 + 1.5 * torch.rand(Hq + 2 * Hk, 1, device=DEV, generator=g))
        x = x.to(dt)
        st["q"], st["k"] = x[..., :Hq, :], x[..., Hq:Hq + Hk, :]
        if case["layout"] == "bhnd" and not token:
            st["q"], st["k"] = (t.transpose(1, 2).contiguous() for t in (st["q"], st["k"]))
        st["q_weight"], st["k_weight"] = 1 + 0.2 * randn(d), 1 + 0.2 * randn(d)
        st["freq"] = 10000.0 ** (-torch.arange(r // 2, device=DEV, dtype=torch.float64) * 2 / r)
        first = torch.randint(0, 64, (B,), device=DEV, generator=g) + case["start"]
        st["positions"] = first if token else first[:, None] + torch.arange(N, device=DEV)
        if case["op"] == "rotate_backward":
            st["gq"], st["gk"] = (randn(*t.shape).to(dt) for t in (st["q"], st["k"]))
        return st

    B, H, N, d, dv = (case[x] for x in ("B", "H", "N", "d", "dv"))
    step = case["op"] == "retention_step"

    def heads(w):  # the shape of a tensor in the case's layout
        if step:
            return (B, H, w)
        return (B, H, N, w) if case["layout"] == "bhnd" else (B, N, H, w)

    # normed queries and keys, queries scaled by d^-1/2
    q, k = randn(*heads(d)), randn(*heads(d))
    st["q"] = (q / q.norm(dim=-1, keepdim=True)).to(dt)
    st["k"] = (k / k.norm(dim=-1, keepdim=True) * d ** 0.5).to(dt)
    st["v"] = randn(*heads(dv)).to(dt)
    # memories of 4 to 8192 tokens, spread over the heads
    st["gamma"] = 1 - torch.exp2(-(2 + 11 * torch.rand(H, device=DEV, generator=g)))
    st["S"] = randn(B, H, d, dv) if case["state"] else None
    if case["op"] == "retention_backward":
        st["dy"] = randn(*heads(dv)).to(dt)
        st["dS"] = 0.3 * randn(B, H, d, dv) if case["state"] else None
    return st


# ---------------------------------------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        from linear_rnn_sequence_gb300 import linattn as la
        if op == "rotate":
            return la.norm_rotate(st["q"], st["k"], freq=st["freq"], positions=st["positions"], norm=c["norm"],
                                  q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS, pairs=c["pairs"],
                                  layout=c["layout"])
        if op == "rotate_backward":
            return la.norm_rotate_backward(st["gq"], st["gk"], st["q"], st["k"], freq=st["freq"],
                                           positions=st["positions"], norm=c["norm"], q_weight=st["q_weight"],
                                           k_weight=st["k_weight"], eps=EPS, pairs=c["pairs"], layout=c["layout"])
        if op == "retention":
            return la.forward_retention(st["q"], st["k"], st["v"], st["gamma"], S_in=st["S"],
                                        return_state=c["state"], layout=c["layout"])
        if op == "retention_backward":
            return la.backward_retention(st["q"], st["k"], st["v"], st["gamma"], st["dy"], S_in=st["S"],
                                         grad_S_out=st["dS"], layout=c["layout"])
        S = torch.empty_like(st["S"])   # a new state beside the old one, so that a pass can be made again
        return la.decode_step_retention(st["q"], st["k"], st["v"], st["gamma"], st["S"], S_out=S), S
    if op == "rotate":
        turn = _turn(st, 1)
        return _norm_rotate(st, "q", turn), _norm_rotate(st, "k", turn)
    if op == "rotate_backward":
        turn = _turn(st, -1)
        gq, wq = _norm_rotate_backward(st, "q", turn)
        gk, wk = _norm_rotate_backward(st, "k", turn)
        return gq, gk, wq, wk
    if op == "retention":
        y, S = _retention(st)
        return (y, S) if c["state"] else y
    if op == "retention_backward":
        return _retention_backward(st)
    return _retention_step(st)


# ---------------------------------------------------------------------------------------------------- plain forms
def _turn(st, sign):
    """x -> x rotated by its token's angles, forwards or backwards."""
    c = st["case"]
    angle = st["positions"][..., None].double() * st["freq"]
    axis = -2 if c["N"] == 0 or c["layout"] == "bnhd" else -3   # the heads' place
    cos, sin = angle.cos().float().unsqueeze(axis), (sign * angle.sin()).float().unsqueeze(axis)
    r = c["rotated"]

    def turn(x):
        rot, rest = x[..., :r], x[..., r:]
        if c["pairs"] == "halves":
            a, b = rot[..., :r // 2], rot[..., r // 2:]
            return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
        a, b = rot[..., 0::2], rot[..., 1::2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)

    return turn


def _scale(x, norm):
    s = x.square().sum(-1, keepdim=True)
    return (s / x.shape[-1] + EPS).rsqrt() if norm == "rms" else (s + EPS).rsqrt()


def _norm_rotate(st, name, turn):
    x = st[name].float()
    return turn(x * _scale(x, st["case"]["norm"]) * st[name + "_weight"]).to(st[name].dtype)


def _norm_rotate_backward(st, name, turn):
    x = st[name].float()
    s = _scale(x, st["case"]["norm"])
    xh = x * s
    u = turn(st["g" + name].float())
    g = u * st[name + "_weight"]
    along = (g * xh).sum(-1, keepdim=True) / (x.shape[-1] if st["case"]["norm"] == "rms" else 1)
    return ((g - xh * along) * s).to(st[name].dtype), (u * xh).flatten(0, -2).sum(0)


def _block(N):   # tokens of a block of the plain form
    return 128 if N <= 16384 else 256


def _cut(t, c):
    """[B, H, blocks, tokens, width] in 32 bits, zeros behind the last token."""
    t = t.float() if c["layout"] == "bhnd" else t.float().transpose(1, 2)
    C = _block(c["N"])
    nc = -(-c["N"] // C)
    return torch.nn.functional.pad(t, (0, 0, 0, nc * C - c["N"])).reshape(c["B"], c["H"], nc, C, -1)


def _uncut(t, c):
    t = t.flatten(2, 3)[:, :, :c["N"]]
    return (t if c["layout"] == "bhnd" else t.transpose(1, 2)).to(_dt(c)).contiguous()


def _decay(c, gamma):
    """log gamma in 64 bits, and gamma^(i-j) within a block (zero above the diagonal)."""
    lg = gamma.double().log()
    n = torch.arange(_block(c["N"]), device=DEV)
    apart = (n[:, None] - n).double()
    return lg, torch.where(apart >= 0, apart * lg[:, None, None], -math.inf).exp().float()[:, None]


def _ahead(lg, tokens):
    """gamma^tokens for a whole tensor of distances, negative ones standing for zero: [H, *tokens.shape]."""
    e = lg.reshape(-1, *[1] * tokens.dim()) * tokens.double()
    return torch.where(tokens >= 0, e, -math.inf).exp().float()


def _states(c, lg, k, v, S):
    """The state before each block, and the last."""
    C, N, nc = k.shape[3], c["N"], k.shape[2]
    n, m = torch.arange(nc + 1, device=DEV), torch.arange(nc, device=DEV)
    at = torch.minimum(n * C, torch.full_like(n, N))   # tokens before each block, and all of them
    # each block's own sum, at the weights of its last token (of a whole block)
    own_sum = (k * _ahead(lg, C - 1 - torch.arange(C, device=DEV))[:, None, :, None]).transpose(-1, -2) @ v
    # that of block m is worth gamma^(at_n - (m + 1) C) before block n; a last, short block is not decayed so far
    apart = at[:, None] - (m + 1) * C
    last = _ahead(lg, apart.clamp(min=0) - (n[:, None] <= m) * 1e9)
    if N < nc * C:
        short = (k[:, :, -1:] * _ahead(lg, N - 1 - (nc - 1) * C - torch.arange(C, device=DEV))[:, None, :, None])
        own_sum = torch.cat((own_sum[:, :, :-1], short.transpose(-1, -2) @ v[:, :, -1:]), 2)
    S_all = (last @ own_sum.flatten(-2)).unflatten(-1, own_sum.shape[-2:])
    if S is not None:
        S_all = S_all + _ahead(lg, at)[None, :, :, None, None] * S[:, :, None]
    return S_all[:, :, :-1], S_all[:, :, -1]


def _retention(st):
    c = st["case"]
    q, k, v = (_cut(st[x], c) for x in "qkv")
    lg, D = _decay(c, st["gamma"])
    before, S = _states(c, lg, k, v, st["S"])
    C = q.shape[3]
    y = (q @ k.transpose(-1, -2) * D) @ v
    y = y + _ahead(lg, torch.arange(1, C + 1, device=DEV))[:, None, :, None] * (q @ before)
    return _uncut(y, c), S.contiguous()


def _retention_backward(st):
    c = st["case"]
    q, k, v, dy = (_cut(st[x], c) for x in ("q", "k", "v", "dy"))
    lg, D = _decay(c, st["gamma"])
    C, N, nc = q.shape[3], c["N"], q.shape[2]
    before, _ = _states(c, lg, k, v, st["S"])
    i = torch.arange(C, device=DEV)
    # G: the gradient of the state behind each block, gamma times that of the token that follows
    n = torch.arange(nc + 1, device=DEV)
    own_sum = (q * _ahead(lg, i + 1)[:, None, :, None]).transpose(-1, -2) @ dy   # seen from before the block
    apart = (n[None, 1:] - 1) * C - n[:, None] * C                               # of block m, seen from before block n
    G = (_ahead(lg, apart) @ own_sum.flatten(-2)).unflatten(-1, own_sum.shape[-2:])
    if st["dS"] is not None:
        left = torch.clamp(N - n * C, min=0)
        G = G + _ahead(lg, left)[None, :, :, None, None] * st["dS"][:, :, None]
    after = G[:, :, 1:]
    # of a short last block, from its own last token on
    L = torch.full((nc,), C, device=DEV)
    L[-1] = N - (nc - 1) * C
    to_end = _ahead(lg, torch.where(i < L[:, None], L[:, None] - 1 - i, -1))[..., None]
    P = dy @ v.transpose(-1, -2) * D
    up = _ahead(lg, i + 1)[:, None, :, None]
    dq = P @ k + up * (dy @ before.transpose(-1, -2))
    dk = P.transpose(-1, -2) @ q + to_end * (v @ after.transpose(-1, -2))
    dv = (q @ k.transpose(-1, -2) * D).transpose(-1, -2) @ dy + to_end * (k @ after)
    return _uncut(dq, c), _uncut(dk, c), _uncut(dv, c), G[:, :, 0].contiguous() if c["state"] else None


def _retention_step(st):
    q, k, v = (st[x].float() for x in "qkv")
    S = st["S"] * st["gamma"][:, None, None] + k[..., None] * v[..., None, :]
    return (S * q[..., None]).sum(-2).to(st["q"].dtype), S


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("rotate"):
        B, Hq, Hk, N, d, r = (case[x] for x in ("B", "Hq", "Hk", "N", "d", "rotated"))
        tokens = B * max(N, 1)
        n = tokens * (Hq + Hk) * d
        if case["op"] == "rotate":   # squares, scale, weight, and six operations for two rotated values
            return {"bytes": 2 * n * es + 8 * tokens + 8 * d + 4 * r, "flops": 4 * n + 3 * n * r // d}
        return {"bytes": 3 * n * es + 8 * tokens + 16 * d + 4 * r, "flops": 12 * n + 3 * n * r // d}
    B, H, N, d, dv = (case[x] for x in ("B", "H", "N", "d", "dv"))
    qk, vs = B * H * N * d * es, B * H * N * dv * es
    state = 4 * B * H * d * dv * case["state"]
    if case["op"] == "retention_backward":
        # the states again and their gradients (4), S dy, G v, G^T k (6) of d x dv a token
        return {"bytes": 4 * qk + 3 * vs + 3 * state + 4 * H, "flops": 10 * B * H * N * d * dv}
    # k v^T and S^T q
    return {"bytes": 2 * qk + 2 * vs + 2 * state + 4 * H, "flops": 4 * B * H * N * d * dv}


# ---------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits; rotations as complex products, gradients by differentiation."""
    st = prepare(case, seed)
    if case["op"].startswith("rotate"):
        return _exact_rotate(st)
    if case["op"] == "retention_step":
        q, k, v, S = (st[x].double() for x in ("q", "k", "v", "S"))
        S = torch.einsum("h,bhde->bhde", st["gamma"].double(), S) + torch.einsum("bhd,bhe->bhde", k, v)
        return torch.einsum("bhd,bhde->bhe", q, S), S
    grad = case["op"] == "retention_backward"
    heads = (lambda t: t) if case["layout"] == "bhnd" else (lambda t: t.transpose(1, 2))
    q, k, v = (heads(st[x]).double().requires_grad_(grad) for x in "qkv")
    S0 = (torch.zeros(case["B"], case["H"], case["d"], case["dv"], device=DEV, dtype=torch.float64)
          if st["S"] is None else st["S"].double()).requires_grad_(grad)
    y, S = _exact_retention(q, k, v, st["gamma"].double(), S0)
    if not grad:
        return (heads(y), S) if case["state"] else heads(y)
    loss = (y * heads(st["dy"]).double()).sum()
    if st["dS"] is not None:
        loss = loss + (S * st["dS"].double()).sum()
    gq, gk, gv, gS = torch.autograd.grad(loss, (q, k, v, S0))
    return heads(gq), heads(gk), heads(gv), gS if case["state"] else None


def _exact_retention(q, k, v, gamma, S):
    """Runs of 64 tokens, one after another."""
    N, out = q.shape[2], []
    g = gamma[:, None, None]
    for a in range(0, N, 64):
        qt, kt, vt = (t[:, :, a:a + 64] for t in (q, k, v))
        L = qt.shape[2]
        i = torch.arange(L, device=DEV, dtype=torch.float64)[:, None]
        lower = (i >= i.T).double() * g ** (i - i.T).clamp(min=0)
        out.append(torch.matmul(torch.einsum("bhid,bhjd->bhij", qt, kt) * lower, vt) + torch.matmul(qt * g ** (i + 1), S))
        S = S * g ** L + torch.einsum("bhjd,bhje->bhde", kt * g ** (L - 1 - i), vt)
    return torch.cat(out, 2), S


def _exact_rotate(st):
    c = st["case"]
    r, grad = c["rotated"], c["op"] == "rotate_backward"
    phase = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), torch.einsum("...,f->...f", st["positions"].double(), st["freq"]))
    phase = phase[:, None] if c["N"] == 0 else phase[:, :, None] if c["layout"] == "bnhd" else phase[:, None]

    def one(x, w):
        n = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        x = x / torch.sqrt((n * n / c["d"] if c["norm"] == "rms" else n * n) + EPS) * w
        z = x[..., :r].unflatten(-1, (2, r // 2) if c["pairs"] == "halves" else (r // 2, 2))
        z = torch.complex(*z.unbind(-2 if c["pairs"] == "halves" else -1)) * phase
        z = torch.stack((z.real, z.imag), -2 if c["pairs"] == "halves" else -1).flatten(-2)
        return torch.cat((z, x[..., r:]), -1)

    q, k, wq, wk = (st[x].double().requires_grad_(grad) for x in ("q", "k", "q_weight", "k_weight"))
    q1, k1 = one(q, wq), one(k, wk)
    if not grad:
        return q1, k1
    loss = (q1 * st["gq"].double()).sum() + (k1 * st["gk"].double()).sum()
    return torch.autograd.grad(loss, (q, k, wq, wk))
