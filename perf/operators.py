"""Calls of the gated delta rule (forward, gradients, single step) and of layer norm, to be timed.

The gated delta rule keeps the state S [d, dv] of a head as

    S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,    y_t = S_t^T q_t

with a_t = exp(log_gate_t).  Its output has no denominator; a layer norm over dv follows it.  ``run`` makes one
call: with ``own`` the library's, otherwise the same operator in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
C = 64  # tokens of a block of the plain form


# ---------------------------------------------------------------------------------------------------- the cases
def _delta(op, name, dtype, B, H, Hk, N, d, dv, layout="bhnd", gate=True, state=True):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "H": H, "Hk": Hk, "N": N, "d": d, "dv": dv,
            "layout": layout, "gate": gate, "state": state}


def _norm(op, name, dtype, rows, D, affine=True):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "D": D, "affine": affine}


def listed():
    return [
        # one layer of a training step: whole sequences from an empty state, nothing carried out
        _delta("forward", "forward_b8h16n8192d128", "bf16", 8, 16, 16, 8192, 128, 128, state=False),
        # the prefill of one long document that decoding goes on from
        _delta("forward", "forward_b1h32n131072d64", "bf16", 1, 32, 32, 131072, 64, 64),
        # the next part of a prompt, of odd length, with heads inside tokens and two value heads to a key head
        _delta("forward", "forward_b3h8n1031d128dv64", "bf16", 3, 8, 4, 1031, 128, 64, layout="bnhd"),
        # a few tokens in float32, without gates: latency
        _delta("forward", "forward_b1h2n256d32_f32", "f32", 1, 2, 2, 256, 32, 32, gate=False),
        # the gradients of one layer of a training step
        _delta("backward", "backward_b8h16n8192d128", "bf16", 8, 16, 16, 8192, 128, 128, state=False),
        # gradients in float32 through a carried state, shared key heads and an odd length
        _delta("backward", "backward_b2h4n777d64_f32", "f32", 2, 4, 2, 777, 64, 64),
        # one token of each of 256 sequences
        _delta("step", "step_b256h32d128", "bf16", 256, 32, 32, 1, 128, 128),
        # one token of a single sequence: latency
        _delta("step", "step_b1h16d128", "bf16", 1, 16, 16, 1, 128, 128),
        # the norm over each head's output, for the tokens of the training step
        _norm("norm", "norm_r1048576d128", "bf16", 1 << 20, 128),
        # the same for one token of a single sequence: latency
        _norm("norm", "norm_r16d128_f32", "f32", 16, 128),
        # the gradients of a norm over the model's width (16 heads of 128)
        _norm("norm_backward", "norm_backward_r65536d2048", "bf16", 65536, 2048),
        # an odd width in float32
        _norm("norm_backward", "norm_backward_r777d1000_f32", "f32", 777, 1000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "step", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        D = _log(rng, 3, 8192)
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, min(1 << 19, (1 << 26) // D)), "D": D,
                "affine": rng.random() < 0.8}
    d, dv = rng.choice([32, 64, 64, 128, 128]), rng.choice([32, 64, 64, 128, 128])
    group = rng.choice([1, 1, 2, 4])
    c = {"op": op, "dtype": dtype, "B": 1, "H": 1, "Hk": 1, "N": 1, "d": d, "dv": dv,
         "layout": rng.choice(["bhnd", "bnhd"]), "gate": rng.random() < 0.8, "state": rng.random() < 0.6}
    if op == "step":
        c["layout"], c["state"] = "bhnd", True
        c["Hk"] = rng.randint(1, 32 // group)
        c["B"] = _log(rng, 1, 192)
    else:
        # at most a quarter of the tokens of the largest training case
        c["N"] = _log(rng, 1, 32768 if op == "forward" else 8192)
        c["Hk"] = rng.randint(1, max(1, min(16 // group, (1 << 18) // (c["N"] * group))))
        c["B"] = _log(rng, 1, max(1, min(16, (1 << 18) // (c["N"] * c["Hk"] * group))))
    c["H"] = c["Hk"] * group
    return c


# ---------------------------------------------------------------------------------------------------- the inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = _dt(case)

    def randn(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    def rand(*shape):
        return torch.rand(shape, device=DEV, generator=g)

    st = {"case": case}
    if case["op"] in ("norm", "norm_backward"):
        R, D = case["rows"], case["D"]
        st["x"] = (randn(R, D) * (0.5 + rand(R, 1)) + 0.3 * randn(R, 1)).to(dt)
        st["weight"] = 1 + 0.2 * randn(D) if case["affine"] else None
        st["bias"] = 0.2 * randn(D) if case["affine"] else None
        if case["op"] == "norm_backward":
            st["dy"] = randn(R, D).to(dt)
            mean, rstd = _stats(st["x"].double())
            st["mean"], st["rstd"] = mean.float(), rstd.float()
        if own:
            from linear_rnn_sequence_gb300 import linattn
            st["la"] = linattn
        return st

    B, H, Hk, N, d, dv = (case[x] for x in ("B", "H", "Hk", "N", "d", "dv"))
    step = case["op"] == "step"

    def heads(n, w):  # the shape of a tensor of n heads in the case's layout
        if step:
            return (B, n, w)
        return (B, n, N, w) if case["layout"] == "bhnd" else (B, N, n, w)

    # queries and keys of unit length, keys with a common direction, queries scaled by d^-1/2
    q, k = randn(*heads(Hk, d)), randn(*heads(Hk, d)) + 0.5 * randn(d)
    st["q"] = (q / q.norm(dim=-1, keepdim=True) * d ** -0.5).to(dt)
    st["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    st["v"] = randn(*heads(H, dv)).to(dt)
    st["beta"] = torch.sigmoid(randn(*heads(H, 1)))[..., 0].contiguous()
    # memories of 4 to 8192 tokens
    st["log_gate"] = (torch.log1p(-torch.exp2(-(2 + 11 * rand(*heads(H, 1)))))[..., 0].contiguous()
                      if case["gate"] else None)
    st["S"] = 0.3 * randn(B, H, d, dv) if case["state"] else None
    if case["op"] == "backward":
        st["dy"] = randn(*heads(H, dv)).to(dt)
        st["dS"] = 0.05 * randn(B, H, d, dv) if case["state"] else None
    if own:
        from linear_rnn_sequence_gb300 import linattn
        st["la"] = linattn
    return st


# ---------------------------------------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        la = st["la"]
        if op == "forward":
            return la.forward_delta(st["q"], st["k"], st["v"], st["beta"], log_gate=st["log_gate"], S_in=st["S"],
                                    return_state=c["state"], layout=c["layout"])
        if op == "backward":
            return la.backward_delta(st["q"], st["k"], st["v"], st["beta"], st["dy"], log_gate=st["log_gate"],
                                     S_in=st["S"], grad_S_out=st["dS"], layout=c["layout"])
        if op == "step":  # a new state beside the old one, so that a pass can be made again
            S = torch.empty_like(st["S"])
            return la.decode_step_delta(st["q"], st["k"], st["v"], st["beta"], st["S"], log_gate=st["log_gate"],
                                        S_out=S), S
        if op == "norm":
            return la.layer_norm(st["x"], st["weight"], st["bias"], return_stats=True)
        return la.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["weight"])
    if op == "forward":
        return _forward(st)
    if op == "backward":
        return _backward(st)
    if op == "step":
        return _step(st)
    if op == "norm":
        return _layer_norm(st)
    return _layer_norm_backward(st)


# ---------------------------------------------------------------------------------------------------- plain forms
def _stats(x, eps=1e-5):
    mean = x.mean(-1)
    var = (x - mean[:, None]).square().mean(-1)
    return mean, (var + eps).rsqrt()


def _layer_norm(st):
    x = st["x"].float()
    mean, rstd = _stats(x)
    y = (x - mean[:, None]) * rstd[:, None]
    if st["weight"] is not None:
        y = y * st["weight"] + st["bias"]
    return y.to(st["x"].dtype), mean, rstd


def _layer_norm_backward(st):
    x, dy = st["x"].float(), st["dy"].float()
    xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
    g = dy if st["weight"] is None else dy * st["weight"]
    dx = (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True)) * st["rstd"][:, None]
    if st["weight"] is None:
        return dx.to(st["x"].dtype), None, None
    return dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _step(st):
    group = st["v"].shape[1] // st["q"].shape[1]
    q, k = (st[n].float().repeat_interleave(group, 1) for n in "qk")
    a = torch.ones_like(st["beta"]) if st["log_gate"] is None else st["log_gate"].exp()
    S = st["S"] * a[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    return (S * q[..., None]).sum(-2).to(st["q"].dtype), S


def _blocks(st):
    """The inputs in blocks: q, k, v [heads, blocks, C, width], beta and the gates' running log sums [heads, blocks, C]."""
    c = st["case"]
    B, H, N = c["B"], c["H"], c["N"]
    nc = -(-N // C)

    def cut(t, value_heads):
        t = t.float() if c["layout"] == "bhnd" else t.float().transpose(1, 2)
        if not value_heads:
            t = t.repeat_interleave(H // c["Hk"], 1)
        t = torch.nn.functional.pad(t, (0, 0, 0, nc * C - N))
        return t.reshape(B * H, nc, C, t.shape[-1])

    q, k, v = cut(st["q"], False), cut(st["k"], False), cut(st["v"], True)
    beta = cut(st["beta"][..., None], True)[..., 0]
    lg = torch.zeros_like(beta) if st["log_gate"] is None else cut(st["log_gate"][..., None], True)[..., 0]
    return q, k, v, beta, lg.double().cumsum(-1), cut


def _uncut(t, c):
    t = t.reshape(c["B"], c["H"], -1, t.shape[-1])[:, :, :c["N"]]
    return (t if c["layout"] == "bhnd" else t.transpose(1, 2)).contiguous()


def _inner(q, k, beta, cum):
    """What of a block does not depend on the state: the gates' products, the inverse, the masked scores."""
    n = torch.arange(C, device=q.device)
    decay = torch.where(n[:, None] >= n[None, :], cum[..., :, None] - cum[..., None, :], -math.inf).exp().float()
    kk = decay.tril(-1) * (k @ k.transpose(-1, -2))
    A = beta[..., None] * kk
    T = torch.eye(C, device=q.device).expand_as(A).contiguous()
    for i in range(1, C):  # (I + A)^-1, row by row
        T[..., i, :i] = -(A[..., i, None, :i] @ T[..., :i, :i])[..., 0, :]
    return decay, kk, T, decay * (q @ k.transpose(-1, -2))


def _states(st, q, k, v, beta, cum, T, decay):
    """The state before each block, and u of each block."""
    c = st["case"]
    a = cum.exp().float()
    S = (torch.zeros(c["B"] * c["H"], c["d"], c["dv"], device=q.device) if st["S"] is None
         else st["S"].reshape(-1, c["d"], c["dv"]))
    W = T @ ((beta * a)[..., None] * k)
    U = T @ (beta[..., None] * v)
    kT = (decay[..., -1, :, None] * k).transpose(-1, -2)
    before = []
    for n in range(q.shape[1]):
        before.append(S)
        U[:, n] -= W[:, n] @ S
        S = a[:, n, -1, None, None] * S + kT[:, n] @ U[:, n]
    return before, S, U, a


def _forward(st):
    c = st["case"]
    q, k, v, beta, cum, _ = _blocks(st)
    decay, _, T, P = _inner(q, k, beta, cum)
    before, S, U, a = _states(st, q, k, v, beta, cum, T, decay)
    y = P @ U
    for n in range(q.shape[1]):
        y[:, n] += a[:, n, :, None] * (q[:, n] @ before[n])
    y = _uncut(y, c).to(_dt(c))
    return (y, S.reshape(c["B"], c["H"], c["d"], c["dv"])) if c["state"] else y


def _backward(st):
    c = st["case"]
    q, k, v, beta, cum, cut = _blocks(st)
    dy = cut(st["dy"], True)
    decay, kk, T, P = _inner(q, k, beta, cum)
    before, S_end, U, a = _states(st, q, k, v, beta, cum, T, decay)
    nc = q.shape[1]
    dS = torch.zeros_like(S_end) if st["dS"] is None else st["dS"].reshape(S_end.shape)
    after, dU, dR = [None] * nc, P.transpose(-1, -2) @ dy, torch.empty_like(U)
    kg = decay[..., -1, :, None] * k
    aq, bk = (a[..., None] * q).transpose(-1, -2), ((beta * a)[..., None] * k).transpose(-1, -2)
    for n in reversed(range(nc)):
        after[n] = dS
        dR[:, n] = T[:, n].transpose(-1, -2) @ (dU[:, n] + kg[:, n] @ dS)
        dS = a[:, n, -1, None, None] * dS + aq[:, n] @ dy[:, n] - bk[:, n] @ dR[:, n]
    S0, dS1 = torch.stack(before, 1), torch.stack(after, 1)
    dv = beta[..., None] * dR
    db = (dR * (v - a[..., None] * (k @ S0) - kk @ U)).sum(-1)
    dP = decay * (dy @ U.transpose(-1, -2))
    F = -beta[..., None] * decay.tril(-1) * (dR @ U.transpose(-1, -2))
    dq = a[..., None] * (dy @ S0.transpose(-1, -2)) + dP @ k
    dk = (kg.new_zeros(()) + decay[..., -1, :, None] * (U @ dS1.transpose(-1, -2)) + dP.transpose(-1, -2) @ q
          - (beta * a)[..., None] * (dR @ S0.transpose(-1, -2)) + F @ k + F.transpose(-1, -2) @ k)
    out = [dq, dk, dv]
    group = c["H"] // c["Hk"]
    for i in range(3):
        t = out[i].reshape(c["B"], c["H"], nc * C, -1)[:, :, :c["N"]]
        if i < 2:
            t = t.reshape(c["B"], c["Hk"], group, c["N"], -1).sum(2)
        out[i] = (t if c["layout"] == "bhnd" else t.transpose(1, 2)).to(_dt(c)).contiguous()
    out.append(_uncut(db[..., None], c)[..., 0].contiguous())
    if c["gate"]:
        # scaling S_t scales what is read of it and what is carried on of it
        x = ((q * dq).sum(-1) - (v * dv).sum(-1)).double()
        carried = torch.stack([(S0[:, n + 1] if n + 1 < nc else S_end).mul(after[n]).double().sum((-1, -2)) for n in range(nc)], 1)
        dlg = x.flip(-1).cumsum(-1).flip(-1) + carried[..., None]
        out.append(_uncut(dlg.float()[..., None], c)[..., 0].contiguous())
    else:
        out.append(None)
    out.append(dS.reshape(c["B"], c["H"], c["d"], c["dv"]) if c["state"] else None)
    return tuple(out)


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["D"]
        return {"bytes": 2 * n * es + 8 * case["rows"] + 8 * case["D"] * case["affine"], "flops": 8 * n}
    if case["op"] == "norm_backward":
        n = case["rows"] * case["D"]
        return {"bytes": 3 * n * es + 8 * case["rows"] + 12 * case["D"] * case["affine"], "flops": 13 * n}
    B, H, Hk, N, d, dv = (case[x] for x in ("B", "H", "Hk", "N", "d", "dv"))
    qk, vs, sc = B * Hk * N * d * es, B * H * N * dv * es, 4 * B * H * N * (2 if case["gate"] else 1)
    state = 4 * B * H * d * dv * case["state"]
    if case["op"] == "backward":
        # the states again (4), and per token q dy^T, G^T k, k du^T, S dy, G u, S du of d x dv (12)
        return {"bytes": 4 * qk + 3 * vs + 2 * sc + 3 * state, "flops": 16 * B * H * N * d * dv}
    # S^T k, k u^T, S^T q
    return {"bytes": 2 * qk + 2 * vs + sc + 2 * state, "flops": 6 * B * H * N * d * dv}


# ---------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions, token by token, in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "norm":
        x = st["x"].double()
        m = x.sum(1, keepdim=True) / case["D"]
        r = 1 / torch.sqrt(((x - m) ** 2).sum(1, keepdim=True) / case["D"] + 1e-5)
        y = (x - m) * r
        y = y if st["weight"] is None else y * st["weight"].double() + st["bias"].double()
        return y, m[:, 0], r[:, 0]
    if case["op"] == "norm_backward":
        x, dy, D = st["x"].double(), st["dy"].double(), case["D"]
        m, r = st["mean"].double()[:, None], st["rstd"].double()[:, None]
        w = torch.ones(D, device=DEV, dtype=torch.float64) if st["weight"] is None else st["weight"].double()
        xh = (x - m) * r
        a, b = (dy * w).sum(1, keepdim=True), (dy * w * xh).sum(1, keepdim=True)
        dx = r * (dy * w - a / D - xh * b / D)
        return (dx, None, None) if st["weight"] is None else (dx, (dy * xh).sum(0), dy.sum(0))

    B, H, N = case["B"], case["H"], case["N"]
    if N > 140000 or (case["op"] == "backward" and N > 10000):
        return None
    group = H // case["Hk"]

    def per_token(t, shared):  # [N, heads, width]
        if t is None:
            return None
        if case["op"] == "step":
            t = t[:, :, None] if t.dim() == 3 else t[:, :, None, None]
        elif t.dim() == 3:
            t = t[..., None]
        if case["op"] != "step" and case["layout"] == "bnhd":
            t = t.transpose(1, 2)
        if shared and group > 1:
            t = t[:, :, None].expand(-1, -1, group, -1, -1).reshape(B, H, N, -1)
        return t.permute(2, 0, 1, 3).reshape(N, B * H, -1).contiguous()

    q, k, v = per_token(st["q"], True), per_token(st["k"], True), per_token(st["v"], False)
    beta, lg = per_token(st["beta"], False), per_token(st["log_gate"], False)
    S = torch.zeros(B * H, case["d"], case["dv"], device=DEV, dtype=torch.float64)
    if st["S"] is not None:
        S += st["S"].reshape(S.shape)

    def advance(S, t):
        kt, vt, bt = k[t].double()[:, :, None], v[t].double()[:, None], beta[t].double()[:, None]
        if lg is not None:
            S = S * lg[t].double().exp()[:, None]
        e = vt - (kt * S).sum(1, keepdim=True)
        return S + kt * (bt * e), e

    if case["op"] != "backward":
        y = torch.empty(N, B * H, case["dv"], device=DEV, dtype=torch.float64)
        for t in range(N):
            S, _ = advance(S, t)
            y[t] = (q[t].double()[:, :, None] * S).sum(1)
        if case["op"] == "step":
            return y[0].reshape(B, H, -1), S.reshape(B, H, case["d"], case["dv"])
        y = y.reshape(N, B, H, -1).permute((1, 2, 0, 3) if case["layout"] == "bhnd" else (1, 0, 2, 3))
        return (y, S.reshape(B, H, case["d"], case["dv"])) if case["state"] else y

    dy = per_token(st["dy"], False)
    f64 = {"device": DEV, "dtype": torch.float64}
    dq, dk, dv = (torch.empty(N, B * H, w, **f64) for w in (case["d"], case["d"], case["dv"]))
    db, dl = torch.empty(N, B * H, 1, **f64), torch.empty(N, B * H, 1, **f64)
    keep, L = [], 96
    for t in range(N):
        if t % L == 0:
            keep.append(S)
        S, _ = advance(S, t)
    G = torch.zeros_like(S) if st["dS"] is None else st["dS"].reshape(S.shape).double()
    for first in reversed(range(0, N, L)):
        states, errs = [keep[first // L]], []
        for t in range(first, min(N, first + L)):
            S1, e = advance(states[-1], t)
            states.append(S1)
            errs.append(e)
        for t in reversed(range(first, min(N, first + L))):
            S0, S1, e = states[t - first], states[t - first + 1], errs[t - first]
            kt, qt = k[t].double()[:, :, None], q[t].double()[:, :, None]
            vt, dyt, bt = v[t].double()[:, None], dy[t].double()[:, None], beta[t].double()[:, None]
            a = 1.0 if lg is None else lg[t].double().exp()[:, None]
            dq[t] = (S1 * dyt).sum(2)
            G = G + qt * dyt
            du = (kt * G).sum(1, keepdim=True)
            dk[t] = (G * (bt * e)).sum(2) - (a * S0 * (bt * du)).sum(2)
            dv[t] = (bt * du)[:, 0]
            db[t] = (du * e).sum(2)
            G = G - kt * (bt * du)
            dl[t] = (G * (a * S0)).sum((1, 2))[:, None]
            G = a * G

    def back(t, shared):
        t = t.reshape(N, B, H, -1)
        if shared:
            t = t.reshape(N, B, case["Hk"], group, -1).sum(3)
        return t.permute((1, 2, 0, 3) if case["layout"] == "bhnd" else (1, 0, 2, 3))

    return (back(dq, True), back(dk, True), back(dv, False), back(db, False)[..., 0],
            back(dl, False)[..., 0] if lg is not None else None,
            G.reshape(B, H, case["d"], case["dv"]) if case["state"] else None)
