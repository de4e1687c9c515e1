"""The gated delta rule and layer norm from their definitions in float64, on the CPU, and the
bounds the GPU tests hold the kernels to.

The recurrence (heads in a leading dimension, tokens one by one):
    e_t = v_t - a_t S_{t-1}^T k_t,  S_t = a_t S_{t-1} + k_t (b_t e_t)^T,  y_t = S_t^T q_t

Bounds.  An output of type T is one rounding away from a float32 computation: |got - ref| <=
eps(T)/2 |ref| + r, eps(T)/2 the largest relative rounding error.  r covers the float32 sums.  With
|k|^2 b <= 1 and gates <= 1 the map S_{t-1} -> S_t has norm <= 1, so what N tokens commit adds up at
most, and as roundings of either sign like sqrt(N): a token's e, u and S each round values of the
size of v and S a few times and sum d products, about (sqrt(d) + 4) 2^-24 relative to the RMS; the
largest of many elements is some 6 of these.  For N = 1000, d = 128: 6 * 15 * 32 * 6e-8 = 1.7e-4 of
the RMS if nothing were forgotten; b near 1/2 and d keys forget within about 2 d tokens: sqrt(256)
instead of sqrt(1000), 9e-5.  So r = 1e-4 RMS, the bound the float32 paths of this library have.
"""
import torch

R_F32 = 1e-4


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, ref, name="", r=R_F32, slack=0.0):
    """|got - ref| <= half a step of got's type + r RMS(ref) + slack, everywhere."""
    got64, ref = got.detach().cpu().double(), ref.double()
    assert got64.shape == ref.shape, (name, got64.shape, ref.shape)
    if not ref.numel():
        return
    assert torch.isfinite(got64).all(), f"{name}: not finite"
    rms = ref.square().mean().sqrt()
    bound = half_step(got.dtype) * ref.abs() + r * rms + slack + 1e-30
    worst = ((got64 - ref).abs() / bound).max().item()
    assert worst <= 1, f"{name}: {worst:.3g} times the bound"


def inputs(B, H, Hk, N, d, dv, dtype=torch.float32, gate="open", state=False, layout="bhnd", seed=0):
    """Random inputs; gate: None, "open" (memories of 4 to 8192 tokens), "any" (gates from 0 to 1,
    some closed for good by log_gate = -inf, some nearly)."""
    g = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=g)

    q, k = rn(B, Hk, N, d), rn(B, Hk, N, d) + 0.5 * rn(d)
    q = q / q.norm(dim=-1, keepdim=True) * d ** -0.5
    # a bf16 key of unit length is off by up to 2^-9: stay below 1
    k = 0.99 * k / k.norm(dim=-1, keepdim=True)
    x = dict(q=q.to(dtype), k=k.to(dtype), v=rn(B, H, N, dv).to(dtype),
             beta=torch.sigmoid(rn(B, H, N)), log_gate=None, S_in=None)
    if gate == "open":
        x["log_gate"] = torch.log1p(-torch.exp2(-(2 + 11 * torch.rand(B, H, N, generator=g))))
    elif gate == "any":
        lg = torch.log(torch.rand(B, H, N, generator=g))
        lg[torch.rand(B, H, N, generator=g) < 0.05] = -float("inf")
        lg[torch.rand(B, H, N, generator=g) < 0.05] = -60.0
        lg[torch.rand(B, H, N, generator=g) < 0.2] = 0.0
        x["log_gate"] = lg
        x["beta"][torch.rand(B, H, N, generator=g) < 0.1] = 0.0
        x["beta"][torch.rand(B, H, N, generator=g) < 0.1] = 1.0
    if state:
        x["S_in"] = rn(B, H, d, dv)
    if layout == "bnhd":
        for n in ("q", "k", "v", "beta", "log_gate"):
            if x[n] is not None:
                x[n] = x[n].transpose(1, 2).contiguous()
    return x


def _heads_first(t, layout):
    if t is None:
        return None
    return (t.transpose(1, 2) if layout == "bnhd" else t).double()


def forward(x, layout="bhnd"):
    """y (in v's layout, float64) and the final state."""
    q, k, v, beta, lg = (_heads_first(x[n], layout) for n in ("q", "k", "v", "beta", "log_gate"))
    B, H, N, dv = v.shape
    group = H // q.shape[1]
    q, k = (t.repeat_interleave(group, 1) for t in (q, k))
    S = torch.zeros(B, H, q.shape[-1], dv, dtype=torch.float64) if x["S_in"] is None else x["S_in"].double()
    y = []
    for t in range(N):
        if lg is not None:
            S = S * lg[:, :, t].exp()[..., None, None]
        e = v[:, :, t] - (S * k[:, :, t, :, None]).sum(-2)
        S = S + k[:, :, t, :, None] * (beta[:, :, t, None] * e)[..., None, :]
        y.append((S * q[:, :, t, :, None]).sum(-2))
    y = torch.stack(y, 2) if N else v
    return (y.transpose(1, 2) if layout == "bnhd" else y), S


def backward(x, dy, dS=None, layout="bhnd"):
    """Gradients by the formulas of include/linattn.h: dq, dk, dv, dbeta, dlog_gate, dS_in."""
    q, k, v, beta, lg, dy = (_heads_first(t, layout) for t in
                             (x["q"], x["k"], x["v"], x["beta"], x["log_gate"], dy))
    B, H, N, dv = v.shape
    Hk, d = q.shape[1], q.shape[-1]
    q, k = (t.repeat_interleave(H // Hk, 1) for t in (q, k))
    S = torch.zeros(B, H, d, dv, dtype=torch.float64) if x["S_in"] is None else x["S_in"].double()
    a = torch.ones(B, H, N, dtype=torch.float64) if lg is None else lg.exp()
    states, errs = [S], []
    for t in range(N):
        aS = a[:, :, t, None, None] * states[-1]
        errs.append(v[:, :, t] - (aS * k[:, :, t, :, None]).sum(-2))
        states.append(aS + k[:, :, t, :, None] * (beta[:, :, t, None] * errs[-1])[..., None, :])
    G = torch.zeros_like(S) if dS is None else dS.double()
    gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    gb, gl = torch.zeros_like(beta), torch.zeros_like(beta)
    for t in reversed(range(N)):
        G = G + q[:, :, t, :, None] * dy[:, :, t, None, :]
        gq[:, :, t] = (states[t + 1] * dy[:, :, t, None, :]).sum(-1)
        du = (G * k[:, :, t, :, None]).sum(-2)
        gb[:, :, t] = (du * errs[t]).sum(-1)
        bdu = beta[:, :, t, None] * du
        gv[:, :, t] = bdu
        aS = a[:, :, t, None, None] * states[t]
        gk[:, :, t] = ((G * (beta[:, :, t, None] * errs[t])[..., None, :]).sum(-1)
                       - (aS * bdu[..., None, :]).sum(-1))
        G = G - k[:, :, t, :, None] * bdu[..., None, :]
        gl[:, :, t] = (G * aS).sum((-1, -2))
        G = a[:, :, t, None, None] * G
    gq, gk = (t.reshape(B, Hk, H // Hk, N, d).sum(2) for t in (gq, gk))
    out = [gq, gk, gv, gb, gl if lg is not None else None]
    if layout == "bnhd":
        out = [t if t is None else t.transpose(1, 2) for t in out]
    return (*out, G)


def log_gate_slack(x, dy, dS, grads, layout="bhnd"):
    """What float32 rounding alone can leave of grad_log_gate where its terms cancel.

    grad_log_gate_m = <G, S> at the end of m's block of 64 tokens + the sum over the block's tokens
    t >= m of q_t . dq_t - v_t . dv_t.  The three terms can cancel altogether (a first token from
    an empty state has gradient 0 and terms of the size of y . dy), so an error relative to them is
    not one relative to their sum.  Each dot product, of float32 values that are themselves sums of
    d products, is off by about (sqrt(d) + 4) 2^-24 <= 16 2^-24 of its size; 64 tokens of either
    sign add sqrt(64) of these, and <G, S> one: 16 * 8 * 2^-24 of the terms' RMS, with 4 for the
    largest of many."""
    v, dyh = _heads_first(x["v"], layout), _heads_first(dy, layout)
    dvv = grads[2].transpose(1, 2) if layout == "bnhd" else grads[2]
    y, S = forward(x, layout)
    y = _heads_first(y, layout)   # q . dq of all a key head's value heads is their y . dy
    ends = torch.zeros(1, dtype=torch.float64) if dS is None else (dS.double() * S).sum((-1, -2)).abs()
    terms = torch.cat([(dyh * y).sum(-1).abs().flatten(), (v * dvv).sum(-1).abs().flatten(), ends.flatten()])
    return 4 * 16 * 8 * 2.0 ** -24 * terms.square().mean().sqrt().item()


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd
    y = y if weight is None else y * weight.double()
    y = y if bias is None else y + bias.double()
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_backward(dy, x, mean, rstd, weight=None):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[..., None], rstd.double()[..., None]
    xh = (x - mean) * rstd
    g = dy if weight is None else dy * weight.double()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    lead = tuple(range(x.dim() - 1))
    return dx, (dy * xh).sum(lead), dy.sum(lead)
