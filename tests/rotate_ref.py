"""Float64 reference of the norm and rotation of queries and keys, and the bounds its tests use.

Bounds, relative to the values that a result is put together from (|u_a| + |u_b| for a rotated value): the sum of
at most 256 squares is at most 37 roundings long, of whose error the square root keeps half (18.5 u, u = 2^-24); the
reciprocal root is off by 4 u, the products by 3 u, sine and cosine by 4 u of 1 each, their argument by u of half a
turn (3.2 u), the rotation's two operations by 2 u: below 39 u.  E is 64 u.  A result in bf16 is off by half a step,
2^-8 of itself, more.  The gradient's second sum is as long as the first and enters once: E2 = 2 E.  Sums over rows:
one rounding a row of a lane, fewer than 256 in every test: E_SUM = 2^-16 of the sum of sizes.  Below the smallest
normal number, 2^-126, steps are 2^-133 in bf16 and 2^-149 in float32 whatever the value: half a step of the result's
type, and up to eight of float32's half steps in between."""
import torch

E = 2.0 ** -18
E2 = 2 * E
E_SUM = 2.0 ** -16


def inputs(B, Hq, Hk, N, d, dtype, layout="bhnd", seed=0, rotated=None):
    g = torch.Generator().manual_seed(seed)

    def rand(h):
        lead = (B, h) if N is None else (B, h, N) if layout == "bhnd" else (B, N, h)
        return (torch.randn(*lead, d, generator=g) * (0.2 + 2 * torch.rand(*lead, 1, generator=g))).to(dtype)

    x = {"q": rand(Hq), "k": rand(Hk), "gq": rand(Hq), "gk": rand(Hk)}
    x["wq"], x["wk"] = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    r = d // 2 if rotated is None else rotated
    x["freq"] = 10000.0 ** (-torch.arange(r, dtype=torch.float64) / max(r, 1)) if r else None
    lead = (B,) if N is None else (B, N)
    x["positions"] = torch.randint(0, 5000, lead, generator=g)
    return x


def angles(x, key, layout, N):
    """cos and sin by (batch, head, token) of x's tensor, in 64 bits; the whole turns are taken off exactly."""
    pos = x["positions"]
    a = pos[..., None].double() * x["freq"]
    if a.numel() and a.abs().max() > 1e6:   # beyond what 64 bits hold: in integers
        import math
        from fractions import Fraction
        two_pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62) * 2
        flat = [[float((Fraction(int(p)) * Fraction(float(f))) % two_pi) for f in x["freq"]] for p in pos.flatten()]
        a = torch.tensor(flat, dtype=torch.float64).reshape(*pos.shape, -1)
        assert math.isfinite(float(a.sum()))
    if N is None:
        a = a[:, None]                                         # [B, 1, r]
    else:
        if a.dim() == 2:
            a = a[None]
        a = a[:, None] if layout == "bhnd" else a[:, :, None]  # a place for the heads
    return a.cos(), a.sin()


def split(t, r, pairs):
    rot = t[..., :2 * r]
    return (rot[..., :r], rot[..., r:]) if pairs == "halves" else (rot[..., 0::2], rot[..., 1::2])


def join(a, b, rest, pairs):
    rot = torch.cat((a, b), -1) if pairs == "halves" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((rot, rest), -1)


def turn(t, cs, r, pairs, sign=1.0):
    if r == 0:
        return t
    (a, b), (c, s) = split(t, r, pairs), cs
    s = sign * s
    return join(a * c - b * s, b * c + a * s, t[..., 2 * r:], pairs)


def around(t, r, pairs):
    """|a| + |b| in the place of both values of a pair."""
    t = t.abs()
    if r == 0:
        return t
    a, b = split(t, r, pairs)
    return join(a + b, a + b, t[..., 2 * r:], pairs)


def scale(t, norm, eps):
    if norm is None:
        return torch.ones_like(t[..., :1])
    ss = (t * t).sum(-1, keepdim=True)
    return 1 / torch.sqrt((ss / t.shape[-1] if norm == "rms" else ss) + eps)


def forward(x, key, layout="bhnd", norm="rms", pairs="halves", eps=1e-6, weight=True, N=0):
    """The output of q or k and what its error is relative to."""
    t = x[key].double()
    r = 0 if x["freq"] is None else len(x["freq"])
    u = t * scale(t, norm, eps) * (x["w" + key].double() if weight else 1.0)
    cs = angles(x, key, layout, N) if r else None
    return turn(u, cs, r, pairs), around(u, r, pairs)


def backward(x, key, layout="bhnd", norm="rms", pairs="halves", eps=1e-6, weight=True, N=0):
    """(grad, its size, grad_weight, its size) of q or k."""
    t, up = x[key].double(), x["g" + key].double()
    r = 0 if x["freq"] is None else len(x["freq"])
    cs = angles(x, key, layout, N) if r else None
    w = x["w" + key].double() if weight else torch.ones(t.shape[-1], dtype=torch.float64)
    s = scale(t, norm, eps)
    xh, u, usize = t * s, turn(up, cs, r, pairs, -1.0), around(up, r, pairs)
    g = u * w
    c = 0.0 if norm is None else 1.0 / t.shape[-1] if norm == "rms" else 1.0
    dx = s * (g - c * xh * (g * xh).sum(-1, keepdim=True))
    size = s * (usize * w.abs() + c * xh.abs() * (usize * w.abs() * xh.abs()).sum(-1, keepdim=True))
    flat = lambda z: z.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731
    return dx, size, flat(u * xh), flat(usize * xh.abs())


def near(got, want, size, e, what):
    half, least = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float32: (2.0 ** -24, 2.0 ** -150)}[got.dtype]
    least += 2.0 ** -147
    got = got.detach().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.numel() == 0:
        return
    over = (got.double() - want).abs() - (half * want.abs() + e * size + least)
    assert bool((over <= 0).all()), f"{what}: {float(over.max())} over the bound"
