"""Float64 reference of retention, and the bounds its tests use.

Bounds are relative to the sizes that a result is put together from: with |.| taken of every input,
size_y = retention of the sizes, size_S = the final state of the sizes.  With u = 2^-24:
 * float32 sums: at most 128 products of a score, 128 terms of a block, 128 of the state's part and one rounding for
   each earlier block (up to 64 in these tests), the powers of gamma 3 u: below 512 u = 2^-15.
 * bf16 inputs with widths of 64 and 128 run on the tensor cores, where each score and each value of the state
   that a query meets is rounded once to bf16 (2^-8 of itself): 2^-8 of size_y more.
 * a result in bf16: 2^-8 of itself more.
The 2-norm of the error is far smaller: roundings to bf16 are spread over a step, 2^-8 / sqrt(3) at most in the mean
square, independent of each other; with terms of both signs that of a result's and of its terms' roundings are
2^-8 sqrt(2 / 3) of the result together.  ROOT is 2^-8.  For float32 results ROOT32 is 2^-19: 2^-24 for each of
up to 512 roundings at random is 2^-19.5."""
import torch

E = 2.0 ** -15
HALF = 2.0 ** -8
ROOT, ROOT32 = 2.0 ** -8, 2.0 ** -19
NAMES = ("q", "k", "v", "dy", "gamma", "S", "dS")


def inputs(B, H, N, d, dv, dtype, layout="bhnd", state=True, seed=0, gamma=None):
    g = torch.Generator().manual_seed(seed)

    def rand(w, s=1.0):
        t = torch.randn(B, H, N, w, generator=g) * s
        return (t if layout == "bhnd" else t.transpose(1, 2).contiguous()).to(dtype)

    x = {"q": rand(d, d ** -0.5), "k": rand(d), "v": rand(dv), "dy": rand(dv)}
    if gamma is None:
        x["gamma"] = 1 - torch.exp2(-(1 + 9 * torch.rand(H, generator=g)))
    else:
        x["gamma"] = torch.tensor([gamma[i % len(gamma)] for i in range(H)], dtype=torch.float32)
    x["S"] = torch.randn(B, H, d, dv, generator=g) if state else None
    x["dS"] = torch.randn(B, H, d, dv, generator=g) if state else None
    return x


def heads(t, layout):
    return t if layout == "bhnd" else t.transpose(1, 2)


def formula(q, k, v, gamma, S):
    """[B, H, N, ...] in 64 bits, the whole sequence at once."""
    N = q.shape[2]
    i = torch.arange(N, dtype=torch.float64)
    g = gamma[:, None, None]
    apart = (i[:, None] - i).clamp(min=0)
    D = (i[:, None] >= i) * torch.where(apart == 0, torch.ones(()), g ** apart)
    y = (q @ k.transpose(-1, -2) * D) @ v + g ** (i[:, None] + 1) * (q @ S)
    end = torch.where(i == N - 1, torch.ones(()), g[..., 0] ** (N - 1 - i))
    S1 = g ** N * S + (k * end[..., None]).transpose(-1, -2) @ v
    return y, S1


def forward(x, layout="bhnd"):
    """y, its size, S, its size."""
    q, k, v = (heads(x[n], layout).double() for n in "qkv")
    gamma = x["gamma"].double()
    S = torch.zeros(q.shape[0], q.shape[1], q.shape[3], v.shape[3], dtype=torch.float64) if x["S"] is None else x["S"].double()
    y, S1 = formula(q, k, v, gamma, S)
    ys, Ss = formula(q.abs(), k.abs(), v.abs(), gamma, S.abs())
    return heads(y, layout), heads(ys, layout), S1, Ss


def backward(x, layout="bhnd"):
    """[(gradient, size)] of q, k, v, S, by the formula and by its own sizes; with differentiation for the values."""
    q, k, v = (heads(x[n], layout).double().requires_grad_() for n in "qkv")
    gamma, dy = x["gamma"].double(), heads(x["dy"], layout).double()
    zero = torch.zeros(q.shape[0], q.shape[1], q.shape[3], v.shape[3], dtype=torch.float64)
    S = (zero if x["S"] is None else x["S"].double()).requires_grad_()
    dS = zero if x["dS"] is None else x["dS"].double()
    out = []
    for sizes in (False, True):
        ins = [t.detach().abs().requires_grad_() if sizes else t for t in (q, k, v, S)]
        y, S1 = formula(*ins[:3], gamma, ins[3])
        loss = (y * (dy.abs() if sizes else dy)).sum() + (S1 * (dS.abs() if sizes else dS)).sum()
        out.append(torch.autograd.grad(loss, ins))
    res = [(a, s) for a, s in zip(*out)]
    return [(heads(a, layout), heads(s, layout)) for a, s in res[:3]] + [res[3]]


def check(got, want, size, what, cores=False):
    """cores: computed on the tensor cores."""
    got, b = got.detach().cpu(), got.dtype == torch.bfloat16
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.numel() == 0:
        return
    err = (got.double() - want).abs()
    over = err - ((HALF if b else 2.0 ** -24) * want.abs() + (E + (HALF * 1.01 if cores and b else 0)) * size + 2.0 ** -130)
    assert bool((over <= 0).all()), f"{what}: {float(over.max())} over the bound"
    if got.numel() >= 64 and float(want.norm()) > 0:
        rel = float(err.norm() / want.norm())
        # terms that cancel more than at random leave the result smaller than their roundings allow for
        spread = max(1.0, float(size.norm() / want.norm()) * min(1.0, 12 / got.numel() ** 0.5))
        assert rel <= (ROOT if b else ROOT32) * spread, f"{what}: {rel} in the 2-norm"


def on_cores(x):
    return x["q"].dtype == torch.bfloat16 and x["q"].shape[-1] > 32 and x["v"].shape[-1] > 32
