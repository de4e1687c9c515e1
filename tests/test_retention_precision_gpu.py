"""Retention where the terms of a result cancel: states, keys and values with a large common part that the queries do not see.

y and the gradients are sums of scores times values and of queries times states.  A prompt's scores and the states that its
queries meet enter the products as two bf16 pieces: the first cut to 8 bits, what is left of it (2^-7 of the value at most)
rounded to 8 bits, off by 2^-8 of that at most (half a step is 2^-9 of the next power of two, 2^-8 of the value itself), so
2^-15 of each term for every value.  With the float32 sums (retention_ref.E, 2^-15 of the sum of sizes) and the one rounding
of the result (2^-8 of itself) an element is off by at most

    2^-8 |y| + 2^-14 size,

which bounds the 2-norm likewise.  One bf16 piece would be off by 2^-8 of each term, 64 times that.  A single token takes
the state in float32."""
import pytest
import torch

import retention_ref as R
from linear_rnn_sequence_gb300 import linattn as la

BF16 = torch.bfloat16
TERM = 2.0 ** -14


def away_from(t, a):
    """t without its part along a (of unit length)."""
    return t - (t * a).sum(-1, keepdim=True) * a


def inputs(N, d, dv, shift, seed):
    """Keys and, in the state, every column with a common part along a that queries are orthogonal to (up to their
    rounding); values and upstream gradients of alternating sign with a common part along b; likewise behind the last token."""
    B, H = 1, 3
    g = torch.Generator().manual_seed(seed)
    a, b = (torch.nn.functional.normalize(torch.randn(w, generator=g), dim=0) for w in (d, dv))
    sign = (1 - 2 * (torch.arange(N) % 2))[:, None]
    r = lambda w: torch.randn(B, H, N, w, generator=g)  # noqa: E731
    x = {"q": away_from(r(d), a) * d ** -0.5, "k": r(d) + shift * a, "v": r(dv) + shift * sign * b,
         "dy": r(dv) + shift * sign * b}
    x = {n: t.to(BF16) for n, t in x.items()}
    x["gamma"] = torch.tensor([0.9999, 0.98, 1.0])
    S, dS = (torch.randn(B, H, d, dv, generator=g) for _ in range(2))
    x["S"] = S + shift * d ** 0.5 * a[:, None]
    x["dS"] = dS + shift * dv ** 0.5 * b
    return x


def near(got, want, size, what):
    got = got.detach().cpu()
    assert got.shape == want.shape
    half = R.HALF if got.dtype == BF16 else 2.0 ** -24
    err = (got.double() - want).abs()
    over = err - (half * want.abs() + TERM * size + 2.0 ** -130)
    rel, most = float(err.norm() / want.norm()), half + TERM * float(size.norm() / want.norm())
    assert rel <= most, f"{what}: {rel} in the 2-norm, at most {most}"
    assert bool((over <= 0).all()), f"{what}: {float(over.max())} over the bound"


def on_gpu(x):
    return {n: t.cuda() for n, t in x.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0.0, 8.0, 64.0])
@pytest.mark.parametrize("d,dv", [(64, 64), (64, 128), (128, 64), (128, 128), (32, 64)])
@pytest.mark.parametrize("N", [1, 100, 300, 1500])
def test_terms_that_cancel(N, d, dv, shift):
    x = inputs(N, d, dv, shift, seed=N + d + dv)
    c = on_gpu(x)
    y, S = la.forward_retention(c["q"], c["k"], c["v"], c["gamma"], S_in=c["S"], return_state=True, check_status=True)
    yr, ys, Sr, Ss = R.forward(x)
    near(y, yr, ys, "y")
    near(S, Sr, Ss, "S")
    grads = la.backward_retention(c["q"], c["k"], c["v"], c["gamma"], c["dy"], S_in=c["S"], grad_S_out=c["dS"], check_status=True)
    for n, g, (w, s) in zip(("grad_q", "grad_k", "grad_v", "grad_S_in"), grads, R.backward(x)):
        near(g, w, s, n)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dv", [64, 128])
def test_a_prompt_and_single_tokens_agree(d, dv):
    """The same tokens as a prompt and one by one, from a state with a large common part."""
    x = inputs(140, d, dv, 64.0, seed=d + dv)
    c = on_gpu(x)
    y = la.forward_retention(c["q"], c["k"], c["v"], c["gamma"], S_in=c["S"])
    S, rows = c["S"].clone(), []
    for t in range(140):
        rows.append(la.decode_step_retention(*(c[n][:, :, t].contiguous() for n in "qkv"), c["gamma"], S))
    yr, ys, _, _ = R.forward(x)
    both = torch.stack(rows, 2).cpu().double()
    err = (y.cpu().double() - both).abs()
    assert bool((err <= 2 * (R.HALF * yr.abs() + TERM * ys)).all())
    near(torch.stack(rows, 2), yr, ys, "token by token")


def emulated(x, pieces):
    """y by the block form in 64 bits, with each score and each value of the first state cut to this many bf16 pieces."""
    def cut(t):
        t, out = t.float(), torch.zeros_like(t.float())
        for i in range(pieces):
            p = t.to(BF16).float() if i == pieces - 1 else (t.view(torch.int32) & -65536).view(torch.float32)
            out, t = out + p, t - p
        return out.double()

    q, k, v, S = (x[n].double() for n in ("q", "k", "v", "S"))
    N = q.shape[2]
    i = torch.arange(N, dtype=torch.float64)
    g = x["gamma"].double()[:, None, None]
    D = torch.where(i[:, None] >= i, g ** (i[:, None] - i).clamp(min=0), torch.zeros(()).double())
    return (cut(q @ k.transpose(-1, -2) * D) @ v + g ** (i[:, None] + 1) * (q @ cut(S))).to(BF16)


@pytest.mark.parametrize("shift,N", [(64.0, 1), (64.0, 100), (8.0, 100)])
def test_the_bound_tells_one_piece_from_two(shift, N):
    x = inputs(N, 128, 128, shift, seed=1)
    yr, ys, _, _ = R.forward(x)
    near(emulated(x, 2), yr, ys, "two pieces")
    with pytest.raises(AssertionError):
        near(emulated(x, 1), yr, ys, "one piece")
