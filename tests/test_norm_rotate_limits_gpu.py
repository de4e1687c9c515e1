"""Norm and rotation at the ends of what the calls accept: far positions and large frequencies, rows next to nothing,
values that are not finite where no norm looks at them (bounds: rotate_ref.py; the angle of a frequency below 2^40 at any
position is off by less than 2^-27 turns, 4.7e-8, of which the bounds' 64 roundings leave room for 25)."""
import pytest
import torch

import rotate_ref as R
from linear_rnn_sequence_gb300 import linattn as la

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def args(x):
    return dict(freq=x["freq"].cuda(), positions=x["positions"].cuda(), q_weight=x["wq"].cuda(), k_weight=x["wk"].cuda())


FAR = [2 ** 46 + 3, 2 ** 50 + 12345, 2 ** 55 - 1, 2 ** 60 + 7, 2 ** 63 - 1, -2 ** 63, -2 ** 52 - 9, 2 ** 31, 2 ** 20 + 1, -1, 0]


# on both sides of where angles go from 64-bit fractions to 128-bit ones
BORDER = [2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, -2 ** 32 + 1, -2 ** 32, -2 ** 32 - 1, 2 ** 31 + 5, 3, 1, 0, -1]
FREQ = [1.0, -0.5, 0.1, 1e-4, 1e-12, 3.0, 6.283185307179586, 100.0, 1e5, -1e5, 2.0 ** 40 - 1, 2.0 ** -40, 0.0, 1e9, 2.0 ** -70, 1e-19]
SLOW = [1.0, -0.5, 0.1, 1e-4, 1e-12, 3.0, 6.283185307179586, 7.999999, 7.0, -7.9, 5.5, 2.0 ** -40, 0.0, 2.5, 2.0 ** -70, 1e-19]


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("positions,freq", [(FAR, FREQ), (FAR, SLOW), (BORDER, SLOW), (BORDER, FREQ), (BORDER, SLOW[:-1] + [8.0]),
                                            (BORDER, [-8.0] + SLOW[1:])])
def test_far_positions_and_large_frequencies(positions, freq, dtype, pairs):
    x = R.inputs(1, 2, 2, len(positions), 32, dtype, seed=1)
    x["positions"] = torch.tensor(positions)
    x["freq"] = torch.tensor(freq, dtype=torch.float64)
    q, k, gq, gk = (x[n].cuda() for n in ("q", "k", "gq", "gk"))
    out = la.norm_rotate(q, k, pairs=pairs, **args(x))
    res = la.norm_rotate_backward(gq, gk, q, k, pairs=pairs, **args(x))
    for key, y, g, gw in zip("qk", out, res[:2], res[2:]):
        want, size = R.forward(x, key, pairs=pairs)
        R.near(y, want, size, R.E, f"{key} out")
        dx, size, dw, wsize = R.backward(x, key, pairs=pairs)
        R.near(g, dx, size, R.E2, f"grad_{key}")
        R.near(gw, dw, wsize, R.E_SUM, f"grad_{key}_weight")


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [32, 30])
def test_gradients_without_a_norm_do_not_see_the_inputs(d, dtype, pairs):
    x = R.inputs(1, 3, 2, 5, d, dtype, rotated=8, seed=2)
    kw = dict(args(x), norm=None, pairs=pairs)
    gq, gk = x["gq"].cuda(), x["gk"].cuda()
    clean = la.norm_rotate_backward(gq, gk, x["q"].cuda(), x["k"].cuda(), **kw)
    q, k = x["q"].clone(), x["k"].clone()
    q[0, 0, 1, 2], q[0, 1, 2, 20], k[0, 1, 4, 3] = float("inf"), float("nan"), -float("inf")
    got = la.norm_rotate_backward(gq, gk, q.cuda(), k.cuda(), **kw)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    # the weights' gradients are sums of gradients times inputs: each in its own column
    for g, c, hurt in ((got[2], clean[2], [2, 20]), (got[3], clean[3], [3])):
        same = torch.ones(d, dtype=torch.bool)
        same[hurt] = False
        assert torch.equal(g.cpu()[same], c.cpu()[same]) and not bool(torch.isfinite(g.cpu()[hurt]).any())


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -133, 2.0 ** -100, 2.0 ** -91, 2.0 ** -90, 2.0 ** -89])
def test_small_rows_and_a_smaller_eps(eps, dtype, norm):
    """Rows whose squares float32 does not hold, beside others."""
    x = R.inputs(1, 3, 2, 8, 64, dtype, seed=3)
    for n in "qk":
        for t, down in enumerate((0.0, 2.0 ** -74, 2.0 ** -66, 2.0 ** -52, 2.0 ** -48, 2.0 ** -45, 2.0 ** -30)):
            x[n][:, :, t] *= down
    q, k, gq, gk = (x[n].cuda() for n in ("q", "k", "gq", "gk"))
    kw = dict(args(x), norm=norm, eps=eps)
    out = la.norm_rotate(q, k, **kw)
    res = la.norm_rotate_backward(gq, gk, q, k, **kw)
    for key, y, g, gw in zip("qk", out, res[:2], res[2:]):
        want, size = R.forward(x, key, norm=norm, eps=eps)
        R.near(y, want, size, R.E, f"{key} out")
        dx, size, dw, wsize = R.backward(x, key, norm=norm, eps=eps)
        R.near(g, dx, size, R.E2, f"grad_{key}")
        R.near(gw, dw, wsize, R.E_SUM, f"grad_{key}_weight")
