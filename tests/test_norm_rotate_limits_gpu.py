"""Norm and rotation at the ends of what the calls accept: values that are not finite where no norm looks at them."""
import pytest
import torch

import rotate_ref as R
from linear_rnn_sequence_gb300 import linattn as la

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def args(x):
    return dict(freq=x["freq"].cuda(), positions=x["positions"].cuda(), q_weight=x["wq"].cuda(), k_weight=x["wk"].cuda())


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
