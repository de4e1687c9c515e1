"""Which outputs of the norm and rotation share memory with what: outputs among other tensors' gaps are taken, and only those
that share an element are refused (for tensors of the same strides; others count as sharing what lies between their ends)."""
import ctypes
import random

import pytest
import torch

import rotate_ref as R
from linear_rnn_sequence_gb300 import linattn as la


def status(q, k, yq, yk, strides, B, Hq, Hk, N, d):
    """Of a call on made-up addresses, float32, without a GPU: refused, or not carried out for want of one."""
    st = (ctypes.c_longlong * 12)(*strides)
    return la.lib().la_norm_rotate(*(ctypes.c_void_p(x) for x in (q, k, yq, yk)), st, B, Hq, Hk, N, d, 0, 0, 1, 1e-6, None, None, None,
                                   0, 0, None, 0, None)


def elements(at, st, B, H, N, d):
    return {at // 4 + b * st[0] + h * st[1] + n * st[2] + e for b in range(B) for h in range(H) for n in range(N) for e in range(d)}


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: for where nothing can be launched")
def test_shared_elements_are_refused_and_nothing_else():
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(4000):
        B, Hq, Hk, N = (rng.randint(1, 3) for _ in range(4))
        d = rng.choice([2, 4])
        # nested strides, in any order of batch, head and token, with gaps of any size
        st, inner = [0, 0, 0], d
        for i in rng.sample(range(3), 3):
            st[i] = inner + rng.choice([0, 0, 1, 2, d, 3 * d])
            inner = st[i] * max((B, max(Hq, Hk), N)[i], rng.randint(1, 4))
        base = 1 << 30
        q, k = base, (1 << 30) + 4 * rng.randint(-40, 40)
        yq = rng.choice([q, base + 4 * rng.randint(-60, 60)])
        yk = rng.choice([k, base + 4 * rng.randint(-60, 60)])
        own = {n: elements(a, st, B, h, N, d) for n, a, h in (("q", q, Hq), ("k", k, Hk), ("yq", yq, Hq), ("yk", yk, Hk))}
        pairs = [("yq", "k"), ("yk", "q"), ("yq", "yk")] + ([] if yq == q else [("yq", "q")]) + ([] if yk == k else [("yk", "k")])
        shared = any(own[a] & own[b] for a, b in pairs)
        got = status(q, k, yq, yk, st * 4, B, Hq, Hk, N, d)
        assert (got == la.LA_ERR_INVALID_ARG) == shared, (q, k, yq, yk, st, B, Hq, Hk, N, d)
        seen[shared] += 1
    assert min(seen) > 400


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bnhd", "bhnd"])
@pytest.mark.parametrize("pad", [8, 20, 64, 100])
def test_parts_of_a_padded_buffer(pad, layout):
    """Sequences that start at no multiple of a token's values: q and k, and where they go, are parts of the same tokens."""
    B, N, H, d = 3, 7, 2, 32
    W = 6 * H * d
    x = R.inputs(B, H, H, N, d, torch.bfloat16, layout, seed=pad)
    big = torch.full((B * (N * W + pad),), 7.0, dtype=torch.bfloat16, device="cuda")
    part = [torch.as_strided(big, (B, N, H, d), (N * W + pad, W, d, 1), i * H * d) for i in range(6)]
    if layout == "bhnd":
        part = [t.transpose(1, 2) for t in part]
    for t, n in zip(part, ("q", "k", "gq", "gk")):
        t.copy_(x[n])
    kw = dict(freq=x["freq"].cuda(), positions=x["positions"].cuda(), q_weight=x["wq"].cuda(), k_weight=x["wk"].cuda(), layout=layout)
    apart = [x[n].cuda() for n in ("q", "k", "gq", "gk")]
    want = la.norm_rotate(apart[0], apart[1], **kw)
    grads = la.norm_rotate_backward(apart[2], apart[3], apart[0], apart[1], **kw)
    got = la.norm_rotate_backward(part[2], part[3], part[0], part[1], out=(part[4], part[5]), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    la.norm_rotate(part[0], part[1], out=(part[4], part[5]), **kw)
    assert torch.equal(part[4], want[0]) and torch.equal(part[5], want[1])
    la.norm_rotate(part[0], part[1], out=(part[0], part[1]), **kw)
    assert torch.equal(part[0], want[0]) and torch.equal(part[1], want[1])
    assert torch.equal(part[2], apart[2]) and torch.equal(part[3], apart[3])
    gaps = torch.ones(big.numel(), dtype=torch.bool)
    for i in range(6):
        torch.as_strided(gaps, (B, N, H, d), (N * W + pad, W, d, 1), i * H * d).fill_(False)
    assert bool((big.cpu()[gaps] == 7).all())
    for bad in ((part[1], part[5]), (part[4], part[0]), (part[4], part[4])):
        with pytest.raises(la.LinAttnError):
            la.norm_rotate(part[0], part[1], out=bad, **kw)
