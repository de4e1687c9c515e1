"""Norm and rotation of queries and keys on the GPU against their float64 reference (bounds: rotate_ref.py)."""
import pytest
import torch

import rotate_ref as R
from linear_rnn_sequence_gb300 import linattn as la

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def args(x, weight=True):
    put = lambda t: None if t is None else t.cuda()  # noqa: E731
    return dict(freq=put(x["freq"]), positions=put(x["positions"]), q_weight=put(x["wq"]) if weight else None,
                k_weight=put(x["wk"]) if weight else None)


def check(x, N, layout="bhnd", norm="rms", pairs="halves", eps=1e-6, weight=True, q=None, k=None, gq=None, gk=None):
    q, k, gq, gk = (x[n].cuda() if t is None else t for n, t in (("q", q), ("k", k), ("gq", gq), ("gk", gk)))
    kw = dict(args(x, weight), layout=layout, norm=norm, pairs=pairs, eps=eps)
    out = la.norm_rotate(q, k, **kw)
    for key, y in zip("qk", out):
        want, size = R.forward(x, key, layout, norm, pairs, eps, weight, N)
        assert y.is_contiguous()
        R.near(y, want, size, R.E, f"{key} out")
    res = la.norm_rotate_backward(gq, gk, q, k, sums=True, **kw)
    for key, g, gw in zip("qk", res[:2], res[2:]):
        dx, size, dw, wsize = R.backward(x, key, layout, norm, pairs, eps, weight, N)
        R.near(g, dx, size, R.E2, f"grad_{key}")
        R.near(gw, dw, wsize, R.E_SUM, f"grad_{key}_weight")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("d", [2, 6, 16, 32, 34, 64, 66, 80, 96, 128, 130, 192, 200, 254, 256])
def test_every_width(d, pairs, dtype):
    layout = "bnhd" if d % 4 else "bhnd"
    norm = ["rms", "l2", None][d // 2 % 3]
    x = R.inputs(2, 3, 2, 37, d, dtype, layout, seed=d)
    check(x, 37, layout, norm, pairs, weight=d != 64)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("d,rotated", [(64, 0), (64, 1), (64, 2), (64, 8), (64, 16), (64, 31), (128, 16), (128, 3),
                                       (128, 24), (256, 64), (256, 100), (30, 7), (6, 1)])
def test_part_of_a_head(d, rotated, pairs, dtype):
    x = R.inputs(1, 2, 2, 19, d, dtype, "bnhd", seed=d + rotated, rotated=rotated)
    check(x, 19, "bnhd", "l2", pairs)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 1, 1), (1, 1, 1, 2), (3, 1, 5, 1), (1, 16, 16, 1), (2, 5, 1, 63), (5, 7, 3, 33),
                                       (1, 33, 2, 129), (1, 2, 2, 4097), (16, 4, 4, 257)])
def test_heads_and_lengths(B, Hq, Hk, N, dtype):
    for layout in ("bhnd", "bnhd"):
        check(R.inputs(B, Hq, Hk, N, 64, dtype, layout, seed=N), N, layout)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hq,Hk,d", [(1, 1, 1, 64), (1, 16, 16, 128), (256, 32, 8, 128), (3, 5, 2, 34)])
def test_single_tokens(B, Hq, Hk, d, dtype):
    check(R.inputs(B, Hq, Hk, None, d, dtype, seed=B), None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(dtype):
    x = R.inputs(2, 3, 2, 0, 64, dtype)
    check(x, 0)
    res = la.norm_rotate_backward(x["gq"].cuda(), x["gk"].cuda(), x["q"].cuda(), x["k"].cuda(), **args(x))
    assert res[2].abs().max() == 0 and res[3].abs().max() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("layout", ["bnhd", "bhnd"])
def test_parts_of_a_projection(layout, shift, dtype):
    """q, k (and v) side by side in each token, from a place that is a multiple of nothing on."""
    B, N, Hq, Hk, d = 2, 21, 4, 2, 64
    x = R.inputs(B, Hq, Hk, N, d, dtype, "bnhd", seed=shift)
    width = (Hq + 2 * Hk) * d + shift
    big = torch.full((B, N, width), 7.0, dtype=dtype, device="cuda")
    q = big[..., shift:shift + Hq * d].unflatten(-1, (Hq, d))
    k = big[..., shift + Hq * d:shift + (Hq + Hk) * d].unflatten(-1, (Hk, d))
    q.copy_(x["q"])
    k.copy_(x["k"])
    if layout == "bhnd":
        q, k = q.transpose(1, 2), k.transpose(1, 2)
        for n in ("q", "k", "gq", "gk"):
            x[n] = x[n].transpose(1, 2).contiguous()
    assert not q.is_contiguous()
    check(x, N, layout, q=q, k=k)
    # in place: the same values, and nothing else is written
    kw = dict(args(x), layout=layout)
    want = la.norm_rotate(q, k, **kw)
    before = big.clone()
    got = la.norm_rotate(q, k, out=(q, k), **kw)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    q.copy_(x["q"])
    k.copy_(x["k"])
    assert torch.equal(big, before)
    # gradients over the inputs, and over the outputs' gradients
    want = la.norm_rotate_backward(x["gq"].cuda(), x["gk"].cuda(), q, k, **kw)
    gq, gk = x["gq"].cuda(), x["gk"].cuda()
    got = la.norm_rotate_backward(gq, gk, q, k, out=(gq, gk), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = la.norm_rotate_backward(x["gq"].cuda(), x["gk"].cuda(), q, k, out=(q, k), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rest = big.clone()
    rest[..., shift:shift + (Hq + Hk) * d] = 7.0
    assert bool((rest == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_broadcast_inputs(dtype):
    """One row of keys for all heads; one upstream gradient for all tokens."""
    x = R.inputs(2, 2, 1, 9, 32, dtype)
    k, gq = x["k"].cuda().expand(2, 5, 9, 32), x["gq"][:, :, :1].cuda().expand(2, 2, 9, 32)
    gk = x["gk"].cuda().expand(2, 5, 9, 32)
    x["k"], x["gq"], x["gk"] = k.cpu(), gq.cpu(), gk.cpu()
    check(x, 9, k=k, gq=gq, gk=gk)


def test_offsets_past_32_bits():
    """Tokens 2^28 values apart: the last begins at value 11 * 2^28."""
    N, d = 12, 64
    x = R.inputs(1, 2, 1, N, d, BF16, "bnhd")
    big = torch.empty(N << 28, dtype=BF16, device="cuda")
    q = torch.as_strided(big, (1, N, 2, d), (N << 28, 1 << 28, d, 1))
    q.copy_(x["q"])
    check(x, N, "bnhd", q=q)
    want = la.norm_rotate(q, x["k"].cuda(), layout="bnhd", **args(x))[0]
    la.norm_rotate(q, x["k"].cuda(), layout="bnhd", out=(q, x["k"].cuda()), **args(x))
    assert torch.equal(q, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_positions(dtype):
    x = R.inputs(3, 2, 2, 11, 64, dtype)
    x["positions"] = torch.arange(100000, 100011)   # of all sequences
    check(x, 11)
    x["positions"] = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 40 + 12345, -1, -7, -2 ** 33, 5, 5])
    check(x, 11)
    # none: the token's index
    kw = args(x)
    kw["positions"] = None
    a = la.norm_rotate(x["q"].cuda(), x["k"].cuda(), **kw)
    kw["positions"] = torch.arange(11).cuda()
    b = la.norm_rotate(x["q"].cuda(), x["k"].cuda(), **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_frequencies():
    """Large, tiny, negative and zero ones; what has no angle gives NaN in its own pair."""
    x = R.inputs(1, 1, 1, 7, 32, F32)
    x["freq"] = torch.tensor([1.0, -0.5, 0.0, 1e-12, 3.0, 6.283185307179586, 1e-300, 100.0, 1e5, 0.1, 2.0 ** -70, 1e-3,
                              7.0, 2.0 ** -40, 1.5, 1e-6], dtype=torch.float64)
    check(x, 7)
    bad = x["freq"].clone()
    bad[3], bad[5], bad[7] = float("inf"), float("nan"), 2.0 ** 64
    kw = dict(args(x), freq=bad.cuda())
    y = la.norm_rotate(x["q"].cuda(), x["k"].cuda(), **kw)[0].cpu()
    nan = torch.zeros(32, dtype=torch.bool)
    nan[[3, 5, 7, 19, 21, 23]] = True
    assert bool((torch.isnan(y) == nan).all())


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sizes_of_values(dtype, norm):
    """Zeros, tiny values, values whose squares pass float32's range, and rows that are not finite."""
    x = R.inputs(1, 2, 2, 12, 64, dtype)
    for n in "qk":
        x[n][:, :, 0] = 0
        x[n][:, :, 1] *= 1e-30
        x[n][:, :, 2] *= 1e-4
        x[n][:, :, 3] *= 2.0 ** 62
        x[n][:, :, 4] *= 2.0 ** 100
        x[n][:, :, 5, 7] = 2.0 ** 125
    check(x, 12, norm=norm, eps=1e-5)
    kw = dict(args(x), norm=norm)
    clean = la.norm_rotate(x["q"].cuda(), x["k"].cuda(), **kw)
    q = x["q"].clone()
    q[0, 0, 6, 3], q[0, 0, 7, 9], q[0, 1, 8, 63] = float("nan"), float("inf"), -float("inf")
    y = la.norm_rotate(q.cuda(), x["k"].cuda(), **kw)
    assert torch.equal(y[1], clean[1])
    hurt = torch.zeros(1, 2, 12, dtype=torch.bool)
    hurt[0, 0, 6] = hurt[0, 0, 7] = hurt[0, 1, 8] = True
    assert torch.equal(y[0].cpu()[~hurt], clean[0].cpu()[~hurt])
    assert bool(torch.isnan(y[0].cpu()[0, 0, 6]).all())
    assert bool(torch.isnan(y[0].cpu()[0, 0, 7]).any()) and bool(torch.isnan(y[0].cpu()[0, 1, 8]).any())


@pytest.mark.parametrize("d", [6, 30, 64, 66, 128, 250])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_rows_beside_rows_that_are_not_numbers(d, dtype):
    """Heads that a lane works on together: each its own row's norm, whatever the others hold."""
    x = R.inputs(1, 9, 9, 3, d, dtype, seed=d)
    for n in "qk":
        x[n][:, 0::3] *= 2.0 ** 100
        x[n][:, 1::3, :, 1] = float("nan")
    want = {n: R.forward({**x, n: torch.nan_to_num(x[n])}, n, norm="rms") for n in "qk"}
    got = la.norm_rotate(x["q"].cuda(), x["k"].cuda(), **args(x))
    res = la.norm_rotate_backward(x["gq"].cuda(), x["gk"].cuda(), x["q"].cuda(), x["k"].cuda(), **args(x))
    whole = torch.tensor([h for h in range(9) if h % 3 != 1])
    for n, y, g in zip("qk", got, res):
        R.near(y[:, whole.cuda()], want[n][0][:, whole], want[n][1][:, whole], R.E, n)
        assert bool(torch.isnan(y[:, 1::3]).all()) and bool(torch.isfinite(g[:, whole.cuda()]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_infinities_without_a_norm(pairs, dtype):
    """They reach the value they are turned with and no other."""
    x = R.inputs(1, 1, 1, 3, 32, dtype, rotated=8)
    q = x["q"].clone()
    q[..., 1, 2], q[..., 1, 20] = float("inf"), float("nan")
    kw = dict(args(x), norm=None, pairs=pairs)
    y = la.norm_rotate(q.cuda(), x["k"].cuda(), **kw)[0].cpu()[0, 0]
    clean = la.norm_rotate(x["q"].cuda(), x["k"].cuda(), **kw)[0].cpu()[0, 0]
    touched = torch.zeros(3, 32, dtype=torch.bool)
    touched[1, [2, 10] if pairs == "halves" else [2, 3]] = True
    touched[1, 20] = True
    assert torch.equal(y[~touched], clean[~touched])
    assert not bool(torch.isfinite(y[touched]).any())


@pytest.mark.parametrize("norm", ["rms", "l2", None])
def test_gradients_against_differences(norm):
    x = R.inputs(2, 3, 2, 17, 64, F32, seed=3)
    kw = dict(args(x), norm=norm)
    q, k, gq, gk = (x[n].cuda() for n in ("q", "k", "gq", "gk"))
    res = la.norm_rotate_backward(gq, gk, q, k, **kw)

    def loss(q, k, wq, wk):
        a, b = la.norm_rotate(q, k, **{**kw, "q_weight": wq, "k_weight": wk})
        return float((a.double() * gq.double()).sum() + (b.double() * gk.double()).sum())

    ins = [q, k, kw["q_weight"], kw["k_weight"]]
    g = torch.Generator().manual_seed(1)
    for i, grad in enumerate(res):
        dirn = torch.randn(ins[i].shape, generator=g).cuda()
        h = 2.0 ** -8
        up, dn = list(ins), list(ins)
        up[i], dn[i] = ins[i] + h * dirn, ins[i] - h * dirn
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        want = float((grad.double() * dirn.double()).sum())
        # outputs are off by E of their size each, at random; the third order of the step by h^2
        slack = float((grad.double() * dirn.double()).abs().sum()) * 2 * h * h * 9 + R.E * 2000 / h
        assert abs(diff - want) <= slack, (i, diff, want, slack)
        assert slack < 40 * float(grad.double().norm())


def test_the_same_every_time_and_on_other_streams():
    x = R.inputs(4, 8, 8, 700, 128, BF16, "bnhd")
    q, k, gq, gk = (x[n].cuda() for n in ("q", "k", "gq", "gk"))
    kw = dict(args(x), layout="bnhd")
    first = (*la.norm_rotate(q, k, **kw), *la.norm_rotate_backward(gq, gk, q, k, **kw))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(*la.norm_rotate(q, k, stream=s, **kw), *la.norm_rotate_backward(gq, gk, q, k, stream=s, **kw)) for s in streams]
    torch.cuda.synchronize()
    for other in got:
        assert all(torch.equal(a, b) for a, b in zip(first, other))


def test_captured_and_replayed():
    x = R.inputs(2, 4, 2, 50, 128, BF16)
    q, k, gq, gk = (x[n].cuda() for n in ("q", "k", "gq", "gk"))
    kw = args(x)
    la.norm_rotate_backward(gq, gk, q, k, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (*la.norm_rotate(q, k, **kw), *la.norm_rotate_backward(gq, gk, q, k, **kw))
    q.mul_(-1.5)
    kw["positions"].add_(3)
    graph.replay()
    torch.cuda.synchronize()
    want = (*la.norm_rotate(q, k, **kw), *la.norm_rotate_backward(gq, gk, q, k, **kw))
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    x = R.inputs(2, 4, 2, 5, 64, BF16)
    q, k = x["q"].cuda(), x["k"].cuda()
    kw = args(x)
    for bad in (dict(layout="hbnd"), dict(norm="max"), dict(pairs="thirds"), dict(positions=kw["positions"].int()),
                dict(positions=kw["positions"][:1]), dict(positions=kw["positions"].cpu()), dict(freq=kw["freq"].float()),
                dict(freq=kw["freq"][None]), dict(q_weight=kw["q_weight"][:32]), dict(k_weight=kw["k_weight"].bfloat16()),
                dict(out=(q.float(), k)), dict(out=(q[:1], k)), dict(out=(q[0], k)), dict(out=(q, k[..., None]))):
        with pytest.raises((ValueError, TypeError)):
            la.norm_rotate(q, k, **{**kw, **bad})
    for a, b in ((q, k.float()), (q, k[:, :, :4]), (q, k[:1]), (q, k[..., :32]), (q[0], k), (q[0, 0], k[0, 0]),
                 (q.transpose(2, 3), k.transpose(2, 3)), (q, k.cpu()), (q.cpu(), k.cpu()), (q.half(), k.half())):
        with pytest.raises((ValueError, TypeError)):
            la.norm_rotate(a, b, norm="rms")
    with pytest.raises(ValueError):   # single tokens without positions
        la.norm_rotate(q[:, :, 0], k[:, :, 0], freq=kw["freq"])
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(freq=torch.ones(33, dtype=torch.float64, device="cuda")),
                dict(out=(q, q[:, :2])), dict(out=(q.flip(0)[:, :1].expand(2, 4, 5, 64), k)),
                dict(out=(kw["q_weight"].view(BF16).new_empty(q.shape), k[:, :1].expand(2, 2, 5, 64)))):
        with pytest.raises(la.LinAttnError):
            la.norm_rotate(q, k, **{**kw, **bad})
    with pytest.raises(la.LinAttnError):   # odd width
        la.norm_rotate(q[..., :33], k[..., :33])
    with pytest.raises(la.LinAttnError):
        la.norm_rotate_backward(q, k, q, k, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), **kw)
    la.norm_rotate(q, k, norm=None, eps=0.0)   # not read
