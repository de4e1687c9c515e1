"""Retention on the GPU against its float64 reference (bounds: retention_ref.py)."""
import pytest
import torch

import retention_ref as R
from linear_rnn_sequence_gb300 import linattn as la

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
GRADS = ("grad_q", "grad_k", "grad_v", "grad_S_in")


def on_gpu(x):
    return {n: t if t is None else t.cuda() for n, t in x.items()}


def forward(x, layout="bhnd", **kw):
    x = on_gpu(x)
    return la.forward_retention(x["q"], x["k"], x["v"], x["gamma"], S_in=x["S"], layout=layout, check_status=True, **kw)


def backward(x, layout="bhnd", **kw):
    x = on_gpu(x)
    return la.backward_retention(x["q"], x["k"], x["v"], x["gamma"], x["dy"], S_in=x["S"], grad_S_out=x["dS"],
                                 layout=layout, check_status=True, **kw)


def check_forward(x, layout="bhnd"):
    y, S = forward(x, layout, return_state=True)
    yr, ys, Sr, Ss = R.forward(x, layout)
    R.check(y, yr, ys, "y", R.on_cores(x))
    R.check(S, Sr, Ss, "S")
    assert torch.equal(forward(x, layout), y)   # without a state asked for


def check_backward(x, layout="bhnd"):
    got = backward(x, layout)
    for n, a, (w, s) in zip(GRADS, got, R.backward(x, layout)):
        if n == "grad_S_in" and x["S"] is None:
            assert a is None
        else:
            R.check(a, w, s, n, R.on_cores(x))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_every_width(d, dv, dtype):
    x = R.inputs(1, 3, 300, d, dv, dtype, seed=d + dv)
    check_forward(x)
    check_backward(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("N", [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500])
def test_lengths(N, layout, dtype):
    x = R.inputs(2, 2, N, 64, 128, dtype, layout, state=N % 3 != 0, seed=N)
    check_forward(x, layout)
    check_backward(x, layout)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gamma", [[0.0], [1.0], [0.5, 0.25], [1e-3, 1e-30], [0.999999, 0.70710677], [0.9, 0.99, 0.0, 1.0]])
def test_decays(gamma, dtype):
    x = R.inputs(1, 4, 333, 128, 64, dtype, gamma=gamma, seed=3)
    check_forward(x)
    check_backward(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (64, 128), (128, 64), (32, 32)])
@pytest.mark.parametrize("N", [3000, 4095])
def test_long_sequences_of_few_heads(N, d, dv, dtype):
    """Split into segments where few heads would leave SMs idle."""
    x = R.inputs(1, 2, N, d, dv, dtype, "bnhd", gamma=[0.9999, 0.97], seed=N)
    check_forward(x, "bnhd")
    check_backward(x, "bnhd")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_heads_than_sms(dtype):
    x = R.inputs(3, 111, 140, 64, 64, dtype, seed=1)
    check_forward(x)
    check_backward(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(dtype):
    x = R.inputs(2, 3, 0, 64, 32, dtype)
    y, S = forward(x, return_state=True)
    assert y.numel() == 0 and torch.equal(S.cpu(), x["S"])
    assert torch.equal(backward(x)[3].cpu(), x["dS"])
    x["S"] = x["dS"] = None
    assert forward(x, return_state=True)[1].abs().max() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cut", [1, 64, 100, 128, 256])
def test_in_parts(cut, dtype):
    """A prompt in two parts, the state carried in place; then token by token."""
    x = R.inputs(2, 3, 300, 64, 64, dtype, seed=cut)
    g = on_gpu(x)
    S = g["S"].clone()
    ys = []
    for a, b in ((0, cut), (cut, 290)):
        part = [g[n][:, :, a:b].contiguous() for n in "qkv"]
        y, S1 = la.forward_retention(*part, g["gamma"], S_in=S, S_out=S, return_state=True)
        assert S1 is S
        ys.append(y)
    for t in range(290, 300):
        ys.append(la.decode_step_retention(*(g[n][:, :, t].contiguous() for n in "qkv"), g["gamma"], S)[:, :, None])
    yr, ysz, Sr, Ssz = R.forward(x)
    R.check(torch.cat(ys, 2), yr, ysz, "y", R.on_cores(x))
    R.check(S, Sr, Ssz, "S")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (5, 3)])
def test_single_tokens(B, H, d, dv, dtype):
    x = R.inputs(B, H, 1, d, dv, dtype, seed=d, gamma=[0.0, 1.0, 0.97] if H > 1 else None)
    g = on_gpu(x)
    q, k, v = (g[n][:, :, 0].contiguous() for n in "qkv")
    S_out = torch.empty_like(g["S"])
    y = la.decode_step_retention(q, k, v, g["gamma"], g["S"], S_out=S_out)
    assert torch.equal(g["S"].cpu(), x["S"])
    yr, ys, Sr, Ss = R.forward(x)
    R.check(y[:, :, None], yr, ys, "y")
    R.check(S_out, Sr, Ss, "S")
    y2 = la.decode_step_retention(q, k, v, g["gamma"], g["S"])   # in place
    assert torch.equal(y2, y) and torch.equal(g["S"], S_out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("at", [0, 5, 127, 128, 190])
def test_what_is_not_finite_reaches_nothing_earlier(at, where, bad, dtype):
    x = R.inputs(1, 2, 270, 64, 128, dtype, gamma=[0.99, 0.5], seed=4)
    clean_y, clean_S = forward(x, return_state=True)
    clean = backward(x)
    y = {n: t if t is None else t.clone() for n, t in x.items()}
    y[where][0, 1, at, 7] = bad
    got, S = forward(y, return_state=True)
    assert torch.equal(got[:, 0], clean_y[:, 0]) and torch.equal(got[0, 1, :at], clean_y[0, 1, :at])
    assert not bool(torch.isfinite(got[0, 1, at]).all())
    if where == "q":
        assert torch.equal(S, clean_S) and torch.equal(got[0, 1, at + 1:], clean_y[0, 1, at + 1:])
    else:
        assert not bool(torch.isfinite(S[0, 1]).all())
        assert not bool(torch.isfinite(got[0, 1, at:]).all(-1).any())
    grads = backward(y)
    assert all(torch.equal(a[:, 0], b[:, 0]) for a, b in zip(grads, clean))
    # grad_q has later tokens' q in it nowhere, grad_k and grad_v earlier tokens' nothing
    assert torch.equal(grads[0][0, 1, :at], clean[0][0, 1, :at])
    assert torch.equal(grads[1][0, 1, at + 1:], clean[1][0, 1, at + 1:])
    assert torch.equal(grads[2][0, 1, at + 1:], clean[2][0, 1, at + 1:])


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("where", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("at", [63, 64, 129, 600])
def test_what_is_not_finite_at_other_widths(at, where, d, dv):
    x = R.inputs(1, 2, 700, d, dv, BF16, gamma=[0.99, 0.0], seed=13)
    clean_y, clean = forward(x), backward(x)
    for head, bad in ((0, float("inf")), (1, float("nan"))):
        y = {n: t if t is None else t.clone() for n, t in x.items()}
        y[where][0, head, at, 0 if at % 2 else -1] = bad
        got, grads = forward(y), backward(y)
        assert torch.equal(got[0, 1 - head], clean_y[0, 1 - head]) and torch.equal(got[0, head, :at], clean_y[0, head, :at])
        if where != "dy":
            assert not bool(torch.isfinite(got[0, head, at]).all())
        for g, c in zip(grads, clean):
            assert torch.equal(g[0, 1 - head], c[0, 1 - head])
        assert torch.equal(grads[0][0, head, :at], clean[0][0, head, :at])
        for g, c in zip(grads[1:3], clean[1:3]):
            assert torch.equal(g[0, head, at + 1:], c[0, head, at + 1:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dv", [64, 128])
def test_what_is_not_finite_in_many_blocks(d, dv):
    """Whatever the other blocks hold, a block's own tokens before its first such value are as they were and those from it on
    are not finite in its column."""
    x = R.inputs(1, 2, 2000, d, dv, BF16, gamma=[0.9], seed=14, state=False)
    clean = forward(x)
    for first in (3, 300):
        y = {n: t if t is None else t.clone() for n, t in x.items()}
        for t in range(first, 2000, 128):
            y["v"][0, 0, t, 7] = float("nan")
            y["v"][0, 1, t, dv - 1] = float("inf")
        for _ in range(5):
            got = forward(y)
            assert torch.equal(got[:, :, :first], clean[:, :, :first])
            assert not bool(torch.isfinite(got[0, 0, first:, 7]).any())
            assert not bool(torch.isfinite(got[0, 1, first:, dv - 1]).any())
            keep = torch.arange(dv) != 7
            assert torch.equal(got[0, 0][:, keep], clean[0, 0][:, keep])


def test_calls_from_several_threads():
    import threading
    xs = [on_gpu(R.inputs(1, 3, 200 + 130 * i, 64, 64, BF16, seed=i)) for i in range(4)]

    def call(x):
        return (*la.forward_retention(x["q"], x["k"], x["v"], x["gamma"], S_in=x["S"], return_state=True),
                *la.backward_retention(x["q"], x["k"], x["v"], x["gamma"], x["dy"], S_in=x["S"], grad_S_out=x["dS"]))

    want, got = [call(x) for x in xs], [None] * 4
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = call(xs[i])
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_what_is_not_finite_in_the_upstream_gradient(dtype):
    x = R.inputs(1, 1, 270, 64, 128, dtype, gamma=[0.99], seed=5)
    clean = backward(x)
    x["dy"][0, 0, 150, 3] = float("inf")
    grads = backward(x)
    assert torch.equal(grads[0][0, 0, :150], clean[0][0, 0, :150])
    assert torch.equal(grads[0][0, 0, 151:], clean[0][0, 0, 151:])
    assert torch.equal(grads[1][0, 0, 151:], clean[1][0, 0, 151:])
    assert torch.equal(grads[2][0, 0, 151:], clean[2][0, 0, 151:])
    assert not bool(torch.isfinite(grads[3]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_padding_in_front(dtype):
    x = R.inputs(1, 2, 200, 64, 64, dtype, state=False, seed=6)
    for n in "kv":
        x[n][:, :, :77] = 0
    y, S = forward(x, return_state=True)
    z = {n: t if t is None or n == "gamma" else t[:, :, 77:].contiguous() for n, t in x.items()}
    yr, ys, Sr, Ss = R.forward(z)
    R.check(y[:, :, 77:], yr, ys, "y", R.on_cores(x))
    R.check(S, Sr, Ss, "S")
    assert y[:, :, :77].abs().max() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nothing_else_is_written(dtype):
    x = R.inputs(2, 2, 150, 64, 128, dtype, "bnhd", seed=7)
    g = on_gpu(x)
    room = torch.full((x["v"].numel() + 512,), 7.0, dtype=dtype, device="cuda")
    out = room[256:-256].view(x["v"].shape)
    need = la.lib().la_retention_workspace_bytes(2, 2, 150, 64, 128, 1 if dtype is BF16 else 0)
    ws = torch.full((need + 512,), 5, dtype=torch.uint8, device="cuda")
    S = torch.full((2 * 2 * 64 * 128 + 128,), 7.0, device="cuda")
    la.forward_retention(g["q"], g["k"], g["v"], g["gamma"], S_in=g["S"], return_state=True, out=out, layout="bnhd",
                         S_out=S[64:-64].view(2, 2, 64, 128), workspace=ws[:need] if need else None)
    assert bool((room[:256] == 7).all()) and bool((room[-256:] == 7).all()) and bool((ws[need:] == 5).all())
    assert bool((S[:64] == 7).all()) and bool((S[-64:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [70, 3000])
def test_captured_replayed_and_sharing_a_workspace(N, dtype):
    x = R.inputs(1, 3, N, 64, 64, dtype, seed=8)
    g = on_gpu(x)
    code = 1 if dtype is BF16 else 0
    need = max(la.lib().la_retention_workspace_bytes(1, 3, N, 64, 64, code),
               la.lib().la_retention_backward_workspace_bytes(1, 3, N, 64, 64, code))
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def both():
        y, S = la.forward_retention(g["q"], g["k"], g["v"], g["gamma"], S_in=g["S"], return_state=True, workspace=ws)
        return (y, S, *la.backward_retention(g["q"], g["k"], g["v"], g["gamma"], g["dy"], S_in=g["S"],
                                             grad_S_out=g["dS"], workspace=ws))

    both()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(both())
    g["v"].mul_(-2)
    g["gamma"].mul_(0.5)
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    want = both()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_several_streams_at_once():
    x = R.inputs(2, 5, 700, 128, 128, BF16, seed=9)
    g = on_gpu(x)
    a = (g["q"], g["k"], g["v"], g["gamma"])
    want = (*la.forward_retention(*a, S_in=g["S"], return_state=True),
            *la.backward_retention(*a, g["dy"], S_in=g["S"], grad_S_out=g["dS"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [(*la.forward_retention(*a, S_in=g["S"], return_state=True, stream=s),
            *la.backward_retention(*a, g["dy"], S_in=g["S"], grad_S_out=g["dS"], stream=s)) for s in streams]
    torch.cuda.synchronize()
    for other in got:
        assert all(torch.equal(u, v) for u, v in zip(other, want))


@pytest.mark.parametrize("dtype", [F32])
def test_gradients_against_differences(dtype):
    x = R.inputs(1, 2, 150, 64, 32, dtype, seed=10)
    g = on_gpu(x)
    grads = backward(x)

    def loss(q, k, v, S):
        y, S1 = la.forward_retention(q, k, v, g["gamma"], S_in=S, return_state=True)
        return float((y.double() * g["dy"].double()).sum() + (S1.double() * g["dS"].double()).sum())

    ins = [g["q"], g["k"], g["v"], g["S"]]
    gen = torch.Generator().manual_seed(2)
    for i, grad in enumerate(grads):
        dirn = torch.randn(ins[i].shape, generator=gen).cuda()
        up, dn = list(ins), list(ins)
        up[i], dn[i] = ins[i] + dirn, ins[i] - dirn   # linear in each: any step
        diff, want = (loss(*up) - loss(*dn)) / 2, float((grad.double() * dirn.double()).sum())
        sizes = abs(loss(*up)) + abs(loss(*dn)) + float((grad.double() * dirn.double()).abs().sum())
        assert abs(diff - want) <= 2.0 ** -15 * sizes


def test_a_layer():
    """Projections' parts normed and rotated, retained, normed: a prompt, then tokens one by one; and the gradients of the
    whole prompt."""
    B, N, H, d, T = 2, 333, 3, 64, 4
    gen = torch.Generator().manual_seed(11)
    qkv = torch.randn(B, N + T, 3 * H, d, generator=gen).bfloat16()
    wq, wk, wn = (1 + 0.1 * torch.randn(d, generator=gen) for _ in range(3))
    freq = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))
    gamma = torch.tensor([0.9, 0.99, 0.999])
    do = torch.randn(B, N, H, d, generator=gen).bfloat16()

    # 64 bits, differentiable; values between the calls are not rounded
    x = qkv.double().requires_grad_()
    wq64, wk64, wn64 = (t.double().requires_grad_() for t in (wq, wk, wn))
    ang = torch.arange(N + T, dtype=torch.float64)[:, None] * freq
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]

    def turned(t, w):
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
        a, b = t[..., :d // 2], t[..., d // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).transpose(1, 2)

    q, k, v = turned(x[:, :, :H], wq64), turned(x[:, :, H:2 * H], wk64), x[:, :, 2 * H:].transpose(1, 2)
    y, _ = R.formula(q, k, v, gamma.double(), torch.zeros(B, H, d, d, dtype=torch.float64))
    o = torch.nn.functional.layer_norm(y.transpose(1, 2), (d,), wn64, torch.zeros(d, dtype=torch.float64))
    want = torch.autograd.grad((o[:, :N] * do.double()).sum(), (x, wq64, wk64, wn64))

    X, f, gm = qkv.cuda(), freq.cuda(), gamma.cuda()
    Wq, Wk, Wn = wq.cuda(), wk.cuda(), wn.cuda()
    P = X[:, :N]
    kw = dict(freq=f, q_weight=Wq, k_weight=Wk, layout="bnhd")
    q, k = la.norm_rotate(P[:, :, :H], P[:, :, H:2 * H], **kw)
    V = P[:, :, 2 * H:].contiguous()
    y, S = la.forward_retention(q, k, V, gm, return_state=True, layout="bnhd")
    out, mean, rstd = la.layer_norm(y, Wn, return_stats=True)
    near = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    # six roundings to bf16 on the way, at random: 2.5 x 2^-8 in the mean, four times that here
    assert near(out, o[:, :N].detach()) <= 10 * 2.0 ** -8
    for t in range(N, N + T):
        q1, k1 = la.norm_rotate(X[:, t, :H], X[:, t, H:2 * H], positions=torch.full((B,), t).cuda(),
                                **{**kw, "layout": "bhnd"})
        y1 = la.decode_step_retention(q1, k1, X[:, t, 2 * H:].contiguous(), gm, S)
        o1 = la.layer_norm(y1, Wn)
        assert near(o1, o[:, t].detach()) <= 10 * 2.0 ** -8
    gy, gwn, _ = la.layer_norm_backward(do.cuda(), y, mean, rstd, Wn)
    gq, gk, gv, _ = la.backward_retention(q, k, V, gm, gy, layout="bnhd")
    dx = torch.zeros_like(P)
    *_, gwq, gwk = la.norm_rotate_backward(gq, gk, P[:, :, :H], P[:, :, H:2 * H], out=(dx[:, :, :H], dx[:, :, H:2 * H]), **kw)
    dx[:, :, 2 * H:] = gv
    assert near(dx, want[0][:, :N]) <= 10 * 2.0 ** -8
    for a, b in ((gwq, want[1]), (gwk, want[2]), (gwn, want[3])):
        assert near(a, b) <= 10 * 2.0 ** -8


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("N", [100, 300, 4000])
def test_a_copy_that_never_comes(N, d, dv):
    """A bounded wait runs out, the call says so, and the next one is right."""
    x = R.inputs(1, 2, N, d, dv, BF16, seed=12)
    la.set_fault(drop_load_item=1, wait_limit_ns=2_000_000)
    try:
        for call in (lambda: forward(x, return_state=True), lambda: backward(x)):
            with pytest.raises(la.LinAttnError) as e:
                call()
            assert e.value.status == la.LA_ERR_TIMEOUT
    finally:
        la.set_fault()
    if N < 4000:
        check_forward(x)
        check_backward(x)
    else:
        forward(x), backward(x)


def test_refusals():
    x = on_gpu(R.inputs(1, 2, 8, 64, 32, BF16))
    q, k, v, g = x["q"], x["k"], x["v"], x["gamma"]
    for bad in ((q, k[:, :1], v, g), (q, k, v[:, :, :4], g), (q, k.float(), v, g), (q, k, v.float(), g), (q, k, v, g.double()),
                (q, k, v, g[:1]), (q, k, v, g.cpu()), (q[0], k[0], v[0], g), (q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), g),
                (q.half(), k.half(), v.half(), g), (q.cpu(), k, v, g)):
        with pytest.raises((ValueError, TypeError)):
            la.forward_retention(*bad)
        with pytest.raises((ValueError, TypeError)):
            la.backward_retention(*bad, x["dy"])
    for bad in (dict(S_in=x["S"][:, :1]), dict(S_in=x["S"].bfloat16()), dict(out=v.float()), dict(layout="nbhd"),
                dict(S_out=x["S"].transpose(2, 3))):
        with pytest.raises(ValueError):
            la.forward_retention(q, k, v, g, **bad)
    with pytest.raises(la.LinAttnError):
        la.forward_retention(q[..., :48].contiguous(), k[..., :48].contiguous(), v, g)
    with pytest.raises(la.LinAttnError):
        la.forward_retention(q, k, v, g, out=v)
    with pytest.raises(ValueError):
        la.decode_step_retention(q, k, v, g, x["S"])
    with pytest.raises(ValueError):
        la.decode_step_retention(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0], g, x["S"])
