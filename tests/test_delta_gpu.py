"""The gated delta rule and layer norm on the GPU against their float64 references, with the bounds
derived in delta_ref.py."""
import pytest
import torch

import delta_ref as R
from linear_rnn_sequence_gb300 import linattn as la

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("grad_q", "grad_k", "grad_v", "grad_beta", "grad_log_gate", "grad_S_in")


def on_gpu(x):
    return {n: t if t is None else t.cuda() for n, t in x.items()}


def gpu_forward(x, layout="bhnd", **kw):
    x = on_gpu(x)
    return la.forward_delta(x["q"], x["k"], x["v"], x["beta"], x["log_gate"], S_in=x["S_in"], layout=layout,
                            check_status=True, **kw)


def gpu_backward(x, dy, dS=None, layout="bhnd"):
    x = on_gpu(x)
    return la.backward_delta(x["q"], x["k"], x["v"], x["beta"], dy.cuda(), x["log_gate"], S_in=x["S_in"],
                             grad_S_out=None if dS is None else dS.cuda(), layout=layout, check_status=True)


def upstream(x, dtype, seed=9, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(x["v"].shape, generator=g).to(dtype)
    dS = None if x["S_in"] is None else scale * torch.randn(x["S_in"].shape, generator=g)
    return dy, dS


def check_forward(x, layout="bhnd"):
    y, S = gpu_forward(x, layout, return_state=True)
    yr, Sr = R.forward(x, layout)
    R.check(y, yr, "y")
    R.check(S, Sr, "S")


def check_backward(x, dtype, layout="bhnd"):
    dy, dS = upstream(x, dtype)
    got, want = gpu_backward(x, dy, dS, layout), R.backward(x, dy, dS, layout)
    for n, a, b in zip(NAMES, got, want):
        if n == "grad_S_in" and dS is None:
            assert a is None
        elif a is None:
            assert n == "grad_log_gate" and x["log_gate"] is None
        else:
            R.check(a, b, n, slack=R.log_gate_slack(x, dy, dS, want, layout) if n == "grad_log_gate" else 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_every_width(d, dv, dtype):
    x = R.inputs(1, 4, 2, 150, d, dv, dtype, state=True, seed=d + dv)
    check_forward(x)
    check_backward(x, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 333])
def test_lengths(N, dtype):
    x = R.inputs(2, 2, 1, N, 64, 128, dtype, state=N % 2 == 0, layout="bnhd", seed=N)
    check_forward(x, "bnhd")
    check_backward(x, dtype, "bnhd")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", [None, "any"])
@pytest.mark.parametrize("group", [1, 4])
def test_gates_and_shared_heads(gate, group, dtype):
    x = R.inputs(2, 4, 4 // group, 200, 128, 64, dtype, gate=gate, state=True, seed=group)
    check_forward(x)
    check_backward(x, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [1, 2])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("gate", [-9999.0, -1234.5, -60.0, -float("inf")])
def test_gates_that_all_but_close(gate, d, dv, group, dtype):
    """Among open gates a few that close as good as wholly: differences of running sums of logarithms that are
    thousands apart, whose last places still are the open gates."""
    for seed, N in ((0, 64), (2, 150)):
        x = R.inputs(1, 4, 4 // group, N, d, dv, dtype, state=seed == 0, seed=seed)
        g = torch.Generator().manual_seed(seed + 1)
        x["log_gate"][torch.rand(1, 4, N, generator=g) < 0.05] = gate
        check_forward(x)
        check_backward(x, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_keys_and_full_writes(dtype):
    # the same key again and again with b = 1: the hardest inverse of a block
    x = R.inputs(1, 2, 2, 140, 64, 64, dtype, gate=None, state=True, seed=4)
    x["k"][:] = x["k"][:, :, :1]
    x["beta"][:] = 1.0
    check_forward(x)
    check_backward(x, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_long_sequence(dtype, layout):
    x = R.inputs(1, 2, 1, 1000, 128, 128, dtype, layout=layout, seed=6)
    check_forward(x, layout)
    check_backward(x, dtype, layout)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("gate,N", [(None, 2500), ("open", 4000), ("any", 1900)])
def test_few_heads_and_many_tokens(d, dv, gate, N):
    """bf16 sequences long enough to be split over the SMs, from a given state.  Without gates the
    state is the one of two orders of the same sums (maps of the state, then the state): the bound
    is that of a sequence of N tokens all the same, sqrt(2 d) tokens being remembered."""
    x = R.inputs(1, 2, 1, N, d, dv, BF16, gate=gate, state=True, layout="bnhd", seed=N + d)
    check_forward(x, "bnhd")
    y, S = gpu_forward(x, "bnhd", return_state=True)
    y2, S2 = gpu_forward(x, "bnhd", return_state=True)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    check_backward(x, BF16, "bnhd")


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("B,H,Hk,N", [(3, 6, 2, 1800), (5, 6, 6, 610), (40, 8, 8, 40)])
def test_more_blocks_than_sms(d, dv, B, H, Hk, N):
    """Persistent CTAs of the gradients' products take several blocks each: of one value head, of three
    that share a key head, and of the ragged ends alone."""
    x = R.inputs(B, H, Hk, N, d, dv, BF16, gate="any" if N > 1000 else "open", state=H != Hk, seed=N + d + dv)
    check_backward(x, BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_sequence_in_parts(dtype):
    x = on_gpu(R.inputs(2, 2, 2, 300, 64, 64, dtype, state=True, seed=8))

    def part(a, b, S):
        c = {n: t[:, :, a:b].contiguous() for n, t in x.items() if n != "S_in"}
        return la.forward_delta(**c, S_in=S, return_state=True)

    y, S = la.forward_delta(**x, return_state=True)
    S1, ys = x["S_in"], []
    for a, b in ((0, 100), (100, 101), (101, 101), (101, 300)):
        y1, S1 = part(a, b, S1)
        ys.append(y1)
    # two summation orders of the same sums: twice the bound
    R.check(torch.cat(ys, 2), y.cpu(), "y", 2 * R.R_F32 + 2 * R.half_step(dtype))
    R.check(S1, S.cpu(), "S", 2 * R.R_F32)


def test_padding_leaves_the_state():
    x = R.inputs(1, 2, 2, 90, 64, 64, BF16, state=True, seed=11)
    x["beta"][:, :, 70:] = 0
    x["log_gate"][:, :, 70:] = 0
    _, S = gpu_forward(x, return_state=True)
    cut = {n: t if n == "S_in" else t[:, :, :70].contiguous() for n, t in x.items()}
    R.check(S, R.forward(cut)[1], "S")


def test_final_state_over_the_initial_one():
    x = R.inputs(1, 2, 2, 130, 64, 128, BF16, state=True, seed=12)
    want = gpu_forward(x, return_state=True)
    xg = on_gpu(x)
    S = xg["S_in"]
    y, S2 = la.forward_delta(**xg, S_out=S, return_state=True)
    assert S2 is S and torch.equal(S, want[1]) and torch.equal(y, want[0])


def test_no_tokens():
    x = on_gpu(R.inputs(1, 2, 1, 0, 64, 64, BF16, state=True))
    y, S = la.forward_delta(**x, return_state=True)
    assert y.shape == (1, 2, 0, 64) and torch.equal(S, x["S_in"])
    x0 = {**x, "S_in": None}
    assert not la.forward_delta(**x0, return_state=True)[1].any()
    dS = torch.randn_like(x["S_in"])
    got = la.backward_delta(x["q"], x["k"], x["v"], x["beta"], x["v"], x["log_gate"], S_in=x["S_in"], grad_S_out=dS)
    assert torch.equal(got[5], dS)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_same_bits_again(dtype):
    x = R.inputs(2, 4, 2, 260, 128, 128, dtype, state=True, seed=13)
    dy, dS = upstream(x, dtype)
    a, b = gpu_forward(x, return_state=True), gpu_forward(x, return_state=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    a, b = gpu_backward(x, dy, dS), gpu_backward(x, dy, dS)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_nothing_is_written_outside():
    """Outputs carved out of one buffer: what lies between them stays."""
    x = on_gpu(R.inputs(1, 2, 2, 77, 64, 64, BF16, state=True, seed=14))
    n = x["v"].numel()
    buf = torch.full((3 * n,), 7.0, dtype=BF16, device="cuda")
    y = buf[n:2 * n].view(x["v"].shape)
    sbuf = torch.full((3 * x["S_in"].numel(),), 7.0, device="cuda")
    m = x["S_in"].numel()
    S = sbuf[m:2 * m].view(x["S_in"].shape)
    la.forward_delta(**x, out=y, S_out=S, return_state=True)
    assert (buf[:n] == 7).all() and (buf[2 * n:] == 7).all() and (sbuf[:m] == 7).all() and (sbuf[2 * m:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,dv,group", [(32, 32, 1), (128, 128, 2), (64, 128, 1), (128, 32, 4)])
@pytest.mark.parametrize("gate", [None, "any"])
def test_single_steps_are_the_sequence(dtype, d, dv, group, gate):
    x = R.inputs(3, 4, 4 // group, 6, d, dv, dtype, gate=gate, state=True, seed=d)
    yr, Sr = R.forward(x)
    xg = on_gpu(x)
    S = xg["S_in"].clone()
    for t in range(6):
        y = la.decode_step_delta(*(xg[n][:, :, t].contiguous() for n in ("q", "k", "v", "beta")), S,
                                 None if gate is None else xg["log_gate"][:, :, t].contiguous())
        R.check(y, yr[:, :, t], f"y {t}")
    R.check(S, Sr, "S")


def test_step_into_another_state():
    x = on_gpu(R.inputs(2, 2, 2, 1, 64, 64, BF16, state=True, seed=15))
    args = [x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "beta")]
    S0, S1 = x["S_in"].clone(), torch.empty_like(x["S_in"])
    y1 = la.decode_step_delta(*args, S0, x["log_gate"][:, :, 0].contiguous(), S_out=S1)
    assert torch.equal(S0, x["S_in"])
    y0 = la.decode_step_delta(*args, S0, x["log_gate"][:, :, 0].contiguous())
    assert torch.equal(S0, S1) and torch.equal(y0, y1)


# ---- layer norm -----------------------------------------------------------------
# float32 sums of D values: mean and rstd are off by a few 2^-24 (a tree of sums) of the RMS of x,
# far below r = 1e-5; the column sums of `rows` values by 2^-24 sqrt(rows) or less
R_NORM = 1e-5


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 32), (700, 64), (1000, 128), (33, 100), (17, 127), (9, 256),
                                    (40, 511), (40, 512), (21, 1000), (6, 2048), (5, 4099), (4, 8192), (3, 16384),
                                    (2, 16383), (20011, 8)])
@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm(dtype, rows, D, affine):
    g = torch.Generator().manual_seed(D)
    x = (torch.randn(rows, D, generator=g) * 2 + torch.randn(rows, 1, generator=g)).to(dtype)
    dy = torch.randn(rows, D, generator=g).to(dtype)
    w, b = (1 + 0.3 * torch.randn(D, generator=g), torch.randn(D, generator=g)) if affine else (None, None)
    dev = [t if t is None else t.cuda() for t in (x, w, b)]
    y, mean, rstd = la.layer_norm(*dev, return_stats=True)
    yr, mr, rr = R.layer_norm(x, w, b)
    if D == 1:   # x - mean is exactly zero, and so is every gradient of x
        assert torch.equal(y.cpu().double(), torch.zeros_like(yr) if b is None else b.expand_as(yr).to(dtype).double())
    else:
        R.check(y, yr, "y", R_NORM)
    R.check(mean, mr, "mean", R_NORM)
    R.check(rstd, rr, "rstd", R_NORM)
    gx, gw, gb = la.layer_norm_backward(dy.cuda(), dev[0], mr.float().cuda(), rr.float().cuda(), dev[1], sums=True)
    gxr, gwr, gbr = R.layer_norm_backward(dy, x, mr.float(), rr.float(), w)
    # of the size of dy rstd, the terms it is the difference of
    scale = (dy.double() * rr[:, None]).square().mean().sqrt() / gxr.square().mean().sqrt().clamp_min(1e-30)
    if D > 2:
        R.check(gx, gxr, "grad_x", R_NORM * max(1.0, scale.item()))
    R.check(gw, gwr, "grad_weight", 4 * R_NORM)
    R.check(gb, gbr, "grad_bias", 4 * R_NORM)
    only = la.layer_norm_backward(dy.cuda(), dev[0], mr.float().cuda(), rr.float().cuda(), dev[1], sums=False)
    assert only[1] is None and torch.equal(only[0], gx)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,D", [(9001, 22), (40009, 31), (30001, 46), (20003, 65), (6007, 158), (5003, 333), (3001, 510),
                                    (777, 1062), (333, 2090), (100, 4431), (50, 6290), (20, 12290), (3, 16382)])
def test_layer_norm_of_rows_that_start_anywhere(dtype, rows, D):
    test_layer_norm(dtype, rows, D, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,D", [(90011, 64), (90011, 128), (45007, 256), (22511, 512), (7001, 768), (5003, 1024), (7001, 1536),
                                    (5003, 2048), (4001, 4096), (2003, 5120), (2003, 8192), (1901, 16384)])
def test_layer_norm_of_many_rows(dtype, rows, D):
    """Whole vectors, several steps of a CTA in both directions, two rows in flight where the rule has them, and a
    last step that is not full: sums and rows read ahead have to be those of their own step."""
    test_layer_norm(dtype, rows, D, True)


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_layer_norm_off_its_vectors(offset):
    """Even widths whose rows start 2, 4 or 8 bytes off: single values or pairs, in x, y, dy and dx alike."""
    for D in (96, 158):
        buf, out = torch.randn(2, 50 * D + offset, device="cuda").to(BF16)
        x, y = buf[offset:].view(50, D), out[offset:].view(50, D)
        got, mean, rstd = la.layer_norm(x, out=y, return_stats=True)
        want, mr, rr = R.layer_norm(x.cpu())
        assert got is y
        R.check(y, want, "y", R_NORM)
        gx, _, _ = la.layer_norm_backward(y, x, mean, rstd)
        gxr, _, _ = R.layer_norm_backward(y.cpu(), x.cpu(), mean.cpu(), rstd.cpu())
        # y lies almost along xh, so the gradient is a small difference of terms of the size of dy rstd
        scale = (y.cpu().double() * rr[:, None]).square().mean().sqrt() / gxr.square().mean().sqrt()
        R.check(gx, gxr, "grad_x", R_NORM * max(1.0, scale.item()))


def test_layer_norm_unaligned_rows_and_in_place():
    # rows that start 2 bytes off a 16-byte boundary, and y written over x
    buf = torch.randn(4 * 128 + 1, device="cuda").to(BF16)
    x = buf[1:].view(4, 128)
    yr, _, _ = R.layer_norm(x.cpu())
    R.check(la.layer_norm(x), yr, "y", R_NORM)
    z = x.clone()
    la.layer_norm(z, out=z)
    R.check(z, yr, "y", R_NORM)


def test_layer_norm_of_equal_values():
    x = torch.full((3, 96), 5.0, device="cuda")
    y, mean, rstd = la.layer_norm(x, return_stats=True)
    assert not y.any() and (mean == 5).all() and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))


def test_layer_norm_no_rows():
    x = torch.empty(0, 64, device="cuda")
    assert la.layer_norm(x).shape == (0, 64)
    s = torch.empty(0, device="cuda")
    gx, gw, gb = la.layer_norm_backward(x, x, s, s, torch.ones(64, device="cuda"))
    assert gx.shape == (0, 64) and not gw.any() and not gb.any()


# ---- together -------------------------------------------------------------------
def test_one_layer_and_its_gradients():
    """The delta rule, its norm, and the gradients back through both, as a training step runs them;
    against float64 autograd through both.  The values between the two are rounded to bf16 on the
    way (y, and dy): two half steps of their RMS on top of the bounds."""
    B, H, N, d, dv = 2, 4, 150, 64, 64
    x = R.inputs(B, H, 2, N, d, dv, BF16, layout="bnhd", seed=21)
    g = torch.Generator().manual_seed(22)
    w, b = 1 + 0.1 * torch.randn(dv, generator=g), 0.1 * torch.randn(dv, generator=g)
    do = torch.randn(B, N, H, dv, generator=g).to(BF16)
    xg = on_gpu(x)
    y = la.forward_delta(**xg, layout="bnhd")
    o, mean, rstd = la.layer_norm(y, w.cuda(), b.cuda(), return_stats=True)
    gy, gw, gb = la.layer_norm_backward(do.cuda(), y, mean, rstd, w.cuda())
    grads = la.backward_delta(xg["q"], xg["k"], xg["v"], xg["beta"], gy, xg["log_gate"], layout="bnhd")

    leaves = {n: t if t is None else t.double().requires_grad_() for n, t in x.items()}
    wl, bl = w.double().requires_grad_(), b.double().requires_grad_()
    yr, _ = R.forward(leaves, "bnhd")
    outr, _, _ = R.layer_norm(yr, wl, bl)
    names = ["q", "k", "v", "beta", "log_gate"]
    want = torch.autograd.grad((outr * do.double()).sum(), [leaves[n] for n in names] + [wl, bl])
    for n, a, r in zip(names + ["weight", "bias"], [*grads[:5], gw, gb], want):
        err = (a.cpu().double() - r).norm() / r.norm()
        assert err <= 4 * R.half_step(BF16), (n, err.item())
    assert (o.cpu().double() - outr).norm() / outr.norm() <= 3 * R.half_step(BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_and_on_another_stream(dtype):
    x = on_gpu(R.inputs(1, 4, 2, 200, 64, 64, dtype, state=True, seed=31))
    dy = torch.randn_like(x["v"])
    w = torch.rand(64, device="cuda")

    def step():
        y, S = la.forward_delta(**x, return_state=True)
        o, mean, rstd = la.layer_norm(y, w, return_stats=True)
        gy, gw, gb = la.layer_norm_backward(dy, y, mean, rstd, w)
        grads = la.backward_delta(x["q"], x["k"], x["v"], x["beta"], gy, x["log_gate"], S_in=x["S_in"])
        st = la.decode_step_delta(x["q"][:, :, 0].contiguous(), x["k"][:, :, 0].contiguous(),
                                  x["v"][:, :, 0].contiguous(), x["beta"][:, :, 0].contiguous(), S)
        return [y, S, o, gy, gw, gb, *grads, st]

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x["v"].mul_(2)
    want2 = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want2))
    assert not torch.equal(want[0], want2[0])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = la.forward_delta(**x, stream=s)
    n = la.layer_norm(y, w, stream=s)
    s.synchronize()
    assert torch.equal(y, want2[0]) and torch.equal(n, want2[2])


# ---- run-time failure, without a GPU fault --------------------------------------
@pytest.mark.parametrize("what,B,H,N", [("forward", 1, 4, 200), ("forward", 1, 2, 4000), ("forward", 40, 4, 130),
                                         ("backward", 1, 4, 200), ("backward", 1, 2, 4000)])
def test_a_dropped_copy_times_out_and_the_next_call_is_right(what, B, H, N):
    """The test hook announces one work item's first tile copy and never issues it: every wait on it
    runs out, the call records LA_ERR_TIMEOUT, and the context stays usable."""
    x = on_gpu(R.inputs(B, H, H, N, 64, 64, BF16, seed=41))
    dy = torch.randn_like(x["v"])

    def call():
        if what == "forward":
            return (la.forward_delta(**x, check_status=True),)
        return la.backward_delta(x["q"], x["k"], x["v"], x["beta"], dy, x["log_gate"], check_status=True)[:5]

    want = call()
    try:
        la.set_fault(drop_load_item=1, wait_limit_ns=5_000_000)
        with pytest.raises(la.LinAttnError) as e:
            call()
        assert e.value.status == la.LA_ERR_TIMEOUT
    finally:
        la.set_fault(-1, 0)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.mark.parametrize("dtype,d,N", [(F32, 64, 70), (F32, 64, 0), (BF16, 32, 70), (BF16, 64, 5), (BF16, 64, 0)])
def test_status_of_a_call_that_needs_no_workspace(dtype, d, N):
    """Such a call leaves a given workspace alone: what an earlier one recorded there is not its status."""
    x = on_gpu(R.inputs(1, 2, 2, N, d, d, dtype, state=True, seed=7))
    marked = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    y = la.forward_delta(**x, workspace=marked, check_status=True)
    assert torch.equal(y, la.forward_delta(**x)) and (marked == 255).all()
    if N == 0:   # the gradients need none either
        la.backward_delta(x["q"], x["k"], x["v"], x["beta"], x["v"], x["log_gate"], workspace=marked, check_status=True)
    if dtype == F32 and N:   # nor do the causal calls of this dtype
        gamma = torch.full((2,), 0.9, device="cuda")
        la.forward_causal(x["q"], x["k"], x["v"], workspace=marked, check_status=True)
        la.forward_causal_decay(x["q"], x["k"], x["v"], gamma, workspace=marked, check_status=True)


@pytest.mark.parametrize("N", [40, 64, 65, 129, 200, 333, 1000, 4000])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128)])
def test_late_output_warps(N, d, dv):
    """The test hook starts the warps that read a block's scores and write y a good deal later than the
    other blocks' inverses take: nothing overtakes them."""
    x = on_gpu(R.inputs(2, 2, 1, N, d, dv, BF16, state=True, seed=N + d))
    want = la.forward_delta(**x, return_state=True, check_status=True)
    try:
        la.set_stall(300_000)
        got = la.forward_delta(**x, return_state=True, check_status=True)
    finally:
        la.set_stall(0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- what the binding refuses ----------------------------------------------------
def test_binding_refuses():
    x = on_gpu(R.inputs(1, 4, 2, 40, 64, 64, BF16, state=True))
    bad = [dict(k=x["k"].float()), dict(v=x["v"][:, :, :39].contiguous()), dict(beta=x["beta"].double()),
           dict(beta=x["beta"][:, :2].contiguous()), dict(log_gate=x["log_gate"].bfloat16()),
           dict(S_in=x["S_in"].bfloat16()), dict(S_in=x["S_in"][:, :1].contiguous()), dict(layout="nbhd"),
           dict(q=x["q"].transpose(2, 3)), dict(v=x["v"].transpose(1, 2).contiguous().transpose(1, 2)),
           dict(out=x["v"].float()), dict(beta=x["beta"].cpu())]
    for change in bad:
        with pytest.raises(ValueError):
            la.forward_delta(**{**x, **change})
    with pytest.raises(TypeError):
        la.forward_delta(**{n: t.half() if n in "qkv" else t for n, t in x.items()})
    with pytest.raises(la.LinAttnError) as e:   # three heads of v to two of q
        la.forward_delta(x["q"], x["k"], x["v"][:, :3].contiguous(), x["beta"][:, :3].contiguous())
    assert e.value.status == la.LA_ERR_INVALID_ARG
    with pytest.raises(la.LinAttnError) as e:   # over one of its inputs
        la.forward_delta(**x, out=x["v"])
    assert e.value.status == la.LA_ERR_INVALID_ARG
    with pytest.raises(la.LinAttnError) as e:   # rows that start 2 bytes off a 16-byte boundary
        buf = torch.zeros(x["v"].numel() + 1, dtype=BF16, device="cuda")
        la.forward_delta(**x, out=buf[1:].view(x["v"].shape))
    assert e.value.status == la.LA_ERR_INVALID_ARG
    with pytest.raises(la.LinAttnError) as e:
        la.backward_delta(x["q"], x["k"], x["v"], x["beta"], x["v"], x["log_gate"],
                          workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == la.LA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        la.layer_norm(torch.zeros(3, 8, device="cuda"), torch.zeros(7, device="cuda"))
    with pytest.raises(la.LinAttnError):
        la.layer_norm(torch.zeros(2, 16385, device="cuda"))


def test_layer_norm_of_a_scalar_is_refused():
    x = torch.zeros((), device="cuda")
    with pytest.raises(ValueError):
        la.layer_norm(x)
    with pytest.raises(ValueError):
        la.layer_norm_backward(x, x, x, x)


@pytest.mark.parametrize("dtype,N", [(BF16, 200), (BF16, 20), (F32, 100)])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v", "beta", "log_gate"])
def test_what_is_not_finite_reaches_no_earlier_token(what, value, d, dv, dtype, N):
    """One such value in one head: y and the state are not finite where the recurrence's are not, and nowhere
    else; all else keeps its bits (and, where a gate that is no number sends its block down the general path of
    the gates, its bound)."""
    for t in (0, 1, 17, 30, 62, 63, 64, 100, 199):
        if t >= N:
            break
        x = R.inputs(1, 3, 3, N, d, dv, dtype, state=t % 2 == 1, seed=t)
        clean = gpu_forward(x, return_state=True)
        x[what] = x[what].clone()
        x[what][(0, 1, t, 5) if what in "qkv" else (0, 1, t)] = value
        got, want = gpu_forward(x, return_state=True), R.forward(x)
        for g, w, c in zip(got, want, clean):
            ok = torch.isfinite(w)
            assert torch.equal(torch.isfinite(g).cpu(), ok), (t, what)
            if what != "log_gate":
                assert torch.equal(g.cpu()[ok], c.cpu()[ok]), (t, what)
            elif ok.any():
                R.check(g.cpu()[ok], w[ok], what)


@pytest.mark.parametrize("B,H,N,t", [(1, 2, 2500, 1400), (40, 5, 100, 70)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_what_is_not_finite_in_long_sequences_and_many_heads(what, B, H, N, t):
    """The same for sequences split into segments, and for more heads than SMs; with the final state written
    over the initial one, and replayed from a captured graph."""
    x = R.inputs(B, H, H, N, 64, 64, BF16, state=True, seed=N)
    clean = gpu_forward(x, return_state=True)
    bad = {**x, what: x[what].clone()}
    bad[what][B - 1, 1, t, 5] = float("nan")
    bad[what][B - 1, 0, N - 1, 7] = float("inf")
    want = R.forward(bad)

    def check(got):
        for g, w, c in zip(got, want, clean):
            ok = torch.isfinite(w)
            assert not ok.all() and torch.equal(torch.isfinite(g).cpu(), ok)
            assert torch.equal(g.cpu()[ok], c.cpu()[ok])

    check(gpu_forward(bad, return_state=True))
    xg = on_gpu(bad)
    y, _ = la.forward_delta(**xg, S_out=xg["S_in"], return_state=True)
    check((y, xg["S_in"]))
    xg = on_gpu(x)
    la.forward_delta(**xg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = la.forward_delta(**xg, return_state=True)
    xg[what].copy_(bad[what])
    graph.replay()
    check(got)
    xg[what].copy_(x[what])
    graph.replay()
    assert all(torch.equal(g, c) for g, c in zip(got, clean))


@pytest.mark.parametrize("N", [40, 200])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("scale", [30.0, 1e4, 1e15, 1e30])
def test_overflow_reaches_no_earlier_token(scale, d, dv, N):
    """Keys and values of any size from token t on, as what lies behind a prompt's end may be: the tokens
    before it keep their bits."""
    for t in (3, 21, 37, 70, 150):
        if t >= N:
            break
        x = R.inputs(2, 2, 1, N, d, dv, BF16, state=True, seed=t)
        clean = gpu_forward(x)
        x["k"][:, :, t:] *= scale
        x["v"][:, :, t:] *= scale
        y = gpu_forward(x)
        assert torch.equal(y[:, :, :t], clean[:, :, :t]), t


def test_values_behind_the_inputs_are_not_read():
    """NaN in memory on either side of every input."""
    def guarded(t):
        if t is None:
            return None
        buf = torch.full((t.numel() + 2 * 4096,), float("nan"), dtype=t.dtype, device="cuda")
        view = buf[4096:4096 + t.numel()].view(t.shape)
        view.copy_(t)
        return view

    for dtype in (BF16, F32):
        for N in (1, 70, 300):
            x = on_gpu(R.inputs(2, 2, 1, N, 64, 64, dtype, state=True, seed=N))
            g = {n: guarded(t) for n, t in x.items()}
            dy = torch.randn_like(x["v"])
            assert all(torch.equal(a, b) for a, b in zip(la.forward_delta(**g, return_state=True),
                                                         la.forward_delta(**x, return_state=True)))
            args = ("q", "k", "v", "beta")
            a = la.backward_delta(*(g[n] for n in args), guarded(dy), g["log_gate"], S_in=g["S_in"])
            b = la.backward_delta(*(x[n] for n in args), dy, x["log_gate"], S_in=x["S_in"])
            assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_two_calls_in_flight_on_two_streams():
    xs = [on_gpu(R.inputs(1, 4, 4, 700, 64, 64, BF16, seed=50 + i)) for i in range(2)]
    dys = [torch.randn_like(x["v"]) for x in xs]

    def call(i, stream=None):
        x = xs[i]
        return [la.forward_delta(**x, stream=stream),
                *la.backward_delta(x["q"], x["k"], x["v"], x["beta"], dys[i], x["log_gate"], stream=stream)[:5]]

    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [call(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
