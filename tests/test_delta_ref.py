"""The float64 references of the gated delta rule and of layer norm against differences and against
closed forms, and the host-side refusals of their entry points.  No GPU."""
import ctypes

import pytest
import torch

import delta_ref as R
from linear_rnn_sequence_gb300 import linattn as la


@pytest.mark.parametrize("gate", [None, "open", "any"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_gradients_match_autograd_and_differences(gate, layout):
    x = R.inputs(2, 4, 2, 7, 6, 5, gate=gate, state=True, layout=layout, seed=3)
    x = {n: t if t is None else t.double() for n, t in x.items()}
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(x["v"].shape, generator=g).double()
    dS = torch.randn(x["S_in"].shape, generator=g).double()

    def loss(z):
        y, S = R.forward(z, layout)
        return (y * dy).sum() + (S * dS).sum()

    got = R.backward(x, dy, dS, layout)
    names = ["q", "k", "v", "beta", "log_gate", "S_in"]
    leaves = {n: t if t is None else t.clone().requires_grad_() for n, t in x.items()}
    auto = torch.autograd.grad(loss(leaves), [leaves[n] for n in names if leaves[n] is not None])
    auto = iter(auto)
    for n, have in zip(names, got):
        if x[n] is None:
            assert have is None
            continue
        want = next(auto)
        assert torch.allclose(have, torch.nan_to_num(want), rtol=1e-9, atol=1e-10), n
        # central differences along one direction that leaves closed gates closed
        way = torch.randn(x[n].shape, generator=g).double()
        way = torch.where(torch.isfinite(x[n]), way, torch.zeros_like(way))
        h = 1e-5
        up, down = ({**x, n: torch.where(torch.isfinite(x[n]), x[n] + s * h * way, x[n])} for s in (1, -1))
        num = (loss(up) - loss(down)) / (2 * h)
        assert torch.allclose((have * way).sum(), num, rtol=1e-6, atol=1e-7), n


def test_recurrence_is_the_matrix_form():
    x = R.inputs(1, 2, 2, 5, 4, 3, state=True, seed=1)
    S = x["S_in"].double()
    for t in range(5):
        k, v = x["k"][:, :, t].double(), x["v"][:, :, t].double()
        b, a = x["beta"][:, :, t].double()[..., None, None], x["log_gate"][:, :, t].double().exp()[..., None, None]
        S = a * (S - b * k[..., None] * (k[..., None, :] @ S)) + b * k[..., None] * v[..., None, :]
    assert torch.allclose(R.forward(x)[1], S, rtol=1e-12)


def test_a_full_write_is_read_back():
    # b = 1 and a unit key: the value just stored is what that key reads
    x = R.inputs(1, 1, 1, 9, 8, 8, gate="open", seed=2)
    x["k"] = torch.nn.functional.normalize(x["k"].double(), dim=-1)
    x["q"], x["beta"] = x["k"], torch.ones(1, 1, 9)
    assert torch.allclose(R.forward(x)[0], x["v"].double(), atol=1e-12)


def test_layer_norm_gradients_match_autograd():
    g = torch.Generator().manual_seed(0)
    x, w, b, dy = (torch.randn(*s, generator=g).double() for s in ((3, 5, 11), (11,), (11,), (3, 5, 11)))
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    want = torch.autograd.grad((R.layer_norm(*leaves)[0] * dy).sum(), leaves)
    _, mean, rstd = R.layer_norm(x, w, b)
    for have, w_ in zip(R.layer_norm_backward(dy, x, mean, rstd, w), want):
        assert torch.allclose(have, w_, rtol=1e-10, atol=1e-12)


# ---- refusals: fake addresses, rejected before anything is dereferenced ---------
def at(i, off=0):
    return ctypes.c_void_p((1 << 20) + i * (1 << 28) + off)


def _forward(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), y=at(3), beta=at(4), lg=at(5), B=1, H=2, Hk=1, N=8, d=64, dv=64, dt=1,
             layout=0, S_in=None, S_out=None, ws=at(8), wsb=1 << 40)
    a.update(kw)
    return la.lib().la_forward_delta(*(a[n] for n in ("q", "k", "v", "y", "beta", "lg", "B", "H", "Hk", "N", "d",
                                                      "dv", "dt", "layout", "S_in", "S_out", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,expected", [
    (dict(q=None), la.LA_ERR_INVALID_ARG), (dict(k=None), la.LA_ERR_INVALID_ARG),
    (dict(v=None), la.LA_ERR_INVALID_ARG), (dict(y=None), la.LA_ERR_INVALID_ARG),
    (dict(beta=None), la.LA_ERR_INVALID_ARG),
    (dict(q=at(0, 8)), la.LA_ERR_INVALID_ARG), (dict(y=at(3, 2)), la.LA_ERR_INVALID_ARG),
    (dict(beta=at(4, 2)), la.LA_ERR_INVALID_ARG), (dict(lg=at(5, 1)), la.LA_ERR_INVALID_ARG),
    (dict(S_in=at(6, 4)), la.LA_ERR_INVALID_ARG), (dict(S_out=at(6, 4)), la.LA_ERR_INVALID_ARG),
    (dict(d=48), la.LA_ERR_UNSUPPORTED), (dict(dv=256), la.LA_ERR_UNSUPPORTED),
    (dict(dt=2), la.LA_ERR_UNSUPPORTED), (dict(layout=2), la.LA_ERR_UNSUPPORTED),
    (dict(layout=-1), la.LA_ERR_UNSUPPORTED),
    (dict(H=3, Hk=2), la.LA_ERR_INVALID_ARG), (dict(Hk=0), la.LA_ERR_INVALID_ARG),
    (dict(H=1, Hk=2), la.LA_ERR_INVALID_ARG),
    (dict(B=0), la.LA_ERR_INVALID_ARG), (dict(N=-1), la.LA_ERR_INVALID_ARG),
    (dict(B=1 << 14, H=1 << 10, N=1 << 10), la.LA_ERR_INVALID_ARG),
    (dict(B=1 << 30, H=1 << 30, N=1 << 30), la.LA_ERR_INVALID_ARG),
    (dict(B=1 << 19, H=1, N=1), la.LA_ERR_INVALID_ARG),                 # the state is too large
    (dict(y=at(0)), la.LA_ERR_INVALID_ARG), (dict(y=at(2)), la.LA_ERR_INVALID_ARG),
    (dict(y=at(4)), la.LA_ERR_INVALID_ARG), (dict(y=at(5)), la.LA_ERR_INVALID_ARG),
    (dict(S_in=at(3)), la.LA_ERR_INVALID_ARG), (dict(S_out=at(3)), la.LA_ERR_INVALID_ARG),
    (dict(S_out=at(1)), la.LA_ERR_INVALID_ARG),
    (dict(S_in=at(6), S_out=at(6, 64)), la.LA_ERR_INVALID_ARG),         # overlap, not the same
])
def test_forward_refuses(kw, expected):
    assert _forward(**kw) == expected


def _backward(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), dy=at(3), beta=at(4), lg=at(5), gq=at(6), gk=at(7), gv=at(8), gb=at(9),
             gl=at(10), B=1, H=2, Hk=1, N=8, d=64, dv=64, dt=1, layout=0, S_in=None, gSo=None, gSi=None,
             ws=at(14), wsb=1 << 30)
    a.update(kw)
    return la.lib().la_backward_delta(*(a[n] for n in ("q", "k", "v", "dy", "beta", "lg", "gq", "gk", "gv", "gb",
                                                       "gl", "B", "H", "Hk", "N", "d", "dv", "dt", "layout", "S_in",
                                                       "gSo", "gSi", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,expected", [
    *[({n: None}, la.LA_ERR_INVALID_ARG) for n in ("q", "k", "v", "dy", "beta", "gq", "gk", "gv", "gb", "gl", "lg")],
    *[({n: at(20, 4)}, la.LA_ERR_INVALID_ARG) for n in ("dy", "gq", "gk", "gv", "S_in", "gSo", "gSi")],
    (dict(gb=at(9, 2)), la.LA_ERR_INVALID_ARG),
    (dict(ws=None), la.LA_ERR_WORKSPACE), (dict(wsb=1 << 10), la.LA_ERR_WORKSPACE),
    (dict(ws=at(14, 16)), la.LA_ERR_WORKSPACE),
    (dict(gq=at(0)), la.LA_ERR_INVALID_ARG), (dict(gk=at(6)), la.LA_ERR_INVALID_ARG),
    (dict(gv=at(3)), la.LA_ERR_INVALID_ARG), (dict(gb=at(4)), la.LA_ERR_INVALID_ARG),
    (dict(gSi=at(11), S_in=at(11)), la.LA_ERR_INVALID_ARG), (dict(gSi=at(14)), la.LA_ERR_INVALID_ARG),
    (dict(gSi=at(11), gSo=at(11)), la.LA_ERR_INVALID_ARG),
    (dict(d=16), la.LA_ERR_UNSUPPORTED), (dict(H=5, Hk=2), la.LA_ERR_INVALID_ARG),
])
def test_backward_refuses(kw, expected):
    assert _backward(**kw) == expected


def _step(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), y=at(3), beta=at(4), lg=at(5), S_in=at(6), S_out=at(6), B=1, H=2, Hk=1, d=64,
             dv=64, dt=1)
    a.update(kw)
    return la.lib().la_decode_step_delta(*(a[n] for n in ("q", "k", "v", "y", "beta", "lg", "S_in", "S_out", "B", "H",
                                                          "Hk", "d", "dv", "dt")), None)


@pytest.mark.parametrize("kw,expected", [
    *[({n: None}, la.LA_ERR_INVALID_ARG) for n in ("q", "k", "v", "y", "beta", "S_in", "S_out")],
    *[({n: at(20, 4)}, la.LA_ERR_INVALID_ARG) for n in ("q", "k", "v", "y", "S_in", "S_out")],
    (dict(S_out=at(6, 64)), la.LA_ERR_INVALID_ARG), (dict(y=at(6)), la.LA_ERR_INVALID_ARG),
    (dict(S_out=at(0), S_in=at(7)), la.LA_ERR_INVALID_ARG),
    (dict(d=65), la.LA_ERR_UNSUPPORTED), (dict(dt=9), la.LA_ERR_UNSUPPORTED),
    (dict(H=3, Hk=2), la.LA_ERR_INVALID_ARG), (dict(B=0), la.LA_ERR_INVALID_ARG),
])
def test_step_refuses(kw, expected):
    assert _step(**kw) == expected


def _norm(**kw):
    a = dict(x=at(0), y=at(1), w=at(2), b=at(3), mean=at(4), rstd=at(5), rows=7, D=100, dt=1, eps=1e-5)
    a.update(kw)
    return la.lib().la_layer_norm(*(a[n] for n in ("x", "y", "w", "b", "mean", "rstd", "rows", "D", "dt", "eps")), None)


@pytest.mark.parametrize("kw,expected", [
    (dict(x=None), la.LA_ERR_INVALID_ARG), (dict(y=None), la.LA_ERR_INVALID_ARG),
    (dict(mean=None), la.LA_ERR_INVALID_ARG), (dict(rstd=None), la.LA_ERR_INVALID_ARG),
    (dict(x=at(0, 1)), la.LA_ERR_INVALID_ARG), (dict(w=at(2, 2)), la.LA_ERR_INVALID_ARG),
    (dict(dt=0, y=at(1, 2)), la.LA_ERR_INVALID_ARG),
    (dict(rows=-1), la.LA_ERR_INVALID_ARG), (dict(D=0), la.LA_ERR_INVALID_ARG),
    (dict(D=16385), la.LA_ERR_UNSUPPORTED), (dict(dt=5), la.LA_ERR_UNSUPPORTED),
    (dict(eps=0.0), la.LA_ERR_INVALID_ARG), (dict(eps=float("nan")), la.LA_ERR_INVALID_ARG),
    (dict(rows=1 << 62, D=16384), la.LA_ERR_INVALID_ARG),
    (dict(y=at(0, 2)), la.LA_ERR_INVALID_ARG), (dict(mean=at(0)), la.LA_ERR_INVALID_ARG),
    (dict(rstd=at(4)), la.LA_ERR_INVALID_ARG), (dict(y=at(0), mean=at(0)), la.LA_ERR_INVALID_ARG),
    (dict(y=at(2)), la.LA_ERR_INVALID_ARG),
    (dict(rows=0), la.LA_OK),
])
def test_layer_norm_refuses(kw, expected):
    assert _norm(**kw) == expected


def _norm_backward(**kw):
    a = dict(dy=at(0), x=at(1), mean=at(2), rstd=at(3), w=at(4), gx=at(5), gw=at(6), gb=at(7), rows=7, D=100, dt=1,
             ws=at(8), wsb=1 << 28)
    a.update(kw)
    return la.lib().la_layer_norm_backward(*(a[n] for n in ("dy", "x", "mean", "rstd", "w", "gx", "gw", "gb", "rows",
                                                            "D", "dt", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,expected", [
    *[({n: None}, la.LA_ERR_INVALID_ARG) for n in ("dy", "x", "mean", "rstd", "gx")],
    (dict(ws=None), la.LA_ERR_WORKSPACE), (dict(wsb=300), la.LA_ERR_WORKSPACE),
    (dict(D=20000), la.LA_ERR_UNSUPPORTED), (dict(rows=-2), la.LA_ERR_INVALID_ARG),
    (dict(gx=at(0, 2)), la.LA_ERR_INVALID_ARG), (dict(gw=at(1)), la.LA_ERR_INVALID_ARG),
    (dict(gw=at(7)), la.LA_ERR_INVALID_ARG), (dict(gx=at(1), gw=at(1)), la.LA_ERR_INVALID_ARG),
    (dict(gb=at(8)), la.LA_ERR_INVALID_ARG), (dict(mean=at(2, 2)), la.LA_ERR_INVALID_ARG),
])
def test_layer_norm_backward_refuses(kw, expected):
    assert _norm_backward(**kw) == expected


def test_workspace_sizes():
    L = la.lib()
    assert L.la_delta_backward_workspace_bytes(1, 2, 1, 0, 64, 64, 1) == 0
    assert L.la_delta_backward_workspace_bytes(1, 3, 2, 8, 64, 64, 1) == 0
    assert L.la_delta_backward_workspace_bytes(1, 2, 1, 8, 64, 64, 1) > 256
    assert L.la_delta_workspace_bytes(1, 3, 2, 8, 64, 64, 1) == 0
    assert L.la_layer_norm_backward_workspace_bytes(0, 64, 1) == 0
    assert L.la_layer_norm_backward_workspace_bytes(5, 64, 1) > 256


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = R.inputs(1, 2, 1, 3, 32, 32)
    with pytest.raises(ValueError):
        la.forward_delta(x["q"], x["k"], x["v"], x["beta"])
    with pytest.raises(ValueError):
        la.layer_norm(torch.zeros(3, 4))
