"""Retention without a GPU: refusals of the C entry points, before anything is launched; the reference against a
recurrence."""
import ctypes

import pytest
import torch

import retention_ref as R
from linear_rnn_sequence_gb300 import linattn as la

AT = {n: (i + 1) << 26 for i, n in enumerate(("q", "k", "v", "y", "dy", "gamma", "S_in", "S_out", "gq", "gk", "gv", "dS", "ws"))}
BASE = dict(B=2, H=2, N=300, d=64, dv=64, dt=1, layout=0)


def sizes(a):
    return [a[n] for n in ("B", "H", "N", "d", "dv", "dt")]


def call(which, **kw):
    a = {**AT, **BASE, **kw}
    L = la.lib()
    p = {n: None if a[n] is None else ctypes.c_void_p(a[n]) for n in AT}
    if which == "step":
        return L.la_decode_step_retention(p["q"], p["k"], p["v"], p["y"], p["gamma"], p["S_in"], p["S_out"], a["B"], a["H"],
                                          a["d"], a["dv"], a["dt"], None)
    wsb = a.get("wsb", 1 << 25)
    if which == "forward":
        return L.la_forward_retention(p["q"], p["k"], p["v"], p["y"], p["gamma"], *sizes(a), a["layout"], p["S_in"],
                                      p["S_out"], p["ws"], wsb, None)
    return L.la_backward_retention(p["q"], p["k"], p["v"], p["dy"], p["gamma"], p["gq"], p["gk"], p["gv"], *sizes(a),
                                   a["layout"], p["S_in"], p["dS"], p["S_out"], p["ws"], wsb, None)


COMMON = [(dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(gamma=None), 1), (dict(q=AT["q"] + 4), 1),
          (dict(gamma=AT["gamma"] + 2), 1), (dict(B=0), 1), (dict(H=0), 1), (dict(d=48), 2), (dict(dv=256), 2), (dict(dt=3), 2),
          (dict(B=1 << 16, H=1 << 15), 1)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(y=None), 1), (dict(y=AT["y"] + 8), 1), (dict(y=AT["q"]), 1), (dict(y=AT["gamma"] - 64), 1), (dict(y=AT["S_in"]), 1),
    (dict(S_out=AT["y"]), 1), (dict(S_out=AT["S_in"] + 16), 1), (dict(S_in=AT["S_in"] + 4), 1), (dict(layout=2), 2),
    (dict(N=-1), 1), (dict(N=1 << 30), 1), (dict(ws=AT["v"]), 1)])
def test_forward_refuses(kw, status):
    assert call("forward", **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dy=None), 1), (dict(gq=None), 1), (dict(gv=AT["gv"] + 2), 1), (dict(gq=AT["gk"]), 1), (dict(gk=AT["dy"]), 1),
    (dict(S_out=AT["S_in"]), 1), (dict(S_out=AT["dS"]), 1), (dict(gv=AT["ws"]), 1), (dict(layout=-1), 2), (dict(N=-1), 1)])
def test_backward_refuses(kw, status):
    assert call("backward", **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(y=None), 1), (dict(S_in=None), 1), (dict(S_out=None), 1), (dict(S_out=AT["S_in"] + 16), 1), (dict(y=AT["S_out"]), 1),
    (dict(y=AT["k"]), 1)])
def test_step_refuses(kw, status):
    assert call("step", **kw) == status


@pytest.mark.parametrize("dt", [0, 1])
def test_workspace(dt):
    L = la.lib()
    for f, which in ((L.la_retention_workspace_bytes, "forward"), (L.la_retention_backward_workspace_bytes, "backward")):
        need = f(2, 2, 300, 64, 64, dt)
        assert need >= 256
        assert call(which, dt=dt, wsb=need - 1) == la.LA_ERR_WORKSPACE
        assert call(which, dt=dt, ws=None) == la.LA_ERR_WORKSPACE
        assert call(which, dt=dt, ws=AT["ws"] + 64) == la.LA_ERR_WORKSPACE
        for bad in ((0, 2, 300, 64, 64, dt), (2, 2, 0, 64, 64, dt), (2, 2, -1, 64, 64, dt), (2, 2, 300, 63, 64, dt), (2, 2, 300, 64, 64, 9)):
            assert f(*bad) == 0


def test_binding_refuses_cpu_tensors():
    q, g = torch.zeros(1, 2, 4, 32), torch.ones(2)
    with pytest.raises(ValueError):
        la.forward_retention(q, q, q, g)
    with pytest.raises(ValueError):
        la.backward_retention(q, q, q, g, q)
    with pytest.raises(ValueError):
        la.decode_step_retention(q[:, :, 0], q[:, :, 0], q[:, :, 0], g, torch.zeros(1, 2, 32, 32))


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_reference_against_the_recurrence(layout):
    x = R.inputs(2, 3, 23, 32, 64, torch.float32, layout, gamma=[0.0, 0.7, 1.0])
    y, _, S, _ = R.forward(x, layout)
    q, k, v = (R.heads(x[n], layout).double() for n in "qkv")
    s = x["S"].double()
    for t in range(23):
        s = x["gamma"].double()[:, None, None] * s + k[:, :, t, :, None] * v[:, :, t, None]
        assert torch.allclose(R.heads(y, layout)[:, :, t], (s * q[:, :, t, :, None]).sum(-2), rtol=1e-12, atol=1e-12)
    assert torch.allclose(S, s, rtol=1e-12, atol=1e-12)
