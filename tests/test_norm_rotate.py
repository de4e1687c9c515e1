"""Norm and rotation of queries and keys without a GPU: refusals of the C entry points, before anything is launched."""
import ctypes

import pytest

from linear_rnn_sequence_gb300 import linattn as la

AT = {n: (i + 1) << 28 for i, n in enumerate(("q", "k", "gq", "gk", "yq", "yk", "wq", "wk", "freq", "pos", "dwq", "dwk", "ws"))}
BASE = dict(B=2, Hq=4, Hk=2, N=8, d=64, dt=1, layout=0, norm=1, eps=1e-6, r=32, pairs=0, pstride=8, strides=None, wsb=1 << 24)


def address(v):
    return None if v is None else ctypes.c_void_p(v)


def call(back=False, **kw):
    a = {**AT, **BASE, **kw}
    st = None if a["strides"] is None else (ctypes.c_longlong * len(a["strides"]))(*a["strides"])
    bufs = ("q", "k", "gq", "gk", "yq", "yk") if back else ("q", "k", "yq", "yk")
    common = [*(address(a[n]) for n in bufs), st, *(a[n] for n in ("B", "Hq", "Hk", "N", "d", "dt", "layout", "norm", "eps")),
              *(address(a[n]) for n in ("wq", "wk", "freq")), a["r"], a["pairs"], address(a["pos"]), a["pstride"]]
    if not back:
        return la.lib().la_norm_rotate(*common, None)
    return la.lib().la_norm_rotate_backward(*common, address(a["dwq"]), address(a["dwk"]), address(a["ws"]), a["wsb"], None)


# as parts of one buffer: 8 heads of 64 in a token, q the first four, k the next two
FUSED = [8 * 8 * 64, 64, 8 * 64]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(yq=None), 1), (dict(yk=None), 1), (dict(freq=None), 1),
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(N=-1), 1), (dict(Hq=65535, Hk=1), 1), (dict(B=1 << 20, N=1 << 12), 1),
    (dict(d=63), 2), (dict(d=0), 2), (dict(d=258), 2), (dict(dt=5), 2), (dict(layout=2), 2), (dict(norm=3), 2), (dict(pairs=2), 2),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(r=33), 1), (dict(r=-1), 1), (dict(pstride=-1), 1), (dict(pstride=1 << 61), 1),
    (dict(q=AT["q"] + 1), 1), (dict(yk=AT["yk"] + 1), 1), (dict(wq=AT["wq"] + 2), 1), (dict(freq=AT["freq"] + 4), 1),
    (dict(pos=AT["pos"] + 4), 1),
    (dict(yq=AT["q"] + 64), 1), (dict(yq=AT["k"]), 1), (dict(yk=AT["q"]), 1), (dict(yq=AT["yk"]), 1), (dict(yq=AT["wk"]), 1),
    (dict(yk=AT["freq"] - 256), 1), (dict(yk=AT["pos"]), 1),
])
def test_refusals(kw, status, back):
    assert call(back, **kw) == status


def strided(back, **over):
    names = ("q", "k", "gq", "gk", "yq", "yk") if back else ("q", "k", "yq", "yk")
    flat = []
    for n in names:
        flat += over.get(n, [4 * 8 * 64, 8 * 64, 64] if n.endswith("q") else [2 * 8 * 64, 8 * 64, 64])
    return flat


@pytest.mark.parametrize("back", [False, True])
def test_strides(back):
    at = AT["q"]
    for bad in (dict(q=[-1, 64, 64]), dict(yq=[0, 512, 64]), dict(yq=[2048, 512, 63]), dict(yk=[1024, 511, 64]),
                dict(yq=[1 << 61, 1, 1]), dict(k=[1 << 62, 0, 1 << 62])):
        assert call(back, strides=strided(back, **bad)) == 1, bad
    # in place needs the same strides; an output inside another tensor's gaps is told from one that is not
    assert call(back, strides=strided(back, q=FUSED, yq=[2048, 512, 64]), yq=at) == 1
    assert call(back, strides=strided(back, q=FUSED, yk=FUSED), yk=at + 2 * 3 * 64) == 1    # over q's last head
    assert call(back, strides=strided(back, q=FUSED, yk=FUSED), yk=at + 2 * 7 * 64) == 1    # its second head is the next token's first
    assert call(back, strides=strided(back, k=FUSED, yk=FUSED, yq=FUSED), k=at, yk=at, yq=at + 2 * 64) == 1


def test_workspace():
    L = la.lib()
    need = L.la_norm_rotate_backward_workspace_bytes(2, 4, 2, 8, 64, 1)
    assert need >= 152 * 2 * 64 * 4
    assert call(True, wsb=need - 1) == la.LA_ERR_WORKSPACE
    assert call(True, ws=None) == la.LA_ERR_WORKSPACE
    assert call(True, ws=AT["ws"] + 16) == la.LA_ERR_WORKSPACE
    assert call(True, dwq=AT["ws"] + 64) == la.LA_ERR_INVALID_ARG
    assert call(True, dwq=AT["dwk"]) == la.LA_ERR_INVALID_ARG
    assert call(True, dwq=AT["dwq"] + 2) == la.LA_ERR_INVALID_ARG
    assert call(True, dwk=AT["yq"]) == la.LA_ERR_INVALID_ARG
    assert call(True, dwk=AT["freq"]) == la.LA_ERR_INVALID_ARG
    assert call(True, ws=AT["gk"]) == la.LA_ERR_INVALID_ARG
    for sizes in ((0, 4, 2, 8, 64, 1), (2, 4, 2, 0, 64, 1), (2, 4, 2, 8, 65, 1), (2, 4, 2, 8, 64, 7)):
        assert L.la_norm_rotate_backward_workspace_bytes(*sizes) == 0


def test_no_tokens_is_nothing_to_do():
    assert call(N=0, q=None, k=None, yq=None, yk=None) == la.LA_OK
    assert call(N=0, freq=None) == la.LA_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    import torch
    q = torch.zeros(1, 2, 4, 32)
    with pytest.raises(ValueError):
        la.norm_rotate(q, q)
    with pytest.raises(ValueError):
        la.norm_rotate_backward(q, q, q, q)
