"""The loss and routing entry points without a GPU: refusals, no-ops and workspace sizes are
decided on the host before any HIP call; the plain forms the GPU tests compare with agree
with differences of their own losses."""

import numpy as np
import pytest

import heads_ref as ref
from roofline_optimisation_amd import binding as gb

P, Q, R, S, T, U, V, WS = (1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32, 6 << 32, 7 << 32, 8 << 32)
BIG = 1 << 31


def xent(**kw):
    a = dict(dtype=2, flags=gb.TRANS_B, M=8, N=100, K=16, X=P, ldx=16, W=Q, ldw=16, labels=R, ignore=-100, loss=S,
             lse=T, ws=WS, n=BIG)
    a.update(kw)
    return gb.gemm355_xent(*[a[k] for k in ("dtype", "flags", "M", "N", "K", "X", "ldx", "W", "ldw", "labels",
                                            "ignore", "loss", "lse", "ws", "n")])


def grad(**kw):
    a = dict(dtype=2, flags=gb.TRANS_B, M=8, N=100, K=16, X=P, ldx=16, W=Q, ldw=16, labels=R, ignore=-100, lse=S,
             dloss=T, dX=U, lddx=16, dW=V, lddw=16, ws=WS, n=BIG)
    a.update(kw)
    return gb.gemm355_xent_grad(*[a[k] for k in ("dtype", "flags", "M", "N", "K", "X", "ldx", "W", "ldw", "labels",
                                                 "ignore", "lse", "dloss", "dX", "lddx", "dW", "lddw", "ws", "n")])


COMMON_BAD = [dict(dtype=3), dict(dtype=-1), dict(flags=gb.TRANS_A), dict(flags=64), dict(M=-1), dict(N=-1),
              dict(K=-1), dict(M=1 << 30), dict(N=1 << 30), dict(N=0), dict(ldx=15), dict(ldw=15),
              dict(flags=0, ldw=99), dict(X=0), dict(W=0), dict(labels=0), dict(ws=0), dict(ws=WS + 8),
              dict(n=16), dict(ws=P), dict(ws=Q + 64)]


@pytest.mark.parametrize("kw", COMMON_BAD + [dict(loss=P), dict(lse=Q + 32), dict(loss=R), dict(loss=S, lse=S + 4),
                                             dict(loss=WS + 128)])
def test_xent_refuses(kw):
    assert xent(**kw) == gb.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", COMMON_BAD + [dict(lse=0), dict(dloss=0), dict(lddx=15), dict(lddw=15), dict(dX=P),
                                             dict(dX=Q), dict(dW=Q), dict(dW=P + 32), dict(dX=U, dW=U + 16),
                                             dict(dX=S), dict(dW=T), dict(dX=WS + 64), dict(dW=R + 8)])
def test_xent_grad_refuses(kw):
    assert grad(**kw) == gb.ERR_INVALID_ARG


def test_xent_noops():
    assert xent(M=0, X=0, W=0, labels=0, ws=0, n=0) == gb.OK
    assert xent(loss=0, lse=0) == gb.OK
    assert grad(dX=0, dW=0) == gb.OK
    assert grad(M=0, dW=0) == gb.OK
    assert grad(K=0, ldx=1, ldw=1, lddx=1, lddw=1) == gb.OK   # both gradients have no elements


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_workspace_sizes(dtype):
    for f in (gb.gemm355_xent_workspace, gb.gemm355_xent_grad_workspace):
        assert f(dtype, gb.TRANS_B, 0, 10, 10) == 0
        assert f(dtype, gb.TRANS_B, 10, 0, 10) == 0
        assert f(3, 0, 10, 10, 10) == 0 and f(dtype, 4, 10, 10, 10) == 0 and f(dtype, 0, -1, 10, 10) == 0
    assert gb.gemm355_xent_workspace(dtype, gb.TRANS_B, 10, 1000, 0) > 0
    assert gb.gemm355_xent_grad_workspace(dtype, gb.TRANS_B, 10, 1000, 0) == 0   # no gradient has elements
    # never the whole logits: 8192 x 131072 of binary32 are 4 GiB
    assert gb.gemm355_xent_workspace(dtype, gb.TRANS_B, 8192, 131072, 4096) < 1 << 30
    assert gb.gemm355_xent_grad_workspace(dtype, gb.TRANS_B, 8192, 131072, 4096) < 4 << 30


def route(**kw):
    a = dict(dtype=0, flags=0, rows=8, E=64, k=4, groups=8, top=4, gtop=2, X=P, ldx=64, bias=Q, scale=1.0, ids=R,
             weights=S, counts=T)
    a.update(kw)
    return gb.gemm355_route(*[a[k] for k in ("dtype", "flags", "rows", "E", "k", "groups", "top", "gtop", "X", "ldx",
                                             "bias", "scale", "ids", "weights", "counts")])


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(flags=4), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(E=0),
                                dict(E=1025, groups=1, top=1, ldx=1025), dict(ldx=63), dict(groups=0),
                                dict(groups=7), dict(groups=128, E=128, ldx=128), dict(top=0), dict(top=9),
                                dict(gtop=0), dict(gtop=3), dict(k=0), dict(k=33), dict(k=65, groups=1, top=1, E=128,
                                                                                        ldx=128),
                                dict(X=0), dict(ids=0), dict(weights=0), dict(ids=P), dict(weights=R + 64),
                                dict(counts=Q + 4), dict(counts=R)])
def test_route_refuses(kw):
    assert route(**kw) == gb.ERR_INVALID_ARG


def rgrad(**kw):
    a = dict(dtype=1, flags=2, rows=8, E=64, k=4, X=P, ldx=64, ids=Q, dw=R, scale=1.0, dX=S, lddx=64)
    a.update(kw)
    return gb.gemm355_route_grad(*[a[k] for k in ("dtype", "flags", "rows", "E", "k", "X", "ldx", "ids", "dw",
                                                  "scale", "dX", "lddx")])


@pytest.mark.parametrize("kw", [dict(dtype=5), dict(flags=8), dict(rows=-2), dict(E=0), dict(E=2000, ldx=2000,
                                                                                            lddx=2000),
                                dict(ldx=63), dict(lddx=63), dict(k=0), dict(k=65), dict(X=0), dict(ids=0),
                                dict(dw=0), dict(dX=0), dict(dX=P + 2), dict(dX=P, lddx=65), dict(dX=Q),
                                dict(dX=R + 4)])
def test_route_grad_refuses(kw):
    assert rgrad(**kw) == gb.ERR_INVALID_ARG


def test_route_noops():
    assert route(rows=0, X=0, ids=0, weights=0, counts=0) == gb.OK
    assert rgrad(rows=0, X=0, ids=0, dw=0, dX=0) == gb.OK


def test_wrappers_refuse():
    import torch
    x, w, y = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        gb.linear_cross_entropy(x, w, y, trans_b=True)          # not on a GPU
    with pytest.raises(ValueError):
        gb.linear_cross_entropy_grad(x, w, y, x[:, 0], x[:, 0], trans_b=True)
    with pytest.raises(ValueError):
        gb.route(x, 2)
    with pytest.raises(ValueError):
        gb.route(x, 2, score="tanh")
    with pytest.raises(ValueError):
        gb.route_grad(x, y, x)
    with pytest.raises(ValueError):
        gb._row_stride(torch.zeros(1, 8).expand(4, 8), "X")     # rows that overlap
    with pytest.raises(ValueError):
        gb._row_stride(torch.zeros(8, 4).t(), "X")              # columns first
    with pytest.raises(ValueError):
        gb._c_ints(3, 1 << 31)
    assert gb._row_stride(torch.zeros(4, 10)[:, :8], "X") == 10
    assert gb._row_stride(torch.zeros(8, 1).t(), "X") == 8
    assert gb._row_stride(torch.zeros(4, 0), "X") == 1


# ------------------------------------------------ the plain forms against differences

def test_plain_gradient_matches_differences():
    rng = np.random.default_rng(3)
    X, W, y = ref.make_head(5, 11, 6, "f32", 3)
    g = rng.standard_normal(5).astype(np.float32)

    def total(x, w):
        z = x @ w.T
        m = z.max(1)
        lse = m + np.log(np.exp(z - m[:, None]).sum(1))
        live = y != -100
        return (g.astype(np.float64) * np.where(live, lse - z[np.arange(5), np.where(live, y, 0)], 0)).sum()

    x, w = X.astype(np.float64), W.astype(np.float64)
    lse = ref.xent(X, W, y, "f32")[1]
    dX, dW, _, _ = ref.xent_grad(X, W, y, lse, g, "f32")
    h = 1e-6
    for got, arr, f in ((dX, x, lambda a: total(a, w)), (dW, w, lambda a: total(x, a))):
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += h
            dn[i] -= h
            # central differences of a smooth sum: error h^2 f''' / 6 + 2^-53 |f| / h, below 1e-7
            assert abs((f(up) - f(dn)) / (2 * h) - got[i]) < 1e-7


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_plain_route_gradient_matches_differences(kind, renorm):
    rng = np.random.default_rng(4)
    X = ref.make_router(4, 12, "f32", 4)
    ids, _, _ = ref.route(X, "f32", 3, kind, renorm=renorm, scale=2.5)
    dw = rng.standard_normal((4, 3)).astype(np.float32)
    dX, _ = ref.route_grad(X, "f32", ids, dw, kind, renorm, 2.5)

    def total(x):
        s = np.take_along_axis(ref.scores(x, kind), ids, 1)
        w = 2.5 * (s / s.sum(1, keepdims=True) if renorm else s)
        return (dw.astype(np.float64) * w).sum()

    x, h = X.astype(np.float64), 1e-6
    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += h
        dn[i] -= h
        assert abs((total(up) - total(dn)) / (2 * h) - dX[i]) < 1e-7
