"""GPU parity of gemm355_xent and gemm355_xent_grad against their plain binary64 forms,
every element within the bound derived beside them (heads_ref.xent, heads_ref.xent_grad).
Operands sit in NaN-padded buffers, results between sentinels."""

from __future__ import annotations

import numpy as np
import pytest

import heads_ref as ref
from gpu_util import nan_fill, place, to_device
from roofline_optimisation_amd import binding as gb

pytestmark = pytest.mark.gpu

CODE = {"f32": gb.F32, "f16": gb.F16, "bf16": gb.BF16}
SENT = 7777


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Head:
    """A projection's operands on the GPU, W as N x K (trans_b) or K x N, with padded rows."""

    def __init__(self, X, W, labels, dtype, trans_b, padx=0, padw=0, offset=0):
        self.X, self.W, self.labels, self.dtype, self.trans_b = X, W, labels, dtype, trans_b
        self.M, self.K = X.shape
        self.N = W.shape[0]
        w = W if trans_b else np.ascontiguousarray(W.T)
        self.ldx, self.ldw = max(self.K, 1) + padx, max(w.shape[1], 1) + padw
        fill = nan_fill(dtype)
        self.dX = to_device(place(X, self.ldx, offset, 1, fill))
        self.dW = to_device(place(w, self.ldw, offset, 1, fill))
        es = self.dX.element_size()
        self.px, self.pw = self.dX.data_ptr() + es * offset, self.dW.data_ptr() + es * offset
        self.dlabels = to_device(labels)
        self.flags = gb.TRANS_B if trans_b else 0

    def head_args(self):
        return (CODE[self.dtype], self.flags, self.M, self.N, self.K, self.px, self.ldx, self.pw, self.ldw,
                self.dlabels.data_ptr())


def scratch(n):
    """Workspace of exactly n bytes followed by a guard, filled with NaN patterns."""
    import torch
    return torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")


def guard_ok(ws, n):
    return bool((ws[n:] == 0xFF).all())


def run_xent(h, ignore=-100):
    import torch
    out = torch.full((2, h.M + 32), float(SENT), device="cuda")
    n = gb.gemm355_xent_workspace(CODE[h.dtype], h.flags, h.M, h.N, h.K)
    ws = scratch(n)
    st = gb.gemm355_xent(*h.head_args(), ignore, out[0, 16:].data_ptr(), out[1, 16:].data_ptr(), ws.data_ptr(), n,
                         torch.cuda.current_stream().cuda_stream)
    assert st == gb.OK, st
    torch.cuda.synchronize()
    assert guard_ok(ws, n), "wrote past the workspace"
    o = out.cpu().numpy()
    assert (o[:, :16] == SENT).all() and (o[:, 16 + h.M:] == SENT).all(), "wrote outside"
    return o[0, 16:16 + h.M].copy(), o[1, 16:16 + h.M].copy()


def check_xent(h, what, ignore=-100):
    loss, lse = run_xent(h, ignore)
    wl, ws, tl, ts = ref.xent(h.X, h.W, h.labels, h.dtype, ignore)
    assert np.all(np.abs(lse - ws) <= ts), (what, float((np.abs(lse - ws) / ts).max()))
    assert np.array_equal(np.isnan(loss), np.isnan(wl)), what
    ok = ~np.isnan(wl)
    assert np.all(np.abs(loss - wl)[ok] <= tl[ok]), (what, np.abs(loss - wl)[ok].max())
    assert np.all(loss[h.labels == ignore] == 0)
    return lse


def run_grad(h, lse, dloss, need=(True, True), padx=0, padw=0, ignore=-100):
    import torch
    wr, wc = (h.N, h.K) if h.trans_b else (h.K, h.N)
    store = np.float32 if h.dtype == "f32" else np.uint16
    ldx, ldw = max(h.K, 1) + padx, max(wc, 1) + padw
    dx = to_device(np.full(16 + h.M * ldx + 16, SENT, store))
    dw = to_device(np.full(16 + wr * ldw + 16, SENT, store))
    es = dx.element_size()
    n = gb.gemm355_xent_grad_workspace(CODE[h.dtype], h.flags, h.M, h.N, h.K)
    ws = scratch(n)
    dl, dg = to_device(lse.astype(np.float32)), to_device(dloss.astype(np.float32))
    st = gb.gemm355_xent_grad(*h.head_args(), ignore, dl.data_ptr(), dg.data_ptr(),
                              dx.data_ptr() + 16 * es if need[0] else 0, ldx,
                              dw.data_ptr() + 16 * es if need[1] else 0, ldw, ws.data_ptr(), n,
                              torch.cuda.current_stream().cuda_stream)
    assert st == gb.OK, st
    torch.cuda.synchronize()
    assert guard_ok(ws, n), "wrote past the workspace"
    got = []
    for t, rows, cols, ld, want in ((dx, h.M, h.K, ldx, need[0]), (dw, wr, wc, ldw, need[1])):
        o = t.cpu().numpy().view(store)
        body = o[16:16 + rows * ld].reshape(rows, ld)
        g = body[:, :cols].copy()
        if want:
            body[:, :cols] = SENT
        assert (o == SENT).all(), "wrote outside"
        got.append(ref.widen(g, h.dtype) if want else None)
    if got[1] is not None and not h.trans_b:
        got[1] = got[1].T
    return got


def check_grad(h, lse, dloss, what, ignore=-100, parts=1, **kw):
    dX, dW = run_grad(h, lse, dloss, ignore=ignore, **kw)
    wX, wW, tX, tW = ref.xent_grad(h.X, h.W, h.labels, lse, dloss, h.dtype, ignore, parts)
    for name, got, want, tol in (("dX", dX, wX, tX), ("dW", dW, wW, tW)):
        if got is None:
            continue
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (what, name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                               tol[bad][:4])


def upstream(M, seed, dtype):
    rng = np.random.default_rng(seed)
    return ((0.5 + rng.random(M)) * (256.0 if dtype == "f16" else 1.0) / max(M, 1)).astype(np.float32)


# rows x classes x hidden: one of each; hidden sizes below, at and past a trip of the ring,
# ragged in every way; rows and classes that end inside a tile of any size
SHAPES = [(1, 1, 1), (1, 1000, 64), (3, 7, 0), (2, 33, 7), (5, 100, 136), (16, 2056, 128), (17, 1001, 256),
          (33, 515, 520), (64, 640, 200), (65, 777, 128), (100, 300, 1000), (128, 512, 384), (130, 1288, 264),
          (255, 1999, 192), (257, 2304, 128), (300, 1000, 72), (513, 520, 256)]


@pytest.mark.parametrize("trans_b", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_loss_and_gradient(M, N, K, dtype, trans_b):
    X, W, y = ref.make_head(M, N, K, dtype, M + N + K)
    h = Head(X, W, y, dtype, trans_b)
    lse = check_xent(h, (M, N, K))
    if K:
        check_grad(h, lse, upstream(M, 1, dtype), (M, N, K))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("padx,padw,offset", [(8, 16, 0), (1, 0, 0), (0, 3, 0), (0, 0, 1), (5, 7, 3), (24, 8, 8)])
@pytest.mark.parametrize("trans_b", [True, False])
def test_strides_and_alignment(padx, padw, offset, dtype, trans_b):
    X, W, y = ref.make_head(70, 400, 160, dtype, 5)
    h = Head(X, W, y, dtype, trans_b, padx, padw, offset)
    lse = check_xent(h, (padx, padw, offset))
    check_grad(h, lse, upstream(70, 2, dtype), (padx, padw, offset), padx=padw, padw=padx)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("need", [(True, False), (False, True)])
def test_one_gradient(dtype, need):
    X, W, y = ref.make_head(90, 600, 128, dtype, 6)
    h = Head(X, W, y, dtype, True)
    lse = check_xent(h, need)
    check_grad(h, lse, upstream(90, 3, dtype), need, need=need)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_labels(dtype):
    """Rows without a label, labels outside the vocabulary, an ignored class inside it."""
    X, W, y = ref.make_head(140, 300, 136, dtype, 7, ignored=False)
    y[:8] = [-1, 300, 1 << 40, -(1 << 40), 299, 0, 1 << 32, -100]
    h = Head(X, W, y, dtype, True)
    lse = check_xent(h, "labels")
    check_grad(h, lse, upstream(140, 4, dtype), "labels")
    y2 = y.copy()
    y2[20:30] = 17
    h = Head(X, W, y2, dtype, True)
    lse = check_xent(h, "ignore 17", ignore=17)
    check_grad(h, lse, upstream(140, 4, dtype), "ignore 17", ignore=17)
    y3 = np.full(140, -100, np.int64)
    h = Head(X, W, y3, dtype, True)
    lse = check_xent(h, "no labels")
    dX, dW = run_grad(h, lse, upstream(140, 4, dtype))
    assert not dX.any() and not dW.any()


@pytest.mark.parametrize("trans_b", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_nan_in_rows_without_a_label(dtype, trans_b):
    """What a padded row holds reaches no gradient and no other row's loss."""
    X, W, y = ref.make_head(150, 520, 128, dtype, 8)
    y[[3, 70, 149]] = -100
    Xn = X.copy()
    for r, v in ((3, np.nan), (70, np.inf), (149, -np.inf)):
        Xn[r] = ref.round_to(np.full(128, v), dtype) if dtype != "bf16" or np.isfinite(v) or np.isinf(v) else 0x7FC0
    lse = ref.xent(X, W, y, dtype)[1].astype(np.float32)
    clean, dirty = Head(X, W, y, dtype, trans_b), Head(Xn, W, y, dtype, trans_b)
    l0, s0 = run_xent(clean)
    l1, s1 = run_xent(dirty)
    rest = np.ones(150, bool)
    rest[[3, 70, 149]] = False
    assert np.array_equal(l0, l1) and np.array_equal(s0[rest], s1[rest]) and not np.isfinite(s1[~rest]).any()
    lse_n = lse.copy()
    lse_n[[3, 70, 149]] = np.nan
    g = upstream(150, 9, dtype)
    gn = g.copy()
    gn[[3, 70, 149]] = np.nan
    a, b = run_grad(clean, lse, g), run_grad(dirty, lse_n, gn)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    check_grad(clean, lse, g, "clean")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_far_apart_logits(dtype):
    """Logits thousands apart: the label's far below, or alone at the top (loss 0)."""
    rng = np.random.default_rng(1)
    W = ref.round_to(rng.standard_normal((300, 128)), dtype)
    y = rng.integers(0, 300, 66).astype(np.int64)
    X = ref.round_to(ref.widen(W, dtype)[y] * rng.choice([-40.0, 40.0], (66, 1)), dtype)
    h = Head(X, W, y, dtype, True)
    lse = check_xent(h, "far apart")
    check_grad(h, lse, upstream(66, 5, dtype), "far apart")


@pytest.mark.parametrize("exponent", [-90, -40, -14, 0, 14])
def test_binary16_upstream_of_any_size(exponent):
    """dZ is scaled before it is rounded, so dX relative to the upstream gradient does not
    depend on its size (until dX itself leaves binary16's range)."""
    X, W, y = ref.make_head(80, 900, 128, "f16", 12)
    h = Head(X, W, y, "f16", True)
    lse = ref.xent(X, W, y, "f16")[1].astype(np.float32)
    check_grad(h, lse, upstream(80, 6, "f32") * np.float32(2.0 ** exponent), exponent)


@pytest.mark.parametrize("trans_b", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 128), (7, 2600, 256), (33, 1003, 136), (64, 5000, 520), (64, 256, 100)])
def test_few_rows_keep_two_parts(M, N, K, dtype, trans_b):
    """Up to 64 rows the rounding of dZ adds next to nothing to the results' own."""
    X, W, y = ref.make_head(M, N, K, dtype, 15 + M, ignored=M > 1)
    h = Head(X, W, y, dtype, trans_b)
    lse = ref.xent(X, W, y, dtype)[1].astype(np.float32)
    check_grad(h, lse, upstream(M, 8, dtype), (M, N, K), parts=2)


def test_zero_upstream():
    for dtype in ("f32", "f16", "bf16"):
        X, W, y = ref.make_head(40, 200, 128, dtype, 13)
        h = Head(X, W, y, dtype, True)
        lse = ref.xent(X, W, y, dtype)[1].astype(np.float32)
        dX, dW = run_grad(h, lse, np.zeros(40, np.float32))
        assert not dX.any() and not dW.any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_many_pieces(dtype):
    """Rows enough that the vocabulary is walked in several pieces, the last one odd
    (checked in binary64 on the GPU)."""
    import torch
    M, N, K = 9000, 20001, 64 if dtype == "f32" else 128
    g = torch.Generator(device="cuda").manual_seed(3)
    t = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    W = (torch.randn(N, K, generator=g, device="cuda") * 0.2).to(t)
    X = torch.randn(M, K, generator=g, device="cuda").to(t)
    y = torch.randint(0, N, (M,), generator=g, device="cuda")
    y[::7] = -100
    loss, lse = gb.linear_cross_entropy(X, W, y, trans_b=True)
    Z = X.double() @ W.double().t()
    e = (K + 8) * 2.0 ** -24 * (X.double().abs() @ W.double().abs().t())
    want = torch.logsumexp(Z, 1)
    tol = e.max(1)[0] + 2.0 ** -24 * (4 * want.abs() + N / 256 + 64)
    assert ((lse - want).abs() <= tol).all()
    live = y != -100
    at = torch.where(live, y, 0)
    wl = torch.where(live, want - Z.gather(1, at[:, None])[:, 0], 0.0)
    assert ((loss - wl).abs() <= 2 * tol + 2.0 ** -22 * (want.abs() + 16)).all()
    dl = torch.rand(M, generator=g, device="cuda") / (1.0 if dtype == "f16" else M)
    dX, dW = gb.linear_cross_entropy_grad(X, W, y, lse, dl, trans_b=True)
    gr = torch.where(live, dl, 0.0).double()
    P = torch.exp(Z - lse.double()[:, None])
    dZ = gr[:, None] * P
    dZ[torch.arange(M, device="cuda"), at] -= gr
    half = 0.0 if dtype == "f32" else ref.HALF[dtype]
    # as in heads_ref.xent_grad, |Z| and |lse| bounded by their largest
    d = e + 2.0 ** -24 * (4 * lse.abs().max().item() + 2 * Z.abs().max().item() + 16)
    err = gr[:, None] * P * torch.expm1(d) + 3 * 2.0 ** -24 * dZ.abs()
    err = err + half * (dZ.abs() + err)
    if dtype == "f16":
        err += 2.0 ** -25 * gr.max() / 2.0 ** 13 * (gr != 0)[:, None]
    tiny = {"f32": 2.0 ** -140, "f16": 2.0 ** -25, "bf16": 2.0 ** -130}[dtype]
    del P, e, d
    w, x = W.double(), torch.where(live[:, None], X.double(), 0.0)
    mag = dZ.abs() + err
    for got, want, tol in ((dX, dZ @ w, err @ w.abs() + (N + 8) * 2.0 ** -24 * (mag @ w.abs())),
                           (dW, dZ.t().contiguous() @ x,
                            err.t().contiguous() @ x.abs() + (M + 8) * 2.0 ** -24 * (mag.t().contiguous() @ x.abs()))):
        tol = tol + ref.HALF[dtype] * (want.abs() + tol) + tiny
        assert ((got.double() - want).abs() <= tol).all()


def test_no_rows():
    import torch
    for t in (torch.float32, torch.bfloat16):
        W = torch.ones(30, 16, device="cuda", dtype=t)
        X = torch.empty(0, 16, device="cuda", dtype=t)
        y = torch.empty(0, dtype=torch.int64, device="cuda")
        e = torch.empty(0, device="cuda")
        loss, lse = gb.linear_cross_entropy(X, W, y, trans_b=True)
        assert loss.shape == lse.shape == (0,)
        dX, dW = gb.linear_cross_entropy_grad(X, W, y, e, e, trans_b=True)
        assert dX.shape == (0, 16) and dW.shape == (30, 16) and not dW.any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [5, 700])
def test_no_hidden_columns(dtype, N):
    """K = 0: every logit is 0, and no gradient has elements."""
    import torch
    t = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    X, W = torch.empty(9, 0, device="cuda", dtype=t), torch.empty(N, 0, device="cuda", dtype=t)
    y = torch.arange(9, device="cuda") % N
    loss, lse = gb.linear_cross_entropy(X, W, y, trans_b=True)
    # log N, to the rounding of the logarithm and the sum
    assert ((loss.double() - np.log(N)).abs() <= 2.0 ** -20 * np.log(N)).all() and torch.equal(loss, lse)
    dX, dW = gb.linear_cross_entropy_grad(X, W, y, lse, loss, trans_b=True)
    assert dX.shape == (9, 0) and dW.shape == (N, 0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("trans_b", [True, False])
@pytest.mark.parametrize("M,N,K", [(1500, 300, 136), (2300, 517, 264), (3000, 256, 100)])
def test_many_rows_of_few_classes(M, N, K, dtype, trans_b):
    """dW of few tiles, summed over ranges of the rows."""
    X, W, y = ref.make_head(M, N, K, dtype, M)
    h = Head(X, W, y, dtype, trans_b, padx=3, padw=1)
    lse = check_xent(h, (M, N, K))
    check_grad(h, lse, upstream(M, 1, dtype), (M, N, K), padx=1, padw=2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rest,N,K", [(500, 1000, 256), (20, 300, 264), (1, 256, 128), (3000, 1000, 260)])
def test_rows_past_a_block_of_rows(rest, N, K, dtype):
    """The loss takes 32768 rows at a time; the few after them may take smaller tiles, with more
    statistics a row."""
    X, W, y = ref.make_head(32768 + rest, N, K, dtype, rest)
    check_xent(Head(X, W, y, dtype, True), (rest, N, K))


@pytest.mark.parametrize("trans_b", [True, False])
def test_more_classes_than_a_launch_takes(trans_b):
    """The loss takes 2^22 classes at a time."""
    import torch
    M, N, K = 70, (1 << 22) + 1000, 136
    torch.manual_seed(1)
    X = torch.randn(M, K, device="cuda").half()
    W = (torch.randn(N, K, device="cuda") / K ** 0.5).half()
    y = torch.randint(0, N, (M,), device="cuda")
    y[:3] = torch.tensor([N - 1, 1 << 22, (1 << 22) - 1])
    loss, lse = gb.linear_cross_entropy(X, W if trans_b else W.t().contiguous(), y, trans_b=trans_b)
    Z = torch.cat([X.double() @ W[v:v + (1 << 18)].double().t() for v in range(0, N, 1 << 18)], 1)
    want = torch.logsumexp(Z, 1)
    # the sum's own error and a logit's, K rounded additions of products at most 2^-24 each of
    # sum |x w| <= |x| |w|
    size = X.double().norm(dim=1) * float(W.float().norm(dim=1).max())
    tol = 2.0 ** -24 * (4 * want.abs() + N / 256 + 64 + K * size)
    assert ((lse - want).abs() <= tol).all()
    zl = Z.gather(1, y[:, None])[:, 0]
    assert ((loss - (want - zl)).abs() <= tol + 2.0 ** -24 * (K * size + want.abs() + zl.abs())).all()


def test_repeated_calls_give_the_same_bits():
    for dtype in ("f32", "bf16"):
        X, W, y = ref.make_head(200, 3001, 256, dtype, 14)
        h = Head(X, W, y, dtype, True)
        a, b = run_xent(h), run_xent(h)
        assert np.array_equal(a[0], b[0], equal_nan=True) and np.array_equal(a[1], b[1])
        g = upstream(200, 7, dtype)
        a, b = run_grad(h, a[1], g), run_grad(h, a[1], g)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
