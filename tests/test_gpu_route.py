"""GPU parity of gemm355_route and gemm355_route_grad against their plain binary64 forms:
ids and counts equal, weights to one rounding, gradients within the bound derived beside the
plain form (heads_ref.route_grad).  Logits sit in NaN-padded buffers, results between
sentinels."""

from __future__ import annotations

import numpy as np
import pytest

import heads_ref as ref
from gpu_util import to_device
from roofline_optimisation_amd import binding as gb

pytestmark = pytest.mark.gpu

SENT = 7777
CODE = {"f32": gb.F32, "f16": gb.F16, "bf16": gb.BF16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def padded(x, ld, dtype):
    """x's rows at stride ld in a NaN-filled device buffer."""
    nan = ref.round_to(np.array([np.nan]), dtype)[0] if dtype != "bf16" else np.uint16(0x7FC0)
    buf = np.full(x.shape[0] * ld + 16, nan, x.dtype)
    if x.size:
        buf[:x.shape[0] * ld].reshape(-1, ld)[:, :x.shape[1]] = x
    return to_device(buf)


def run_route(X, dtype, k, kind="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0,
              pad=0, counts=True):
    import torch
    rows, E = X.shape
    ld = E + pad
    dX = padded(X, ld, dtype)
    db = None if bias is None else to_device(bias.astype(np.float32))
    ids = torch.full((rows * k + 32,), SENT, dtype=torch.int32, device="cuda")
    wts = torch.full((rows * k + 32,), float(SENT), device="cuda")
    cnt = torch.full((E + 32,), SENT, dtype=torch.int32, device="cuda")
    flags = (gb.ROUTE_SIGMOID if kind == "sigmoid" else 0) | (gb.ROUTE_RENORM if renorm else 0)
    st = gb.gemm355_route(CODE[dtype], flags, rows, E, k, groups, top_groups, group_top, dX.data_ptr(), ld,
                          0 if db is None else db.data_ptr(), scale, ids.data_ptr() + 64, wts.data_ptr() + 64,
                          cnt.data_ptr() + 64 if counts else 0, torch.cuda.current_stream().cuda_stream)
    assert st == gb.OK, st
    torch.cuda.synchronize()
    out = []
    for t, n in ((ids, rows * k), (wts, rows * k), (cnt, E if counts else 0)):
        h = t.cpu().numpy()
        assert (h[:16] == SENT).all() and (h[16 + n:] == SENT).all(), "wrote outside"
        out.append(h[16:16 + n])
    return out[0].reshape(rows, k), out[1].reshape(rows, k), out[2]


def check_route(X, dtype, k, **kw):
    pad = kw.pop("pad", 0)
    if kw.get("bias") is not None:
        kw["bias"] = kw["bias"].astype(np.float32)   # the plain form adds what the kernel is given
    ids, w, n = run_route(X, dtype, k, pad=pad, **kw)
    rids, rw, rn = ref.route(X, dtype, k, **{**kw, "scale": float(np.float32(kw.get("scale", 1.0)))})
    assert np.array_equal(ids, rids), np.argwhere(ids != rids)[:4]
    assert np.array_equal(n, rn)
    # one rounding to binary32, and the binary64 scores' own (sums of up to 1024 terms: 2^-40)
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    live = ~np.isnan(rw)
    assert np.all(np.abs(w[live] - rw[live]) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(rw[live]) + 2.0 ** -149)


SHAPES = [(1, 1, 1), (1, 64, 8), (3, 2, 2), (5, 65, 3), (7, 63, 6), (9, 128, 8), (33, 96, 1), (130, 256, 8),
          (17, 257, 4), (6, 512, 16), (5, 1000, 64), (4, 1024, 10), (64, 8, 2), (2050, 16, 4)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,E,k", SHAPES)
def test_route_shapes(rows, E, k, dtype):
    X = ref.make_router(rows, E, dtype, rows + E)
    bias = np.random.default_rng(E).standard_normal(E) * 0.1
    check_route(X, dtype, k, kind="softmax", renorm=True, pad=3)
    check_route(X, dtype, k, kind="sigmoid", bias=bias, scale=2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,gtop", [(64, 8, 4, 2), (256, 8, 4, 2), (256, 8, 1, 1), (96, 3, 2, 2),
                                               (64, 64, 5, 2), (60, 4, 3, 1), (512, 16, 15, 2), (1024, 64, 8, 2),
                                               (8, 4, 4, 2), (1000, 8, 3, 2), (7, 7, 3, 1), (6, 2, 1, 2)])
def test_route_groups(E, groups, top, gtop, kind):
    bias = np.random.default_rng(E + groups).standard_normal(E) * 0.2
    k = min(8, top * (E // groups))
    for dtype in ("f32", "bf16"):
        X = ref.make_router(37, E, dtype, 5)
        check_route(X, dtype, k, kind=kind, bias=bias, groups=groups, top_groups=top, group_top=gtop, renorm=True,
                    scale=2.5)
        check_route(X, dtype, k, kind=kind, groups=groups, top_groups=top, group_top=gtop)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_index(kind):
    X = np.zeros((9, 200), np.float32)
    X[1:] = np.random.default_rng(1).integers(0, 3, (8, 200))
    check_route(X, "f32", 12, kind=kind, renorm=True)
    check_route(X, "f32", 12, kind=kind, groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_masked_experts(kind):
    inf = np.float32(np.inf)
    X = ref.make_router(8, 64, "f32", 9)
    X[0] = -inf                  # nothing left
    X[1, 5:] = -inf              # five left for eight places
    X[2, :8] = -inf              # a whole group
    X[3, ::2] = -inf
    X[4, 10] = np.nan
    X[5, 11] = inf
    X[6] = np.finfo(np.float32).min   # masked with the lowest finite value: an ordinary logit
    X[7, 1:] = np.finfo(np.float32).min
    bias = np.zeros(64)
    bias[[3, 40]] = -np.inf
    bias[41] = np.nan
    for kw in ({}, dict(bias=bias), dict(groups=8, top_groups=4, group_top=2, bias=bias),
               dict(groups=8, top_groups=4, group_top=1)):
        for renorm in (False, True):
            check_route(X, "f32", 8, kind=kind, renorm=renorm, **kw)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 200, 512, 1000])
def test_route_choices_a_rounding_apart(kind, E):
    """Choices and group scores that binary32 cannot order, and some it can: steps of 2^-30 and
    2^-22 of the scores, hidden in logits that the bias evens out."""
    rng = np.random.default_rng(E)
    X = ref.make_router(40, E, "f32", E)
    s = ref.scores(X.astype(np.float64), kind)
    # rows 0..: every choice near 0.5, its distance from it the rounding of the bias
    bias = (0.5 - s[0]).astype(np.float32)
    X[1:20] = X[0]
    X[1:20] += (rng.integers(-1, 2, (19, E)) * np.spacing(np.abs(X[0]))).astype(np.float32)
    check_route(X, "f32", 8, kind=kind, bias=bias, renorm=True)
    check_route(X, "f32", 8, kind=kind, bias=bias, groups=4, top_groups=2, group_top=2)
    # group scores equal but for the last bits: the same logits in every group, reordered
    per = E // 4
    for r in range(20, 40):
        base = X[r, :per].copy()
        for g in range(4):
            X[r, g * per:(g + 1) * per] = rng.permutation(base)
        X[r, rng.integers(E)] += np.float32(1e-6)
    check_route(X, "f32", 8, kind=kind, groups=4, top_groups=2, group_top=2, renorm=True)
    check_route(X, "f32", 8, kind=kind, groups=4, top_groups=1, group_top=1)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(32, 8), (20, 3), (48, 33), (64, 32)])
def test_route_many_rows(E, k, kind):
    """More rows than the grid has waves: a wave takes two rows at once (one for k > 32), either
    of which may have nothing to choose."""
    rows = 8192 + 2600
    X = ref.make_router(rows, E, "f32", 3)
    X[5] = -np.inf                       # the first of a wave's two
    X[8192 + 6] = -np.inf                # the second
    X[[7, 8192 + 7, 8192 + 8], [1, 2, 3]] = np.nan
    X[9, 2:] = -np.inf                   # fewer than k left
    X[8192 + 10, 2:] = -np.inf
    bias = np.random.default_rng(E).standard_normal(E) * 0.1
    check_route(X, "f32", k, kind=kind)
    check_route(X, "f32", k, kind=kind, bias=bias, renorm=True, pad=1)


def test_route_chosen_scores_of_zero():
    # the bias chooses experts whose softmax is 0 in binary64 (800 below the maximum)
    X = np.full((2, 32), -800.0, np.float32)
    X[:, 0] = 0.0
    bias = np.zeros(32)
    bias[4:8] = 2.0
    check_route(X, "f32", 3, bias=bias, renorm=True)


def test_route_without_counts_and_without_rows():
    import torch
    X = ref.make_router(20, 64, "f32", 2)
    ids, w, _ = run_route(X, "f32", 4, counts=False)
    assert np.array_equal(ids, ref.route(X, "f32", 4)[0])
    i, w, n = gb.route(torch.empty((0, 16), device="cuda"), 2)
    assert i.shape == (0, 2) and w.shape == (0, 2) and n.tolist() == [0] * 16


# ------------------------------------------------------------------ gradient

def run_grad(X, dtype, ids, dw, kind="softmax", renorm=False, scale=1.0, pad=0, in_place=False):
    import torch
    rows, E = X.shape
    ld = E + pad
    dX = padded(X, ld, dtype)
    if in_place:
        out, ldo, off = dX, ld, 0
    else:
        ldo, off = E + 2 * pad, 16
        out = to_device(np.full(rows * ldo + 32, SENT, np.float32 if dtype == "f32" else np.uint16))
    flags = (gb.ROUTE_SIGMOID if kind == "sigmoid" else 0) | (gb.ROUTE_RENORM if renorm else 0)
    di, dd = to_device(np.ascontiguousarray(ids)), to_device(np.ascontiguousarray(dw))
    es = out.element_size()
    st = gb.gemm355_route_grad(CODE[dtype], flags, rows, E, ids.shape[1], dX.data_ptr(), ld, di.data_ptr(),
                               dd.data_ptr(), scale, out.data_ptr() + es * off, ldo,
                               torch.cuda.current_stream().cuda_stream)
    assert st == gb.OK, st
    torch.cuda.synchronize()
    h = out.cpu().numpy()
    if dtype != "f32":
        h = h.view(np.uint16)
    got = h[off:off + rows * ldo].reshape(rows, ldo)[:, :E].copy()
    if not in_place:
        h[off:off + rows * ldo].reshape(rows, ldo)[:, :E] = SENT
        assert (h == SENT).all(), "wrote outside"
    return ref.widen(got, dtype)


def check_grad(X, dtype, ids, dw, what, **kw):
    got = run_grad(X, dtype, ids, dw, **kw)
    kw = {k: v for k, v in kw.items() if k in ("kind", "renorm", "scale")}
    want, tol = ref.route_grad(X, dtype, ids, dw, **kw)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("rows,E,k", SHAPES)
def test_route_grad(rows, E, k, dtype, kind, renorm):
    X = ref.make_router(rows, E, dtype, rows + 2 * E)
    ids = ref.route(X, dtype, k, kind)[0]
    dw = np.random.default_rng(rows).standard_normal((rows, k)).astype(np.float32)
    check_grad(X, dtype, ids, dw, (rows, E, k), kind=kind, renorm=renorm, scale=1.5, pad=rows % 3)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_odd_ids(kind, renorm):
    """Places without an expert, ids outside the experts, the same id twice."""
    X = ref.make_router(5, 70, "f32", 1)
    X[3, 10:] = -np.inf
    X[4] = -np.inf
    ids = np.array([[0, -1, 3], [-1, -1, -1], [7, 7, 69], [1, 2, 70], [5, 6, 1 << 30]], np.int32)
    dw = np.random.default_rng(2).standard_normal(ids.shape).astype(np.float32)
    check_grad(X, "f32", ids, dw, "odd ids", kind=kind, renorm=renorm)
    check_grad(X, "f32", ids, dw, "odd ids in place", kind=kind, renorm=renorm, in_place=True, pad=2)


def test_more_rows_than_a_launch_has_threads_for():
    """2^26 rows and more: 64 threads a row would be 2^32."""
    import torch
    rows = (1 << 26) + 5
    X = torch.randint(-4, 5, (rows, 2), device="cuda").to(torch.bfloat16)
    ids, w, counts = gb.route(X, 1, score="sigmoid")
    want = (X[:, 1] > X[:, 0]).to(torch.int32)
    assert torch.equal(ids[:, 0], want)
    ones = int(want.sum(dtype=torch.int64))
    assert counts.tolist() == [rows - ones, ones]
    del want
    s = torch.sigmoid(torch.maximum(X[:, 0], X[:, 1]).float())
    assert ((w[:, 0] - s).abs() <= 2.0 ** -20).all()
    dX = gb.route_grad(X, ids, w, score="sigmoid")
    chosen = torch.gather(dX, 1, ids.long())[:, 0].float()
    # one rounding to bfloat16, and binary32's own
    assert ((chosen - w[:, 0] * s * (1 - s)).abs() <= 2.0 ** -8 * chosen.abs() + 2.0 ** -20).all()
    assert not torch.gather(dX, 1, 1 - ids.long()).any()
    dX = gb.route_grad(X, ids, w, score="softmax")
    assert torch.equal(dX[-3:], gb.route_grad(X[-3:], ids[-3:], w[-3:], score="softmax"))


def test_infinite_bias():
    """A bias of +infinity chooses its expert first, of several the lowest; with NaN or -infinity
    an expert is out."""
    bias = np.zeros(40)
    bias[[7, 30]] = np.inf
    bias[9] = -np.inf
    bias[12] = np.nan
    X = ref.make_router(12, 40, "f32", 3)
    X[3, 7] = -np.inf
    for kind in ("softmax", "sigmoid"):
        for kw in ({}, dict(groups=5, top_groups=2, group_top=2), dict(groups=5, top_groups=3, group_top=1)):
            check_route(X, "f32", 6, kind=kind, bias=bias, renorm=True, **kw)
