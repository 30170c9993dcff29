"""The operators as a training step uses them together: a router's logits and choice, the
experts' products weighted by it, the vocabulary head's loss, and the way back through all of
them to the router's weights; on other streams, in graphs, and beside themselves."""

from __future__ import annotations

import pytest

from roofline_optimisation_amd import binding as gb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(M=96, K=64, E=16, N=517, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, f=1.0: torch.randn(*s, generator=g, device="cuda") * f  # noqa: E731
    s = dict(X=r(M, K), Wr=r(K, E, f=K ** -0.5), We=r(E, K, K, f=K ** -0.5), W=r(N, K, f=K ** -0.5),
             y=torch.randint(0, N, (M,), generator=g, device="cuda"))
    s["y"][::5] = -100
    return s


def step(s, k=4):
    """Loss per row, and the gradients of its mean to the head's and the router's weights."""
    import torch
    X, Wr, We, W, y = s["X"], s["Wr"], s["We"], s["W"], s["y"]
    logits = gb.matmul(X, Wr)
    ids, w, counts = gb.route(logits, k, score="sigmoid", groups=4, top_groups=2, group_top=2, renorm=True, scale=2.0)
    outs = torch.stack([gb.matmul(X, We[e]) for e in range(We.shape[0])], 1)     # M x E x K
    chosen = torch.gather(outs, 1, ids.long()[:, :, None].expand(-1, -1, X.shape[1]))
    H = X + (w[:, :, None] * chosen).sum(1)
    loss, lse = gb.linear_cross_entropy(H, W, y, trans_b=True)
    live = (y != -100).sum()
    dloss = (1.0 / live).expand(y.shape[0]).contiguous().float()
    dH, dW = gb.linear_cross_entropy_grad(H, W, y, lse, dloss, trans_b=True)
    dw = (dH[:, None, :] * chosen).sum(2).contiguous()
    dlogits = gb.route_grad(logits, ids, dw, score="sigmoid", renorm=True, scale=2.0)
    dWr = gb.matmul(X, dlogits, trans_a=True)
    return loss, dW, dWr, ids, counts, dlogits


def test_a_training_step_against_autograd():
    """binary32 throughout; reference in binary64 with the step's own choice of experts.
    Relative 2-norm errors: every stage is a sum of at most N = 517 binary32 products of
    values the earlier stages hold to about 1e-6, none of which cancels to below a thousandth
    of its terms in norm: 1e-4."""
    import torch
    s = make()
    loss, dW, dWr, ids, counts, _ = step(s)
    d = {k: v.double() for k, v in s.items() if k != "y"}
    W, Wr = d["W"].requires_grad_(True), d["Wr"].requires_grad_(True)
    logits = d["X"] @ Wr
    p = torch.sigmoid(logits)
    q = torch.gather(p, 1, ids.long())
    w = 2.0 * q / q.sum(1, keepdim=True)
    outs = torch.stack([d["X"] @ d["We"][e] for e in range(16)], 1)
    chosen = torch.gather(outs, 1, ids.long()[:, :, None].expand(-1, -1, 64))
    H = d["X"] + (w[:, :, None] * chosen).sum(1)
    z = H @ W.t()
    live = s["y"] != -100
    at = torch.where(live, s["y"], 0)
    want = torch.where(live, torch.logsumexp(z, 1) - z.gather(1, at[:, None])[:, 0], 0.0)
    (want.sum() / live.sum()).backward()
    assert int(counts.sum()) == ids.numel() and (counts == torch.bincount(ids.flatten().long(), minlength=16)).all()
    for got, ref in ((loss, want.detach()), (dW, W.grad), (dWr, Wr.grad)):
        assert (got.double() - ref).norm() <= 1e-4 * ref.norm()


def test_a_step_replayed_from_a_graph():
    """Replays with new inputs, with eager work of the same operators between them, equal
    the eager results bit for bit."""
    import torch
    s = make(seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s)
    for seed in (2, 3, 4):
        new = make(seed=seed)
        for k in s:
            s[k].copy_(new[k])
        want = step(new)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        step(make(seed=seed + 10))
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,N,K", [(70, 1501, 256), (300, 2048, 128)])
def test_a_captured_16_bit_head(M, N, K):
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    W = (torch.randn(N, K, generator=g, device="cuda") / 8).bfloat16()
    y = torch.randint(0, N, (M,), generator=g, device="cuda")
    dl = torch.rand(M, generator=g, device="cuda")

    def both():
        loss, lse = gb.linear_cross_entropy(X, W, y, trans_b=True)
        return (loss, lse) + gb.linear_cross_entropy_grad(X, W, y, lse, dl, trans_b=True)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        X.copy_(torch.randn(M, K, generator=g, device="cuda"))
        y.copy_(torch.randint(0, N, (M,), generator=g, device="cuda"))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    """Each call has its own workspace, also when two run at the same time and when a stream
    other than the current one is given."""
    import torch
    sets = [make(M=200, N=3000, seed=20 + i) for i in range(2)]
    want = [step(s) for s in sets]
    grads = []
    for s in sets:
        H, w = s["X"].bfloat16(), s["W"].bfloat16()
        loss, lse = gb.linear_cross_entropy(H, w, s["y"], trans_b=True)
        dl = torch.ones(200, device="cuda") / 200
        grads.append((H, w, s["y"], loss, lse, dl, *gb.linear_cross_entropy_grad(H, w, s["y"], lse, dl, trans_b=True)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [[], []]
        for i in range(2):
            H, w, y, loss, lse, dl, dX, dW = grads[i]
            handle = streams[i].cuda_stream if i else streams[i]    # a stream, or its handle
            got[i] = [*gb.linear_cross_entropy(H, w, y, trans_b=True, stream=handle),
                      *gb.linear_cross_entropy_grad(H, w, y, lse, dl, trans_b=True, stream=handle)]
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] += step(sets[i])
        torch.cuda.synchronize()
        for i in range(2):
            _, _, _, loss, lse, _, dX, dW = grads[i]
            for a, b in zip(got[i], [loss, lse, dX, dW, *want[i]]):
                assert torch.equal(a, b)


def test_wrappers_refuse_on_the_gpu():
    import torch
    X, W = torch.zeros(4, 8, device="cuda"), torch.zeros(16, 8, device="cuda")
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    v = torch.zeros(4, device="cuda")
    bad = [lambda: gb.linear_cross_entropy(X, W, y),                                   # K x N expected
           lambda: gb.linear_cross_entropy(X, W, y[:3], trans_b=True),
           lambda: gb.linear_cross_entropy(X, W, y.int(), trans_b=True),
           lambda: gb.linear_cross_entropy(X, W, y.cpu(), trans_b=True),
           lambda: gb.linear_cross_entropy(X[:1].expand(4, 8), W, y, trans_b=True),
           lambda: gb.linear_cross_entropy(X, W, y, trans_b=True, ignore_index=1 << 63),
           lambda: gb.linear_cross_entropy_grad(X, W, y, v, v[:3], trans_b=True),
           lambda: gb.linear_cross_entropy_grad(X, W, y, v.double(), v, trans_b=True),
           lambda: gb.route(X, 0), lambda: gb.route(X, 65), lambda: gb.route(X[0], 1),
           lambda: gb.route(X, 2, bias=v), lambda: gb.route(X, 2, groups=1 << 33),
           lambda: gb.route_grad(X, y[:, None], v[:, None]),
           lambda: gb.route_grad(X, y.int()[:, None], v[:3, None])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: gb.route(X, 9), lambda: gb.route(X, 2, groups=3), lambda: gb.route(X, 2, groups=2, top_groups=3)):
        with pytest.raises(gb.Gemm355Error):
            f()
    with pytest.raises(TypeError):
        gb.linear_cross_entropy(X, W.half(), y, trans_b=True)
    with pytest.raises(TypeError):
        gb.linear_cross_entropy(X.double(), W.double(), y, trans_b=True)
