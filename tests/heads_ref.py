"""Plain binary64 forms of the vocabulary head's loss and the router's head, with the bounds
their tests hold the kernels to.  numpy only: nothing here is the library's code."""

from __future__ import annotations

import numpy as np

U24 = 2.0 ** -24
# half a step of the storage type, relative to the value
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def round_to(x: np.ndarray, dtype: str) -> np.ndarray:
    """x rounded to the storage type (binary32 values or 16-bit patterns)."""
    x = np.asarray(x, np.float32)
    if dtype == "f32":
        return x
    if dtype == "f16":
        return x.astype(np.float16).view(np.uint16)
    bits = x.view(np.uint32)
    return ((bits + 0x7FFF + ((bits >> 16) & 1)) >> 16).astype(np.uint16)


def widen(b: np.ndarray, dtype: str) -> np.ndarray:
    """Stored values as binary64."""
    if dtype == "f32":
        return b.astype(np.float64)
    if dtype == "f16":
        return b.view(np.float16).astype(np.float64)
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def make_head(M, N, K, dtype, seed, ignore=-100, ignored=True):
    """Stored X (M x K), W (N x K) and labels; rows lean towards their label's weights by
    differing amounts; some rows carry no label."""
    rng = np.random.default_rng(seed)
    W = rng.standard_normal((N, K)) * (1.5 / np.sqrt(max(K, 1)))
    labels = rng.integers(0, N, M) if M else np.zeros(0, np.int64)
    X = rng.standard_normal((M, K)) + rng.uniform(0, 8, (M, 1)) * W[labels]
    if ignored and M > 2:
        labels[rng.random(M) < 0.2] = ignore
        labels[M // 2] = ignore
    return round_to(X, dtype), round_to(W, dtype), labels.astype(np.int64)


def logits(X, W, dtype):
    """(Z, error bound of a binary32 dot product of it) in binary64."""
    x, w = widen(X, dtype), widen(W, dtype)
    K = x.shape[1]
    return x @ w.T, (K + 8) * U24 * (np.abs(x) @ np.abs(w).T)


def xent(X, W, labels, dtype, ignore=-100):
    """(loss, lse, bound of loss, bound of lse) in binary64.  The bound of lse: no
    logit's error is larger than the row's largest (lse moves by a weighted mean of them);
    then, in units of 2^-24, the stored maximum, shifts and result (4 |lse|), the sequential
    sums (N / 256), and 64 for the exponentials' arguments (a weighted mean of |z - m| is at
    most log N), the exponentials, merges and logarithm."""
    Z, e = logits(X, W, dtype)
    N = W.shape[0]
    m = Z.max(1)
    lse = m + np.log(np.exp(Z - m[:, None]).sum(1))
    tol = e.max(1) + U24 * (4 * np.abs(lse) + N / 256 + 64)
    live = (labels != ignore) & (labels >= 0) & (labels < N)
    at = np.where(live, labels, 0)
    r = np.arange(len(labels))
    loss = np.where(labels == ignore, 0.0, np.where(live, lse - Z[r, at], np.nan))
    ltol = np.where(live, tol + e[r, at] + 2 * U24 * (np.abs(lse) + np.abs(Z[r, at])), 0.0)
    return loss, lse, ltol, tol


def xent_grad(X, W, labels, lse, dloss, dtype, ignore=-100, parts=1):
    """(dX, dW as N x K, bound of dX, bound of dW) in binary64, for the given lse.

    dZ = g (p - onehot), p = exp(Z - lse).  An error d of the argument moves p by p d: d is
    the logit's error plus 2^-24 (4 |lse| + 2 |Z| + 16) (the shift by lse, the scaling to
    base 2, the exponential); the subtraction and the product with g round twice more.  dZ is
    rounded to the storage type (half a step of it, and for binary16, whose values are scaled
    so that the largest |g| is at least 2^13, half of the least subnormal, 2^-25, over that
    scale).  The products are summed in binary32 (n + 8 roundings of the sum of magnitudes,
    n their length) and rounded once to the storage type (with its least subnormal)."""
    Z, e = logits(X, W, dtype)
    x, w = widen(X, dtype), widen(W, dtype)
    M, N = Z.shape
    live = (labels != ignore) & (labels >= 0) & (labels < N)
    g = np.where(live, dloss.astype(np.float64), 0.0)
    hot = np.zeros_like(Z)
    hot[np.flatnonzero(live), labels[live]] = 1.0
    lse = np.where(live, lse.astype(np.float64), 0.0)
    x = np.where(live[:, None], x, 0.0)
    Z, e = np.where(live[:, None], Z, 0.0), np.where(live[:, None], e, 0.0)
    p = np.exp(Z - lse[:, None])
    dz = g[:, None] * (p - hot)
    moved = np.expm1(e + U24 * (4 * np.abs(lse[:, None]) + 2 * np.abs(Z) + 16))
    # rounded in two parts, the second is off by half a step of what the first leaves
    half = HALF[dtype] ** parts if dtype != "f32" else 0.0
    err = np.abs(g)[:, None] * p * moved + 3 * U24 * np.abs(dz)
    err += half * (np.abs(dz) + err)
    if dtype == "f16" and np.abs(g).max() > 0:
        err += 2.0 ** -25 * np.abs(g).max() / 2.0 ** 13 * (g != 0)[:, None]
    # below the least normal binary32, 2^-126, p and its product with g may be flushed to zero:
    # p, in [0, 2^-126), is then off by less than 2^-126, and so is g p
    err += 2.0 ** -126 * (1 + np.abs(g)[:, None]) * (g != 0)[:, None]
    tiny = {"f32": 2.0 ** -140, "f16": 2.0 ** -25, "bf16": 2.0 ** -130}[dtype]
    mag = np.abs(dz) + err
    dX, dW = dz @ w, dz.T @ x
    tX = err @ np.abs(w) + (N + 8) * U24 * (mag @ np.abs(w))
    tW = err.T @ np.abs(x) + (M + 8) * U24 * (mag.T @ np.abs(x))
    tX += HALF[dtype] * (np.abs(dX) + tX) + tiny
    tW += HALF[dtype] * (np.abs(dW) + tW) + tiny
    return dX, dW, tX, tW


def scores(x, kind):
    """Softmax or sigmoid of binary64 logits; rows without a finite logit give 0."""
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(m), 0.0, m))
        s = e.sum(1, keepdims=True)
        return e / np.where(s == 0, 1.0, s)


def route(X, dtype, k, kind="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0):
    """(ids, weights, counts) row by row, as the header states them."""
    x = widen(X, dtype)
    rows, E = x.shape
    per = E // groups
    s = scores(x, kind)
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    ids = np.full((rows, k), -1, np.int32)
    wts = np.zeros((rows, k))
    for r in range(rows):
        if np.isnan(x[r]).any() or (kind == "softmax" and np.isposinf(x[r]).any()):
            wts[r] = np.nan
            continue
        with np.errstate(invalid="ignore"):
            c = s[r] + b
            c = np.where((x[r] > -np.inf) & (c > -np.inf), c, -np.inf)
        if top_groups < groups:
            gs = []
            for g in range(groups):
                top = [v for v in sorted(c[g * per:(g + 1) * per], reverse=True)[:group_top] if v > -np.inf]
                gs.append(sum(top) if top else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
            mask = np.ones(E, bool)
            for g in keep:
                mask[g * per:(g + 1) * per] = False
            c = np.where(mask, -np.inf, c)
        by = c if bias is not None else np.where(c > -np.inf, x[r], -np.inf)
        order = [e for e in sorted(range(E), key=lambda e: (-by[e], e)) if c[e] > -np.inf][:k]
        ids[r, :len(order)] = order
        w = s[r][order]
        if renorm:
            t = w.sum()
            w = w / t if t > 0 else np.zeros_like(w)
        wts[r, :len(order)] = w * scale
    counts = np.bincount(ids[ids >= 0], minlength=E).astype(np.int32)
    return ids, wts, counts


def route_grad(X, dtype, ids, dweights, kind="softmax", renorm=False, scale=1.0):
    """(dX, bound) in binary64.  The bound: a score's relative error is r = 2^-24 (4 max|x -
    m| + E / 64 + 16) (argument, exponential, sum, division); each of the at most three sums
    and quotients that follow adds its own 2^-24 (2 k + E / 64 + 16), all of them relative to
    the magnitudes summed; then half a step of the storage type."""
    x = widen(X, dtype)
    rows, E = x.shape
    k = ids.shape[1]
    s = scores(x, kind)
    q = np.float64(np.float32(scale)) * dweights.astype(np.float64)
    dX, tol = np.zeros((rows, E)), np.zeros((rows, E))
    for r in range(rows):
        on = (ids[r] >= 0) & (ids[r] < E)
        e, qq = ids[r][on], q[r][on]
        mag = np.abs(qq)
        if renorm:
            S = s[r][e].sum()
            if S > 0:
                mean, mmag = (qq * s[r][e]).sum() / S, (mag * s[r][e]).sum() / S
                qq, mag = (qq - mean) / S, (mag + mmag) / S
            else:
                qq, mag = np.zeros_like(qq), np.zeros_like(mag)
        ds, dm = np.zeros(E), np.zeros(E)
        np.add.at(ds, e, qq)
        np.add.at(dm, e, mag)
        if kind == "sigmoid":
            dX[r] = ds * s[r] * (1 - s[r])
            # 1 - s cancels: its error is that of s, relative to s
            tol[r] = dm * s[r]
            spread = np.abs(x[r][np.isfinite(x[r])]).max(initial=0.0)
        else:
            dX[r] = s[r] * (ds - (ds * s[r]).sum())
            tol[r] = s[r] * (dm + (dm * s[r]).sum())
            f = x[r][np.isfinite(x[r])]
            spread = f.max() - f.min() if f.size else 0.0
        tol[r] *= U24 * (3 * (4 * spread + E / 64 + 16) + 3 * (2 * k + E / 64 + 16))
    tiny = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}[dtype]
    return dX, tol + HALF[dtype] * (np.abs(dX) + tol) + tiny


def make_router(rows, E, dtype, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    return round_to(rng.standard_normal((rows, E)) * spread, dtype)


__all__ = ["HALF", "U24", "logits", "make_head", "make_router", "round_to", "route", "route_grad",
           "scores", "widen", "xent", "xent_grad"]
