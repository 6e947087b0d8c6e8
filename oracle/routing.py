"""Float64 definitions of the expert routing, its gradient, and the int8 product
and quantisation (test infrastructure; shares no code with the CUDA path).

Routing: s = softmax(l) or sigmoid(l), c = s + bias; groups by their best or the
sum of their two best c; the topk best experts of the kept groups, ties to the
lowest index (of experts and of groups), compared by logits where there is no
bias; weights scale * s, optionally divided by their sum over the chosen ones.
"""
from __future__ import annotations

import numpy as np


def scores(l: np.ndarray, score: str) -> np.ndarray:
    """softmax or sigmoid of float64 rows; a row of -inf gives zeros."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            e = np.exp(-np.abs(l))
            return np.where(l >= 0, 1 / (1 + e), e / (1 + e))
        top = l.max(axis=1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total == 0, 1.0, total)


def chosen_weights(l: np.ndarray, ids: np.ndarray, score: str, renormalize: bool, scale: float) -> np.ndarray:
    """Weights of the given experts (-1: 0), from log scores so that none underflows before the division."""
    none = ids < 0
    at = np.where(none, 0, ids)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if score == "softmax":
            top = l.max(axis=1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0.0)
            log_s = l - top - np.log(np.exp(l - top).sum(axis=1, keepdims=True))
        else:
            log_s = -np.logaddexp(0.0, -l)
        s = np.where(none, -np.inf, np.take_along_axis(log_s, at, axis=1))
        if renormalize:
            top = s.max(axis=1, keepdims=True)
            e = np.exp(s - np.where(np.isneginf(top), 0.0, top))
            total = e.sum(axis=1, keepdims=True)
            w = e / np.where(total == 0, 1.0, total)
        else:
            w = np.exp(s)
    return np.where(none, 0.0, scale * w)


def moe_gate(logits, topk, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=False,
             scale=1.0):
    """(ids int32 [T, topk], weights float64 [T, topk], bad rows [T])."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    bad = np.isnan(l).any(axis=1) | np.isposinf(l).any(axis=1)
    dead = np.isneginf(l)
    key = group_by = l
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        bad |= np.isnan(b).any() or np.isposinf(b).any()
        dead = dead | np.isneginf(b)[None]
        key = group_by = scores(l, score) + b
    elif n_group > 1 and group_top > 1:
        group_by = scores(l, score)
    ids = np.full((T, topk), -1, dtype=np.int32)
    gsize = E // n_group
    for t in range(T):
        if bad[t]:
            continue
        live = ~dead[t]
        if n_group > 1:
            totals = []
            for g in range(n_group):
                span = slice(g * gsize, (g + 1) * gsize)
                best = np.sort(group_by[t, span][live[span]])[::-1][:group_top]
                totals.append(best.sum() if len(best) else -np.inf)
            order = sorted(range(n_group), key=lambda g: (-totals[g], g))[:topk_group]
            kept = np.isin(np.arange(E) // gsize, order)
            live = live & kept
        pick = sorted(np.nonzero(live)[0], key=lambda e: (-key[t, e], e))[:topk]
        ids[t, :len(pick)] = pick
    w = np.zeros((T, topk))
    ok = (ids >= 0).any(axis=1)
    w[ok] = chosen_weights(l[ok], ids[ok], score, renormalize, scale)
    return ids, w, bad


def moe_gate_backward(logits, ids, d_weights, score="softmax", renormalize=False, scale=1.0):
    """(d_logits, size), both float64 [T, E]: the gradient by its formulas, and the sum of the magnitudes of
    the terms that it is made of, to which rounding errors are relative."""
    l = np.asarray(logits, dtype=np.float64)
    g = np.asarray(d_weights, dtype=np.float64)
    T, E = l.shape
    none = (ids < 0) | (ids >= E)
    at = np.where(none, 0, ids)
    g = np.where(none, 0.0, g)
    d, size = np.zeros((T, E)), np.zeros((T, E))
    if score == "softmax" and not renormalize:
        p = scores(l, score)
        G = np.zeros((T, E))
        for j in range(ids.shape[1]):
            np.add.at(G, (np.arange(T), at[:, j]), g[:, j])
        live = (~none).any(axis=1)
        d[live] = (scale * p * (G - (p * G).sum(axis=1, keepdims=True)))[live]
        size[live] = (abs(scale) * p * (np.abs(G) + (p * np.abs(G)).sum(axis=1, keepdims=True)))[live]
        return d, size
    sel = np.where(none, -np.inf, np.take_along_axis(l, at, axis=1))
    s = scores(sel, "sigmoid")
    slope = scores(-sel, "sigmoid")
    if renormalize:
        r = chosen_weights(l, np.where(none, -1, ids), score, True, 1.0)
        f = abs(scale) * r * (slope if score == "sigmoid" else 1.0)
        v = np.sign(scale) * f * (g - (r * g).sum(axis=1, keepdims=True))
        z = f * (np.abs(g) + (r * np.abs(g)).sum(axis=1, keepdims=True))
    else:
        v = scale * s * slope * g
        z = np.abs(v)
    for j in range(ids.shape[1]):
        rows = np.nonzero(~none[:, j])[0]
        np.add.at(d, (rows, at[rows, j]), v[rows, j])
        np.add.at(size, (rows, at[rows, j]), z[rows, j])
    return d, size


def quantize_int8_per_token(x: np.ndarray):
    """(codes int8, scale float32 [rows]) of float32-valued rows: scale = fp32(amax / 127), codes the integers
    nearest (ties to even) to the exact product x * fp32(127 / amax)."""
    x = np.asarray(x, dtype=np.float32)
    least = np.float32(2.0 ** -126)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.abs(x).max(axis=-1)
        finite = np.isfinite(x).all(axis=-1)
        tiny = amax < np.float32(127) * least
        scale = np.where(tiny, least, amax / np.float32(127)).astype(np.float32)
        inverse = np.where(tiny, np.float32(1) / least, np.float32(127) / amax).astype(np.float32)
        scale = np.where(amax == 0, np.float32(1), scale)
        scale = np.where(finite, scale, np.float32(np.nan))
        # a float32 times a float32 is exact in float64
        codes = np.rint(x.astype(np.float64) * inverse.astype(np.float64)[..., None])
    codes = np.where(finite[..., None], codes, 0)
    return codes.astype(np.int8), scale.astype(np.float32)


def int8_gemm(a: np.ndarray, sa: np.ndarray, b: np.ndarray, sb: np.ndarray) -> np.ndarray:
    """sa[m] * sb[n] * (A . B^T) in float64; the integer sums are exact (below 2^53)."""
    acc = a.astype(np.float64) @ b.astype(np.float64).T
    return acc * sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :]
