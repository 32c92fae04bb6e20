"""Plain 64-bit statements of the operators for rows that choose their
weights, with bounds on the error of a correct fp32 evaluation.  numpy (and
torch's fp64 erf), written from the definitions; nothing here calls the package.

Rounding model: u = 2^-24 is half a step of fp32 relative to the value; a
bf16 result is off by at most 2^-8 of itself on top (half a step)."""

from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


# ------------------------------------------------------------------ routing

def route(logits, k, score, bias=None, groups=1, top_groups=1, renormalise=True, scale=1.0):
    """ids [M, k] (-1: none left) and fp64 weights, row by row."""
    x = np.minimum(np.asarray(logits, dtype=np.float64), float(np.finfo(np.float32).max))
    M, E = x.shape
    per = E // groups
    ids = np.full((M, k), -1, dtype=np.int32)
    weights = np.zeros((M, k))
    for m in range(M):
        open_ = [i for i in range(E) if not np.isnan(x[m, i]) and x[m, i] != -np.inf]
        if score == "softmax":
            top = max((x[m, i] for i in open_), default=0.0)
            e = {i: math.exp(x[m, i] - top) for i in open_}
            total = sum(e.values())
            s = {i: v / total for i, v in e.items()}
        else:
            s = {i: 1.0 / (1.0 + math.exp(-x[m, i])) if x[m, i] > -700 else 0.0 for i in open_}
        c = {i: s[i] + (float(bias[i]) if bias is not None else 0.0) for i in open_}
        open_ = [i for i in open_ if not np.isnan(c[i]) and c[i] != -np.inf]
        if groups > 1:
            value = {}
            for g in range(groups):
                v = sorted((c[i] for i in open_ if i // per == g), reverse=True)[:2]
                if v:
                    value[g] = sum(v)
            kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            open_ = [i for i in open_ if i // per in kept]
        # the score is monotone in the logit: without a bias the logits decide
        rank = (lambda i: (-c[i], i)) if bias is not None else (lambda i: (-x[m, i], i))
        for j, i in enumerate(sorted(open_, key=rank)[:k]):
            ids[m, j], weights[m, j] = i, s[i]
        if renormalise:
            t = weights[m].sum()
            weights[m] = weights[m] / t if t > 0 else 0.0
    return ids, weights * scale


def choice_values(x, score, bias):
    """fp64 choice values of one row of finite logits."""
    x = np.asarray(x, dtype=np.float64)
    s = np.exp(x - x.max()) / np.exp(x - x.max()).sum() if score == "softmax" else 1 / (1 + np.exp(-x))
    return s if bias is None else s + np.asarray(bias, dtype=np.float64)


def plan(ids, E):
    """(order, offsets) of flat ids: a stable sort with the pairs outside
    0..E-1 last."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    return order.astype(np.int32), np.searchsorted(key[order], np.arange(E + 1)).astype(np.int32)


# --------------------------------------------------------- experts' products

def _activate(z, act):
    if act is None:
        return z
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    erf = torch.erf(torch.from_numpy(z / math.sqrt(2.0))).numpy()  # fp64, on the CPU
    return 0.5 * z * (1.0 + erf)


def _affine(x, sx, w, sw, b):
    """Value and error bound of fma(acc, sx sw, b): the exact accumulator
    is rounded to fp32, the scales' product once, the result once."""
    p = (x.astype(np.float64) @ w.astype(np.float64).T) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    z = p if b is None else p + b.astype(np.float64)
    return z, 2.01 * U * np.abs(p) + U * np.abs(z)


def _activation_error(z, dz, act):
    """Error of the activation of a value off by dz: the slope is below
    1.13; the exponential's argument (at most 2.4 |z| (1 + 0.045 z^2), a
    few roundings) moves it by that many units relative to the result; exp2
    and reciprocal are good to one unit each; the erf form adds 7.5e-8 |z|."""
    if act is None:
        return dz
    arg = np.abs(z) * (1 + 0.05 * z * z)
    return 1.13 * dz + (8 * arg + 16) * U * np.abs(_activate(z, act)) + (7.5e-8 * np.abs(z) if act == "gelu_erf" else 0)


def grouped(x, sx, ids, E, w, sw, b=None, act=None, source="by_row", dest="by_pair", w2=None, sw2=None, b2=None,
            dtype="f32"):
    """(Y [pairs, N] fp64, bound, written rows): act(x W_e^T ..) or, with w2,
    act(gate) * up; rows of pairs without a group stay zero."""
    ids = np.asarray(ids)
    k = ids.shape[1] if ids.ndim == 2 else 1
    order, offsets = plan(ids, E)
    N = w.shape[0] // E
    Y, bound = np.zeros((ids.size, N)), np.zeros((ids.size, N))
    written = np.zeros(ids.size, dtype=bool)
    for e in range(E):
        pos = np.arange(offsets[e], offsets[e + 1])
        if pos.size == 0:
            continue
        pair = order[pos]
        src = {"by_row": pair // k, "by_pair": pair, "sorted": pos}[source]
        cols = slice(e * N, (e + 1) * N)
        z, dz = _affine(x[src], sx[src], w[cols], sw[cols], None if b is None else b[cols])
        y, dy = _activate(z, act), _activation_error(z, dz, act)
        if w2 is not None:
            u, du = _affine(x[src], sx[src], w2[cols], sw2[cols], None if b2 is None else b2[cols])
            y, dy = y * u, dy * np.abs(u) + np.abs(y) * du + dy * du + U * np.abs(y * u)
        to = pair if dest == "by_pair" else pos
        Y[to], bound[to], written[to] = y, dy + HALF_STEP[dtype] * (np.abs(y) + dy) + 1e-38, True
    return Y, bound, written


def combine(y, weights, ids, E, dtype="f32"):
    """sum_j w y in fp32 fused multiply-adds, rounded once."""
    M, k = ids.shape
    used = ((ids >= 0) & (ids < E)).astype(np.float64)
    w = weights.astype(np.float64) * used
    y = np.where(used.reshape(-1, 1) > 0, y.astype(np.float64), 0.0).reshape(M, k, y.shape[1])
    out = (w[..., None] * y).sum(1)
    err = k * U * (np.abs(w)[..., None] * np.abs(y)).sum(1)
    return out, err + HALF_STEP[dtype] * (np.abs(out) + err) + 1e-38


# ------------------------------------------------------------------ adapters

def lora(x, a, b, scales, y, ids, dtype="f32"):
    """y + scale (x A^T) B^T per row, and the bound: K fp32 additions of the
    first sum, the split of T into two (bf16) or three bf16 terms, r additions
    per term of the second, the final fused multiply-add and rounding."""
    E, r, K = a.shape
    terms = 3 if dtype == "f32" else 2
    out = y.astype(np.float64).copy()
    bound = np.zeros_like(out)
    for e in range(E):
        rows = np.nonzero(np.asarray(ids) == e)[0]
        if rows.size == 0:
            continue
        X, A, B = x[rows].astype(np.float64), a[e].astype(np.float64), b[e].astype(np.float64)
        s = float(scales[e])
        t = X @ A.T
        dt = K * U * (np.abs(X) @ np.abs(A).T)
        dt = dt + 2.0 ** (-8 * terms) * np.abs(t)
        out[rows] += s * (t @ B.T)
        bound[rows] = abs(s) * (dt @ np.abs(B).T + (r * terms + 2) * U * ((np.abs(t) + dt) @ np.abs(B).T))
    return out, bound + HALF_STEP[dtype] * (np.abs(out) + bound) * (np.asarray(ids)[:, None] >= 0) + 1e-38
