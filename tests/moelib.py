"""Plain 64-bit forms of the mixture-of-experts operators, on the CPU, for the
tests: each from its formula, row by row."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle

FLT_MAX = float(np.finfo(np.float32).max)


def route(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0):
    """weights float64 [T, k], ids int32 [T, k]."""
    x = np.minimum(np.nan_to_num(logits.double().cpu().numpy(), nan=-np.inf, posinf=np.inf, neginf=-np.inf), FLT_MAX)
    T, E = x.shape
    b = None if bias is None else bias.double().cpu().numpy()
    per = E // groups
    W, I = np.zeros((T, k)), np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        live = x[t] > -np.inf
        s = np.zeros(E)
        if live.any():
            if score == "softmax":
                s[live] = np.exp(x[t][live] - x[t].max())
                s /= s.sum()
            else:
                with np.errstate(over="ignore"):
                    s[live] = 1.0 / (1.0 + np.exp(-x[t][live]))
        c = s.copy() if b is None else s + b
        key = x[t].copy() if b is None else c.copy()
        if b is not None:
            live = live & (c > -np.inf)
        key[~live] = -np.inf
        c[~live] = -np.inf
        if topk_groups < groups:
            val = np.full(groups, -np.inf)
            for g in range(groups):
                v = np.sort((key if group_top == 1 else c)[g * per:(g + 1) * per])[::-1]
                val[g] = v[0]
                if group_top == 2 and per > 1 and v[1] > -np.inf:
                    val[g] += v[1]
            keep = np.argsort(-val, kind="stable")[:topk_groups]
            for g in range(groups):
                if g not in keep:
                    key[g * per:(g + 1) * per] = -np.inf
        best = np.argsort(-key, kind="stable")[:k]
        best = best[key[best] > -np.inf]
        w = s[best]
        if renormalize and w.sum() > 0:
            w = w / w.sum()
        I[t, :len(best)], W[t, :len(best)] = best, w * float(np.float32(scale))
    return W, I


def sort(ids, E):
    """offsets [E + 1], order [P], pos like ids."""
    flat = ids.cpu().numpy().reshape(-1)
    order = [p for e in range(E) for p in np.flatnonzero(flat == e)]
    pos = np.full(flat.size, -1, dtype=np.int32)
    pos[order] = np.arange(len(order))
    full = np.full(flat.size, -1, dtype=np.int32)
    full[:len(order)] = order
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    return offsets, full, pos.reshape(tuple(ids.shape))


def experts(x, wq, sw, offsets, order, top_k, act, int8):
    """float64 [rows, N], NaN where no expert has the row; and the sum of the
    products' magnitudes [rows, all weight rows] (scaled), for tolerances."""
    x = x.float().cpu().to(torch.bfloat16)
    codes, sx = oracle.quant_rows(x.contiguous(), oracle.INT8 if int8 else oracle.E4M3)
    val = codes.view(np.int8).astype(np.float64) if int8 else \
        torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()
    w = wq.cpu().double().numpy() if int8 else wq.cpu().view(torch.float8_e4m3fn).double().numpy()
    sw, off = sw.cpu().double().numpy(), offsets.cpu().numpy()
    rows = x.shape[0] if order is None else order.numel()
    src = np.arange(rows) if order is None else order.cpu().numpy() // top_k
    n_all = w.shape[1]
    N = n_all // 2 if act else n_all
    out, mag = np.full((rows, N), np.nan), np.zeros((rows, n_all))
    for e in range(w.shape[0]):
        a, b = off[e], off[e + 1]
        if b <= a:
            continue
        r = src[a:b]
        v = (val[r] @ w[e].T) * sx.astype(np.float64)[r][:, None] * sw[e]
        mag[a:b] = (np.abs(val[r]) @ np.abs(w[e]).T) * sx.astype(np.float64)[r][:, None] * np.abs(sw[e])
        if act:
            g, u = v[:, :N], v[:, N:]
            with np.errstate(over="ignore"):
                out[a:b] = g / (1.0 + np.exp(-g)) * u
        else:
            out[a:b] = v
    return out, mag


def experts_tolerance(ref, mag, K, act, int8):
    """Error bound of the kernel against the 64-bit form.

    One bf16 rounding (half a step: 2^-8 relative) of a value that carries the
    error of the accumulator and of a few fp32 operations (the two scale
    products, and with the activation the fast exponential and quotient; 2^-19
    together).  int8 accumulators are exact until their conversion to fp32
    (2^-24).  The e4m3 accumulator takes K / 32 steps; each adds 32 products
    and the running sum, every one of the 33 cut off at worst 2^-24 below the
    largest, which is at most `mag`, the sum of the products' magnitudes:
    K * 33 / 32 * 2^-24 * mag, and 64 more roundings where K ranges are joined.
    With the activation each factor's bound passes through the product:
    |d silu / d g| <= 1.1 and |silu(g)| <= |g|."""
    eps = 2.0 ** -24 if int8 else (K * 33 / 32 + 64) * 2.0 ** -24
    if act:
        N = ref.shape[1]
        g, u = mag[:, :N], mag[:, N:]
        acc = (2.1 * eps + 1.1 * eps * eps) * g * u
    else:
        acc = eps * mag
    return np.abs(ref) * (2.0 ** -8 + 2.0 ** -19) + acc + 2.0 ** -133


def combine(h, pos, weights, add):
    h, pos = h.double().cpu().numpy(), pos.cpu().numpy()
    w = weights.double().cpu().numpy()
    T, k = pos.shape
    y = np.zeros((T, h.shape[1])) if add is None else add.double().cpu().numpy().copy()
    mag = np.abs(y)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < h.shape[0]:
                y[t] += w[t, j] * h[pos[t, j]]
                mag[t] += np.abs(w[t, j] * h[pos[t, j]])
    return y, mag


def combine_tolerance(ref, mag, k):
    """Half a bf16 step (2^-8 relative) plus k + 1 fp32 steps of the partial sums."""
    return np.abs(ref) * 2.0 ** -8 + (k + 1) * 2.0 ** -24 * mag * (1 + 2.0 ** -8) + 2.0 ** -133


def close(y, ref, tol, what=""):
    y = y.double().cpu().numpy() if isinstance(y, torch.Tensor) else y
    err = np.abs(y - ref)
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err - tol, -math.inf)), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; at {i}: y={y[i]!r} ref={ref[i]!r} "
                             f"tol={tol[i]!r}")
