"""The int8 routed experts in 64 bits (numpy): routing, int8 quantization of
rows, the int8 product and the experts' products. No counterpart on the pages;
include/sk.h states the formulas (sk_route, sk_int8_quantize, sk_gemm_int8,
sk_experts_int8). Test infrastructure, like the rest of this package: it shares
no code with the CUDA path. Pinned by tests/test_oracle_experts.py.

Float inputs are FP32 or FP64 arrays (BF16 values widened by the caller).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a unit in the last place of FP32, relative


def route(logits, top_k, bias=None, n_groups=1, topk_groups=1, score="softmax", renormalize=True,
          scale=1.0):
    """(ids [m, top_k], weights [m, top_k] FP64), one row at a time."""
    logits = np.asarray(logits, np.float64)
    m, n = logits.shape
    ids = np.full((m, top_k), -1, np.int32)
    weights = np.zeros((m, top_k))
    per = n // n_groups
    for i in range(m):
        a = logits[i]
        can = ~(np.isnan(a) | (a == -np.inf))
        p = np.zeros(n)
        if can.any():
            if score == "softmax":
                top = a[can].max()
                with np.errstate(invalid="ignore"):
                    d = np.where(a[can] == top, 0.0, a[can] - top)
                p[can] = np.exp(d) / np.exp(d).sum()
            else:
                with np.errstate(over="ignore"):
                    p[can] = 1.0 / (1.0 + np.exp(-a[can]))
        v = a if bias is None else p + np.asarray(bias, np.float64)
        can &= ~(np.isnan(v) | (v == -np.inf))
        if n_groups > 1:
            value = []
            for g in range(n_groups):
                best = sorted((float(v[e]) for e in range(g * per, (g + 1) * per) if can[e]), reverse=True)
                if best:
                    value.append((-(best[0] if bias is None else sum(best[:2])), g))
            kept = {g for _, g in sorted(value)[:topk_groups]}
            can &= np.array([e // per in kept for e in range(n)])
        order = sorted((-float(v[e]), e) for e in range(n) if can[e])[:top_k]
        for j, (_, e) in enumerate(order):
            ids[i, j], weights[i, j] = e, p[e]
        total = weights[i].sum()
        if renormalize:
            weights[i] = weights[i] / total if total > 0 else 0.0
    return ids, weights * scale


def int8_quantize(z):
    """(q int8, scale FP64 [m]) of each row of z."""
    z = np.asarray(z, np.float64)
    amax = np.abs(z).max(1)
    fine = np.isfinite(amax)
    div = np.where(fine & (amax > 0), amax, 1.0)[:, None]
    q = np.where((fine & (amax > 0))[:, None], np.rint(127.0 * np.where(fine[:, None], z, 0.0) / div), 0.0)
    return q.astype(np.int8), np.where(fine, amax / 127.0, np.nan)


def gemm_int8(xq, x_scale, wq, w_scale):
    """The product, unrounded (FP64; the integer sum is exact)."""
    s = np.asarray(xq, np.int64) @ np.asarray(wq, np.int64).T
    return s.astype(np.float64) * np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)


def gemm_int8_bound(y):
    """How far a BF16 result may be from ``y``: the FP32 sum, two FP32 products
    (2^-24 each) and the rounding to BF16 (2^-8), or half its smallest step."""
    return np.abs(y) * (2.0 ** -8 + 4 * U) + 2.0 ** -134


def experts_int8(xq, x_scale, w13, s13, w2, s2, ids, weights):
    """(y [m, hidden] FP64, bound): the routed experts' output and how far a
    BF16 result with FP32 steps may be from it.

    The FP32 activation has a relative error of at most c = (6 |gate| + 32)
    2^-24: three roundings in each of gate and up; exp(-gate), whose argument's
    error grows by |gate|, twice for the pair of an element and the row's
    largest; the functions' own ulps. So a code may differ by one where the exact
    quotient is that near to half an integer, which moves an output by at most
    |w2| hs s2; hs differs by c too. The sum over the choices adds (top_k + 4)
    2^-24 of the summands' magnitudes, the result 2^-8.
    """
    m, top_k = ids.shape
    n_experts, hidden, inter = w2.shape
    y, off, mag = (np.zeros((m, hidden)) for _ in range(3))
    for i in range(m):
        for j in range(top_k):
            e = int(ids[i, j])
            if not 0 <= e < n_experts:
                continue
            h = gemm_int8(xq[i:i + 1], x_scale[i:i + 1], w13[e], s13[e])[0]
            gate, up = h[:inter], h[inter:]
            with np.errstate(over="ignore"):
                act = gate / (1.0 + np.exp(-gate)) * up
            q, hs = int8_quantize(act[None])
            o = gemm_int8(q, hs, w2[e], s2[e])[0]
            g = float(weights[i, j])
            y[i] += g * o
            c = (6 * np.abs(gate).max() + 32) * U
            amax = np.abs(act).max()
            quot = 127.0 * act / amax if amax > 0 else np.zeros(inter)
            near = np.abs(np.abs(quot - np.floor(quot)) - 0.5) <= np.abs(quot) * c
            flips = np.abs(w2[e][:, near].astype(np.float64)).sum(1) * hs[0] * np.abs(s2[e].astype(np.float64))
            off[i] += abs(g) * (flips * (1 + c) + np.abs(o) * (c + 4 * U))
            mag[i] += abs(g) * (np.abs(o) + flips)
    off += mag * (top_k + 4) * U
    return y, off + (np.abs(y) + off) * 2.0 ** -8 + 2.0 ** -134
