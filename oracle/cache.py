"""The key/value cache held in 4 bits, in 64 bits (numpy): its layout, appending,
attention and the pages, one row at a time as include/sk.h states them
(sk_kv_append, sk_attn_nvfp4, sk_kv_resize, sk_kv_fork, sk_kv_compact). No
counterpart on the pages. Test infrastructure, like the rest of this package: it
shares no code with the CUDA path. Pinned by tests/test_oracle_cache.py.

A cache is uint8 [pages, kv_heads, block] (of all layers: [layers, ...]); BF16 inputs
are their 16-bit words for ``append`` and widened values elsewhere.
"""
from __future__ import annotations

import numpy as np

import oracle


def parts(cache, ps, d):
    """Views of a cache [..., block]: K codes, V codes [..., ps, d/2], K scales
    [..., ps, d/16], V scales [..., d/16, ps]."""
    code, scale = ps * d // 2, ps * d // 16
    assert cache.shape[-1] == 2 * (code + scale)

    def at(lo, n, shape):
        return _split(cache[..., lo:lo + n], shape)

    return (at(0, code, (ps, d // 2)), at(code, code, (ps, d // 2)),
            at(2 * code, scale, (ps, d // 16)), at(2 * code + scale, scale, (d // 16, ps)))


def _split(v, shape):
    """v [..., a * b] as a view [..., a, b]."""
    s = v.strides
    return np.lib.stride_tricks.as_strided(v, v.shape[:-1] + shape, s[:-1] + (shape[1] * s[-1], s[-1]))


def append(k, v, k_gs, v_gs, cache, table, lens, ps, new_lens=None, fresh=None):
    """A copy of ``cache`` with the tokens k, v (BF16 bits [b, t, hk, d]) in it: the last
    fresh[i] of rows that have the length new_lens[i]."""
    b, t, hk, d = k.shape
    out = cache.copy()
    kc, vc, ks, vs = parts(out, ps, d)
    for i in range(b):
        if new_lens is not None and (lens[i] != new_lens[i] or lens[i] > table.shape[1] * ps):
            continue
        for j in range(t):
            pos = int(lens[i]) - t + j
            if fresh is not None and t - j > fresh[i]:
                continue
            if not 0 <= pos < table.shape[1] * ps:
                continue
            page, at = int(table[i, pos // ps]), pos % ps
            if not 0 <= page < len(cache):
                continue
            kc[page, :, at], ks[page, :, at] = oracle.nvfp4_quantize(k[i, j], k_gs)
            vc[page, :, at], vs[page, :, :, at] = oracle.nvfp4_quantize(v[i, j], v_gs)
    return out


def keys(cache, row, n, ps, d, gs, which):
    """(values [hk, n, d] FP64, there [n]) of the first n tokens of a row of the
    table: K (which 0) or V (1); tokens without a page are not there (0)."""
    hk = cache.shape[1]
    p = parts(cache, ps, d)
    codes, scales = p[which], p[2 + which]
    x = np.zeros((hk, n, d))
    there = np.zeros(n, bool)
    for first in range(0, n, ps):
        page, m = int(row[first // ps]), min(ps, n - first)
        if not 0 <= page < len(cache):
            continue
        there[first:first + m] = True
        for h in range(hk):
            sc = scales[page, h].T[:m] if which else scales[page, h, :m]
            x[h, first:first + m] = oracle.nvfp4_dequant(np.ascontiguousarray(codes[page, h, :m]),
                                                         np.ascontiguousarray(sc))
    return x / float(np.float32(gs)), there


def attn(q, k_gs, v_gs, cache, table, lens, ps, scale=None, window=0):
    """(out, lse, size, reach, mass): attention in FP64 of q [b, t, hq, d]; what
    rounding errors go with: size is sum_k p |v| / sum_k p, reach the largest
    sum_c |scale q K| of a key that is seen, mass the sum of their |v|."""
    b, t, hq, d = q.shape
    hk = cache.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, size, mass = (np.zeros((b, t, hq, d)) for _ in range(3))
    lse, reach = np.full((b, t, hq), -np.inf), np.zeros((b, t, hq))
    for i in range(b):
        n = min(max(int(lens[i]), 0), table.shape[1] * ps)
        kk, there = keys(cache, table[i], n, ps, d, k_gs, 0)
        vv, _ = keys(cache, table[i], n, ps, d, v_gs, 1)
        for j in range(t):
            pos = int(lens[i]) - t + j
            at = np.arange(n)
            seen = there & (at <= pos) & (at > pos - window if window else True)
            if not seen.any():
                continue
            for h in range(hq):
                c = h // (hq // hk)
                s = scale * (kk[c, seen] @ q[i, j, h])
                p = np.exp(s - s.max())
                out[i, j, h] = p @ vv[c, seen] / p.sum()
                size[i, j, h] = p @ np.abs(vv[c, seen]) / p.sum()
                mass[i, j, h] = np.abs(vv[c, seen]).sum(0)
                lse[i, j, h] = s.max() + np.log(p.sum())
                reach[i, j, h] = np.abs(scale) * (np.abs(kk[c, seen]) @ np.abs(q[i, j, h])).max()
    return out, lse, size, reach, mass


def resize(new_lens, cache, table, lens, refs, ps):
    """(status, cache, table, lens, refs) after sk_kv_resize: one row after another,
    pages taken from those that are free before the call."""
    cache, table, lens, refs = cache.copy(), table.copy(), lens.copy(), refs.copy()
    width = table.shape[1]
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    given = np.zeros_like(refs)  # given back: free after the call
    status = np.zeros(len(lens), np.int32)
    short = False
    for i in range(len(lens)):
        old, want = int(lens[i]), int(new_lens[i])
        if not 0 <= old <= width * ps or want > width * ps:
            status[i] = 2
            continue
        if want < 0 or want == old:
            continue
        have, after = -(-old // ps), -(-want // ps)
        if want < old:
            for c in range(after, have):
                if 0 <= table[i, c] < len(refs):
                    given[table[i, c]] += 1
                table[i, c] = -1
            lens[i] = want
            continue
        last = int(table[i, have - 1]) if old % ps else -1
        copy = 0 <= last < len(refs) and refs[last] > 1
        need = after - have + copy
        if need and (short or need > len(free)):
            short, status[i] = True, 1
            continue
        if copy:
            page = free.pop(0)
            cache[:, page] = cache[:, last]
            refs[last] -= 1
            refs[page] = 1
            table[i, have - 1] = page
        for c in range(have, after):
            page = free.pop(0)
            refs[page] = 1
            table[i, c] = page
        lens[i] = want
    return status, cache, table, lens, refs - given


def fork(parents, table, lens, refs, ps):
    """(status, table, lens, refs) after sk_kv_fork."""
    old, old_lens = table.copy(), lens.copy()
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    status = np.zeros(len(lens), np.int32)
    width = table.shape[1]

    def used(i):
        return -(-min(max(int(old_lens[i]), 0), width * ps) // ps)

    for i, p in enumerate(parents):
        if p >= len(lens):
            status[i] = 2
        if p < 0 or p >= len(lens) or p == i:
            continue
        for page in old[i, : used(i)]:
            if 0 <= page < len(refs):
                refs[page] -= 1
        for page in old[p, : used(p)]:
            if 0 <= page < len(refs):
                refs[page] += 1
        table[i] = -1
        table[i, : used(p)] = old[p, : used(p)]
        lens[i] = old_lens[p]
    return status, table, lens, refs


def compact(cache, table, lens, refs, ps):
    """(page_map, cache, table, refs) after sk_kv_compact."""
    cache, table, refs = cache.copy(), table.copy(), refs.copy()
    count = int((refs > 0).sum())
    holes = [p for p in range(count) if refs[p] <= 0]
    moved = [p for p in range(count, len(refs)) if refs[p] > 0]
    page_map = np.where(refs > 0, np.arange(len(refs)), -1).astype(np.int32)
    for p, to in zip(moved, holes):
        cache[:, to] = cache[:, p]
        refs[to], refs[p] = refs[p], 0
        page_map[p] = to
    for i in range(len(lens)):
        for c in range(-(-min(max(int(lens[i]), 0), table.shape[1] * ps) // ps)):
            if 0 <= table[i, c] < len(refs):
                table[i, c] = page_map[table[i, c]]
    return page_map, cache, table, refs
