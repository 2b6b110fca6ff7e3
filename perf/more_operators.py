"""The operators of a key/value cache held in 4 bits, as cases to be measured:
appending to it, attention over it, and its pages (growing and shrinking rows,
forking them, moving the pages in use together).

``run`` computes a case's operator in its plain form (elementary torch
operations in FP32, FP64 where a value next to a rounding border decides), or,
where ``own`` is true, by the calls of nvfp4_sm_skinny_gb300. ``exact`` gives
the same outputs from the definition in 64 bits.

The cache of one layer is uint8 [pages, KV heads, block]; a block holds one KV
head's part of a page of ps tokens of d values, in this order: the K codes
[ps, d/2] and V codes [ps, d/2] (two e2m1 codes per byte, the even column in
the low nibble), the K scales [ps, d/16] and the V scales [d/16, ps] (e4m3, one
per 16 columns of a token). A value is code * scale / global scale. table
[rows, width] names the page of each ps tokens of a row, lens [rows] its
tokens, refs [pages] how many rows hold a page.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases ----
def _attn(name, b, t, hq, hk, d, ps, lo, hi, window=0, lse=False):
    return dict(name=name, op="attn", b=b, t=t, hq=hq, hk=hk, d=d, ps=ps, lo=lo, hi=hi,
                window=window, lse=lse)


def _append(name, b, t, hq, hk, d, ps, lo, hi):
    return dict(name=name, op="append", b=b, t=t, hq=hq, hk=hk, d=d, ps=ps, lo=lo, hi=hi)


def _resize(name, rows, family, ps, hk, d, layers, pages, lo, hi, grow):
    return dict(name=name, op="resize", rows=rows, family=family, ps=ps, hk=hk, d=d, layers=layers,
                pages=pages, lo=lo, hi=hi, grow=grow)


def _fork(name, rows, ps, lo, hi, keep):
    return dict(name=name, op="fork", rows=rows, ps=ps, lo=lo, hi=hi, keep=keep)


def _compact(name, rows, ps, hk, d, layers, lo, hi, share):
    return dict(name=name, op="compact", rows=rows, ps=ps, hk=hk, d=d, layers=layers, lo=lo, hi=hi,
                share=share)


def listed():
    return [
        # the first tokens of a single conversation: nothing but latency
        _attn("attn b1 d64 len 200", 1, 1, 128, 8, 64, 64, 200, 200),
        # a batch whose four tokens were drafted, lengths far apart, a sliding window, log sums
        _attn("attn b16 t4 d64 ragged window", 16, 4, 128, 8, 64, 16, 100, 8192, 4096, True),
        # one very long document
        _attn("attn b1 d128 len 131071", 1, 1, 64, 8, 128, 64, 131071, 131071),
        # a large serving batch of ragged lengths
        _attn("attn b64 d128 ragged", 64, 1, 64, 8, 128, 64, 512, 16384),
        # the tokens of one decode step, as they lie in the rows of the qkv product
        _append("append b16 t1 d64", 16, 1, 128, 8, 64, 64, 100, 8192),
        # two prompts written at once
        _append("append b2 t16384 d128", 2, 16384, 64, 8, 128, 32, 16384, 20000),
        # the rows of a decode batch grow by a token each, few of them by a page
        _resize("resize 16 rows by 1", 16, 1, 64, 8, 64, 4, 1024, 100, 2000, 1),
        # samples of the same prompts part: partly filled pages are copied in every layer
        _resize("resize 128 rows of 32 prompts", 128, 4, 64, 8, 128, 16, 4096, 1000, 5000, 4),
        # the beams of a few short searches change places
        _fork("fork 64 rows", 64, 64, 100, 2000, 0.5),
        # a thousand rows, a quarter of them replaced by others
        _fork("fork 1021 rows", 1021, 16, 400, 8000, 0.75),
        # a small pool after its rows have come and gone
        _compact("compact 13 rows", 13, 16, 8, 64, 4, 50, 900, 0.7),
        # a large pool, half of it in use, all layers
        _compact("compact 160 rows", 160, 64, 8, 128, 16, 200, 4000, 0.5),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "resize", "fork", "compact"])
    d, ps = rng.choice([64, 128]), rng.choice([16, 32, 64])
    hk = rng.choice([1, 2, 4, 8, 8, 5])
    if op in ("attn", "append"):
        hq = hk * rng.choice([1, 2, 4, 7, 8, 16])
        b, t = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4, 8])
        most = 4 * 10 ** 9 // (b * t * hq * d) if op == "attn" else 32768 // b
        hi = _log(rng, 16, min(131071, 300000 // b, most))
        lo = _log(rng, 1, hi)
        if op == "append":
            t = _log(rng, 1, hi)
            return dict(op=op, b=b, t=t, hq=hq, hk=hk, d=d, ps=ps, lo=lo, hi=hi)
        return dict(op=op, b=b, t=t, hq=hq, hk=hk, d=d, ps=ps, lo=lo, hi=hi,
                    window=rng.choice([0, 0, _log(rng, 1, hi)]), lse=rng.random() < 0.5)
    lo = _log(rng, 1, 2000)
    hi = lo + _log(rng, 1, 2000)
    if op == "resize":
        family = rng.choice([1, 2, 4, 8])
        rows = family * _log(rng, 1, 128 // family)
        pages = sum(_ceil(n, ps) for n in _lengths(rows // family, lo, hi)) + 5 * rows + 1
        return dict(op=op, rows=rows, family=family, ps=ps, hk=hk, d=d, layers=_log(rng, 1, 8),
                    pages=pages, lo=lo, hi=hi, grow=_log(rng, 1, 64))
    if op == "fork":
        return dict(op=op, rows=_log(rng, 1, 1021), ps=ps, lo=lo, hi=hi, keep=rng.random())
    return dict(op=op, rows=_log(rng, 1, 160), ps=ps, hk=hk, d=d, layers=_log(rng, 1, 8), lo=lo,
                hi=hi, share=0.3 + 0.6 * rng.random())


def _lengths(count, lo, hi):
    """Lengths from lo to hi, evenly spread over their logarithm."""
    return [int(round(lo * (hi / lo) ** (i / max(1, count - 1)))) for i in range(count)][::-1]


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------- the cache's form ----
def _parts(cache, ps, d):
    """Views of a cache [..., block]: K codes, V codes [..., ps, d/2], K scales
    [..., ps, d/16], V scales [..., d/16, ps]."""
    code, scale = ps * d // 2, ps * d // 16
    kc, vc, ks, vs = cache.split([code, code, scale, scale], -1)
    return (kc.unflatten(-1, (ps, d // 2)), vc.unflatten(-1, (ps, d // 2)),
            ks.unflatten(-1, (ps, d // 16)), vs.unflatten(-1, (d // 16, ps)))


def _f32(x):
    """FP64 values rounded to FP32: one FP32 operation of the definition."""
    return x.float().double()


def _nvfp4(z, gs):
    """Codes [..., d/2] and scales [..., d/16] (both uint8) of z [..., d]. The
    definition rounds every step to FP32; a code may turn on such a rounding, and
    torch divides by a number through its reciprocal, so the steps are in FP64."""
    z, gs = z.double().unflatten(-1, (-1, 16)), gs.double()
    amax = z.abs().amax(-1)
    sf = _f32(_f32(amax / 6) * gs).clamp_max(448).float().to(torch.float8_e4m3fn)
    wide = sf.double()
    one = _f32(1 / _f32(wide * _f32(1 / gs))).masked_fill(wide == 0, 0)
    y = _f32(z * one.unsqueeze(-1)).float()
    m = y.abs()
    code = (m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)
    code = (code + 8 * torch.signbit(y).byte()).flatten(-2)
    return code[..., ::2] + 16 * code[..., 1::2], sf.view(torch.uint8)


def _values(codes, scales, dtype):
    """code * scale of codes [..., d/2] and scales [..., d/16]."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)  # of a byte
    v = pair[codes.int()].flatten(-2)
    return v.unflatten(-1, (-1, 16)).mul_(scales.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1)).flatten(-2)


# --------------------------------------------------------------- inputs ----
def _table(lens, ps, width, pages, g):
    """Rows of pages in a random order, none of them twice; -1 behind a row's end."""
    used = [_ceil(n, ps) for n in lens]
    order = torch.randperm(pages, generator=g, device=DEV)[: sum(used)].int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV) < torch.tensor(used, device=DEV).unsqueeze(1)] = order
    return table


def _prepare_cache(s, case, seed, g):
    b, t, hq, hk, d, ps = (case[n] for n in ("b", "t", "hq", "hk", "d", "ps"))
    lens = _lengths(b, case["lo"], case["hi"])
    pages, width = sum(_ceil(n, ps) for n in lens) + 3, _ceil(max(lens), ps) + 1
    s["table"], s["lens"] = _table(lens, ps, width, pages, g), torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["k_gs"], s["v_gs"] = (300 + 200 * torch.rand(1, generator=g, device=DEV) for _ in range(2))
    rows = torch.randn(b * t, (hq + 2 * hk) * d, generator=g, device=DEV).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = (x.view(b, t, -1, d) for x in rows.split([hq * d, hk * d, hk * d], 1))
    s["cache"] = torch.randint(0, 256, (pages, hk, ps * d * 9 // 8), generator=g, device=DEV, dtype=torch.uint8)
    if case["op"] == "append":
        return
    s["q"].mul_(2)  # scores that tell keys apart
    parts = _parts(s["cache"], ps, d)
    for at in range(0, pages, 2048):
        kc, vc, ks, vs = (p[at:at + 2048] for p in parts)
        for codes, scales, gs in ((kc, ks, s["k_gs"]), (vc, vs.transpose(-1, -2), s["v_gs"])):
            c, sf = _nvfp4(torch.randn(*codes.shape[:-1], d, generator=g, device=DEV).bfloat16(), gs)
            codes.copy_(c)
            scales.copy_(sf)
    # behind a row's last token its page holds what is left from others: scales that are no number
    last = s["table"].gather(1, ((s["lens"].long() - 1) // ps).unsqueeze(1)).squeeze(1).long()
    behind = torch.zeros(pages, 1, ps, 1, dtype=torch.bool, device=DEV)
    behind[last, 0, :, 0] = torch.arange(ps, device=DEV) > ((s["lens"] - 1) % ps).unsqueeze(1)
    parts[2].masked_fill_(behind, 0x7F)
    parts[3].transpose(-1, -2).masked_fill_(behind, 0xFF)


def _prepare_pages(s, case, seed, g):
    op, rows, ps = case["op"], case["rows"], case["ps"]
    family = case.get("family", 1)
    lens = _lengths(rows // family, case["lo"], case["hi"])
    used = sum(_ceil(n, ps) for n in lens)
    width = _ceil(case["hi"] + case.get("grow", 0), ps) + 1
    pages = case["pages"] if op == "resize" else _ceil(int(used / case.get("share", 1.0)), 1)
    table = _table(lens, ps, width, pages, g).repeat_interleave(family, 0)
    held = torch.bincount(table[table >= 0].long(), minlength=pages).int()
    # table, lens and refs in one buffer, so that a pass starts from the same ones with one copy
    s["book"] = torch.cat([table.flatten(), torch.tensor(lens, dtype=torch.int32, device=DEV).repeat_interleave(family), held])
    s["work"] = torch.empty_like(s["book"])
    s["sizes"] = (rows, width, pages)
    if op == "fork":
        other = torch.randint(0, rows, (rows,), generator=g, device=DEV, dtype=torch.int32)
        stays = torch.rand(rows, generator=g, device=DEV) < case["keep"]
        s["parents"] = torch.where(stays, -1, other)
        return
    s["cache"] = torch.randint(0, 256, (case["layers"], pages, case["hk"], ps * case["d"] * 9 // 8),
                               generator=g, device=DEV, dtype=torch.uint8)
    if op == "resize":
        s["new_lens"] = torch.tensor(_new_lengths(case), dtype=torch.int32, device=DEV)


def _new_lengths(case):
    """Of every 16 rows one has ended, one gives three tokens back, one waits, the others grow."""
    lens = [n for n in _lengths(case["rows"] // case["family"], case["lo"], case["hi"])
            for _ in range(case["family"])]
    return [0 if i % 16 == 5 else max(0, n - 3) if i % 16 == 6 else -1 if i % 16 == 11 else n + case["grow"]
            for i, n in enumerate(lens)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    (_prepare_cache if case["op"] in ("attn", "append") else _prepare_pages)(s, case, seed, g)
    return s


# ------------------------------------------------------------ plain forms ----
def _plain_attn(s):
    b, t, hq, hk, d, ps = (s[n] for n in ("b", "t", "hq", "hk", "d", "ps"))
    width = s["table"].shape[1]
    at = torch.arange(width * ps, device=DEV)
    there = (at < s["lens"].unsqueeze(1)) & (s["table"] >= 0).repeat_interleave(ps, 1)  # [b, keys]
    kc, vc, ks, vs = _parts(s["cache"][s["table"].clamp_min(0).long()], ps, d)  # [b, width, hk, ..]
    k = _values(kc, ks, torch.float32).transpose(1, 2).flatten(2, 3)  # [b, hk, keys, d]
    q = s["q"].float().view(b, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = (q @ k.transpose(2, 3)) * (1 / math.sqrt(d) / s["k_gs"])
    del k
    pos = s["lens"].unsqueeze(1) - t + torch.arange(t, device=DEV)  # [b, t]
    seen = there.unsqueeze(1) & (at <= pos.unsqueeze(2))
    if s["window"]:
        seen &= at > pos.unsqueeze(2) - s["window"]
    seen = seen.repeat_interleave(hq // hk, 1).unsqueeze(1)  # [b, 1, t group, keys]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(3, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = (scores - top).exp()
    total = p.sum(3, keepdim=True)
    v = _values(vc, vs.transpose(-1, -2).contiguous(), torch.float32).transpose(1, 2).flatten(2, 3)
    v = v.masked_fill(~there.unsqueeze(1).unsqueeze(3), 0.0)
    out = (p @ v) / s["v_gs"] / total.masked_fill(total == 0, 1.0)
    out = out.view(b, hk, t, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(torch.bfloat16)
    if not s["lse"]:
        return out
    lse = (top + total.log()).view(b, hk, t, hq // hk).transpose(1, 2).reshape(b, t, hq)
    return out, lse


def _plain_append(s):
    t, d, ps = s["t"], s["d"], s["ps"]
    pos = s["lens"].unsqueeze(1) - t + torch.arange(t, device=DEV)
    row, token = torch.nonzero(pos >= 0, as_tuple=True)
    at = pos[row, token].long()
    page, at = s["table"][row, at // ps].long(), at % ps
    kc, vc, ks, vs = _parts(s["cache"], ps, d)
    kc[page, :, at], ks[page, :, at] = _nvfp4(s["k"][row, token], s["k_gs"])
    vc[page, :, at], vs[page, :, :, at] = _nvfp4(s["v"][row, token], s["v_gs"])
    return s["cache"]


def _plain_resize(new, cache, table, lens, refs, ps):
    rows, width = table.shape
    old, want = lens.long(), torch.where(new < 0, lens, new).long()
    status = torch.where(want > width * ps, 2, 0)
    want = torch.where(status > 0, old, want)
    have, after = -(-old // ps), -(-want // ps)
    grows = want > old
    last = table.gather(1, (have - 1).clamp_min(0).unsqueeze(1)).squeeze(1).long()
    held = refs[last.clamp_min(0)]
    shared = grows & (old % ps != 0) & (held > 1)
    before = ((last.unsqueeze(1) == last) & shared.unsqueeze(1) & shared).tril(-1)
    copies = shared & (before.sum(1) < held - 1)  # the last one that holds it keeps it
    need = torch.where(grows, after - have, 0) + copies
    upto = need.cumsum(0)
    free = torch.nonzero(refs <= 0).squeeze(1)
    refused = (need > 0) & (upto > len(free))
    refused |= shared & ~copies & (before & refused).any(1)
    status = torch.where(refused, 1, status).int()
    after, want = torch.where(refused, have, after), torch.where(refused, old, want)
    copies &= ~refused
    col = torch.arange(width, device=DEV)
    fresh = (col >= have.unsqueeze(1)) & (col < after.unsqueeze(1))
    gone = (col < have.unsqueeze(1)) & (col >= after.unsqueeze(1))
    given = (upto - need + copies).unsqueeze(1) + col - have.unsqueeze(1)
    free = torch.cat([free, free.new_zeros(1)])
    pages = free[given.clamp(0, len(free) - 1)].int()
    into = free[(upto - need).clamp(0, len(free) - 1)]
    refs.index_add_(0, table[gone].long(), torch.full_like(table[gone], -1))
    refs.index_add_(0, last[copies], torch.full_like(last[copies], -1).int())
    refs[pages[fresh].long()] = 1
    refs[into[copies]] = 1
    cache[:, into[copies]] = cache[:, last[copies]]
    table.copy_(torch.where(fresh, pages, torch.where(gone, -1, table)))
    table[copies, have[copies] - 1] = into[copies].int()
    lens.copy_(want)
    return status, table, lens, refs, cache


def _plain_fork(parents, table, lens, refs, ps):
    rows, width = table.shape
    status = torch.where(parents >= rows, 2, 0).int()
    me = torch.arange(rows, device=DEV)
    p = torch.where((parents < 0) | (parents >= rows), me, parents.long())
    used = torch.arange(width, device=DEV) < (-(-lens // ps)).unsqueeze(1)
    moved = (p != me).unsqueeze(1)
    refs.index_add_(0, table[used & moved].long(), torch.full_like(table[used & moved], -1))
    taken = table[p][used[p] & moved]
    refs.index_add_(0, taken.long(), torch.ones_like(taken))
    table.copy_(torch.where(moved, table[p].masked_fill(~used[p], -1), table))
    lens.copy_(lens[p])
    return status, table, lens, refs


def _plain_compact(cache, table, lens, refs, ps):
    live = refs > 0
    count = live.sum()
    number = torch.arange(len(refs), device=DEV)
    holes = torch.nonzero(~live & (number < count)).squeeze(1)
    moved = torch.nonzero(live & (number >= count)).squeeze(1)
    page_map = torch.where(live, number, -1).int()
    page_map[moved] = holes.int()
    cache[:, holes] = cache[:, moved]
    refs[holes] = refs[moved]
    refs[moved] = 0
    used = torch.arange(table.shape[1], device=DEV) < (-(-lens // ps)).unsqueeze(1)
    table.copy_(torch.where(used, page_map[table.clamp_min(0).long()], table))
    return page_map, table, refs, cache


def run(state):
    s, op = state, state["op"]
    if own:
        import nvfp4_sm_skinny_gb300 as sk
    if op == "attn":
        if own:
            out, lse, _ = sk.attn_nvfp4(s["q"], s["k_gs"], s["v_gs"], s["cache"], s["table"], s["lens"],
                                        s["ps"], window=s["window"], lse=True if s["lse"] else None)
            return (out, lse) if s["lse"] else out
        return _plain_attn(s)
    if op == "append":  # codes and scales by the definition's FP32 steps: equal bytes on every side
        if own:
            sk.kv_append(s["k"], s["v"], s["k_gs"], s["v_gs"], s["cache"], s["table"], s["lens"], s["ps"])
            return s["cache"]
        return _plain_append(s)
    rows, width, pages = s["sizes"]
    s["work"].copy_(s["book"])
    table, lens, refs = s["work"].split([rows * width, rows, pages])
    table = table.view(rows, width)
    if op == "resize":
        if own:
            status, _ = sk.kv_resize(s["new_lens"], s["cache"], table, lens, refs, s["ps"])
            return status, table, lens, refs, s["cache"]
        return _plain_resize(s["new_lens"], s["cache"], table, lens, refs, s["ps"])
    if op == "fork":
        if own:
            return sk.kv_fork(s["parents"], table, lens, refs, s["ps"]), table, lens, refs
        return _plain_fork(s["parents"], table, lens, refs, s["ps"])
    if own:
        page_map, _ = sk.kv_compact(s["cache"], table, lens, refs, s["ps"])
        return page_map, table, refs, s["cache"]
    return _plain_compact(s["cache"], table, lens, refs, s["ps"])


# ------------------------------------------------------------------ work ----
def work(case):
    op = case["op"]
    if op in ("attn", "append"):
        b, t, hq, hk, d = (case[n] for n in ("b", "t", "hq", "hk", "d"))
        lens = _lengths(b, case["lo"], case["hi"])
        if op == "append":
            tokens = sum(min(n, t) for n in lens)
            return dict(bytes=tokens * hk * d * 2 * (2 + 9 / 16), flops=tokens * hk * d * 2 * 4)
        w = case["window"] or max(lens)
        read = sum(min(n, w + t - 1) for n in lens)
        pairs = sum(max(0, min(n - j, w)) for n in lens for j in range(t))
        return dict(bytes=read * hk * d * 9 / 8 + b * t * hq * (4 * d + (4 if case["lse"] else 0)),
                    flops=4 * d * hq * pairs)
    ps, rows = case["ps"], case["rows"]
    family = case.get("family", 1)
    lens = [n for n in _lengths(rows // family, case["lo"], case["hi"]) for _ in range(family)]
    if op == "fork":
        entries = sum(_ceil(n, ps) for n in lens) * (1 - case["keep"])
        return dict(bytes=entries * 16 + rows * 16, flops=entries)  # entries and counts, in and out
    used = sum(_ceil(n, ps) for n in lens) // family
    page = case["layers"] * case["hk"] * ps * case["d"] * 9 // 8
    if op == "compact":
        pages = _ceil(int(used / case["share"]), 1)
        return dict(bytes=2 * page * used * (1 - used / pages) + 12 * pages + 8 * used, flops=pages)
    copied = 0
    new = _new_lengths(case)
    for at in range(0, rows, family):
        n = lens[at]
        grown = sum(m > n for m in new[at:at + family])
        copied += min(grown, family - 1) if n % ps else 0
    return dict(bytes=2 * page * copied + 8 * case["pages"] + 16 * rows, flops=case["pages"])


# ---------------------------------------------------------------- 64 bits ----
def _exact_codes(z, gs):
    """The definition of the codes: the nearest e2m1 value, of two the even code."""
    d = z.shape[-1]
    z, gs = z.double().reshape(-1, 16), float(gs)
    sixth = (z.abs().max(1).values / 6).float()
    sf = (sixth.double() * gs).float().clamp(max=448.0).to(torch.float8_e4m3fn)
    back = torch.tensor(1.0 / gs, dtype=torch.float32).item()
    step = (sf.double() * back).float().double()
    y = (z * torch.where(sf.double() > 0, (1 / step).float().double(), 0.0)[:, None]).float().double()
    e = torch.tensor(E2M1, dtype=torch.float64, device=z.device)
    low = (torch.searchsorted(e, y.abs(), right=True) - 1).clamp(0, 6)
    below, above = y.abs() - e[low], e[low + 1] - y.abs()
    code = low + ((above < below) | ((above == below) & (low % 2 == 1)))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).view(-1, d // 2, 2)
    return code[..., 0] | code[..., 1] << 4, sf.view(torch.uint8).view(-1, d // 16)


def _exact_values(codes, scales):
    """The values that codes [n, d/2] with scales [n, d/16] stand for, [n, d]."""
    code = torch.stack([codes & 15, codes >> 4], 2).flatten(1).long()
    e = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)[code & 7]
    byte = scales.long()
    exponent, mantissa = byte >> 3 & 15, (byte & 7).double() / 8
    scale = torch.where(exponent == 0, mantissa * 2.0 ** -6, (1 + mantissa) * 2.0 ** (exponent - 7).double())
    return torch.where(code > 7, -e, e) * scale.repeat_interleave(16, 1)


def _exact_append(s):
    hk, d, ps = s["hk"], s["d"], s["ps"]
    kc, vc, ks, vs = _parts(s["cache"], ps, d)
    for r, n in enumerate(s["lens"].tolist()):
        first = max(0, n - s["t"])
        at = torch.arange(first, n, device=DEV)
        page, at = s["table"][r, at // ps].long(), at % ps
        for x, gs, codes, scales in ((s["k"], s["k_gs"], kc, ks), (s["v"], s["v_gs"], vc, vs.transpose(-1, -2))):
            c, sf = _exact_codes(x[r, s["t"] - (n - first):], gs)
            codes[page, :, at] = c.view(-1, hk, d // 2)
            scales[page, :, at] = sf.view(-1, hk, d // 16)
    return s["cache"]


def _exact_attn(s):
    b, t, hq, hk, d, ps = (s[n] for n in ("b", "t", "hq", "hk", "d", "ps"))
    out = torch.zeros(b, t, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64, device=DEV)
    kc, vc, ks, vs = _parts(s["cache"], ps, d)
    for r, n in enumerate(s["lens"].tolist()):
        at = torch.arange(n, device=DEV)
        page, at = s["table"][r, at // ps].long(), at % ps
        k = _exact_values(kc[page, :, at].flatten(0, 1), ks[page, :, at].flatten(0, 1)) / s["k_gs"].double()
        v = _exact_values(vc[page, :, at].flatten(0, 1), vs[page, :, :, at].flatten(0, 1)) / s["v_gs"].double()
        k, v = (x.view(n, hk, d).transpose(0, 1) for x in (k, v))
        for j in range(t):
            end = n - t + j + 1
            if end <= 0:
                continue
            keys = slice(max(0, end - s["window"]) if s["window"] else 0, end)
            a = torch.einsum("hgd,hkd->hgk", s["q"][r, j].double().view(hk, -1, d), k[:, keys]) / math.sqrt(d)
            w = torch.softmax(a, 2)
            out[r, j] = torch.einsum("hgk,hkd->hgd", w, v[:, keys]).reshape(hq, d)
            lse[r, j] = torch.logsumexp(a, 2).flatten()
    return (out, lse) if s["lse"] else out


def exact(case, seed):
    if case["op"] not in ("attn", "append"):
        return None  # pages are moved and counted: nothing is computed
    s = prepare(case, seed)
    return _exact_attn(s) if case["op"] == "attn" else _exact_append(s)
