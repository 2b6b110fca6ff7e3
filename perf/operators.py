"""The operators of the routed experts, as cases to be measured: routing,
int8 quantization of rows, the int8 matrix product and the experts' products.

``run`` computes a case's operator in its plain form (elementary torch
operations in FP32, FP64 where the order of near-equal scores matters), or,
where ``own`` is true, by the calls of nvfp4_sm_skinny_gb300. ``exact`` gives
the same outputs from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases ----
def _route(name, m, experts, k, groups=1, topk_groups=1, score="softmax", bias=False, dtype="bf16",
           scale=1.0):
    return dict(name=name, op="route", m=m, experts=experts, k=k, groups=groups,
                topk_groups=topk_groups, score=score, bias=bias, dtype=dtype, scale=scale)


def _gemm(name, m, n, k):
    return dict(name=name, op="gemm", m=m, n=n, k=k)


def _experts(name, m, experts, k, hidden, inter, masked=0.0):
    return dict(name=name, op="experts", m=m, experts=experts, k=k, hidden=hidden, inter=inter,
                masked=masked)


def listed():
    return [
        # one token of a small model: nothing but latency
        _route("route m1 e16 k2", 1, 16, 2),
        # a full decode batch, grouped sigmoid scores with a balance bias, BF16 logits of the GEMM
        _route("route m16 e256 k8 grouped", 16, 256, 8, 8, 4, "sigmoid", True, scale=2.5),
        # a long prompt's tokens at once
        _route("route m16384 e256 k8 grouped", 16384, 256, 8, 8, 4, "sigmoid", True, "fp32", 2.5),
        # the pooled rows of a decode batch, before the experts
        dict(name="quantize 16x4096", op="quantize", m=16, n=4096),
        # an o_proj weight, quantized per output channel when a model is loaded
        dict(name="quantize 8192x8192", op="quantize", m=8192, n=8192),
        # the unpooler shard at one token: latency
        _gemm("gemm m1 1024x4096", 1, 1024, 4096),
        # the o_proj shard at a full batch
        _gemm("gemm m16 8192x1024", 16, 8192, 1024),
        # ragged features and K
        _gemm("gemm m5 4100x2064", 5, 4100, 2064),
        # the whole o_proj at a full batch: the weight stream
        _gemm("gemm m16 8192x8192", 16, 8192, 8192),
        # one token through eight experts of the pooled width
        _experts("experts m1 e128 k8 4096/2048", 1, 128, 8, 4096, 2048),
        # a padded batch, odd widths, a quarter of the choices masked
        _experts("experts m7 e60 k4 1040/528", 7, 60, 4, 1040, 528, 0.25),
        # a full batch: most experts are chosen by someone
        _experts("experts m16 e128 k8 4096/2048", 16, 128, 8, 4096, 2048),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "gemm", "experts", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 2 if groups > 1 else 8, 512 // groups)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, experts // groups * topk_groups))
        return dict(op=op, m=_log(rng, 1, 16384), experts=experts, k=k, groups=groups,
                    topk_groups=topk_groups, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp32"]),
                    scale=rng.choice([1.0, 2.5]))
    if op == "quantize":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 16, 8192, 16))
    if op == "gemm":
        return dict(op=op, m=rng.randint(1, 16), n=_log(rng, 16, 8192), k=_log(rng, 64, 8192, 16))
    experts = _log(rng, 8, 128)
    return dict(op=op, m=rng.randint(1, 16), experts=experts, k=rng.randint(1, 8),
                hidden=_log(rng, 256, 4096, 16), inter=_log(rng, 64, 2048, 16),
                masked=rng.choice([0.0, 0.25]))


# --------------------------------------------------------------- inputs ----
def _codes(shape, g):
    """int8 codes of normal values, quantized so that about four sigma fill the range."""
    t = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)
    return t.mul_(31.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, g, unit):
    return (torch.rand(shape, generator=g, device=DEV) + 0.5) * unit


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, m = case["op"], case["m"]
    s = dict(case)
    if op == "route":
        t = torch.randn(m, case["experts"], generator=g, device=DEV) * 1.5
        s["logits"] = t.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["b"] = torch.randn(case["experts"], generator=g, device=DEV) * 0.05 if case["bias"] else None
    elif op == "quantize":
        s["z"] = torch.randn(m, case["n"], generator=g, device=DEV).to(torch.bfloat16)
    elif op == "gemm":
        s["xq"], s["xs"] = _codes((m, case["k"]), g), _scales((m,), g, 1 / 31)
        s["wq"], s["ws"] = _codes((case["n"], case["k"]), g), _scales((case["n"],), g, 0.02 / 31)
    else:
        e, h, i = case["experts"], case["hidden"], case["inter"]
        s["xq"], s["xs"] = _codes((m, h), g), _scales((m,), g, 1 / 31)
        s["w13"], s["s13"] = _codes((e, 2 * i, h), g), _scales((e, 2 * i), g, 0.02 / 31)
        s["w2"], s["s2"] = _codes((e, h, i), g), _scales((e, h), g, 0.02 / 31)
        score, ids = torch.rand(m, e, generator=g, device=DEV).topk(case["k"], dim=1)
        if case["masked"]:
            ids = ids.masked_fill(torch.rand(ids.shape, generator=g, device=DEV) < case["masked"], -1)
        s["ids"], s["g"] = ids.to(torch.int32), score / score.sum(1, keepdim=True)
    return s


# ------------------------------------------------------------ plain forms ----
def _plain_route(s):
    neg = float("-inf")
    a = s["logits"].double()
    m, e = a.shape
    a = torch.where(a.isnan(), neg, a)
    if s["score"] == "softmax":
        top = a.amax(1, keepdim=True)
        p = torch.where(a == top, 0.0, a - top).exp().masked_fill(a == neg, 0.0)
        p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1 / (1 + torch.exp(-a))
    v = a if s["b"] is None else p + s["b"].double()
    v = v.masked_fill((a == neg) | v.isnan(), neg)
    if s["groups"] > 1:
        per = e // s["groups"]
        best = v.view(m, s["groups"], per).sort(2, descending=True).values
        gv = best[..., 0]
        if s["b"] is not None and per > 1:
            gv = torch.where(best[..., 1] == neg, gv, gv + best[..., 1])
        order = gv.sort(stable=True, dim=1, descending=True).indices[:, : s["topk_groups"]]
        keep = torch.zeros_like(gv, dtype=torch.bool).scatter_(1, order, True)
        v = v.masked_fill(~keep.repeat_interleave(per, 1), neg)
    best, ids = v.sort(stable=True, dim=1, descending=True)
    best, ids = best[:, : s["k"]], ids[:, : s["k"]]
    w = p.gather(1, ids).masked_fill(best == neg, 0.0)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0) * s["scale"]
    return ids.masked_fill(best == neg, -1).to(torch.int32), w.float()


def _plain_quantize(z):
    z = z.float()
    amax = z.abs().amax(1, keepdim=True)
    f = torch.where(amax >= 1, 2.0 ** -8, 1.0)  # keeps 127 z finite; a power of two, so exact
    q = torch.round((z * f * 127) / (amax * f)).nan_to_num(0.0).masked_fill(~amax.isfinite(), 0.0)
    return q, torch.where(amax.isfinite(), amax / 127, float("nan"))


def _plain_experts(s):
    m, k = s["ids"].shape
    i = s["inter"]
    ids = s["ids"].long().clamp_min(0).flatten()
    x = (s["xq"].float()).repeat_interleave(k, 0).unsqueeze(2)
    h = torch.bmm(s["w13"][ids].float(), x).squeeze(2)
    h = h * s["xs"].repeat_interleave(k).unsqueeze(1) * s["s13"][ids]
    gate, up = h[:, :i], h[:, i:]
    act = gate / (1 + torch.exp(-gate)) * up
    hq, hs = _plain_quantize(act)
    o = torch.bmm(s["w2"][ids].float(), hq.unsqueeze(2)).squeeze(2) * hs * s["s2"][ids]
    g = s["g"].masked_fill(s["ids"] < 0, 0.0)
    return (o.view(m, k, -1) * g.unsqueeze(2)).sum(1).to(torch.bfloat16)


def run(state):
    s, op = state, state["op"]
    if own:
        import nvfp4_sm_skinny_gb300 as sk

        if op == "route":
            return sk.route(s["logits"], s["k"], bias=s["b"], n_groups=s["groups"],
                            topk_groups=s["topk_groups"], score=s["score"], scale=s["scale"])
        if op == "quantize":
            return sk.int8_quantize(s["z"])  # the codes are whole numbers, equal on every side
        if op == "gemm":
            return sk.gemm_int8(s["xq"], s["xs"], s["wq"], s["ws"])
        return sk.experts_int8(s["xq"], s["xs"], s["w13"], s["s13"], s["w2"], s["s2"], s["ids"],
                               s["g"])[0]
    if op == "route":
        return _plain_route(s)
    if op == "quantize":
        q, scale = _plain_quantize(s["z"])
        return q.to(torch.int8), scale.squeeze(1)
    if op == "gemm":
        return ((s["xq"].float() @ s["wq"].float().T) * s["xs"].unsqueeze(1) * s["ws"]).to(torch.bfloat16)
    return _plain_experts(s)


# ------------------------------------------------------------------ work ----
def work(case):
    op, m = case["op"], case["m"]
    if op == "route":
        e, k = case["experts"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=m * e * size + 8 * m * k + (4 * e if case["bias"] else 0), flops=8 * m * e)
    if op == "quantize":
        n = case["n"]
        return dict(bytes=3 * m * n + 4 * m, flops=3 * m * n)
    if op == "gemm":
        n, k = case["n"], case["k"]
        return dict(bytes=n * k + m * k + 4 * (m + n) + 2 * m * n, flops=2 * m * n * k)
    e, k, h, i = case["experts"], case["k"], case["hidden"], case["inter"]
    picks = min(k, e) * (1 - case["masked"])
    chosen = e * (1 - (1 - picks / e) ** m)  # distinct experts, on average
    return dict(bytes=chosen * (3 * i * h + 4 * (2 * i + h)) + m * (h + 4) + 8 * m * k + 2 * m * h,
                flops=2 * m * picks * 3 * i * h)


# ---------------------------------------------------------------- 64 bits ----
def _exact_route(s):
    a = s["logits"].double().cpu().numpy()
    m, e = a.shape
    b = None if s["b"] is None else s["b"].double().cpu().numpy()
    if s["score"] == "softmax":
        p = np.exp(a - a.max(1)[:, None])
        p /= p.sum(1)[:, None]
    else:
        p = 1 / (1 + np.exp(-a))
    v = a if b is None else p + b
    groups, per = s["groups"], e // s["groups"]
    if groups > 1:
        u = np.sort(v.reshape(m, groups, per), axis=2)
        value = u[:, :, -1] if b is None else u[:, :, -2:].sum(2)
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        v = np.where(np.repeat(rank < s["topk_groups"], per, axis=1), v, -np.inf)
    ids = np.argsort(-v, axis=1, kind="stable")[:, : s["k"]]
    w = np.take_along_axis(p, ids, 1)
    return ids.astype(np.int32), w / w.sum(1)[:, None] * s["scale"]


def _exact_rows(t):
    """int8 codes and scales of each row, from the definition."""
    amax = t.abs().max(1, keepdim=True).values
    return torch.round(t * 127 / torch.where(amax > 0, amax, 1.0)), amax / 127


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "quantize":
        q, scale = _exact_rows(s["z"].double())
        return q.to(torch.int8), scale.squeeze(1)
    if op == "gemm":
        total = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        for at in range(0, case["k"], 1024):
            total += s["xq"][:, at:at + 1024].double() @ s["wq"][:, at:at + 1024].double().T
        return total * torch.outer(s["xs"].double(), s["ws"].double())
    y = torch.zeros(case["m"], case["hidden"], dtype=torch.float64, device=DEV)
    for e in range(case["experts"]):
        tok, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if len(tok) == 0:
            continue
        x = s["xq"][tok].double() * s["xs"][tok].double()[:, None]
        gate, up = (x @ (s["w13"][e].double() * s["s13"][e].double()[:, None]).T).chunk(2, 1)
        q, scale = _exact_rows(gate * torch.sigmoid(gate) * up)
        o = (q * scale) @ (s["w2"][e].double() * s["s2"][e].double()[:, None]).T
        y.index_add_(0, tok, o * s["g"][tok, slot].double()[:, None])
    return y
