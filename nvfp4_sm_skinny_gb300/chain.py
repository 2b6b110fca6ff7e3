"""The per-layer decode chain of the hot path, wired from the public calls.

One layer, at M token rows (HIDDEN H = 8192, POOLED P = 4096):

    partial = h_l @ W_o^T                 o_proj      [8192, 8192]   (sk_gemm_dual_norm)
    s, u    = dual_norm(partial, s)       attention boundary, FP32 residual s in place
    a, a_sf, z = nvfp4(rmsnorm(u @ W_p^T)) pooler     [4096, 8192]   (sk_gemm_rmsnorm_nvfp4)
    h_{l+1} = z @ W_u^T                   unpooler    [8192, 4096]   (sk_gemm_bf16)

The routed experts stand between the pooler and the unpooler (the order of
the pages: o_proj -> attention boundary -> pooler -> experts -> unpooler ->
next boundary). The pages leave them to another package, and by default so does
the chain: the unpooler reads the expert input z in their place. With
``experts`` = E > 0 (a multiple of 16, the router being a GEMM) each layer runs E
routed experts in int8 on z:

    logits  = z @ W_r^T                   router       [E, 4096]      (sk_gemm_bf16)
    ids, g  = top_k of sigmoid(logits) + bias                         (sk_route)
    zq, zs  = int8 codes of z's rows                                  (sk_int8_quantize)
    e       = sum_j g_j W2(silu(W1 z) * W3 z)  [E, 2 I, 4096], [E, 4096, I] (sk_experts_int8)

and the unpooler reads e; the NVFP4 codes a and a_sf have no reader then.

The attention stands before the o_proj (attention width 128 heads of 64, H). The
pages start at its output, and so does the chain by default: the o_proj reads h in
its place. With ``context`` > 0 each layer runs it on h, one token of each of the m
rows per pass, with kv_heads KV heads and a key/value cache held in 4 bits, of
``context`` tokens per row:

    q, k, v = h_l @ W_qkv^T               qkv   [8192 + 2 kv_heads 64, 8192]  (sk_gemm_bf16)
    cache  <- k, v                        at the last position of each row    (sk_kv_append)
    o       = attention of q over it                                          (sk_attn_nvfp4)

and the o_proj reads o. A pass starts by giving the rows the lengths in ``want``
(sk_kv_resize), which the caller sets before it, each row's tokens so far and one
more (0: a row without a sequence; negative: a row that waits). A row that waits, or for
which there are no pages (``row_status``), keeps its cache as it is, and its outputs of
the pass mean nothing. This
module only allocates buffers and calls the binding; every step runs in libsk's
kernels. ``capture()`` records one pass into a CUDA graph (the calls allocate
nothing and are capturable).
"""
from __future__ import annotations

import copy

import torch

import nvfp4_sm_skinny_gb300 as sk
from nvfp4_sm_skinny_gb300 import synth

H = synth.HIDDEN
P = synth.POOLED
HEAD = 64  # columns of a query, key or value head


def layer_bytes(m: int) -> dict:
    """Algorithmic bytes of one layer (each input read once, each output
    written once; internal round trips such as the o_proj partial and the
    pooler's pre-norm y are not counted)."""
    oproj = 2 * H * H + 2 * m * H + 2 * m * H + 3 * 2 * H + 2 * 4 * m * H
    pooler = 2 * P * H + 2 * m * H + 2 * P + 4 + m * P // 2 + m * P // 16 + 2 * m * P
    unpooler = 2 * H * P + 2 * m * P + 2 * m * H
    return dict(oproj_dual=oproj, pooler_nvfp4=pooler, unpooler=unpooler,
                total=oproj + pooler + unpooler)


def gemm_bytes(m: int) -> int:
    """Algorithmic bytes of the three GEMMs of one layer taken alone."""
    return (2 * H * H + 2 * m * H + 2 * m * H) + (2 * P * H + 2 * m * H + 2 * m * P) + \
        (2 * H * P + 2 * m * P + 2 * m * H)


class DecodeChain:
    """Weights and buffers of an L-layer chain at M rows on one device."""

    def __init__(self, layers: int = 48, m: int = 16, device="cuda", eps: float = synth.EPS,
                 gain_center: float = synth.GAIN_CENTER, splits: int = 0,
                 prefetch_next: bool = True, experts: int = 0, top_k: int = 8,
                 inter: int = 1024, context: int = 0, kv_heads: int = 8, page_size: int = 64):
        self.L, self.m, self.device = layers, m, torch.device(device)
        self.experts, self.top_k, self.inter = experts, top_k, inter
        # each GEMM starts the next GEMM's first weight stages towards L2
        self.prefetch_next = prefetch_next
        self.eps, self.gc, self.splits = eps, gain_center, splits
        dev = self.device
        self.w_o, self.w_p, self.w_u = [], [], []
        self.post_w, self.pre_w, self.beta, self.norm_w = [], [], [], []
        for l in range(layers):
            self.w_o.append(synth.chain_weight(l, 0, (H, H), device=dev))
            self.w_p.append(synth.chain_weight(l, 1, (P, H), device=dev))
            self.w_u.append(synth.chain_weight(l, 2, (H, P), device=dev))
            self.post_w.append(synth.chain_weight(l, 3, (H,), std=0.1, mean=1.0, device=dev))
            self.pre_w.append(synth.chain_weight(l, 4, (H,), std=0.1, mean=1.0, device=dev))
            self.beta.append(synth.chain_beta(l, device=dev))
            self.norm_w.append(synth.chain_weight(l, 6, (P,), std=0.1, device=dev))
        self.alpha = 1.0
        self.gs = torch.full((layers, 1), 448.0, dtype=torch.float32, device=dev)
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.h = torch.zeros(layers + 1, m, H, **bf)           # h[0] is the input
        self.s = torch.zeros(m, H, dtype=torch.float32, device=dev)
        self.u = torch.zeros(layers, m, H, **bf)               # dual-norm outputs
        self.z = torch.zeros(layers, m, P, **bf)               # normalised pooler rows
        self.a = torch.zeros(layers, m, P // 2, dtype=torch.uint8, device=dev)
        self.a_sf = torch.zeros(layers, m, P // 16, dtype=torch.uint8, device=dev)
        self.ws_o = torch.zeros(layers, sk.gemm_dual_norm_workspace(m, H), dtype=torch.uint8, device=dev)
        self.ws_p = torch.zeros(layers, sk.gemm_rmsnorm_nvfp4_workspace(m, P), dtype=torch.uint8,
                                device=dev)

        self.context = context
        if context:
            self._add_attention(bf, kv_heads, page_size)
        if experts:
            self._add_experts(bf)

    def _add_attention(self, bf, kv_heads, page_size) -> None:
        L, m, dev, d = self.L, self.m, self.device, HEAD
        self.kv_heads, self.page_size = kv_heads, page_size
        self.heads = [H, kv_heads * d, kv_heads * d]           # columns of q, k and v
        self.w_qkv = [synth.chain_weight(l, 11, (sum(self.heads), H), device=dev) for l in range(L)]
        self.k_gs = torch.full((L, 1), 448.0, dtype=torch.float32, device=dev)
        self.v_gs = torch.full((L, 1), 448.0, dtype=torch.float32, device=dev)
        self.qkv = torch.zeros(L, m, sum(self.heads), **bf)
        self.o = torch.zeros(L, m, H, **bf)                    # attention outputs
        width = -(-self.context // page_size)
        i32 = dict(dtype=torch.int32, device=dev)
        self.cache = torch.zeros(L, m * width, kv_heads, sk.kv_block_bytes(page_size, d), dtype=torch.uint8,
                                 device=dev)
        self.table = torch.full((m, width), -1, **i32)
        self.lens, self.want, self.row_status = (torch.zeros(m, **i32) for _ in range(3))
        self.refs = torch.zeros(m * width, **i32)
        self.ws_a = torch.zeros(sk.attn_nvfp4_workspace(m, 1, H // d, kv_heads, d), dtype=torch.uint8, device=dev)
        self.ws_r = torch.zeros(sk.kv_resize_workspace(m, m * width), dtype=torch.uint8, device=dev)

    def _add_experts(self, bf) -> None:
        L, m, E, I, dev = self.L, self.m, self.experts, self.inter, self.device
        self.w_r, self.bias, self.w13, self.s13, self.w2, self.s2 = ([] for _ in range(6))
        for l in range(L):
            self.w_r.append(synth.chain_weight(l, 7, (E, P), device=dev))
            self.bias.append(synth.chain_weight(l, 8, (E,), std=0.05, device=dev).float())
            for rows, k, role, codes, scales in ((2 * I, P, 9, self.w13, self.s13),
                                                 (P, I, 10, self.w2, self.s2)):
                w = synth.chain_weight(l, role, (E * rows, k), device=dev)
                q, s = sk.int8_quantize(w)
                codes.append(q.view(E, rows, k))
                scales.append(s.view(E, rows))
        self.logits = torch.zeros(L, m, E, **bf)
        self.ids = torch.zeros(L, m, self.top_k, dtype=torch.int32, device=dev)
        self.gates = torch.zeros(L, m, self.top_k, dtype=torch.float32, device=dev)
        self.zq = torch.zeros(L, m, P, dtype=torch.int8, device=dev)
        self.zs = torch.zeros(L, m, dtype=torch.float32, device=dev)
        self.e = torch.zeros(L, m, P, **bf)                    # routed experts' outputs
        self.ws_e = torch.zeros(sk.experts_int8_workspace(m, self.top_k, P, I), dtype=torch.uint8,
                                device=dev)

    def twin(self) -> "DecodeChain":
        """A chain on the same weights and global scales with its own
        activation buffers and workspaces, so that two steps can be in flight
        (one copying its inputs in or results out while the other runs)."""
        t = copy.copy(self)
        names = ("h", "s", "u", "z", "a", "a_sf", "ws_o", "ws_p")
        if self.experts:
            names += ("logits", "ids", "gates", "zq", "zs", "e", "ws_e")
        if self.context:
            names += ("qkv", "o", "cache", "table", "lens", "want", "row_status", "refs", "ws_a", "ws_r")
        for name in names:
            setattr(t, name, torch.zeros_like(getattr(self, name)))
        return t

    def set_input(self, h0: torch.Tensor, s0: torch.Tensor) -> None:
        self.h[0].copy_(h0)
        self.s.copy_(s0)

    def layer_op(self, l: int, op: int, stream=None) -> None:
        """One of the layer's three calls: 0 o_proj + dual norm, 1 pooler +
        RMSNorm + NVFP4, 2 unpooler."""
        if op == 0:
            x = self.o[l] if self.context else self.h[l]
            sk.gemm_dual_norm(x, self.w_o[l], self.s, self.post_w[l], self.alpha,
                              self.beta[l], self.pre_w[l], out=self.u[l], eps_post=self.eps,
                              eps_pre=self.eps, workspace=self.ws_o[l], splits=self.splits,
                              stream=stream)
        elif op == 1:
            sk.gemm_rmsnorm_nvfp4(self.u[l], self.w_p[l], self.norm_w[l], self.eps, self.gc,
                                  self.gs[l], a=self.a[l], a_sf=self.a_sf[l], z_out=self.z[l],
                                  workspace=self.ws_p[l], splits=self.splits, stream=stream)
        else:
            x = self.e[l] if self.experts else self.z[l]
            sk.gemm_bf16(x, self.w_u[l], out=self.h[l + 1], splits=self.splits, stream=stream)

    def routed(self, l: int, stream=None) -> None:
        """The routed experts of layer l: z[l] to e[l] (a chain with experts)."""
        sk.gemm_bf16(self.z[l], self.w_r[l], out=self.logits[l], stream=stream)
        sk.route(self.logits[l], self.top_k, bias=self.bias[l], score="sigmoid", ids=self.ids[l],
                 weights=self.gates[l], stream=stream)
        sk.int8_quantize(self.z[l], q=self.zq[l], scale=self.zs[l], stream=stream)
        sk.experts_int8(self.zq[l], self.zs[l], self.w13[l], self.s13[l], self.w2[l], self.s2[l],
                        self.ids[l], self.gates[l], out=self.e[l], workspace=self.ws_e,
                        stream=stream)

    def rows(self, stream=None) -> None:
        """The rows take the lengths in ``want`` (a chain with attention)."""
        sk.kv_resize(self.want, self.cache, self.table, self.lens, self.refs, self.page_size,
                     status=self.row_status, workspace=self.ws_r, stream=stream)

    def attend(self, l: int, stream=None) -> None:
        """The attention of layer l: h[l] to o[l] (a chain with attention)."""
        m, d = self.m, HEAD
        if self.prefetch_next:
            sk.gemm_prefetch_next(self.w_o[l])
        sk.gemm_bf16(self.h[l], self.w_qkv[l], out=self.qkv[l], splits=self.splits, stream=stream)
        q, k, v = (x.unflatten(1, (1, -1, d)) for x in self.qkv[l].split(self.heads, 1))
        sk.kv_append(k, v, self.k_gs[l], self.v_gs[l], self.cache[l], self.table, self.lens, self.page_size,
                     stream=stream, new_lens=self.want)
        sk.attn_nvfp4(q, self.k_gs[l], self.v_gs[l], self.cache[l], self.table, self.lens, self.page_size,
                      out=self.o[l].view(m, 1, H // d, d), workspace=self.ws_a, stream=stream)

    def next_weight(self, l: int, op: int):
        """The weight of the GEMM after layer l's call `op` (None after the last)."""
        if op == 0:
            return self.w_p[l]
        if op == 1:
            return self.w_r[l] if self.experts else self.w_u[l]
        first = self.w_qkv if self.context else self.w_o
        return first[l + 1] if l + 1 < self.L else None

    def layer(self, l: int, stream=None) -> None:
        if self.context:
            self.attend(l, stream)
        for op in range(3):
            if self.prefetch_next:
                sk.gemm_prefetch_next(self.next_weight(l, op))
            self.layer_op(l, op, stream)
            if op == 1 and self.experts:
                self.routed(l, stream)

    def forward(self, stream=None) -> None:
        if self.context:
            self.rows(stream)
        for l in range(self.L):
            self.layer(l, stream)

    def gemms_only(self, stream=None) -> None:
        """The chain's three GEMMs per layer without their epilogues (same
        shapes, weights and launch configuration), for timing the GEMM kernel."""
        hint = sk.gemm_prefetch_next if self.prefetch_next else (lambda w: None)
        for l in range(self.L):
            hint(self.next_weight(l, 0))
            sk.gemm_bf16(self.h[l], self.w_o[l], out=self.ws_o[l][: self.m * H * 2].view(
                torch.bfloat16).view(self.m, H), splits=self.splits, stream=stream)
            hint(self.w_u[l])  # next here, routed experts or not
            sk.gemm_bf16(self.u[l], self.w_p[l], out=self.ws_p[l][: self.m * P * 2].view(
                torch.bfloat16).view(self.m, P), splits=self.splits, stream=stream)
            hint(self.w_o[l + 1] if l + 1 < self.L else None)  # next here, attention or not
            sk.gemm_bf16(self.z[l], self.w_u[l], out=self.h[l + 1], splits=self.splits,
                         stream=stream)

    def calibrate(self, x_cal: torch.Tensor, s_cal: torch.Tensor) -> None:
        """Sets each layer's NVFP4 global scale to 448 * 6 / amax(z) of one
        calibration pass (set-up, outside any timed region). With attention also
        those of K and V; the pass takes one token of each row, the rows' first, and
        leaves them without any."""
        self.set_input(x_cal, s_cal)
        self.gs.fill_(1.0)
        if self.context:
            self.want.fill_(1)
            self.rows()
        for l in range(self.L):
            self.layer(l)
            amax = self.z[l].float().abs().amax()
            self.gs[l].copy_(2688.0 / amax.clamp_min(1e-30))
            if self.context:
                _, k, v = self.qkv[l].float().abs().split(self.heads, 1)
                self.k_gs[l].copy_(2688.0 / k.amax().clamp_min(1e-30))
                self.v_gs[l].copy_(2688.0 / v.amax().clamp_min(1e-30))
        if self.context:
            self.want.fill_(0)
            self.rows()
        torch.cuda.synchronize(self.device)

    def capture(self, fn=None) -> torch.cuda.CUDAGraph:
        """One pass recorded as a CUDA graph (run once eagerly first)."""
        fn = fn or self.forward
        s = torch.cuda.Stream(self.device)
        s.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(s):
            fn()
        torch.cuda.synchronize(self.device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fn()
        torch.cuda.synchronize(self.device)
        return g

    launches_per_layer = 5          # without experts, which add 7, and attention, which adds 4
    gemm_launches_per_layer = 3
