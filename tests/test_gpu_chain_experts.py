"""The decode chain with routed experts between the pooler and the unpooler: each
step of a layer against the oracle on that layer's GPU inputs, the unpooler's
input, repeats, and a captured pass. (Without experts the chain is the one of
test_gpu_chain.py.)"""
import numpy as np
import pytest
import torch

import oracle
from nvfp4_sm_skinny_gb300 import synth
from oracle import experts as ox
from parity import check_gemm

pytestmark = pytest.mark.gpu
DEV = "cuda"
E, K, I, P, H = 32, 4, 192, synth.POOLED, synth.HIDDEN


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.fixture(scope="module", params=[1, 16])
def chain(request):
    import nvfp4_sm_skinny_gb300 as sk
    from nvfp4_sm_skinny_gb300.chain import DecodeChain

    m = request.param
    c = DecodeChain(layers=2, m=m, device=DEV, experts=E, top_k=K, inter=I)
    c.h0 = synth.normal_bf16((m, H), 1.0, 0).to(DEV)
    c.s0 = synth.normal_f32((m, H), 503).to(DEV)
    c.set_input(c.h0, c.s0)
    c.forward()
    torch.cuda.synchronize()
    yield c
    assert sk.device_status() == 0


def test_layer_matches_the_oracle(chain):
    import nvfp4_sm_skinny_gb300 as sk

    c = chain
    b = synth.bits
    for l in range(c.L):
        zb, wr = b(c.z[l]), b(c.w_r[l])
        acc, absacc = oracle.gemm_f64(zb, wr)
        check_gemm(b(c.logits[l]), oracle.gemm_bf16(zb, wr), acc, absacc, P, sk.gemm_splits(c.m, E, P))
        ids, g = ox.route(f64(c.logits[l]), K, bias=f64(c.bias[l]), score="sigmoid")
        assert np.array_equal(c.ids[l].cpu().numpy(), ids)
        # exponents up to 8, as in the routing tests: (2 * 2 * 8 + 96) roundings
        assert np.abs(f64(c.logits[l])).max() < 8
        assert np.all(np.abs(f64(c.gates[l]) - g) <= g * 128 * ox.U)
        q, s = ox.int8_quantize(f64(c.z[l]))
        assert np.array_equal(c.zq[l].cpu().numpy(), q)
        assert np.all(np.abs(f64(c.zs[l]) - s) <= s * ox.U)
        ref, bound = ox.experts_int8(*(t[l].cpu().numpy() for t in (c.zq, c.zs, c.w13, c.s13, c.w2, c.s2,
                                                                    c.ids, c.gates)))
        assert np.all(np.abs(f64(c.e[l]) - ref) <= bound)
        assert np.abs(ref).max() > 0
        # the unpooler reads the experts' output
        eb, wu = b(c.e[l]), b(c.w_u[l])
        acc, absacc = oracle.gemm_f64(eb, wu)
        check_gemm(b(c.h[l + 1]), oracle.gemm_bf16(eb, wu), acc, absacc, P, sk.gemm_splits(c.m, H, P))


def test_replay_and_twin_repeat_the_eager_pass(chain):
    c = chain
    c.set_input(c.h0, c.s0)
    c.forward()
    torch.cuda.synchronize()
    want = {n: getattr(c, n).clone() for n in ("h", "e", "ids", "gates")}
    graph = c.capture()
    for _ in range(3):
        c.e.fill_(7.0)
        c.h[1:].fill_(7.0)
        c.set_input(c.h0, c.s0)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in want.items():
            assert torch.equal(getattr(c, n), t), n
    t = c.twin()
    t.set_input(c.h0, c.s0)
    t.forward()
    torch.cuda.synchronize()
    assert torch.equal(t.h, want["h"]) and t.e.data_ptr() != c.e.data_ptr()
    assert t.ws_e.data_ptr() != c.ws_e.data_ptr() and t.w13[0] is c.w13[0]
