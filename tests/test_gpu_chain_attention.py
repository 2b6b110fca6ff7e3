"""The decode chain with attention over the 4-bit cache before the o_proj: each
step of a layer against the oracle on that layer's GPU inputs, over several passes,
eager and from a captured graph. (Without attention the chain is the one of
test_gpu_chain.py.)"""
import numpy as np
import pytest
import torch

import oracle
from nvfp4_sm_skinny_gb300 import synth
from oracle import cache as oc
from parity import check_gemm
from test_gpu_cache import attn_bounds, host

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, D, HK, CONTEXT, PS = synth.HIDDEN, 64, 8, 40, 16


@pytest.fixture(scope="module", params=[1, 5])
def chain(request):
    import nvfp4_sm_skinny_gb300 as sk
    from nvfp4_sm_skinny_gb300.chain import DecodeChain

    m = request.param
    c = DecodeChain(layers=2, m=m, device=DEV, context=CONTEXT, kv_heads=HK, page_size=PS)
    c.h0 = synth.normal_bf16((m, H), 1.0, 0).to(DEV)
    c.s0 = synth.normal_f32((m, H), 503).to(DEV)
    c.calibrate(c.h0, c.s0)
    yield c
    assert sk.device_status() == 0


def inputs(c, step):
    c.set_input(synth.normal_bf16((c.m, H), 1.0, 700 + step).to(DEV), synth.normal_f32((c.m, H), 800 + step).to(DEV))


def test_rows_are_empty_after_calibration(chain):
    c = chain
    assert not c.lens.any() and not c.refs.any() and (c.table == -1).all()
    assert (c.k_gs != 448).all() and torch.isfinite(c.k_gs).all() and torch.isfinite(c.v_gs).all()


def test_passes_match_the_oracle(chain):
    import nvfp4_sm_skinny_gb300 as sk

    c = chain
    b = synth.bits
    skip = 0 if c.m == 1 else 3  # a row of the batch without a sequence
    start = [0, 0, 7, 0, 15][: c.m]  # rows that begin with tokens of a prompt: zeros here
    c.want.copy_(torch.tensor(start, dtype=torch.int32))
    c.cache.zero_()
    c.rows()
    graph = None
    for step in range(20):
        inputs(c, step)
        c.want.copy_(torch.tensor([0 if i == skip and c.m > 1 else start[i] + step + 1 for i in range(c.m)],
                                  dtype=torch.int32))
        before = c.cache.cpu().numpy()
        if step == 2:
            graph = c.capture()  # runs the pass once, too
        if graph is None:
            c.forward()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert not c.row_status.any() and torch.equal(c.lens, c.want)
        table, lens = c.table.cpu().numpy(), c.lens.cpu().numpy()
        for l in range(c.L):
            hb, w = b(c.h[l]), b(c.w_qkv[l])
            if step == 0:
                acc, absacc = oracle.gemm_f64(hb, w)
                check_gemm(b(c.qkv[l]), oracle.gemm_bf16(hb, w), acc, absacc, H, sk.gemm_splits(c.m, w.shape[0], H))
            q, k, v = (x.unflatten(1, (1, -1, D)) for x in c.qkv[l].split(c.heads, 1))
            cache = c.cache[l].cpu().numpy()
            k_gs, v_gs = float(c.k_gs[l]), float(c.v_gs[l])
            assert np.array_equal(cache, oc.append(b(k.contiguous()), b(v.contiguous()), k_gs, v_gs, before[l], table, lens, PS))
            ref = oc.attn(host(q), k_gs, v_gs, cache, table, lens, PS)
            off = np.abs(host(c.o[l]).reshape(ref[0].shape) - ref[0])
            assert np.all(off <= attn_bounds(ref, D, lens.max())[0])
            if c.m > 1:
                assert not c.o[l][skip].any()
    # what the o_proj reads is the attention's output
    s = c.s0.clone()
    u = sk.gemm_dual_norm(c.o[0], c.w_o[0], s.copy_(synth.normal_f32((c.m, H), 800 + 19)), c.post_w[0], c.alpha,
                          c.beta[0], c.pre_w[0], eps_post=c.eps, eps_pre=c.eps)[0]
    assert torch.equal(u, c.u[0])


def test_twin_has_rows_of_its_own(chain):
    c = chain
    t = c.twin()
    t.table.fill_(-1)
    inputs(t, 0)
    t.want.fill_(1)
    t.forward()
    torch.cuda.synchronize()
    assert (t.lens == 1).all() and not torch.equal(t.lens, c.lens)
    assert t.w_qkv is c.w_qkv and t.cache.data_ptr() != c.cache.data_ptr()
