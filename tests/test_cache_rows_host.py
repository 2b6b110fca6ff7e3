"""sk_kv_append_ex without a GPU: its refusals, and what the 64-bit statement makes of rows
that bring no tokens or fewer than others."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

P = 1 << 20  # an aligned address that nothing reads
ARGS = dict(k=P, v=P, k_gs=P, v_gs=P, cache=P, table=P, lens=P, new_lens=P, fresh=P, b=2, t=1, kv_heads=8, head_dim=64,
            page_size=64, pages=10, width=4, k_stride=512, v_stride=512, stream=None)


@pytest.fixture(scope="module")
def sk():
    from nvfp4_sm_skinny_gb300 import build

    build.build()
    import nvfp4_sm_skinny_gb300 as sk

    return sk


@pytest.mark.parametrize("change,word", [(dict(new_lens=P + 2), "new_lens"), (dict(fresh=P + 1), "fresh"), (dict(b=0), "b=0"),
                                         (dict(lens=None), "lens"), (dict(k_stride=8), "k_stride")])
def test_refusals(sk, change, word):
    assert sk.lib().sk_kv_append_ex(*{**ARGS, **change}.values()) == 1 and word in sk.last_error()


@pytest.mark.parametrize("change", [{}, dict(new_lens=None), dict(fresh=None), dict(new_lens=None, fresh=None)])
def test_valid_calls_without_gpu_report_a_device_error(sk, change):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    assert sk.lib().sk_kv_append_ex(*{**ARGS, **change}.values()) in (3, 5) and sk.last_error()


def test_the_statement_leaves_rows_out():
    rng = np.random.default_rng(0)
    k = rng.integers(0, 2 ** 14, (5, 2, 1, 64)).astype(np.uint16)
    table, lens = np.arange(10, dtype=np.int32).reshape(5, 2), np.array([3, 3, 17, 32, 40], np.int32)
    zero = np.zeros((10, 1, 1152), np.uint8)
    new, fresh = np.array([3, -1, 17, 33, 40], np.int32), np.array([2, 2, 1, 2, 2], np.int32)
    got = oc.append(k, k, 1.0, 1.0, zero, table, lens, 16, new, fresh)
    kc = oc.parts(got, 16, 64)[0]
    written = sorted((int(p), int(i)) for p, _, i in np.argwhere(kc.any(-1)))
    # row 0 both tokens, row 1 waits, row 2 its last one, row 3 was refused, row 4 is out of range
    assert written == [(0, 1), (0, 2), (5, 0)]
    assert np.array_equal(oc.append(k, k, 1.0, 1.0, zero, table, lens, 16, lens.clip(0, 32), np.full(5, 9)),
                          oc.append(k[:4], k[:4], 1.0, 1.0, zero, table[:4], lens[:4], 16))
