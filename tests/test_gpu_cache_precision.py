"""What attention over the 4-bit cache promises of its 16-bit operands: P's rounding in
tiles of 128 rows after the base moved, and the queries' range, against the 64-bit
statement (oracle/cache.py) within attn_bounds (test_gpu_cache.py)."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import BF16, DEV, F32, I32, U8, attn_bounds, gpu, host, random_cache, random_table, sk  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [4, 16, 40, 64, 100])
def test_the_largest_p_stays_above_what_the_bound_says(sk, hq, d):  # noqa: F811
    """Scores, in powers of two below the largest: 8.39 for the first key, 0 for one behind it,
    31.45 for all others, of which the V of 64 behind these two alone is not 0. So the base moves,
    in tiles of 128 rows by a whole number, and what is added up then is 2^-31.45 of the largest
    p: lost if that is below 2^7 (0.48 steps of FP16's subnormal numbers with 2^6.39, 0.96 with
    2^7.39)."""
    ps, n, copies = 64, 640, 304
    cache = np.zeros((4, 1, ps * d * 9 // 8), np.uint8)
    kc, vc, ks, vs = oc.parts(cache, ps, d)
    kc[..., 0] = 0x0F         # column 0 is -6 * 1.25
    ks[...] = 0x3A
    vs[...] = 0x38            # 1.0
    kc[0, :, 0, 0] = 0x0C     # -2
    ks[0, :, 0, 0] = 0x38
    kc[1, :, 0, 0] = 0x00
    vc[2] = 0x77              # 6.0
    # chunks of 128 keys: the first, the next even one, and the one behind that, in their first halves
    table = np.array([[0, 3, 3, 3, 1, 3, 3, 3, 2, 3]], np.int32)
    lens = np.array([n - ps])
    q = np.zeros((1, 1, hq, d))
    q[..., 0] = 1.0
    scale = 31.45 / 7.5 * np.log(2.0)
    # so many rows of the same pages that most of them are not cut into parts
    out, _, _ = sk.attn_nvfp4(torch.as_tensor(q).to(BF16).to(DEV).expand(copies, 1, hq, d).contiguous(), gpu([1.0], F32),
                              gpu([1.0], F32), gpu(cache, U8), gpu(np.repeat(table, copies, 0), I32),
                              gpu(np.repeat(lens, copies), I32), ps, scale=scale)
    ref = oc.attn(q, 1.0, 1.0, cache, table, lens, ps, scale=scale)
    off = np.abs(host(out) - ref[0])
    bound = attn_bounds(ref, d, n)[0]
    assert np.all(off <= bound), np.max(off / bound)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [3, 13, 40, 100])
@pytest.mark.parametrize("below", [29, 30, 31, 32, 33])
def test_queries_far_below_the_row_s_largest(sk, below, hq, d):  # noqa: F811
    """A query's largest value meets keys of 0, so that its scores are those of values 2^below
    smaller. Their eight significant bits are exact through 2^31; below that each is off by at
    most half a step of FP16's subnormal numbers, 2^-25 where the largest is at least 2^14:
    2^-39 of the largest."""
    rng = np.random.default_rng(below)
    n, ps = 300, 64
    table = random_table(rng, [n], 5, 5, ps)
    cache = random_cache(rng, 5, 1, ps, d)
    kc = oc.parts(cache, ps, d)[0]
    kc[..., 0] &= 0xF0                                          # column 0
    q = rng.choice([-1.0, 1.0], (1, 1, hq, d)) * rng.integers(128, 256, (1, 1, hq, d)) / 128.0  # [1, 2)
    q[..., 0] *= 2.0 ** below
    scale = 0.02
    out, lse, _ = sk.attn_nvfp4(torch.as_tensor(q).to(BF16).to(DEV), gpu([1.0], F32), gpu([9.0], F32), gpu(cache, U8),
                                gpu(table, I32), gpu([n], I32), ps, scale=scale, lse=True)
    out_ref, lse_ref, size, reach, mass = oc.attn(q, 1.0, 9.0, cache, table, np.array([n]), ps, scale=scale)
    if below > 31:  # attn_bounds makes (d / 8 + 16) 2^-23 of `reach`, which is scale sum |q K|, |q| >= 1
        reach = reach * (1 + 2.0 ** (below + 1 - 39) / ((d / 8 + 16) * 2.0 ** -23))
    b_out, b_lse = attn_bounds((out_ref, lse_ref, size, reach, mass), d, n)
    assert np.all(np.abs(host(out) - out_ref) <= b_out)
    assert np.all(np.abs(host(lse) - lse_ref) <= b_lse)
