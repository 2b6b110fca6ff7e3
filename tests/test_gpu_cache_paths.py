"""Forms of the 4-bit cache's calls that only large sizes take (GPU): tables so wide that the work is
counted in 64 bits, thousands of rows that part from one page, families of rows over shared pages."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import (BF16, DEV, F32, I32, U8, check_attn, check_resize, gpu, host, random_cache, random_table,  # noqa: F401
                            sk)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,d", [(1, 64), (1, 128), (3, 64), (20, 64), (20, 128)])
def test_tables_so_wide_that_work_counts_in_64_bits(sk, t, d):  # noqa: F811
    # 16 rows of 2^24 pages (1 GB) and 8 KV heads; the rows themselves are short
    rng = np.random.default_rng(t)
    b, hk, hq, ps = 16, 8, 64, 64
    lens = np.concatenate([[0, 700, -3], rng.integers(1, 700, b - 3)])
    table = random_table(rng, lens, 11, 200, ps)
    cache = gpu(random_cache(rng, 200, hk, ps, d), U8)
    q = torch.as_tensor(rng.normal(size=(b, t, hq, d))).to(BF16).to(DEV)
    wide = torch.full((b, 2 ** 24), -1, dtype=I32, device=DEV)
    wide[:, :11] = gpu(table, I32)
    one, ln = gpu([9.0], F32), gpu(lens, I32)
    for window in (0, 100):
        near, near_lse, _ = sk.attn_nvfp4(q, one, one, cache, gpu(table, I32), ln, ps, window=window, lse=True)
        far, far_lse, _ = sk.attn_nvfp4(q, one, one, cache, wide, ln, ps, window=window, lse=True)
        assert torch.equal(near, far) and torch.equal(near_lse, far_lse)


@pytest.mark.parametrize("rows,free", [(4096, 4096), (4096, 3000), (2500, 0)])
def test_thousands_of_rows_part_from_one_page(sk, rows, free):  # noqa: F811
    cache = np.random.default_rng(rows).integers(0, 256, (1, 4200, 1, 1152)).astype(np.uint8)
    table = np.full((rows, 2), -1, np.int32)
    table[:, 0] = 7
    lens = np.full(rows, 5, np.int32)
    refs = np.ones(4200, np.int32)
    refs[100:100 + free] = 0
    refs[7] = rows
    got = check_resize(sk, lens + 1, cache, table, lens, refs, 16)
    served = min(free, rows - 1) + (free >= rows - 1)  # the last one keeps the page
    assert (got[0] == 0).sum() == served


@pytest.mark.parametrize("t,hq,hk,d", [(1, 16, 2, 128), (1, 32, 2, 64), (5, 16, 1, 64), (3, 64, 2, 128)])
def test_families_of_rows_over_one_prompt(sk, t, hq, hk, d):  # noqa: F811
    # four prompts, each with rows that share its pages but the last, as after a fork and a step
    rng = np.random.default_rng(t * d)
    ps, rows = 32, 24
    prompt = np.array([900, 64, 31, 333])[np.arange(rows) % 4]
    lens = prompt + t + rng.integers(0, 40, rows)
    width = -(-int(lens.max()) // ps)
    table = np.full((rows, width), -1, np.int32)
    order = iter(rng.permutation(400))
    first = {}
    for i in range(rows):
        shared = prompt[i] // ps
        if prompt[i] not in first:
            first[prompt[i]] = [next(order) for _ in range(shared)]
        table[i, :shared] = first[prompt[i]]
        for c in range(shared, -(-int(lens[i]) // ps)):
            table[i, c] = next(order)
    cache = random_cache(rng, 400, hk, ps, d)
    check_attn(sk, rng.normal(size=(rows, t, hq, d)), 20.0, 9.0, cache, table, lens, ps)
