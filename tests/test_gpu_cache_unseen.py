"""A token's attention over the 4-bit cache does not depend on keys that it does not see,
be their scales no numbers, although other tokens of the same call see them."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import BF16, DEV, F32, I32, U8, attn_bounds, gpu, host, random_cache, random_table, sk  # noqa: F401

pytestmark = pytest.mark.gpu


def spoil(cache, table, ps, d, row, pos, blocks, k_too):
    """Scales that are no number: of V in some blocks of 16 columns, of K if wanted."""
    _, _, ks, vs = oc.parts(cache, ps, d)
    page, at = table[row, pos // ps], pos % ps
    for x in blocks:
        vs[page, :, x, at] = 0xFF if x % 2 else 0x7F
    if k_too:
        ks[page, :, at] = 0x7F


@pytest.mark.parametrize("t,hq,hk,d,ps", [
    (4, 2, 1, 64, 16), (3, 2, 2, 128, 64), (4, 4, 1, 64, 64), (5, 6, 2, 128, 16), (9, 1, 1, 128, 32), (2, 16, 1, 64, 32),
    (3, 16, 1, 64, 32), (4, 16, 1, 128, 64), (8, 12, 1, 64, 16), (7, 32, 2, 128, 32), (140, 2, 2, 64, 64), (70, 4, 1, 128, 16),
])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("k_too", [False, True])
def test_keys_that_some_tokens_do_not_see(sk, t, hq, hk, d, ps, window, k_too):  # noqa: F811
    rng = np.random.default_rng(t + window)
    lens = np.array([300, t, 131 + t, 2])
    table = random_table(rng, lens, -(-300 // ps) + 1, 90, ps)
    cache = random_cache(rng, 90, hk, ps, d)
    q = torch.as_tensor(rng.normal(size=(4, t, hq, d))).to(BF16).to(DEV)
    args = (gpu([9.0], F32), gpu([9.0], F32))
    rest = (gpu(table, I32), gpu(lens, I32), ps)
    clean, clean_lse, _ = sk.attn_nvfp4(q, *args, gpu(cache, U8), *rest, window=window, lse=True)
    ref = oc.attn(host(q), 9.0, 9.0, cache, table, lens, ps, window=window)
    blocks = [0, d // 16 - 1]
    hurt = np.zeros((4, t, d), bool)        # what may be no number
    all_hurt = np.zeros((4, t), bool)       # seen with a K that is no number
    for i, n in enumerate(lens):
        first = n - t  # position of the first token; some of the call's tokens see these places, some do not
        places = [n - 1, first + t // 2 + 1] + ([first + 1 - window, first + t // 2 - window] if window else [])
        for pos in places:
            if not 0 <= pos < n:
                continue
            spoil(cache, table, ps, d, i, pos, blocks, k_too)
            for j in range(t):
                at = first + j
                if pos <= at and (not window or pos > at - window):
                    for x in blocks:
                        hurt[i, j, 16 * x:16 * x + 16] = True
                    all_hurt[i, j] |= k_too
    dirty, dirty_lse, _ = sk.attn_nvfp4(q, *args, gpu(cache, U8), *rest, window=window, lse=True)
    well = ~(hurt | all_hurt[..., None])
    x, y = dirty.float().cpu().numpy(), clean.float().cpu().numpy()
    keep = np.broadcast_to(well[:, :, None], x.shape)
    b_out, b_lse = attn_bounds(ref, d, 300)
    assert np.all(np.abs(x - ref[0])[keep] <= b_out[keep])
    assert np.isnan(x[np.broadcast_to(hurt[:, :, None], x.shape)]).all()
    seen = ~np.broadcast_to(all_hurt[:, :, None], ref[1].shape) & (ref[1] != -np.inf)
    lse = dirty_lse.cpu().numpy()
    assert np.all(np.abs(lse[seen] - ref[1][seen]) <= b_lse[seen])
    if not k_too:  # scores that are no numbers move the base of other rows too
        assert np.array_equal(x[keep], y[keep]) and np.array_equal(lse, clean_lse.cpu().numpy())


@pytest.mark.parametrize("d,hq,t", [(64, 4, 20), (64, 4, 40), (128, 4, 20), (128, 4, 70)])
def test_keys_that_some_tokens_do_not_see_in_rows_that_are_not_cut(sk, d, hq, t):  # noqa: F811
    # so many rows that most are the work of one CTA, over 12 chunks and more: the first ones, which
    # the window leaves in part, are long behind when the row ends
    rng = np.random.default_rng(t)
    b, ps, window = 400, 64, 1500
    lens = rng.integers(1800, 2500, b)
    table = random_table(rng, np.full(8, 2500), 40, 320, ps)[rng.integers(0, 8, b)]
    pages = np.unique(table)
    cache = random_cache(rng, 320, 1, ps, d)
    q = torch.as_tensor(rng.normal(size=(b, t, hq, d))).to(BF16).to(DEV)
    args = (gpu([9.0], F32), gpu([9.0], F32))
    rest = (gpu(table, I32), gpu(lens, I32), ps)
    clean, clean_lse, _ = sk.attn_nvfp4(q, *args, gpu(cache, U8), *rest, window=window, lse=True)
    # one place in every fourth page, one block of it each: rows see a few of them, at their ends in part
    _, _, _, vs = oc.parts(cache, ps, d)
    where = {int(p): (int(rng.integers(0, d // 16)), int(rng.integers(0, ps))) for p in pages[::4]}
    for p, (x, at) in where.items():
        vs[p, 0, x, at] = 0x7F
    hurt = np.zeros((b, t, d // 16), bool)
    for i in range(b):
        for c, p in enumerate(table[i]):
            if int(p) in where:
                x, at = where[int(p)]
                pos, first = c * ps + at, lens[i] - t
                hurt[i, max(0, pos - first):max(0, pos + window - first), x] = True
    dirty, dirty_lse, _ = sk.attn_nvfp4(q, *args, gpu(cache, U8), *rest, window=window, lse=True)
    lost = torch.as_tensor(hurt).to(DEV)[:, :, None, :, None].expand(b, t, hq, d // 16, 16).reshape(b, t, hq, d)
    assert torch.equal(dirty.isnan(), lost) and torch.equal(dirty[~lost], clean[~lost])
    assert torch.equal(dirty_lse, clean_lse)


@pytest.mark.parametrize("hq", [4, 16, 40, 100])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_no_number_counts_however_little_it_weighs(sk, d, hq):  # noqa: F811
    # a V of that kind where p = exp(-400), 0 in FP32, in each chunk of the row in turn
    ps, n, copies = 64, 640, 304
    table = np.arange(10, dtype=np.int32)[None]
    for where in range(10):
        cache = np.zeros((10, 1, ps * d * 9 // 8), np.uint8)
        kc, vc, ks, vs = oc.parts(cache, ps, d)
        kc[..., 0] = 0x0F                       # column 0 is -6
        kc[(where + 3) % 10, 0, 5, 0] = 0       # but of one key
        vc[...], ks[...], vs[...] = 0x22, 0x38, 0x38
        vs[where, 0, 1, 9] = 0x7F
        q = torch.zeros(copies, 1, hq, d, dtype=BF16, device=DEV)
        q[..., 0] = 1.0
        out = sk.attn_nvfp4(q, gpu([1.0], F32), gpu([1.0], F32), gpu(cache, U8), gpu(np.repeat(table, copies, 0), I32),
                            gpu(np.full(copies, n), I32), ps, scale=400 / 6)[0]
        assert out[..., 16:32].isnan().all() and (out[..., :16] == 1).all() and (out[..., 32:] == 1).all()
