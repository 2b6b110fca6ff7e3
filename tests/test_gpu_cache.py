"""GPU parity of the 4-bit key/value cache (sk_kv_append, sk_attn_nvfp4,
sk_kv_resize, sk_kv_fork, sk_kv_compact) against its 64-bit statement
(oracle/cache.py). Bytes and whole numbers have to be equal; what attention may be
off by is derived in attn_bounds."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def sk(oracle_mod):
    import nvfp4_sm_skinny_gb300 as sk

    sk.lib()
    return sk


@pytest.fixture(autouse=True)
def _no_device_errors(sk):
    yield
    assert sk.device_status(clear=True) == 0


def gpu(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV).to(dtype)


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def random_table(rng, lens, width, pages, ps, spare=-1):
    """Rows of pages in a random order, none twice, `spare` behind a row's end."""
    order = iter(rng.permutation(pages))
    table = np.full((len(lens), width), spare, np.int32)
    for i, n in enumerate(lens):
        for c in range(-(-min(max(int(n), 0), width * ps) // ps)):
            table[i, c] = next(order)
    return table


def random_cache(rng, pages, hk, ps, d, lo=0x20, hi=0x58):
    """Codes of any value and scales of 2^-3 to 2^4, signs among them."""
    cache = rng.integers(0, 256, (pages, hk, ps * d * 9 // 8)).astype(np.uint8)
    for p in oc.parts(cache, ps, d)[2:]:
        p[...] = rng.integers(lo, hi, p.shape)
    return cache


# ------------------------------------------------------------------ append ----
@pytest.mark.parametrize("b,t,hk,d,ps,lens", [
    (1, 1, 1, 64, 16, [1]), (1, 1, 8, 128, 64, [64]), (3, 2, 2, 64, 32, [5, 33, 1]),
    (2, 70, 3, 128, 32, [70, 90]), (4, 17, 5, 64, 16, [0, 16, 17, 200]), (1, 300, 1, 128, 64, [1000]),
])
def test_append(sk, b, t, hk, d, ps, lens):
    rng = np.random.default_rng(b + t)
    width = -(-max(lens) // ps) + 1
    pages = sum(-(-n // ps) for n in lens) + 2
    table = random_table(rng, lens, width, pages, ps)
    cache = rng.integers(0, 256, (pages, hk, ps * d * 9 // 8)).astype(np.uint8)
    x = torch.as_tensor(rng.normal(size=(2, b, t, hk, d)) * np.exp(rng.normal(size=(2, b, t, hk, 1)) * 2)).to(BF16)
    x[0, 0, 0, 0, :16] = 0.0           # a block without a scale
    x[1, 0, -1, -1, 16:32] *= 1e6      # one beyond the largest
    k_gs, v_gs = 300.0, 41.5
    c, k, v = gpu(cache, U8), x[0].to(DEV), x[1].to(DEV)
    sk.kv_append(k, v, gpu([k_gs], F32), gpu([v_gs], F32), c, gpu(table, I32), gpu(lens, I32), ps)
    assert np.array_equal(host(c), oc.append(bits(x[0]), bits(x[1]), k_gs, v_gs, cache, table, np.array(lens), ps))


def test_append_from_the_rows_of_one_product(sk):
    rng = np.random.default_rng(3)
    b, t, hq, hk, d, ps, lens = 3, 2, 4, 2, 64, 16, [2, 20, 33]
    rows = torch.as_tensor(rng.normal(size=(b * t, (hq + 2 * hk) * d))).to(BF16)
    _, k, v = (x.view(b, t, -1, d) for x in rows.split([hq * d, hk * d, hk * d], 1))
    table = random_table(rng, lens, 3, 8, ps)
    cache = np.zeros((8, hk, ps * d * 9 // 8), np.uint8)
    c = gpu(cache, U8)
    r = rows.to(DEV)
    _, kd, vd = (x.view(b, t, -1, d) for x in r.split([hq * d, hk * d, hk * d], 1))
    one = gpu([100.0], F32)
    sk.kv_append(kd, vd, one, one, c, gpu(table, I32), gpu(lens, I32), ps)
    assert np.array_equal(host(c), oc.append(bits(k), bits(v), 100.0, 100.0, cache, table, np.array(lens), ps))
    with pytest.raises(ValueError, match="k: needs"):
        sk.kv_append(kd.transpose(0, 1), vd.transpose(0, 1), one, one, c, gpu(table[:2], I32), gpu(lens[:2], I32), ps)


def test_append_of_every_largest_value(sk):
    # a block for each finite BF16 magnitude, which its scale's division by 6 starts from
    ps, d, hk, t = 64, 128, 2, 2048
    mag = np.arange(t * hk * d // 16, dtype=np.uint16)  # 32,768 bit patterns, the last 128 not finite
    mag[mag >= 0x7F80] = 0
    rng = np.random.default_rng(5)
    z = (rng.random((len(mag), 16)) * mag[:, None]).astype(np.uint16)  # smaller patterns are smaller values
    z[:, 7] = mag
    z |= (rng.integers(0, 2, z.shape) << 15).astype(np.uint16)
    k = torch.as_tensor(z.view(np.int16)).view(BF16).view(1, t, hk, d)
    table = rng.permutation(32)[None].astype(np.int32)
    cache = np.zeros((32, hk, ps * d * 9 // 8), np.uint8)
    for k_gs, v_gs in ((1.0, 448.0), (3e-30, 7e30)):
        c = gpu(cache, U8)
        sk.kv_append(k.to(DEV), k.flip(1).to(DEV), gpu([k_gs], F32), gpu([v_gs], F32), c, gpu(table, I32),
                     gpu([t], I32), ps)
        want = oc.append(bits(k), bits(k.flip(1)), k_gs, v_gs, cache, table, np.array([t]), ps)
        assert np.array_equal(host(c), want)


def test_append_leaves_out_what_has_no_place(sk):
    # pages outside the cache, positions before the row and beyond the table
    rng = np.random.default_rng(4)
    cache = rng.integers(0, 256, (4, 2, 16 * 64 * 9 // 8)).astype(np.uint8)
    table = np.array([[-1, 2], [4, 1], [2 ** 31 - 1, -2 ** 31], [0, 3]], np.int32)
    lens = np.array([18, 17, 32, 40], np.int32)
    x = torch.as_tensor(rng.normal(size=(4, 20, 2, 64))).to(BF16)
    c = gpu(cache, U8)
    one = gpu([1.0], F32)
    sk.kv_append(x.to(DEV), x.to(DEV), one, one, c, gpu(table, I32), gpu(lens, I32), 16)
    assert np.array_equal(host(c), oc.append(bits(x), bits(x), 1.0, 1.0, cache, table, lens, 16))


# --------------------------------------------------------------- attention ----
def attn_bounds(ref, d, keys):
    """(out, lse) bounds. A score is a sum of d exact products in FP32, d / 16 steps of
    the tensor core, each within 2 units of its largest part, times a factor of five
    roundings, minus the base: off by ds = reach (d / 8 + 16) 2^-23 + 2^-20 (the
    exponential 2^-22 of itself, the base). P is rounded to FP16: 2^-11 of itself, or
    2^-25, half the step below FP16's normal numbers, however small it is, where a
    row's largest p and so its sum are at least 2^7: 2^-32 of every |v|. Products with
    V are exact and summed in FP32: `keys` terms in chains of keys / 8 + 64 additions.
    The last rounding is to BF16, half a step."""
    out, lse, size, reach, mass = ref
    ds = reach * (d / 8 + 16) * 2.0 ** -23 + 2.0 ** -20
    sums = (keys / 8 + 64) * 2.0 ** -23
    rel = 2.0 ** -11 + 2 * ds + 2 * sums
    return np.abs(out) * 2.0 ** -8 + (size * rel[..., None] + mass * 2.0 ** -32) * 1.01 + 1e-38, ds + sums + np.abs(lse) * 2.0 ** -22


def check_attn(sk, q, k_gs, v_gs, cache, table, lens, ps, **kw):
    q = torch.as_tensor(q).to(BF16)
    c, table, lens = gpu(cache, U8), np.asarray(table, np.int32), np.asarray(lens, np.int32)
    args = (q.to(DEV), gpu([k_gs], F32), gpu([v_gs], F32), c, gpu(table, I32), gpu(lens, I32), ps)
    out, lse, _ = sk.attn_nvfp4(*args, lse=True, **kw)
    again, none, _ = sk.attn_nvfp4(*args, **kw)
    assert none is None and torch.equal(out, again)
    ref = oc.attn(host(q), k_gs, v_gs, cache, table, lens, ps, **kw)
    b_out, b_lse = attn_bounds(ref, q.shape[3], max(1, lens.max()))
    off = np.abs(host(out) - ref[0])
    assert np.all(off <= b_out), (np.max(off - b_out), np.argwhere(off > b_out)[:5])
    empty = ref[1] == -np.inf
    assert (host(lse)[empty] == -np.inf).all() and not host(out)[empty].any()
    assert np.all(np.abs(host(lse)[~empty] - ref[1][~empty]) <= b_lse[~empty])
    return out, lse


ATTN = [  # t, hq, hk, d, ps, lens
    (1, 1, 1, 64, 16, [1]), (1, 8, 8, 64, 64, [63, 64, 65]), (1, 16, 2, 128, 64, [129, 1, 0, 300]),
    (1, 128, 8, 64, 64, [200]), (1, 64, 8, 128, 16, [257, 255]), (2, 8, 1, 128, 32, [1, 2, 47]),
    (1, 16, 1, 128, 64, [700]), (1, 9, 1, 64, 32, [333]), (4, 32, 4, 64, 16, [3, 100, 511]),
    (4, 16, 2, 128, 64, [400, 5]), (3, 33, 3, 64, 64, [130]), (8, 16, 1, 128, 32, [300]),
    (5, 14, 2, 64, 16, [64, 63, 0, 1]), (1, 100, 1, 128, 64, [190]), (70, 2, 1, 64, 32, [70, 90]),
    (1, 7, 1, 128, 16, [2500]), (1, 32, 4, 64, 64, list(range(0, 300, 7))),
]


@pytest.mark.parametrize("t,hq,hk,d,ps,lens", ATTN)
def test_attention(sk, t, hq, hk, d, ps, lens):
    rng = np.random.default_rng(hq * 100 + lens[0])
    width = -(-max(lens) // ps) + 1
    pages = sum(-(-n // ps) for n in lens) + 2
    table = random_table(rng, lens, width, pages, ps, spare=pages + 5)
    cache = random_cache(rng, pages, hk, ps, d)
    q = rng.normal(size=(len(lens), t, hq, d)) * np.exp2(rng.integers(-3, 2, (len(lens), t, hq, 1)))
    check_attn(sk, q, 30.0, 7.0, cache, table, lens, ps)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 1000])
@pytest.mark.parametrize("t,d,ps", [(1, 128, 64), (5, 64, 16), (20, 64, 32)])
def test_window(sk, window, t, d, ps):
    rng = np.random.default_rng(window)
    lens = [700, 64, 65, 3, 0]
    table = random_table(rng, lens, -(-700 // ps), 200, ps)
    cache = random_cache(rng, 200, 2, ps, d)
    q = rng.normal(size=(5, t, 8, d)) * 0.3
    check_attn(sk, q, 20.0, 3.0, cache, table, lens, ps, window=window)


@pytest.mark.parametrize("d,ps", [(64, 16), (128, 32), (128, 64)])
def test_what_no_token_sees_does_not_matter(sk, d, ps):
    # scales that are no number behind the end of rows, in pages of others and in pieces not there
    rng = np.random.default_rng(7)
    lens = np.array([100, 37, 64, 250])
    table = random_table(rng, lens, 16, 60, ps)
    cache = random_cache(rng, 60, 2, ps, d)
    q = rng.normal(size=(4, 2, 8, d))
    clean, _ = check_attn(sk, q, 9.0, 9.0, cache, table, lens, ps)
    held = np.zeros((60, ps), bool)
    for i, n in enumerate(lens):
        for p in range(n):
            held[table[i, p // ps], p % ps] = True
    _, _, ks, vs = oc.parts(cache, ps, d)
    ks[:] = np.where(held[:, None, :, None], ks, 0x7F)
    vs[:] = np.where(held[:, None, None, :], vs, 0xFF)
    dirty, _ = check_attn(sk, q, 9.0, 9.0, cache, table, lens, ps)
    assert torch.equal(clean, dirty)


@pytest.mark.parametrize("t,hq,d,ps,window", [(1, 4, 64, 16, 70), (1, 4, 128, 64, 1), (2, 16, 128, 32, 100), (4, 32, 64, 64, 33),
                                              (8, 32, 128, 16, 150)])
def test_what_lies_before_the_window_does_not_matter(sk, t, hq, d, ps, window):
    # scales that are no number before the first key that a row's first token sees
    rng = np.random.default_rng(window)
    lens = np.array([300, 130, 64, 9])
    table = random_table(rng, lens, -(-300 // ps), 60, ps)
    cache = random_cache(rng, 60, 2, ps, d)
    q = rng.normal(size=(4, t, hq, d))
    clean, _ = check_attn(sk, q, 9.0, 9.0, cache, table, lens, ps, window=window)
    _, _, ks, vs = oc.parts(cache, ps, d)
    for i, n in enumerate(lens):
        for p in range(n - t - window + 1):
            ks[table[i, p // ps], :, p % ps] = 0x7F
            vs[table[i, p // ps], :, :, p % ps] = 0xFF
    dirty = sk.attn_nvfp4(torch.as_tensor(q).to(BF16).to(DEV), gpu([9.0], F32), gpu([9.0], F32),
                          gpu(cache, U8), gpu(table, I32), gpu(lens, I32), ps, window=window)[0]
    assert torch.equal(clean, dirty)


def test_missing_pages_are_left_out(sk):
    rng = np.random.default_rng(8)
    ps, d = 16, 64
    table = random_table(rng, [300, 300, 20, 64], 19, 80, ps)
    table[0, [0, 5, 18]] = -1, 80, 2 ** 31 - 1
    table[1] = -2 ** 31
    table[2, 0] = 1000
    cache = random_cache(rng, 80, 1, ps, d)
    check_attn(sk, rng.normal(size=(4, 3, 4, d)), 5.0, 5.0, cache, table, [300, 300, 20, 64], ps)
    check_attn(sk, rng.normal(size=(4, 3, 4, d)), 5.0, 5.0, cache, table, [300, 300, 20, 64], ps, window=40)


def test_lengths_out_of_range(sk):
    # negative: a row of nothing; beyond the table: the keys that it names
    rng = np.random.default_rng(9)
    table = random_table(rng, [64, 64, 64], 4, 20, 16)
    cache = random_cache(rng, 20, 1, 16, 64)
    q = rng.normal(size=(3, 2, 2, 64))
    out, lse = check_attn(sk, q, 5.0, 5.0, cache, table, [-7, 80, 2 ** 31 - 1], 16)
    assert not host(out)[0].any() and (host(lse)[0] == -np.inf).all()
    # a window counts from the position, whatever of it the table names
    check_attn(sk, q, 5.0, 5.0, cache, table, [66, 80, 2 ** 31 - 1], 16, window=10)
    check_attn(sk, q, 5.0, 5.0, cache, table, [65, 100, 73], 16, window=40)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 8.0])
def test_scales_and_queries_far_apart(sk, scale):
    # one key that outweighs all, rising and falling scores, rows of zeros and of tiny and huge values
    rng = np.random.default_rng(10)
    d, n = 128, 900
    table = random_table(rng, [n], 15, 15, 64)
    cache = random_cache(rng, 15, 1, 64, d)
    q = rng.normal(size=(1, 1, 16, d))
    q[0, 0, 0] = 0.0
    q[0, 0, 1] *= 1e-30
    q[0, 0, 2] = 1e-39
    q[0, 0, 3] *= 8
    q[0, 0, 4, 1:] *= 2.0 ** -20
    q[0, 0, 5] *= 1e4 if scale <= 0 else 1
    check_attn(sk, q, 40.0, 1.0, cache, table, [n], 64, scale=scale)


def test_queries_of_the_largest_values(sk):
    rng = np.random.default_rng(11)
    table = random_table(rng, [200], 4, 4, 64)
    cache = random_cache(rng, 4, 1, 64, 64)
    q = np.sign(rng.normal(size=(1, 1, 8, 64))) * 3e38
    check_attn(sk, q, 1.0, 1.0, cache, table, [200], 64, scale=1e-39)


def test_scores_that_grow_along_the_row(sk):
    # every chunk outdoes the one before it, by much and by little: the base moves each time
    d, n = 64, 1500
    cache = np.zeros((24, 1, 64 * d * 9 // 8), np.uint8)
    kc, vc, ks, vs = oc.parts(cache, 64, d)
    rng = np.random.default_rng(12)
    kc[...] = 0x22                                           # 1.0
    ks[...] = (0x20 + np.arange(24) * 2)[:, None, None, None]  # growing scales
    vc[...] = rng.integers(0, 256, vc.shape)
    vs[...] = 0x38
    q = np.ones((1, 1, 4, d)) * np.array([0.01, 0.1, 1.0, -1.0])[None, None, :, None]
    check_attn(sk, q, 1.0, 1.0, cache, np.arange(24)[None], [n], 64, scale=1.0)


def test_shared_pages_and_queries_in_longer_rows(sk):
    rng = np.random.default_rng(13)
    lens = [100, 90, 100]
    table = np.array([[1, 2], [1, 3], [1, 2]], np.int32)
    cache = random_cache(rng, 4, 2, 64, 64)
    rows = torch.as_tensor(rng.normal(size=(3 * 2, 8 * 64 + 256))).to(BF16).to(DEV)
    q = rows[:, 128:128 + 8 * 64].unflatten(0, (3, 2)).unflatten(2, (8, 64))
    one, c, tb, ln = gpu([3.0], F32), gpu(cache, U8), gpu(table, I32), gpu(lens, I32)
    out, _, _ = sk.attn_nvfp4(q, one, one, c, tb, ln, 64)
    flat, _ = check_attn(sk, host(q), 3.0, 3.0, cache, table, lens, 64)
    assert torch.equal(out, flat)


@pytest.mark.parametrize("b,hq,hk,d,ps,n", [(1, 16, 2, 128, 64, 20000), (1, 4, 1, 64, 16, 9001), (300, 8, 2, 64, 64, 40),
                                            (150, 16, 1, 128, 16, 33)])
def test_many_parts_and_many_rows(sk, b, hq, hk, d, ps, n):
    rng = np.random.default_rng(14)
    lens = [n] if b == 1 else rng.integers(0, n, b)
    width = -(-n // ps)
    pages = sum(-(-int(x) // ps) for x in lens) + 1
    table = random_table(rng, lens, width, pages, ps)
    cache = random_cache(rng, pages, hk, ps, d)
    check_attn(sk, rng.normal(size=(b, 1, hq, d)), 30.0, 9.0, cache, table, lens, ps)


# More than 32 rows per KV head, in tiles of 128: up to 64 rows, up to 128, several tiles,
# rows before the first token, windows that end within a chunk of 128.
MANY = [  # t, hq, hk, d, ps, lens
    (3, 12, 1, 64, 16, [5, 200, 129, 0]), (4, 16, 1, 128, 64, [128, 127, 1, 0, 2, 256]), (1, 64, 1, 64, 32, [300]),
    (5, 13, 1, 128, 16, [700]), (8, 16, 1, 64, 64, [513, 3, 8]), (8, 32, 2, 128, 32, [640, 1000]),
    (130, 1, 1, 64, 16, [130, 200, 40]), (70, 4, 2, 128, 64, [70, 333]), (300, 2, 1, 64, 64, [300, 777]),
    (40, 9, 3, 128, 16, [90] * 5), (1, 33, 1, 64, 64, [1, 2500]),
]


@pytest.mark.parametrize("window", [0, 1, 100, 129])
@pytest.mark.parametrize("t,hq,hk,d,ps,lens", MANY)
def test_many_rows(sk, t, hq, hk, d, ps, lens, window):
    rng = np.random.default_rng(t + hq)
    width = -(-max(lens) // ps) + 1
    pages = sum(-(-n // ps) for n in lens) + 2
    table = random_table(rng, lens, width, pages, ps, spare=pages + 5)
    cache = random_cache(rng, pages, hk, ps, d)
    q = rng.normal(size=(len(lens), t, hq, d)) * np.exp2(rng.integers(-3, 2, (len(lens), t, hq, 1)))
    check_attn(sk, q, 30.0, 7.0, cache, table, lens, ps, window=window)


@pytest.mark.parametrize("d,t,hq", [(64, 4, 10), (64, 9, 10), (128, 4, 10), (128, 9, 10)])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 8.0])
def test_many_rows_with_scores_that_move_the_base(sk, scale, d, t, hq):
    # scales of keys that grow from page to page, and queries of every size and sign
    rng = np.random.default_rng(16)
    n = 1400
    table = np.arange(24)[None]
    cache = random_cache(rng, 24, 1, 64, d)
    kc, _, ks, _ = oc.parts(cache, 64, d)
    kc[:, :, :, :4] = 0x22                                   # 1.0
    ks[...] = (0x20 + np.arange(24) * 2)[:, None, None, None]
    q = rng.normal(size=(1, t, hq, d)) * np.exp2(rng.integers(-12, 3, (1, t, hq, 1)))
    q[0, 0, 0] = 0.0
    q[0, 1, 1] = 1e-39
    q[0, 2, 2, 1:] *= 2.0 ** -20
    check_attn(sk, q, 40.0, 1.0, cache, table, [n], 64, scale=scale)


@pytest.mark.parametrize("d,ps", [(64, 16), (128, 32), (128, 64)])
def test_many_rows_with_missing_pages_and_strange_lengths(sk, d, ps):
    rng = np.random.default_rng(17)
    width = 320 // ps
    lens = [300, 300, 20, 320, -7, 400, 2 ** 31 - 1]
    table = random_table(rng, [320] * 7, width, 7 * width, ps)
    table[0, [0, 3]] = -1, 7 * width
    table[1] = -2 ** 31
    table[2, 0] = 2 ** 31 - 1
    cache = random_cache(rng, 7 * width, 1, ps, d)
    q = rng.normal(size=(7, 12, 4, d))
    check_attn(sk, q, 5.0, 5.0, cache, table, lens, ps)
    check_attn(sk, q, 5.0, 5.0, cache, table, lens, ps, window=90)
    # scales that are no number where nobody looks
    _, _, ks, vs = oc.parts(cache, ps, d)
    clean = sk.attn_nvfp4(torch.as_tensor(q).to(BF16).to(DEV), gpu([5.0], F32), gpu([5.0], F32), gpu(cache, U8),
                          gpu(table, I32), gpu(lens, I32), ps)[0]
    held = np.zeros((7 * width, ps), bool)
    for i, n in enumerate(lens):
        for p in range(min(max(n, 0), 320)):
            if 0 <= table[i, p // ps] < 7 * width:
                held[table[i, p // ps], p % ps] = True
    ks[:] = np.where(held[:, None, :, None], ks, 0x7F)
    vs[:] = np.where(held[:, None, None, :], vs, 0xFF)
    dirty = sk.attn_nvfp4(torch.as_tensor(q).to(BF16).to(DEV), gpu([5.0], F32), gpu([5.0], F32), gpu(cache, U8),
                          gpu(table, I32), gpu(lens, I32), ps)[0]
    assert torch.equal(clean, dirty)


@pytest.mark.parametrize("b,t,hq,hk,d,ps,n", [(1, 4, 10, 1, 128, 64, 20000), (1, 9, 10, 1, 64, 16, 9001),
                                              (300, 5, 8, 1, 64, 64, 40), (150, 4, 20, 2, 128, 16, 33)])
def test_many_rows_in_many_parts(sk, b, t, hq, hk, d, ps, n):
    rng = np.random.default_rng(18)
    lens = [n] if b == 1 else rng.integers(0, n, b)
    width = -(-n // ps)
    pages = sum(-(-int(x) // ps) for x in lens) + 1
    table = random_table(rng, lens, width, pages, ps)
    cache = random_cache(rng, pages, hk, ps, d)
    check_attn(sk, rng.normal(size=(b, t, hq, d)), 30.0, 9.0, cache, table, lens, ps)


def test_many_rows_of_longer_rows_and_captured(sk):
    # queries as they lie in a product's rows; the same result from a replayed graph, with other lengths
    rng = np.random.default_rng(19)
    d, ps, t, hq, hk = 64, 32, 6, 16, 2
    lens = np.array([100, 600])
    table = random_table(rng, [700, 700], 22, 44, ps)
    cache = random_cache(rng, 44, hk, ps, d)
    rows = torch.as_tensor(rng.normal(size=(2 * t, hq * d + 256))).to(BF16).to(DEV)
    q = rows[:, 128:128 + hq * d].unflatten(0, (2, t)).unflatten(2, (hq, d))
    one, c, tb, ln = gpu([3.0], F32), gpu(cache, U8), gpu(table, I32), gpu(lens, I32)
    out, _, ws = sk.attn_nvfp4(q, one, one, c, tb, ln, ps)
    flat, _ = check_attn(sk, host(q), 3.0, 3.0, cache, table, lens, ps)
    assert torch.equal(out, flat)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        sk.attn_nvfp4(q, one, one, c, tb, ln, ps, out=out, workspace=ws, stream=stream)
    for lens in ([700, 1], [129, 350]):
        ln.copy_(gpu(lens, I32))
        graph.replay()
        want, _ = check_attn(sk, host(q), 3.0, 3.0, cache, table, lens, ps)
        assert torch.equal(out, want)


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_between_products(sk, d):
    # products before and after, which hold tensor memory too, one launch overlapping the next
    rng = np.random.default_rng(20)
    b, t, hk, ps = 4, 4, 2, 64
    hq, lens = 32, np.array([500, 64, 300, 129])
    table = random_table(rng, lens, 8, 32, ps)
    cache = random_cache(rng, 32, hk, ps, d)
    def bf16(*shape):
        return torch.as_tensor(rng.normal(size=shape) * 0.1).to(BF16).to(DEV)
    x, w_in, w_out = bf16(b * t, 1024), bf16((hq + 2 * hk) * d, 1024), bf16(1024, hq * d)
    one, c, tb, ln = gpu([3.0], F32), gpu(cache, U8), gpu(table, I32), gpu(lens, I32)
    def step():
        qkv = sk.gemm_bf16(x, w_in).view(b, t, hq + 2 * hk, d)
        q, k, v = qkv.split([hq, hk, hk], 2)
        sk.kv_append(k, v, one, one, c, tb, ln, ps)
        out, _, _ = sk.attn_nvfp4(q, one, one, c, tb, ln, ps)
        return q, out, sk.gemm_bf16(out.view(b * t, hq * d), w_out)
    q, first, y = step()
    ref = oc.attn(host(q), 3.0, 3.0, host(c), table, lens, ps)
    assert np.all(np.abs(host(first) - ref[0]) <= attn_bounds(ref, d, lens.max())[0])
    assert torch.equal(y, sk.gemm_bf16(first.view(b * t, hq * d), w_out))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        results = [step() for _ in range(8)]
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, first) and torch.equal(z, y) for _, out, z in results)


def test_many_rows_on_two_streams(sk):
    # two calls at once, of head sizes that take different shares of an SM
    rng = np.random.default_rng(21)
    calls = []
    for d, t in ((64, 5), (128, 40)):
        lens = [2000, 700, 41]
        table = random_table(rng, lens, 32, 96, 64)
        q = torch.as_tensor(rng.normal(size=(3, t, 16, d))).to(BF16).to(DEV)
        calls.append((q, gpu([9.0], F32), gpu([9.0], F32), gpu(random_cache(rng, 96, 2, 64, d), U8),
                      gpu(table, I32), gpu(lens, I32), 64))
    alone = [sk.attn_nvfp4(*a)[0] for a in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    results = [[], []]
    for _ in range(10):
        for a, st, r in zip(calls, streams, results):
            r.append(sk.attn_nvfp4(*a, stream=st)[0])
    torch.cuda.synchronize()
    for r, want in zip(results, alone):
        assert all(torch.equal(x, want) for x in r)


def test_cache_beyond_31_bits(sk):
    # the last pages of a cache of 2.4 GB
    ps, d, hk = 64, 128, 8
    pages = 2 ** 31 // (hk * ps * d * 9 // 8) + 4000
    rng = np.random.default_rng(15)
    small = random_cache(rng, 3, hk, ps, d)
    c = torch.zeros(pages, hk, ps * d * 9 // 8, dtype=U8, device=DEV)
    c[-3:] = gpu(small, U8)
    table = np.array([[2, 0, 1]], np.int32)
    q = torch.as_tensor(rng.normal(size=(1, 1, 16, d))).to(BF16)
    one, ln = gpu([5.0], F32), gpu([180], I32)
    near = sk.attn_nvfp4(q.to(DEV), one, one, gpu(small, U8), gpu(table, I32), ln, ps)[0]
    far = sk.attn_nvfp4(q.to(DEV), one, one, c, gpu(table + pages - 3, I32), ln, ps)[0]
    assert torch.equal(near, far)
    kv = torch.as_tensor(rng.normal(size=(1, 2, hk, d))).to(BF16)
    sk.kv_append(kv.to(DEV), kv.to(DEV), one, one, c, gpu(table + pages - 3, I32), gpu([130], I32), ps)
    want = oc.append(bits(kv), bits(kv), 5.0, 5.0, small, table, np.array([130]), ps)
    assert np.array_equal(host(c[-3:]), want) and not c[:-3].any()


# ------------------------------------------------------------------- pages ----
def random_state(rng, rows, width, pages, ps, layers, share, fill=0.7, block=288):
    """A table whose rows partly share pages, with refs that count them."""
    table = np.full((rows, width), -1, np.int32)
    lens = np.zeros(rows, np.int32)
    order = list(rng.permutation(int(pages * fill)))
    for i in range(rows):
        if i and rng.random() < share:
            p = rng.integers(0, i)
            keep = rng.integers(0, lens[p] + 1)
            lens[i] = keep
            table[i, : -(-keep // ps)] = table[p, : -(-keep // ps)]
        else:
            n = min(int(rng.integers(0, width * ps + 1)), len(order) * ps)
            lens[i] = n
            for c in range(-(-n // ps)):
                table[i, c] = order.pop()
    refs = np.zeros(pages, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    cache = rng.integers(0, 256, (layers, pages, 1, 64 * ps * 9 // 8)).astype(np.uint8)
    return cache, table, lens, refs


def put(cache, table, lens, refs):
    return gpu(cache, U8), gpu(table, I32), gpu(lens, I32), gpu(refs, I32)


def check_resize(sk, new, cache, table, lens, refs, ps):
    c, t, n, r = put(cache, table, lens, refs)
    st, _ = sk.kv_resize(gpu(new, I32), c, t, n, r, ps)
    got = [host(x) for x in (st, c, t, n, r)]
    want = oc.resize(np.asarray(new), cache, table, lens, refs, ps)
    for name, x, y in zip(("status", "cache", "table", "lens", "refs"), got, want):
        assert np.array_equal(x, y), name
    return got


@pytest.mark.parametrize("rows,width,pages,ps,layers,share", [
    (1, 1, 1, 16, 1, 0.0), (4, 4, 20, 16, 2, 0.5), (33, 9, 400, 32, 3, 0.6), (200, 6, 900, 16, 1, 0.7),
    (1030, 4, 3001, 16, 1, 0.5), (64, 30, 5000, 64, 2, 0.3), (4096, 2, 9000, 16, 1, 0.6),
])
def test_resize(sk, rows, width, pages, ps, layers, share):
    rng = np.random.default_rng(rows)
    cache, table, lens, refs = random_state(rng, rows, width, pages, ps, layers, share)
    most = width * ps
    grow = np.minimum(lens + rng.integers(0, 2 * ps, rows), most)
    kind = rng.integers(0, 6, rows)
    new = np.where(kind == 0, 0, np.where(kind == 1, -1, np.where(kind == 2, lens // 2, grow))).astype(np.int32)
    got = check_resize(sk, new, cache, table, lens, refs, ps)
    held = np.zeros(pages, np.int32)  # refs still count the table's pages
    np.add.at(held, got[2][got[2] >= 0], 1)
    assert np.array_equal(held, got[4])
    check_resize(sk, np.minimum(lens + 1, most), cache, table, lens, refs, ps)


@pytest.mark.parametrize("free", [0, 1, 2, 3, 5, 8])
def test_resize_with_too_few_pages(sk, free):
    rng = np.random.default_rng(free)
    cache, table, lens, refs = random_state(rng, 12, 6, 60, 16, 2, 0.6, fill=0.6)
    spare = np.flatnonzero(refs == 0)
    refs[rng.permutation(spare)[free:]] = 1  # held by others
    new = np.minimum(lens + rng.integers(0, 40, 12), 96)
    check_resize(sk, new, cache, table, lens, refs, 16)


def test_resize_refuses_lengths_out_of_range(sk):
    rng = np.random.default_rng(3)
    cache, table, lens, refs = random_state(rng, 6, 4, 40, 16, 1, 0.0, fill=0.3)
    lens[2], lens[3] = -1, 65
    got = check_resize(sk, [65, 2 ** 31 - 1, 3, 3, -2 ** 31, 64], cache, table, lens, refs, 16)
    assert list(got[0][:5]) == [2, 2, 2, 2, 0]
    table[:] = rng.integers(-5, 60, table.shape)  # pages that are not there are not given back
    lens[2:4] = 20
    check_resize(sk, [0, 0, 5, 64, 0, 1], cache, table, lens, refs, 16)


@pytest.mark.parametrize("rows,width,ps,share", [(1, 1, 16, 0), (5, 3, 16, 0.5), (64, 33, 64, 0.3), (1021, 13, 32, 0.2),
                                                 (4096, 3, 16, 0.5)])
def test_fork(sk, rows, width, ps, share):
    rng = np.random.default_rng(rows)
    _, table, lens, refs = random_state(rng, rows, width, 2 * rows * width, ps, 1, share, fill=1.0, block=1)
    parents = np.where(rng.random(rows) < 0.3, -1, rng.integers(0, rows + 1 + rows // 10, rows)).astype(np.int32)
    t, n, r = gpu(table, I32), gpu(lens, I32), gpu(refs, I32)
    st = sk.kv_fork(gpu(parents, I32), t, n, r, ps)
    for x, y in zip((st, t, n, r), oc.fork(parents, table, lens, refs, ps)):
        assert np.array_equal(host(x), y)
    turn = np.roll(np.arange(rows), 1).astype(np.int32)  # all change places, twice in a row
    table, lens, refs = (host(x) for x in (t, n, r))
    sk.kv_fork(gpu(turn, I32), t, n, r, ps)
    want = oc.fork(turn, *oc.fork(turn, table, lens, refs, ps)[1:], ps)
    sk.kv_fork(gpu(turn, I32), t, n, r, ps)
    for x, y in zip((t, n, r), want[1:]):
        assert np.array_equal(host(x), y)


@pytest.mark.parametrize("rows,width,pages,ps,layers,fill", [
    (1, 1, 1, 16, 1, 0.0), (1, 2, 3, 16, 1, 1.0), (6, 4, 60, 16, 3, 0.9), (40, 20, 3000, 32, 2, 1.0),
    (100, 9, 5001, 16, 1, 1.0),
])
def test_compact(sk, rows, width, pages, ps, layers, fill):
    rng = np.random.default_rng(pages)
    cache, table, lens, refs = random_state(rng, rows, width, pages, ps, layers, 0.3, fill=fill)
    table[:, -1] = np.where(lens <= (width - 1) * ps, 2 ** 30, table[:, -1])  # behind the end: not looked at
    c, t, n, r = put(cache, table, lens, refs)
    m, _ = sk.kv_compact(c, t, n, r, ps)
    for x, y in zip((m, c, t, r), oc.compact(cache, table, lens, refs, ps)):
        assert np.array_equal(host(x), y)
    before = host(c)
    m, _ = sk.kv_compact(c, t, n, r, ps)  # nothing is left to move
    used = int((refs > 0).sum())
    assert np.array_equal(host(m), np.where(np.arange(pages) < used, np.arange(pages), -1))
    assert np.array_equal(host(c), before)


# -------------------------------------------------------------- all together ----
def test_a_run_of_them_together(sk):
    """A prompt, three samples forked from it, a few steps of two tokens, one sample given
    up, the pool compacted, more steps: attention against the 64-bit statement on
    what the cache has to hold by then, in two layers, from replayed graphs."""
    rng = np.random.default_rng(21)
    rows, width, pages, ps, layers, hq, hk, d, t = 4, 6, 30, 16, 2, 8, 2, 64, 2
    table = torch.full((rows, width), -1, dtype=I32, device=DEV)
    lens, refs = torch.zeros(rows, dtype=I32, device=DEV), torch.zeros(pages, dtype=I32, device=DEV)
    refs[[0, 3, 4]] = 1  # held by somebody else
    cache = torch.randint(0, 256, (layers, pages, hk, ps * d * 9 // 8), dtype=U8, device=DEV)
    gs = gpu([50.0], F32)
    k0, v0 = (torch.as_tensor(rng.normal(size=(layers, 1, 21, hk, d))).to(BF16).to(DEV) for _ in range(2))
    new = torch.tensor([21, -1, -1, -1], dtype=I32, device=DEV)
    sk.kv_resize(new, cache, table, lens, refs, ps)
    for l in range(layers):
        sk.kv_append(k0[l], v0[l], gs, gs, cache[l], table[:1], lens[:1], ps)
    parents = torch.tensor([-1, 0, 0, 0], dtype=I32, device=DEV)
    assert not host(sk.kv_fork(parents, table, lens, refs, ps)).any()
    told = [[np.concatenate([bits(k0[l])[0]], 0) for l in range(layers)] for _ in range(rows)]
    told_v = [[bits(v0[l])[0] for l in range(layers)] for _ in range(rows)]

    qkv = torch.zeros(layers, rows * t, (hq + 2 * hk) * d, dtype=BF16, device=DEV)
    outs = torch.zeros(layers, rows, t, hq, d, dtype=BF16, device=DEV)
    ws = torch.zeros(sk.attn_nvfp4_workspace(rows, t, hq, hk, d), dtype=U8, device=DEV)
    ws_r = torch.zeros(sk.kv_resize_workspace(rows, pages), dtype=U8, device=DEV)
    status = torch.zeros(rows, dtype=I32, device=DEV)
    want = torch.zeros(rows, dtype=I32, device=DEV)

    def step():
        sk.kv_resize(want, cache, table, lens, refs, ps, status=status, workspace=ws_r)
        for l in range(layers):
            q, k, v = (x.unflatten(0, (rows, t)).unflatten(2, (-1, d))
                       for x in qkv[l].split([hq * d, hk * d, hk * d], 1))
            sk.kv_append(k, v, gs, gs, cache[l], table, lens, ps)
            sk.attn_nvfp4(q, gs, gs, cache[l], table, lens, ps, out=outs[l], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = [x.clone() for x in (cache, table, lens, refs)]
    with torch.cuda.stream(side):
        want.fill_(-1)
        step()  # once before it is captured
    torch.cuda.synchronize()
    for x, y in zip((cache, table, lens, refs), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()

    alive = [True] * rows
    for at in range(9):
        if at == 4:  # a sample is given up, the rest moves together
            gone = torch.tensor([-1, 0, -1, -1], dtype=I32, device=DEV)
            sk.kv_resize(gone, cache, table, lens, refs, ps)
            sk.kv_compact(cache, table, lens, refs, ps)
            assert int((refs > 0).sum()) == int((refs > 0).nonzero().max()) + 1
            alive[1] = False
            told[1], told_v[1] = [[x[:0] for x in told[1]], [x[:0] for x in told_v[1]]]
        new = torch.as_tensor(rng.normal(size=tuple(qkv.shape))).to(BF16)
        qkv.copy_(new)
        want.copy_(torch.tensor([len(told[i][0]) + t if alive[i] else -1 for i in range(rows)], dtype=I32))
        graph.replay()
        torch.cuda.synchronize()
        assert not host(status).any()
        x = new.view(layers, rows, t, -1, d)
        n = host(lens)
        for l in range(layers):
            for i in range(rows):
                if alive[i]:
                    told[i][l] = np.concatenate([told[i][l], bits(x[l, i, :, hq:hq + hk])], 0)
                    told_v[i][l] = np.concatenate([told_v[i][l], bits(x[l, i, :, hq + hk:])], 0)
            # every row in pages of its own, filled by the statement
            own = np.arange(rows * width, dtype=np.int32).reshape(rows, width)
            ref = np.zeros((rows * width, hk, ps * d * 9 // 8), np.uint8)
            for i in range(rows):
                m = len(told[i][l])
                assert m == n[i]
                if m:
                    ref = oc.append(told[i][l][None], told_v[i][l][None], 50.0, 50.0, ref, own[i:i + 1], np.array([m]), ps)
            r = oc.attn(host(x[l, :, :, :hq]), 50.0, 50.0, ref, own, n, ps)
            off = np.abs(host(outs[l]) - r[0])
            assert np.all(off <= attn_bounds(r, d, n.max())[0])


def test_two_streams_at_once(sk):
    rng = np.random.default_rng(22)
    lens = [3000, 17]
    table = random_table(rng, lens, 47, 60, 64)
    cache = random_cache(rng, 60, 2, 64, 128)
    q = [torch.as_tensor(rng.normal(size=(2, 1, 16, 128))).to(BF16).to(DEV) for _ in range(2)]
    one, c, tb, ln = gpu([5.0], F32), gpu(cache, U8), gpu(table, I32), gpu(lens, I32)
    alone = [sk.attn_nvfp4(x, one, one, c, tb, ln, 64)[0] for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(20):
        got = [sk.attn_nvfp4(x, one, one, c, tb, ln, 64, stream=s)[0] for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, got))


def test_tensors_of_other_devices_and_strides_are_refused(sk):
    c = torch.zeros(4, 1, 1152, dtype=U8, device=DEV)
    table, lens = torch.zeros(1, 2, dtype=I32, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    one, q = torch.ones(1, device=DEV), torch.zeros(1, 1, 2, 64, dtype=BF16, device=DEV)
    with pytest.raises(ValueError, match="lens"):
        sk.attn_nvfp4(q, one, one, c, table, lens.cpu(), 16)
    with pytest.raises(ValueError, match="q: needs"):
        sk.attn_nvfp4(q.transpose(2, 3).contiguous().transpose(2, 3), one, one, c, table, lens, 16)
    with pytest.raises(ValueError, match="q_heads"):
        sk.attn_nvfp4(q, one, one, torch.zeros(4, 4, 1152, dtype=U8, device=DEV), table, lens, 16)
    with pytest.raises(ValueError, match="table"):
        sk.attn_nvfp4(q, one, one, c, torch.zeros(1, 4, dtype=I32, device=DEV)[:, ::2], lens, 16)
    with pytest.raises(ValueError, match="workspace"):
        sk.attn_nvfp4(q, one, one, c, table, lens, 16, workspace=torch.zeros(256, dtype=U8, device=DEV))
    with pytest.raises(ValueError, match="refs"):
        sk.kv_fork(lens, table, lens, torch.zeros(4, device=DEV), 16)
