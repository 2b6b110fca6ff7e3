"""Pins of the 64-bit statement of the 4-bit key/value cache (oracle/cache.py)
against hand-worked layouts, closed forms and invariants (no GPU)."""
import numpy as np
import pytest

from oracle import cache as oc


@pytest.fixture(autouse=True)
def _built(oracle_mod):
    return oracle_mod


def bf16_bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_parts_name_the_bytes_of_a_block():
    ps, d = 16, 64
    block = np.arange(ps * d * 9 // 8, dtype=np.int64)
    kc, vc, ks, vs = oc.parts(block, ps, d)
    assert kc.shape == vc.shape == (16, 32) and ks.shape == (16, 4) and vs.shape == (4, 16)
    assert kc[3, 5] == 3 * 32 + 5 and vc[0, 0] == 512 and vc[15, 31] == 1023
    assert ks[2, 1] == 1024 + 9 and vs[1, 2] == 1024 + 64 + 18
    a = np.zeros((2, 3, ps * d * 9 // 8), np.uint8)
    oc.parts(a, ps, d)[3][1, 2, 3, 4] = 7  # a view of the cache
    assert a[1, 2, 1024 + 64 + 3 * 16 + 4] == 7


def test_append_puts_exact_values_where_they_belong():
    # gs 1: a block with amax 6 has scale 1, and its values are the codes' own
    ps, d, hk = 16, 64, 2
    cache = np.full((3, hk, ps * d * 9 // 8), 0xAA, np.uint8)
    table = np.array([[2, 0, -1]], np.int32)
    k = np.zeros((1, 2, hk, d), np.float32)
    k[..., 0::16] = 6.0
    k[..., 1] = -0.5
    k[0, 1, 1, 17] = 3.0
    out = oc.append(bf16_bits(k), bf16_bits(2 * k), 1.0, 1.0, cache, table, np.array([17]), ps)
    kc, vc, ks, vs = oc.parts(out, ps, d)
    # token 0 is position 15 (page 2, place 15), token 1 position 16 (page 0, place 0)
    assert kc[2, 0, 15, 0] == 0x97 and kc[0, 1, 0, 8] == 0x57 and ks[2, 0, 15, 0] == 0x38
    assert vs[0, 1, 1, 0] == 0x40 and vc[0, 1, 0, 8] == 0x57
    kk, there = oc.keys(out, table[0], 17, ps, d, 1.0, 0)
    assert there.all() and np.array_equal(kk[:, 15:], k[0].transpose(1, 0, 2))
    vv, _ = oc.keys(out, table[0], 17, ps, d, 1.0, 1)
    assert np.array_equal(vv[:, 15:], 2 * k[0].transpose(1, 0, 2))
    kept = oc.append(bf16_bits(k), bf16_bits(k), 1.0, 1.0, cache, table, np.array([1]), ps)
    assert (kept != cache).any() and np.array_equal(kept[:2], cache[:2])  # position -1 is left out
    none = oc.append(bf16_bits(k), bf16_bits(k), 1.0, 1.0, cache, np.array([[7, -1, 3]]), np.array([18]), ps)
    assert np.array_equal(none, cache)


def random_cache(rng, pages, hk, ps, d):
    cache = rng.integers(0, 256, (pages, hk, ps * d * 9 // 8)).astype(np.uint8)
    for p in oc.parts(cache, ps, d)[2:]:
        p[...] = rng.integers(0x20, 0x50, p.shape)
    return cache


@pytest.mark.parametrize("window", [0, 5])
def test_attention_by_brute_force(window):
    rng = np.random.default_rng(1)
    ps, d, hk, hq, t, n = 16, 64, 2, 6, 3, 37
    cache = random_cache(rng, 5, hk, ps, d)
    table = np.array([[4, 1, 3, 0]], np.int32)
    q = rng.normal(size=(1, t, hq, d))
    out, lse, size, reach, _ = oc.attn(q, 2.0, 4.0, cache, table, np.array([n]), ps, scale=0.25, window=window)
    kk, _ = oc.keys(cache, table[0], n, ps, d, 2.0, 0)
    vv, _ = oc.keys(cache, table[0], n, ps, d, 4.0, 1)
    for j in range(t):
        pos = n - t + j
        lo = max(0, pos - window + 1) if window else 0
        for h in range(hq):
            w = [np.exp(0.25 * sum(q[0, j, h, c] * kk[h // 3, k, c] for c in range(d))) for k in range(lo, pos + 1)]
            ref = sum(x * vv[h // 3, k] for x, k in zip(w, range(lo, pos + 1))) / sum(w)
            assert np.allclose(out[0, j, h], ref, rtol=1e-12, atol=1e-12)
            assert np.isclose(lse[0, j, h], np.log(sum(w)), rtol=1e-12)
    assert (size >= np.abs(out) - 1e-12).all() and (reach > 0).all()


def test_attention_of_nothing_is_zero():
    rng = np.random.default_rng(2)
    cache = random_cache(rng, 2, 1, 16, 64)
    q = rng.normal(size=(3, 2, 1, 64))
    table = np.array([[0, -1], [1, 0], [-1, 9]], np.int32)
    out, lse, _, _, mass = oc.attn(q, 1.0, 1.0, cache, table, np.array([0, 1, 20]), 16)
    assert not out[0].any() and not out[1, 0].any() and out[1, 1].any() and not out[2].any()
    assert (lse[0] == -np.inf).all() and lse[1, 1, 0] > -np.inf
    v = oc.keys(cache, table[1], 1, 16, 64, 1.0, 1)[0]
    assert np.allclose(out[1, 1, 0], v[0, 0])  # one key: its value
    assert np.allclose(mass[1, 1, 0], np.abs(v[0, 0])) and not mass[1, 0].any()


def state():
    """Rows 0 and 1 share page 3 (full) and page 0 (4 of 16 tokens); row 2 has page 5."""
    table = np.full((4, 4), -1, np.int32)
    table[0, :2] = table[1, :2] = 3, 0
    table[2, 0] = 5
    lens = np.array([20, 20, 16, 0], np.int32)
    refs = np.array([2, 0, 0, 2, 0, 1, 0, 0], np.int32)
    cache = np.arange(2 * 8 * 4, dtype=np.uint8).reshape(2, 8, 4)
    return cache, table, lens, refs


def test_resize_by_hand():
    cache, table, lens, refs = state()
    st, c, t, n, r = oc.resize(np.array([21, 40, -1, 5]), cache, table, lens, refs, 16)
    assert not st.any() and list(n) == [21, 40, 16, 5]
    # row 0 copies page 0 to 1; row 1 holds it alone by then, and adds 2; row 3 gets 4
    assert list(t[0]) == [3, 1, -1, -1] and list(t[1]) == [3, 0, 2, -1] and list(t[3]) == [4, -1, -1, -1]
    assert list(r) == [1, 1, 1, 2, 1, 1, 0, 0]
    assert np.array_equal(c[:, 1], cache[:, 0]) and np.array_equal(c[:, 2:], cache[:, 2:])
    st, _, t, n, r = oc.resize(np.array([3, 0, 0, 65]), cache, table, lens, refs, 16)
    assert list(st) == [0, 0, 0, 2] and list(n) == [3, 0, 0, 0] and list(r) == [0, 0, 0, 1, 0, 0, 0, 0]
    # of the free pages 1, 2, 4, 6, 7 row 0 takes three and row 1 two; none is left for row 3
    st, _, t, n, r = oc.resize(np.array([64, 60, 3, 1]), cache, table, lens, refs, 16)
    assert list(st) == [0, 0, 0, 1] and list(n) == [64, 60, 3, 0]
    assert list(t[0]) == [3, 1, 2, 4] and list(t[1]) == [3, 0, 6, 7] and list(r) == [1, 1, 1, 2, 1, 1, 1, 1]
    refs[[1, 2, 4]] = 1
    st, _, t, n, r = oc.resize(np.array([64, 22, 3, 1]), cache, table, lens, refs, 16)
    # row 0 needs three of two; row 1 would have kept page 0 alone, but row 0 still holds it
    assert list(st) == [1, 1, 0, 1] and list(n) == [20, 20, 3, 0] and np.array_equal(t[:2], table[:2])


def test_fork_by_hand():
    _, table, lens, refs = state()
    st, t, n, r = oc.fork(np.array([2, 0, -1, 0]), table, lens, refs, 16)
    assert not st.any() and list(n) == [16, 20, 16, 20]
    assert list(t[0]) == [5, -1, -1, -1] and list(t[3, :2]) == [3, 0]
    assert list(r) == [2, 0, 0, 2, 0, 2, 0, 0]
    st, t, n, r = oc.fork(np.array([0, 4, 3, -5]), table, lens, refs, 16)
    assert list(st) == [0, 2, 0, 0] and list(n) == [20, 20, 0, 0] and list(r) == [2, 0, 0, 2, 0, 0, 0, 0]


def test_compact_by_hand():
    cache, table, lens, refs = state()
    m, c, t, r = oc.compact(cache, table, lens, refs, 16)
    assert list(m) == [0, -1, -1, 1, -1, 2, -1, -1] and list(r) == [2, 2, 1, 0, 0, 0, 0, 0]
    assert list(t[0, :2]) == [1, 0] and t[2, 0] == 2
    assert np.array_equal(c[:, 1], cache[:, 3]) and np.array_equal(c[:, 2], cache[:, 5])
