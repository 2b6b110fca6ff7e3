"""Rows of a batch that bring no tokens, or fewer than others (sk_kv_append_ex): what they
have cached, and rows that share it, stay as they are (GPU)."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_gpu_cache import BF16, DEV, F32, I32, U8, bits, gpu, host, put, random_state, random_table, sk  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,t,hk,d,ps", [(1, 1, 1, 64, 16), (7, 1, 8, 128, 64), (9, 4, 2, 64, 16), (40, 5, 3, 128, 32),
                                         (6, 70, 1, 64, 64), (3, 2, 40, 128, 16)])
def test_append_of_some_rows(sk, b, t, hk, d, ps):  # noqa: F811
    rng = np.random.default_rng(b * t)
    width = -(-200 // ps)
    lens = rng.integers(0, 200, b)
    pages = int((-(-lens // ps)).sum()) + 2
    table = random_table(rng, lens, width, pages, ps)
    cache = rng.integers(0, 256, (pages, hk, ps * d * 9 // 8)).astype(np.uint8)
    x = torch.as_tensor(rng.normal(size=(2, b, t, hk, d))).to(BF16)
    kind = rng.integers(0, 4, b)
    new = np.where(kind == 0, -1, np.where(kind == 1, lens + 3, lens)).astype(np.int32)
    fresh = rng.integers(-1, t + 2, b).astype(np.int32)
    fresh[-1] = rng.choice([-2 ** 31, 2 ** 31 - 1])
    one = gpu([90.0], F32)
    for n, f in ((new, None), (None, fresh), (new, fresh)):
        c = gpu(cache, U8)
        sk.kv_append(x[0].to(DEV), x[1].to(DEV), one, one, c, gpu(table, I32), gpu(lens, I32), ps,
                     new_lens=None if n is None else gpu(n, I32), fresh=None if f is None else gpu(f, I32))
        want = oc.append(bits(x[0]), bits(x[1]), 90.0, 90.0, cache, table, lens, ps, n, f)
        assert np.array_equal(host(c), want)


def test_append_to_rows_whose_length_is_out_of_range(sk):  # noqa: F811
    # a resize refuses them, although they "have" what they were to have
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 256, (4, 1, 1152)).astype(np.uint8)
    x = torch.as_tensor(rng.normal(size=(3, 4, 1, 64))).to(BF16).to(DEV)
    lens = gpu([33, -3, 2 ** 31 - 1], I32)
    c, one = gpu(cache, U8), gpu([1.0], F32)
    sk.kv_append(x, x, one, one, c, gpu([[0, 1], [2, 3], [2, 3]], I32), lens, 16, new_lens=lens)
    assert np.array_equal(host(c), cache)


@pytest.mark.parametrize("free", [0, 1, 3, 7])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_resize_and_append_of_rows_that_share_pages(sk, free, seed):  # noqa: F811
    """Rows of forks grow with too few free pages, some wait, each brings as many tokens as it
    grows by: afterwards every row that was not served reads what it read before, every other
    one that and its tokens behind it; from a captured graph too."""
    rng = np.random.default_rng(seed)
    rows, width, ps, t, d = 12, 6, 16, 5, 64
    cache, table, lens, refs = random_state(rng, rows, width, 60, ps, 1, 0.6, fill=0.6)
    spare = np.flatnonzero(refs == 0)
    refs[rng.permutation(spare)[free:]] = 1  # held by others
    grow = rng.integers(0, t + 1, rows).astype(np.int32)
    new = np.where(rng.random(rows) < 0.3, -1, lens + grow).astype(np.int32)
    x = torch.as_tensor(rng.normal(size=(2, rows, t, 1, d))).to(BF16)
    gs = gpu([90.0], F32)
    kd, vd, nl, fr = x[0].to(DEV), x[1].to(DEV), gpu(new, I32), gpu(grow, I32)
    ws = torch.zeros(sk.kv_resize_workspace(rows, 60), dtype=U8, device=DEV)
    c, tb, ln, rf = put(cache, table, lens, refs)
    status = torch.zeros(rows, dtype=I32, device=DEV)

    def step():
        sk.kv_resize(nl, c, tb, ln, rf, ps, status=status, workspace=ws)
        sk.kv_append(kd, vd, gs, gs, c[0], tb, ln, ps, new_lens=nl, fresh=fr)

    def tokens(cache, row, n):  # codes and scales of the first n tokens of a row of the table
        p = oc.parts(cache[0], ps, d)
        at = [(row[i // ps], i % ps) for i in range(n)]
        return [[p[0][a, 0, i].tolist(), p[1][a, 0, i].tolist(), p[2][a, 0, i].tolist(), p[3][a, 0, :, i].tolist()]
                for a, i in at]

    step()
    own = np.arange(rows * width, dtype=np.int32).reshape(rows, width)
    blank = np.zeros((1, rows * width, 1, 1152), np.uint8)
    results = [[host(y) for y in (status, c, tb, ln, rf)]]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step()
    for y, z in zip((c, tb, ln, rf), put(cache, table, lens, refs)):
        y.copy_(z)
    graph.replay()
    results.append([host(y) for y in (status, c, tb, ln, rf)])
    for st, c1, t1, n1, _ in results:
        assert any(st == 1) or free > 1
        for i in range(rows):
            before = tokens(cache, table[i], lens[i])
            served = new[i] >= 0 and st[i] == 0
            assert n1[i] == (new[i] if served else lens[i])
            if served and grow[i]:
                alone = oc.append(bits(x[0, i:i + 1]), bits(x[1, i:i + 1]), 90.0, 90.0, blank[0], own[i:i + 1],
                                  n1[i:i + 1], ps, fresh=grow[i:i + 1])
                before = before + tokens(alone[None], own[i], n1[i])[lens[i]:]
            assert tokens(c1, t1[i], n1[i]) == before


def test_rows_that_ask_for_more_pages_than_32_bits_count(sk):  # noqa: F811
    # 70 rows, 66 of which want the 2^26 pages that a row of the table has places for: 2^32 and more
    rows, width, ps, pages = 70, 2 ** 26, 16, 9
    table = torch.full((rows, width), -1, dtype=I32, device=DEV)
    table[3, 0] = 5
    lens, refs = torch.zeros(rows, dtype=I32, device=DEV), torch.zeros(pages, dtype=I32, device=DEV)
    lens[3], refs[5] = 7, 1
    cache = torch.full((1, pages, 1, 1152), 9, dtype=U8, device=DEV)
    new = torch.full((rows,), 2 ** 30, dtype=I32, device=DEV)
    new[0], new[2], new[-1], new[-2] = 17, -1, 0, 1
    status, _ = sk.kv_resize(new, cache, table, lens, refs, ps)
    # served before the first refusal: row 0; rows that need no page: 2 and the last; row 68 needs one
    want = torch.ones(rows, dtype=I32)
    want[0] = want[2] = want[-1] = 0
    assert torch.equal(status.cpu(), want)
    assert lens.tolist() == [17, 0, 0, 7] + [0] * (rows - 4) and refs.tolist() == [1, 1, 0, 0, 0, 1, 0, 0, 0]
    assert table[0, :2].tolist() == [0, 1] and int(table[3, 0]) == 5 and (cache == 9).all()
    table[0, :2] = table[3, 0] = -1
    assert all((table[i] == -1).all() for i in range(rows))
