"""Host-side checks of the 4-bit cache's entry points: every refusal comes before
any CUDA call, with a status and a message that names the argument (no GPU)."""
import ctypes

import pytest
import torch

P = 1 << 20  # an aligned address that nothing reads
BIG = 1 << 40


@pytest.fixture(scope="module")
def sk():
    from nvfp4_sm_skinny_gb300 import build

    build.build()
    import nvfp4_sm_skinny_gb300 as sk

    return sk


APPEND = dict(k=P, v=P, k_gs=P, v_gs=P, cache=P, table=P, lens=P, b=2, t=1, kv_heads=8, head_dim=64,
              page_size=64, pages=10, width=4, k_stride=512, v_stride=512, stream=None)
ATTN = dict(q=P, k_gs=P, v_gs=P, cache=P, table=P, lens=P, out=P, lse=P, workspace=P,
            workspace_bytes=BIG, b=2, t=1, q_heads=64, kv_heads=8, head_dim=64, page_size=64, pages=10,
            width=4, q_stride=4096, scale=0.125, window=0, stream=None)
RESIZE = dict(new_lens=P, cache=P, table=P, lens=P, refs=P, status=P, workspace=P, workspace_bytes=BIG,
              rows=4, width=8, pages=100, layers=2, kv_heads=8, head_dim=64, page_size=16, stream=None)
FORK = dict(parents=P, table=P, lens=P, refs=P, status=P, rows=4, width=8, pages=100, page_size=16,
            stream=None)
COMPACT = dict(cache=P, table=P, lens=P, refs=P, page_map=P, workspace=P, workspace_bytes=BIG, rows=4,
               width=8, pages=100, layers=2, kv_heads=8, head_dim=64, page_size=16, stream=None)


def refused(sk, call, args, change, word, status=1):
    assert getattr(sk.lib(), call)(*{**args, **change}.values()) == status
    assert word in sk.last_error()


@pytest.mark.parametrize("change,word", [
    (dict(b=0), "b=0"), (dict(b=2 ** 20 + 1), "b="), (dict(t=0), "t=0"), (dict(t=2 ** 24), "b * t"),
    (dict(kv_heads=0), "kv_heads"), (dict(kv_heads=1025), "kv_heads"), (dict(head_dim=96), "head_dim"),
    (dict(head_dim=0), "head_dim"), (dict(page_size=8), "page_size"), (dict(page_size=128), "page_size"),
    (dict(pages=0), "pages"), (dict(width=0), "width"), (dict(width=2 ** 25), "width"),
    (dict(k_stride=511), "k_stride"), (dict(k_stride=516), "k_stride"), (dict(v_stride=0), "v_stride"),
    (dict(k=None), "k is"), (dict(v=P + 8), "v ("), (dict(cache=P + 4), "cache"),
    (dict(k_gs=None), "k_global_scale"), (dict(v_gs=P + 2), "v_global_scale"),
    (dict(table=None), "table"), (dict(lens=P + 1), "lens"),
])
def test_append_refusals(sk, change, word):
    refused(sk, "sk_kv_append", APPEND, change, word)


@pytest.mark.parametrize("change,status,word", [
    (dict(b=0), 1, "b=0"), (dict(t=0), 1, "t=0"), (dict(t=2 ** 24), 1, "b * t"), (dict(q_heads=4), 1, "q_heads"),
    (dict(q_heads=60), 1, "q_heads"), (dict(q_heads=4104), 1, "q_heads"), (dict(t=2 ** 23, q_heads=128, q_stride=8192), 1, "q_heads"),
    (dict(kv_heads=0), 1, "kv_heads"), (dict(head_dim=80), 1, "head_dim"), (dict(page_size=48), 1, "page_size"),
    (dict(pages=-1), 1, "pages"), (dict(width=2 ** 25), 1, "width"), (dict(q_stride=4088), 1, "q_stride"),
    (dict(q_stride=4100), 1, "q_stride"), (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"), (dict(window=-1), 1, "window"), (dict(q=None), 1, "q is"),
    (dict(out=P + 8), 1, "out"), (dict(cache=None), 1, "cache"), (dict(lse=P + 2), 1, "lse"),
    (dict(k_gs=None), 1, "k_global_scale"), (dict(table=P + 2), 1, "table"), (dict(lens=None), 1, "lens"),
    (dict(workspace=P + 64), 1, "workspace"), (dict(workspace=None), 1, "workspace"),
    (dict(workspace_bytes=1024), 4, "workspace"),
])
def test_attn_refusals(sk, change, status, word):
    refused(sk, "sk_attn_nvfp4", ATTN, change, word, status)


@pytest.mark.parametrize("change,status,word", [
    (dict(rows=0), 1, "rows"), (dict(rows=4097), 1, "rows"), (dict(pages=0), 1, "pages"),
    (dict(width=0), 1, "width"), (dict(width=2 ** 27), 1, "width"), (dict(layers=0), 1, "layers"),
    (dict(layers=65537), 1, "layers"), (dict(kv_heads=0), 1, "kv_heads"), (dict(head_dim=32), 1, "head_dim"),
    (dict(page_size=0), 1, "page_size"), (dict(cache=P + 8), 1, "cache"), (dict(table=None), 1, "table"),
    (dict(lens=None), 1, "lens"), (dict(refs=P + 2), 1, "refs"), (dict(workspace=P + 16), 1, "workspace"),
    (dict(workspace_bytes=64), 4, "workspace"),
])
def test_pages_refusals(sk, change, status, word):
    refused(sk, "sk_kv_resize", RESIZE, change, word, status)
    refused(sk, "sk_kv_compact", COMPACT, change, word, status)
    if set(change) <= set(FORK):
        refused(sk, "sk_kv_fork", FORK, change, word, status)


@pytest.mark.parametrize("call,args,name", [
    ("sk_kv_resize", RESIZE, "new_lens"), ("sk_kv_resize", RESIZE, "status"), ("sk_kv_fork", FORK, "parents"),
    ("sk_kv_fork", FORK, "status"), ("sk_kv_compact", COMPACT, "page_map"),
])
def test_lists_have_to_be_there(sk, call, args, name):
    refused(sk, call, args, {name: None}, name)
    refused(sk, call, args, {name: P + 2}, name)


def test_sizes(sk):
    assert sk.kv_block_bytes(64, 128) == 9216 and sk.kv_block_bytes(16, 64) == 1152
    assert sk.kv_block_bytes(24, 64) == 0 and "page_size" in sk.last_error()
    assert sk.kv_block_bytes(2 ** 33, 64) == 0
    assert sk.attn_nvfp4_workspace(1, 1, 64, 8, 128) > 0 and sk.attn_nvfp4_workspace(1, 1, 60, 8, 128) == 0
    assert sk.kv_resize_workspace(4, 100) >= 4 * 24 + 400 and sk.kv_resize_workspace(5000, 100) == 0
    assert sk.kv_compact_workspace(100) >= 800 and sk.kv_compact_workspace(0) == 0


def test_valid_calls_without_gpu_report_a_device_error(sk):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    for call, args in (("sk_kv_append", APPEND), ("sk_attn_nvfp4", ATTN), ("sk_kv_resize", RESIZE),
                       ("sk_kv_fork", FORK), ("sk_kv_compact", COMPACT)):
        assert getattr(sk.lib(), call)(*args.values()) in (3, 5) and sk.last_error()


def test_binding_refuses_other_tensors(sk):
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(2, 1, 8, 64, dtype=bf)
    gs = torch.ones(1)
    cache = torch.zeros(10, 8, 4608, dtype=torch.uint8)
    table, lens = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        sk.kv_append(k, k, gs, gs, cache, table, lens, 64)
    with pytest.raises(ValueError, match="dtype"):
        sk.kv_append(k.float(), k, gs, gs, cache, table, lens, 64)
    with pytest.raises(ValueError, match="v: shape"):
        sk.kv_append(k, k[:1], gs, gs, cache, table, lens, 64)
    with pytest.raises(ValueError, match="q: dtype"):
        sk.attn_nvfp4(k.half(), gs, gs, cache, table, lens, 64)
    whole = cache[None]
    refs = torch.zeros(10, dtype=i32)
    with pytest.raises(ValueError, match="cache: shape .*needs 4 dimensions"):
        sk.kv_resize(lens, cache, table, lens, refs, 64)
    with pytest.raises(ValueError, match="cache: blocks"):
        sk.kv_compact(whole[..., :4600], table, lens, refs, 64)
    with pytest.raises(ValueError, match="cache"):
        sk.kv_resize(lens, whole, table, lens, refs, 64)
    with pytest.raises(ValueError, match="table"):
        sk.kv_fork(lens, table, lens, refs, 64)
    for bad, name in (((k[0], k, gs, gs, cache, table, lens), "k"), ((k, k, gs, gs, whole, table, lens), "cache"),
                      ((k, k, gs, gs, cache, lens, lens), "table")):
        with pytest.raises(ValueError, match="k|cache|table"):
            sk.kv_append(*bad, 64)
    with pytest.raises(ValueError, match="refs: shape"):
        sk.kv_fork(lens, table, lens, table, 64)
