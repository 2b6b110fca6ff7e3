"""Host-side checks of the int8 routed experts' entry points: every refusal
comes before any CUDA call, with a status and a message (no GPU)."""
import ctypes

import pytest
import torch

P = 1 << 20  # an aligned address that nothing reads
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def sk():
    from nvfp4_sm_skinny_gb300 import build

    build.build()
    import nvfp4_sm_skinny_gb300 as sk

    return sk


ROUTE = dict(logits=P, logits_type=1, bias=P, ids=P, weights=P, m=4, n_experts=64, n_groups=8,
             topk_groups=4, top_k=8, score=1, renormalize=1, scale=1.0, stream=None)


@pytest.mark.parametrize("change,word", [
    (dict(logits_type=2), "logits_type"), (dict(score=2), "score"), (dict(m=0), "m=0"),
    (dict(m=-3), "m=-3"), (dict(n_experts=0), "n_experts"), (dict(n_experts=1032), "n_experts"),
    (dict(n_groups=0), "n_groups"), (dict(n_groups=7), "n_groups"), (dict(n_groups=64), "n_groups"),
    (dict(topk_groups=0), "topk_groups"), (dict(topk_groups=9), "topk_groups"),
    (dict(top_k=0), "top_k"), (dict(top_k=17), "top_k"), (dict(topk_groups=1, top_k=9), "top_k"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(logits=None), "logits"), (dict(logits=P + 2), "logits"), (dict(bias=P + 2), "bias"),
    (dict(ids=None), "ids"), (dict(weights=P + 1), "weights"),
])
def test_route_refusals(sk, change, word):
    assert sk.lib().sk_route(*{**ROUTE, **change}.values()) == 1
    assert word in sk.last_error()


@pytest.mark.parametrize("z,q,scale,m,n,word", [
    (P, P, P, 0, 64, "m=0"), (P, P, P, 1, 0, "n=0"), (P, P, P, 1, 24, "n=24"),
    (P, P, P, 1, 131072, "n=131072"), (None, P, P, 1, 64, "z"), (P + 8, P, P, 1, 64, "z"),
    (P, P + 4, P, 1, 64, "q"), (P, P, P + 2, 1, 64, "scale"), (P, P, None, 1, 64, "scale"),
])
def test_quantize_refusals(sk, z, q, scale, m, n, word):
    assert sk.lib().sk_int8_quantize(z, q, scale, m, n, None) == 1
    assert word in sk.last_error()


GEMM = dict(xq=P, x_scale=P, wq=P, w_scale=P, y=P, m=1, n=128, k=256, splits=0, stream=None)


@pytest.mark.parametrize("change,status,word", [
    (dict(m=0), 1, "m=0"), (dict(m=17), 1, "m=17"), (dict(n=0), 1, "n=0"),
    (dict(n=2 ** 30 + 1), 1, "n=1073741825"), (dict(n=2 ** 31 - 1), 1, "n=2147483647"), (dict(k=0), 1, "k=0"),
    (dict(k=24), 1, "k=24"), (dict(k=131072), 1, "k=131072"), (dict(splits=3), 2, "split"),
    (dict(splits=16), 2, "split"), (dict(xq=None), 1, "xq"), (dict(wq=P + 8), 1, "wq"),
    (dict(y=P + 2), 1, "y "), (dict(x_scale=P + 2), 1, "x_scale"), (dict(w_scale=None), 1, "w_scale"),
])
def test_gemm_refusals(sk, change, status, word):
    a = {**GEMM, **change}
    assert sk.lib().sk_gemm_int8(*a.values()) == status
    assert word in sk.last_error()
    if set(change) & {"m", "n", "k", "splits"}:
        assert sk.lib().sk_gemm_int8_supported(a["m"], a["n"], a["k"], a["splits"]) == status
        assert word in sk.gemm_int8_supported(a["m"], a["n"], a["k"], a["splits"])


def test_gemm_supported(sk):
    for shape in ((1, 1, 16, 0), (16, 8192, 8192, 8), (5, 4100, 2064, 2), (16, 17, 131056, 0)):
        assert sk.gemm_int8_supported(*shape) is None


EXPERTS = dict(xq=P, x_scale=P, w13=P, s13=P, w2=P, s2=P, ids=P, weights=P, y=P, workspace=P,
               workspace_bytes=1 << 30, m=2, n_experts=8, top_k=2, hidden=64, inter=32, stream=None)


@pytest.mark.parametrize("change,status,word", [
    (dict(m=0), 1, "m=0"), (dict(m=17), 1, "m=17"), (dict(n_experts=0), 1, "n_experts"),
    (dict(n_experts=1025), 1, "n_experts"), (dict(top_k=0), 1, "top_k"), (dict(top_k=17), 1, "top_k"),
    (dict(hidden=40), 1, "hidden"), (dict(inter=8), 1, "inter"), (dict(inter=131072), 1, "inter"),
    (dict(w13=None), 1, "w13"), (dict(w2=P + 8), 1, "w2"), (dict(ids=P + 2), 1, "ids"),
    (dict(workspace=P + 16), 1, "workspace"), (dict(workspace_bytes=1024), 4, "workspace"),
])
def test_experts_refusals(sk, change, status, word):
    assert sk.lib().sk_experts_int8(*{**EXPERTS, **change}.values()) == status
    assert word in sk.last_error()


def test_experts_workspace(sk):
    # act and codes and scales of every choice, outputs of every choice
    assert sk.experts_int8_workspace(3, 2, 64, 32) == 6 * 32 * 4 + 256 + 256 + 6 * 64 * 4
    assert sk.experts_int8_workspace(16, 16, 131056, 131056) > 1 << 27
    assert sk.experts_int8_workspace(17, 2, 64, 32) == 0 and "m=17" in sk.last_error()


def test_valid_calls_without_gpu_report_a_device_error(sk):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    L = sk.lib()
    for st in (L.sk_route(*ROUTE.values()), L.sk_int8_quantize(P, P, P, 1, 64, None),
               L.sk_gemm_int8(*GEMM.values()), L.sk_experts_int8(*EXPERTS.values())):
        assert st in (3, 5) and sk.last_error()


def test_binding_refuses_other_tensors(sk):
    def t(*shape, dtype=torch.int8):
        return torch.zeros(*shape, dtype=dtype)

    f = torch.float32
    with pytest.raises(ValueError, match="logits"):
        sk.route(t(2, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="CUDA"):
        sk.route(t(2, 8, dtype=f), 2)
    with pytest.raises(ValueError, match="z"):
        sk.int8_quantize(t(2, 32, dtype=f))
    with pytest.raises(ValueError, match="xq"):
        sk.gemm_int8(t(2, 32, dtype=torch.uint8), t(2, dtype=f), t(4, 32), t(4, dtype=f))
    with pytest.raises(ValueError, match="xq"):
        sk.experts_int8(t(2, 32, dtype=f), t(2, dtype=f), t(4, 32, 32), t(4, 32, dtype=f), t(4, 32, 16),
                        t(4, 32, dtype=f), t(2, 2, dtype=torch.int32), t(2, 2, dtype=f))


def test_binding_refuses_other_devices(sk, monkeypatch):
    class Tensor:
        def __init__(self, dev):
            self.dev, self.device = dev, f"cuda:{dev}"

        def get_device(self):
            return self.dev

    class Stream:
        cuda_stream = 5

        def __init__(self, dev):
            self.device = torch.device("cuda", dev)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 7, raising=False)
    assert sk._launch_on(None, 0, Tensor(0), None) == 7
    assert sk._launch_on(Stream(0), 0, Tensor(0)) == 5
    with pytest.raises(ValueError, match="one device"):
        sk._launch_on(None, 0, Tensor(0), Tensor(1))
    with pytest.raises(ValueError, match="current"):
        sk._launch_on(None, 1, Tensor(1))
    with pytest.raises(ValueError, match="current"):
        sk._launch_on(Stream(1), 0, Tensor(0))


@pytest.mark.parametrize("change,message", [
    (dict(z=None), "sk_int8_quantize: z is a null pointer"), (dict(z=P + 8), "sk_int8_quantize: z (0x100008) is not 16-byte"),
    (dict(q=None), "sk_int8_quantize: q is a null pointer"), (dict(q=P + 4), "sk_int8_quantize: q (0x100004) is not 16-byte"),
    (dict(scale=None), "sk_int8_quantize: scale is a null"), (dict(scale=P + 2), "sk_int8_quantize: scale (0x100002) is not 4-byte"),
])
def test_quantize_refusals_name_the_argument(sk, change, message):
    a = {**dict(z=P, q=P, scale=P, m=1, n=64, stream=None), **change}
    assert sk.lib().sk_int8_quantize(*a.values()) == 1
    assert sk.last_error().startswith(message)


def test_binding_refusals_name_the_argument(sk):
    def t(*shape, dtype=torch.int8):
        return torch.zeros(*shape, dtype=dtype)

    f = torch.float32
    with pytest.raises(ValueError, match="^z: dtype"):
        sk.int8_quantize(t(2, 32, dtype=f))
    with pytest.raises(ValueError, match="^xq: dtype"):
        sk.gemm_int8(t(2, 32, dtype=torch.uint8), t(2, dtype=f), t(4, 32), t(4, dtype=f))
    with pytest.raises(ValueError, match="^logits: dtype"):
        sk.route(t(2, 8, dtype=torch.float16), 2)


def test_binding_refuses_sizes_beyond_32_bits(sk, monkeypatch):
    # the C arguments are 32-bit: 2^32 + 4 rows would run as 4
    class Tensor:
        is_cuda, device = True, "cuda:0"

        def __init__(self, dtype, *shape):
            self.dtype, self.shape = dtype, torch.Size(shape)

        def is_contiguous(self):
            return True

        def get_device(self):
            return 0

        def data_ptr(self):
            return P

        def numel(self):
            return self.shape.numel()

    class Lib:
        def __getattr__(self, name):
            raise AssertionError(f"{name} is called")

    monkeypatch.setattr(sk, "lib", Lib)
    monkeypatch.setattr(sk, "_launch_on", lambda *args: 0)
    bf, f, i8, i32, many = torch.bfloat16, torch.float32, torch.int8, torch.int32, 2 ** 32
    for change in (dict(), dict(n_groups=many + 1), dict(n_groups=1 - many), dict(topk_groups=many + 1)):
        m = 2 if change else many + 4
        with pytest.raises(ValueError, match=f"^{next(iter(change), 'm')}=-?429496"):
            sk.route(Tensor(bf, m, 8), 2, ids=Tensor(i32, m, 2), weights=Tensor(f, m, 2), **change)
    with pytest.raises(ValueError, match="^m=4294967297"):
        sk.int8_quantize(Tensor(bf, many + 1, 16), q=Tensor(i8, many + 1, 16), scale=Tensor(f, many + 1))
    for m, n, k, splits in ((1, many + 5, 16, 0), (many + 1, 8, 16, 0), (1, 8, many + 16, 0), (1, 8, 16, many)):
        with pytest.raises(ValueError, match="=429496"):
            sk.gemm_int8(Tensor(i8, m, k), Tensor(f, m), Tensor(i8, n, k), Tensor(f, n), out=Tensor(bf, m, n), splits=splits)
        assert "=429496" in sk.gemm_int8_supported(m, n, k, splits)
    for m, e, k, hidden, inter in ((1, 1, many + 2, 16, 16), (1, 1, 2, many + 16, 16), (1, 1, 2, 16, many + 16),
                                   (1, many + 1, 2, 16, 16), (many + 1, 1, 2, 16, 16)):
        assert max(m, k, hidden, inter) < many or sk.experts_int8_workspace(m, k, hidden, inter) == 0
        with pytest.raises(ValueError, match="=429496"):
            sk.experts_int8(Tensor(i8, m, hidden), Tensor(f, m), Tensor(i8, e, 2 * inter, hidden), Tensor(f, e, 2 * inter),
                            Tensor(i8, e, hidden, inter), Tensor(f, e, hidden), Tensor(i32, m, k), Tensor(f, m, k),
                            out=Tensor(bf, m, hidden), workspace=Tensor(torch.uint8, 4096))


@pytest.mark.parametrize("experts", [0, 4])
def test_chain_hints_name_the_next_gemm(sk, monkeypatch, experts):
    from nvfp4_sm_skinny_gb300 import chain

    c = chain.DecodeChain.__new__(chain.DecodeChain)
    c.L, c.m, c.experts, c.prefetch_next, c.splits, c.eps, c.gc = 2, 1, experts, True, 0, 0.0, 0.0
    for name in ("w_o", "w_p", "w_u", "w_r"):
        setattr(c, name, [f"{name}{l}" for l in range(c.L)])
    for name, n in (("ws_o", chain.H), ("ws_p", chain.P)):
        setattr(c, name, torch.zeros(c.L, 2 * n, dtype=torch.uint8))
    c.h, c.u, c.z = ([None] * (c.L + 1) for _ in range(3))
    calls = []
    monkeypatch.setattr(sk, "gemm_prefetch_next", lambda w: calls.append(("hint", w)))
    monkeypatch.setattr(sk, "gemm_bf16", lambda x, w, **kw: calls.append(("gemm", w)))
    c.gemms_only()
    order = [f"{name}{l}" for l in range(c.L) for name in ("w_o", "w_p", "w_u")]
    assert calls == [call for w, ahead in zip(order, order[1:] + [None]) for call in (("hint", ahead), ("gemm", w))]
    assert c.next_weight(0, 1) == ("w_r0" if experts else "w_u0")  # with routed experts the router's GEMM follows
