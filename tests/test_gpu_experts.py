"""GPU parity of the int8 routed experts (sk_route, sk_int8_quantize,
sk_gemm_int8, sk_experts_int8) against their 64-bit statement
(oracle/experts.py). Whole numbers have to be equal; the tolerances of the
others count roundings and are stated beside each check."""
import numpy as np
import pytest
import torch

from oracle import experts as ox

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, I8, I32 = torch.float32, torch.bfloat16, torch.int8, torch.int32


@pytest.fixture(scope="module")
def sk():
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
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


# ---------------------------------------------------------------- routing ----
def check_route(sk, logits, k, bias=None, **kw):
    """ids equal; weights within (2 |d| + 96) 2^-24 of the exact ones, d the
    exponents of the chosen: the rounding of an exponent moves exp by |d| 2^-24,
    a sum of up to 1024 terms in any tree of at most 37 additions a path and the
    sum and quotient of the renormalisation add less than 96 roundings."""
    ids, w = sk.route(logits, k, bias=bias, **kw)
    torch.cuda.synchronize()
    a = host(logits)
    rids, rw = ox.route(a, k, bias=None if bias is None else host(bias), **kw)
    assert np.array_equal(host(ids), rids)
    with np.errstate(invalid="ignore"):
        top = np.where(np.isfinite(a), a, 0.0)
        d = np.abs(top).max() * 2
    assert np.all(np.abs(host(w) - rw) <= np.abs(rw) * (2 * d + 96) * ox.U + 2.0 ** -126)
    return ids, w


ROUTE = [  # m, experts, k, groups, topk_groups
    (1, 1, 1, 1, 1), (1, 16, 2, 1, 1), (3, 7, 7, 1, 1), (16, 128, 8, 1, 1), (5, 60, 4, 1, 1),
    (16, 256, 8, 8, 4), (33, 96, 6, 3, 2), (2, 1024, 16, 32, 5), (4, 1023, 16, 1, 1),
    (7, 32, 16, 32, 16), (257, 160, 6, 8, 3), (9, 33, 3, 11, 2),
]


@pytest.mark.parametrize("m,n,k,groups,topk_groups", ROUTE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route(sk, m, n, k, groups, topk_groups, score, with_bias, dtype):
    rng = np.random.default_rng(m * 1000 + n)
    logits = gpu(rng.normal(0, 1.5, (m, n)), dtype)
    bias = gpu(rng.normal(0, 0.05, n), F32) if with_bias else None
    check_route(sk, logits, k, bias, n_groups=groups, topk_groups=topk_groups, score=score)
    check_route(sk, logits, k, bias, n_groups=groups, topk_groups=topk_groups, score=score,
                renormalize=False, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3), (16, 16)])
def test_route_masks_and_specials(sk, score, with_bias, groups, topk_groups):
    inf, nan, n = np.inf, np.nan, 64
    rng = np.random.default_rng(11)
    a = rng.normal(size=(12, n)).astype(np.float32)
    a[0] = -inf                                  # nothing to choose
    a[1] = nan
    a[2, 1:] = -inf                              # one expert
    a[3, ::2] = -inf                             # half of them
    a[4, 5:] = nan
    a[5, [7, 40]] = inf                          # two take everything
    a[6] = np.finfo(np.float32).min              # the type's lowest value is a value
    a[7] = 0.0
    a[7, 3] = -0.0                               # equal to its neighbours
    a[8] = np.finfo(np.float32).max
    a[9, :8] = [inf, -inf, nan, 1, 2, 3, nan, -inf]
    a[10] = np.repeat(a[10, :8], 8)              # many equal values
    a[11] *= 60                                  # saturated sigmoids
    bias = None
    if with_bias:
        b = rng.normal(0, 0.05, n).astype(np.float32)
        b[[9, 17]] = -inf, nan                   # never chosen
        b[20] = inf                              # always chosen
        b[40:48] = 0.0
        bias = gpu(b, F32)
    ids, w = sk.route(gpu(a, F32), 8, bias=bias, n_groups=groups, topk_groups=topk_groups, score=score)
    rids, rw = ox.route(a, 8, bias=None if bias is None else b, n_groups=groups,
                        topk_groups=topk_groups, score=score)
    assert np.array_equal(host(ids), rids)
    finite = np.where(np.isfinite(a), np.abs(a), 0.0).max(1, keepdims=True)
    d = 2 * np.minimum(finite, 100.0)            # exp underflows beyond
    assert np.all(np.abs(host(w) - rw) <= np.abs(rw) * (2 * d + 96) * ox.U + 2.0 ** -126)
    assert (host(ids)[0] == -1).all() and not host(w)[0].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 4)])
def test_route_order_of_values_that_fp32_cannot_tell_apart(sk, score, groups, topk_groups):
    # logits one to three FP32 steps apart, whose scores round to the same FP32
    # value, and biases that bring far scores within less than an FP32 step
    rng = np.random.default_rng(13)
    n, k = 64, 8
    base = np.float32(1.7)
    a = (base.view(np.int32) + rng.integers(0, 3, (40, n))).astype(np.int32).view(np.float32)
    check_route(sk, gpu(a, F32), k, gpu(np.zeros(n), F32), n_groups=groups, topk_groups=topk_groups,
                score=score)
    a = rng.normal(size=(40, n)).astype(np.float32)
    a[:] = a[0]
    p = np.exp(a[0].astype(np.float64))
    p = p / p.sum() if score == "softmax" else p / (1 + p)
    b = (p.max() - p).astype(np.float32)         # p + b equal to within FP32 rounding
    check_route(sk, gpu(a, F32), k, gpu(b, F32), n_groups=groups, topk_groups=topk_groups, score=score)
    a = np.repeat(a[:1], 3, 0)
    a[1] += np.float32(1e-6) * rng.integers(0, 2, n)
    check_route(sk, gpu(a, F32), k, gpu(b, F32), n_groups=groups, topk_groups=topk_groups, score=score)


@pytest.mark.parametrize("base", [0.01, 1.7, -1.7, 6.0, -6.0, 12.0, 16.0, 20.0, 36.0, -40.0, -90.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 4)])
def test_route_order_of_neighbouring_logits(sk, base, score, groups, topk_groups):
    # scores from 1e-7 apart to equal in 64 bits, by the slope of the score there
    rng = np.random.default_rng(17)
    steps = rng.integers(0, 40, (24, 64)).astype(np.int32)
    a = (np.float32(base).view(np.int32) + steps).astype(np.int32).view(np.float32)
    a[:, 0] = 1.0                                # a largest one for softmax, elsewhere
    for bias in (np.zeros(64), np.full(64, -0.25), np.where(np.arange(64) % 2, 0.125, -3.0)):
        check_route(sk, gpu(a, F32), 8, gpu(bias, F32), n_groups=groups, topk_groups=topk_groups, score=score)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
def test_route_weights_of_tiny_scores(sk, with_bias, groups, topk_groups):
    # renormalized weights are ratios, however small the scores are: below FP32's
    # smallest values they still add up to one
    rng = np.random.default_rng(19)
    a = rng.normal(size=(12, 32)).astype(np.float32)
    a -= np.array([0, 30, 59, 61, 85, 88, 90, 100, 104, 200, 500, 650], np.float32)[:, None]
    bias = gpu(rng.normal(0, 0.05, 32), F32) if with_bias else None
    # ratios of exp(x - the largest chosen): exponents of at most 8
    kw = dict(n_groups=groups, topk_groups=topk_groups, score="sigmoid")
    ids, w = sk.route(gpu(a, F32), 4, bias=bias, **kw)
    rids, rw = ox.route(a, 4, bias=None if bias is None else host(bias), **kw)
    assert np.array_equal(host(ids), rids)
    assert np.all(np.abs(host(w) - rw) <= rw * (2 * np.minimum(np.abs(a).max(1, keepdims=True), 60 + 8) + 96) * ox.U)
    # softmax with its likeliest experts masked by the bias
    a = rng.normal(size=(8, 32)).astype(np.float32)
    a[:, 5], a[:, 20] = np.array([0, 10, 60, 90, 120, 300, 650, 1e30]), 90.0
    b = np.zeros(32)
    b[[5, 20]] = -np.inf
    kw["score"] = "softmax"
    ids, w = sk.route(gpu(a, F32), 4, bias=gpu(b, F32), **kw)
    rids, rw = ox.route(a, 4, bias=b.astype(np.float32), **kw)
    # where scores are nothing in 64 bits either, the order is the index's, the weights 0
    assert np.array_equal(host(ids), rids)
    assert np.all(np.abs(host(w) - rw) <= rw * (2 * 8 + 96) * ox.U)
    assert not host(w)[-1].any() and np.all(np.abs(host(w)[:-1].sum(1) - 1) < 1e-6)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_at_the_last_choice(sk, score):
    # the last choice ties with the next ones, and the one after those is above
    # them by less than FP32 can tell
    n, k = 64, 4
    a = np.linspace(-3, -1, n).astype(np.float32)[None].repeat(6, 0)
    a[:, 40:44] = 1.5
    a[:, 50] = np.nextafter(np.float32(1.5), np.float32(2))   # the largest, by its index not
    a[1, 3:7] = 1.5
    a[2, 10] = np.nextafter(np.float32(1.5), np.float32(1))
    a[3] = 1.5
    a[3, 63] = np.nextafter(np.float32(1.5), np.float32(2))
    a[4, :] = np.nextafter(np.float32(1.5), np.float32(1))
    a[4, 20:60:2] = 1.5
    a[5, ::3] = 1.5
    for bias in (np.zeros(n), np.full(n, 100.0), np.full(n, -1e-3)):
        check_route(sk, gpu(a, F32), k, gpu(bias, F32), score=score)
        check_route(sk, gpu(a, F32), k, gpu(bias, F32), score=score, n_groups=4, topk_groups=2)


def test_route_many_rows(sk):
    g = torch.Generator(device=DEV).manual_seed(3)
    logits = torch.randn(5000, 64, generator=g, device=DEV)
    bias = torch.randn(64, generator=g, device=DEV) * 0.1
    check_route(sk, logits, 6, bias, n_groups=8, topk_groups=4, score="sigmoid", scale=2.0)


LOW, HIGH = (float(v) for v in (np.finfo(np.float32).min, np.finfo(np.float32).max))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_of_the_largest_biases(sk, score):
    # sums of two biases beyond FP32: the type's lowest value is a mask that still
    # leaves its experts to be chosen where nothing else is left
    bias = np.array([0, 0] + 6 * [LOW])
    ids, _ = check_route(sk, gpu(np.zeros((1, 8)), F32), 4, gpu(bias, F32), n_groups=4, topk_groups=2, score=score)
    assert host(ids).tolist() == [[0, 1, 2, 3]]
    rng = np.random.default_rng(29)
    for _ in range(60):
        a = rng.normal(size=(12, 32))
        values = [0.0, 0.25, LOW, LOW / 2, HIGH, HIGH / 2, -np.inf, np.inf, np.nan]
        bias = rng.choice(values, 32, p=[0.2, 0.1, 0.3, 0.1, 0.08, 0.08, 0.06, 0.04, 0.04])
        for topk_groups, k in ((1, 3), (3, 12), (7, 16)):
            check_route(sk, gpu(a, F32), k, gpu(bias, F32), n_groups=8, topk_groups=topk_groups, score=score)


def test_route_groups_of_cancelling_biases(sk):
    # a group whose two best biases nearly cancel is known far worse than its sum's
    # size says, wherever it ranks
    h = float.fromhex
    bias = np.array([h("0x1.ffe006p+9"), h("-0x1.ffep+9"), -3000, -3000, 0, h("0x1.98f1d4p-13"), -3000, -3000,
                     0, h("0x1.83f91ep-13"), -3000, -3000, -1, -1, -1, -1])
    kw = dict(n_groups=4, topk_groups=2, score="sigmoid")
    ids, _ = check_route(sk, gpu(np.zeros((1, 16)), F32), 2, gpu(bias, F32), **kw)
    assert host(ids).tolist() == [[5, 9]]


@pytest.mark.parametrize("score,spread", [("softmax", 1e-6), ("sigmoid", 1e-7)])
@pytest.mark.parametrize("pin", [30.0, 1e3, 1e5])
def test_route_groups_pinned_and_dropped(sk, score, spread, pin):
    # two groups have one expert pinned, one dropped as far and two further; the groups
    # are as far apart as an FP32 step of the pin
    rng = np.random.default_rng(31)
    a = rng.normal(0, spread * pin, (3000, 32))
    bias = np.zeros((8, 4))
    bias[:, 2:] = -3 * pin
    bias[[1, 4], :2] = pin, -pin
    for topk_groups in (2, 5):
        check_route(sk, gpu(a, F32), 4, gpu(bias.reshape(-1), F32), n_groups=8, topk_groups=topk_groups, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups,k", [(1, 1, 6), (1, 1, 16), (8, 2, 8), (8, 2, 5)])
def test_route_doubtful_rows_that_run_out_of_experts(sk, score, groups, topk_groups, k):
    # scores that FP32 cannot tell apart, and no more experts than choices, or fewer
    rng = np.random.default_rng(41)
    steps = rng.integers(0, 4, (200, 32)).astype(np.int32)
    a = (np.float32(1.7).view(np.int32) + steps).astype(np.int32).view(np.float32)
    bias = np.full(32, 0.125)
    if groups == 1:
        bias[6:] = -np.inf
    check_route(sk, gpu(a, F32), k, gpu(bias, F32), n_groups=groups, topk_groups=topk_groups, score=score)
    a[::2, 3::2] = -np.inf
    check_route(sk, gpu(a, F32), k, gpu(bias, F32), n_groups=groups, topk_groups=topk_groups, score=score)


@pytest.mark.parametrize("score,base", [("sigmoid", 8.0), ("softmax", 0.01)])
@pytest.mark.parametrize("topk_groups", [2, 4, 7])
def test_route_groups_that_pairs_cannot_tell_apart(sk, score, base, topk_groups):
    # groups some 1e-10 apart, which pairs of FP32 tell, and among them one whose
    # biases cancel, which these know to some 1e-9 only
    rng = np.random.default_rng(37)
    a = np.repeat(rng.normal(size=(2000, 1)), 16, 1).astype(np.float32)
    steps = rng.integers(0, 40, (2000, 8)).astype(np.int32)
    a[:, ::2] = (np.float32(base).view(np.int32) + steps).astype(np.int32).view(np.float32)
    bias = np.zeros(16)
    bias[6:8] = 2.0 ** 22, -2.0 ** 22
    check_route(sk, gpu(a, F32), 2 * topk_groups - 1, gpu(bias, F32), n_groups=8, topk_groups=topk_groups, score=score)


@pytest.mark.parametrize("with_bias", [False, True])
def test_route_weights_of_sigmoids_far_apart(sk, with_bias):
    # ratios of scores of which some are beyond FP32 and others are not
    a = np.array([[-30, -95, -100, -88], [-50, -100, -110, -120], [-59, -61, -87.5, -88.5], [-60, -60.001, -140, -90],
                  [3, -70, -80, -60], [100, -61, 0, -59], [-0.5, -87, -61, -100], [-61, -62, -150, -95]])
    bias = gpu(np.array([0.5, 0.25, 0.125, 0]), F32) if with_bias else None
    for k in (2, 4):
        check_route(sk, gpu(a, F32), k, bias, score="sigmoid")


@pytest.mark.parametrize("doubt", [False, True])
def test_route_weights_of_scores_that_are_nothing_in_64_bits(sk, doubt):
    # sigmoids below -709.78 and softmaxes 746 below the largest logit are 0 in FP64:
    # they weigh nothing, whether the row's order took FP64 or not
    bias = np.zeros(8) if doubt else np.arange(8, 0, -1) / 8
    a = np.array([[-705, -712, -720, -800, -720, -712, -706, -900], [-710, -715, -720, -730, -740, -744, -746, -800],
                  [-3, -650, -705, -711, -800, -900, -1000, -709]])
    check_route(sk, gpu(a, F32), 6, gpu(bias, F32), score="sigmoid")
    bias[0] = -np.inf
    a = np.array([[0, -735, -747, -748, -760, -800, -900, -1000]])
    check_route(sk, gpu(a, F32), 6, gpu(bias, F32), score="softmax")


# ----------------------------------------------------------- quantization ----
def check_quantize(sk, z):
    q, scale = sk.int8_quantize(z)
    torch.cuda.synchronize()
    rq, rs = ox.int8_quantize(host(z))
    assert np.array_equal(host(q), rq)
    s = host(scale)
    assert np.array_equal(np.isnan(s), np.isnan(rs))
    fine = ~np.isnan(rs)
    # one FP32 rounding: half a step, also of the smallest values
    assert np.all(np.abs(s - rs)[fine] <= np.abs(rs)[fine] * ox.U + 2.0 ** -150)
    return q, scale


@pytest.mark.parametrize("m,n", [(1, 16), (1, 4096), (16, 4096), (3, 48), (16, 8192), (7, 1040),
                                 (300, 528), (2, 33024), (1, 131056)])
def test_quantize(sk, m, n):
    g = torch.Generator(device=DEV).manual_seed(m + n)
    check_quantize(sk, torch.randn(m, n, generator=g, device=DEV).to(BF16))


def test_quantize_special_rows(sk):
    g = torch.Generator(device=DEV).manual_seed(5)
    z = torch.randn(14, 272, generator=g, device=DEV).to(BF16)
    big = torch.finfo(BF16).max
    z[0] = 0
    z[1, 100] = float("inf")
    z[2, 271] = float("nan")
    z[3] *= 1e38                                    # 127 z beyond FP32
    z[4, 7] = big
    z[5] = z[5].sign() * 2.0 ** -133                # subnormals
    z[6] *= 2.0 ** -130
    z[7] = (torch.arange(272, device=DEV) - 135).to(BF16) / 2  # codes at exact halves
    z[7, 0] = 127
    z[8] = -big
    z[9] = -0.0
    z[10, :] = 0
    z[10, 3] = -1e-30
    z[11, 0], z[11, 1] = float("-inf"), float("nan")
    z[12] *= 1.0 / 256
    z[13, :] = 1
    q, scale = check_quantize(sk, z)
    assert not host(q)[[0, 1, 2, 9, 11]].any()


@pytest.mark.parametrize("exponent", [-120, -8, 0, 110])
def test_quantize_every_quotient(sk, exponent):
    # every significand of the row's largest value against every one of a value, with
    # codes from 127 to below 1: the nearest to half an integer, but not one, is
    # 127 (255 / 256) / 253 = 1/2 + 1/64768
    amax = np.arange(128, 256.0)[:, None]
    z = (np.arange(128, 256.0)[:, None] * 2.0 ** -np.arange(9)).reshape(1, -1)
    z = np.where(z <= amax, z, 0.0) * (-1) ** np.arange(z.size)
    z = np.concatenate([amax, z, np.zeros((128, 15))], 1) * 2.0 ** exponent
    t = gpu(z, torch.float64).to(BF16)
    assert np.array_equal(host(t), z) and z.shape[1] == 1168
    check_quantize(sk, t)


# ------------------------------------------------------------------- gemm ----
def codes(rng, *shape):
    return rng.integers(-128, 128, shape).astype(np.int8)


def check_gemm(sk, xq, xs, wq, ws, splits=0):
    y = torch.full((len(xq), len(wq)), 77.0, dtype=BF16, device=DEV)
    sk.gemm_int8(gpu(xq, I8), gpu(xs, F32), gpu(wq, I8), gpu(ws, F32), out=y, splits=splits)
    torch.cuda.synchronize()
    ref = ox.gemm_int8(xq, xs.astype(np.float32), wq, ws.astype(np.float32))
    got = host(y)
    assert np.all(np.abs(got - ref) <= ox.gemm_int8_bound(ref))
    assert not (y.view(torch.int16) == -32768).any()  # no -0.0
    return y


@pytest.mark.parametrize("m", [1, 2, 5, 8, 9, 16])
@pytest.mark.parametrize("n,k", [(1, 16), (16, 64), (33, 80), (100, 512), (64, 1040), (1024, 4096),
                                 (515, 2064), (40, 16384)])
def test_gemm(sk, m, n, k):
    rng = np.random.default_rng(m * n + k)
    check_gemm(sk, codes(rng, m, k), rng.uniform(0.01, 0.02, m), codes(rng, n, k),
               rng.uniform(0.001, 0.002, n))


@pytest.mark.parametrize("m,n,k", [(16, 96, 8192), (3, 40, 4112), (1, 31, 16)])
def test_gemm_splits_agree(sk, m, n, k):
    rng = np.random.default_rng(k)
    args = (codes(rng, m, k), rng.uniform(0.01, 0.02, m), codes(rng, n, k), rng.uniform(0.001, 0.002, n))
    ys = [check_gemm(sk, *args, splits=s) for s in (0, 1, 2, 4, 8)]
    assert all(torch.equal(y.view(torch.int16), ys[0].view(torch.int16)) for y in ys)


@pytest.mark.parametrize("k", [1024, 1040, 8192, 131056])
@pytest.mark.parametrize("splits", [1, 8])
def test_gemm_sums_are_exact(sk, k, splits):
    # extremes of the codes, and sums of large terms that cancel to a small one
    rng = np.random.default_rng(k)
    xq = np.full((9, k), -128, np.int8)
    xq[1], xq[2] = 127, rng.choice([-128, 127], k)
    xq[3, ::2], xq[4] = 127, codes(rng, k)
    wq = np.full((35, k), -128, np.int8)
    wq[1], wq[2] = 127, rng.choice([-128, 127], k)
    wq[3, ::2] = 127
    wq[4, : k // 2] = 127
    wq[5:] = codes(rng, 30, k)
    one = np.ones(35, np.float32)
    check_gemm(sk, xq, one[:9], wq, one, splits)
    # differences of almost equal sums, exact through a tiny scale: codes that
    # differ in one place
    wq[7] = wq[6]
    wq[7, k - 1] ^= 1
    y = check_gemm(sk, xq, one[:9], wq, one, splits)
    assert y.shape == (9, 35)


def cancelling(rng, rows, half):
    """Weight codes [rows, 2 half] whose halves are alike: extremes or random."""
    first = np.stack([(np.full(half, 127), np.full(half, -128), rng.integers(-128, 128, half))[r % 3] for r in range(rows)])
    return np.concatenate([first, first], 1).astype(np.int8)


@pytest.mark.parametrize("m", [1, 2, 8, 16])
@pytest.mark.parametrize("k", [1024, 8208, 16384, 33024, 131056])
@pytest.mark.parametrize("splits", [1, 8])
def test_gemm_sums_that_cancel_are_exact(sk, m, k, splits):
    # the first half of K adds up to as much as sums can hold, the second takes it off
    # again; a token code and a weight code one step off leave an integer of at most
    # 128 + 128, which BF16 holds
    rng = np.random.default_rng(k + m)
    half, n = k // 2, 42
    xq = np.full((m, k), 127, np.int8)
    xq[1::2] = -127
    xq[:, half:] *= -1
    wq = cancelling(rng, n, half)
    for x in xq[2:]:
        c = rng.integers(k)
        x[c] -= np.sign(x[c])
    for w in wq[1::2]:
        c = rng.integers(k)
        w[c] += 1 if w[c] < 0 else -1
    ref = xq.astype(np.int64) @ wq.astype(np.int64).T
    assert np.abs(ref).max() <= 256 and ref.any()
    y = sk.gemm_int8(gpu(xq, I8), gpu(np.ones(m), F32), gpu(wq, I8), gpu(np.ones(n), F32), splits=splits)
    assert np.array_equal(host(y), ref)


def test_gemm_scales(sk):
    rng = np.random.default_rng(2)
    xq, wq = codes(rng, 6, 128), codes(rng, 48, 128)
    xs = np.array([0.0, -1.0, 1e-30, 1e20, np.nan, np.inf], np.float32)
    ws = rng.uniform(0.5, 2, 48).astype(np.float32)
    ws[3], ws[4] = 0.0, 1e25
    y = sk.gemm_int8(gpu(xq, I8), gpu(xs, F32), gpu(wq, I8), gpu(ws, F32))
    got = host(y)
    with np.errstate(all="ignore"):
        ref = ox.gemm_int8(xq, xs, wq, ws)
        f32 = (xq.astype(np.int64) @ wq.astype(np.int64).T).astype(np.float32) * xs[:, None] * ws
        ref = np.where(np.isfinite(f32), ref, f32)
        over = np.abs(ref) > float(torch.finfo(BF16).max) * (1 + 2.0 ** -9)
        ref = np.where(over, np.sign(ref) * np.inf, ref)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    assert np.all(np.abs(got[fine] - ref[fine]) <= ox.gemm_int8_bound(ref[fine]))
    assert not (y.view(torch.int16) == -32768).any()


def test_gemm_reads_a_weight_quantized_just_before(sk):
    # the weight's codes come from the call ahead on the stream; the previous
    # contents of the buffer would give other results
    g = torch.Generator(device=DEV).manual_seed(1)
    xq, xs = sk.int8_quantize(torch.randn(4, 2048, generator=g, device=DEV).to(BF16))
    ws_ = [torch.randn(4096, 2048, generator=g, device=DEV).to(BF16) for _ in range(2)]
    want = []
    for w in ws_:
        q, s = sk.int8_quantize(w)
        torch.cuda.synchronize()
        want.append(sk.gemm_int8(xq, xs, q, s))
    torch.cuda.synchronize()
    q = torch.zeros(4096, 2048, dtype=I8, device=DEV)
    s = torch.zeros(4096, dtype=F32, device=DEV)
    got = []
    for r in range(40):
        sk.int8_quantize(ws_[r % 2], q=q, scale=s)
        got.append(sk.gemm_int8(xq, xs, q, s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[r % 2]) for r, y in enumerate(got))


# ---------------------------------------------------------------- experts ----
def make_experts(rng, m, experts, k, hidden, inter):
    return dict(xq=codes(rng, m, hidden), xs=rng.uniform(0.01, 0.03, m).astype(np.float32),
                w13=codes(rng, experts, 2 * inter, hidden),
                s13=rng.uniform(2e-4, 6e-4, (experts, 2 * inter)).astype(np.float32) * np.float32((512 / hidden) ** 0.5),
                w2=codes(rng, experts, hidden, inter),
                s2=rng.uniform(2e-4, 6e-4, (experts, hidden)).astype(np.float32),
                ids=np.stack([rng.permutation(experts)[:k] for _ in range(m)]).astype(np.int32),
                g=rng.uniform(0.1, 1.0, (m, k)).astype(np.float32))


def run_experts(sk, c, **kw):
    return sk.experts_int8(gpu(c["xq"], I8), gpu(c["xs"], F32), gpu(c["w13"], I8), gpu(c["s13"], F32),
                           gpu(c["w2"], I8), gpu(c["s2"], F32), gpu(c["ids"], I32), gpu(c["g"], F32), **kw)


def check_experts(sk, c):
    m, k = c["ids"].shape
    hidden, inter = c["w2"].shape[1:]
    ws = torch.full((sk.experts_int8_workspace(m, k, hidden, inter),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((m, hidden), 77.0, dtype=BF16, device=DEV)
    y, _ = run_experts(sk, c, out=out, workspace=ws)
    torch.cuda.synchronize()
    ref, bound = ox.experts_int8(*(c[n] for n in ("xq", "xs", "w13", "s13", "w2", "s2", "ids", "g")))
    got = host(y)
    assert np.all(np.abs(got - ref) <= bound), float((np.abs(got - ref) / bound).max())
    assert not (y.view(torch.int16) == -32768).any()
    return y


@pytest.mark.parametrize("m,experts,k,hidden,inter", [
    (1, 1, 1, 16, 16), (1, 8, 2, 64, 32), (2, 16, 4, 528, 272), (16, 8, 2, 256, 128),
    (16, 4, 4, 1040, 80), (7, 60, 4, 1040, 528), (5, 40, 16, 128, 48), (16, 32, 8, 512, 1040),
    (3, 1024, 8, 32, 16), (9, 3, 1, 2064, 560), (16, 24, 16, 64, 48), (16, 1024, 16, 32, 16),
    (2, 2, 1, 131056, 16), (1, 2, 2, 16, 131056),
])
def test_experts(sk, m, experts, k, hidden, inter):
    k = min(k, experts)
    check_experts(sk, make_experts(np.random.default_rng(m * experts + hidden), m, experts, k, hidden, inter))


def test_experts_masked_repeated_and_shared(sk):
    rng = np.random.default_rng(21)
    c = make_experts(rng, 16, 12, 4, 144, 112)
    c["ids"][0] = -1                                # a padded token: zeros
    c["ids"][1] = [3, -1, 12, 5]                    # masked, and one past the last expert
    c["ids"][2] = [4, 4, 4, 4]                      # one expert four times
    c["ids"][3] = [2, 7, 2, 7]
    c["ids"][4] = [2 ** 31 - 1, -2 ** 31, 0, 11]
    c["ids"][5:, 0] = 9                             # most tokens share an expert
    c["ids"][5:, 1:] = [1, 2, 3]
    c["g"][6] = 0.0
    c["g"][7] *= -1
    y = check_experts(sk, c)
    assert not host(y)[0].any()
    c["ids"][:] = -1
    assert not host(check_experts(sk, c)).any()
    c["ids"][:] = 6                                 # everybody, everywhere
    check_experts(sk, c)
    c["ids"][:] = -1
    c["ids"][15, 3] = 11                            # one choice of one token
    check_experts(sk, c)


def test_experts_leave_masked_weights_unread_and_nan_rows_alone(sk):
    rng = np.random.default_rng(22)
    c = make_experts(rng, 4, 6, 2, 96, 64)
    c["ids"][:] = [[0, 1], [1, 2], [2, 0], [3, -1]]
    c["s13"][4:], c["s2"][4:] = np.nan, np.nan      # experts nobody names
    check_experts(sk, c)
    c["xs"][3] = np.nan                             # one bad token stays its own
    y, _ = run_experts(sk, c)
    got = host(y)
    assert np.isnan(got[3]).all() and np.isfinite(got[:3]).all()
    c["xs"][3] = 0.0                                # a row of zeros: scale 0
    assert not host(run_experts(sk, c)[0])[3].any()


def test_experts_extreme_activations(sk):
    rng = np.random.default_rng(23)
    c = make_experts(rng, 5, 4, 2, 64, 64)
    c["xs"][:] = [1e-30, 10.0, 0.3, 1.0, 3.0]       # gates far into silu's tails
    check_experts(sk, c)


def small_sums(rng, w, places):
    """Makes the sums of `cancelling` rows small integers, by changes at places where the
    other operand is 1."""
    w[:, places] = 100
    w[:, places + w.shape[1] // 2] = 100
    w[:, places] += rng.integers(-5, 6, (len(w), len(places))).astype(np.int8)


@pytest.mark.parametrize("m", [1, 2, 8, 16])
@pytest.mark.parametrize("k", [1040, 16384, 131056])
def test_experts_sums_that_cancel_are_exact(sk, m, k):
    # as above, in gate and up (over hidden) and in down (over inter): sums of a few
    # units, of which one would be far outside the bound
    rng = np.random.default_rng(k + m)
    half = k // 2
    places = rng.choice(half, 3, replace=False)
    sign = np.where(np.arange(m) % 2, -1, 1)
    row = np.full(k, 127)
    row[places] = 1
    row[half:] = -row[:half]
    c = make_experts(rng, m, 2, 2, k, 16)
    c["xq"] = (sign[:, None] * row).astype(np.int8)
    c["xs"][:], c["s13"][:] = 0.25, 1.0
    for w in c["w13"]:
        w[:] = cancelling(rng, 32, half)
        small_sums(rng, w, places)
    check_experts(sk, c)
    c = make_experts(rng, m, 2, 2, 16, k)
    c["xq"][:], c["xq"][:, 0], c["xq"][:, 1] = 0, 127, 127 * sign
    c["xs"][:], c["s13"][:] = 1 / 127, 1 / 127
    c["w13"][:] = 0
    c["w13"][:, :k, 0], c["w13"][:, k:, 1] = 127, row  # gates of 1, ups of the row / 127
    for w in c["w2"]:
        w[:] = cancelling(rng, 16, half)
        small_sums(rng, w, places)
    y = check_experts(sk, c)
    assert host(y).any()


# ------------------------------------------------- calls as a program makes ----
def test_repeats_are_bitwise_equal(sk):
    rng = np.random.default_rng(31)
    c = make_experts(rng, 16, 24, 6, 512, 256)
    t = {k: gpu(v, {np.int8: I8, np.float32: F32, np.int32: I32}[v.dtype.type]) for k, v in c.items()}
    first = None
    for _ in range(50):
        y, _ = sk.experts_int8(*t.values())
        d = sk.gemm_int8(t["xq"], t["xs"], t["w13"][3], t["s13"][3])
        first = first or (y, d)
        assert torch.equal(y, first[0]) and torch.equal(d, first[1])


class Layer:
    """Router, routed experts and a shared int8 product, as a decode step runs them."""

    def __init__(self, sk, m, experts, k, hidden, inter, seed=0):
        self.sk, self.k = sk, k
        self.rng = np.random.default_rng(seed)
        c = make_experts(self.rng, m, experts, k, hidden, inter)
        self.c = c
        self.z = gpu(self.rng.normal(size=(m, hidden)), BF16)
        self.w_r = gpu(self.rng.normal(0, 0.05, (experts, hidden)), BF16)
        self.bias = gpu(self.rng.normal(0, 0.05, experts), F32)
        self.t = {n: gpu(c[n], I8 if c[n].dtype == np.int8 else F32) for n in ("w13", "s13", "w2", "s2")}
        self.w_s = gpu(self.rng.normal(0, 0.02, (hidden, hidden)), BF16)
        self.wq, self.ws = sk.int8_quantize(self.w_s)
        self.ws_buf = torch.empty(sk.experts_int8_workspace(m, k, hidden, inter), dtype=torch.uint8, device=DEV)
        self.out = torch.empty(m, hidden, dtype=BF16, device=DEV)
        self.dense = torch.empty(m, hidden, dtype=BF16, device=DEV)
        self.logits = torch.empty(m, experts, dtype=BF16, device=DEV)

    def step(self, stream=None):
        sk, t = self.sk, self.t
        logits = sk.gemm_bf16(self.z, self.w_r, out=self.logits, stream=stream)
        ids, g = sk.route(logits, self.k, bias=self.bias, score="sigmoid", stream=stream)
        xq, xs = sk.int8_quantize(self.z, stream=stream)
        sk.experts_int8(xq, xs, t["w13"], t["s13"], t["w2"], t["s2"], ids, g, out=self.out,
                        workspace=self.ws_buf, stream=stream)
        sk.gemm_int8(xq, xs, self.wq, self.ws, out=self.dense, stream=stream)
        return logits, ids, g, xq, xs

    def check(self, logits, ids, g, xq, xs):
        torch.cuda.synchronize()
        rids, _ = ox.route(host(logits), self.k, bias=host(self.bias), score="sigmoid")
        assert np.array_equal(host(ids), rids)
        rq, _ = ox.int8_quantize(host(self.z))
        assert np.array_equal(host(xq), rq)
        c = self.c
        ref, bound = ox.experts_int8(host(xq), host(xs), c["w13"], c["s13"], c["w2"], c["s2"], host(ids), host(g))
        assert np.all(np.abs(host(self.out) - ref) <= bound)
        ref = ox.gemm_int8(host(xq), host(xs), host(self.wq), host(self.ws))
        assert np.all(np.abs(host(self.dense) - ref) <= ox.gemm_int8_bound(ref))


@pytest.mark.parametrize("m", [1, 6, 16])
def test_layer_together(sk, m):
    layer = Layer(sk, m, 16, 4, 512, 192, seed=m)
    for _ in range(3):
        layer.check(*layer.step())


def test_layer_captured_and_replayed_with_new_inputs(sk):
    layer = Layer(sk, 16, 16, 4, 512, 192, seed=5)
    layer.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = layer.step()
    for seed in range(3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        layer.z.copy_(torch.randn(layer.z.shape, generator=g, device=DEV))
        layer.out.fill_(77.0)
        graph.replay()
        layer.check(*held)


def test_layers_on_two_streams(sk):
    layers = [Layer(sk, 8, 16, 3, 512, 160, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(10):
        held = [layer.step(stream=s) for layer, s in zip(layers, streams)]
    for layer, h in zip(layers, held):
        layer.check(*h)


def test_offsets_beyond_31_bits(sk):
    # the last expert's weights start past 2^31 codes
    experts, hidden, inter, m = 70, 4096, 4096, 2
    g = torch.Generator(device=DEV).manual_seed(9)
    w13 = torch.zeros(experts, 2 * inter, hidden, dtype=I8, device=DEV)
    w2 = torch.zeros(experts, hidden, inter, dtype=I8, device=DEV)
    last = experts - 1
    w13[last] = torch.randint(-127, 128, w13[last].shape, generator=g, device=DEV, dtype=I8)
    w2[last] = torch.randint(-127, 128, w2[last].shape, generator=g, device=DEV, dtype=I8)
    assert last * 2 * inter * hidden > 2 ** 31 and w13.numel() > 2 ** 31
    s13 = torch.full((experts, 2 * inter), 1e-4, device=DEV)
    s2 = torch.full((experts, hidden), 1e-4, device=DEV)
    xq = torch.randint(-127, 128, (m, hidden), generator=g, device=DEV, dtype=I8)
    xs = torch.full((m,), 0.02, device=DEV)
    ids = torch.tensor([[last], [last]], dtype=I32, device=DEV)
    gw = torch.tensor([[1.0], [0.5]], device=DEV)
    y, _ = sk.experts_int8(xq, xs, w13, s13, w2, s2, ids, gw)
    one = lambda t: host(t[last:])  # noqa: E731
    ref, bound = ox.experts_int8(host(xq), host(xs), one(w13), one(s13), one(w2), one(s2),
                                 np.zeros((m, 1), np.int32), host(gw))
    assert np.all(np.abs(host(y) - ref) <= bound)


def test_large_offsets_of_routing_and_quantization(sk):
    g = torch.Generator(device=DEV).manual_seed(9)
    m, n = 16400, 131056
    z = torch.zeros(m, n, dtype=BF16, device=DEV)
    z[-3:] = torch.randn(3, n, generator=g, device=DEV).to(BF16)
    assert z.numel() > 2 ** 31
    q, scale = sk.int8_quantize(z)
    rq, rs = ox.int8_quantize(host(z[-3:]))
    assert np.array_equal(host(q[-3:]), rq) and not host(scale[:-3]).any()
    del z, q
    m, n = 2 ** 21 + 5, 1024
    a = torch.zeros(m, n, dtype=BF16, device=DEV)
    a[-4:] = torch.randn(4, n, generator=g, device=DEV).to(BF16)
    assert a.numel() > 2 ** 31
    ids, w = sk.route(a, 3)
    rids, rw = ox.route(host(a[-4:]), 3)
    assert np.array_equal(host(ids[-4:]), rids)
    assert torch.equal(ids[:-4], torch.arange(3, dtype=I32, device=DEV).expand(m - 4, 3))


def test_gemm_offsets_beyond_31_bits(sk):
    g = torch.Generator(device=DEV).manual_seed(10)
    m, n, k = 3, 16400, 131056
    wq = torch.zeros(n, k, dtype=I8, device=DEV)
    wq[-40:] = torch.randint(-128, 128, (40, k), generator=g, device=DEV, dtype=I8)
    xq = torch.randint(-128, 128, (m, k), generator=g, device=DEV, dtype=I8)
    assert wq.numel() > 2 ** 31
    xs, ws = torch.full((m,), 0.01, device=DEV), torch.full((n,), 0.01, device=DEV)
    y = host(sk.gemm_int8(xq, xs, wq, ws))
    ref = ox.gemm_int8(host(xq), host(xs), host(wq[-40:]), host(ws[-40:]))
    assert np.all(np.abs(y[:, -40:] - ref) <= ox.gemm_int8_bound(ref)) and not y[:, :-40].any()
