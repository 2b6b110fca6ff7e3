// C entry points of the int8 routed experts: sk_route, sk_int8_quantize,
// sk_gemm_int8 and sk_experts_int8. Arguments are checked here, before any CUDA
// call; the kernels are in sk_experts.cu.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "sk.h"
#include "sk_internal.h"

namespace {

constexpr int kMaxInt8N = 1 << 30;    // row indices of whole tiles stay below 2^31
constexpr int kMaxInt8K = 131056;  // the largest multiple of 16 with k * 2^14 < 2^31

sk_status fail(sk_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return sk::report_error(st, buf);
}

sk_status ok() { return sk::report_error(SK_OK, ""); }

struct PtrArg {
  const char *name;
  const void *p;
};

sk_status check_ptrs(const char *call, unsigned align, std::initializer_list<PtrArg> ps) {
  for (const PtrArg &a : ps) {
    if (!a.p) return fail(SK_ERR_INVALID_ARG, "%s: %s is a null pointer", call, a.name);
    if (reinterpret_cast<uintptr_t>(a.p) & (align - 1))
      return fail(SK_ERR_INVALID_ARG, "%s: %s (%p) is not %u-byte aligned", call, a.name, a.p, align);
  }
  return SK_OK;
}

sk_status launch_status(cudaError_t e, const char *what) {
  if (e != cudaSuccess) return fail(SK_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
  return ok();
}

cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

sk_status check_width(const char *name, int v) {
  if (v < 16 || v % 16 || v > kMaxInt8K)
    return fail(SK_ERR_INVALID_ARG, "%s=%d: needs a multiple of 16 in [16, %d]", name, v, kMaxInt8K);
  return SK_OK;
}

sk_status check_rows(int m) {
  if (m < 1 || m > SK_MAX_M)
    return fail(SK_ERR_INVALID_ARG, "m=%d: needs 1 <= m <= %d token rows", m, SK_MAX_M);
  return SK_OK;
}

sk_status check_gemm(int m, int n, int k, int splits) {
  sk_status st;
  if ((st = check_rows(m)) != SK_OK) return st;
  if (n < 1 || n > kMaxInt8N)
    return fail(SK_ERR_INVALID_ARG, "n=%d: needs 1 <= n <= %d output features", n, kMaxInt8N);
  if ((st = check_width("k", k)) != SK_OK) return st;
  if (splits != 0 && splits != 1 && splits != 2 && splits != 4 && splits != 8)
    return fail(SK_ERR_UNSUPPORTED, "unsupported split count %d (0, 1, 2, 4 or 8)", splits);
  return SK_OK;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

struct ExpertsWorkspace {
  size_t act, hq, hs, o, total;  // byte offsets
};

ExpertsWorkspace experts_workspace(int m, int top_k, int hidden, int inter) {
  const size_t rows = static_cast<size_t>(m) * top_k;
  ExpertsWorkspace w;
  w.act = 0;
  w.hq = w.act + round256(rows * inter * 4);
  w.hs = w.hq + round256(rows * inter);
  w.o = w.hs + round256(rows * 4);
  w.total = w.o + round256(rows * hidden * 4);
  return w;
}

}  // namespace

extern "C" {

sk_status sk_route(const void *logits, int logits_type, const float *bias, int32_t *ids,
                   float *weights, int m, int n_experts, int n_groups, int topk_groups, int top_k,
                   int score, int renormalize, float scale, void *stream) {
  sk_status st;
  if (logits_type != SK_TYPE_BF16 && logits_type != SK_TYPE_FP32)
    return fail(SK_ERR_INVALID_ARG, "logits_type=%d: needs SK_TYPE_BF16 or SK_TYPE_FP32", logits_type);
  if (score != SK_SCORE_SOFTMAX && score != SK_SCORE_SIGMOID)
    return fail(SK_ERR_INVALID_ARG, "score=%d: needs SK_SCORE_SOFTMAX or SK_SCORE_SIGMOID", score);
  if (m < 1) return fail(SK_ERR_INVALID_ARG, "m=%d: needs m >= 1 token rows", m);
  if (n_experts < 1 || n_experts > SK_MAX_EXPERTS)
    return fail(SK_ERR_INVALID_ARG, "n_experts=%d: needs 1 <= n_experts <= %d", n_experts, SK_MAX_EXPERTS);
  if (n_groups < 1 || n_groups > SK_MAX_GROUPS || n_experts % n_groups)
    return fail(SK_ERR_INVALID_ARG, "n_groups=%d: needs a divisor of n_experts=%d in [1, %d]", n_groups,
                n_experts, SK_MAX_GROUPS);
  if (topk_groups < 1 || topk_groups > n_groups)
    return fail(SK_ERR_INVALID_ARG, "topk_groups=%d: needs 1 <= topk_groups <= n_groups=%d", topk_groups,
                n_groups);
  if (top_k < 1 || top_k > SK_MAX_TOP_K || top_k > n_experts / n_groups * topk_groups)
    return fail(SK_ERR_INVALID_ARG,
                "top_k=%d: needs 1 <= top_k <= %d and at most the %d experts of %d groups", top_k,
                SK_MAX_TOP_K, n_experts / n_groups * topk_groups, topk_groups);
  if (!std::isfinite(scale)) return fail(SK_ERR_INVALID_ARG, "scale=%g: needs a finite factor", scale);
  const bool fp32 = logits_type == SK_TYPE_FP32;
  if ((st = check_ptrs("sk_route", fp32 ? 4 : 2, {{"logits", logits}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_route", 4, {{"ids", ids}, {"weights", weights}})) != SK_OK) return st;
  if (bias && (st = check_ptrs("sk_route", 4, {{"bias", bias}})) != SK_OK) return st;
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  sk::RouteArgs a{logits, bias, ids, weights, m, n_experts, n_groups, topk_groups, top_k, fp32,
                  score == SK_SCORE_SIGMOID, renormalize != 0, scale};
  return launch_status(sk::launch_route(a, as_stream(stream), sk::pdl_on()), "route");
}

sk_status sk_int8_quantize(const void *z, int8_t *q, float *scale, int m, int n, void *stream) {
  sk_status st;
  if (m < 1) return fail(SK_ERR_INVALID_ARG, "m=%d: needs m >= 1 rows", m);
  if ((st = check_width("n", n)) != SK_OK) return st;
  if ((st = check_ptrs("sk_int8_quantize", 16, {{"z", z}, {"q", q}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_int8_quantize", 4, {{"scale", scale}})) != SK_OK) return st;
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  return launch_status(sk::launch_int8_quantize(static_cast<const uint16_t *>(z), q, scale, m, n,
                                                as_stream(stream), sk::pdl_on()),
                       "int8_quantize");
}

sk_status sk_gemm_int8_supported(int m, int n, int k, int splits) {
  sk_status st = check_gemm(m, n, k, splits);
  return st == SK_OK ? ok() : st;
}

sk_status sk_gemm_int8(const int8_t *xq, const float *x_scale, const int8_t *wq,
                       const float *w_scale, void *y, int m, int n, int k, int splits,
                       void *stream) {
  sk_status st;
  if ((st = check_gemm(m, n, k, splits)) != SK_OK) return st;
  if ((st = check_ptrs("sk_gemm_int8", 16, {{"xq", xq}, {"wq", wq}, {"y", y}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_gemm_int8", 4, {{"x_scale", x_scale}, {"w_scale", w_scale}})) != SK_OK)
    return st;
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  sk::Int8GemmArgs a{xq, wq, x_scale, w_scale, static_cast<uint16_t *>(y), m, n, k,
                     splits ? splits : sk::int8_splits(n, k, info.sm_count)};
  return launch_status(sk::launch_gemm_int8(a, as_stream(stream), sk::pdl_on()), "gemm_int8");
}

static sk_status check_experts(int m, int top_k, int hidden, int inter) {
  sk_status st;
  if ((st = check_rows(m)) != SK_OK) return st;
  if (top_k < 1 || top_k > SK_MAX_TOP_K)
    return fail(SK_ERR_INVALID_ARG, "top_k=%d: needs 1 <= top_k <= %d", top_k, SK_MAX_TOP_K);
  if ((st = check_width("hidden", hidden)) != SK_OK) return st;
  return check_width("inter", inter);
}

size_t sk_experts_int8_workspace(int m, int top_k, int hidden, int inter) {
  if (check_experts(m, top_k, hidden, inter) != SK_OK) return 0;
  ok();
  return experts_workspace(m, top_k, hidden, inter).total;
}

sk_status sk_experts_int8(const int8_t *xq, const float *x_scale, const int8_t *w13,
                          const float *s13, const int8_t *w2, const float *s2, const int32_t *ids,
                          const float *weights, void *y, void *workspace, size_t workspace_bytes,
                          int m, int n_experts, int top_k, int hidden, int inter, void *stream) {
  sk_status st;
  if ((st = check_experts(m, top_k, hidden, inter)) != SK_OK) return st;
  if (n_experts < 1 || n_experts > SK_MAX_EXPERTS)
    return fail(SK_ERR_INVALID_ARG, "n_experts=%d: needs 1 <= n_experts <= %d", n_experts, SK_MAX_EXPERTS);
  if ((st = check_ptrs("sk_experts_int8", 16, {{"xq", xq}, {"w13", w13}, {"w2", w2}, {"y", y}})) != SK_OK)
    return st;
  if ((st = check_ptrs("sk_experts_int8", 4,
                       {{"x_scale", x_scale}, {"s13", s13}, {"s2", s2}, {"ids", ids},
                        {"weights", weights}})) != SK_OK)
    return st;
  if ((st = check_ptrs("sk_experts_int8", 256, {{"workspace", workspace}})) != SK_OK) return st;
  const ExpertsWorkspace w = experts_workspace(m, top_k, hidden, inter);
  if (workspace_bytes < w.total)
    return fail(SK_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, w.total);
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  sk::ExpertsArgs a{xq, x_scale, w13, s13, w2, s2, ids, weights, static_cast<uint16_t *>(y),
                    reinterpret_cast<float *>(ws + w.act), reinterpret_cast<int8_t *>(ws + w.hq),
                    reinterpret_cast<float *>(ws + w.hs), reinterpret_cast<float *>(ws + w.o),
                    m, n_experts, top_k, hidden, inter};
  return launch_status(sk::launch_experts_int8(a, info.sm_count, as_stream(stream), sk::pdl_on()),
                       "experts_int8");
}

}  // extern "C"
