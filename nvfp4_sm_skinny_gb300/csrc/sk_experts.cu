// Device code of the int8 routed experts: routing (sk_route), int8 quantization
// of rows (sk_int8_quantize), the int8 GEMM (sk_gemm_int8) and the experts'
// products (sk_experts_int8). include/sk.h has the formulas.
#include <math_constants.h>

#include <type_traits>

#include "sk.h"
#include "sk_internal.h"
#include "sk_ptx.cuh"

namespace sk {
namespace {

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                   bool pdl, int cluster_y, typename std::remove_reference<Args>::type... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  int na = 0;
  if (pdl) {
    attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster_y > 1) {
    attrs[na].id = cudaLaunchAttributeClusterDimension;
    attrs[na].val.clusterDim.x = 1;
    attrs[na].val.clusterDim.y = static_cast<unsigned>(cluster_y);
    attrs[na++].val.clusterDim.z = 1;
  }
  cfg.attrs = attrs;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A load that stays in its place.
__device__ __forceinline__ int load_id(const int32_t *p) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// ------------------------------------------------------------------ routing
// One warp per token row, kVals logits per lane (expert 32 j + lane in value j).
// What a row costs is the chain of selections, each two warp reductions, not
// its bytes; so the values are compared as order-preserving 32-bit integers, for
// which a reduction is one instruction.
//
// Without a bias the order is that of the logits, exactly. With one it is that
// of p + bias, computed in FP32 here, and two values nearer than the rounding
// errors of either decide nothing: such a row (about one in a thousand of random
// ones) is done again in pairs of FP32, and one that these cannot settle either in
// FP64, whose exponential alone takes microseconds on this GPU.
constexpr int kRouteWarps = 4;  // token rows per CTA

__device__ __forceinline__ float route_logit(const RouteArgs &a, size_t at) {
  const float x = a.fp32 ? static_cast<const float *>(a.logits)[at]
                         : bf16_bits_to_f32(static_cast<const uint16_t *>(a.logits)[at]);
  return isnan(x) ? -CUDART_INF_F : x + 0.0f;  // -0 becomes 0
}

// The last step of a row: lane c holds choice c (id -1: none), its logit x and its
// score p. Renormalized weights are ratios of scores, which FP32 would lose where
// some of them are tiny (the likely experts masked by the bias, far negative logits):
// those of a softmax are ratios of exp(x - the largest chosen x), those of sigmoids
// where one is that small, of exp(x - ref) / (1 + exp(x)), ref the largest chosen x
// or 0 if that is positive. `top`: the logit that scores refer to (softmax). A score
// weighs nothing where it is 0 in FP64, where exp(-x) is infinite or exp(x - top) 0.
__device__ __forceinline__ void route_store(const RouteArgs &a, int row, int id, float x, float p, float top) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31;
  const bool mine = lane < a.top_k && id >= 0;
  float w = mine ? p : 0.0f;
  if (a.renormalize) {
    if (!a.sigmoid || __any_sync(kAll, mine && x < -60.0f)) {
      float most = mine ? x : -CUDART_INF_F;
#pragma unroll
      for (int d = SK_MAX_TOP_K / 2; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, d));
      const bool nothing = !mine || (a.sigmoid ? x < -709.78266f : x != top && x - top < -745.13f);
      if (!a.sigmoid) w = nothing ? 0.0f : __expf(x == most ? 0.0f : x - most);
      else if (!(x > 0.0f)) w = nothing ? 0.0f : __expf(x - fminf(most, 0.0f)) / (1.0f + __expf(x));
    }
    float total = w;  // of the first lanes, which hold the choices
#pragma unroll
    for (int d = SK_MAX_TOP_K / 2; d; d >>= 1) total += __shfl_xor_sync(kAll, total, d);
    w = total > 0.0f ? w / total : 0.0f;
  }
  if (lane < a.top_k) {
    a.ids[static_cast<size_t>(row) * a.top_k + lane] = id;
    a.weights[static_cast<size_t>(row) * a.top_k + lane] = w * a.scale;
  }
}

// Largest value of the warp's lanes and, among equals, the lowest index; lanes
// without a candidate give -inf and index INT_MAX.
__device__ __forceinline__ void warp_best(double &v, int &at) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const double ov = __shfl_xor_sync(0xFFFFFFFFu, v, d);
    const int oat = __shfl_xor_sync(0xFFFFFFFFu, at, d);
    if (ov > v || (ov == v && oat < at)) {
      v = ov;
      at = oat;
    }
  }
}

// A row in FP64, its selection values in v[n_experts] (shared memory).
__device__ __noinline__ void route_row_f64(const RouteArgs &a, int row, double *v) {
  const int lane = threadIdx.x & 31;
  const int E = a.n_experts;
  const size_t base = static_cast<size_t>(row) * E;

  double top = -CUDART_INF;
  for (int e = lane; e < E; e += 32) {
    const double x = static_cast<double>(route_logit(a, base + e));
    v[e] = x;
    top = fmax(top, x);
  }
  for (int d = 16; d; d >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  double sum = 0.0;
  if (!a.sigmoid) {
    for (int e = lane; e < E; e += 32)
      if (v[e] != -CUDART_INF) sum += exp(v[e] == top ? 0.0 : v[e] - top);
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  }
  auto score = [&](double x) {
    if (x == -CUDART_INF) return 0.0;
    return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x == top ? 0.0 : x - top) / sum;
  };
  if (a.bias) {
    for (int e = lane; e < E; e += 32) {
      double s = v[e] == -CUDART_INF ? v[e] : score(v[e]) + static_cast<double>(a.bias[e]);
      if (isnan(s)) s = -CUDART_INF;
      v[e] = s;
    }
  }
  __syncwarp();

  const int per = E / a.n_groups;
  uint32_t keep = a.n_groups > 1 ? 0u : 1u;
  if (a.n_groups > 1) {
    double gv = -CUDART_INF;
    if (lane < a.n_groups) {
      double b0 = -CUDART_INF, b1 = -CUDART_INF;
      for (int j = 0; j < per; ++j) {
        const double x = v[lane * per + j];
        b1 = fmax(b1, fmin(b0, x));
        b0 = fmax(b0, x);
      }
      gv = a.bias && b1 != -CUDART_INF ? b0 + b1 : b0;
    }
    for (int j = 0; j < a.topk_groups; ++j) {
      double b = gv;
      int at = gv == -CUDART_INF ? INT_MAX : lane;
      warp_best(b, at);
      if (at == INT_MAX) break;
      keep |= 1u << at;
      if (lane == at) gv = -CUDART_INF;
    }
  }

  int id = -1;  // lane j holds choice j
  double w = 0.0;
  for (int j = 0; j < a.top_k; ++j) {
    double b = -CUDART_INF;
    int at = INT_MAX;
    for (int e = lane; e < E; e += 32)
      if ((keep >> (a.n_groups > 1 ? e / per : 0)) & 1u)
        if (v[e] > b) {
          b = v[e];
          at = e;
        }
    warp_best(b, at);
    if (at == INT_MAX) break;
    if (lane == 0) v[at] = -CUDART_INF;
    __syncwarp();
    if (lane == j) {
      id = at;
      w = score(static_cast<double>(route_logit(a, base + at)));
    }
  }
  double total = w;
  for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
  if (a.renormalize) w = total > 0.0 ? w / total : 0.0;
  if (lane < a.top_k) {
    a.ids[static_cast<size_t>(row) * a.top_k + lane] = id;
    a.weights[static_cast<size_t>(row) * a.top_k + lane] = static_cast<float>(w * a.scale);
  }
}


// A value as the sum of two FP32, hi the nearest to it: about 45 significant bits,
// by the error-free sums and products of Dekker and Knuth.
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ Pair quick_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair exact_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = exact_sum(a.hi, b.hi), t = exact_sum(a.lo, b.lo);
  const Pair r = quick_sum(s.hi, __fadd_rn(s.lo, t.hi));
  return quick_sum(r.hi, __fadd_rn(r.lo, t.lo));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float p = __fmul_rn(a.hi, b.hi);
  const float e = __fmaf_rn(a.hi, b.hi, -p);
  return quick_sum(p, __fadd_rn(e, __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}
__device__ __forceinline__ Pair operator/(Pair a, Pair b) {
  const float q = __fdiv_rn(a.hi, b.hi);
  const float r = __fadd_rn(__fmaf_rn(-q, b.hi, a.hi), __fmaf_rn(-q, b.lo, a.lo));
  return quick_sum(q, __fdiv_rn(r, b.hi));
}
__device__ __forceinline__ bool above(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

// exp(x) for -80 <= x <= 80: x = k ln 2 + r, and exp(r) - 1 from that of r / 8 by
// its series and three squarings, 1 + y -> (1 + y)^2.
__device__ __forceinline__ Pair pair_exp(Pair x) {
  constexpr float kLn2Hi = 0x1.62ep-1f;                  // 12 bits, so that k times it is exact
  constexpr float kLn2Mid = 0x1.0bfbe8p-15f;             // the next 24
  constexpr float kLn2Lo = 0x1.cf79acp-40f;              // and the rest
  const float k = rintf(__fmul_rn(x.hi, 1.44269504f));
  const float a = __fmaf_rn(-k, kLn2Hi, x.hi);           // exact
  const float m = __fmul_rn(-k, kLn2Mid), e = __fmaf_rn(-k, kLn2Mid, -m);
  const Pair s = exact_sum(a, m);
  const Pair r = quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(__fmaf_rn(-k, kLn2Lo, e), x.lo)));
  const Pair z = {r.hi * 0.125f, r.lo * 0.125f};
  // z^4 / 24 + ... + z^8 / 40320, below 2e-7 with |z| <= 0.0434
  const float h = z.hi, t = __fmul_rn(__fmul_rn(__fmul_rn(h, h), __fmul_rn(h, h)),
                                      1.0f / 24 + h * (1.0f / 120 + h * (1.0f / 720 + h * (1.0f / 5040 + h * (1.0f / 40320)))));
  const Pair z2 = z * z, z3 = z2 * z;
  Pair y = z + Pair{0.5f * z2.hi, 0.5f * z2.lo} + z3 * Pair{0x1.555556p-3f, -0x1.555556p-28f} + Pair{t, 0.0f};
#pragma unroll
  for (int i = 0; i < 3; ++i) y = Pair{2.0f * y.hi, 2.0f * y.lo} + y * y;
  const Pair v = Pair{1.0f, 0.0f} + y;
  const float scale = __int_as_float((static_cast<int>(k) + 127) << 23);
  return {v.hi * scale, v.lo * scale};
}

// exp(x - top) of a softmax or exp(-x) of a sigmoid; tiny ones to FP32 only,
// within the tolerance of `close`.
__device__ __forceinline__ Pair pair_power(bool sigmoid, float x, float top) {
  const Pair d = sigmoid ? Pair{-x, 0.0f} : x == top ? Pair{0.0f, 0.0f} : exact_sum(x, -top);
  if (!(fabsf(d.hi) <= 80.0f)) return {d.hi > 0.0f ? CUDART_INF_F : __expf(d.hi), 0.0f};
  return pair_exp(d);
}
__device__ __forceinline__ Pair pair_sigmoid(float x) {
  const Pair p = pair_power(true, x, 0.0f);
  if (p.hi == CUDART_INF_F) return {__expf(x), 0.0f};
  return Pair{1.0f, 0.0f} / (Pair{1.0f, 0.0f} + p);
}
__device__ __forceinline__ Pair pair_biased(Pair p, float b) {  // b > -inf
  return b < CUDART_INF_F ? p + Pair{b, 0.0f} : Pair{CUDART_INF_F, 0.0f};
}
// Whether a, not below b, may be b all the same. Scores are within 2^-38 of their
// size (1e-34 for tiny ones), values and sums of two another 2^-44.
__device__ __forceinline__ bool close(Pair a, Pair b, float scores, float sizes) {
  return !(__fadd_rn(a.hi - b.hi, a.lo - b.lo) > scores * 0x1p-37f + sizes * 0x1p-43f + 1e-34f);
}

// route_row_f64 in pairs: false where these cannot tell two values apart. The
// selection values are in hi[n_experts], lo[n_experts] (shared memory).
__device__ __noinline__ bool route_row_pairs(const RouteArgs &a, int row, float *hi, float *lo) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, E = a.n_experts;
  const size_t base = static_cast<size_t>(row) * E;
  float top = -CUDART_INF_F;
  if (!a.sigmoid) {
    for (int e = lane; e < E; e += 32) top = fmaxf(top, route_logit(a, base + e));
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
  }
  Pair sum = {0.0f, 0.0f};
  if (!a.sigmoid) {
    for (int e = lane; e < E; e += 32) {
      const float x = route_logit(a, base + e);
      if (x > -CUDART_INF_F) sum = sum + pair_power(false, x, top);
    }
    for (int d = 16; d; d >>= 1)
      sum = sum + Pair{__shfl_xor_sync(kAll, sum.hi, d), __shfl_xor_sync(kAll, sum.lo, d)};
  }
  auto score = [&](float x) { return a.sigmoid ? pair_sigmoid(x) : pair_power(false, x, top) / sum; };
  const Pair none = {-CUDART_INF_F, 0.0f};
#pragma unroll 2
  for (int e = lane; e < E; e += 32) {
    const float x = route_logit(a, base + e), b = a.bias[e];
    Pair v = none;
    if (x > -CUDART_INF_F && b > -CUDART_INF_F) v = pair_biased(score(x), b);
    hi[e] = v.hi;
    lo[e] = v.lo;
  }
  __syncwarp();
  const int per = E / a.n_groups;
  uint32_t keep = a.n_groups > 1 ? 0u : 1u;
  if (a.n_groups > 1) {
    Pair gv = none;
    float size = 0.0f;
    if (lane < a.n_groups) {
      Pair b0 = none, b1 = none;
      int j = lane % per;  // apart, so that groups do not meet in one bank
#pragma unroll 4
      for (int i = 0; i < per; ++i, j = j + 1 == per ? 0 : j + 1) {
        const Pair x = {hi[lane * per + j], lo[lane * per + j]};
        if (above(x, b0)) {
          b1 = b0;
          b0 = x;
        } else if (above(x, b1)) {
          b1 = x;
        }
      }
      // half of the sum, as the whole may be beyond FP32
      const bool two = b1.hi > -CUDART_INF_F;
      const Pair h0 = {0.5f * b0.hi, 0.5f * b0.lo}, h1 = {0.5f * b1.hi, 0.5f * b1.lo};
      gv = !two ? h0 : fmaxf(b0.hi, b1.hi) < CUDART_INF_F ? h0 + h1 : Pair{CUDART_INF_F, 0.0f};
      size = fabsf(h0.hi) + (two ? fabsf(h1.hi) : 0.0f);
    }
    int rank = 0;
    for (int o = 0; o < a.n_groups; ++o) {
      const Pair v = {__shfl_sync(kAll, gv.hi, o), __shfl_sync(kAll, gv.lo, o)};
      rank += above(v, gv) || (!above(gv, v) && o < lane);
    }
    keep = __ballot_sync(kAll, lane < a.n_groups && rank < a.topk_groups && gv.hi > -CUDART_INF_F);
    // Each kept group against each of the others, with the sizes of both: what a sum
    // has cancelled to does not tell how well it is known.
    const bool in = (keep >> lane) & 1u;
    bool doubt = false;
    for (int o = 0; o < a.n_groups; ++o) {
      const Pair v = {__shfl_sync(kAll, gv.hi, o), __shfl_sync(kAll, gv.lo, o)};
      const float other = __shfl_sync(kAll, size, o);
      if (in && !((keep >> o) & 1u) && v.hi > -CUDART_INF_F)
        doubt = doubt || close(gv, v, 2.0f, size + other);  // halves of four scores
    }
    if (__any_sync(kAll, doubt)) return false;
  }

  if (a.n_groups > 1)
    for (int e = lane; e < E; e += 32)
      if (!((keep >> (e / per)) & 1u)) hi[e] = -CUDART_INF_F, lo[e] = 0.0f;  // as `none`: never above it
  __syncwarp();

  // The choices and those after them, down to one that is clearly apart.
  int id = -1, found = 0;
  Pair mine = none, before = none;
  bool apart = false;
  while (found < 32 && !apart) {
    Pair b = none;
    int at = INT_MAX;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) {
      const Pair x = {hi[e], lo[e]};
      if (above(x, b)) {
        b = x;
        at = e;
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const Pair o = {__shfl_xor_sync(kAll, b.hi, d), __shfl_xor_sync(kAll, b.lo, d)};
      const int oat = __shfl_xor_sync(kAll, at, d);
      if (above(o, b) || (!above(b, o) && oat < at)) {
        b = o;
        at = oat;
      }
    }
    if (at == INT_MAX) break;
    if (lane == 0) hi[at] = -CUDART_INF_F, lo[at] = 0.0f;
    __syncwarp();
    if (lane == found) {
      id = at;
      mine = b;
    }
    apart = found >= a.top_k && !close(before, b, 2.0f, fabsf(before.hi) + fabsf(b.hi));
    before = b;
    ++found;
  }
  if (found == 32 && !apart) return false;
  const int count = apart ? found - 1 : found;  // all of them but the one apart
  const float x = id >= 0 ? route_logit(a, base + id) : 0.0f, b = id >= 0 ? a.bias[id] : 0.0f;
  const Pair v1 = {__shfl_down_sync(kAll, mine.hi, 1), __shfl_down_sync(kAll, mine.lo, 1)};
  const float x1 = __shfl_down_sync(kAll, x, 1), b1 = __shfl_down_sync(kAll, b, 1);
  const Pair p = id >= 0 ? score(x) : Pair{0.0f, 0.0f};
  const float p1 = __shfl_down_sync(kAll, p.hi, 1);
  if (__any_sync(kAll, lane + 1 < count && !(x1 == x && b1 == b) &&
                           close(mine, v1, p.hi + p1, fabsf(mine.hi) + fabsf(v1.hi))))
    return false;
  route_store(a, row, id, x, p.hi, a.sigmoid ? 0.0f : top);
  return true;
}

// FP32 -> integer with the same order; 0 stands for "cannot be chosen" (-inf and
// NaN, and nothing else).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  if (!(v > -CUDART_INF_F)) return 0u;
  return b ^ (static_cast<int>(b) < 0 ? 0xFFFFFFFFu : 0x80000000u);
}

// The two largest of a lane's keys and their experts (key 0: none).
struct Best {
  uint32_t key, next;
  int at, next_at;
  __device__ __forceinline__ Best() : key(0u), next(0u), at(0), next_at(0) {}
  __device__ __forceinline__ void offer(uint32_t k, int e) {  // in ascending order of e
    const bool first = k > key, second = k > next;
    next_at = first ? at : second ? e : next_at;
    next = max(next, min(key, k));
    at = first ? e : at;
    key = max(key, k);
  }
};

template <int kVals>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ double route_smem[];
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned row = blockIdx.x * kRouteWarps + warp;
  if (row >= static_cast<unsigned>(a.m)) return;
  const int E = a.n_experts;
  const size_t base = static_cast<size_t>(row) * E;
  double *scratch = route_smem + warp * max(E, 16);

  float x[kVals];  // NaN where the logit is: no comparison below takes one
  if (a.fp32) {
    const float *p = static_cast<const float *>(a.logits) + base + lane;
#pragma unroll
    for (int j = 0; j < kVals; ++j) x[j] = j * 32 + lane < E ? p[j * 32] : -CUDART_INF_F;
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(a.logits) + base + lane;
#pragma unroll
    for (int j = 0; j < kVals; ++j) x[j] = j * 32 + lane < E ? bf16_bits_to_f32(p[j * 32]) : -CUDART_INF_F;
  }
  float top = -CUDART_INF_F, unit = 1.0f;  // softmax: the largest logit, 1 / sum
  if (!a.sigmoid) {
#pragma unroll
    for (int j = 0; j < kVals; ++j) top = fmaxf(top, x[j]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kVals; ++j)
      if (x[j] > -CUDART_INF_F) sum += __expf(x[j] == top ? 0.0f : x[j] - top);
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    unit = 1.0f / sum;
  }
  auto score = [&](float v) {
    return a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-v)) : __expf(v == top ? 0.0f : v - top) * unit;
  };
  uint32_t key[kVals];
#pragma unroll
  for (int j = 0; j < kVals; ++j) {
    float v = x[j];
    if (a.bias && j * 32 + lane < E) v = v > -CUDART_INF_F ? score(v) + a.bias[j * 32 + lane] : v;
    key[j] = order_key(v);
  }
  auto value = [](uint32_t k) {  // of a key
    return k == 0u ? -CUDART_INF_F : __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
  };

  bool near = false;  // FP32 cannot tell
  if (a.n_groups > 1) {
    // The two best of each group, that of group `lane` in b0, b1.
    const int per = E / a.n_groups;
    uint32_t b0 = 0u, b1 = 0u;
    if (per % 32 == 0) {
      // whole values of all lanes: group g is values j with 32 j in [g per, ...)
      uint32_t l0 = 0u, l1 = 0u;
      int left = per, grp = 0;
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        if (j * 32 >= E) break;
        l1 = max(l1, min(l0, key[j]));
        l0 = max(l0, key[j]);
        left -= 32;
        if (left == 0) {
          const uint32_t m0 = __reduce_max_sync(kAll, l0);
          uint32_t m1 = 0u;
          if (a.bias) {
            const int who = __ffs(__ballot_sync(kAll, l0 == m0)) - 1;
            m1 = __reduce_max_sync(kAll, lane == who ? l1 : l0);
          }
          if (lane == grp) {
            b0 = m0;
            b1 = m1;
          }
          l0 = l1 = 0u;
          left = per;
          ++grp;
        }
      }
    } else {
      // `lanes` lanes per group read them from shared memory, starting apart so
      // that groups do not meet in one bank
      uint32_t *keys = reinterpret_cast<uint32_t *>(scratch);
#pragma unroll
      for (int j = 0; j < kVals; ++j)
        if (j * 32 + lane < E) keys[j * 32 + lane] = key[j];
      __syncwarp();
      int lanes = 1;
      while (2 * lanes * a.n_groups <= 32) lanes *= 2;
      const int grp = lane / lanes, sub = lane % lanes;
      if (grp < a.n_groups) {
        const uint32_t *k = keys + grp * per;
        const int turns = (per + lanes - 1) / lanes;
        for (int i = 0, s = grp % turns; i < turns; ++i) {
          const int at = s * lanes + sub;
          const uint32_t v = at < per ? k[at] : 0u;
          b1 = max(b1, min(b0, v));
          b0 = max(b0, v);
          s = s + 1 == turns ? 0 : s + 1;
        }
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const uint32_t o0 = __shfl_xor_sync(kAll, b0, d), o1 = __shfl_xor_sync(kAll, b1, d);
        b1 = max(max(b1, o1), min(b0, o0));
        b0 = max(b0, o0);
      }
      b0 = __shfl_sync(kAll, b0, lane * lanes);
      b1 = __shfl_sync(kAll, b1, lane * lanes);
    }
    // With a bias half of the sum, as the whole may be beyond FP32 (two biases of its
    // lowest value, as a mask).
    float gv = a.bias ? 0.5f * value(b0) : value(b0), size = fabsf(gv);
    if (a.bias && b1) {
      gv += 0.5f * value(b1);
      size += 0.5f * fabsf(value(b1));
    }
    // (infinities of opposite signs never meet: -inf is no value)
    uint32_t gk = lane < a.n_groups ? order_key(gv) : 0u, kept = 0u;
    for (int o = 0; o < a.topk_groups; ++o) {  // the best groups one by one
      const uint32_t k = __reduce_max_sync(kAll, gk);
      if (!k) break;
      const int who = __ffs(__ballot_sync(kAll, gk == k)) - 1;
      kept |= 1u << who;
      if (lane == who) gk = 0u;
    }
    if (a.bias && a.topk_groups < a.n_groups) {
      // The least that each kept group may be against the most that another may. With
      // u = 2^-24, a group's half sum is within 2 u of its size, whatever it cancels
      // to, and the bound's own rounding takes another. Its scores count apart: halves
      // of four meet, each sigmoid's within 4 u (3 p, and the exponential's error
      // p (1 - p) times), all softmax's together within 75 u.
      const float slack = size < CUDART_INF_F ? 1.8e-7f * size : 0.0f;  // +inf is exact
      const uint32_t most = __reduce_max_sync(kAll, gk ? order_key(gv + slack) : 0u);
      const bool clear = gv - slack - value(most) > (a.sigmoid ? 0.55e-6f : 0.75e-5f);
      near = most && __any_sync(kAll, ((kept >> lane) & 1u) && !clear);
    }
    if (per % 32 == 0) {
      int left = per, g = 0;
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        if (!((kept >> g) & 1u)) key[j] = 0u;
        left -= 32;
        if (left == 0) {
          left = per;
          ++g;
        }
      }
    } else {
      const uint32_t magic = per == 1 ? 0u : 0xFFFFFFFFu / per + 1;
      int at = lane;  // expert of value j
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const uint32_t g = per == 1 ? at : __umulhi(static_cast<uint32_t>(at), magic);  // at / per
        if (at < E && !((kept >> g) & 1u)) key[j] = 0u;
        at += 32;
      }
    }
  }

  // The choices: lane c holds choice c. With a bias also those after them, down to
  // one that is clearly apart (by the largest tolerance that there is).
  int *list = reinterpret_cast<int *>(scratch), found = 0;
  const int want = a.bias ? 32 : a.top_k;
  float before = 0.0f;
  bool apart = false;
  Best best;
#pragma unroll
  for (int j = 0; j < kVals; ++j) best.offer(key[j], j * 32 + lane);
  bool whole = true;  // best.next is this lane's second
  __syncwarp();
  while (found < want && !apart) {
    const uint32_t k = __reduce_max_sync(kAll, best.key);
    if (!k) break;
    bool win = best.key == k;
    const uint32_t who = __ballot_sync(kAll, win);
    if (who & (who - 1)) {
      const uint32_t e = __reduce_min_sync(kAll, win ? static_cast<uint32_t>(best.at) : kAll);
      win = win && best.at == static_cast<int>(e);
    }
    if (win) list[found] = best.at;
    if (win && !whole) {  // look for the two best below this one
      const int e = best.at;
      best = Best();
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const int o = j * 32 + lane;
        best.offer(key[j] < k || (key[j] == k && o > e) ? key[j] : 0u, o);
      }
      whole = true;
    } else {
      best.key = win ? best.next : best.key;
      best.at = win ? best.next_at : best.at;
      whole = whole && !win;
    }
    if (a.bias) {
      const float v = value(k);
      apart = found >= a.top_k &&
              before - v > 7.5e-8f * ((a.sigmoid ? 16.0f : 102.0f) + fabsf(before) + fabsf(v));
      before = v;
    }
    ++found;
  }
  __syncwarp();
  int id = lane < found ? list[lane] : -1;
  float chosen = id >= 0 ? route_logit(a, base + id) : 0.0f;
  float w = id >= 0 ? score(chosen) : 0.0f;
  if (a.bias) {
    const float b = id >= 0 ? a.bias[id] : 0.0f, v = w + b;
    const float v1 = __shfl_down_sync(kAll, v, 1), w1 = __shfl_down_sync(kAll, w, 1);
    const float c1 = __shfl_down_sync(kAll, chosen, 1), b1 = __shfl_down_sync(kAll, b, 1);
    // Rounding errors in units of 2^-24: of p, the exponential's 4 + 2.4 times its
    // argument (in a sigmoid (1 - p) times that, and three more), and 64 of
    // softmax's sum (37 of adding, and its terms' own, whose arguments average at
    // most ln 1024); one of p + bias.
    auto error = [&](float p, float x, float v) {
      const float grow = a.sigmoid ? 3.0f + (1.0f - p) * (4.0f + 2.4f * fabsf(x)) : 70.0f + 2.4f * (top - x);
      return p * grow + fabsf(v);
    };
    const float tol = 7.5e-8f * (error(w, chosen, v) + error(w1, c1, v1));
    const bool same = c1 == chosen && b1 == b;  // equal in any precision
    const int count = apart ? found - 1 : found;  // all of them but the one apart
    near = near || (found == 32 && !apart);
    bool again = near || __any_sync(kAll, lane + 1 < count && !same && !(v - v1 > tol));
    if (again && !near && a.sigmoid) {
      // Nobody else can be among them: their values decide in pairs, a lane each.
      Pair p = {-CUDART_INF_F, 0.0f};
      if (lane < count) p = pair_biased(pair_sigmoid(chosen), b);
      int rank = 0;
      bool doubt = false;
      for (int o = 0; o < count; ++o) {
        const Pair q = {__shfl_sync(kAll, p.hi, o), __shfl_sync(kAll, p.lo, o)};
        const float qc = __shfl_sync(kAll, chosen, o), qb = __shfl_sync(kAll, b, o), qw = __shfl_sync(kAll, w, o);
        const int qid = __shfl_sync(kAll, id, o);
        const bool equal = qc == chosen && qb == b;
        rank += equal ? qid < id : above(q, p);
        doubt = doubt || (!equal && close(above(q, p) ? q : p, above(q, p) ? p : q, w + qw, fabsf(p.hi) + fabsf(q.hi)));
      }
      if (!__any_sync(kAll, doubt && lane < count)) {
        again = false;
        int from = lane;
        for (int o = 0; o < count; ++o)
          if (__shfl_sync(kAll, rank, o) == lane) from = o;
        id = __shfl_sync(kAll, id, from);
        w = __shfl_sync(kAll, w, from);
        chosen = __shfl_sync(kAll, chosen, from);
      }
    }
    if (again) {
      __syncwarp();
      float *parts = reinterpret_cast<float *>(scratch);
      if (!route_row_pairs(a, row, parts, parts + E)) {
        __syncwarp();
        route_row_f64(a, row, scratch);
      }
      return;
    }
  }
  route_store(a, row, id, chosen, w, a.sigmoid ? 0.0f : top);
}

// ------------------------------------------------------------- quantization
// Largest of a row's values, W warps to a row, as FP32 bits of a magnitude; NaN
// when the row holds an Inf or NaN (the bits of |z| order as integers, Inf and NaN
// above every finite value).
template <int W>
__device__ __forceinline__ float row_max(uint32_t bits) {
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if constexpr (W > 1) {
    __shared__ uint32_t part[W];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = bits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) bits = max(bits, part[w]);
  }
  return bits >= 0x7F800000u ? CUDART_NAN_F : __uint_as_float(bits);
}

// A row's codes: round to nearest even of 127 v / amax, as of the exact quotient.
// The product with 127 / amax, within 127 2^-23 = 1.51e-5 of it, settles all that are
// further than 1e-4 from half an integer. The others take an IEEE division, whose
// rounding crosses no half, nor lands on one from a quotient of BF16 inputs: the
// nearest is 127 (255 / 256) / 253, 1/64768 = 1.54e-5 away. For it f (2^-8 for
// amax >= 1, else 1) keeps 127 v finite.
struct RowCodes {
  float amax, inv, f;
  bool plain;  // neither zero nor NaN
  bool quick;  // 127 / amax is finite
  __device__ __forceinline__ explicit RowCodes(float row_max) {
    amax = row_max;
    inv = __fdiv_rn(127.0f, amax);
    f = amax >= 1.0f ? 0x1p-8f : 1.0f;
    plain = amax > 0.0f;
    quick = inv < CUDART_INF_F;
  }
  // The codes of two values in their low bytes. Adding 1.5 2^23 rounds to an
  // integer and leaves it, in two's complement, in the low bits; `far` grows to the
  // largest distance from the quotient.
  __device__ __forceinline__ void two(float2 v, uint32_t &c0, uint32_t &c1, float &far) const {
    const float2 t = __fmul2_rn(v, make_float2(inv, inv));
    const float2 b = __fadd2_rn(t, make_float2(12582912.0f, 12582912.0f));
    const float2 r = __fadd2_rn(b, make_float2(-12582912.0f, -12582912.0f));
    const float2 d = __ffma2_rn(r, make_float2(-1.0f, -1.0f), t);
    far = fmaxf(fmaxf(far, fabsf(d.x)), fabsf(d.y));
    c0 = __float_as_uint(b.x);
    c1 = __float_as_uint(b.y);
  }
  __device__ __forceinline__ uint32_t slow(float v) const {
    return static_cast<uint32_t>(
        __float2int_rn(__fdiv_rn(__fmul_rn(__fmul_rn(v, f), 127.0f), __fmul_rn(amax, f))));
  }
};

// 16 bytes of a row as values: 8 BF16 or 4 FP32.
template <typename T>
struct Chunk {
  static constexpr int kVals = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(word(i));
    else return __uint_as_float(i & 1 ? word(i >> 1) & 0xFFFF0000u : word(i >> 1) << 16);
  }
  // The largest magnitude's bits: of BF16, in either half.
  __device__ __forceinline__ uint32_t max_bits(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) m = max(m, word(i) & 0x7FFFFFFFu);
      else m = __vmaxu2(m, word(i) & 0x7FFF7FFFu);
    }
    return m;
  }
  static __device__ __forceinline__ uint32_t fp32_bits(uint32_t m) {  // of max_bits' result
    if constexpr (sizeof(T) == 4) return m;
    else return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void store(int8_t *q, const RowCodes &code) const {
    uint32_t c[kVals];
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; i += 2) code.two(make_float2(value(i), value(i + 1)), c[i], c[i + 1], far);
    if (!code.quick || far > 0.4999f) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) c[i] = code.plain ? code.slow(value(i)) : 0u;
    }
    uint32_t w[kVals / 4];
#pragma unroll
    for (int i = 0; i < kVals / 4; ++i)
      w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040),
                         0x5410);
    if constexpr (kVals == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(q) = w[0];
  }
};

// CTAs of four warps, W of them (1 or 4) to a row. kKeep > 0: rows of at most
// kKeep 16-byte chunks per thread, kept in registers, so that a row is read once;
// 0: rows of any length, read twice. The row's maximum is all that its codes wait
// for, so what counts is rows in flight: ten CTAs per SM where registers allow
// ([8192, 8192]: 36.4 us, 5.5 TB/s; before the packed arithmetic 38 us, when 256
// threads per row took 42 us and CTAs that stay and load the next row ahead 48 us),
// and one warp to a short row (starting a CTA takes 1.3 ns). A caller's codes (ids
// null) may be the weight of a call that reads it ahead of its dependency wait, so
// dependents start only once they are written; the codes of the experts' activations
// are read after the wait.
constexpr int kQuantThreads = 128;
template <typename T, int kKeep, int W>
__global__ void __launch_bounds__(kQuantThreads, 10)
    quantize_kernel(const T *z, int8_t *q, float *scale, int rows, int n, const int32_t *ids, int n_experts) {
  constexpr int kVals = Chunk<T>::kVals, kThreads = 32 * W;
  if (ids) griddep_launch_dependents();
  const unsigned row = blockIdx.x * (kQuantThreads / kThreads) + threadIdx.x / kThreads;
  const int tid = threadIdx.x % kThreads, chunks = n / kVals;
  // (all the warps of a row, and with W = 4 all of the CTA, agree; the kernel
  // ahead started after the one that wrote the ids was done)
  const bool done = row >= static_cast<unsigned>(rows) || (ids && static_cast<unsigned>(load_id(ids + row)) >= static_cast<unsigned>(n_experts));
  griddep_wait();
  if (!done) {
    const uint4 *from = reinterpret_cast<const uint4 *>(z + static_cast<size_t>(row) * n);
    int8_t *to = q + static_cast<size_t>(row) * n;
    uint32_t bits = 0;
    float amax;
    if constexpr (kKeep > 0) {
      Chunk<T> c[kKeep];
#pragma unroll
      for (int j = 0; j < kKeep; ++j) {
        const int at = tid + j * kThreads;
        c[j].raw = at < chunks ? from[at] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kKeep; ++j) bits = c[j].max_bits(bits);
      amax = row_max<W>(Chunk<T>::fp32_bits(bits));
      const RowCodes code(amax);
#pragma unroll
      for (int j = 0; j < kKeep; ++j) {
        const int at = tid + j * kThreads;
        if (at < chunks) c[j].store(to + at * kVals, code);
      }
    } else {
      for (int at = tid; at < chunks; at += kThreads) bits = Chunk<T>{from[at]}.max_bits(bits);
      amax = row_max<W>(Chunk<T>::fp32_bits(bits));
      const RowCodes code(amax);
      for (int at = tid; at < chunks; at += kThreads) Chunk<T>{from[at]}.store(to + at * kVals, code);
    }
    if (tid == 0) scale[row] = __fdiv_rn(amax, 127.0f);
  }
  if (ids) return;
  __threadfence();
  __syncthreads();
  griddep_launch_dependents();
}

template <typename T>
cudaError_t launch_quantize(const T *z, int8_t *q, float *scale, int rows, int n, const int32_t *ids,
                            int n_experts, cudaStream_t stream, bool pdl) {
  const int chunks = n / Chunk<T>::kVals, lane = (chunks + 31) / 32, thread = (chunks + 127) / 128;
  auto *kernel = lane <= 1 ? quantize_kernel<T, 1, 1> : lane <= 2 ? quantize_kernel<T, 2, 1>
               : lane <= 4 ? quantize_kernel<T, 4, 1> : thread <= 2 ? quantize_kernel<T, 2, 4>
               : thread <= 4 ? quantize_kernel<T, 4, 4> : thread <= 8 ? quantize_kernel<T, 8, 4>
               : quantize_kernel<T, 0, 4>;
  const int per_cta = lane <= 4 ? 4 : 1;
  return launch(kernel, dim3((static_cast<unsigned>(rows) + per_cta - 1) / per_cta), dim3(kQuantThreads), 0, stream, pdl, 1, z, q, scale,
                rows, n, ids, n_experts);
}

// ------------------------------------------------------- the int8 product core
//
// Products at up to 16 tokens stream each weight once; 1 byte of weight meets
// at most 16 tokens, far below what the tensor cores need to be busy, so HBM
// is the bound and the rest has to stay out of its way. A CTA owns 32 weight
// rows; its eight warps take blocks of 64 columns in turn.
//
// Each thread streams for itself: 16-byte asynchronous copies bring the pieces
// that this thread multiplies into a queue of its own in shared memory, kDepth
// blocks ahead, where no other thread reads or writes. So nothing but the
// thread's own copies is ever waited for. (A shared ring filled by TMA was
// slower: its boxes of 128-byte rows passed the copy engine at about four
// cycles a row, 60 GB/s for an SM with two CTAs, and a producer, its barriers
// and the slowest of the warps held back the refill.)
//
// The tensor cores multiply int8 codes at FP16, exactly. A weight code w goes
// in as the FP16 subnormal (w + 128) 2^-24, which costs no arithmetic: masked
// bytes with the sign bit flipped (two three-input logic operations and a shift
// for four codes). A token code x becomes the FP16 integer x: code + 128 in the
// mantissa of 1024, less 1152. What is summed is (w + 128) x; the 128 sum x that
// this adds is known from the token row alone and taken off at the end. Every
// product is an integer below 2^15 (times 2^-24) and FP32 holds every partial
// sum exactly up to 2^24, i.e. over 512 columns of a warp, after which the
// accumulators move to 32-bit integers. The warps' and CTAs' sums are added as
// integers (modulo 2^32), so neither the order nor the split count can change a
// result. (The integer tensor-core product of the same size issues at an eighth
// of the FP16 one's rate on this GPU.)
//
// K order within a block is free as long as both operands agree: thread t of a
// quad holds columns 16 t .. 16 t + 15 (one 16-byte piece of a weight row, one of
// a token row) and feeds four of them to each of four m16n8k16 products.
constexpr int kRows = 32;                        // weight rows of a CTA
constexpr int kBlockCols = 64;                   // columns of a warp's block
constexpr int kWarps = 8;
constexpr int kCoreThreads = 32 * kWarps;
constexpr int kExactBlocks = 8;                  // a warp's blocks between moves to integers
constexpr int kRedPitch = kRows + 4;             // ints per token of the sum buffer: rows, then the token's own sum
constexpr int kRedInts = SK_MAX_M * kRedPitch;
constexpr uint64_t kCoreWaitNs = 2000000000ull;  // 2 s of wall time per wait

__device__ uint32_t g_core_status;  // OR of SK_DEVICE_WAIT_* bits

// Blocks in flight per thread, and pieces of a block: four of the weight, one
// for each eight tokens. About 100 KiB of queue per CTA, two CTAs per SM.
template <int NT>
struct Queue {
  static constexpr int kPieces = 4 + NT;
  static constexpr int kDepth = NT == 1 ? 5 : 4;
  static constexpr int kBytes = kWarps * kDepth * kPieces * 512;
};

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const int8_t *from, bool real) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16_once(uint32_t to, const int8_t *from, bool real, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2, %3;" ::"r"(to),
               "l"(from), "r"(real ? 16 : 0), "l"(policy)
               : "memory");
}
// Starts `bytes` (a multiple of 16) towards L2.
__device__ __forceinline__ void prefetch_l2(const int8_t *from, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(from)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The constants of widen_weight in registers: a three-input logic operation
// takes one immediate only.
struct WidenConst {
  uint32_t mask, flip;
  __device__ __forceinline__ WidenConst() {
    asm volatile("mov.u32 %0, 0x00FF00FF;" : "=r"(mask));
    asm volatile("mov.u32 %0, 0x00800080;" : "=r"(flip));
  }
};

// Four codes of a weight -> two FP16 pairs (bytes 0 and 2, 1 and 3) of
// (code + 128) 2^-24.
__device__ __forceinline__ void widen_weight(const WidenConst &c, uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(lo) : "r"(w), "r"(c.mask), "r"(c.flip));  // (w & mask) ^ flip
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(hi) : "r"(w >> 8), "r"(c.mask), "r"(c.flip));
}

// Four codes of a token -> two FP16 pairs of the codes, in the same order.
__device__ __forceinline__ void widen_token(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4240), b = __byte_perm(u, 0x64646464u, 0x4341);
  __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
  __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
  lo = *reinterpret_cast<uint32_t *>(&x);
  hi = *reinterpret_cast<uint32_t *>(&y);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void red_shared(uint32_t addr, int v) {
  asm volatile("red.shared.add.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A warp's sums of one item: its products with the first 8 NT token rows.
template <int NT>
struct Sums {
  float acc[2][NT][4];
  int xsum[NT];  // this thread's columns of token nt * 8 + lane / 4
  int blocks;    // since the last move to integers

  __device__ __forceinline__ Sums() : blocks(0) {
#pragma unroll
    for (int i = 0; i < 2 * NT * 4; ++i) (&acc[0][0][0])[i] = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xsum[nt] = 0;
  }

  // Adds a block's products; x[nt], w[tile][row half]: this thread's pieces.
  __device__ __forceinline__ void add(const WidenConst &wc, const uint4 (&x)[NT], const uint4 (&w)[2][2]) {
    uint32_t b[NT][8];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t xw[4] = {x[nt].x, x[nt].y, x[nt].z, x[nt].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        widen_token(xw[i], b[nt][2 * i], b[nt][2 * i + 1]);
        xsum[nt] = __dp4a(static_cast<int>(xw[i]), 0x01010101, xsum[nt]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const uint4 &w0 = w[rt][0], &w1 = w[rt][1];
        uint32_t a0, a1, a2, a3;
        widen_weight(wc, i == 0 ? w0.x : i == 1 ? w0.y : i == 2 ? w0.z : w0.w, a0, a2);
        widen_weight(wc, i == 0 ? w1.x : i == 1 ? w1.y : i == 2 ? w1.z : w1.w, a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(acc[rt][nt], a0, a1, a2, a3, b[nt][2 * i], b[nt][2 * i + 1]);
      }
  }

  // Moves the products' sums of the first `tokens` tokens to red[token][row]
  // (a shared address).
  __device__ __forceinline__ void move(uint32_t red, int tokens) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    blocks = 0;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int token = nt * 8 + 2 * t + (i & 1), row = rt * 16 + g + (i >> 1) * 8;
          if (token < tokens)
            red_shared(red + 4u * (token * kRedPitch + row), __float2int_rn(acc[rt][nt][i] * 0x1p24f));
          acc[rt][nt][i] = 0.0f;
        }
  }

  // The same for the last time, and the tokens' own sums to red[token][kRows].
  __device__ __forceinline__ void finish(uint32_t red, int tokens) {
    const int g = (threadIdx.x & 31) >> 2;
    if (blocks) move(red, tokens);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (nt * 8 + g < tokens) red_shared(red + 4u * ((nt * 8 + g) * kRedPitch + kRows), xsum[nt]);
  }
};

// The same for one or two tokens (C), without the tensor cores: four-way integer
// products of the codes as they are, half the instructions of widening them. Every
// lane needs the pieces of all token rows, which the lanes 4 c + t brought.
template <int C>
struct Dots {
  static constexpr int kTokens = C;
  int acc[4][C];

  __device__ __forceinline__ Dots() {
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) (&acc[0][0])[i] = 0;
  }
  __device__ __forceinline__ void add(const uint4 (&x)[C], const uint4 (&w)[2][2]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint4 &v = w[h >> 1][h & 1];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        int s = acc[h][c];
        s = __dp4a(static_cast<int>(v.x), static_cast<int>(x[c].x), s);
        s = __dp4a(static_cast<int>(v.y), static_cast<int>(x[c].y), s);
        s = __dp4a(static_cast<int>(v.z), static_cast<int>(x[c].z), s);
        acc[h][c] = __dp4a(static_cast<int>(v.w), static_cast<int>(x[c].w), s);
      }
    }
  }
  // To red[token][row]; the tokens' own sums stay 0, as nothing is to be taken off.
  __device__ __forceinline__ void finish(uint32_t red) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        int s = acc[h][c];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
        if (t == 0) red_shared(red + 4u * (c * kRedPitch + h * 8 + g), s);
      }
  }
};

// The sum of products of a token with a tile row: the correction of the weights'
// offset by 128 (modulo 2^32).
__device__ __forceinline__ int red_sum(const int *red, int token, int row) {
  const uint32_t s = red[token * kRedPitch + row], x = red[token * kRedPitch + kRows];
  return static_cast<int>(s - 128u * x);
}

// ----------------------------------------------------------------- int8 GEMM
// Grid (tiles of 32 output features, S slices of K), cluster (1, S, 1): every
// CTA is resident from the start, two per SM, so that the stream does not wait
// for scheduling. The S sums of a tile meet in shared memory: rank r receives
// rows [32 r / S, ...) of every other rank (st.async, counted by its exchange
// barrier) and finishes them.
template <int NT>
struct GemmShared {
  uint8_t queue[Queue<NT>::kBytes];
  int red[kRedInts];
  int recv[SK_MAX_M * kRows];  // [S ranks][16 tokens][32 / S rows]
  uint64_t exchange;
  int abort;
};

// C > 0: C tokens, without the tensor cores (m1 [8192, 8192]: 12.5 us with them).
template <int NT, int C>
__global__ void __launch_bounds__(kCoreThreads, 2) gemm_int8_kernel(Int8GemmArgs a) {
  using Q = Queue<NT>;
  extern __shared__ __align__(16) uint8_t raw[];
  GemmShared<NT> &sh = *reinterpret_cast<GemmShared<NT> *>(raw);
  const int S = a.splits, rows = kRows / S, rank = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows;
  griddep_launch_dependents();

  // This warp's blocks: every eighth of the slice [k0, k1).
  const int slices = (a.k + kWarps * kBlockCols - 1) / (kWarps * kBlockCols);
  const int k0 = static_cast<int>(static_cast<long long>(slices) * rank / S) * kWarps * kBlockCols;
  const int k1 = min(a.k, static_cast<int>(static_cast<long long>(slices) * (rank + 1) / S) * kWarps * kBlockCols);
  const int col = k0 + warp * kBlockCols + 16 * t;  // this thread's first column
  const int blocks = max(0, (k1 - k0 - warp * kBlockCols + kWarps * kBlockCols - 1) / (kWarps * kBlockCols));
  const uint32_t queue = smem_u32(sh.queue) + warp * (Q::kDepth * Q::kPieces * 512) + lane * 16;
  const uint64_t policy = l2_policy_evict_first();
  const int8_t *wp[2][2], *xp[NT];
  const int from = col < k1 ? col : 0;  // a thread without columns copies zeros, but names an address all the same
#pragma unroll
  for (int h = 0; h < 4; ++h)  // rows past n repeat the last one; their sums are not stored
    wp[h >> 1][h & 1] = a.wq + static_cast<size_t>(min(n0 + h * 8 + g, a.n - 1)) * a.k + from;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xp[nt] = a.xq + static_cast<size_t>(min(nt * 8 + g, a.m - 1)) * a.k + from;
  auto copy_weights = [&](int i, int slot) {
    const bool real = i < blocks && col + i * kWarps * kBlockCols < k1;
    const int off = real ? i * kWarps * kBlockCols : 0;
#pragma unroll
    for (int h = 0; h < 4; ++h)
      copy16_once(queue + (slot * Q::kPieces + h) * 512, wp[h >> 1][h & 1] + off, real, policy);
  };
  auto copy_tokens = [&](int i, int slot) {
    const bool real = i < blocks && col + i * kWarps * kBlockCols < k1;
    const int off = real ? i * kWarps * kBlockCols : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      copy16(queue + (slot * Q::kPieces + 4 + nt) * 512, xp[nt] + off, real && nt * 8 + g < a.m);
  };
#pragma unroll
  for (int i = 0; i < Q::kDepth; ++i) copy_weights(i, i);  // ahead of the kernel before this one

  // The next four slices beyond the queue start towards L2, a row per lane: they
  // keep HBM busy until the token rows are there (m16 [8192, 8192]: 14.2 us
  // without, 13.6 with four, 14.3 with all of K).
  const int ahead = k0 + Q::kDepth * kWarps * kBlockCols;
  if (warp == 0 && n0 + lane < a.n && ahead < k1)
    prefetch_l2(a.wq + static_cast<size_t>(n0 + lane) * a.k + ahead, min(4 * kWarps * kBlockCols, k1 - ahead));

  for (int i = tid; i < kRedInts; i += kCoreThreads) sh.red[i] = 0;
  if (S > 1 && tid == 0) {
    mbar_init(smem_u32(&sh.exchange), 1);
    mbar_arrive_expect_tx(smem_u32(&sh.exchange), (S - 1) * a.m * rows * 4);
    sh.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (S > 1) cluster_arrive();
  griddep_wait();
#pragma unroll
  for (int i = 0; i < Q::kDepth; ++i) {
    copy_tokens(i, i);
    copy_commit();
  }
  // The scales of the outputs that this thread finishes: one output feature
  // (rows divides the threads), kKeep tokens; fetched before the stream ends.
  constexpr int kKeep = NT * 8 * kRows / kCoreThreads;
  const int n = n0 + rank * rows + tid % rows;
  const float w_scale = n < a.n ? a.w_scale[n] : 0.0f;
  float x_scale[kKeep];
#pragma unroll
  for (int q = 0; q < kKeep; ++q) {
    const int token = (tid + q * kCoreThreads) / rows;
    x_scale[q] = token < a.m ? a.x_scale[token] : 0.0f;
  }

  const uint32_t red = smem_u32(sh.red);
  int slot = 0;
  // The next block's pieces into registers, and its slot to the one kDepth ahead.
  auto pop = [&](int i, uint4 (&w)[2][2], auto &x, uint32_t x_at, uint32_t x_step) {
    copy_wait<Q::kDepth - 1>();
    if (C > 0) __syncwarp();  // the token rows' pieces are other lanes'
    const uint32_t at = slot * (Q::kPieces * 512);
#pragma unroll
    for (int h = 0; h < 4; ++h) w[h >> 1][h & 1] = lds128(queue + at + h * 512);
#pragma unroll
    for (int c = 0; c < static_cast<int>(sizeof(x) / sizeof(uint4)); ++c) x[c] = lds128(x_at + at + c * x_step);
    if (C > 0) __syncwarp();
    if (i + Q::kDepth < blocks) {
      copy_weights(i + Q::kDepth, slot);
      copy_tokens(i + Q::kDepth, slot);
    }
    copy_commit();
    slot = slot + 1 == Q::kDepth ? 0 : slot + 1;
  };
  uint4 w[2][2];
  if constexpr (C > 0) {
    Dots<C> dots;
    uint4 x[C];
    for (int i = 0; i < blocks; ++i) {
      pop(i, w, x, queue + 4 * 512 + (t - lane) * 16, 64);
      dots.add(x, w);
    }
    dots.finish(red);
  } else {
    const WidenConst wc;
    Sums<NT> sums;
    uint4 x[NT];
    for (int i = 0; i < blocks; ++i) {
      pop(i, w, x, queue + 4 * 512, 512);
      sums.add(wc, x, w);
      if (++sums.blocks == kExactBlocks) sums.move(red, a.m);
    }
    sums.finish(red, a.m);
  }
  copy_wait<0>();
  __syncthreads();

  if (S > 1) {
    cluster_wait();  // every rank has started
    for (int i = tid; i < a.m * kRows / 4; i += kCoreThreads) {
      const int row = i * 4 % kRows, token = i * 4 / kRows, to = row / rows;
      int v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = red_sum(sh.red, token, row + j);
      int *at = sh.recv + (rank * SK_MAX_M + token) * rows + row % rows;
      if (to == rank) {
        *reinterpret_cast<int4 *>(at) = make_int4(v[0], v[1], v[2], v[3]);
      } else {
        st_async_v4_f32(dsmem_map(smem_u32(at), to), __int_as_float(v[0]), __int_as_float(v[1]),
                        __int_as_float(v[2]), __int_as_float(v[3]), dsmem_map(smem_u32(&sh.exchange), to));
      }
    }
    __syncthreads();  // the rank's own part
    if (!mbar_wait_bounded(smem_u32(&sh.exchange), 0, kCoreWaitNs)) {
      sh.abort = 1;
      atomicOr(&g_core_status, SK_DEVICE_WAIT_EPILOGUE);
    }
    cluster_arrive();  // this rank has what it waits for, and sends no more
  }
  if (S == 1 || !*reinterpret_cast<volatile int *>(&sh.abort)) {
#pragma unroll
    for (int q = 0; q < kKeep; ++q) {
      const int i = tid + q * kCoreThreads, token = i / rows;
      if (i >= a.m * rows || n >= a.n) break;
      int s = 0;
      if (S > 1)
        for (int p = 0; p < S; ++p) s += sh.recv[(p * SK_MAX_M + token) * rows + tid % rows];
      else
        s = red_sum(sh.red, token, tid % rows);
      a.y[static_cast<size_t>(token) * a.n + n] =
          bf16_store_bits(__fmul_rn(__fmul_rn(__int2float_rn(s), x_scale[q]), w_scale));
    }
  }
  if (S > 1) cluster_wait();  // shared memory stays until every rank is done with it
}

// ------------------------------------------------------------------- experts
// Who named which expert, in shared memory: the active experts in ascending
// order, and for each the workspace rows (token * top_k + first choice) of its
// tokens in ascending order.
struct Roster {
  uint16_t mask[SK_MAX_EXPERTS];               // tokens of an expert
  uint16_t offset[SK_MAX_EXPERTS];             // its first entry of `rows`
  uint16_t active[SK_MAX_M * SK_MAX_TOP_K];
  int16_t ids[SK_MAX_M * SK_MAX_TOP_K];        // -1: masked
  uint8_t rows[SK_MAX_M * SK_MAX_TOP_K];
  uint8_t some[SK_MAX_EXPERTS / 32], count[SK_MAX_EXPERTS / 32];  // per 32 experts: active ones, their tokens
  int n_active;
};

// The workspace row of choice c of ids (shared memory, -1 where masked): that of
// the token's first choice of the same expert, or -1.
template <typename Id>
__device__ __forceinline__ int choice_row(const Id *ids, int c, int top_k) {
  const int e = ids[c];
  if (e < 0) return -1;
  int f = c / top_k * top_k;
  while (ids[f] != e) ++f;
  return f;
}

__device__ __forceinline__ void clear_roster(Roster &q, int n_experts) {
  uint32_t *mask = reinterpret_cast<uint32_t *>(q.mask);
  for (int e = threadIdx.x; e < (n_experts + 31) / 32 * 16; e += kCoreThreads) mask[e] = 0;
}

// By all threads, after clear_roster.
__device__ __forceinline__ void build_roster(Roster &q, const ExpertsArgs &a) {
  const int choices = a.m * a.top_k, c = threadIdx.x;  // at most 256 choices, as many threads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (c < choices) {
    const int e = load_id(a.ids + c);
    q.ids[c] = static_cast<int16_t>(static_cast<unsigned>(e) < static_cast<unsigned>(a.n_experts) ? e : -1);
  }
  __syncthreads();
  const bool mine = c < choices && choice_row(q.ids, c, a.top_k) == c;
  const int e = mine ? q.ids[c] : 0, token = c / a.top_k;
  if (mine) atomicOr(reinterpret_cast<uint32_t *>(q.mask) + e / 2, 1u << (token + 16 * (e & 1)));
  __syncthreads();
  // Prefix sums over the experts: within groups of 32, a warp each ...
  const int groups = (a.n_experts + 31) / 32;
  for (int g = warp; g < groups; g += kWarps) {
    const int tokens = __popc(static_cast<uint32_t>(q.mask[g * 32 + lane]));
    int sum = tokens;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    q.offset[g * 32 + lane] = static_cast<uint16_t>(sum - tokens);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, tokens);
    if (lane == 31) {
      q.some[g] = static_cast<uint8_t>(__popc(some));
      q.count[g] = static_cast<uint8_t>(min(sum, 255));  // 256 only if nothing comes after
    }
  }
  __syncthreads();
  // ... then over the groups, by every warp for itself.
  int n = lane < groups ? q.some[lane] : 0, tokens = lane < groups ? q.count[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int on = __shfl_up_sync(0xFFFFFFFFu, n, d), ot = __shfl_up_sync(0xFFFFFFFFu, tokens, d);
    if (lane >= d) {
      n += on;
      tokens += ot;
    }
  }
  if (threadIdx.x == 31) q.n_active = n;
  for (int g = warp; g < groups; g += kWarps) {
    const int n0 = g ? __shfl_sync(0xFFFFFFFFu, n, g - 1) : 0, t0 = g ? __shfl_sync(0xFFFFFFFFu, tokens, g - 1) : 0;
    const int x = g * 32 + lane;
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, q.mask[x]);
    q.offset[x] = static_cast<uint16_t>(q.offset[x] + t0);
    if (q.mask[x]) q.active[n0 + __popc(some & ((1u << lane) - 1))] = static_cast<uint16_t>(x);
  }
  __syncthreads();
  if (mine) q.rows[q.offset[e] + __popc(static_cast<uint32_t>(q.mask[e]) & ((1u << token) - 1))] = static_cast<uint8_t>(c);
  __syncthreads();
}

// Gate and up (kUp), or down: persistent CTAs, two per SM, that take items
// (active expert, tile) in turn, expert-major, so that at any time the grid
// streams neighbouring tiles. An up item is 16 gate rows and their 16 up rows, a
// down item 32 rows of the output. The token rows come from the caller (up) or
// from the codes of the activations (down). The queues run on over the items'
// ends: while one item is finished the next one's weights arrive.
template <int NT>
struct ExpertShared {
  uint8_t queue[Queue<NT>::kBytes];
  int red[2][kRedInts];
  Roster roster;
};

template <bool kUp, int NT>
__global__ void __launch_bounds__(kCoreThreads, 2) experts_kernel(ExpertsArgs a) {
  using Q = Queue<NT>;
  extern __shared__ __align__(16) uint8_t raw[];
  ExpertShared<NT> &sh = *reinterpret_cast<ExpertShared<NT> *>(raw);
  const Roster &q = sh.roster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  for (int i = tid; i < 2 * kRedInts; i += kCoreThreads) (&sh.red[0][0])[i] = 0;
  clear_roster(sh.roster, a.n_experts);
  // The ids may come from the kernel ahead. The kernels after this one start
  // only now, so they may read the ids at once, and start on their weights.
  if (kUp) griddep_wait();
  griddep_launch_dependents();
  build_roster(sh.roster, a);

  const int K = kUp ? a.hidden : a.inter, N = kUp ? a.inter : a.hidden;
  constexpr int kTile = kUp ? kRows / 2 : kRows;
  const int tiles = (N + kTile - 1) / kTile, items = q.n_active * tiles;
  const int col = warp * kBlockCols + 16 * t;  // this thread's first column
  const int blocks = max(0, (K - warp * kBlockCols + kWarps * kBlockCols - 1) / (kWarps * kBlockCols));
  const uint32_t queue = smem_u32(sh.queue) + warp * (Q::kDepth * Q::kPieces * 512) + lane * 16;
  const uint64_t policy = l2_policy_evict_first();

  // What is copied next: block fb of item fi, from these rows.
  const int from = col < K ? col : 0;  // a thread without columns copies zeros, but names an address all the same
  int fi = blockIdx.x, fb = 0, count = 0;
  const int8_t *wp[2][2], *xp[NT];
  auto open = [&] {
    if (fi >= items) return;
    const int e = q.active[fi / tiles], n0 = fi % tiles * kTile;
    count = __popc(static_cast<uint32_t>(q.mask[e]));
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // rows past N repeat the last one; their sums are not stored
      const size_t row = kUp ? (static_cast<size_t>(e) * 2 + (h >> 1)) * N + min(n0 + (h & 1) * 8 + g, N - 1)
                             : static_cast<size_t>(e) * N + min(n0 + h * 8 + g, N - 1);
      wp[h >> 1][h & 1] = (kUp ? a.w13 : a.w2) + row * K + from;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = q.rows[q.offset[e] + min(nt * 8 + g, count - 1)];
      xp[nt] = kUp ? a.xq + static_cast<size_t>(row / a.top_k) * K + from : a.hq + static_cast<size_t>(row) * K + from;
    }
  };
  auto copy_weights = [&](int slot) {
    const bool real = col + fb * kWarps * kBlockCols < K;
    const int off = real ? fb * kWarps * kBlockCols : 0;
#pragma unroll
    for (int h = 0; h < 4; ++h)
      copy16_once(queue + (slot * Q::kPieces + h) * 512, wp[h >> 1][h & 1] + off, real, policy);
  };
  auto copy_tokens = [&](int slot) {
    const bool real = col + fb * kWarps * kBlockCols < K;
    const int off = real ? fb * kWarps * kBlockCols : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (nt * 8 + g < count) copy16(queue + (slot * Q::kPieces + 4 + nt) * 512, xp[nt] + off, real);
  };
  auto next = [&] {
    if (++fb == blocks) {
      fb = 0;
      fi += gridDim.x;
      open();
    }
  };

  open();
  if (!kUp && blocks) {  // the weights go ahead of the kernel before this one
    for (int d = 0; d < Q::kDepth && fi < items; ++d, next()) copy_weights(d);
    fi = blockIdx.x;
    fb = 0;
    open();
  }
  if (!kUp) griddep_wait();
  if (blocks)
    for (int d = 0; d < Q::kDepth; ++d) {
      if (fi < items) {
        if (kUp) copy_weights(d);
        copy_tokens(d);
        next();
      }
      copy_commit();
    }

  const WidenConst wc;
  int slot = 0, side = 0, turn = 0;
  for (int i = blockIdx.x; i < items; i += gridDim.x, side ^= 1, ++turn) {
    const int e = q.active[i / tiles], n = i % tiles * kTile + lane % kTile;
    const uint8_t *rows = q.rows + q.offset[e];
    const int tokens = __popc(static_cast<uint32_t>(q.mask[e]));
    int *red = sh.red[side];
    // A warp finishes whole tokens, kTile outputs each, and the warps take turns
    // over the items; what it needs besides the sums is fetched ahead of them.
    const int first = (warp + turn) % kWarps;
    const bool store = lane < kTile && n < N;
    float scale0 = 0.0f, scale1 = 0.0f, row_scale[NT];
    if (store) {
      const size_t at = static_cast<size_t>(e) * (kUp ? 2 * N : N) + n;
      scale0 = (kUp ? a.s13 : a.s2)[at];
      if (kUp) scale1 = a.s13[at + N];
    }
#pragma unroll
    for (int k = 0; k < NT; ++k)
      if (first + k * kWarps < tokens) {
        const int row = rows[first + k * kWarps];
        row_scale[k] = kUp ? a.x_scale[row / a.top_k] : a.hs[row];
      }
    auto stream = [&](auto sums) {
      constexpr int kT = sizeof(sums.xsum) / sizeof(int);
      for (int b = 0; b < blocks; ++b) {
        copy_wait<Q::kDepth - 1>();
        const uint32_t at = queue + slot * (Q::kPieces * 512);
        uint4 w[2][2], x[kT];
#pragma unroll
        for (int h = 0; h < 4; ++h) w[h >> 1][h & 1] = lds128(at + h * 512);
#pragma unroll
        for (int nt = 0; nt < kT; ++nt) x[nt] = lds128(at + (4 + nt) * 512);
        if (fi < items) {
          copy_weights(slot);
          copy_tokens(slot);
          next();
        }
        copy_commit();
        slot = slot + 1 == Q::kDepth ? 0 : slot + 1;
        sums.add(wc, x, w);
        if (++sums.blocks == kExactBlocks) sums.move(smem_u32(red), tokens);
      }
      sums.finish(smem_u32(red), tokens);
    };
    auto stream_few = [&](auto dots) {
      constexpr int C = decltype(dots)::kTokens;
      for (int b = 0; b < blocks; ++b) {
        copy_wait<Q::kDepth - 1>();
        __syncwarp();
        const uint32_t at = queue + slot * (Q::kPieces * 512);
        uint4 w[2][2], x[C];
#pragma unroll
        for (int h = 0; h < 4; ++h) w[h >> 1][h & 1] = lds128(at + h * 512);
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = lds128(at + 4 * 512 + (4 * c + t - lane) * 16);
        __syncwarp();
        if (fi < items) {
          copy_weights(slot);
          copy_tokens(slot);
          next();
        }
        copy_commit();
        slot = slot + 1 == Q::kDepth ? 0 : slot + 1;
        dots.add(x, w);
      }
      dots.finish(smem_u32(red));
    };
    if (tokens == 1) stream_few(Dots<1>());
    else if (tokens == 2) stream_few(Dots<2>());
    else if (NT == 2 && tokens > 8) stream(Sums<NT>());
    else stream(Sums<1>());
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int c = first + k * kWarps;
      if (c >= tokens) break;
      const size_t at = static_cast<size_t>(rows[c]) * N + n;
      if (store) {
        const float s0 = __fmul_rn(__fmul_rn(__int2float_rn(red_sum(red, c, lane)), row_scale[k]), scale0);
        if (kUp) {
          const float up =
              __fmul_rn(__fmul_rn(__int2float_rn(red_sum(red, c, kTile + lane)), row_scale[k]), scale1);
          a.act[at] = s0 / (1.0f + expf(-s0)) * up;
        } else {
          a.o[at] = s0;
        }
      }
      // The token's sums are zero again before this warp passes the barrier of the
      // next item, after which this buffer's turn comes again.
      __syncwarp();
      for (int j = lane; j <= kRows; j += 32) red[c * kRedPitch + j] = 0;
    }
  }
  copy_wait<0>();
}

// Weighted sum of a token's choices, in their order; four columns per thread.
// (Summing in the down kernel, by the last to write a tile, was slower: the fence
// before its counter waits for all of a thread's copies in flight; m16 318 -> 464
// us.)
constexpr int kSumThreads = 64;
__global__ void __launch_bounds__(kSumThreads) experts_sum_kernel(ExpertsArgs a) {
  __shared__ int ids[SK_MAX_TOP_K];
  __shared__ float weights[SK_MAX_TOP_K];
  griddep_launch_dependents();
  const int i = blockIdx.y, n = 4 * (blockIdx.x * kSumThreads + threadIdx.x);
  // (the products' kernels, which this one waits for, started after what wrote
  // the ids and the weights)
  if (static_cast<int>(threadIdx.x) < a.top_k) {
    const int e = load_id(a.ids + i * a.top_k + threadIdx.x);
    ids[threadIdx.x] = static_cast<unsigned>(e) < static_cast<unsigned>(a.n_experts) ? e : -1;
    weights[threadIdx.x] = __int_as_float(load_id(reinterpret_cast<const int32_t *>(a.weights) + i * a.top_k + threadIdx.x));
  }
  __syncthreads();
  griddep_wait();
  if (n >= a.hidden) return;
  float4 o[SK_MAX_TOP_K], s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < SK_MAX_TOP_K; ++j) {
    const int f = j < a.top_k ? choice_row(ids, j, SK_MAX_TOP_K) : -1;
    if (f >= 0) o[j] = *reinterpret_cast<const float4 *>(a.o + static_cast<size_t>(i * a.top_k + f) * a.hidden + n);
  }
#pragma unroll
  for (int j = 0; j < SK_MAX_TOP_K; ++j) {
    if (j >= a.top_k || ids[j] < 0) continue;
    s.x = fmaf(weights[j], o[j].x, s.x);
    s.y = fmaf(weights[j], o[j].y, s.y);
    s.z = fmaf(weights[j], o[j].z, s.z);
    s.w = fmaf(weights[j], o[j].w, s.w);
  }
  const uint32_t lo = bf16_store_bits(s.x) | static_cast<uint32_t>(bf16_store_bits(s.y)) << 16;
  const uint32_t hi = bf16_store_bits(s.z) | static_cast<uint32_t>(bf16_store_bits(s.w)) << 16;
  *reinterpret_cast<uint2 *>(a.y + static_cast<size_t>(i) * a.hidden + n) = make_uint2(lo, hi);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream, bool pdl) {
  const int per = (a.n_experts + 31) / 32;
  auto *kernel = per <= 1 ? route_kernel<1> : per <= 2 ? route_kernel<2> : per <= 4 ? route_kernel<4>
               : per <= 8 ? route_kernel<8> : per <= 16 ? route_kernel<16> : route_kernel<32>;
  return launch(kernel, dim3((static_cast<unsigned>(a.m) + kRouteWarps - 1) / kRouteWarps), dim3(32 * kRouteWarps),
                sizeof(double) * kRouteWarps * (a.n_experts > 16 ? a.n_experts : 16), stream, pdl, 1, a);
}

cudaError_t launch_int8_quantize(const uint16_t *z, int8_t *q, float *scale, int m, int n,
                                 cudaStream_t stream, bool pdl) {
  return launch_quantize(z, q, scale, m, n, static_cast<const int32_t *>(nullptr), 0, stream, pdl);
}

cudaError_t experts_setup() {
  cudaError_t e;
  auto smem = [&](auto *kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  };
  if ((e = smem(gemm_int8_kernel<1, 1>, sizeof(GemmShared<1>)))) return e;
  if ((e = smem(gemm_int8_kernel<1, 2>, sizeof(GemmShared<1>)))) return e;
  if ((e = smem(gemm_int8_kernel<1, 0>, sizeof(GemmShared<1>)))) return e;
  if ((e = smem(gemm_int8_kernel<2, 0>, sizeof(GemmShared<2>)))) return e;
  if ((e = smem(experts_kernel<true, 1>, sizeof(ExpertShared<1>)))) return e;
  if ((e = smem(experts_kernel<true, 2>, sizeof(ExpertShared<2>)))) return e;
  if ((e = smem(experts_kernel<false, 1>, sizeof(ExpertShared<1>)))) return e;
  return smem(experts_kernel<false, 2>, sizeof(ExpertShared<2>));
}

// Slices of K: as many as leave every CTA resident (two per SM) with a block
// for each of its warps.
int int8_splits(int n, int k, int sm_count) {
  const int tiles = (n + kRows - 1) / kRows, slices = (k + kWarps * kBlockCols - 1) / (kWarps * kBlockCols);
  int s = 1;
  while (s < 8 && 2 * s <= slices && static_cast<long long>(tiles) * 2 * s <= 2 * sm_count) s *= 2;
  return s;
}

cudaError_t launch_gemm_int8(const Int8GemmArgs &a, cudaStream_t stream, bool pdl) {
  const dim3 grid((a.n + kRows - 1) / kRows, a.splits);
  auto *kernel = a.m == 1 ? gemm_int8_kernel<1, 1> : a.m == 2 ? gemm_int8_kernel<1, 2>
               : a.m <= 8 ? gemm_int8_kernel<1, 0> : gemm_int8_kernel<2, 0>;
  return launch(kernel, grid, dim3(kCoreThreads),
                a.m > 8 ? sizeof(GemmShared<2>) : sizeof(GemmShared<1>), stream, pdl, a.splits, a);
}

cudaError_t launch_experts_int8(const ExpertsArgs &a, int sm_count, cudaStream_t stream, bool pdl) {
  const unsigned rows = static_cast<unsigned>(a.m * a.top_k);
  const bool many = a.m > 8;
  const size_t smem = many ? sizeof(ExpertShared<2>) : sizeof(ExpertShared<1>);
  // no more CTAs than items if every choice names another expert
  const int active = a.n_experts < a.m * a.top_k ? a.n_experts : a.m * a.top_k;
  auto ctas = [&](int tiles) {
    const long long items = static_cast<long long>(active) * tiles;
    return dim3(static_cast<unsigned>(items < 2 * sm_count ? items : 2 * sm_count));
  };
  cudaError_t e = launch(many ? experts_kernel<true, 2> : experts_kernel<true, 1>,
                         ctas((a.inter + kRows / 2 - 1) / (kRows / 2)), dim3(kCoreThreads), smem, stream, pdl, 1, a);
  if (e != cudaSuccess) return e;
  e = launch_quantize(static_cast<const float *>(a.act), a.hq, a.hs, static_cast<int>(rows), a.inter, a.ids,
                      a.n_experts, stream, pdl);
  if (e != cudaSuccess) return e;
  e = launch(many ? experts_kernel<false, 2> : experts_kernel<false, 1>, ctas((a.hidden + kRows - 1) / kRows),
             dim3(kCoreThreads), smem, stream, pdl, 1, a);
  if (e != cudaSuccess) return e;
  return launch(experts_sum_kernel, dim3((a.hidden / 4 + kSumThreads - 1) / kSumThreads, a.m), dim3(kSumThreads), 0,
                stream, pdl, 1, a);
}

cudaError_t read_core_status(uint32_t *out, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_core_status, sizeof(uint32_t));
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_core_status, &zero, sizeof zero);
}

}  // namespace sk
