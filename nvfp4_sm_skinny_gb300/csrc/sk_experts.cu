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
                   bool pdl, typename std::remove_reference<Args>::type... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------ routing
constexpr int kRouteWarps = 4;  // token rows per CTA

__device__ __forceinline__ float route_logit(const RouteArgs &a, size_t at) {
  if (a.fp32) return static_cast<const float *>(a.logits)[at];
  return bf16_bits_to_f32(static_cast<const uint16_t *>(a.logits)[at]);
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

// One warp per token row, all selection values in FP64 in shared memory.
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(RouteArgs a) {
  extern __shared__ double route_smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kRouteWarps + warp;
  if (row >= a.m) return;
  const int E = a.n_experts;
  double *v = route_smem + warp * E;
  const size_t base = static_cast<size_t>(row) * E;

  double top = -CUDART_INF;
  for (int e = lane; e < E; e += 32) {
    double x = static_cast<double>(route_logit(a, base + e)) + 0.0;
    if (isnan(x)) x = -CUDART_INF;
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

// ------------------------------------------------------------- quantization
// Row maximum of |z| over the CTA; NaN when the row holds an Inf or NaN (the
// bits of |z| order as integers, Inf and NaN above every finite value).
__device__ __forceinline__ float cta_row_max(uint32_t bits) {
  __shared__ uint32_t part[32];
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = bits;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  bits = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0u;
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  return bits >= 0x7F800000u ? CUDART_NAN_F : __uint_as_float(bits);
}

// Code of v in a row of maximum amax (not 0, not NaN): round to nearest even of
// 127 v / amax. f (2^-8 for amax >= 1, else 1) keeps 127 v finite.
__device__ __forceinline__ int int8_code(float v, float amax, float f) {
  return __float2int_rn(__fdiv_rn(__fmul_rn(__fmul_rn(v, f), 127.0f), __fmul_rn(amax, f)));
}

template <typename T>  // uint16_t (BF16 bits) or float
__device__ __forceinline__ float as_f32(T v) {
  if constexpr (std::is_same<T, float>::value) return v;
  else return bf16_bits_to_f32(v);
}

// One CTA per row, two passes over it. The codes may be the weight of a call
// that reads it ahead of its dependency wait, so dependents start only once
// they are written.
template <typename T>
__global__ void __launch_bounds__(256)
    quantize_kernel(const T *z, int8_t *q, float *scale, int n, const int32_t *ids, int n_experts) {
  griddep_wait();
  const size_t row = blockIdx.x;
  if (ids && static_cast<unsigned>(ids[row]) >= static_cast<unsigned>(n_experts)) return;
  uint32_t bits = 0;
  for (int j = threadIdx.x; j < n; j += blockDim.x)
    bits = max(bits, __float_as_uint(as_f32(z[row * n + j])) & 0x7FFFFFFFu);
  const float amax = cta_row_max(bits);
  const float f = amax >= 1.0f ? 0x1p-8f : 1.0f;
  const bool plain = amax > 0.0f;  // neither zero nor NaN
  for (int j = threadIdx.x; j < n; j += blockDim.x)
    q[row * n + j] = static_cast<int8_t>(plain ? int8_code(as_f32(z[row * n + j]), amax, f) : 0);
  if (threadIdx.x == 0) scale[row] = __fdiv_rn(amax, 127.0f);
  __threadfence();
  __syncthreads();
  griddep_launch_dependents();
}

// ----------------------------------------------------------------- int8 GEMM
// sum_k x[k] w[k] over the warp, 16 codes at a time.
__device__ __forceinline__ int warp_dot(const int8_t *x, const int8_t *w, int k) {
  int s = 0;
  for (int c = threadIdx.x & 31; c < k / 16; c += 32) {
    const int4 a = reinterpret_cast<const int4 *>(x)[c], b = reinterpret_cast<const int4 *>(w)[c];
    s = __dp4a(a.x, b.x, s);
    s = __dp4a(a.y, b.y, s);
    s = __dp4a(a.z, b.z, s);
    s = __dp4a(a.w, b.w, s);
  }
  return __reduce_add_sync(0xFFFFFFFFu, s);
}

// One warp per output feature and token.
__global__ void __launch_bounds__(256) gemm_int8_kernel(Int8GemmArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), i = blockIdx.y;
  if (n >= a.n) return;
  const int s = warp_dot(a.xq + static_cast<size_t>(i) * a.k, a.wq + static_cast<size_t>(n) * a.k, a.k);
  if ((threadIdx.x & 31) == 0)
    a.y[static_cast<size_t>(i) * a.n + n] =
        bf16_store_bits(__fmul_rn(__fmul_rn(__int2float_rn(s), a.x_scale[i]), a.w_scale[n]));
}

// ------------------------------------------------------------------- experts
// The workspace row of choice j of token i: that of the token's first choice of
// the same expert, or -1 where the choice is masked.
__device__ __forceinline__ int choice_row(const ExpertsArgs &a, int i, int j) {
  const int e = a.ids[i * a.top_k + j];
  if (static_cast<unsigned>(e) >= static_cast<unsigned>(a.n_experts)) return -1;
  int f = 0;
  while (a.ids[i * a.top_k + f] != e) ++f;
  return i * a.top_k + f;
}

// One warp per choice and activation column.
__global__ void __launch_bounds__(256) experts_up_kernel(ExpertsArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), row = blockIdx.y;
  const int i = row / a.top_k;
  if (n >= a.inter || choice_row(a, i, row % a.top_k) != row) return;
  const size_t e = a.ids[row];
  const int8_t *x = a.xq + static_cast<size_t>(i) * a.hidden;
  const size_t gate = e * 2 * a.inter + n, up = gate + a.inter;
  const int sg = warp_dot(x, a.w13 + gate * a.hidden, a.hidden);
  const int su = warp_dot(x, a.w13 + up * a.hidden, a.hidden);
  if ((threadIdx.x & 31) == 0) {
    const float g = __int2float_rn(sg) * a.x_scale[i] * a.s13[gate];
    const float u = __int2float_rn(su) * a.x_scale[i] * a.s13[up];
    a.act[static_cast<size_t>(row) * a.inter + n] = g / (1.0f + expf(-g)) * u;
  }
}

// One warp per choice and output column.
__global__ void __launch_bounds__(256) experts_down_kernel(ExpertsArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), row = blockIdx.y;
  if (n >= a.hidden || choice_row(a, row / a.top_k, row % a.top_k) != row) return;
  const size_t at = static_cast<size_t>(a.ids[row]) * a.hidden + n;
  const int s = warp_dot(a.hq + static_cast<size_t>(row) * a.inter, a.w2 + at * a.inter, a.inter);
  if ((threadIdx.x & 31) == 0)
    a.o[static_cast<size_t>(row) * a.hidden + n] = __int2float_rn(s) * a.hs[row] * a.s2[at];
}

// Weighted sum of a token's choices, in their order.
__global__ void __launch_bounds__(256) experts_sum_kernel(ExpertsArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = blockIdx.x * 256 + threadIdx.x, i = blockIdx.y;
  if (n >= a.hidden) return;
  float s = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    const int row = choice_row(a, i, j);
    if (row >= 0) s = fmaf(a.weights[i * a.top_k + j], a.o[static_cast<size_t>(row) * a.hidden + n], s);
  }
  a.y[static_cast<size_t>(i) * a.hidden + n] = bf16_store_bits(s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream, bool pdl) {
  return launch(route_kernel, dim3((a.m + kRouteWarps - 1) / kRouteWarps), dim3(32 * kRouteWarps),
                static_cast<size_t>(kRouteWarps) * a.n_experts * sizeof(double), stream, pdl, a);
}

cudaError_t launch_int8_quantize(const uint16_t *z, int8_t *q, float *scale, int m, int n,
                                 cudaStream_t stream, bool pdl) {
  return launch(quantize_kernel<uint16_t>, dim3(m), dim3(256), 0, stream, pdl, z, q, scale, n,
                static_cast<const int32_t *>(nullptr), 0);
}

cudaError_t launch_gemm_int8(const Int8GemmArgs &a, cudaStream_t stream, bool pdl) {
  return launch(gemm_int8_kernel, dim3((a.n + 7) / 8, a.m), dim3(256), 0, stream, pdl, a);
}

cudaError_t launch_experts_int8(const ExpertsArgs &a, cudaStream_t stream, bool pdl) {
  const unsigned rows = static_cast<unsigned>(a.m * a.top_k);
  cudaError_t e = launch(experts_up_kernel, dim3((a.inter + 7) / 8, rows), dim3(256), 0, stream, pdl, a);
  if (e != cudaSuccess) return e;
  e = launch(quantize_kernel<float>, dim3(rows), dim3(256), 0, stream, pdl,
             static_cast<const float *>(a.act), a.hq, a.hs, a.inter, a.ids, a.n_experts);
  if (e != cudaSuccess) return e;
  e = launch(experts_down_kernel, dim3((a.hidden + 7) / 8, rows), dim3(256), 0, stream, pdl, a);
  if (e != cudaSuccess) return e;
  return launch(experts_sum_kernel, dim3((a.hidden + 255) / 256, a.m), dim3(256), 0, stream, pdl, a);
}

}  // namespace sk
