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

// One CTA per row, two passes over it. A caller's codes (ids null) may be the
// weight of a call that reads it ahead of its dependency wait, so dependents
// start only once they are written. The codes of the experts' activations are
// read after the wait.
template <typename T>
__global__ void __launch_bounds__(256)
    quantize_kernel(const T *z, int8_t *q, float *scale, int n, const int32_t *ids, int n_experts) {
  if (ids) griddep_launch_dependents();
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
  if (ids) return;
  __threadfence();
  __syncthreads();
  griddep_launch_dependents();
}

// ------------------------------------------------------- the int8 product core
//
// Products at up to 16 tokens stream each weight once; 1 byte of weight meets
// at most 16 tokens, far below what the tensor cores need to be busy, so HBM
// is the bound and the rest has to stay out of its way. Each CTA owns items of
// 32 weight rows and a K range. One producer thread copies them with TMA, a
// stage of 32 rows x 512 codes (16 KiB) at a time, into a ring; eight consumer
// warps each take one 64-code column block of every stage.
//
// The tensor cores multiply int8 codes at FP16: a code widens to FP16 exactly
// by placing code + 128 in the mantissa of 1024 and subtracting 1152 (one
// exclusive-or, two byte permutes and two FP16x2 additions for four codes).
// Products are integers below 2^15 and FP32 holds every partial sum exactly up
// to 2^24, i.e. over 1024 columns of a warp: 16 stages, after which the
// accumulators move to 32-bit integers. The warps' and CTAs' sums are added as
// integers, so neither the order nor the split count can change a result.
//
// K order within a block is free as long as both operands agree: thread t of a
// quad holds columns 16 t .. 16 t + 15 (one 16-byte load of a weight row, one of
// a token row) and feeds four of them to each of four m16n8k16 products.
constexpr int kTileRows = 32;
constexpr int kStageK = 512;
constexpr int kBoxK = 128;                                // one TMA box: 128-byte rows, swizzled
constexpr int kBoxBytes = kTileRows * kBoxK;              // 4 KiB
constexpr int kStageBytes = kTileRows * kStageK;          // 16 KiB
constexpr int kConsumers = 8;                             // warps
constexpr int kCoreThreads = 32 * (kConsumers + 1);
constexpr int kExactStages = 16;                          // stages between moves to integers
constexpr int kRedPitch = kTileRows + 4;                  // ints per token of the sum buffer
constexpr int kRedInts = SK_MAX_M * kRedPitch;
constexpr uint64_t kCoreWaitNs = 2000000000ull;           // 2 s of wall time per wait

__device__ uint32_t g_core_status;  // OR of SK_DEVICE_WAIT_* bits

struct Ring {
  uint32_t data, full, empty;  // shared addresses: stages, then their barriers
  int stages;
  volatile uint32_t *abort;
};

// A wait that runs out raises the abort flag, after which no wait of the CTA
// waits: every role runs through its loops, nothing is stored.
__device__ __forceinline__ void ring_wait(const Ring &r, uint32_t bar, uint32_t parity, uint32_t bit) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*r.abort) return;
    if (globaltimer_ns() - t0 > kCoreWaitNs) {
      *r.abort = 1;
      atomicOr(&g_core_status, bit);
      return;
    }
  }
}

// Copies stage by stage the box rows at (row, batch) of the weight map for
// columns [k0, k1) into the ring; `it` counts the CTA's stages.
__device__ __forceinline__ void produce(const Ring &r, const CUtensorMap *map, int row, int batch,
                                        int k0, int k1, int &it, uint64_t policy) {
  for (int k = k0; k < k1; k += kStageK, ++it) {
    const int st = it % r.stages, lap = it / r.stages;
    if (lap) ring_wait(r, r.empty + 8 * st, (lap - 1) & 1, SK_DEVICE_WAIT_PRODUCER);
    if (*r.abort) continue;
    const int boxes = min(kStageK / kBoxK, (k1 - k + kBoxK - 1) / kBoxK);
    mbar_arrive_expect_tx(r.full + 8 * st, boxes * kBoxBytes);
    for (int b = 0; b < boxes; ++b)
      tma_load_3d(r.data + st * kStageBytes + b * kBoxBytes, map, r.full + 8 * st, k + b * kBoxK, row,
                  batch, policy);
  }
}

// After an abort: waits (again with a limit) for the copies still in flight.
__device__ __forceinline__ void drain(const Ring &r, int it) {
  if (!*r.abort) return;
  for (int i = max(0, it - r.stages); i < it; ++i)
    mbar_wait_bounded(r.full + 8 * (i % r.stages), (i / r.stages) & 1, kCoreWaitNs / 100);
}

// Four int8 codes -> two FP16 pairs, exact.
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
  __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
  lo = *reinterpret_cast<uint32_t *>(&x);
  hi = *reinterpret_cast<uint32_t *>(&y);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of a token row, not through the read-only path: the kernel ahead
// wrote them.
__device__ __forceinline__ uint4 ldg128(const int8_t *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One consumer warp's part of an item: adds to red[token][row] its column
// blocks' products of the 32 tile rows with NT * 8 tokens (red: a shared address). xp[nt]: this lane's
// token row (token nt * 8 + lane / 4) at column 16 (lane % 4), or null.
template <int NT>
__device__ __forceinline__ void consume(const Ring &r, const int8_t *const (&xp)[NT], int k0, int k1,
                                        int &it, uint32_t red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // Tile row of the lane within eight: rows g = 2 i and 2 i + 1, which a load
  // phase reads together, are four apart, so their swizzles use both halves of
  // the 128-byte row and no two lanes of the phase meet in a bank.
  const int pg = ((g & 1) << 2) | (g >> 1);
  const uint32_t chunk = static_cast<uint32_t>((((warp & 1) << 2) | t) ^ pg) << 4;
  const uint32_t at = (warp >> 1) * kBoxBytes + pg * kBoxK + chunk;
  const int kw = warp * 64;
  float acc[2][NT][4];
#pragma unroll
  for (int i = 0; i < 2 * NT * 4; ++i) (&acc[0][0][0])[i] = 0.0f;
  auto flush = [&] {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int token = nt * 8 + 2 * t + (i & 1), row = rt * 16 + pg + (i >> 1) * 8;
          asm volatile("red.shared.add.s32 [%0], %1;" ::"r"(red + 4u * (token * kRedPitch + row)),
                       "r"(__float2int_rn(acc[rt][nt][i]))
                       : "memory");
          acc[rt][nt][i] = 0.0f;
        }
  };
  uint4 xn[NT];
  auto load_x = [&](int k) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      xn[nt] = xp[nt] && k + kw + 16 * t < k1 ? ldg128(xp[nt] + k + kw) : make_uint4(0, 0, 0, 0);
  };
  load_x(k0);
  int done = 0;
  for (int k = k0; k < k1; k += kStageK, ++it) {
    const int st = it % r.stages;
    uint32_t b[NT][8];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      widen(xn[nt].x, b[nt][0], b[nt][1]);
      widen(xn[nt].y, b[nt][2], b[nt][3]);
      widen(xn[nt].z, b[nt][4], b[nt][5]);
      widen(xn[nt].w, b[nt][6], b[nt][7]);
    }
    load_x(k + kStageK);
    ring_wait(r, r.full + 8 * st, (it / r.stages) & 1, SK_DEVICE_WAIT_MMA);
    if (k + kw < k1) {
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const uint32_t base = r.data + st * kStageBytes + at + rt * 16 * kBoxK;
        const uint4 w0 = lds128(base), w1 = lds128(base + 8 * kBoxK);
        const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          widen(lo[i], a0, a2);
          widen(hi[i], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(acc[rt][nt], a0, a1, a2, a3, b[nt][2 * i], b[nt][2 * i + 1]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(r.empty + 8 * st);
    if (++done == kExactStages) {
      flush();
      done = 0;
    }
  }
  if (done) flush();
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}

// Shared memory of a core kernel, from its 1024-aligned base: the ring, two
// sum buffers, the barriers and the abort flag, then `extra` bytes.
struct CoreLayout {
  int red, bars, flag, extra, total;
};
__host__ __device__ inline CoreLayout core_layout(int stages, int extra) {
  CoreLayout l;
  l.red = stages * kStageBytes;
  l.bars = l.red + 2 * kRedInts * 4;
  l.flag = l.bars + 2 * stages * 8;
  l.extra = l.flag + 16;
  l.total = l.extra + extra;
  return l;
}

__device__ __forceinline__ uint8_t *core_smem(uint8_t *raw) {
  return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
}

// Set-up by all threads of a core kernel: barriers, abort flag, zeroed sums.
__device__ __forceinline__ Ring core_setup(uint8_t *smem, const CoreLayout &l, int stages,
                                           const CUtensorMap *map) {
  Ring r;
  r.data = smem_u32(smem);
  r.full = smem_u32(smem + l.bars);
  r.empty = r.full + 8 * stages;
  r.stages = stages;
  r.abort = reinterpret_cast<volatile uint32_t *>(smem + l.flag);
  int *red = reinterpret_cast<int *>(smem + l.red);
  for (int i = threadIdx.x; i < 2 * kRedInts; i += kCoreThreads) red[i] = 0;
  if (threadIdx.x == 32 * kConsumers) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(r.full + 8 * s, 1);
      mbar_init(r.empty + 8 * s, kConsumers);
    }
    *r.abort = 0;
    fence_barrier_init();
    tma_prefetch_map(map);
  }
  __syncthreads();
  return r;
}

// ----------------------------------------------------------------- int8 GEMM
// Grid (tiles of 32 output features, S slices of K), cluster (1, S, 1): every
// CTA holds its whole share in flight at once, two CTAs per SM, so that the
// stream does not wait for scheduling. The S sums of a tile meet in shared
// memory: rank r receives 32 / S rows of every rank and finishes them.
template <int NT>
__global__ void __launch_bounds__(kCoreThreads, 2)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap map, Int8GemmArgs a, int stages) {
  extern __shared__ uint8_t raw[];
  uint8_t *smem = core_smem(raw);
  const int S = a.splits;
  const CoreLayout l = core_layout(stages, 0);
  const Ring r = core_setup(smem, l, stages, &map);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = blockIdx.x * kTileRows, rank = blockIdx.y;
  const int blocks = (a.k + kStageK - 1) / kStageK;
  const int k0 = static_cast<int>(static_cast<long long>(blocks) * rank / S) * kStageK;
  const int k1 = min(a.k, static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / S) * kStageK);
  int *red = reinterpret_cast<int *>(smem + l.red);
  int *recv = red + kRedInts;  // the second sum buffer: [S ranks][16 tokens][32 / S rows]
  griddep_launch_dependents();
  if (S > 1) cluster_arrive();

  if (warp == kConsumers) {
    if (lane == 0) {
      int it = 0;
      produce(r, &map, n0, 0, k0, k1, it, l2_policy_evict_first());
      drain(r, it);
    }
    __syncwarp();
    griddep_wait();
  } else {
    griddep_wait();
    const int8_t *xp[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int token = nt * 8 + (lane >> 2);
      xp[nt] = token < a.m ? a.xq + static_cast<size_t>(token) * a.k + 16 * (lane & 3) : nullptr;
    }
    int it = 0;
    consume<NT>(r, xp, k0, k1, it, smem_u32(red));
    consumer_sync();
  }
  const int rows = kTileRows / S;
  if (S > 1) {
    cluster_wait();  // every rank has started
    if (warp < kConsumers)
      for (int i = tid; i < NT * 8 * kTileRows; i += 32 * kConsumers) {
        const int row = i % kTileRows, token = i / kTileRows;
        const uint32_t to = smem_u32(recv + (rank * SK_MAX_M + token) * rows + row % rows);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_map(to, row / rows)),
                     "r"(red[token * kRedPitch + row])
                     : "memory");
      }
    cluster_arrive();
    cluster_wait();
  }
  if (warp == kConsumers || *r.abort) return;
  for (int i = tid; i < a.m * rows; i += 32 * kConsumers) {
    const int token = i / rows, j = i % rows, n = n0 + rank * rows + j;
    if (n >= a.n) continue;
    int s = 0;
    if (S > 1)
      for (int q = 0; q < S; ++q) s += recv[(q * SK_MAX_M + token) * rows + j];
    else
      s = red[token * kRedPitch + j];
    a.y[static_cast<size_t>(token) * a.n + n] =
        bf16_store_bits(__fmul_rn(__fmul_rn(__int2float_rn(s), a.x_scale[token]), a.w_scale[n]));
  }
}

// ------------------------------------------------------------------- experts
// Who named which expert, in shared memory: the active experts in ascending
// order, and for each the workspace rows (token * top_k + first choice) of its
// tokens in ascending order.
struct Roster {
  uint32_t mask[SK_MAX_EXPERTS];               // tokens of an expert
  uint16_t offset[SK_MAX_EXPERTS];             // its first entry of `rows`
  uint16_t rows[SK_MAX_M * SK_MAX_TOP_K];
  uint16_t active[SK_MAX_M * SK_MAX_TOP_K];
  int n_active;
};

__device__ __forceinline__ int load_id(const int32_t *p) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// The workspace row of choice `c` (token * top_k + j): that of the token's
// first choice of the same expert, or -1 where the choice is masked.
__device__ __forceinline__ int choice_row(const ExpertsArgs &a, int c) {
  const int e = load_id(a.ids + c);
  if (static_cast<unsigned>(e) >= static_cast<unsigned>(a.n_experts)) return -1;
  int f = c / a.top_k * a.top_k;
  while (load_id(a.ids + f) != e) ++f;
  return f;
}

__device__ __forceinline__ void build_roster(Roster &q, const ExpertsArgs &a) {
  const int choices = a.m * a.top_k;
  for (int e = threadIdx.x; e < a.n_experts; e += kCoreThreads) q.mask[e] = 0;
  __syncthreads();
  const int c = threadIdx.x;  // at most 256 choices, 288 threads
  const bool mine = c < choices && choice_row(a, c) == c;
  const int e = mine ? load_id(a.ids + c) : 0, token = c / a.top_k;
  if (mine) atomicOr(&q.mask[e], 1u << token);
  __syncthreads();
  if (threadIdx.x < 32) {
    int n = 0, rows = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += 32) {
      const int x = e0 + threadIdx.x;
      const int count = x < a.n_experts ? __popc(q.mask[x]) : 0;
      const uint32_t some = __ballot_sync(0xFFFFFFFFu, count);
      if (!some) continue;
      int sum = count;  // inclusive prefix
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (static_cast<int>(threadIdx.x) >= d) sum += o;
      }
      if (count) {
        q.active[n + __popc(some & ((1u << threadIdx.x) - 1))] = static_cast<uint16_t>(x);
        q.offset[x] = static_cast<uint16_t>(rows + sum - count);
      }
      n += __popc(some);
      rows += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (threadIdx.x == 0) q.n_active = n;
  }
  __syncthreads();
  if (mine) q.rows[q.offset[e] + __popc(q.mask[e] & ((1u << token) - 1))] = static_cast<uint16_t>(c);
  __syncthreads();
}

// Gate and up (kUp), or down: persistent CTAs, two per SM, that take items
// (active expert, tile) in turn, expert-major, so that at any time the grid
// streams neighbouring tiles. An up item is 16 gate rows and their 16 up rows
// (one box of two batches of the [2 n_experts, inter, hidden] view), a down item
// 32 rows of the output. The token rows come from the caller (up) or from the
// codes of the activations (down).
template <bool kUp>
__global__ void __launch_bounds__(kCoreThreads, 2)
    experts_kernel(const __grid_constant__ CUtensorMap map, ExpertsArgs a, int stages) {
  extern __shared__ uint8_t raw[];
  uint8_t *smem = core_smem(raw);
  const CoreLayout l = core_layout(stages, sizeof(Roster));
  const Ring r = core_setup(smem, l, stages, &map);
  Roster &q = *reinterpret_cast<Roster *>(smem + l.extra);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The ids may come from the kernel ahead. The kernels after this one start
  // only now, so they may read the ids at once, and start on their weights.
  if (kUp) griddep_wait();
  griddep_launch_dependents();
  build_roster(q, a);

  const int K = kUp ? a.hidden : a.inter, N = kUp ? a.inter : a.hidden;
  constexpr int kRows = kUp ? kTileRows / 2 : kTileRows;
  const int tiles = (N + kRows - 1) / kRows, items = q.n_active * tiles;
  int it = 0;
  if (warp == kConsumers) {
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_first();
      for (int i = blockIdx.x; i < items; i += gridDim.x) {
        const int e = q.active[i / tiles];
        produce(r, &map, i % tiles * kRows, kUp ? 2 * e : e, 0, K, it, policy);
      }
      drain(r, it);
    }
    __syncwarp();
    if (!kUp) griddep_wait();
    return;
  }
  if (!kUp) griddep_wait();
  int *red = reinterpret_cast<int *>(smem + l.red);
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int e = q.active[i / tiles], n0 = i % tiles * kRows;
    const uint16_t *rows = q.rows + q.offset[e];
    const int count = __popc(q.mask[e]);
    auto token_row = [&](int c) -> const int8_t * {
      if (c >= count) return nullptr;
      const size_t row = kUp ? rows[c] / a.top_k : rows[c];
      return (kUp ? a.xq : a.hq) + row * K + 16 * (lane & 3);
    };
    if (count > 8) {
      const int8_t *const xp[2] = {token_row(lane >> 2), token_row(8 + (lane >> 2))};
      consume<2>(r, xp, 0, K, it, smem_u32(red));
    } else {
      const int8_t *const xp[1] = {token_row(lane >> 2)};
      consume<1>(r, xp, 0, K, it, smem_u32(red));
    }
    consumer_sync();
    const bool store = !*r.abort;
    for (int j = tid; j < count * kRows; j += 32 * kConsumers) {
      const int c = j / kRows, n = n0 + j % kRows, row = rows[c];
      int *sum = &red[c * kRedPitch + j % kRows];
      if (kUp) {
        if (store && n < N) {
          const size_t gate = static_cast<size_t>(e) * 2 * N + n;
          const float xs = a.x_scale[row / a.top_k];
          const float g = __fmul_rn(__fmul_rn(__int2float_rn(sum[0]), xs), a.s13[gate]);
          const float u = __fmul_rn(__fmul_rn(__int2float_rn(sum[kRows]), xs), a.s13[gate + N]);
          a.act[static_cast<size_t>(row) * N + n] = g / (1.0f + expf(-g)) * u;
        }
        sum[kRows] = 0;
      } else if (store && n < N) {
        a.o[static_cast<size_t>(row) * N + n] =
            __fmul_rn(__fmul_rn(__int2float_rn(sum[0]), a.hs[row]), a.s2[static_cast<size_t>(e) * N + n]);
      }
      sum[0] = 0;
    }
    // The next item adds to the other buffer; this one is zero again before the
    // item after it, whose adds come after the next item's barrier.
    red = reinterpret_cast<int *>(smem + l.red) + (red == reinterpret_cast<int *>(smem + l.red) ? kRedInts : 0);
  }
}

// Weighted sum of a token's choices, in their order.
__global__ void __launch_bounds__(256) experts_sum_kernel(ExpertsArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = blockIdx.x * 256 + threadIdx.x, i = blockIdx.y;
  if (n >= a.hidden) return;
  float s = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    const int row = choice_row(a, i * a.top_k + j);
    if (row >= 0) s = fmaf(a.weights[i * a.top_k + j], a.o[static_cast<size_t>(row) * a.hidden + n], s);
  }
  a.y[static_cast<size_t>(i) * a.hidden + n] = bf16_store_bits(s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream, bool pdl) {
  return launch(route_kernel, dim3((a.m + kRouteWarps - 1) / kRouteWarps), dim3(32 * kRouteWarps),
                static_cast<size_t>(kRouteWarps) * a.n_experts * sizeof(double), stream, pdl, 1, a);
}

cudaError_t launch_int8_quantize(const uint16_t *z, int8_t *q, float *scale, int m, int n,
                                 cudaStream_t stream, bool pdl) {
  return launch(quantize_kernel<uint16_t>, dim3(m), dim3(256), 0, stream, pdl, 1, z, q, scale, n,
                static_cast<const int32_t *>(nullptr), 0);
}

cudaError_t experts_setup(const DeviceInfo &info) {
  cudaFuncAttributes fa;
  cudaError_t e;
  auto all_smem = [&](auto *kernel) {
    if ((e = cudaFuncGetAttributes(&fa, kernel))) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(info.max_smem_optin - fa.sharedSizeBytes));
  };
  if ((e = all_smem(gemm_int8_kernel<1>))) return e;
  if ((e = all_smem(gemm_int8_kernel<2>))) return e;
  if ((e = all_smem(experts_kernel<true>))) return e;
  return all_smem(experts_kernel<false>);
}

// Ring stages of a core kernel with two CTAs per SM.
static int core_stages(int extra) {
  int st = 1;
  while (1024 + core_layout(st + 1, extra).total <= static_cast<int>(kTwoPerSmSmem)) ++st;
  return st;
}

// Slices of K: as many as leave every CTA resident (two per SM) with at least
// one stage each.
int int8_splits(int n, int k, int sm_count) {
  const int tiles = (n + kTileRows - 1) / kTileRows, blocks = (k + kStageK - 1) / kStageK;
  int s = 1;
  while (s < 8 && 2 * s <= blocks && static_cast<long long>(tiles) * 2 * s <= 2 * sm_count) s *= 2;
  return s;
}

cudaError_t launch_gemm_int8(const CUtensorMap &map, const Int8GemmArgs &a, cudaStream_t stream, bool pdl) {
  const int blocks = (a.k + kStageK - 1) / kStageK;
  const int per = (blocks + a.splits - 1) / a.splits;
  const int most = core_stages(0), stages = per < most ? per : most;
  const size_t smem = 1024 + core_layout(stages, 0).total;
  const dim3 grid((a.n + kTileRows - 1) / kTileRows, a.splits);
  return launch(a.m > 8 ? gemm_int8_kernel<2> : gemm_int8_kernel<1>, grid, dim3(kCoreThreads), smem,
                stream, pdl, a.splits, map, a, stages);
}

cudaError_t launch_experts_int8(const CUtensorMap &map13, const CUtensorMap &map2, const ExpertsArgs &a,
                                int sm_count, cudaStream_t stream, bool pdl) {
  const unsigned rows = static_cast<unsigned>(a.m * a.top_k);
  const int stages = core_stages(sizeof(Roster));
  const size_t smem = 1024 + core_layout(stages, sizeof(Roster)).total;
  // no more CTAs than items if every choice names another expert
  const int active = a.n_experts < a.m * a.top_k ? a.n_experts : a.m * a.top_k;
  auto ctas = [&](int tiles) {
    const long long items = static_cast<long long>(active) * tiles;
    return dim3(static_cast<unsigned>(items < 2 * sm_count ? items : 2 * sm_count));
  };
  cudaError_t e = launch(experts_kernel<true>, ctas((a.inter + kTileRows / 2 - 1) / (kTileRows / 2)),
                         dim3(kCoreThreads), smem, stream, pdl, 1, map13, a, stages);
  if (e != cudaSuccess) return e;
  e = launch(quantize_kernel<float>, dim3(rows), dim3(256), 0, stream, pdl, 1,
             static_cast<const float *>(a.act), a.hq, a.hs, a.inter, a.ids, a.n_experts);
  if (e != cudaSuccess) return e;
  e = launch(experts_kernel<false>, ctas((a.hidden + kTileRows - 1) / kTileRows), dim3(kCoreThreads), smem,
             stream, pdl, 1, map2, a, stages);
  if (e != cudaSuccess) return e;
  return launch(experts_sum_kernel, dim3((a.hidden + 255) / 256, a.m), dim3(256), 0, stream, pdl, 1, a);
}

cudaError_t read_core_status(uint32_t *out, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_core_status, sizeof(uint32_t));
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_core_status, &zero, sizeof zero);
}

}  // namespace sk
