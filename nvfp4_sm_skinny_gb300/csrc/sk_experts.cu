// Device code of the int8 routed experts: routing (sk_route), int8 quantization
// of rows (sk_int8_quantize), the int8 GEMM (sk_gemm_int8) and the experts'
// products (sk_experts_int8). include/sk.h has the formulas.
#include <math_constants.h>

#include <cstdlib>
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
// is the bound and the rest has to stay out of its way. One producer thread
// copies weights with TMA, a stage of 16 KiB at a time, into a ring, and the
// token rows' columns with them; eight consumer warps multiply.
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
// result.
//
// K order within a block is free as long as both operands agree: thread t of a
// quad holds columns 16 t .. 16 t + 15 (one 16-byte load of a weight row, one of
// a token row) and feeds four of them to each of four m16n8k16 products.
constexpr int kBoxK = 128;                                // columns of a TMA box, swizzled over 128 bytes
constexpr int kStageWBytes = 16 * 1024;                   // weights of a stage
constexpr int kConsumers = 8;                             // warps
constexpr int kCoreThreads = 32 * (kConsumers + 1);
constexpr int kExactStages = 8;                           // a warp's stages between moves to integers
constexpr uint64_t kCoreWaitNs = 2000000000ull;           // 2 s of wall time per wait

// A stage's shape: kRows rows by 16 KiB / kRows columns. A warp takes 64 columns
// and 16 kTiles rows of a stage, kWarps warps a whole stage; with kSets > 1 the
// sets of warps take turns, so that one set's latency hides behind another's.
// kGather: the token rows come one by one (bulk copies to rows of a fixed
// pitch); else they are a tile of the activations ([m, k], TMA boxes of 8 or 16
// rows).
template <int kRows_, int kTiles_, bool kGather_>
struct Shape {
  static constexpr bool kGather = kGather_;
  static constexpr int kRows = kRows_, kTiles = kTiles_;
  static constexpr int kStageK = kStageWBytes / kRows;
  static constexpr int kRowGroups = kRows / (16 * kTiles);
  static constexpr int kWarps = kStageK / 64 * kRowGroups;
  static constexpr int kSets = kConsumers / kWarps;
  static constexpr int kBoxes = kStageK / kBoxK;
  static constexpr int kBoxBytes = kRows * kBoxK;
  static constexpr int kXPitch = kStageK + 64;           // kGather: bytes per token row of a stage
  // ints per token of the sum buffer: the rows' sums, then the token's own
  static constexpr int kRedPitch = kRows + (kGather ? 4 : 8);
  static constexpr int kRedInts = SK_MAX_M * kRedPitch;
  __host__ __device__ static constexpr int x_rows(int m) { return m > 8 ? 16 : 8; }
  __host__ __device__ static constexpr int stage_bytes(int m) {
    return (kStageWBytes + x_rows(m) * (kGather ? kXPitch : kStageK) + 1023) / 1024 * 1024;
  }
};
using TallShape = Shape<128, 4, false>;   // 128 rows x 128 columns, two sets of four warps
using LowShape = Shape<32, 2, false>;     // 32 rows x 512 columns
using ExpertShape = Shape<32, 2, true>;

__device__ uint32_t g_core_status;  // OR of SK_DEVICE_WAIT_* bits

struct Ring {
  uint32_t data, full, empty;  // shared addresses: stages, then their barriers
  int stages, stage_bytes, x_rows;
  volatile uint32_t *abort;
};

// A role's place in the ring.
struct RingPos {
  int st = 0;
  uint32_t lap = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      ++lap;
    }
  }
};

// A wait that runs out raises the abort flag, after which no wait of the CTA
// waits: every role runs through its loops, nothing is stored. False after an
// abort.
__device__ __forceinline__ bool ring_wait(const Ring &r, uint32_t bar, uint32_t parity, uint32_t bit) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*r.abort) return false;
    if (globaltimer_ns() - t0 > kCoreWaitNs) {
      *r.abort = 1;
      atomicOr(&g_core_status, bit);
      return false;
    }
  }
  return true;
}

// After an abort: waits (again with a limit) for the copies still in flight, of
// the last of the `it` stages sent.
__device__ __forceinline__ void drain(const Ring &r, int it) {
  for (int i = max(0, it - r.stages); i < it; ++i)
    mbar_wait_bounded(r.full + 8 * (i % r.stages), (i / r.stages) & 1, kCoreWaitNs / 100);
}

// One item's sources: the weight tile's coordinates; with kGather the token row
// of each of the first `tokens` lanes.
struct Source {
  int row, batch, tokens;
  const int8_t *x;
};

// The copies of a stage, each by a lane of its own in one instruction: the
// producer shares its scheduler with busy warps, and a loop over the copies by
// one thread held the ring back (m1 [8192, 32768] in 32-row tiles: 60 us, the
// copies alone 44 us). `tokens` tells whether the token rows are sent too, or
// the weights alone, or (weights false) the token rows alone.
template <typename T>
__device__ __forceinline__ void copy_stage(const Ring &r, const CUtensorMap *map, const CUtensorMap *xmap,
                                           const Source &s, int st, int k, int k1, bool weights,
                                           bool tokens, uint64_t policy) {
  const int lane = threadIdx.x & 31, left = k1 - k;
  const uint32_t to = r.data + st * r.stage_bytes, bar = r.full + 8 * st;
  if (weights) {
    if (lane == 0) {
      const int boxes = left >= T::kStageK ? T::kBoxes : (left + kBoxK - 1) / kBoxK;
      mbar_arrive_expect_tx(bar, boxes * T::kBoxBytes + (T::kGather ? s.tokens * min(T::kStageK, left)
                                                                    : boxes * r.x_rows * kBoxK));
    }
    __syncwarp();  // a stage's bytes are announced before any of them arrives
  }
  // lanes 0 .. kBoxes - 1: weight boxes; the next kBoxes: token boxes
  const int b = lane % T::kBoxes;
  const bool w = lane < T::kBoxes;
  const bool mine = w ? weights : !T::kGather && tokens && lane < 2 * T::kBoxes;
  if (mine && b * kBoxK < left)
    tma_load_3d(to + (w ? b * T::kBoxBytes : kStageWBytes + b * r.x_rows * kBoxK), w ? map : xmap, bar,
                k + b * kBoxK, w ? s.row : 0, w ? s.batch : 0, policy);
  if (T::kGather && tokens && lane < s.tokens)
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            to + kStageWBytes + lane * T::kXPitch),
        "l"(__cvta_generic_to_global(s.x + k)), "r"(min(T::kStageK, left)), "r"(bar)
        : "memory");
}

// The producer warp: copies columns [k0, k1) of the items first, first + step,
// ... below last, stage by stage. With `early` the token rows are not written
// yet: the first ring of weights goes out before the wait for the kernel ahead,
// its token rows after it.
template <typename T, typename Items>
__device__ __forceinline__ void produce(const Ring &r, const CUtensorMap *map, const CUtensorMap *xmap,
                                        Items source, int first, int last, int step, int k0, int k1,
                                        bool early) {
  constexpr int kStageK = T::kStageK;
  const int lane = threadIdx.x & 31;
  // each weight is read once, the token rows by every tile
  const uint64_t policy = lane < T::kBoxes ? l2_policy_evict_first() : l2_policy_evict_last();
  int sent = 0;
  if (early) {
    for (int i = first; i < last && sent < r.stages; i += step) {
      const Source s = source(i);
      for (int k = k0; k < k1 && sent < r.stages; k += kStageK, ++sent)
        copy_stage<T>(r, map, xmap, s, sent, k, k1, true, false, policy);
    }
    griddep_wait();
    int n = 0;
    for (int i = first; i < last && n < sent; i += step) {
      const Source s = source(i);
      for (int k = k0; k < k1 && n < sent; k += kStageK, ++n)
        copy_stage<T>(r, map, xmap, s, n, k, k1, false, true, policy);
    }
  }
  RingPos pos;
  int it = 0;
  for (int i = first; i < last; i += step) {
    const Source s = source(i);
    for (int k = k0; k < k1; k += kStageK, ++it, pos.next(r.stages)) {
      if (it < sent) continue;
      const bool go = !pos.lap || ring_wait(r, r.empty + 8 * pos.st, (pos.lap - 1) & 1,
                                            SK_DEVICE_WAIT_PRODUCER);
      if (!__all_sync(0xFFFFFFFFu, go)) {
        drain(r, it);
        return;
      }
      copy_stage<T>(r, map, xmap, s, pos.st, k, k1, true, true, policy);
    }
  }
  if (__any_sync(0xFFFFFFFFu, *r.abort)) drain(r, it);
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

// One consumer warp's part of an item: adds its products with the first `tokens`
// (at most 8 NT) token rows of the stages to red[token][row] (a shared address),
// and the token rows' own sums to red[token][kRows]. Rows of a stage beyond
// `tokens` hold zeros or leftovers, whose sums are not added. seq counts the
// CTA's stages, for the sets' turns.
template <typename T, int NT>
__device__ __forceinline__ void consume(const Ring &r, int tokens, int k0, int k1, int &seq, RingPos &pos,
                                        uint32_t red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int set = warp / T::kWarps, w = warp % T::kWarps;
  const int cg = w / T::kRowGroups, rg = w % T::kRowGroups;  // column and row group
  // Tile row of the lane within eight: rows g = 2 i and 2 i + 1, which a load
  // phase reads together, are four apart, so their swizzles use both halves of
  // the 128-byte row and no two lanes of the phase meet in a bank. Gathered
  // token rows, at a pitch of an odd number of 64 bytes, need no reordering.
  const int pg = ((g & 1) << 2) | (g >> 1);
  const uint32_t chunk = static_cast<uint32_t>((((cg & 1) << 2) | t) ^ pg) << 4;
  const uint32_t at = r.data + (cg >> 1) * T::kBoxBytes + (rg * 16 * T::kTiles + pg) * kBoxK + chunk;
  const uint32_t xat = r.data + kStageWBytes +
                       (T::kGather ? g * T::kXPitch + cg * 64 + t * 16
                                   : (cg >> 1) * r.x_rows * kBoxK + pg * kBoxK + chunk);
  constexpr uint32_t kXStep = 8 * (T::kGather ? T::kXPitch : kBoxK);
  const WidenConst wc;
  const int ones = rg == 0 ? 0x01010101 : 0;  // one row group sums the token's codes
  float acc[T::kTiles][NT][4];
  int xsum[NT];
#pragma unroll
  for (int i = 0; i < T::kTiles * NT * 4; ++i) (&acc[0][0][0])[i] = 0.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xsum[nt] = 0;
  auto flush = [&] {
#pragma unroll
    for (int rt = 0; rt < T::kTiles; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int token = nt * 8 + (T::kGather ? 2 * t + (i & 1) : t + 4 * (i & 1));
          const int row = (rg * T::kTiles + rt) * 16 + pg + (i >> 1) * 8;
          if (token < tokens)
            red_shared(red + 4u * (token * T::kRedPitch + row), __float2int_rn(acc[rt][nt][i] * 0x1p24f));
          acc[rt][nt][i] = 0.0f;
        }
  };
  int done = 0;
  for (int k = k0; k < k1; k += T::kStageK, pos.next(r.stages), ++seq) {
    if (T::kSets > 1 && seq % T::kSets != set) continue;
    const uint32_t off = pos.st * r.stage_bytes;
    ring_wait(r, r.full + 8 * pos.st, pos.lap & 1, SK_DEVICE_WAIT_MMA);
    if (k + cg * 64 < k1) {
      uint4 x[NT], wt[T::kTiles][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt] = lds128(xat + off + nt * kXStep);
#pragma unroll
      for (int rt = 0; rt < T::kTiles; ++rt) {
        wt[rt][0] = lds128(at + off + rt * 16 * kBoxK);
        wt[rt][1] = lds128(at + off + (rt * 16 + 8) * kBoxK);
      }
      uint32_t b[NT][8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t xw[4] = {x[nt].x, x[nt].y, x[nt].z, x[nt].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          widen_token(xw[i], b[nt][2 * i], b[nt][2 * i + 1]);
          xsum[nt] = __dp4a(static_cast<int>(xw[i]), ones, xsum[nt]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int rt = 0; rt < T::kTiles; ++rt) {
          const uint4 &w0 = wt[rt][0], &w1 = wt[rt][1];
          uint32_t a0, a1, a2, a3;
          widen_weight(wc, i == 0 ? w0.x : i == 1 ? w0.y : i == 2 ? w0.z : w0.w, a0, a2);
          widen_weight(wc, i == 0 ? w1.x : i == 1 ? w1.y : i == 2 ? w1.z : w1.w, a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(acc[rt][nt], a0, a1, a2, a3, b[nt][2 * i], b[nt][2 * i + 1]);
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(r.empty + 8 * pos.st);
    if (++done == kExactStages) {
      flush();
      done = 0;
    }
  }
  if (done) flush();
  if (rg == 0)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int token = nt * 8 + (T::kGather ? g : pg);
      if (token < tokens) red_shared(red + 4u * (token * T::kRedPitch + T::kRows), xsum[nt]);
    }
}

// The sum of products of a token with a tile row: the correction of the weights'
// offset by 128 (modulo 2^32).
template <typename T>
__device__ __forceinline__ int red_sum(const int *red, int token, int row) {
  const uint32_t s = red[token * T::kRedPitch + row], x = red[token * T::kRedPitch + T::kRows];
  return static_cast<int>(s - 128u * x);
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}

// Shared memory of a core kernel, from its 1024-aligned base: the ring, two
// sum buffers, the barriers and the abort flag, then `extra` bytes.
struct CoreLayout {
  int red, bars, flag, extra, total;
};
template <typename T>
__host__ __device__ inline CoreLayout core_layout(int m, int stages, int extra) {
  CoreLayout l;
  l.red = stages * T::stage_bytes(m);
  l.bars = l.red + 2 * T::kRedInts * 4;
  l.flag = l.bars + 2 * stages * 8;
  l.extra = l.flag + 16;
  l.total = l.extra + extra;
  return l;
}

__device__ __forceinline__ uint8_t *core_smem(uint8_t *raw) {
  return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
}

// Set-up by all threads of a core kernel: barriers, abort flag, zeroed sums.
template <typename T>
__device__ __forceinline__ Ring core_setup(uint8_t *smem, const CoreLayout &l, int m, int stages,
                                           const CUtensorMap *map) {
  Ring r;
  r.data = smem_u32(smem);
  r.full = smem_u32(smem + l.bars);
  r.empty = r.full + 8 * stages;
  r.stages = stages;
  r.stage_bytes = T::stage_bytes(m);
  r.x_rows = T::x_rows(m);
  r.abort = reinterpret_cast<volatile uint32_t *>(smem + l.flag);
  int *red = reinterpret_cast<int *>(smem + l.red);
  for (int i = threadIdx.x; i < 2 * T::kRedInts; i += kCoreThreads) red[i] = 0;
  if (threadIdx.x == 32 * kConsumers) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(r.full + 8 * s, 1);
      mbar_init(r.empty + 8 * s, T::kWarps);
    }
    *r.abort = 0;
    fence_barrier_init();
    tma_prefetch_map(map);
  }
  __syncthreads();
  return r;
}

// ----------------------------------------------------------------- int8 GEMM
// Grid (tiles of kRows output features, S slices of K), cluster (1, S, 1):
// every CTA is resident from the start, two per SM, so that the stream does not
// wait for scheduling. The S sums of a tile meet in shared memory: rank r
// receives a slice of the rows from every rank and finishes them.
template <typename T, int NT>
__global__ void __launch_bounds__(kCoreThreads, 2)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap xmap,
                     Int8GemmArgs a, int stages) {
  extern __shared__ uint8_t raw[];
  uint8_t *smem = core_smem(raw);
  const int S = a.splits;
  const CoreLayout l = core_layout<T>(a.m, stages, 0);
  const Ring r = core_setup<T>(smem, l, a.m, stages, &map);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int n0 = blockIdx.x * T::kRows, rank = blockIdx.y;
  const int blocks = (a.k + T::kStageK - 1) / T::kStageK;
  const int k0 = static_cast<int>(static_cast<long long>(blocks) * rank / S) * T::kStageK;
  const int k1 = min(a.k, static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / S) * T::kStageK);
  int *red = reinterpret_cast<int *>(smem + l.red);
  int *recv = red + T::kRedInts;  // the second sum buffer: [S ranks][16 tokens][rows / S]
  griddep_launch_dependents();
  if (S > 1) cluster_arrive();

  if (warp == kConsumers) {
    produce<T>(r, &map, &xmap, [&](int) { return Source{n0, 0, a.m, nullptr}; }, 0, 1, 1, k0, k1,
                       true);
    __syncwarp();
  } else {
    RingPos pos;
    int seq = 0;
    consume<T, NT>(r, a.m, k0, k1, seq, pos, smem_u32(red));
    consumer_sync();
    griddep_wait();  // the scales, and the order of the stores to y
  }
  const int rows = T::kRows / S;
  if (S > 1) {
    cluster_wait();  // every rank has started
    if (warp < kConsumers)
      for (int i = tid; i < a.m * T::kRows; i += 32 * kConsumers) {
        const int row = i % T::kRows, token = i / T::kRows;
        const uint32_t to = smem_u32(recv + (rank * SK_MAX_M + token) * rows + row % rows);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_map(to, row / rows)),
                     "r"(red_sum<T>(red, token, row))
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
      s = red_sum<T>(red, token, j);
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
  using T = ExpertShape;
  const CoreLayout l = core_layout<T>(a.m, stages, sizeof(Roster));
  const Ring r = core_setup<T>(smem, l, a.m, stages, &map);
  Roster &q = *reinterpret_cast<Roster *>(smem + l.extra);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The ids may come from the kernel ahead. The kernels after this one start
  // only now, so they may read the ids at once, and start on their weights.
  if (kUp) griddep_wait();
  griddep_launch_dependents();
  build_roster(q, a);

  const int K = kUp ? a.hidden : a.inter, N = kUp ? a.inter : a.hidden;
  constexpr int kRows = kUp ? T::kRows / 2 : T::kRows;
  const int tiles = (N + kRows - 1) / kRows, items = q.n_active * tiles;
  if (warp == kConsumers) {
    produce<T>(r, &map, nullptr,
            [&](int i) {
              const int e = q.active[i / tiles], count = __popc(q.mask[e]);
              const int row = q.rows[q.offset[e] + (lane < count ? lane : 0)];
              return Source{i % tiles * kRows, kUp ? 2 * e : e, count,
                            (kUp ? a.xq + static_cast<size_t>(row / a.top_k) * K
                                 : a.hq + static_cast<size_t>(row) * K)};
            },
            blockIdx.x, items, gridDim.x, 0, K, !kUp);
    return;
  }
  if (!kUp) griddep_wait();
  int *red = reinterpret_cast<int *>(smem + l.red);
  RingPos pos;
  int seq = 0;
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int e = q.active[i / tiles], n0 = i % tiles * kRows;
    const uint16_t *rows = q.rows + q.offset[e];
    const int count = __popc(q.mask[e]);
    if (count > 8) consume<T, 2>(r, count, 0, K, seq, pos, smem_u32(red));
    else consume<T, 1>(r, count, 0, K, seq, pos, smem_u32(red));
    consumer_sync();
    const bool store = !*r.abort;
    for (int j = tid; j < count * kRows; j += 32 * kConsumers) {
      const int c = j / kRows, at = j % kRows, n = n0 + at, row = rows[c];
      if (!store || n >= N) continue;
      const float s0 = __int2float_rn(red_sum<T>(red, c, at));
      if (kUp) {
        const size_t gate = static_cast<size_t>(e) * 2 * N + n;
        const float xs = a.x_scale[row / a.top_k];
        const float g = __fmul_rn(__fmul_rn(s0, xs), a.s13[gate]);
        const float u = __fmul_rn(__fmul_rn(__int2float_rn(red_sum<T>(red, c, kRows + at)), xs),
                                  a.s13[gate + N]);
        a.act[static_cast<size_t>(row) * N + n] = g / (1.0f + expf(-g)) * u;
      } else {
        a.o[static_cast<size_t>(row) * N + n] =
            __fmul_rn(__fmul_rn(s0, a.hs[row]), a.s2[static_cast<size_t>(e) * N + n]);
      }
    }
    consumer_sync();
    for (int j = tid; j < count * T::kRedPitch; j += 32 * kConsumers) red[j] = 0;
    // The next item adds to the other buffer; this one is zero again before the
    // item after it, whose adds come after the next item's barrier.
    red = reinterpret_cast<int *>(smem + l.red) + (red == reinterpret_cast<int *>(smem + l.red) ? T::kRedInts : 0);
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
  if ((e = all_smem(gemm_int8_kernel<LowShape, 1>))) return e;
  if ((e = all_smem(gemm_int8_kernel<LowShape, 2>))) return e;
  if ((e = all_smem(gemm_int8_kernel<TallShape, 1>))) return e;
  if ((e = all_smem(gemm_int8_kernel<TallShape, 2>))) return e;
  if ((e = all_smem(experts_kernel<true>))) return e;
  return all_smem(experts_kernel<false>);
}

// Ring stages of a core kernel with two CTAs per SM, for `need` stages of work.
// A multiple of the sets: a slot then belongs to one set, which waits for each
// of its laps in turn (a wait for a lap before the one ahead has landed would
// fall through, as it goes by the lap's parity).
template <typename T>
static int core_stages(int m, int extra, long long need) {
  int st = T::kSets;
  while (st < need && 1024 + core_layout<T>(m, st + T::kSets, extra).total <= static_cast<int>(kTwoPerSmSmem))
    st += T::kSets;
  return st;
}

// Tiles of 128 rows where K can be cut into enough slices to fill the SMs, of
// 32 rows otherwise: the tokens' codes pass L2 once per tile, at 16 tokens
// 12.5 % of the weights' bytes with 128 rows and 50 % with 32. S is the largest
// of 1, 2, 4, 8 that leaves every CTA resident (two per SM) with a stage at
// least.
Int8Plan plan_int8(int m, int n, int k, int splits, int sm_count) {
  auto best = [&](int rows, int stage_k) {
    const int tiles = (n + rows - 1) / rows, blocks = (k + stage_k - 1) / stage_k;
    int s = 1;
    while (s < 8 && 2 * s <= blocks && static_cast<long long>(tiles) * 2 * s <= 2 * sm_count) s *= 2;
    return s;
  };
  const int tall = splits ? splits : best(128, 128);
  Int8Plan p;
  p.tall = m > 2 && static_cast<long long>((n + 127) / 128) * tall >= sm_count;
  if (const char *v = std::getenv("SK_INT8_TALL")) p.tall = v[0] == '1';
  p.splits = p.tall ? tall : splits ? splits : best(32, 512);
  return p;
}

template <typename T>
static cudaError_t launch_gemm_int8_rows(const CUtensorMap &map, const CUtensorMap &xmap,
                                         const Int8GemmArgs &a, cudaStream_t stream, bool pdl) {
  const int blocks = (a.k + T::kStageK - 1) / T::kStageK;
  const int per = (blocks + a.splits - 1) / a.splits;
  const int stages = core_stages<T>(a.m, 0, per);
  const size_t smem = 1024 + core_layout<T>(a.m, stages, 0).total;
  const dim3 grid((a.n + T::kRows - 1) / T::kRows, a.splits);
  return launch(a.m > 8 ? gemm_int8_kernel<T, 2> : gemm_int8_kernel<T, 1>, grid, dim3(kCoreThreads),
                smem, stream, pdl, a.splits, map, xmap, a, stages);
}

cudaError_t launch_gemm_int8(const CUtensorMap &map, const CUtensorMap &xmap, const Int8GemmArgs &a,
                             bool tall, cudaStream_t stream, bool pdl) {
  return tall ? launch_gemm_int8_rows<TallShape>(map, xmap, a, stream, pdl)
              : launch_gemm_int8_rows<LowShape>(map, xmap, a, stream, pdl);
}

cudaError_t launch_experts_int8(const CUtensorMap &map13, const CUtensorMap &map2, const ExpertsArgs &a,
                                int sm_count, cudaStream_t stream, bool pdl) {
  const unsigned rows = static_cast<unsigned>(a.m * a.top_k);
  const int stages = core_stages<ExpertShape>(a.m, sizeof(Roster), 64);
  const size_t smem = 1024 + core_layout<ExpertShape>(a.m, stages, sizeof(Roster)).total;
  // no more CTAs than items if every choice names another expert
  const int active = a.n_experts < a.m * a.top_k ? a.n_experts : a.m * a.top_k;
  auto ctas = [&](int tiles) {
    const long long items = static_cast<long long>(active) * tiles;
    return dim3(static_cast<unsigned>(items < 2 * sm_count ? items : 2 * sm_count));
  };
  cudaError_t e = launch(experts_kernel<true>, ctas((a.inter + 15) / 16),
                         dim3(kCoreThreads), smem, stream, pdl, 1, map13, a, stages);
  if (e != cudaSuccess) return e;
  e = launch(quantize_kernel<float>, dim3(rows), dim3(256), 0, stream, pdl, 1,
             static_cast<const float *>(a.act), a.hq, a.hs, a.inter, a.ids, a.n_experts);
  if (e != cudaSuccess) return e;
  e = launch(experts_kernel<false>, ctas((a.hidden + 31) / 32), dim3(kCoreThreads), smem,
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
