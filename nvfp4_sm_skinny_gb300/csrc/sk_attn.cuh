// What the kernels of the 4-bit key/value cache share: conversions of codes and
// scales, arithmetic on pairs, and how attention cuts its work and keeps its sums.
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "sk.h"
#include "sk_internal.h"
#include "sk_ptx.cuh"

namespace sk {
namespace {

constexpr uint64_t kCacheWaitNs = 2000000000ull;   // 2 s of wall time per wait
constexpr uint32_t kAll = 0xFFFFFFFFu;

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

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Untiled bulk copy global -> shared, completion counted on `bar` in bytes. What is
// copied leaves L2 first: the cache is read once, and table, queries and unfinished
// results stay (b64 d128: 66.2 us without, 64.0 with).
__device__ __forceinline__ void bulk_load_once(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(l2_policy_evict_first())
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two e2m1 codes of byte i of a word as an FP16 pair, the low nibble in the low half.
__device__ __forceinline__ uint32_t widen_e2m1(uint32_t w, int i) {
  uint32_t r;
  if (i == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if (i == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if (i == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Two e4m3 bytes as an FP16 pair, exact.
__device__ __forceinline__ uint32_t widen_e4m3(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

__device__ __forceinline__ void mma_f16(float &c0, float &c1, float &c2, float &c3, uint32_t a0, uint32_t a1,
                                        uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// As mma_f16, into a sum that starts at 0.
__device__ __forceinline__ void mma_f16_first(float &c0, float &c1, float &c2, float &c3, uint32_t a0, uint32_t a1,
                                              uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c0), "=f"(c1), "=f"(c2), "=f"(c3)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Two FP32 operations in one instruction: (x, y) = (x, y) * (cx, cy) + (dx, dy), and + (dx, dy).
__device__ __forceinline__ void fma_f32x2(float &x, float &y, float cx, float cy, float dx, float dy) {
  asm("{\n\t.reg .b64 v, c, d;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 c, {%2, %3};\n\tmov.b64 d, {%4, %5};\n\t"
      "fma.rn.f32x2 v, v, c, d;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(cx), "f"(cy), "f"(dx), "f"(dy));
}
__device__ __forceinline__ void add_f32x2(float &x, float &y, float dx, float dy) {
  asm("{\n\t.reg .b64 v, d;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 d, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, d;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(dx), "f"(dy));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ---------------------------------------------------------------- attention
// Scores are kept as powers of two relative to a base that is at most 15 and after
// an update 7 (in tiles of 128 rows, 7 to 8) below the largest, so that P fits FP16 and
// what is 2^31 times smaller than the largest still counts: a p below 2^-14 is rounded to
// the step of FP16's subnormal numbers, off by 2^-25, which is 2^-32 of 2^7. (What is scaled
// in FP16 as the base moves is rounded twice, by 2^-26 at most the first time.) The base
// moves, and the sums are scaled, only when a score exceeds it by 2^15, or where scores are
// looked at for another reason.
constexpr float kTop = 15.0f, kAim = 7.0f;

constexpr int kBegins = 1, kEnds = 2;  // the part holds the first, the last chunk of the item

// Floats of a part's result: a base and a sum per row, then the rows.
__host__ __device__ constexpr int attn_part_floats(int d, int nt) { return 16 * nt + 8 * nt * d; }

// G equal parts of U, the first U % G one longer: where part c starts, and the part
// of place u. 64-bit divisions take hundreds of instructions, and U rarely needs them.
struct Parts {
  long long q, rest;
  __host__ __device__ Parts(long long U, int G) {
    if (U >> 31) {
      q = U / G;
      rest = U % G;
    } else {
      q = static_cast<uint32_t>(U) / static_cast<uint32_t>(G);
      rest = static_cast<uint32_t>(U) % static_cast<uint32_t>(G);
    }
  }
  __host__ __device__ long long start(int c) const { return c * q + (c < rest ? c : rest); }
  __host__ __device__ int of(long long u) const {
    const long long longer = rest * (q + 1);
    if ((u | q) >> 31) return static_cast<int>(u < longer ? u / (q + 1) : rest + (u - longer) / q);
    return static_cast<int>(u < longer ? static_cast<uint32_t>(u) / static_cast<uint32_t>(q + 1)
                                       : rest + static_cast<uint32_t>(u - longer) / static_cast<uint32_t>(q));
  }
};

__device__ __forceinline__ int token_of(const AttnArgs &a, int r) { return a.t == 1 ? 0 : r / a.group; }

// Where row r of a KV head's rows stands in q and out (in rows of head_dim), and in lse.
__device__ __forceinline__ size_t attn_row(const AttnArgs &a, int seq, int h, int r) {
  const int token = token_of(a, r);
  return (static_cast<size_t>(seq) * a.t + token) * a.hq + h * a.group + r - token * a.group;
}

// Of four scale bytes those that are no number: bit i of the result for byte i, which becomes 0.
// (A key that a row does not see has p = 0 there, but 0 times what is no number is none.)
__device__ __forceinline__ uint32_t take_nans(uint32_t &scales) {
  const uint32_t ones = ((scales & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u;
  scales &= ~(ones * 0xFFu);
  return ones * 0x01020408u >> 24;
}

__device__ __forceinline__ float row_lse(float base, float sum) {
  return sum == 0.0f ? -CUDART_INF_F : (base + log2f(sum)) * 0.693147180559945f;
}

__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  return bf16_store_bits(x) | static_cast<uint32_t>(bf16_store_bits(y)) << 16;
}

}  // namespace
}  // namespace sk
