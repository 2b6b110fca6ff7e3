// Attention over the 4-bit key/value cache (sk_attn_nvfp4) for many rows per KV head:
// several tokens at once, drafted or of a prompt.
#include "sk_attn.cuh"

namespace sk {
namespace {

__device__ uint32_t g_tile_status;  // OR of SK_DEVICE_WAIT_* bits

// 128 rows of a KV head at a time (group query heads times t tokens), with chunks of 128
// tokens; the products run on tcgen05, whose sums lie in tensor memory:
//   S [128 rows, 128 tokens] = Q [128 rows, d] K^T     both in shared memory
//   O [128 rows, d] += P [128 rows, 128 tokens] V      P in tensor memory, V^T in shared
// Eight warps widen codes to FP16 in shared memory (code times scale, exact), in the
// 128-byte swizzle that the products read; two groups of four warps make P of S, a thread
// per row, one the even chunks, one the odd, each with its own base, sum and O; one warp
// issues the products, one the copies. So P of two chunks is made while the next are
// multiplied and widened.
//
// Up to 64 rows lie there twice: each copy sees half of a chunk's tokens (P is 0
// elsewhere), has its own base and sum, and all threads have work. Copies and groups are
// added at the end of an item.
//
// The work is cut as in attn_kernel, in a part per CTA; the items of a tile of rows count
// for the chunks that any of its rows sees, so a prompt's first tiles are cheap.
//
// b16 of 8192 tokens, 128 query heads: d64, 64 rows 59 us (84 in tiles of 16 rows), d128, 64
// rows 79 (136), 128 rows 90 (261). A prompt of 2048 tokens behind 14,336, 64 query heads,
// d128: 926 us (4200). A chunk takes 1440 clocks with 64 rows of d64, 2010 with 128 of d128,
// of which the products take 770 and 1090 at their rate. What bounds it is latency: of the
// issue slots 39 to 42 % are used and of no pipe more than two fifths (in the long prompt 57 %,
// the tensor pipe 47 %), with four or five warps per scheduler that wait for tensor memory, for
// one another and for instructions.
constexpr int kTileRows = 128, kTileChunk = 128;
// An item's beginning and end count for so many chunks (64 query heads, a prompt of 4096
// tokens, d64: 317 us with 5, 292 with 6, 286 with 7, 290 with 8; 128, 4 tokens of 16 rows of
// 100 to 8192, window 4096, d64: 28.6, 27.7, 27.9, 28.7; before the kernels were parted by C).
constexpr int kTileCost = 7;
constexpr int kSoftWarps = 8, kWidenWarps = 8, kMmaWarp = kSoftWarps + kWidenWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kSoft = 32 * kSoftWarps, kSumStride = kSoft + 1;
constexpr int kTileThreads = 32 * (kCopyWarp + 1);
// The warp of the copies runs ahead of the others by what the ring holds and two chunks:
// the chunks whose pieces, and the items, that are remembered.
constexpr int kHave = 8, kItems = 16;
constexpr int kTileNt = kTileRows / 8;
constexpr float kMost = 32768.0f;  // 2^kTop

// Columns of tensor memory, of even and odd chunks: S, O and P, which with d128 takes the
// place of the S that it is made of.
constexpr uint32_t kCols = 512;
__device__ __forceinline__ constexpr uint32_t col_s(int b) { return 128 * b; }
template <int D>
__device__ __forceinline__ constexpr uint32_t col_o(int b) { return 256 + D * b; }
template <int D>
__device__ __forceinline__ constexpr uint32_t col_p(int b) { return D == 128 ? col_s(b) : 384 + 64 * b; }

struct TileKeys {
  int c0, c1;  // chunks [c0, c1) of a sequence that some row of the tile sees
  __device__ int cost() const { return c1 > c0 ? c1 - c0 + kTileCost : 0; }
};

// Rows [128 tile, 128 tile + 128) of a sequence of len >= 0.
__device__ __forceinline__ TileKeys tile_keys(const AttnArgs &a, int len, int tile) {
  const int r0 = tile * kTileRows, first = tile ? token_of(a, r0) : 0;
  const int last = tile + 1 == a.tiles ? a.t - 1 : token_of(a, r0 + kTileRows - 1);
  const int hi = min(max(len - a.t + last + 1, 0), a.width * a.ps);
  const int lo = a.window ? max(0, len - a.t + first + 1 - a.window) : 0;
  return {lo / kTileChunk, ceil_div(hi, kTileChunk)};
}

// The sequence of a pair of a sequence and a tile.
__device__ __forceinline__ int seq_of(const AttnArgs &a, int pair) { return a.tiles == 1 ? pair : pair / a.tiles; }

__device__ __forceinline__ int pair_cost(const AttnArgs &a, int pair, int len) {
  return tile_keys(a, max(len, 0), pair - seq_of(a, pair) * a.tiles).cost();
}

// A part's share of an item: chunks [from, from + 128 count), or none at the end of the
// part. All rows see what is in [all_lo, all_hi).
struct TileItem {
  int seq, tile, h, len, from, count, flags, first, all_lo, all_hi;
};

template <int D>
struct TileShared {
  static constexpr int kStageBytes = kTileChunk * D * 9 / 8;
  static constexpr int kStages = D == 128 ? 3 : 6;
  uint8_t k[2][kTileChunk * D * 2];  // [d / 64][128 tokens][64], swizzled
  uint8_t v[2][kTileChunk * D * 2];  // [2][d channels][64 tokens], swizzled
  // Sums of copies and groups on their way into one, 32 columns at a time: with d128 they
  // take Q's place, which the next item's then waits for.
  static constexpr bool kApart = D == 64;
  static constexpr int kSums = 4 * 32 * kSumStride;
  uint8_t q[kApart ? kTileRows * D * 2 : kSums];  // [d / 64][128 rows][64], swizzled
  uint8_t apart[kApart ? kSums : 16];
  uint8_t ring[kStages * kStageBytes];
  __device__ float *sums() { return reinterpret_cast<float *>(kApart ? apart : q); }
  float2 stat[kSoft];
  uint32_t top[kSoft];
  float out_f[kTileRows];        // what a row's sums are multiplied with
  long long out_at[kTileRows];   // where they go, -1: nowhere
  uint64_t ring_full[kStages], ring_empty[kStages], k_full[2], v_full[2], qk_done[2], pv_done[2], p_full[2];
  uint64_t q_full, soft, drained, item_full[kItems];
  TileItem item[kItems];
  int have[kHave];
  // There was a scale of V that is no number in a chunk that not all rows see: it is left out
  // of the product, which would bring it to all rows.
  int any_nans;
  uint32_t tmem;
};

// Untiled bulk copy global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

// Each thread of the warp reads 16 consecutive 32-bit columns of its lane of tensor memory;
// they are there after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(float (&v)[16]);
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, float (&v)[32]) {
  float(&x)[2][16] = reinterpret_cast<float(&)[2][16]>(v);
  tmem_ld_x16(taddr, x[0]);
  tmem_ld_x16(taddr + 16, x[1]);
  tmem_ld_wait(x[0]);
  tmem_ld_wait(x[1]);
}
// Names the registers, so that no use is scheduled before it.
__device__ __forceinline__ void tmem_ld_wait(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Instruction descriptor of kind::f16 with FP16 operands (0 at bits 7-9 and 10-12), FP32
// sums, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return 1u << 4 | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(m >> 4) << 24;
}

// D[tmem] (+)= A[tmem] B[smem]^T of the types in idesc, 16 of K (as tc_mma_bf16 is for A in shared memory).
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  tc_mma_bf16_tmem_a(d, a, b, idesc, accumulate);
}

// True for one lane of a whole warp. The compiler knows that it is one, and so takes the
// products' operands from uniform registers as they are (with lane == 0, about 100 clocks
// per product).
__device__ __forceinline__ bool one_lane() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Makes a row's sums O no number in the blocks of 16 columns of which it sees a V with such a
// scale, in chunks that not all rows see; [lo, hi) are the row's keys. Called where such scales
// were met, which is rare: out of line, and reads them again.
template <int D>
__device__ __noinline__ void put_nans(const AttnArgs &a, const volatile TileItem &t, int lo, int hi, uint32_t o_at) {
  const int end = min(t.from + kTileChunk * t.count, hi);
  uint32_t lost = 0;
  for (int at = max(t.from, lo); at < end; ++at) {
    const int chunk = at & -kTileChunk;
    if (chunk >= t.all_lo && chunk + kTileChunk <= t.all_hi) {
      at = chunk + kTileChunk - 1;
      continue;
    }
    const int page = a.table[static_cast<size_t>(t.seq) * a.width + at / a.ps];
    if (page < 0 || page >= a.pages) continue;
    const uint8_t *scales = a.cache + (static_cast<size_t>(page) * a.hk + t.h) * (a.ps * D * 9 / 8) +
                            a.ps * D + a.ps * (D / 16) + at % a.ps;
    for (int b = 0; b < D / 16; ++b) lost |= ((scales[b * a.ps] & 0x7F) == 0x7F) << b;
  }
#pragma unroll 1
  for (int b = 0; b < D / 16; ++b) {
    const bool none = lost >> b & 1;
    if (!__any_sync(kAll, none)) continue;
    float y[16];
    uint32_t z[16];
    tmem_ld_32x32b_x16(o_at + 16 * b, y);
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = none ? 0x7FFFFFFFu : __float_as_uint(y[i]);
    tmem_st_x16(o_at + 16 * b, z);
  }
  tmem_st_wait();
}

// C: how many times a row lies there.
template <int D, int C>
__global__ void __launch_bounds__(kTileThreads, 1) attn_tile_kernel(const __grid_constant__ AttnArgs a) {
  using Sh = TileShared<D>;
  constexpr int kStages = Sh::kStages;
  // Where a token's row of K and its column of V^T lie: its low bits are changed by those
  // above, which keeps the lanes that widen V on different banks.
  constexpr int kFlip = D == 128 ? 1 : 3;
  extern __shared__ uint8_t raw[];
  Sh &sh = *reinterpret_cast<Sh *>(raw + (1024 - (smem_u32(raw) & 1023)) % 1024);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, G = gridDim.x, me = blockIdx.x;
  if (threadIdx.x == 0) {
    sh.any_nans = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sh.ring_full[s]), 1);
      mbar_init(smem_u32(&sh.ring_empty[s]), kWidenWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), kWidenWarps);
      mbar_init(smem_u32(&sh.v_full[i]), D == 128 ? kWidenWarps : kWidenWarps / 2);
      mbar_init(smem_u32(&sh.qk_done[i]), 1);
      mbar_init(smem_u32(&sh.pv_done[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), kSoftWarps / 2);
    }
    mbar_init(smem_u32(&sh.q_full), kSoftWarps);
    mbar_init(smem_u32(&sh.soft), kSoftWarps);
    mbar_init(smem_u32(&sh.drained), 1);
    for (int i = 0; i < kItems; ++i) mbar_init(smem_u32(&sh.item_full[i]), 1);
    fence_barrier_init();
  }
  griddep_wait();
  // All of tensor memory: not before the kernels ahead are done, and before those behind
  // start, as either might hold a part of it and wait for the other.
  if (w == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), kCols);
    tmem_relinquish();
  }

  const int pairs = a.b * a.tiles;
  // This CTA's part [u, end) of all, and the pair it starts in, for the warp of the copies;
  // a lane for four pairs.
  long long u = 0, end = 0, at = 0;  // at: the place of u within its pair
  int pair = 0;
  Parts parts(0, 1);
  if (w == kCopyWarp) {
    auto find = [&](auto zero) {  // in 32 bits where the sum of all fits
      using T = decltype(zero);
      auto cost_of4 = [&](int p, T(&cost)[4]) {
        int len[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) len[k] = p + k < pairs ? a.lens[seq_of(a, p + k)] : 0;
        T sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          cost[k] = p + k < pairs ? static_cast<T>(pair_cost(a, p + k, len[k])) * a.hk : 0;
          sum += cost[k];
        }
        return sum;
      };
      T U = 0, cost[4], mine = 0;
      for (int p = 4 * lane; p < pairs; p += 128) U += mine = cost_of4(p, cost);
#pragma unroll
      for (int d = 16; d; d >>= 1) U += __shfl_xor_sync(kAll, U, d);
      parts = Parts(U, G);
      u = parts.start(me);
      end = parts.start(me + 1);
      if (u >= end) return;
      const T from = static_cast<T>(u);
      T before = 0;
      for (int base = 0; base < pairs; base += 128) {
        if (pairs > 128) mine = cost_of4(base + 4 * lane, cost);  // else still at hand
        T upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const T o = __shfl_up_sync(kAll, upto, d);
          if (lane >= d) upto += o;
        }
        const uint32_t behind = __ballot_sync(kAll, before + upto > from);
        if (behind) {
          T off = from - before - (upto - mine);  // from this lane's first pair
          int p = base + 4 * lane;
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (p == base + 4 * lane + k && off >= cost[k]) {
              off -= cost[k];
              ++p;
            }
          pair = __shfl_sync(kAll, p, __ffs(behind) - 1);
          at = __shfl_sync(kAll, off, __ffs(behind) - 1);
          return;
        }
        before += __shfl_sync(kAll, upto, 31);
      }
      u = end;  // lengths that somebody changes meanwhile are no reason to search on
    };
    if (a.small) find(0);
    else find(0ll);
  }

  // Tiles of which nothing is seen, and no item to join yet.
  if (threadIdx.x == 0) a.joins[me] = make_int2(-1, 0);
  for (int p = w * G + me; w < kMmaWarp && p < pairs; p += G * kMmaWarp) {
    if (pair_cost(a, p, a.lens[seq_of(a, p)])) continue;
    const int seq = p / a.tiles, r0 = p % a.tiles * kTileRows, rows = min(kTileRows, a.rows - r0);
    for (int h = 0; h < a.hk; ++h)
      for (int i = lane; i < rows * (D / 8); i += 32) {
        const size_t row = attn_row(a, seq, h, r0 + i / (D / 8));
        reinterpret_cast<uint4 *>(a.out + row * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
        if (a.lse && i % (D / 8) == 0) a.lse[row] = -CUDART_INF_F;
      }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  griddep_launch_dependents();
  const uint32_t tmem = sh.tmem;

  // A wait of a whole warp, bounded: whoever waits in vain says so and leaves.
  auto wait = [&](uint64_t &bar, int parity, uint32_t bit) {
    if (__all_sync(kAll, mbar_wait_bounded(smem_u32(&bar), parity & 1, kCacheWaitNs))) return true;
    if (lane == 0) atomicOr(&g_tile_status, bit);
    return false;
  };
  auto arrive = [&](uint64_t &bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
  };

  const int ps_bits = 31 - __clz(a.ps), blk = a.ps * D * 9 / 8, pieces = kTileChunk / a.ps, codes = a.ps * (D / 2);
  const int most = a.width * a.ps;  // tokens that the table has places for
  // Item i of the part, as the warp of the copies has it.
  auto item = [&](int i) -> volatile TileItem & { return sh.item[i % kItems]; };
  auto comes = [&](int i) { return wait(sh.item_full[i % kItems], i / kItems, SK_DEVICE_WAIT_PRODUCER); };
  int n = 0;  // chunks so far
  bool good = true;

  if (w < kSoftWarps) {
    // ------------------------------------------------- P of S, a thread per row
    const int g = w >> 2, m = threadIdx.x & 127, R = kTileRows / C, rt = m & (R - 1);
    const int s0 = m / R * (8 / C), s1 = s0 + 8 / C;  // this copy's tokens, 16 at a time
    const uint32_t mine = tmem + (static_cast<uint32_t>(32 * (w & 3)) << 16);
    const uint32_t s_at = mine + col_s(g), p_at = mine + col_p<D>(g), o_at = mine + col_o<D>(g);
    const float c_all = __fmul_rn(a.scale, 1.44269504088896f) / *a.k_gs;
    // P of the tokens that are the other copy's, which with d64 stays 0
    auto hide_others = [&] {
      const uint32_t zero[8] = {};
      for (int s = 0; s < 8; ++s)
        if (s < s0 || s >= s1) tmem_st_x8(p_at + 8 * s, zero);
    };
    if (D == 64 && C > 1) hide_others();
    int soft = 0;
    auto together = [&] {  // the threads of all rows
      arrive(sh.soft);
      return wait(sh.soft, soft++, SK_DEVICE_WAIT_EPILOGUE);
    };
    // Queries as FP16, each row times a power of two that brings its largest value to
    // [2^14, 2^15): BF16's eight bits are exact in steps of 2^-24, down to 2^-31 of that value,
    // and off by at most 2^-25, 2^-39 of it, below. A negative scale changes their sign. Each
    // group takes half of the columns.
    uint4 half[D / 16];
    float c = 0.0f;  // what a score is multiplied with
    auto load_q = [&](const volatile TileItem &t) {
      const int r = t.tile * kTileRows + rt, token = r < a.rows ? token_of(a, r) : 0;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + (static_cast<size_t>(t.seq) * a.t + token) * a.q_stride + (t.h * a.group + r - token * a.group) * D);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) half[i] = r < a.rows ? src[g * (D / 16) + i] : make_uint4(0, 0, 0, 0);
    };
    auto put_q = [&] {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t x[4] = {half[i].x, half[i].y, half[i].z, half[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(x[k] & 0x7FFFu, x[k] >> 16 & 0x7FFFu));
      }
      sh.top[threadIdx.x] = top;
      if (!together()) return false;
      top = max(top, sh.top[threadIdx.x ^ 128]);
      const int shift = 14 - max(static_cast<int>(top >> 7) - 127, -126);
      // two factors, as 2^shift alone may not be an FP32 number
      const float f0 = copysignf(__uint_as_float((127 + shift / 2) << 23), c_all);
      const float f1 = __uint_as_float((127 + shift - shift / 2) << 23);
      c = fabsf(c_all) * __uint_as_float((127 - shift / 2) << 23) * __uint_as_float((127 - shift + shift / 2) << 23);
      // not 0, as that times the -inf of what is not seen is no number; S is below 2^34
      c = c < 1e-30f ? 1e-30f : c;
      auto two = [&](uint32_t x) {
        return cvt_f16x2(__uint_as_float(x << 16) * f0 * f1, __uint_as_float(x & 0xFFFF0000u) * f0 * f1);
      };
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int chunk = g * (D / 16) + i;  // 16 bytes of the row
        sts128(smem_u32(sh.q) + (chunk >> 3) * (kTileRows * 128) + m * 128 + (((chunk ^ m) & 7) << 4),
               make_uint4(two(half[i].x), two(half[i].y), two(half[i].z), two(half[i].w)));
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      arrive(sh.q_full);
      return true;
    };
    good = comes(0);
    if (good && item(0).count) {
      load_q(item(0));
      good = put_q();
    }
    for (int at_item = 0; good && item(at_item).count; ++at_item) {
      const volatile TileItem &t = item(at_item);
      const int r = t.tile * kTileRows + rt;
      const bool real = r < a.rows;
      int hi = real ? t.len - a.t + token_of(a, r) + 1 : 0;  // the tokens that the row sees
      const int lo = a.window ? hi - a.window : 0;
      float base = 0.0f, sum = 0.0f;  // the base with its sign changed
      bool unseen = hi > 0;           // without any key so far
      hi = min(hi, most);
      int done = -1;  // the last chunk of this group
      for (int i = (n ^ g) & 1; i < t.count; i += 2) {
        const int at_chunk = n + i, from = t.from + i * kTileChunk;
        if (!(good = wait(sh.qk_done[g], at_chunk >> 1, SK_DEVICE_WAIT_MMA))) break;
        tc_fence_after_sync();
        const int have = sh.have[at_chunk % kHave];
        const bool whole = have == (1 << pieces) - 1 && from + kTileChunk <= t.all_hi && from >= t.all_lo;
        // Scores of tokens that the row does not see are replaced where they lie; token i of 32
        // lies in column i ^ (i / 8 & kFlip).
        if (!whole) {
#pragma unroll 1
          for (int s = s0; s < s1; s += 2) {
            const int at = from + 16 * s, over = hi - at, under = lo - at;
            uint32_t ok = over >= 32 ? kAll : over <= 0 ? 0 : (1u << over) - 1;
            if (under > 0) ok &= under >= 32 ? 0 : kAll << under;
            if (!(have >> (16 * s >> ps_bits) & 1)) ok &= a.ps == 16 ? 0xFFFF0000u : 0;
            if (a.ps == 16 && !(have >> (s + 1) & 1)) ok &= 0xFFFFu;
            float x[32];
            tmem_ld_x32(s_at + 16 * s, x);
            uint32_t y[32];
#pragma unroll
            for (int k = 0; k < 32; ++k)
              y[k] = ok >> (k ^ (k >> 3 & kFlip)) & 1 ? __float_as_uint(x[k]) : 0xFF800000u;  // -inf
            tmem_st_32x32b_x32(s_at + 16 * s, y);
          }
          tmem_st_wait();
        }
        bool waited = false;
        auto free_p = [&] {  // the chunk before the last has been added to O, and its P read
          if (!waited && at_chunk >= 2) good = wait(sh.pv_done[g], (at_chunk >> 1) - 1, SK_DEVICE_WAIT_MMA);
          if (!waited) tc_fence_after_sync();
          waited = true;
        };
        // 64 columns at a time. It is assumed that the base need not move, and their P made again
        // if it has to, which the sums tell: no p is above 2^kTop if they are not.
        for (int s = s0; C == 1 ? s < s1 : s == s0; s += 4) {
          float sum0, sum1;
          uint32_t p[32];
          bool look = __any_sync(kAll, unseen);
          for (;;) {
            if (look) {
              float top = -CUDART_INF_F;
#pragma unroll 1
              for (int i = 0; i < 4; i += 2) {
                float x[32];
                tmem_ld_x32(s_at + 16 * (s + i), x);
#pragma unroll
                for (int k = 0; k < 32; k += 2) top = max3(top, x[k], x[k + 1]);
              }
              // the largest score, relative to the base, moves the base by a whole number, so
              // that a power of two takes all before along: P loses nothing that it has, and the
              // largest p is in [2^kAim, 2^(kAim + 1)) then
              top = top == -CUDART_INF_F ? top : fmaf(top, c, base);
              float by = top > kAim ? floorf(top - kAim) : 0.0f;
              float f = by < 127.0f ? __uint_as_float((127 - static_cast<int>(by)) << 23) : 0.0f;
              if (unseen) {  // the row's first keys set its base
                by = top == -CUDART_INF_F ? 0.0f : top - kAim;
                f = 1.0f;
                unseen = top == -CUDART_INF_F;
              }
              base -= by;
              sum *= f;
              if (__any_sync(kAll, f != 1.0f)) {
                free_p();
                tmem_st_wait();
#pragma unroll 1
                for (int k = 0; done >= 0 && k < D; k += 16) {
                  float y[16];
                  uint32_t z[16];
                  tmem_ld_32x32b_x16(o_at + k, y);
#pragma unroll
                  for (int i = 0; i < 16; ++i) z[i] = __float_as_uint(y[i] * f);
                  tmem_st_x16(o_at + k, z);
                }
#pragma unroll 1
                for (int k = 8 * s0; C == 1 && k < 8 * s; k += 16) {  // this chunk's
                  float y[16];
                  uint32_t z[16];
                  tmem_ld_32x32b_x16(p_at + k, y);
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const uint32_t two = __float_as_uint(y[i]);
                    z[i] = cvt_f16x2(__half2float(__ushort_as_half(two & 0xFFFFu)) * f,
                                     __half2float(__ushort_as_half(two >> 16)) * f);
                  }
                  tmem_st_x16(p_at + k, z);
                }
              }
            }
            sum0 = sum1 = 0.0f;
            auto make = [&](auto step, float(&x)[16]) {
#pragma unroll
              for (int k = 0; k < 16; k += 2) fma_f32x2(x[k], x[k + 1], c, c, base, base);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float y = ex2(x[k]), z = ex2(x[k + 1]);
                add_f32x2(sum0, sum1, y, z);
                p[8 * decltype(step)::value + k / 2] = cvt_f16x2(y, z);
              }
            };
            // 16 columns at a time, the next on their way meanwhile
            float x[16], y[16];
            tmem_ld_x16(s_at + 16 * s, x);
            tmem_ld_wait(x);
            tmem_ld_x16(s_at + 16 * s + 16, y);
            make(std::integral_constant<int, 0>(), x);
            tmem_ld_wait(y);
            tmem_ld_x16(s_at + 16 * s + 32, x);
            make(std::integral_constant<int, 1>(), y);
            tmem_ld_wait(x);
            tmem_ld_x16(s_at + 16 * s + 48, y);
            make(std::integral_constant<int, 2>(), x);
            tmem_ld_wait(y);
            make(std::integral_constant<int, 3>(), y);
            if (look || !__any_sync(kAll, !(sum0 <= kMost && sum1 <= kMost))) break;
            look = true;
          }
          free_p();
          tmem_st_32x32b_x32(p_at + 8 * s, p);  // at once; what it covers of S is read
          sum += sum0 + sum1;
        }
        if (D == 128 && C > 1) hide_others();
        tmem_st_wait();
        done = at_chunk;
        tc_fence_before_sync();
        arrive(sh.p_full[g]);
        if (!good) break;
      }
      n += t.count;
      // with d64 the next item's queries are put in place, and its S made, meanwhile
      if (good) good = comes(at_item + 1);
      const bool more = good && item(at_item + 1).count;
      if (more && Sh::kApart) {
        load_q(item(at_item + 1));
        // the products with the queries at hand are done
        good = wait(sh.qk_done[(n - 1) & 1], (n - 1) >> 1, SK_DEVICE_WAIT_MMA) &&
               (t.count < 2 || wait(sh.qk_done[n & 1], (n - 2) >> 1, SK_DEVICE_WAIT_MMA)) && put_q();
      }
      if (good && done >= 0) good = wait(sh.pv_done[g], done >> 1, SK_DEVICE_WAIT_EPILOGUE);
      if (!good) break;
      tc_fence_after_sync();
      if (__any_sync(kAll, *static_cast<volatile int *>(&sh.any_nans) && done >= 0)) put_nans<D>(a, t, lo, hi, o_at);

      // The whole item's output, or the result of a part: of one that the item began
      // before in slot 2 me, of one that it begins in in slot 2 me + 1.
      const bool whole = t.flags == (kBegins | kEnds);
      float *part = a.parts + (2 * static_cast<size_t>(me) + (t.flags & kBegins ? 1 : 0)) * attn_part_floats(D, kTileNt);
      const float own = sum == 0.0f ? -CUDART_INF_F : -base;
      sh.stat[threadIdx.x] = make_float2(own, sum);
      if (!(good = together())) break;
      float top = -CUDART_INF_F, l = 0.0f;
#pragma unroll
      for (int k = 0; k < 2 * C; ++k) top = fmaxf(top, sh.stat[rt + k * R].x);
#pragma unroll
      for (int k = 0; k < 2 * C; ++k) {
        const float2 x = sh.stat[rt + k * R];
        if (x.x != -CUDART_INF_F) l = fmaf(ex2(x.x - top), x.y, l);
      }
      const float f = own == -CUDART_INF_F ? 0.0f : ex2(own - top);
      if (threadIdx.x < R) {
        const size_t row = real ? attn_row(a, t.seq, t.h, r) : 0;
        if (real) {
          if (!whole) reinterpret_cast<float2 *>(part)[rt] = make_float2(top, l);
          else if (a.lse) a.lse[row] = row_lse(top, l);
        }
        sh.out_f[rt] = l == 0.0f ? 0.0f : 1.0f / *a.v_gs / l;
        sh.out_at[rt] = !real ? -1 : whole ? static_cast<long long>(row) * D : 2 * kTileRows + rt * D;
      }
      // Four channels of a row per thread, so that a warp writes runs of 128 bytes; channel
      // 8 i + k lies in column 8 i + (k ^ (i % 8)).
      auto put = [&](int b) {
        const int q4 = threadIdx.x & 7, i = q4 >> 1;
        for (int row = threadIdx.x >> 3; row < R; row += kSoft / 8) {
          float x[4] = {};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float *src = sh.sums() + (8 * i + ((4 * (q4 & 1) + k) ^ ((4 * b + i) & 7))) * kSumStride + row;
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) x[k] += src[j * R];
          }
          const long long to = sh.out_at[row];
          const float g = sh.out_f[row];
          if (to < 0) continue;
          if (whole)
            *reinterpret_cast<uint2 *>(a.out + to + 32 * b + 4 * q4) =
                make_uint2(bf16_pair(x[0] * g, x[1] * g), bf16_pair(x[2] * g, x[3] * g));
          else
            *reinterpret_cast<float4 *>(part + to + 32 * b + 4 * q4) = make_float4(x[0], x[1], x[2], x[3]);
        }
      };
      // (of a thread that saw no key O may hold anything; what is no number counts however small f is)
      for (int b = 0; good && b < D / 32; ++b) {
        __syncwarp();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float o[16];
          tmem_ld_32x32b_x16(o_at + 32 * b + 16 * s, o);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sh.sums()[(16 * s + i) * kSumStride + threadIdx.x] = own == -CUDART_INF_F ? 0.0f : o[i] * f;
        }
        if (!(good = together())) break;
        put(b);
        good = together();
      }
      tc_fence_before_sync();
      // the part that an item ends in says where it lies, for attn_join_kernel
      if (threadIdx.x == 0 && t.flags == kEnds) a.joins[me] = make_int2(t.first, (t.seq * a.tiles + t.tile) * a.hk + t.h);
      if (more && !Sh::kApart && good) {
        load_q(item(at_item + 1));
        good = put_q();
      }
    }
  } else if (w < kMmaWarp) {
    // -------------------------------------------------------------- K and V widened
    const int wid = w - kSoftWarps, id = 32 * wid + lane;
    const uint32_t ring = smem_u32(sh.ring);
    // K of chunk c: a lane takes 32 columns of a token, in 16-byte rows of 8.
    int k_slot = 0, k_round = 0;
    auto widen_k = [&](int c) {
      if (!wait(sh.ring_full[k_slot], k_round, SK_DEVICE_WAIT_PRODUCER)) return false;
      if (c >= 2 && !wait(sh.qk_done[c & 1], (c >> 1) - 1, SK_DEVICE_WAIT_MMA)) return false;
      const uint32_t stage = ring + k_slot * Sh::kStageBytes, k_to = smem_u32(sh.k[c & 1]);
#pragma unroll
      for (int it = 0; it < D / 64; ++it) {
        constexpr int kLanes = D / 32;  // of a token
        const int idx = it * 32 * kWidenWarps + id, part = idx % kLanes, token = idx / kLanes;
        const uint32_t src = stage + (token >> ps_bits) * blk, in = token & (a.ps - 1);
        const uint4 x = lds128(src + in * (D / 2) + 16 * part);
        const uint32_t two = widen_e4m3(lds16(src + 2 * codes + in * (D / 16) + 2 * part));
        const int s = token ^ (token >> 3 & kFlip);
        // with d128 the upper lanes begin with their second half, to be on other banks
        const int turn = D == 128 ? part & 2 : 0;
        const uint32_t f0 = __byte_perm(two, 0, turn ? 0x3232 : 0x1010), f1 = __byte_perm(two, 0, turn ? 0x1010 : 0x3232);
        const uint32_t q[4] = {turn ? x.z : x.x, turn ? x.w : x.y, turn ? x.x : x.z, turn ? x.y : x.w};
        const uint32_t row = k_to + (part >> 1) * (kTileChunk * 128) + s * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f = i < 2 ? f0 : f1;
          const int chunk = 4 * (part & 1) + (i ^ turn);
          sts128(row + ((chunk ^ (s & 7)) << 4),
                 make_uint4(mul_f16x2(widen_e2m1(q[i], 0), f), mul_f16x2(widen_e2m1(q[i], 1), f),
                            mul_f16x2(widen_e2m1(q[i], 2), f), mul_f16x2(widen_e2m1(q[i], 3), f)));
        }
      }
      fence_proxy_async_smem();
      arrive(sh.k_full[c & 1]);
      if (++k_slot == kStages) {
        k_slot = 0;
        ++k_round;
      }
      return true;
    };
    int slot = 0;
    good = comes(0) && (!item(0).count || widen_k(0));
    for (int at_item = 0; good && item(at_item).count; ++at_item) {
      const volatile TileItem &t = item(at_item);
      const int seen_hi = min(t.len, most), seen_lo = a.window ? t.len - a.t - a.window + 1 : 0;
      const int all_hi = t.all_hi, all_lo = t.all_lo;
      for (int from = t.from, to = from + kTileChunk * t.count; from < to; from += kTileChunk, ++n) {
        // K of the next chunk, of the next item's first after the last, goes before V
        const bool last = from + kTileChunk == to;
        if (last && !(good = comes(at_item + 1))) break;
        if ((!last || item(at_item + 1).count) && !(good = widen_k(n + 1))) break;
        const uint32_t stage = ring + slot * Sh::kStageBytes;
        // V: a lane takes 8 columns of 8 tokens; with d64 half the warps, in turn
        if (D == 128 || wid >> 2 == (n & 1)) {
          if (n >= 2 && !(good = wait(sh.pv_done[n & 1], (n >> 1) - 1, SK_DEVICE_WAIT_MMA))) break;
          constexpr int kLanes = D / 8;  // of a token
          const int wd = id % kLanes, tg = D == 128 ? id / kLanes : id % 128 / kLanes, flip = tg & kFlip;
          const int in = 8 * tg & (a.ps - 1), piece = 8 * tg >> ps_bits;
          const uint32_t src = stage + piece * blk + codes + in * (D / 2) + 4 * wd;
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = lds32(src + (i ^ flip) * (D / 2));
          uint2 sc = lds64(stage + piece * blk + 2 * codes + a.ps * (D / 16) + (wd >> 1) * a.ps + in);
          const int have = sh.have[n % kHave];
          const bool some = from + kTileChunk > all_hi || from < all_lo;  // rows do not see all
          if (have != (1 << pieces) - 1 || some) {
            // what is not seen weighs 0, but its scale may be no number
            const bool there = have >> piece & 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int at = from + 8 * tg + q;
              if (!there || at >= seen_hi || at < seen_lo) sc.x &= ~(0xFFu << 8 * q);
              if (!there || at + 4 >= seen_hi || at + 4 < seen_lo) sc.y &= ~(0xFFu << 8 * q);
            }
            if (some) {
              if (take_nans(sc.x) | take_nans(sc.y)) sh.any_nans = 1;
            }
          }
          const uint32_t order = flip == 0 ? 0x3210u : flip == 1 ? 0x2301u : flip == 2 ? 0x1032u : 0x0123u;
          sc.x = __byte_perm(sc.x, 0, order);
          sc.y = __byte_perm(sc.y, 0, order);
          const uint32_t f[4] = {widen_e4m3(sc.x & 0xFFFFu), widen_e4m3(sc.x >> 16), widen_e4m3(sc.y & 0xFFFFu),
                                 widen_e4m3(sc.y >> 16)};
          const uint32_t v_to = smem_u32(sh.v[n & 1]) + (tg >> 3) * (D * 128) + wd * 1024;
          const uint32_t turned = (wd & 7) << 7 | ((tg ^ wd) & 7) << 4;
#pragma unroll
          for (int par = 0; par < 2; ++par) {
            // bytes of (code of one token, code of the next)
            uint32_t both[4];
#pragma unroll
            for (int p = 0; p < 4; ++p)
              both[p] = par ? (v[2 * p] >> 4 & 0x0F0F0F0Fu) | (v[2 * p + 1] & 0xF0F0F0F0u)
                            : (v[2 * p] & 0x0F0F0F0Fu) | (v[2 * p + 1] << 4 & 0xF0F0F0F0u);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              sts128(v_to + (turned ^ (2 * y + par) * 144),
                     make_uint4(mul_f16x2(widen_e2m1(both[0], y), f[0]), mul_f16x2(widen_e2m1(both[1], y), f[1]),
                                mul_f16x2(widen_e2m1(both[2], y), f[2]), mul_f16x2(widen_e2m1(both[3], y), f[3])));
          }
          fence_proxy_async_smem();
          arrive(sh.v_full[n & 1]);
        }
        arrive(sh.ring_empty[slot]);
        if (++slot == kStages) slot = 0;
      }
    }
  } else if (w == kMmaWarp) {
    // ------------------------------------------------------------------ products
    constexpr uint32_t kQk = idesc_f16_f32(kTileRows, kTileChunk), kPv = idesc_f16_f32(kTileRows, D);
    auto qk = [&](int c) {  // S of chunk c
      const int b = c & 1;
      if (!wait(sh.k_full[b], c >> 1, SK_DEVICE_WAIT_MMA)) return false;
      tc_fence_after_sync();
      if (one_lane()) {
        const uint32_t q = smem_u32(sh.q), k = smem_u32(sh.k[b]);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          tc_mma_bf16(tmem + col_s(b), smem_desc_k128(q + s / 4 * (kTileRows * 128)) + 2 * (s % 4),
                      smem_desc_k128(k + s / 4 * (kTileChunk * 128)) + 2 * (s % 4), kQk, s > 0);
        tc_commit(smem_u32(&sh.qk_done[b]));
      }
      __syncwarp();
      return true;
    };
    for (int at_item = 0; (good = good && comes(at_item)) && item(at_item).count; ++at_item) {
      if (!(good = wait(sh.q_full, at_item, SK_DEVICE_WAIT_MMA))) break;
      const int count = item(at_item).count;
      for (int i = 0; good && i < min(count, 2); ++i) good = qk(n + i);
      for (int i = 0; good && i < count; ++i) {
        const int c = n + i, b = c & 1;
        if (!(good = wait(sh.p_full[b], c >> 1, SK_DEVICE_WAIT_MMA))) break;
        // S of the next chunk but one first, if P does not lie there
        if (D == 64 && i + 2 < count && !(good = qk(c + 2))) break;
        if (!(good = wait(sh.v_full[b], c >> 1, SK_DEVICE_WAIT_MMA))) break;
        tc_fence_after_sync();
        if (one_lane()) {
          const uint32_t v = smem_u32(sh.v[b]);
#pragma unroll
          for (int s = 0; s < kTileChunk / 16; ++s)
            mma_tmem_a(tmem + col_o<D>(b), tmem + col_p<D>(b) + 8 * s, smem_desc_k128(v + s / 4 * (D * 128)) + 2 * (s % 4),
                       kPv, i > 1 || s > 0);
          tc_commit(smem_u32(&sh.pv_done[b]));
        }
        __syncwarp();
        if (D == 128 && i + 2 < count)  // S takes P's place, whose product is waited for
          good = wait(sh.pv_done[b], c >> 1, SK_DEVICE_WAIT_MMA) && qk(c + 2);
      }
      n += count;
    }
    // nothing is in flight when tensor memory is given back
    if (one_lane()) tc_commit(smem_u32(&sh.drained));
    __syncwarp();
    wait(sh.drained, 0, SK_DEVICE_WAIT_MMA);
  } else {
    // -------------------------------------------------------------------- copies
    const uint32_t ring = smem_u32(sh.ring);
    int slot = 0, round = 0, items = 0;
    auto publish = [&](const TileItem &t) {
      if (lane == 0) {
        sh.item[items % kItems] = t;
        mbar_arrive(smem_u32(&sh.item_full[items % kItems]));
      }
      ++items;
    };
    // The items: pairs of a sequence and a tile, and of each the KV heads.
    while (good && u < end && pair < pairs) {
      const int seq = seq_of(a, pair), tile = pair - seq * a.tiles, len = max(a.lens[seq], 0);
      const TileKeys keys = tile_keys(a, len, tile);
      const int cost = keys.cost();
      if (at >= static_cast<long long>(cost) * a.hk) {
        at = 0;
        ++pair;
        continue;
      }
      const int h = at >> 31 ? static_cast<int>(at / cost) : static_cast<int>(at) / cost;
      // of its cost, [x, x + take) is this part's; the first kTileCost are no chunks
      const int x = static_cast<int>(at - static_cast<long long>(h) * cost);
      const int take = static_cast<int>(min(static_cast<long long>(cost - x), end - u));
      const int from_chunk = max(x - kTileCost, 0), count = x + take - kTileCost - from_chunk;
      const bool ends = x + take == cost;
      const long long begun = u - x + kTileCost;
      u += take;
      at += take;
      if (count <= 0) continue;
      const int from = (keys.c0 + from_chunk) * kTileChunk, to = from + count * kTileChunk;
      const int r0 = tile * kTileRows, begin = len - a.t + 1;  // behind the first token
      publish({seq, tile, h, len, from, count, (from_chunk ? 0 : kBegins) | (ends ? kEnds : 0),
               from_chunk && ends ? parts.of(begun) : me,
               a.window ? begin + token_of(a, min(r0 + kTileRows, a.rows) - 1) - a.window : 0,
               min(begin + token_of(a, r0), most)});
      // queries on their way to L2
      for (int i = lane; i < min(kTileRows, a.rows - r0) * (D / 64); i += 32) {
        const int r = r0 + i / (D / 64), token = token_of(a, r);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + (static_cast<size_t>(seq) * a.t + token) * a.q_stride +
                                                      (h * a.group + r - token * a.group) * D + i % (D / 64) * 64));
      }
      auto page_of = [&](int chunk) {
        const int token = chunk + lane * a.ps;
        return chunk < to && lane < pieces && token < len && token < most
                   ? a.table[static_cast<size_t>(seq) * a.width + (token >> ps_bits)]
                   : -1;
      };
      int page = page_of(from);
      for (int chunk = from; chunk < to; chunk += kTileChunk, ++n) {
        const int next = page_of(chunk + kTileChunk);
        if (round && !(good = wait(sh.ring_empty[slot], round - 1, SK_DEVICE_WAIT_PRODUCER))) break;
        const bool real = page >= 0 && page < a.pages;
        const uint32_t mask = __ballot_sync(kAll, real), bar = smem_u32(&sh.ring_full[slot]);
        if (lane == 0) {
          sh.have[n % kHave] = static_cast<int>(mask);
          mbar_arrive_expect_tx(bar, __popc(mask) * blk);
        }
        __syncwarp();
        if (real) {
          const uint32_t dst = ring + slot * Sh::kStageBytes + lane * blk;
          const uint8_t *src = a.cache + (static_cast<size_t>(page) * a.hk + h) * blk;
          if (a.tiles == 1) bulk_load_once(dst, src, blk, bar);
          else bulk_load(dst, src, blk, bar);  // other tiles read it too
        }
        page = next;
        if (++slot == kStages) {
          slot = 0;
          ++round;
        }
      }
    }
    publish({});
    if (!good)  // the copies in flight
      for (int i = max(n - kStages, 0); i < n; ++i)
        mbar_wait_bounded(smem_u32(&sh.ring_full[i % kStages]), i / kStages & 1, kCacheWaitNs);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (w == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kCols);
  }
}

template <int D>
constexpr int tile_smem() {
  return static_cast<int>(sizeof(TileShared<D>)) + 1024;
}

}  // namespace

int attn_tile_nt() { return kTileNt; }

cudaError_t launch_attn_tile(AttnArgs a, int d, int sm_count, cudaStream_t stream, bool pdl, int *parts) {
  const long long most = static_cast<long long>(ceil_div(a.width * a.ps, kTileChunk) + kTileCost) * a.b * a.hk * a.tiles;
  const int grid = static_cast<int>(most < sm_count ? most : sm_count);
  a.small = most < (1ll << 31);
  *parts = grid;
  auto go = [&](auto kernel, int smem) {
    return launch(kernel, dim3(grid), dim3(kTileThreads), smem, stream, pdl, a);
  };
  if (d == 64) return a.rows <= 64 ? go(attn_tile_kernel<64, 2>, tile_smem<64>()) : go(attn_tile_kernel<64, 1>, tile_smem<64>());
  return a.rows <= 64 ? go(attn_tile_kernel<128, 2>, tile_smem<128>()) : go(attn_tile_kernel<128, 1>, tile_smem<128>());
}

cudaError_t attn_tile_setup() {
  auto set = [](auto kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  cudaError_t e;
  if ((e = set(attn_tile_kernel<64, 1>, tile_smem<64>()))) return e;
  if ((e = set(attn_tile_kernel<64, 2>, tile_smem<64>()))) return e;
  if ((e = set(attn_tile_kernel<128, 1>, tile_smem<128>()))) return e;
  return set(attn_tile_kernel<128, 2>, tile_smem<128>());
}

cudaError_t read_tile_status(uint32_t *out, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_tile_status, sizeof(uint32_t));
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_tile_status, &zero, sizeof zero);
}

}  // namespace sk
