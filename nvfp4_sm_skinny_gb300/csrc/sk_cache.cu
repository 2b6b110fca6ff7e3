// Device code of the key/value cache held in 4 bits: appending to it
// (sk_kv_append), attention over it (sk_attn_nvfp4) and its pages
// (sk_kv_resize, sk_kv_fork, sk_kv_compact). include/sk.h has the formulas and
// the cache's layout.
#include "sk_attn.cuh"

namespace sk {
namespace {

__device__ uint32_t g_cache_status;                // OR of SK_DEVICE_WAIT_* bits
// The transpose of an 8 x 8 matrix of 16-bit values, row l / 4, columns 2 (l % 4)
// and the next in lane l's register.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// ---------------------------------------------------------------- attention
// out = sum_k p_k v_k / sum_k p_k, p = exp(scale q . k - max): one pass over the
// keys with a running maximum and sum.
//
// A warp works by itself on chunks of 64 tokens of one KV head, which bulk copies
// bring into its own ring in shared memory (a block of the cache is one run of
// bytes). Codes are widened in registers into operands of the tensor instruction (16 x
// 8 x 16): one conversion and one product with the scale per pair, both exact in FP16.
// The rows of a KV head, group query heads times t tokens, are taken 8 or 16 at a time,
// and every code is widened once for them:
//   8 rows:   S^T [16 tokens, 8 rows] = K [16 tokens, d] Q^T
//   16 rows:  S [16 rows, 8 tokens] = Q [16 rows, d] K^T, for two sets of tokens
//   O^T [16 channels, 8 rows] += V^T [16 channels, 16 tokens] P^T, for 8 rows each
// What S holds is P^T's operand as it stands with 16 rows, transposed with 8.
// The order of an inner product is free, so lanes take what lies together in
// memory: of K, lane (g, j) of the instruction (g = lane / 4, j = lane % 4) the j-th
// quarter of a token's d columns; of V, the g-th eighth of the columns of the 16
// tokens [16 j, 16 j + 16). Row r = 2 j + e + 8 h of token tile mt is therefore
// token 16 j + 4 mt + ((2 h + e) ^ f(j)); f = 0, 2, 1, 3 keeps the lanes of a
// shared-memory access apart.
//
// The work is cut evenly whatever the lengths: the chunks of an item (a sequence, a
// KV head, a tile of rows), item after item, in as many equal parts as the GPU holds
// warps, an item's beginning counting like kItemCost chunks more. An item that falls
// into several parts is joined by attn_join_kernel, in the order of its tokens. Warps
// share nothing, and a CTA is all that fit on an SM: three CTAs of four did not always
// fit beside the last CTAs of the kernel before (b64 d128, 5400 tokens on average:
// 114 us, 85 where the kernel ran alone), and four warps that join their sums in
// shared memory item by item waited for one another (93 us).
constexpr int kChunk = 64;
constexpr int kItemCost = 3;
constexpr int kAttnWarps = 12;  // of a CTA: their sums and queries fill the registers

template <int D, int NT>
struct AttnWarp {
  static constexpr int kStageBytes = kChunk * D * 9 / 8;
  static constexpr int kStages = D == 128 ? 2 : 4;
  alignas(256) uint8_t ring[kStages * kStageBytes];
  uint64_t full[kStages];
  // What the loop over chunks does not need, kept here as registers are short (b16 of
  // 8192 tokens, d128, 16 rows: 63 us with them).
  struct Place {
    long long u, end, at;
    int seq, item, flags, first, h, r0;  // first: the part that the item begins in
  } place;
};

struct Keys {
  int c0, c1;  // chunks [c0, c1) of a sequence that some of its tokens see
  // what an item of the sequence counts for
  __device__ int cost() const { return c1 > c0 ? c1 - c0 + kItemCost : 0; }
};

__device__ __forceinline__ Keys keys_of(const AttnArgs &a, int len) {
  Keys k;
  const int hi = min(max(len, 0), a.width * a.ps);
  const int lo = a.window ? max(0, len - a.t - a.window + 1) : 0;
  k.c0 = lo / kChunk;
  k.c1 = ceil_div(hi, kChunk);
  return k;
}

// What four sequences from s on count for, with all their items.
template <typename T>
__device__ __forceinline__ T cost_of4(const AttnArgs &a, int s, T (&n)[4]) {
  int len[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) len[k] = s + k < a.b ? a.lens[s + k] : 0;
  T sum = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    n[k] = static_cast<T>(keys_of(a, len[k]).cost()) * (a.hk * a.tiles);
    sum += n[k];
  }
  return sum;
}

// Bits i of 32 tokens from `token` on that lie in [lo, hi).
__device__ __forceinline__ uint32_t tokens_in(int token, int lo, int hi) {
  const int over = hi - token, under = lo - token;
  const uint32_t below = over >= 32 ? kAll : over <= 0 ? 0 : (1u << over) - 1;
  return under >= 32 ? 0 : under > 0 ? below & kAll << under : below;
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * kAttnWarps, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
  using Sh = AttnWarp<D, NT>;
  constexpr int kMt = D / 16, kSub = NT == 2 ? 2 : 4, kSteps = D / 16;
  constexpr bool kWide = NT == 2;       // 16 rows: they are the instruction's M in Q K^T
  constexpr int R = kWide ? 1 : 2;      // rows per N tile whose statistics a lane holds
  extern __shared__ __align__(128) uint8_t raw[];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  Sh &sh = reinterpret_cast<Sh *>(raw)[w];
  griddep_launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < Sh::kStages; ++s) mbar_init(smem_u32(&sh.full[s]), 1);
    fence_barrier_init();
  }
  griddep_wait();

  // This warp's part [u, end) of all, and the sequence it starts in. Few parts go to
  // different SMs.
  const int per = a.hk * a.tiles, G = gridDim.x * kAttnWarps;
  const int me = w * gridDim.x + blockIdx.x;
  long long u, end, at = 0;  // at: the place of u within its sequence
  int seq = 0;
  Parts parts(0, 1);
  // A warp finds its part by itself, a lane for four sequences, in 32 bits where the sum
  // of all fits.
  auto find = [&](auto zero) {
    using T = decltype(zero);
    T U = 0, n[4], mine = 0;
    for (int s = 4 * lane; s < a.b; s += 128) U += mine = cost_of4(a, s, n);
#pragma unroll
    for (int d = 16; d; d >>= 1) U += __shfl_xor_sync(kAll, U, d);
    parts = Parts(U, G);
    u = parts.start(me);
    end = parts.start(me + 1);
    if (u >= end) return;
    const T from = static_cast<T>(u);
    T before = 0;
    for (int base = 0; base < a.b; base += 128) {
      if (a.b > 128) mine = cost_of4(a, base + 4 * lane, n);  // else still at hand
      T upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += o;
      }
      const uint32_t behind = __ballot_sync(kAll, before + upto > from);
      if (behind) {
        T off = from - before - (upto - mine);  // from this lane's first sequence
        int s = base + 4 * lane;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (s == base + 4 * lane + k && off >= n[k]) {
            off -= n[k];
            ++s;
          }
        seq = __shfl_sync(kAll, s, __ffs(behind) - 1);
        at = __shfl_sync(kAll, off, __ffs(behind) - 1);
        return;
      }
      before += __shfl_sync(kAll, upto, 31);
    }
    u = end;  // lengths that somebody changes meanwhile are no reason to search on
  };
  if (a.small) find(0);
  else find(0ll);

  // Sequences of which nothing is seen.
  for (int s = me; s < a.b; s += G) {
    if (keys_of(a, a.lens[s]).cost()) continue;
    uint4 *o = reinterpret_cast<uint4 *>(a.out + static_cast<size_t>(s) * a.t * a.hq * D);
    const long long rows = static_cast<long long>(a.t) * a.hq;
    for (long long i = lane; i < rows * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    for (long long i = lane; a.lse && i < rows; i += 32) a.lse[s * rows + i] = -CUDART_INF_F;
    for (int i = lane; i < per; i += 32) a.joins[static_cast<size_t>(s) * per + i] = make_int2(0, -1);
  }
  if (u >= end) return;

  // Row e of those of N tile nt that this lane holds statistics of.
  auto row_at = [&](int nt, int e) { return 8 * nt + (kWide ? g : 2 * j + e); };

  // Places of this lane's values within a chunk, whose tokens [16 i, 16 i + 16) lie in
  // piece 16 i / ps: of K and its scales for row h = 0, of V for e = h = 0. The others
  // differ in the bits of the token alone, which no other term has: they follow by
  // exclusive or, where more addresses would take more registers.
  const int ps_bits = 31 - __clz(a.ps);
  const int blk = a.ps * D * 9 / 8, pieces = kChunk / a.ps, codes = a.ps * (D / 2);
  const int gj = g >> 1, ge = g & 1;
  const int fk = (gj & 1) << 1 | gj >> 1, fv = (j & 1) << 1 | j >> 1;
  const int k_piece = 16 * gj / a.ps * blk, k_in = 16 * gj % a.ps;
  const int v_piece = 16 * j / a.ps * blk, v_in = 16 * j % a.ps;
  const int k_at = k_piece + (k_in + (ge ^ fk)) * (D / 2) + j * (D / 8);
  const int ks_at = k_piece + 2 * codes + (k_in + (ge ^ fk)) * (D / 16) + j * (D / 64);
  const int v_at = v_piece + codes + (v_in + fv) * (D / 2) + g * (D / 16);
  const int vs_at = v_piece + 2 * codes + a.ps * (D / 16) + (D == 128 ? g : g >> 1) * a.ps + v_in;
  const uint32_t vs_order = fv == 0 ? 0x3210u : fv == 1 ? 0x2301u : fv == 2 ? 0x1032u : 0x0123u;
  uint8_t *const ring = sh.ring;

  int slot = 0, phase = 0;  // the next stage to consume
  int held = 0;             // 4 bits per stage: the pieces that it holds

  while (u < end) {
    const int len = a.lens[seq];
    const Keys keys = keys_of(a, len);
    const int cost = keys.cost();
    if (at >= static_cast<long long>(cost) * per) {
      at = 0;
      if (++seq >= a.b) break;  // as above
      continue;
    }
    const int item = at >> 31 ? static_cast<int>(at / cost) : static_cast<int>(at) / cost;
    // of its cost, [x, x + take) is this part's; the first kItemCost are no chunks
    const int x = static_cast<int>(at - static_cast<long long>(item) * cost);
    const int take = static_cast<int>(min(static_cast<long long>(cost - x), end - u));
    const int from_chunk = max(x - kItemCost, 0), count = x + take - kItemCost - from_chunk;
    __syncwarp();  // the last item's is read
    if (count > 0 && lane == 0)
      sh.place = {u + take, end, at + take, seq, item, (from_chunk ? 0 : kBegins) | (x + take == cost ? kEnds : 0),
                  from_chunk && x + take == cost ? parts.of(u - x + kItemCost) : me, item / a.tiles,
                  item % a.tiles * 8 * NT};
    __syncwarp();
    u += take;
    at += take;
    if (count <= 0) continue;
    const volatile typename Sh::Place &place = sh.place;
    int from = (keys.c0 + from_chunk) * kChunk;  // first token of the chunk at hand
    const int to = from + count * kChunk;

    // The page of this lane's piece of a chunk (-1: none), and the copy of a chunk.
    auto page_of = [&](int chunk) {
      const int token = chunk + lane * a.ps;
      return chunk < to && lane < pieces && token < len && token < a.width * a.ps
                 ? a.table[static_cast<size_t>(place.seq) * a.width + (token >> ps_bits)]
                 : -1;
    };
    auto issue = [&](int page, int s) {
      const bool real = page >= 0 && page < a.pages;
      const uint32_t bar = smem_u32(&sh.full[s]);
      const uint32_t mask = __ballot_sync(kAll, real);
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc(mask) * blk);
      __syncwarp();
      if (real)
        bulk_load_once(smem_u32(ring + s * Sh::kStageBytes + lane * blk),
                       a.cache + (static_cast<size_t>(page) * a.hk + place.h) * blk, blk, bar);
      held = (held & ~(15 << 4 * s)) | static_cast<int>(mask) << 4 * s;
    };
    // The first pages' numbers and the queries are on their way before the copies, which
    // would hold them up (b1 of 131,071 tokens: the queries came 5 us after the copies).
    int pages_at[Sh::kStages];
#pragma unroll
    for (int i = 0; i < Sh::kStages; ++i) pages_at[i] = page_of(from + i * kChunk);
    int page = page_of(from + Sh::kStages * kChunk);
    uint4 raw_q[NT][D / 32];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = place.r0 + 8 * nt + g;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw_q[nt][i] = make_uint4(0, 0, 0, 0);
      if (r < a.rows) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            a.q + (static_cast<size_t>(place.seq) * a.t + token_of(a, r)) * a.q_stride +
            (place.h * a.group + r - token_of(a, r) * a.group) * D + j * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw_q[nt][i] = src[i];
      }
    }
    const float c_all = __fmul_rn(a.scale, 1.44269504088896f) / *a.k_gs;
    int ahead = slot;  // the stage of the next copy
#pragma unroll
    for (int i = 0; i < Sh::kStages; ++i) {
      if (from + i * kChunk < to) {
        issue(pages_at[i], ahead);
        ahead = ahead + 1 == Sh::kStages ? 0 : ahead + 1;
      }
    }

    // one past the position of a row's token
    auto row_end = [&](int r) { return r < a.rows ? len - a.t + token_of(a, r) + 1 : 0; };

    // Queries as FP16, each row times a power of two that brings its largest value
    // to [2^14, 2^15): BF16's eight bits are exact in steps of 2^-24, down to 2^-31 of that
    // value, and off by at most 2^-25, 2^-39 of it, below. Lane (g, j) holds row g of each N
    // tile, the j-th quarter of the columns.
    uint32_t qf[NT][kSteps][2];
    float c[NT][R];       // what a score is multiplied with
    uint32_t unseen = 0;  // rows (bit R nt + e) without any key so far
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4(&v)[D / 32] = raw_q[nt];
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) most = max(most, max(x[q] & 0x7FFFu, x[q] >> 16 & 0x7FFFu));
      }
      most = max(most, __shfl_xor_sync(kAll, most, 1));
      most = max(most, __shfl_xor_sync(kAll, most, 2));
      const int shift = 14 - max(static_cast<int>(most >> 7) - 127, -126);
      // two factors, as 2^shift alone may not be an FP32 number
      const float f0 = __uint_as_float((127 + shift / 2) << 23), f1 = __uint_as_float((127 + shift - shift / 2) << 23);
      const float back = c_all * __uint_as_float((127 - shift / 2) << 23) * __uint_as_float((127 - shift + shift / 2) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          qf[nt][2 * i + q / 2][q & 1] =
              cvt_f16x2(__uint_as_float(x[q] << 16) * f0 * f1, __uint_as_float(x[q] & 0xFFFF0000u) * f0 * f1);
      }
#pragma unroll
      for (int e = 0; e < R; ++e) {
        c[nt][e] = kWide ? back : __shfl_sync(kAll, back, 4 * (2 * j + e));
        if (row_end(place.r0 + row_at(nt, e)) > 0) unseen |= 1u << (R * nt + e);
      }
    }

    float o[kMt][NT][4], base[NT][R];  // the base with its sign changed
    float sum[NT][2];                  // of rows 2 j and 2 j + 1, or of row g in two parts
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[i][nt][q] = 0.0f;
      base[nt][0] = base[nt][R - 1] = sum[nt][0] = sum[nt][1] = 0.0f;
    }

    for (; from < to; from += kChunk) {
      if (__any_sync(kAll, !mbar_wait_bounded(smem_u32(&sh.full[slot]), phase, kCacheWaitNs))) {
        // a copy never landed: wait for those in flight, within the same limit, and leave
        if (lane == 0) atomicOr(&g_cache_status, SK_DEVICE_WAIT_PRODUCER);
        for (int s = 0; s < Sh::kStages; ++s)
          mbar_wait_bounded(smem_u32(&sh.full[s]), phase ^ (s < slot), kCacheWaitNs);
        return;
      }
      const int stage = w * static_cast<int>(sizeof(Sh)) + slot * Sh::kStageBytes;  // within raw
      const int have = held >> 4 * slot & 15;
      // every token of the chunk is there and seen by every row
      const bool whole = have == (1 << pieces) - 1 && from + kChunk <= len - a.t + 1 &&
                         from + kChunk <= a.width * a.ps && (!a.window || from >= len - a.window);
#pragma unroll
      for (int part = 0; part < 4 / kSub; ++part) {
        float s[kSub][NT][4];
        const int k0_at = stage + k_at, s0_at = stage + ks_at;
#pragma unroll
        for (int m = 0; m < kSub; ++m) {
          const int mt = part * kSub + m;
          uint32_t k0[D / 32], k1[D / 32];
          uint32_t sc0[D / 64], sc1[D / 64];
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(raw + k0_at + mt * 4 * (D / 2));
            const uint4 y = *reinterpret_cast<const uint4 *>(raw + (k0_at ^ D) + mt * 4 * (D / 2));
            k0[0] = x.x, k0[1] = x.y, k0[2] = x.z, k0[3] = x.w;
            k1[0] = y.x, k1[1] = y.y, k1[2] = y.z, k1[3] = y.w;
            const uint32_t p = widen_e4m3(*reinterpret_cast<const uint16_t *>(raw + s0_at + mt * 4 * (D / 16)));
            const uint32_t q = widen_e4m3(*reinterpret_cast<const uint16_t *>(raw + (s0_at ^ D / 8) + mt * 4 * (D / 16)));
            sc0[0] = __byte_perm(p, 0, 0x1010), sc0[1] = __byte_perm(p, 0, 0x3232);
            sc1[0] = __byte_perm(q, 0, 0x1010), sc1[1] = __byte_perm(q, 0, 0x3232);
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(raw + k0_at + mt * 4 * (D / 2));
            const uint2 y = *reinterpret_cast<const uint2 *>(raw + (k0_at ^ D) + mt * 4 * (D / 2));
            k0[0] = x.x, k0[1] = x.y;
            k1[0] = y.x, k1[1] = y.y;
            sc0[0] = __byte_perm(widen_e4m3(raw[s0_at + mt * 4 * (D / 16)]), 0, 0x1010);
            sc1[0] = __byte_perm(widen_e4m3(raw[(s0_at ^ D / 8) + mt * 4 * (D / 16)]), 0, 0x1010);
          }
          float(&t)[NT][4] = s[m];
#pragma unroll
          for (int wd = 0; wd < D / 32; ++wd) {
            uint32_t x[4], y[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              x[q] = mul_f16x2(widen_e2m1(k0[wd], q), sc0[wd / 2]);
              y[q] = mul_f16x2(widen_e2m1(k1[wd], q), sc1[wd / 2]);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              auto go = [&](float &s0, float &s1, float &s2, float &s3, uint32_t a0, uint32_t a1, uint32_t a2,
                            uint32_t a3, uint32_t b0, uint32_t b1) {
                if (wd == 0 && q == 0) mma_f16_first(s0, s1, s2, s3, a0, a1, a2, a3, b0, b1);
                else mma_f16(s0, s1, s2, s3, a0, a1, a2, a3, b0, b1);
              };
              const int k = 2 * wd + q;
              if constexpr (kWide) {
                go(t[0][0], t[0][1], t[1][0], t[1][1], qf[0][k][0], qf[1][k][0], qf[0][k][1], qf[1][k][1], x[2 * q],
                   x[2 * q + 1]);
                go(t[0][2], t[0][3], t[1][2], t[1][3], qf[0][k][0], qf[1][k][0], qf[0][k][1], qf[1][k][1], y[2 * q],
                   y[2 * q + 1]);
              } else {
                go(t[0][0], t[0][1], t[0][2], t[0][3], x[2 * q], y[2 * q], x[2 * q + 1], y[2 * q + 1], qf[0][k][0],
                   qf[0][k][1]);
              }
            }
          }
        }

        // scores relative to the base of their row, as powers of two; s[m][nt][2 h + e] is
        // that of row 2 j + e with the token that row g + 8 h of tile m stands for, or if
        // wide, of row g with the token of row 2 j + e + 8 h
#pragma unroll
        for (int m = 0; m < kSub; ++m)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; q += 2)
              fma_f32x2(s[m][nt][q], s[m][nt][q + 1], c[nt][0], c[nt][R - 1], base[nt][0], base[nt][R - 1]);
        if (!whole) {
          const bool there = have >> (16 * (kWide ? j : gj) / a.ps) & 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int last = row_end(place.r0 + row_at(nt, e)), lo = a.window ? last - a.window : 0;
              const int hi = there ? min(last, a.width * a.ps) : 0;
#pragma unroll
              for (int m = 0; m < kSub; ++m)
#pragma unroll
                for (int half = 0; half < 4; half += 2) {
                  const int token = from + 4 * (part * kSub + m) +
                                    (kWide ? 16 * j + ((half + e) ^ fv) : 16 * gj + ((half + ge) ^ fk));
                  if (token >= hi || token < lo) s[m][nt][half + e] = -CUDART_INF_F;
                }
            }
        }
        float most = -CUDART_INF_F;
#pragma unroll
        for (int m = 0; m < kSub; ++m)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; q += 2) most = max3(most, s[m][nt][q], s[m][nt][q + 1]);
        if (__any_sync(kAll, unseen != 0 || most > kTop)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int e = 0; e < R; ++e) {
              float x = -CUDART_INF_F;
#pragma unroll
              for (int m = 0; m < kSub; ++m) {
                x = max3(x, s[m][nt][e], s[m][nt][2 + e]);
                if (kWide) x = max3(x, s[m][nt][1], s[m][nt][3]);
              }
#pragma unroll
              for (int d = kWide ? 1 : 4; d < (kWide ? 4 : 32); d <<= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
              const uint32_t bit = 1u << (R * nt + e);
              float by = x > kAim ? x - kAim : 0.0f;
              f[e] = ex2(-by);
              if (unseen & bit) {  // the row's first keys set its base
                by = x == -CUDART_INF_F ? 0.0f : x - kAim;
                f[e] = 1.0f;
                if (x != -CUDART_INF_F) unseen &= ~bit;
              }
              base[nt][e] -= by;
              sum[nt][e] *= f[e];
              if (kWide) sum[nt][1] *= f[e];
#pragma unroll
              for (int m = 0; m < kSub; ++m)
#pragma unroll
                for (int q = e; q < 4; q += R) s[m][nt][q] -= by;
            }
            if (kWide) {  // O^T has rows 2 j and 2 j + 1 here
              f[1] = __shfl_sync(kAll, f[0], 4 * (2 * j + 1));
              f[0] = __shfl_sync(kAll, f[0], 4 * (2 * j));
            }
#pragma unroll
            for (int i = 0; i < kMt; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q) o[i][nt][q] *= f[q & 1];
          }
        }
        uint32_t p[kSub][NT][2];  // P^T: rows 2 j, 2 j + 1 (+ 8) of tile m by row g
#pragma unroll
        for (int m = 0; m < kSub; ++m)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = ex2(s[m][nt][2 * h]), y = ex2(s[m][nt][2 * h + 1]);
              add_f32x2(sum[nt][0], sum[nt][1], x, y);
              p[m][nt][h] = kWide ? cvt_f16x2(x, y) : transpose8(cvt_f16x2(x, y));
            }

        // this lane's scales of V for its 16 tokens, in the order of the rows
        uint32_t vs[kSub];
        if constexpr (kSub == 4) {
          const uint4 x = *reinterpret_cast<const uint4 *>(raw + stage + vs_at);
          vs[0] = x.x, vs[1] = x.y, vs[2] = x.z, vs[3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2 *>(raw + stage + vs_at + 8 * part);
          vs[0] = x.x, vs[1] = x.y;
        }
        if (!whole) {
          // What is not seen weighs 0, but its scale may be no number. One that only some rows
          // see is left out of the product, and makes the sums of these rows no number.
          const bool there = have >> (16 * j / a.ps) & 1;
          uint32_t nans = 0;
#pragma unroll
          for (int m = 0; m < kSub; ++m) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int token = from + 16 * j + 4 * (part * kSub + m) + q;
              if (!there || token >= len || token >= a.width * a.ps || (a.window && token <= len - a.t - a.window))
                vs[m] &= ~(0xFFu << 8 * q);
            }
            nans |= take_nans(vs[m]) << 4 * m;
          }
          if (__any_sync(kAll, nans != 0)) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {  // the tokens of the lanes that share this one's columns
              const uint32_t theirs = __shfl_sync(kAll, nans, (lane & ~3) | i);
              const int token = from + 16 * i + 4 * kSub * part;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int last = row_end(place.r0 + 8 * nt + 2 * j + e), lo = a.window ? last - a.window : 0;
                  if (theirs & tokens_in(token, lo, last)) {
#pragma unroll
                    for (int k = 0; k < kMt; ++k) o[k][nt][e] = o[k][nt][2 + e] = CUDART_NAN_F;
                  }
                }
            }
          }
        }
#pragma unroll
        for (int m = 0; m < kSub; ++m) {
          const int mt = part * kSub + m;
          const uint32_t order = __byte_perm(vs[m], 0, vs_order);
          const uint32_t f0 = widen_e4m3(order & 0xFFFFu), f1 = widen_e4m3(order >> 16);
          constexpr int kWords = D / 64;
          uint32_t v[4][kWords];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint8_t *src = raw + (stage + v_at ^ q * (D / 2)) + 4 * mt * (D / 2);
            if constexpr (D == 128) {
              const uint2 x = *reinterpret_cast<const uint2 *>(src);
              v[q][0] = x.x, v[q][1] = x.y;
            } else {
              v[q][0] = *reinterpret_cast<const uint32_t *>(src);
            }
          }
          // bytes of (code of one token, code of the next) for the even and odd columns
          auto even = [](uint32_t x, uint32_t y) { return (x & 0x0F0F0F0Fu) | (y << 4 & 0xF0F0F0F0u); };
          auto odd = [](uint32_t x, uint32_t y) { return (x >> 4 & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u); };
          // channel tiles i to i + 3, of their operand's four registers one in each word
          auto add_pv = [&](int i, const uint32_t(&both)[4]) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t x[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) x[q] = mul_f16x2(widen_e2m1(both[q], y), q & 2 ? f1 : f0);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float(&t)[4] = o[i + y][nt];
                mma_f16(t[0], t[1], t[2], t[3], x[0], x[1], x[2], x[3], p[m][nt][0], p[m][nt][1]);
              }
            }
          };
          if constexpr (D == 128) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t both[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                both[q] = half ? odd(v[q & 2][q & 1], v[(q & 2) + 1][q & 1]) : even(v[q & 2][q & 1], v[(q & 2) + 1][q & 1]);
              add_pv(4 * half, both);
            }
          } else {
            uint32_t both[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              both[q] = q & 1 ? odd(v[q & 2][0], v[(q & 2) + 1][0]) : even(v[q & 2][0], v[(q & 2) + 1][0]);
            add_pv(0, both);
          }
        }
      }
      __syncwarp();
      if (from + Sh::kStages * kChunk < to) {
        issue(page, slot);
        page = page_of(from + (Sh::kStages + 1) * kChunk);
      }
      if (++slot == Sh::kStages) {
        slot = 0;
        phase ^= 1;
      }
    }

    // The whole item's output, or the result of a part: of one that the item began
    // before in slot 2 me, of one that it begins in in slot 2 me + 1.
    u = place.u, end = place.end, at = place.at, seq = place.seq;
    const int now = place.item, flags = place.flags;
    const bool whole = flags == (kBegins | kEnds);
    const float v_inv = 1.0f / *a.v_gs;
    const int head = place.h, row0 = place.r0;
    float *part = a.parts + (2 * static_cast<size_t>(me) + (flags & kBegins ? 1 : 0)) * attn_part_floats(D, NT);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float l[2], top[2];  // of rows 2 j and 2 j + 1
      if constexpr (kWide) {
        float x = sum[nt][0] + sum[nt][1];
        x += __shfl_xor_sync(kAll, x, 1);
        x += __shfl_xor_sync(kAll, x, 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[e] = __shfl_sync(kAll, x, 4 * (2 * j + e));
          top[e] = -__shfl_sync(kAll, base[nt][0], 4 * (2 * j + e));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[e] = sum[nt][e];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(kAll, l[e], d);
          top[e] = -base[nt][e];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rt = 8 * nt + 2 * j + e, r = row0 + rt;
        if (r >= a.rows) continue;
        // a lane's channels: 16 of its own, or 8
        constexpr int C = D / 8;
        float v[C];
#pragma unroll
        for (int k = 0; k < C; ++k) {
          if constexpr (D == 128) v[k] = o[k % 8 / 2 + k % 2 * 4][nt][k / 8 * 2 + e];
          else v[k] = o[k / 2][nt][k % 2 * 2 + e];
        }
        if (whole) {
          const size_t row = attn_row(a, seq, head, r);
          const float f = l[e] == 0.0f ? 0.0f : v_inv / l[e];
          uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * D + C * g);
#pragma unroll
          for (int k = 0; k < C; k += 8)
            dst[k / 8] = make_uint4(bf16_pair(v[k] * f, v[k + 1] * f), bf16_pair(v[k + 2] * f, v[k + 3] * f),
                                    bf16_pair(v[k + 4] * f, v[k + 5] * f), bf16_pair(v[k + 6] * f, v[k + 7] * f));
          if (a.lse && g == 0) a.lse[row] = row_lse(top[e], l[e]);
        } else {
          float4 *dst = reinterpret_cast<float4 *>(part + 16 * NT + rt * D + C * g);
#pragma unroll
          for (int k = 0; k < C; k += 4) dst[k / 4] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          if (g == 0) reinterpret_cast<float2 *>(part)[rt] = make_float2(l[e] == 0.0f ? -CUDART_INF_F : top[e], l[e]);
        }
      }
    }
    // the part that an item ends in says where it lies, for attn_join_kernel
    if (lane == 0 && flags & kEnds)
      a.joins[static_cast<size_t>(seq) * per + now] = make_int2(place.first, whole ? -1 : me);
  }
}

// Joins the items that fell into several parts. S warps of a CTA take a row of an item
// together, so that each has few results, whose loads do not wait for one another (b64
// d128: 512 items of five results, with 16 warps on one row after another 25 us, a
// warp per row 5).
constexpr int kJoinWarps = 32;  // of a row, at most

template <int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const __grid_constant__ AttnArgs a, int S, int G) {
  constexpr int V = D / 32;  // neighbouring channels per lane
  constexpr int kBatch = 8;
  __shared__ float2 stat[kJoinWarps];
  __shared__ float sums[kJoinWarps][D];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = (blockDim.x >> 5) / S;
  griddep_launch_dependents();
  griddep_wait();
  // the parts that the item begins and ends in; with NT = 16 the part that an item of
  // several ends in says which it is and where it begins
  const int2 join = a.joins[blockIdx.x];
  const int p0 = join.x, ends = NT == 16 ? blockIdx.x : join.y;
  if (p0 < 0 || ends < p0 || ends >= G) return;
  const float v_inv = 1.0f / *a.v_gs;
  int seq, h, tile;
  if constexpr (NT == 16) {
    const int pair = join.y / a.hk;
    h = join.y % a.hk, seq = pair / a.tiles, tile = pair % a.tiles;
  } else {
    const int per = a.hk * a.tiles, item = blockIdx.x % per;
    seq = blockIdx.x / per, h = item / a.tiles, tile = item % a.tiles;
  }
  const int r0 = tile * 8 * NT, results = ends - p0 + 1;
  const int sub = w % S;
  const int rt = blockIdx.y * rows + w / S, r = r0 + rt;
  const bool mine = rt < 8 * NT && r < a.rows;
  float top = -CUDART_INF_F, l = 0.0f, acc[V] = {};
  for (int i0 = sub; mine && i0 < results; i0 += kBatch * S) {
    float2 st[kBatch];
    float v[kBatch][V];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * S;
      st[k] = make_float2(-CUDART_INF_F, 0.0f);
      if (i < results) {
        const float *p = a.parts + (2 * static_cast<size_t>(p0 + i) + (i == 0)) * attn_part_floats(D, NT);
        st[k] = reinterpret_cast<const float2 *>(p)[rt];
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(p + 16 * NT + rt * D + V * lane);
          v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(p + 16 * NT + rt * D + V * lane);
          v[k][0] = x.x, v[k][1] = x.y;
        }
      }
    }
    float most = top;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) most = fmaxf(most, st[k].x);
    const float f0 = top == -CUDART_INF_F ? 0.0f : ex2(top - most);
    l *= f0;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (st[k].x == -CUDART_INF_F) continue;
      const float f = ex2(st[k].x - most);
      l = fmaf(f, st[k].y, l);
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(f, v[k][c], acc[c]);
    }
    top = most;
  }
  if (S > 1) {
    if (lane == 0) stat[w] = make_float2(top, l);
#pragma unroll
    for (int c = 0; c < V; ++c) sums[w][V * lane + c] = acc[c];
    __syncthreads();
    if (sub == 0) {  // a lane per warp of the row weighs its sums
      const float2 x = lane < S ? stat[w + lane] : make_float2(-CUDART_INF_F, 0.0f);
      top = x.x;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
      const float f = x.x == -CUDART_INF_F ? 0.0f : ex2(x.x - top);
      l = f * x.y;
#pragma unroll
      for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(kAll, l, d);
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = 0.0f;
#pragma unroll 4
      for (int k = 0; k < S; ++k) {
        const float fk = __shfl_sync(kAll, f, k);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(fk, sums[w + k][V * lane + c], acc[c]);
      }
    }
  }
  if (mine && sub == 0) {
    const float f = l == 0.0f ? 0.0f : v_inv / l;
    const size_t row = attn_row(a, seq, h, r);
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + row * D + V * lane);
#pragma unroll
    for (int c = 0; c < V; c += 2) dst[c / 2] = bf16_pair(acc[c] * f, acc[c + 1] * f);
    if (a.lse && lane == 0) a.lse[row] = row_lse(top, l);
  }
}

// ------------------------------------------------------------------- append
// A thread takes 16 columns of a token's head, of K and of V. What a block of 16 costs is
// instructions (a thread per block with three IEEE divisions: 51 us for 32,768 tokens
// of 8 heads, d128, twice what its bytes take), so the divisions go. That by 6 is
// Markstein's: with y the FP32 number next to 1/6, q = a y is within a unit of a / 6, r = a - 6 q
// is exact in one fused step, and q + r y in another is a / 6 correctly rounded (1990,
// Computation of elementary functions on the IBM RISC System/6000 processor); every finite
// BF16 magnitude is tested. 1 / (scale / gs) is looked up by the scale's byte.
constexpr int kAppendThreads = 256;

struct AppendShared {
  float step[2][256];  // of K and V: what a scale byte's values are multiplied with
};

__device__ __forceinline__ void append_steps(AppendShared &sh, const AppendArgs &a) {
  for (int i = threadIdx.x; i < 512; i += kAppendThreads) {
    const float gs = i < 256 ? *a.k_gs : *a.v_gs, sf = cvt_e4m3_f32(i & 255);
    sh.step[i >> 8][i & 255] = sf == 0.0f ? 0.0f : __fdiv_rn(1.0f, __fmul_rn(sf, __fdiv_rn(1.0f, gs)));
  }
}

__device__ __forceinline__ void mul_f32x2(float &x, float &y, float c) {
  asm("{\n\t.reg .b64 v, c;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 c, {%2, %2};\n\t"
      "mul.rn.f32x2 v, v, c;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(c));
}

// Eight values to a word of e2m1 codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t codes_e2m1(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// As nvfp4_block16, with 1 / (scale / gs) from a table: the scale byte of 16 BF16 values,
// their codes in `packed`.
__device__ __forceinline__ uint32_t append_block(const uint4 &x, const uint4 &y, float gs, const float *step,
                                                 uint2 &packed) {
  const uint32_t z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %1;\n\tmax.bf16x2 %0, %0, t;\n\t}" : "+r"(most) : "r"(z[i]));
  const float amax = fmaxf(bf16_bits_to_f32(most & 0xFFFFu), __uint_as_float(most & 0xFFFF0000u));
  const float sixth = 0.166666666666666667f, q = amax * sixth;
  const float by6 = amax < CUDART_INF_F ? fmaf(fmaf(-6.0f, q, amax), sixth, q) : amax;
  const uint32_t sf = cvt_f32_e4m3(__fmul_rn(by6, gs));
  const float os = step[sf];
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(z[i] << 16);
    v[2 * i + 1] = __uint_as_float(z[i] & 0xFFFF0000u);
    mul_f32x2(v[2 * i], v[2 * i + 1], os);
  }
  packed = make_uint2(codes_e2m1(v), codes_e2m1(v + 8));
  return sf;
}

// A CTA takes a.tile tokens at a time, its threads as many of them at once as they hold
// whole; a thread keeps its place within a token.
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ AppendShared sh;
  griddep_launch_dependents();
  griddep_wait();
  const int ps_bits = 31 - __clz(a.ps), bits = a.d == 128 ? 3 : 2;
  const int blocks = 1 << bits, per = a.hk << bits;  // blocks of a token
  const int codes = a.ps * a.d / 2, scales = a.ps * blocks, blk = 2 * (codes + scales);
  const int tokens = a.b * a.t, most = a.width * a.ps;
  const int once = per < kAppendThreads ? kAppendThreads / per : 1;  // tokens at once
  const int in = threadIdx.x / per < once ? threadIdx.x / per : once;
  bool ready = false;
  const int first = blockIdx.x * a.tile, end = min(first + a.tile, tokens);
  for (int token = first + in, step = 0; first + step < end; step += once, token += once) {
    const bool mine = in < once && token < end;
    const int seq = mine ? token / a.t : 0;
    const int len = mine ? a.lens[seq] : 0, from_end = a.t - (token - seq * a.t);
    int pos = mine ? len - from_end : -1;
    // rows without the length that they were to have, and what is not among a row's fresh tokens
    if (mine && a.new_lens && (a.new_lens[seq] != len || len > most)) pos = -1;
    if (mine && a.fresh && a.fresh[seq] < from_end) pos = -1;
    int page = -1;
    if (pos >= 0 && pos < most) page = a.table[static_cast<size_t>(seq) * a.width + (pos >> ps_bits)];
    for (int r = threadIdx.x - in * per, more = 0; more < per; more += kAppendThreads, r += kAppendThreads) {
      const int h = r >> bits, block = r & (blocks - 1);
      uint4 x[2], y[2];
      if (mine && r < per) {
        const uint4 *k = reinterpret_cast<const uint4 *>(a.k + token * a.k_stride + h * a.d + 16 * block);
        const uint4 *v = reinterpret_cast<const uint4 *>(a.v + token * a.v_stride + h * a.d + 16 * block);
        x[0] = k[0], y[0] = k[1], x[1] = v[0], y[1] = v[1];
      }
      if (!ready) {  // the first values are on their way
        append_steps(sh, a);
        __syncthreads();
        ready = true;
      }
      if (!mine || r >= per || page < 0 || page >= a.pages) continue;
      uint8_t *base = a.cache + (static_cast<size_t>(page) * a.hk + h) * blk;
      const int at = pos & (a.ps - 1), code = at * (a.d / 2) + 8 * block;
      uint2 packed;
      uint32_t sf = append_block(x[0], y[0], *a.k_gs, sh.step[0], packed);
      *reinterpret_cast<uint2 *>(base + code) = packed;
      base[2 * codes + at * blocks + block] = static_cast<uint8_t>(sf);
      sf = append_block(x[1], y[1], *a.v_gs, sh.step[1], packed);
      *reinterpret_cast<uint2 *>(base + codes + code) = packed;
      base[2 * codes + scales + block * a.ps + at] = static_cast<uint8_t>(sf);
    }
  }
}

// -------------------------------------------------------------------- pages
constexpr int kPageThreads = 1024;

// Exclusive prefix sum over a CTA of kPageThreads threads; total in `all`.
template <typename T>
__device__ __forceinline__ T cta_scan(T v, T *warps, T &all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T upto = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) warps[w] = upto;
  __syncthreads();
  if (w == 0) {
    T x = warps[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T o = __shfl_up_sync(kAll, x, d);
      if (lane >= d) x += o;
    }
    warps[lane] = x;
  }
  __syncthreads();
  all = warps[31];
  const T before = upto - v + (w ? warps[w - 1] : 0);
  __syncthreads();
  return before;
}

// Which of pages [p, p + 16) are in use, and which there are. A scan of the CTA is a
// microsecond whatever it scans, so a thread takes 16 pages at a time.
constexpr int kPagesEach = 16;

__device__ __forceinline__ uint32_t pages_in_use(const int32_t *refs, int p, int pages, bool vectors, uint32_t &there) {
  int r[kPagesEach];
  if (vectors && p + kPagesEach <= pages) {
#pragma unroll
    for (int i = 0; i < kPagesEach; i += 4) {
      const int4 v = *reinterpret_cast<const int4 *>(refs + p + i);
      r[i] = v.x, r[i + 1] = v.y, r[i + 2] = v.z, r[i + 3] = v.w;
    }
    there = 0xFFFF;
  } else {
    there = 0;
#pragma unroll
    for (int i = 0; i < kPagesEach; ++i) {
      r[i] = p + i < pages ? refs[p + i] : 0;
      there |= (p + i < pages) << i;
    }
  }
  uint32_t used = 0;
#pragma unroll
  for (int i = 0; i < kPagesEach; ++i) used |= (r[i] > 0) << i;
  return used;
}

// What becomes of a row: its length before and after, the first of its fresh
// pages, and whether that one is a copy of its last page.
struct RowPlan {
  int old_len, new_len, first, copy;
};

struct ResizeShared {
  int need[SK_MAX_CACHE_ROWS];    // fresh pages of each row, then the sum before it
  int page[SK_MAX_CACHE_ROWS];    // rows that grow from a page that others hold too:
  int who[SK_MAX_CACHE_ROWS];     //   the page, the row,
  int before[SK_MAX_CACHE_ROWS];  //   the copying row before it (-1: none), -2: this one copies
  int warps[32];
  long long wide[32];
};

__global__ void __launch_bounds__(kPageThreads) kv_resize_plan_kernel(const __grid_constant__ ResizeArgs a) {
  extern __shared__ __align__(128) uint8_t raw[];
  ResizeShared &sh = *reinterpret_cast<ResizeShared *>(raw);
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  RowPlan *plan = reinterpret_cast<RowPlan *>(a.plan);
  const int most = a.width * a.ps;
  int sharers = 0, all;
  for (int base = 0; base < a.rows; base += kPageThreads) {
    const int row = base + tid;
    bool shared = false;
    int page = -1;
    if (row < a.rows) {
      const int old = a.lens[row], want = a.new_lens[row];
      const bool bad = old < 0 || old > most || want > most;
      const int next = bad || want < 0 ? old : want;
      const int have = bad ? 0 : ceil_div(old, a.ps);
      if (!bad && next > old && old % a.ps) {
        page = a.table[static_cast<size_t>(row) * a.width + have - 1];
        shared = page >= 0 && page < a.pages && a.refs[page] > 1;
      }
      sh.need[row] = !bad && next > old ? ceil_div(next, a.ps) - have : 0;
      a.status[row] = bad ? 2 : 0;
    }
    const int at = sharers + cta_scan<int>(shared, sh.warps, all);
    if (shared) {
      sh.page[at] = page;
      sh.who[at] = row;
    }
    sharers += all;
  }
  __syncthreads();
  // In the order of rows, who holds a page as its last keeps it; the others copy it.
  for (int i = tid; i < sharers; i += kPageThreads) {
    int rank = 0, latest = -1;
    for (int k = 0; k < i; ++k)
      if (sh.page[k] == sh.page[i]) {
        ++rank;
        latest = sh.who[k];
      }
    const bool copies = rank < a.refs[sh.page[i]] - 1;
    sh.before[i] = copies ? -2 : latest;
    if (copies) ++sh.need[sh.who[i]];
  }
  __syncthreads();
  // 4096 rows may ask for 2^26 pages each: summed in 64 bits. Where more than all pages are
  // taken by then, it does not matter how many more.
  long long total = 0, sum;
  for (int base = 0; base < a.rows; base += kPageThreads) {
    const int row = base + tid;
    const int need = row < a.rows ? sh.need[row] : 0;
    const long long at = total + cta_scan<long long>(need, sh.wide, sum);
    if (row < a.rows) plan[row] = {a.lens[row], need, static_cast<int>(min(at, a.pages + 1ll)), 0};
    total += sum;
  }
  // The free pages, lowest number first, as many as are needed.
  int got = 0;
  for (int base = 0; base < a.pages && got < total; base += kPagesEach * kPageThreads) {
    const int p = base + kPagesEach * tid;
    uint32_t there, free = pages_in_use(a.refs, p, a.pages, a.refs_vector, there);
    free = there & ~free;
    int at = got + cta_scan(__popc(free), sh.warps, all);
    for (; free && at < total; free &= free - 1) a.fresh[at++] = p + __ffs(free) - 1;
    got += all;
  }
  __syncthreads();
  // Rows whose pages are not there are refused, and one that was to keep a page
  // which a refused row before it still holds.
  for (int row = tid; row < a.rows; row += kPageThreads) {
    const RowPlan r = plan[row];
    const bool bad = a.status[row] != 0, refused = !bad && r.new_len > 0 && r.first + r.new_len > got;
    const int want = a.new_lens[row];
    if (refused) a.status[row] = 1;
    sh.need[row] = refused;
    plan[row] = {r.old_len, bad || refused || want < 0 ? r.old_len : want, r.first, 0};
  }
  __syncthreads();
  int copies = 0;
  for (int base = 0; base < sharers; base += kPageThreads) {
    const int i = base + tid;
    bool copy = false;
    if (i < sharers) {
      const int row = sh.who[i];
      copy = sh.before[i] == -2 && !sh.need[row];
      if (copy) plan[row].copy = 1;
      if (sh.before[i] >= 0 && sh.need[sh.before[i]]) {
        a.status[row] = 1;
        plan[row].new_len = plan[row].old_len;
      }
    }
    const int at = copies + cta_scan<int>(copy, sh.warps, all);
    if (copy) a.copies[at] = make_int2(sh.page[i], a.fresh[plan[sh.who[i]].first]);
    copies += all;
  }
  if (tid == 0) *a.count = copies;
}

// Copies pages (source, destination) of every layer: runs of page_bytes, in pieces
// of kCopyBytes spread over the grid.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyBytes = 16 * kCopyThreads * kCopyUnroll;

template <typename Pair>
__device__ __forceinline__ void copy_pages(uint8_t *cache, int layers, size_t layer_bytes, int page_bytes, int count,
                                           Pair pair) {
  const int pieces = ceil_div(page_bytes, kCopyBytes);
  const long long all = static_cast<long long>(count) * layers * pieces;
  for (long long i = blockIdx.x; i < all; i += gridDim.x) {
    const int2 move = pair(static_cast<int>(i / pieces / layers));
    uint8_t *layer = cache + static_cast<size_t>(i / pieces % layers) * layer_bytes;
    const int at = static_cast<int>(i % pieces) * kCopyBytes + 16 * threadIdx.x;
    const uint8_t *from = layer + static_cast<size_t>(move.x) * page_bytes;
    uint8_t *to = layer + static_cast<size_t>(move.y) * page_bytes;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k)
      if (at + k * 16 * kCopyThreads < page_bytes)
        v[k] = *reinterpret_cast<const uint4 *>(from + at + k * 16 * kCopyThreads);
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k)
      if (at + k * 16 * kCopyThreads < page_bytes)
        *reinterpret_cast<uint4 *>(to + at + k * 16 * kCopyThreads) = v[k];
  }
}

__global__ void __launch_bounds__(kCopyThreads) kv_resize_apply_kernel(const __grid_constant__ ResizeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const RowPlan *plan = reinterpret_cast<const RowPlan *>(a.plan);
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const RowPlan r = plan[row];
    if (r.new_len == r.old_len) continue;
    int32_t *table = a.table + static_cast<size_t>(row) * a.width;
    const int have = ceil_div(r.old_len, a.ps), after = ceil_div(r.new_len, a.ps);
    if (threadIdx.x == 0) {
      a.lens[row] = r.new_len;
      if (r.copy) {
        const int page = a.fresh[r.first];
        const int old = table[have - 1];
        if (old >= 0 && old < a.pages) atomicSub(a.refs + old, 1);
        a.refs[page] = 1;
        table[have - 1] = page;
      }
    }
    for (int c = have + threadIdx.x; c < after; c += kCopyThreads) {
      const int page = a.fresh[r.first + r.copy + c - have];
      table[c] = page;
      a.refs[page] = 1;
    }
    for (int c = after + threadIdx.x; c < have; c += kCopyThreads) {
      const int page = table[c];
      if (page >= 0 && page < a.pages) atomicSub(a.refs + page, 1);
      table[c] = -1;
    }
  }
  copy_pages(a.cache, a.layers, a.layer_bytes, a.page_bytes, *a.count, [&](int i) { return a.copies[i]; });
}

// A CTA takes four columns of the table, of all rows: what a row becomes depends on
// other rows in these columns alone, which it reads before it writes. A thread takes a
// row, whose four loads wait for nothing.
constexpr int kForkCols = 4;

__global__ void __launch_bounds__(kPageThreads) kv_fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ __align__(128) uint8_t raw[];
  int4 *old = reinterpret_cast<int4 *>(raw);  // [rows]; -1 where a row has no page
  griddep_launch_dependents();
  griddep_wait();
  const int c0 = blockIdx.x * kForkCols;
  for (int row = threadIdx.x; row < a.rows; row += kPageThreads) {
    const int32_t *t = a.table + static_cast<size_t>(row) * a.width + c0;
    int v[kForkCols];
#pragma unroll
    for (int c = 0; c < kForkCols; ++c) v[c] = c0 + c < a.width ? t[c] : -1;
    const int used = ceil_div(min(max(a.lens[row], 0), a.width * a.ps), a.ps) - c0;
    old[row] = make_int4(used > 0 ? v[0] : -1, used > 1 ? v[1] : -1, used > 2 ? v[2] : -1, used > 3 ? v[3] : -1);
  }
  __syncthreads();
  for (int row = threadIdx.x; row < a.rows; row += kPageThreads) {
    const int p = a.parents[row];
    if (p < 0 || p >= a.rows || p == row) continue;
    int32_t *t = a.table + static_cast<size_t>(row) * a.width + c0;
    const int4 gone = old[row], got = old[p];
    auto change = [&](int c, int from, int to) {
      if (c0 + c >= a.width) return;
      t[c] = to;
      if (from == to) return;
      if (from >= 0 && from < a.pages) atomicSub(a.refs + from, 1);
      if (to >= 0 && to < a.pages) atomicAdd(a.refs + to, 1);
    };
    change(0, gone.x, got.x);
    change(1, gone.y, got.y);
    change(2, gone.z, got.z);
    change(3, gone.w, got.w);
  }
}

// The lengths of forked rows, after their tables: one CTA, which reads all before it writes.
__global__ void __launch_bounds__(kPageThreads) kv_fork_lens_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int32_t old[SK_MAX_CACHE_ROWS];
  griddep_launch_dependents();
  griddep_wait();
  for (int row = threadIdx.x; row < a.rows; row += kPageThreads) old[row] = a.lens[row];
  __syncthreads();
  for (int row = threadIdx.x; row < a.rows; row += kPageThreads) {
    const int p = a.parents[row];
    a.status[row] = p >= a.rows ? 2 : 0;
    if (p >= 0 && p < a.rows && p != row) a.lens[row] = old[p];
  }
}

// Of L pages in use, those numbered L and up move to the free ones below L, k-th to
// k-th, so no page is both source and destination.
__global__ void __launch_bounds__(kPageThreads) kv_compact_plan_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ unsigned long long warps[32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  unsigned long long all, mine = 0;
  for (int p = kPagesEach * tid; p < a.pages; p += kPagesEach * kPageThreads) {
    uint32_t there;
    mine += __popc(pages_in_use(a.refs, p, a.pages, a.refs_vector, there));
  }
  cta_scan(mine, warps, all);
  const int used = static_cast<int>(all);
  unsigned long long sum = 0;  // holes in the low half, pages to move in the high one
  for (int base = 0; base < a.pages; base += kPagesEach * kPageThreads) {
    const int p = base + kPagesEach * tid;
    uint32_t there = 0, live = 0;
    if (p < a.pages) live = pages_in_use(a.refs, p, a.pages, a.refs_vector, there);
    const uint32_t below = used <= p ? 0 : used - p >= kPagesEach ? 0xFFFF : (1u << (used - p)) - 1;
    uint32_t holes = there & ~live & below, moves = live & ~below;
    const unsigned long long at =
        sum + cta_scan<unsigned long long>(__popc(holes) | static_cast<unsigned long long>(__popc(moves)) << 32, warps, all);
    sum += all;
    int h = static_cast<int>(at), m = static_cast<int>(at >> 32);
    for (; holes; holes &= holes - 1) a.holes[h++] = p + __ffs(holes) - 1;
    for (; moves; moves &= moves - 1) a.moves[m++] = p + __ffs(moves) - 1;
    if (there == 0xFFFF && a.map_vector) {
#pragma unroll
      for (int i = 0; i < kPagesEach; i += 4)
        *reinterpret_cast<int4 *>(a.page_map + p + i) =
            make_int4(live >> i & 1 ? p + i : -1, live >> i & 2 ? p + i + 1 : -1, live >> i & 4 ? p + i + 2 : -1,
                      live >> i & 8 ? p + i + 3 : -1);
    } else {
      for (int i = 0; i < kPagesEach; ++i)
        if (there >> i & 1) a.page_map[p + i] = live >> i & 1 ? p + i : -1;
    }
  }
  __syncthreads();
  const int moved = min(static_cast<int>(sum >> 32), static_cast<int>(sum));  // as many as there are holes
  for (int m = tid; m < moved; m += kPageThreads) a.page_map[a.moves[m]] = a.holes[m];
  if (tid == 0) *a.count = moved;
}

__global__ void __launch_bounds__(kCopyThreads) kv_compact_apply_kernel(const __grid_constant__ CompactArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int count = *a.count;
  const long long step = static_cast<long long>(gridDim.x) * kCopyThreads;
  const long long first = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x;
  for (long long m = first; m < count; m += step) {
    a.refs[a.holes[m]] = a.refs[a.moves[m]];
    a.refs[a.moves[m]] = 0;
  }
  const long long entries = static_cast<long long>(a.rows) * a.width;
  for (long long i = first; i < entries; i += step) {
    const int row = static_cast<int>(i / a.width), c = static_cast<int>(i % a.width);
    const int len = min(max(a.lens[row], 0), a.width * a.ps);
    if (c >= ceil_div(len, a.ps)) continue;
    const int page = a.table[i];
    if (page >= 0 && page < a.pages) a.table[i] = a.page_map[page];
  }
  copy_pages(a.cache, a.layers, a.layer_bytes, a.page_bytes, count,
             [&](int m) { return make_int2(a.moves[m], a.holes[m]); });
}

// Calls f with the attention kernels' instance for a head size and rows per tile.
template <typename F>
cudaError_t with_attn(int d, int nt, F f) {
  auto at = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (nt == 1) return f(std::integral_constant<int, D>(), std::integral_constant<int, 1>());
    return f(std::integral_constant<int, D>(), std::integral_constant<int, 2>());
  };
  return d == 64 ? at(std::integral_constant<int, 64>()) : at(std::integral_constant<int, 128>());
}

}  // namespace

// Tiles of 8 rows, or of 16: of 32 the sums alone take 128 registers (d128, b16 of 8192
// tokens, 32 rows: 121 us, in two tiles of 16, which read and widen all twice, 80). From
// 33 rows on attn_tile_kernel's 128 (b16 of 8192 tokens; d128, 32 rows: 76 us here, 78
// there; 64 rows: 136 and 81; d64, 32 rows: 49 and 56; 64 rows: 84 and 59).
int attn_row_tiles(int rows) { return rows <= 8 ? 1 : rows <= 32 ? 2 : attn_tile_nt(); }

size_t attn_part_bytes(int d, int nt) { return sizeof(float) * attn_part_floats(d, nt); }

int attn_max_parts(int sm_count, int nt) { return nt == attn_tile_nt() ? sm_count : kAttnWarps * sm_count; }

size_t attn_joins(int nt, size_t items, int sm_count) { return nt == attn_tile_nt() ? sm_count : items; }

cudaError_t launch_attn(AttnArgs a, int d, int sm_count, cudaStream_t stream, bool pdl) {
  const int nt = attn_row_tiles(a.rows);
  // Warps of a row: as many as take eight results each on average, or four where the
  // GPU holds them all at once (512 items of 16 rows: 32.7 us with four, 30.6 with
  // eight; b1 of 2048 tokens: 11.0 and 11.9).
  auto join = [&](auto kernel, long long joins, long long results, int G) {
    const int rows = a.rows < 8 * nt ? a.rows : 8 * nt;
    int S = 1;
    while (S < kJoinWarps && (8 * S < results || (4 * S < results && 2 * S * joins * rows <= 32 * sm_count))) S *= 2;
    const int warps = S > 8 ? S : rows * S < 8 ? rows * S : 8;
    return launch(kernel, dim3(static_cast<unsigned>(joins), ceil_div(rows * S, warps)), dim3(32 * warps), 0, stream,
                  pdl, a, S, G);
  };
  if (nt == attn_tile_nt()) {
    int parts = 0;
    cudaError_t e = launch_attn_tile(a, d, sm_count, stream, pdl, &parts);
    if (e != cudaSuccess) return e;
    const long long items = static_cast<long long>(a.b) * a.hk * a.tiles, results = parts / items + 2;
    return d == 64 ? join(attn_join_kernel<64, 16>, parts, results, parts)
                   : join(attn_join_kernel<128, 16>, parts, results, parts);
  }
  return with_attn(d, nt, [&](auto dim, auto tiles) {
    constexpr int D = decltype(dim)::value, NT = decltype(tiles)::value;
    // no more SMs than there can be chunks
    const long long items = static_cast<long long>(a.b) * a.hk * a.tiles;
    const long long chunks = ceil_div(a.width * a.ps, kChunk);  // of an item, at most
    a.small = (chunks + kItemCost) * items < (1ll << 31);
    const int grid = static_cast<int>((chunks + kItemCost) * items < sm_count ? (chunks + kItemCost) * items : sm_count);
    cudaError_t e = launch(attn_kernel<D, NT>, dim3(grid), dim3(32 * kAttnWarps),
                           kAttnWarps * sizeof(AttnWarp<D, NT>), stream, pdl, a);
    if (e != cudaSuccess) return e;
    const long long most = grid * kAttnWarps / items + 2;
    return join(attn_join_kernel<D, NT>, items, most < chunks ? most : chunks, grid * kAttnWarps);
  });
}

cudaError_t launch_kv_append(AppendArgs a, int sm_count, cudaStream_t stream, bool pdl) {
  // Four rounds of a CTA's threads per tile (32,768 tokens of 8 heads, d128: 32.3 us; two
  // 34.0, eight 35.3), or one token where that leaves SMs idle.
  const int per = a.hk * (a.d / 16), tokens = a.b * a.t;
  a.tile = 4 * kAppendThreads / per;
  if (a.tile < 1 || tokens / a.tile < sm_count) a.tile = 1;
  return launch(kv_append_kernel, dim3(ceil_div(tokens, a.tile)), dim3(kAppendThreads), 0, stream, pdl, a);
}

cudaError_t launch_kv_resize(const ResizeArgs &a, int sm_count, cudaStream_t stream, bool pdl) {
  cudaError_t e = launch(kv_resize_plan_kernel, dim3(1), dim3(kPageThreads), sizeof(ResizeShared), stream, pdl, a);
  if (e != cudaSuccess) return e;
  return launch(kv_resize_apply_kernel, dim3(4 * sm_count), dim3(kCopyThreads), 0, stream, pdl, a);
}

cudaError_t launch_kv_fork(const ForkArgs &a, cudaStream_t stream, bool pdl) {
  cudaError_t e = launch(kv_fork_kernel, dim3(ceil_div(a.width, kForkCols)), dim3(kPageThreads),
                         sizeof(int4) * a.rows, stream, pdl, a);
  if (e != cudaSuccess) return e;
  return launch(kv_fork_lens_kernel, dim3(1), dim3(kPageThreads), 0, stream, pdl, a);
}

cudaError_t launch_kv_compact(const CompactArgs &a, int sm_count, cudaStream_t stream, bool pdl) {
  cudaError_t e = launch(kv_compact_plan_kernel, dim3(1), dim3(kPageThreads), 0, stream, pdl, a);
  if (e != cudaSuccess) return e;
  return launch(kv_compact_apply_kernel, dim3(4 * sm_count), dim3(kCopyThreads), 0, stream, pdl, a);
}

cudaError_t cache_setup() {
  cudaError_t e = attn_tile_setup();
  if (e != cudaSuccess) return e;
  for (int d : {64, 128})
    for (int nt : {1, 2})
      if ((e = with_attn(d, nt, [&](auto dim, auto tiles) {
             constexpr int D = decltype(dim)::value, NT = decltype(tiles)::value;
             return cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kAttnWarps * sizeof(AttnWarp<D, NT>)));
           })))
        return e;
  if ((e = cudaFuncSetAttribute(kv_resize_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sizeof(ResizeShared)))))
    return e;
  return cudaFuncSetAttribute(kv_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(sizeof(int4) * SK_MAX_CACHE_ROWS));
}

cudaError_t read_cache_status(uint32_t *out, bool clear) {
  uint32_t tile = 0;
  cudaError_t e = read_tile_status(&tile, clear);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(out, g_cache_status, sizeof(uint32_t));
  *out |= tile;
  if (e != cudaSuccess || !clear) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_cache_status, &zero, sizeof zero);
}

}  // namespace sk
