// C entry points of the key/value cache held in 4 bits: sk_kv_append,
// sk_attn_nvfp4, sk_kv_resize, sk_kv_fork and sk_kv_compact. Arguments are
// checked here, before any CUDA call; the kernels are in sk_cache.cu.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "sk.h"
#include "sk_internal.h"

namespace {

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

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

sk_status check_count(const char *name, long long v, long long most) {
  if (v < 1 || v > most) return fail(SK_ERR_INVALID_ARG, "%s=%lld: needs 1 <= %s <= %lld", name, v, name, most);
  return SK_OK;
}

sk_status check_block(int page_size, int head_dim) {
  if (page_size != 16 && page_size != 32 && page_size != 64)
    return fail(SK_ERR_INVALID_ARG, "page_size=%d: needs 16, 32 or 64 tokens", page_size);
  if (head_dim != 64 && head_dim != 128)
    return fail(SK_ERR_INVALID_ARG, "head_dim=%d: needs 64 or 128", head_dim);
  return SK_OK;
}

int block_bytes(int page_size, int head_dim) { return page_size * head_dim / 8 * 9; }

// The cache of a layer and what names its pages; 2^30 tokens keep positions within 31 bits.
sk_status check_cache(int rows, int most_rows, int pages, int width, int page_size) {
  sk_status st;
  if ((st = check_count("rows", rows, most_rows)) != SK_OK) return st;
  if ((st = check_count("pages", pages, 1 << 30)) != SK_OK) return st;
  if (width < 1 || width > (1 << 30) / page_size)
    return fail(SK_ERR_INVALID_ARG, "width=%d: needs 1 <= width <= %d pages in a row of the table", width,
                (1 << 30) / page_size);
  return SK_OK;
}

sk_status check_tokens(int b, int t, int kv_heads) {
  sk_status st;
  if ((st = check_count("b", b, 1 << 20)) != SK_OK) return st;
  if ((st = check_count("t", t, 1 << 24)) != SK_OK) return st;
  if ((st = check_count("kv_heads", kv_heads, 1024)) != SK_OK) return st;
  return check_count("b * t", static_cast<long long>(b) * t, 1 << 24);
}

sk_status check_stride(const char *name, long long stride, long long least) {
  if (stride < least || stride % 8)
    return fail(SK_ERR_INVALID_ARG, "%s=%lld: needs a multiple of 8 that is at least %lld", name, stride, least);
  return SK_OK;
}

sk_status check_attn(int b, int t, int q_heads, int kv_heads, int head_dim) {
  sk_status st;
  if ((st = check_block(64, head_dim)) != SK_OK) return st;
  if ((st = check_tokens(b, t, kv_heads)) != SK_OK) return st;
  if (q_heads < kv_heads || q_heads > 4096 || q_heads % kv_heads)
    return fail(SK_ERR_INVALID_ARG, "q_heads=%d: needs a multiple of kv_heads=%d, at most 4096", q_heads, kv_heads);
  // rows of all KV heads, in tiles of 8 at least: one CTA each
  return check_count("b * t * q_heads", static_cast<long long>(b) * t * q_heads, 1 << 30);
}

sk_status check_layers(int layers, int kv_heads, int page_size, int head_dim, int *page_bytes) {
  sk_status st;
  if ((st = check_block(page_size, head_dim)) != SK_OK) return st;
  if ((st = check_count("layers", layers, 1 << 16)) != SK_OK) return st;
  if ((st = check_count("kv_heads", kv_heads, 1024)) != SK_OK) return st;
  *page_bytes = kv_heads * block_bytes(page_size, head_dim);
  return SK_OK;
}

struct AttnWorkspace {
  int nt, tiles;
  size_t joins, parts, total;
};

AttnWorkspace attn_workspace(int b, int t, int q_heads, int kv_heads, int head_dim) {
  AttnWorkspace w;
  const int rows = q_heads / kv_heads * t;
  w.nt = sk::attn_row_tiles(rows);
  w.tiles = (rows + 8 * w.nt - 1) / (8 * w.nt);
  w.joins = 0;
  const size_t items = static_cast<size_t>(b) * kv_heads * w.tiles;
  w.parts = w.joins + round256(8 * sk::attn_joins(w.nt, items, SK_MAX_SMS));
  w.total = w.parts + round256(2 * sk::attn_max_parts(SK_MAX_SMS, w.nt) * sk::attn_part_bytes(head_dim, w.nt));
  return w;
}

struct ResizeWorkspace {
  size_t plan, copies, fresh, count, total;
};

ResizeWorkspace resize_workspace(int rows, int pages) {
  ResizeWorkspace w;
  w.plan = 0;
  w.copies = w.plan + round256(16 * static_cast<size_t>(rows));
  w.fresh = w.copies + round256(8 * static_cast<size_t>(rows));
  w.count = w.fresh + round256(4 * static_cast<size_t>(pages));
  w.total = w.count + 256;
  return w;
}

}  // namespace

extern "C" {

size_t sk_kv_block_bytes(int page_size, int head_dim) {
  if (check_block(page_size, head_dim) != SK_OK) return 0;
  ok();
  return block_bytes(page_size, head_dim);
}

sk_status sk_kv_append(const void *k, const void *v, const float *k_global_scale,
                       const float *v_global_scale, uint8_t *cache, const int32_t *table,
                       const int32_t *lens, int b, int t, int kv_heads, int head_dim, int page_size,
                       int pages, int width, int64_t k_stride, int64_t v_stride, void *stream) {
  return sk_kv_append_ex(k, v, k_global_scale, v_global_scale, cache, table, lens, nullptr, nullptr, b, t, kv_heads,
                         head_dim, page_size, pages, width, k_stride, v_stride, stream);
}

sk_status sk_kv_append_ex(const void *k, const void *v, const float *k_global_scale,
                          const float *v_global_scale, uint8_t *cache, const int32_t *table,
                          const int32_t *lens, const int32_t *new_lens, const int32_t *fresh, int b,
                          int t, int kv_heads, int head_dim, int page_size, int pages, int width,
                          int64_t k_stride, int64_t v_stride, void *stream) {
  sk_status st;
  if ((st = check_block(page_size, head_dim)) != SK_OK) return st;
  if ((st = check_tokens(b, t, kv_heads)) != SK_OK) return st;
  if ((st = check_cache(b, 1 << 20, pages, width, page_size)) != SK_OK) return st;
  if ((st = check_stride("k_stride", k_stride, static_cast<long long>(kv_heads) * head_dim)) != SK_OK) return st;
  if ((st = check_stride("v_stride", v_stride, static_cast<long long>(kv_heads) * head_dim)) != SK_OK) return st;
  if ((st = check_ptrs("sk_kv_append", 16, {{"k", k}, {"v", v}, {"cache", cache}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_kv_append", 4,
                       {{"k_global_scale", k_global_scale}, {"v_global_scale", v_global_scale},
                        {"table", table}, {"lens", lens}})) != SK_OK)
    return st;
  if (new_lens && (st = check_ptrs("sk_kv_append", 4, {{"new_lens", new_lens}})) != SK_OK) return st;
  if (fresh && (st = check_ptrs("sk_kv_append", 4, {{"fresh", fresh}})) != SK_OK) return st;
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  sk::AppendArgs a{static_cast<const uint16_t *>(k), static_cast<const uint16_t *>(v), k_global_scale,
                   v_global_scale, cache, table, lens, new_lens, fresh, b, t, kv_heads, head_dim, page_size, pages, width,
                   k_stride, v_stride, 1};
  return launch_status(sk::launch_kv_append(a, info.sm_count, as_stream(stream), sk::pdl_on()), "kv_append");
}

size_t sk_attn_nvfp4_workspace(int b, int t, int q_heads, int kv_heads, int head_dim) {
  if (check_attn(b, t, q_heads, kv_heads, head_dim) != SK_OK) return 0;
  ok();
  return attn_workspace(b, t, q_heads, kv_heads, head_dim).total;
}

sk_status sk_attn_nvfp4(const void *q, const float *k_global_scale, const float *v_global_scale,
                        const uint8_t *cache, const int32_t *table, const int32_t *lens, void *out,
                        float *lse, void *workspace, size_t workspace_bytes, int b, int t,
                        int q_heads, int kv_heads, int head_dim, int page_size, int pages, int width,
                        int64_t q_stride, float scale, int window, void *stream) {
  sk_status st;
  if ((st = check_attn(b, t, q_heads, kv_heads, head_dim)) != SK_OK) return st;
  if ((st = check_block(page_size, head_dim)) != SK_OK) return st;
  if ((st = check_cache(b, 1 << 20, pages, width, page_size)) != SK_OK) return st;
  if ((st = check_stride("q_stride", q_stride, static_cast<long long>(q_heads) * head_dim)) != SK_OK) return st;
  if (!std::isfinite(scale)) return fail(SK_ERR_INVALID_ARG, "scale=%g: needs a finite factor", scale);
  if (window < 0) return fail(SK_ERR_INVALID_ARG, "window=%d: needs 0 (none) or a number of keys", window);
  if ((st = check_ptrs("sk_attn_nvfp4", 16, {{"q", q}, {"cache", cache}, {"out", out}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_attn_nvfp4", 4,
                       {{"k_global_scale", k_global_scale}, {"v_global_scale", v_global_scale},
                        {"table", table}, {"lens", lens}})) != SK_OK)
    return st;
  if (lse && (st = check_ptrs("sk_attn_nvfp4", 4, {{"lse", lse}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_attn_nvfp4", 256, {{"workspace", workspace}})) != SK_OK) return st;
  const AttnWorkspace w = attn_workspace(b, t, q_heads, kv_heads, head_dim);
  if (workspace_bytes < w.total)
    return fail(SK_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, w.total);
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  const int group = q_heads / kv_heads;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  // a window beyond the last position hides nothing
  sk::AttnArgs a{static_cast<const uint16_t *>(q), cache, k_global_scale, v_global_scale, table, lens,
                 static_cast<uint16_t *>(out), lse, reinterpret_cast<int2 *>(ws + w.joins),
                 reinterpret_cast<float *>(ws + w.parts), b, t, q_heads, kv_heads, page_size, pages,
                 width, window > (1 << 30) ? 0 : window, group, group * t, w.tiles, q_stride, scale, false};
  const int sms = info.sm_count < SK_MAX_SMS ? info.sm_count : SK_MAX_SMS;
  return launch_status(sk::launch_attn(a, head_dim, sms, as_stream(stream), sk::pdl_on()), "attn_nvfp4");
}

size_t sk_kv_resize_workspace(int rows, int pages) {
  if (check_cache(rows, SK_MAX_CACHE_ROWS, pages, 1, 16) != SK_OK) return 0;
  ok();
  return resize_workspace(rows, pages).total;
}

sk_status sk_kv_resize(const int32_t *new_lens, uint8_t *cache, int32_t *table, int32_t *lens,
                       int32_t *refs, int32_t *status, void *workspace, size_t workspace_bytes,
                       int rows, int width, int pages, int layers, int kv_heads, int head_dim,
                       int page_size, void *stream) {
  sk_status st;
  int page_bytes = 0;
  if ((st = check_layers(layers, kv_heads, page_size, head_dim, &page_bytes)) != SK_OK) return st;
  if ((st = check_cache(rows, SK_MAX_CACHE_ROWS, pages, width, page_size)) != SK_OK) return st;
  if ((st = check_ptrs("sk_kv_resize", 16, {{"cache", cache}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_kv_resize", 4,
                       {{"new_lens", new_lens}, {"table", table}, {"lens", lens}, {"refs", refs},
                        {"status", status}})) != SK_OK)
    return st;
  if ((st = check_ptrs("sk_kv_resize", 256, {{"workspace", workspace}})) != SK_OK) return st;
  const ResizeWorkspace w = resize_workspace(rows, pages);
  if (workspace_bytes < w.total)
    return fail(SK_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, w.total);
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  sk::ResizeArgs a{new_lens, cache, table, lens, refs, status, rows, width, pages, page_size, layers,
                   page_bytes, static_cast<size_t>(pages) * page_bytes,
                   (reinterpret_cast<uintptr_t>(refs) & 15) == 0, reinterpret_cast<int4 *>(ws + w.plan),
                   reinterpret_cast<int2 *>(ws + w.copies), reinterpret_cast<int32_t *>(ws + w.fresh),
                   reinterpret_cast<int32_t *>(ws + w.count)};
  return launch_status(sk::launch_kv_resize(a, info.sm_count, as_stream(stream), sk::pdl_on()), "kv_resize");
}

sk_status sk_kv_fork(const int32_t *parents, int32_t *table, int32_t *lens, int32_t *refs,
                     int32_t *status, int rows, int width, int pages, int page_size, void *stream) {
  sk_status st;
  if ((st = check_block(page_size, 64)) != SK_OK) return st;
  if ((st = check_cache(rows, SK_MAX_CACHE_ROWS, pages, width, page_size)) != SK_OK) return st;
  if ((st = check_ptrs("sk_kv_fork", 4,
                       {{"parents", parents}, {"table", table}, {"lens", lens}, {"refs", refs},
                        {"status", status}})) != SK_OK)
    return st;
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  sk::ForkArgs a{parents, table, lens, refs, status, rows, width, pages, page_size};
  return launch_status(sk::launch_kv_fork(a, as_stream(stream), sk::pdl_on()), "kv_fork");
}

size_t sk_kv_compact_workspace(int pages) {
  if (check_count("pages", pages, 1 << 30) != SK_OK) return 0;
  ok();
  return 2 * round256(4 * static_cast<size_t>(pages)) + 256;
}

sk_status sk_kv_compact(uint8_t *cache, int32_t *table, const int32_t *lens, int32_t *refs,
                        int32_t *page_map, void *workspace, size_t workspace_bytes, int rows,
                        int width, int pages, int layers, int kv_heads, int head_dim, int page_size,
                        void *stream) {
  sk_status st;
  int page_bytes = 0;
  if ((st = check_layers(layers, kv_heads, page_size, head_dim, &page_bytes)) != SK_OK) return st;
  if ((st = check_cache(rows, SK_MAX_CACHE_ROWS, pages, width, page_size)) != SK_OK) return st;
  if ((st = check_ptrs("sk_kv_compact", 16, {{"cache", cache}})) != SK_OK) return st;
  if ((st = check_ptrs("sk_kv_compact", 4,
                       {{"table", table}, {"lens", lens}, {"refs", refs}, {"page_map", page_map}})) != SK_OK)
    return st;
  if ((st = check_ptrs("sk_kv_compact", 256, {{"workspace", workspace}})) != SK_OK) return st;
  const size_t need = sk_kv_compact_workspace(pages);
  if (workspace_bytes < need)
    return fail(SK_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
  sk::DeviceInfo info;
  int dev = 0;
  if ((st = sk::checked_device(&info, &dev)) != SK_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const size_t list = round256(4 * static_cast<size_t>(pages));
  sk::CompactArgs a{cache, table, lens, refs, page_map, rows, width, pages, page_size, layers, page_bytes,
                    static_cast<size_t>(pages) * page_bytes, (reinterpret_cast<uintptr_t>(refs) & 15) == 0,
                    (reinterpret_cast<uintptr_t>(page_map) & 15) == 0, reinterpret_cast<int32_t *>(ws),
                    reinterpret_cast<int32_t *>(ws + list), reinterpret_cast<int32_t *>(ws + 2 * list)};
  return launch_status(sk::launch_kv_compact(a, info.sm_count, as_stream(stream), sk::pdl_on()), "kv_compact");
}

}  // extern "C"
