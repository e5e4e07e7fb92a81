// kv4_api.cu -- C entry points of the 4-bit key/value cache: argument checks
// and launches.  Nothing here allocates or synchronises (ra_kv4_status does).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/ring_attn.h"
#include "kv4.h"
#include "ring_attn_internal.h"

namespace {

ra_status fail(ra_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return ra::set_last_error(st, buf);
}
ra_status cuda_fail(cudaError_t e, const char* what) { return fail(RA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Do `na` bytes at a and `nb` at b share any?  (Outputs that lie over what the call reads, or
// over one another, are refused: CTAs would read what others have written.)
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

constexpr size_t kHeader = 256;
constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int page_shift(int32_t page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

ra_status check_geometry(int64_t num_pages, int32_t page_size, int32_t Hkv, int32_t D) {
  if (D != 64 && D != 128 && D != 256) return fail(RA_ERR_UNSUPPORTED, "head_dim %d: 64, 128 or 256", D);
  if (page_shift(page_size) < 0) return fail(RA_ERR_UNSUPPORTED, "page_size %d: 16, 32, 64, 128 or 256", page_size);
  if (Hkv < 1 || Hkv > 4096) return fail(RA_ERR_INVALID_ARG, "num_kv_heads %d outside [1, 4096]", Hkv);
  if (num_pages < 1 || num_pages > (int64_t(1) << 30))
    return fail(RA_ERR_INVALID_ARG, "num_pages %lld outside [1, 2^30]", (long long)num_pages);
  return RA_OK;
}

ra_status check_cache(const ra_kv4_cache* c, ra::Kv4Cache* out) {
  if (!c) return fail(RA_ERR_INVALID_ARG, "cache is NULL");
  ra_status rs = check_geometry(c->num_pages, c->page_size, c->num_kv_heads, c->head_dim);
  if (rs != RA_OK) return rs;
  if (!c->pages || !aligned(c->pages, 16)) return fail(RA_ERR_INVALID_ARG, "pages must be a 16-byte aligned device pointer");
  *out = ra::Kv4Cache{reinterpret_cast<uint8_t*>(c->pages), c->num_pages, page_shift(c->page_size), c->num_kv_heads};
  return RA_OK;
}

size_t page_bytes(int32_t page_size, int32_t Hkv, int32_t D) {
  return (size_t)(page_size / ra::kKv4Tile) * ra::kv4_tile_bytes(D) * Hkv;
}

// Requests with at least this many rows (tokens x heads of a group) go to the
// tile kernel, where a call can have them.  Its time hardly depends on the rows
// up to 128 a request, the other's grows with each 24 (head_dim 256: 8) of them;
// over 131072 cached tokens in 8 requests (8 heads at head_dim 128 and 64, 2 at
// 256) they take, in us,
//    64 rows  179 / 117 / 100 (tiles), 150 /  98 / 100 (few rows)
//    80 rows  184 / 119 / 108 (tiles), 193 / 125 / 122 (few rows)
//    96 rows  185 / 121 / 116 (tiles), 193 / 125 / 144 (few rows)
//   128 rows  190 / 126 / 137 (tiles), 282 / 177 / 187 (few rows),
// in calls of one kind: in a call that has both, the few-rows kernel is sized for one
// token (few_rows below), and 60 requests of 5 tokens over 4096 take 157 us instead of 110.
constexpr int kTileMinRows = 96;
bool has_tiles(int32_t G, int32_t max_q_len) { return (int64_t)G * max_q_len >= kTileMinRows; }
// Rows that the other kernel's CTAs take: those of the longest request, or of
// one token where the tile kernel takes the long ones.
int64_t few_rows(int32_t G, int32_t max_q_len) {
  return has_tiles(G, max_q_len) ? G : (int64_t)G * max_q_len;
}

// SMs of the current device (a property of the hardware: asked once).
cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

struct AttnLayout {
  size_t tickets, partials, total;
};
// The counters lie in the same place for every variant, so that one workspace
// serves calls of different kinds in turn.
AttnLayout attn_layout(int32_t D, int32_t G, int32_t max_q_len) {
  const ra::Kv4AttnShape s = ra::kv4_attn_shape(D, few_rows(G, max_q_len), ra::kKv4MaxSms);
  size_t floats = (size_t)s.ctas * 2 * s.slot_floats;
  if (has_tiles(G, max_q_len)) floats = std::max(floats, (size_t)ra::kKv4MaxSms * 2 * ra::kv4_tile_slot_floats(D));
  AttnLayout l;
  l.tickets = kHeader;
  l.partials = align256(l.tickets + 3 * (size_t)ra::kKv4MaxCtas * sizeof(int32_t));
  l.total = align256(l.partials + floats * sizeof(float));
  return l;
}

}  // namespace

extern "C" {

ra_status ra_kv4_cache_bytes(int64_t num_pages, int32_t page_size, int32_t num_kv_heads, int32_t head_dim,
                             size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "NULL output");
  ra_status rs = check_geometry(num_pages, page_size, num_kv_heads, head_dim);
  if (rs != RA_OK) return rs;
  *bytes = (size_t)num_pages * page_bytes(page_size, num_kv_heads, head_dim);
  return RA_OK;
}

ra_status ra_kv4_tables(const int32_t* kv_lens, const int32_t* new_lens, int32_t num_requests, int32_t* block_table,
                        int32_t table_width, int64_t table_stride, int32_t page_size, int32_t* free_pages,
                        int32_t num_pages, const int32_t* free_count, int64_t num_slots, int32_t* kv_lens_out,
                        int32_t* cu_new, int64_t* slot_map, int32_t* positions, int32_t* free_count_out,
                        int32_t* status, void* stream) {
  if (num_requests < 1 || num_requests > ra::kKv4MaxRequests)
    return fail(RA_ERR_INVALID_ARG, "num_requests %d outside [1, %d]", num_requests, ra::kKv4MaxRequests);
  if (page_shift(page_size) < 0) return fail(RA_ERR_UNSUPPORTED, "page_size %d: 16, 32, 64, 128 or 256", page_size);
  if (table_width < 1 || table_stride < table_width)
    return fail(RA_ERR_INVALID_ARG, "table_width %d, table_stride %lld: need 1 <= width <= stride", table_width,
                (long long)table_stride);
  if (num_slots < 0 || num_slots > (int64_t(1) << 30))
    return fail(RA_ERR_INVALID_ARG, "num_slots %lld outside [0, 2^30]", (long long)num_slots);
  if (!kv_lens || !new_lens || !block_table || !kv_lens_out || !cu_new || !status ||
      (num_slots > 0 && (!slot_map || !positions)))
    return fail(RA_ERR_INVALID_ARG, "NULL pointer");
  if (free_pages && (!free_count || !free_count_out || num_pages < 1 || num_pages > (1 << 30)))
    return fail(RA_ERR_INVALID_ARG, "a free list needs free_count, free_count_out and num_pages in [1, 2^30]");
  const void* words[] = {kv_lens, new_lens, block_table, kv_lens_out, cu_new, status, positions, free_pages,
                         free_count, free_count_out};
  for (const void* w : words)
    if (!aligned(w, 4)) return fail(RA_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  if (!aligned(slot_map, 8)) return fail(RA_ERR_INVALID_ARG, "slot_map must be 8-byte aligned");
  // Arrays that are written, then those that are only read; an output may be the input
  // that it replaces.
  const size_t R4 = (size_t)num_requests * 4, table_bytes = ((size_t)(num_requests - 1) * table_stride + table_width) * 4;
  const struct { const void* at; size_t bytes; const char* name; } arrays[] = {
      {kv_lens_out, R4, "kv_lens_out"}, {cu_new, R4 + 4, "cu_new"}, {slot_map, (size_t)num_slots * 8, "slot_map"},
      {positions, (size_t)num_slots * 4, "positions"}, {free_count_out, 4, "free_count_out"}, {status, 4, "status"},
      {block_table, table_bytes, "block_table"}, {free_pages, (size_t)num_pages * 4, "free_pages"},
      {kv_lens, R4, "kv_lens"}, {new_lens, R4, "new_lens"}, {free_count, 4, "free_count"}};
  for (int i = 0; i < 8; ++i)
    for (int j = i + 1; j < 11; ++j) {
      if (arrays[i].at == arrays[j].at && ((i == 0 && j == 8) || (i == 4 && j == 10))) continue;
      if (overlap(arrays[i].at, arrays[i].bytes, arrays[j].at, arrays[j].bytes))
        return fail(RA_ERR_INVALID_ARG, "%s lies over %s (only kv_lens_out may be kv_lens, and free_count_out free_count)",
                    arrays[i].name, arrays[j].name);
    }
  ra::Kv4TablesParams p{kv_lens, new_lens, block_table, table_stride, table_width, num_requests,
                        page_shift(page_size), free_pages, num_pages, free_count, num_slots, kv_lens_out, cu_new,
                        slot_map, positions, free_count_out, status};
  const cudaError_t e = ra::launch_kv4_tables(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache tables launch");
}

static ra_status check_rows(const ra_kv4_cache* cache, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const int64_t* slot_map, int64_t T, ra::Kv4RowsParams* p) {
  ra_status rs = check_cache(cache, &p->cache);
  if (rs != RA_OK) return rs;
  if (T < 0 || T > (int64_t(1) << 31)) return fail(RA_ERR_INVALID_ARG, "num_tokens %lld outside [0, 2^31]", (long long)T);
  if (T > 0 && (!k || !v || !slot_map)) return fail(RA_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(RA_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
  if (!aligned(slot_map, 8)) return fail(RA_ERR_INVALID_ARG, "slot_map must be 8-byte aligned");
  const int64_t row = (int64_t)cache->num_kv_heads * cache->head_dim;
  if (T > 1 && (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8))
    return fail(RA_ERR_INVALID_ARG, "row strides %lld, %lld: multiples of 8 elements, at least %lld",
                (long long)k_stride, (long long)v_stride, (long long)row);
  p->slots = slot_map;
  p->T = T;
  return RA_OK;
}

ra_status ra_kv4_store(const ra_kv4_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                       const int64_t* slot_map, int64_t num_tokens, void* stream) {
  ra::Kv4RowsParams p{};
  ra_status rs = check_rows(cache, k, k_stride, v, v_stride, slot_map, num_tokens, &p);
  if (rs != RA_OK || num_tokens == 0) return rs;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  const cudaError_t e = ra::launch_kv4_store(cache->head_dim, p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache store launch");
}

ra_status ra_kv4_load(const ra_kv4_cache* cache, const int64_t* slot_map, int64_t num_tokens, void* k, void* v,
                      void* stream) {
  ra::Kv4RowsParams p{};
  const int64_t row = cache ? (int64_t)cache->num_kv_heads * cache->head_dim : 0;
  ra_status rs = check_rows(cache, k, row, v, row, slot_map, num_tokens, &p);
  if (rs != RA_OK || num_tokens == 0) return rs;
  const size_t bytes = (size_t)num_tokens * row * 2;
  if (overlap(k, bytes, v, bytes) || overlap(k, bytes, slot_map, (size_t)num_tokens * 8) ||
      overlap(v, bytes, slot_map, (size_t)num_tokens * 8))
    return fail(RA_ERR_INVALID_ARG, "k and v must not lie over one another or over slot_map");
  p.k_out = k;
  p.v_out = v;
  const cudaError_t e = ra::launch_kv4_load(cache->head_dim, p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache load launch");
}

static ra_status check_heads(int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q_len) {
  if (D != 64 && D != 128 && D != 256) return fail(RA_ERR_UNSUPPORTED, "head_dim %d: 64, 128 or 256", D);
  if (Hkv < 1 || Hq < 1 || Hq > 65536 || Hq % Hkv)
    return fail(RA_ERR_INVALID_ARG, "num_q_heads %d must be a multiple of num_kv_heads %d", Hq, Hkv);
  if (max_q_len < 1) return fail(RA_ERR_INVALID_ARG, "max_q_len %d must be at least 1", max_q_len);
  return RA_OK;
}

ra_status ra_kv4_attention_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                           int32_t max_q_len, size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "NULL output");
  ra_status rs = check_heads(num_q_heads, num_kv_heads, head_dim, max_q_len);
  if (rs != RA_OK) return rs;
  *bytes = attn_layout(head_dim, num_q_heads / num_kv_heads, max_q_len).total;
  return RA_OK;
}

ra_status ra_kv4_attention(const ra_kv4_cache* cache, const void* q, int64_t q_stride, int32_t num_q_tokens,
                           int32_t num_q_heads, const int32_t* block_table, int32_t table_width, int64_t table_stride,
                           const int32_t* kv_lens, const int32_t* cu_q, int32_t num_requests, int32_t max_q_len,
                           int32_t causal, float softmax_scale, void* o, int32_t o_is_fp32, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  ra::Kv4AttnParams p{};
  ra_status rs = check_cache(cache, &p.cache);
  if (rs != RA_OK) return rs;
  const int32_t D = cache->head_dim, Hkv = cache->num_kv_heads;
  rs = check_heads(num_q_heads, Hkv, D, max_q_len);
  if (rs != RA_OK) return rs;
  if (num_q_tokens < 0 || num_requests < 0)
    return fail(RA_ERR_INVALID_ARG, "num_q_tokens %d, num_requests %d must not be negative", num_q_tokens, num_requests);
  if ((int64_t)num_q_tokens * num_q_heads > (int64_t(1) << 30))
    return fail(RA_ERR_INVALID_ARG, "%d query tokens of %d heads: more than 2^30 rows in one call", num_q_tokens, num_q_heads);
  if (table_width < 1 || table_stride < table_width)
    return fail(RA_ERR_INVALID_ARG, "table_width %d, table_stride %lld: need 1 <= width <= stride", table_width,
                (long long)table_stride);
  const AttnLayout l = attn_layout(D, num_q_heads / Hkv, max_q_len);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < l.total)
    return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes: need %zu, 256-byte aligned", workspace ? workspace_bytes : 0,
                l.total);
  if (num_q_tokens == 0 || num_requests == 0) {  // no row to write; the status is still this call's
    const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int32_t), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "status reset");
  }
  if (!q || !o || !lse || !block_table || !kv_lens || !cu_q) return fail(RA_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(kv_lens, 4) ||
      !aligned(cu_q, 4))
    return fail(RA_ERR_INVALID_ARG, "q and o must be 16-byte aligned, the other arrays 4-byte aligned");
  const int64_t row = (int64_t)num_q_heads * D;
  if (num_q_tokens > 1 && (q_stride < row || q_stride % 8))
    return fail(RA_ERR_INVALID_ARG, "q row stride %lld: a multiple of 8 elements, at least %lld", (long long)q_stride,
                (long long)row);
  const size_t q_bytes = ((size_t)(num_q_tokens - 1) * (num_q_tokens > 1 ? q_stride : row) + row) * 2;
  const size_t o_bytes = (size_t)num_q_tokens * row * (o_is_fp32 ? 4 : 2), lse_bytes = (size_t)num_q_tokens * num_q_heads * 4;
  if (overlap(o, o_bytes, q, q_bytes) || overlap(lse, lse_bytes, q, q_bytes) || overlap(o, o_bytes, lse, lse_bytes))
    return fail(RA_ERR_INVALID_ARG, "o and lse must not lie over q or over one another");
  if (!std::isfinite(softmax_scale)) return fail(RA_ERR_INVALID_ARG, "softmax_scale is not finite");
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  p.q = q;
  p.q_stride = q_stride;
  p.Tq = num_q_tokens;
  p.Hq = num_q_heads;
  p.R = num_requests;
  p.causal = causal != 0;
  p.block_table = block_table;
  p.table_stride = table_stride;
  p.table_width = table_width;
  p.kv_lens = kv_lens;
  p.cu_q = cu_q;
  p.scale = softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)D);
  p.page_bytes = (int64_t)page_bytes(cache->page_size, Hkv, D);
  p.o = o;
  p.o_is_fp32 = o_is_fp32 != 0;
  p.lse = lse;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.found = p.status + 1;
  p.ended = p.status + 2;
  p.tickets = reinterpret_cast<int32_t*>(ws + l.tickets);
  p.partials = reinterpret_cast<float*>(ws + l.partials);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const int32_t G = num_q_heads / Hkv;
  const bool tiles = has_tiles(G, max_q_len);
  if (!tiles || num_requests > 1) {  // (a single long request is the tile kernel's, whatever its real length)
    p.split_rows = tiles ? kTileMinRows : 0;
    e = ra::launch_kv4_attn(D, ra::kv4_attn_shape(D, few_rows(G, max_q_len), sms), p, st);
    if (e != cudaSuccess) return cuda_fail(e, "cache attention launch");
    p.status_kept = 1;
  }
  if (tiles) {
    e = ra::launch_kv4_tile(D, std::min(sms, ra::kKv4MaxSms), p, st);
    if (e != cudaSuccess) return cuda_fail(e, "cache attention launch (row tiles)");
  }
  return RA_OK;
}

ra_status ra_kv4_status(const void* status, void* stream_) {
  if (!status) return fail(RA_ERR_INVALID_ARG, "status is NULL");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream_);
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, status, sizeof(word), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  switch (word) {
    case 0: return RA_OK;
    case RA_KV4_BAD_PAGE: return fail(RA_ERR_INVALID_ARG, "a block table entry or free page is not a page of the cache");
    case RA_KV4_BAD_LENGTH: return fail(RA_ERR_INVALID_ARG, "a length is negative or passes the block table's row");
    case RA_KV4_BAD_OFFSET: return fail(RA_ERR_INVALID_ARG, "query offsets fall or pass the number of query tokens");
    case RA_KV4_TOO_MANY_TOKENS: return fail(RA_ERR_INVALID_ARG, "more new tokens than slots");
    case RA_KV4_NO_PAGES: return fail(RA_ERR_WORKSPACE, "not enough free pages");
    case RA_KV4_BAD_FREE_COUNT: return fail(RA_ERR_INVALID_ARG, "the free count is negative or passes the number of pages");
  }
  return fail(RA_ERR_TIMEOUT, "a kernel gave up on a pipeline wait (site %d)", word - ra::kKv4GaveUp);
}

}  // extern "C"
