// kv4.h -- the 4-bit key/value cache: format, tile layout, parameter blocks and
// launch wrappers shared by its kernels (kv4_cache.cu, kv4_attn.cu) and its C
// entry points (kv4_api.cu).  Not part of the public ABI; the layout is
// documented in ring_attn.h.
#pragma once

#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/ring_attn.h"

namespace ra {

constexpr int kKv4Tile = 16;               // tokens of one tile
constexpr int kKv4Group = 16;              // elements sharing one scale
constexpr float kKv4MaxScale = 10240.f;    // largest scale: 6 * 10240 is finite in fp16
constexpr int kKv4NanScale = 0xff;         // scale byte of a group with a non-finite element
constexpr int kKv4MaxLength = 1 << 30;     // cached tokens of a request (positions a few tiles on still fit 32 bits)
// Status of a kernel that gave up on a pipeline wait: this plus the wait's site.  Above the
// codes of the public header, so that it wins where both occur: rows are missing then.
constexpr int kKv4GaveUp = 2000;
static_assert(kKv4GaveUp > RA_KV4_BAD_FREE_COUNT, "the largest status wins");
constexpr int kKv4MaxRequests = 4096;      // kv4_tables keeps per-request prefix sums in shared memory

// One tile: K codes (8 D bytes), K scales (D), V codes (8 D), V scales (D).
constexpr int kv4_tile_bytes(int D) { return 18 * D; }

// Byte offsets inside a tile.  The orders follow the operand registers of the
// m16n8k16 tensor-core product that attention uses (kv4_attn.cu), so that one
// lane's share of a tile is whole 16-byte words:
//   K (16 tokens x 16 dims an MMA): lane 4 r + c holds tokens r and r + 8 and
//     the contiguous dims [c D/4, (c+1) D/4);
//   V^T (16 dims x 16 tokens an MMA): lane 4 r + c holds dims [r D/8, (r+1) D/8)
//     and tokens 2c, 2c + 1, 2c + 8, 2c + 9.
// `t` is the token within the tile, `g` the group of 16 dims.
template <int D>
struct Kv4Layout {
  static constexpr int kKCodes = 0;
  static constexpr int kKScales = 8 * D;
  static constexpr int kVCodes = 9 * D;
  static constexpr int kVScales = 17 * D;
  static constexpr int kBytes = 18 * D;
  static constexpr int kGroups = D / 16;

  // 8 bytes: the codes of one token's group of keys, two dims a byte
  __host__ __device__ static constexpr int k_code(int t, int g) {
    const int r = t & 7, h = t >> 3;
    if (D == 64) return (4 * r + g) * 16 + h * 8;
    if (D == 128) return h * 512 + (4 * r + (g >> 1)) * 16 + (g & 1) * 8;
    return (2 * h + ((g & 3) >> 1)) * 512 + (4 * r + (g >> 2)) * 16 + (g & 1) * 8;
  }
  __host__ __device__ static constexpr int k_scale(int t, int g) {
    constexpr int per = D / 64;  // groups of one lane and token
    return kKScales + (4 * (t & 7) + g / per) * (2 * per) + (t >> 3) * per + g % per;
  }
  // `half` selects 8 of the group's dims: 4 bytes.  At head_dim 128 and 256 the
  // two halves are neighbours.
  __host__ __device__ static constexpr int v_code(int t, int g, int half) {
    const int h = t >> 3, c = (t & 7) >> 1, e = t & 1;
    if (D == 64) return kVCodes + (4 * (2 * g + half) + c) * 16 + (2 * h + e) * 4;
    if (D == 128) return kVCodes + h * 512 + (4 * g + c) * 16 + e * 8 + half * 4;
    return kVCodes + (2 * h + e) * 512 + (4 * (g >> 1) + c) * 16 + (g & 1) * 8 + half * 4;
  }
  __host__ __device__ static constexpr int v_scale(int t, int g) {
    const int h = t >> 3, c = (t & 7) >> 1, e = t & 1;
    if (D == 256) return kVScales + (4 * (g >> 1) + c) * 8 + (g & 1) * 4 + 2 * h + e;
    return kVScales + (4 * g + c) * 4 + 2 * h + e;
  }
};

// A cache as the kernels see it.
struct Kv4Cache {
  uint8_t* pages;
  int64_t num_pages;
  int32_t page_shift;  // log2 of the page size in tokens
  int32_t Hkv;
};

// Byte offset of the tile that holds token `t` (within the page) of a page and head.
template <int D>
__device__ __forceinline__ size_t kv4_tile_offset(const Kv4Cache& c, int64_t page, int head, int t) {
  const size_t tiles = size_t(1) << (c.page_shift - 4);
  return (((size_t)page * c.Hkv + head) * tiles + (t >> 4)) * Kv4Layout<D>::kBytes;
}

// Launches of a kernel whose dynamic shared memory limit has to be raised: once on
// every device (the attribute call costs about as much host time as a launch),
// and again if a launch is refused, as after a cudaDeviceReset.  One per kernel.
struct Kv4SmemLimit {
  std::atomic<uint64_t> done{0};
  template <typename F>
  cudaError_t launch(const void* kernel, int bytes, F launch_kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    const bool known = (done.load(std::memory_order_relaxed) & bit) != 0;
    if (known && (e = launch_kernel()) != cudaErrorInvalidValue) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
    return launch_kernel();
  }
};

struct Kv4TablesParams {
  const int32_t* kv_lens;
  const int32_t* new_lens;
  int32_t* block_table;
  int64_t table_stride;
  int32_t table_width, num_requests, page_shift;
  int32_t* free_pages;  // null: the block table already holds every page
  int32_t num_pages;
  const int32_t* free_count;
  int64_t num_slots;
  int32_t* kv_lens_out;
  int32_t* cu_new;
  int64_t* slot_map;
  int32_t* positions;
  int32_t* free_count_out;
  int32_t* status;
};

struct Kv4RowsParams {
  Kv4Cache cache;
  const int64_t* slots;
  int64_t T;
  const void* k;  // store: bf16 rows in
  const void* v;
  int64_t k_stride, v_stride;  // elements between rows
  void* k_out;  // load: bf16 rows out, dense
  void* v_out;
};

struct Kv4AttnParams {
  Kv4Cache cache;
  const void* q;  // bf16 [Tq, Hq, D], rows q_stride elements apart
  int64_t q_stride;
  int32_t Tq, Hq, R, causal;
  const int32_t* block_table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  float scale;
  int64_t page_bytes;
  void* o;
  int32_t o_is_fp32;
  float* lse;  // [Hq, Tq]
  int32_t* status;
  // Zero between calls: what the CTAs found wrong (RA_KV4_BAD_...), how many of
  // them have ended, and how many of the partial results that are merged together
  // are there (by the slot of the first one, then by the CTA that began the unit).
  int32_t *found, *ended, *tickets;
  int32_t status_kept;  // the status holds what the other kernel of this call found
  int32_t split_rows;   // rows (query tokens x heads of a group) from which a request is the tile kernel's; 0: see kv4_walk.cuh
  float* partials;  // two slots per CTA: [0] of a unit that an earlier CTA began, [1] of one that this CTA began
};

cudaError_t launch_kv4_tables(const Kv4TablesParams& p, cudaStream_t stream);
cudaError_t launch_kv4_store(int D, const Kv4RowsParams& p, cudaStream_t stream);
cudaError_t launch_kv4_load(int D, const Kv4RowsParams& p, cudaStream_t stream);

// Variant of the kernel for few rows (kv4_attn.cu): query rows of one CTA, CTAs
// on a GPU with `sms` SMs, and the floats of one partial-result slot (two slots a
// CTA).  `rows`: the rows (tokens x heads of a group) that most requests bring.
struct Kv4AttnShape {
  int rows, ctas;
  size_t slot_floats;
};
constexpr int kKv4MaxSms = 160;            // workspaces are sized for this many SMs
constexpr int kKv4MaxCtas = 4 * kKv4MaxSms;  // and at most four CTAs on each
Kv4AttnShape kv4_attn_shape(int D, long long rows, int sms);
// The tile kernel (kv4_tile.cu): one CTA an SM.
constexpr size_t kv4_tile_slot_floats(int D) { return 256 * ((size_t)D + 2); }
cudaError_t launch_kv4_tile(int D, int ctas, const Kv4AttnParams& p, cudaStream_t stream);
cudaError_t launch_kv4_attn(int D, const Kv4AttnShape& shape, const Kv4AttnParams& p, cudaStream_t stream);

}  // namespace ra
