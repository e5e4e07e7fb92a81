// kv4_cache.cu -- the 4-bit key/value cache around its attention:
//   * tables: pages taken and released, block table, slot map and positions
//     of a step, from the requests' lengths;
//   * store: bf16 rows rounded to 4 bits into the pages;
//   * load: cached rows back as bf16.
// All three move bytes.  131072 rows (8 heads, head_dim 128) load in 106 us, 6.5 of
// the measured 6.78 TB/s; 32768 rows store in 42 us, 4.1 TB/s (16 loads
// and 128 registers a thread leave 22 % of the warps, and rounding follows loading);
// a step of the tables is three dependent reads and a launch.
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.h"
#include "kv4.cuh"
#include "tc.cuh"

namespace ra {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ tables

// Sums of the three per-request counts: tokens added, pages taken, pages given back.
struct Counts {
  int32_t add, need, back;
};

// One launch runs the whole step.  Every CTA computes the prefix sums of all
// requests for itself (at most 4096 of them: a few loads a thread), then the
// CTAs share out the pages and the slots.  What one CTA reads no other writes:
// pages taken in this step are computed again rather than read back, table
// entries and free pages are written only where none are read.  The new lengths
// and the new free count are the exception when they replace the old ones in
// place: the grid is then one cluster, which waits until all have read them.
// 262144 slots of 256 requests, one call with cold caches: 42 us in place (one cluster of
// 8 CTAs), 15 us as 257 CTAs.
constexpr int kTablesCluster = 8;  // a grid of at most so many CTAs is one cluster; a step in place has no larger one

template <int kThreads>
__global__ void __launch_bounds__(kThreads) kv4_tables_kernel(const Kv4TablesParams p) {
  extern __shared__ int32_t sm[];
  const int R = p.num_requests, P = 1 << p.page_shift;
  int32_t* s_len = sm;                // length before the step
  int32_t* s_cu = sm + R;             // [R + 1] tokens added before request r
  int32_t* s_need = s_cu + R + 1;     // [R + 1] pages taken before request r
  int32_t* s_back = s_need + R + 1;   // [R + 1] pages given back before request r
  __shared__ Counts s_warp[kThreads / 32];
  __shared__ int s_bad, s_none;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const cg::cluster_group cluster = cg::this_cluster();
  const bool alloc = p.free_pages != nullptr;
  const int32_t count = p.free_count ? *p.free_count : 0;
  if (tid == 0) s_bad = s_none = 0;
  __syncthreads();

  const int per = (R + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, R), r1 = min(r0 + per, R);
  // sums over this thread's requests; 64-bit, so that lengths without sense
  // cannot wrap around before they are refused
  long long add64 = 0, need64 = 0, back64 = 0;
  int bad = 0;
  auto counts = [&](int r, int32_t& len) {
    len = p.kv_lens[r];
    const int32_t nw = p.new_lens[r];
    const long long cap = min((long long)p.table_width * P, (long long)kKv4MaxLength);
    Counts c{0, 0, 0};
    if (len < 0 || nw < -1 || (long long)len + max(nw, 0) > cap) {
      bad = RA_KV4_BAD_LENGTH;
      return c;
    }
    const int32_t held = (int32_t)(((long long)len + P - 1) >> p.page_shift);
    if (nw < 0) {
      c.back = alloc ? held : 0;
    } else {
      c.add = nw;
      c.need = alloc ? (int32_t)(((long long)len + nw + P - 1) >> p.page_shift) - held : 0;
    }
    return c;
  };
  for (int r = r0; r < r1; ++r) {
    int32_t len;
    const Counts c = counts(r, len);
    add64 += c.add; need64 += c.need; back64 += c.back;
  }
  // block-wide exclusive prefix of the three sums, and their totals
  long long ta = add64, tn = need64, tb = back64;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    ta += __shfl_xor_sync(0xffffffffu, ta, d);
    tn += __shfl_xor_sync(0xffffffffu, tn, d);
    tb += __shfl_xor_sync(0xffffffffu, tb, d);
  }
  // A warp's sums that pass 2^30 are refused here; below that, 32 warps' sums
  // are added in 64 bits again.
  if (ta > (1ll << 30) || tn > (1ll << 30) || tb > (1ll << 30)) {
    bad = max(bad, (int)(ta > (1ll << 30) ? RA_KV4_TOO_MANY_TOKENS : RA_KV4_BAD_FREE_COUNT));
    add64 = need64 = back64 = 0;
    ta = tn = tb = 0;
  }
  int32_t xa = (int32_t)add64, xn = (int32_t)need64, xb = (int32_t)back64;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t ya = __shfl_up_sync(0xffffffffu, xa, d), yn = __shfl_up_sync(0xffffffffu, xn, d),
                  yb = __shfl_up_sync(0xffffffffu, xb, d);
    if (lane >= d) { xa += ya; xn += yn; xb += yb; }
  }
  if (lane == 31) s_warp[warp] = Counts{(int32_t)ta, (int32_t)tn, (int32_t)tb};
  if (bad) atomicMax(&s_bad, bad);
  __syncthreads();
  long long ba = 0, bn = 0, bb = 0, suma = 0, sumn = 0, sumb = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const Counts c = s_warp[w];
    if (w < warp) { ba += c.add; bn += c.need; bb += c.back; }
    suma += c.add; sumn += c.need; sumb += c.back;
  }
  int code = s_bad;
  if (code == 0) {
    if (suma > p.num_slots || suma > 0x7fffffffll) code = RA_KV4_TOO_MANY_TOKENS;
    else if (alloc && (count < 0 || count + sumb > p.num_pages)) code = RA_KV4_BAD_FREE_COUNT;
    else if (alloc && sumn > count + sumb) code = RA_KV4_NO_PAGES;
  }
  const bool ok = code == 0;
  int32_t ea = (int32_t)ba + xa - (int32_t)add64, en = (int32_t)bn + xn - (int32_t)need64,
          eb = (int32_t)bb + xb - (int32_t)back64;
  const bool lead = blockIdx.x == 0;
  for (int r = r0; r < r1; ++r) {
    int32_t len;
    const Counts c = counts(r, len);
    s_len[r] = len;
    s_cu[r] = ok ? ea : 0;
    s_need[r] = ok ? en : 0;
    s_back[r] = ok ? eb : 0;
    ea += c.add; en += c.need; eb += c.back;
  }
  const int32_t add = ok ? (int32_t)suma : 0, need = ok ? (int32_t)sumn : 0, back = ok ? (int32_t)sumb : 0;
  if (tid == 0) { s_cu[R] = add; s_need[R] = need; s_back[R] = back; }
  // which requests leave: read before anything is written
  bool gone[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) gone[i] = r0 + i < r1 && p.new_lens[r0 + i] < 0;
  cluster.sync();  // the cluster has read its inputs; this CTA's prefix sums are in place

  if (lead) {
    for (int r = r0; r < r1; ++r) {
      const int i = r - r0;
      const bool leaves = ok && (i == 0 ? gone[0] : i == 1 ? gone[1] : i == 2 ? gone[2] : gone[3]);
      p.kv_lens_out[r] = leaves ? 0 : s_len[r] + (s_cu[r + 1] - s_cu[r]);
      p.cu_new[r] = s_cu[r];
    }
    if (tid == 0) {
      p.cu_new[R] = add;
      if (p.free_count_out) *p.free_count_out = count + back - need;
    }
  }
  // last index i with a[i] <= x (a non-decreasing, a[0] = 0, x < a[R])
  auto find = [&](const int32_t* a, int32_t x) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  // page number `i` of the free list after the step's releases: what was free
  // before, then the released pages in request order
  const int32_t top = count + back;
  auto free_page = [&](int32_t i) -> int32_t {
    if (i < count) return p.free_pages[i];
    const int r = find(s_back, i - count);
    return p.block_table[(size_t)r * p.table_stride + (i - count - s_back[r])];
  };
  // Pages given back, taken, or with place for new tokens that are none: the step is
  // made, but its tokens there have no slot, and the status says so.  A grid of more CTAs than a
  // cluster leaves this to its first one, which then takes no slots: 262144 slots
  // of 256 requests, 24 of them leaving and 32 new, take 10.2 us a call, 12.3 where it does.
  const bool apart = gridDim.x > kTablesCluster;
  if (lead || !apart) {
    const int c0 = apart ? tid : blockIdx.x * kThreads + tid, cn = apart ? kThreads : gridDim.x * kThreads;
    int none = 0;
    // (taken pages that were not given back are a run of the free list)
#pragma unroll 8
    for (int32_t i = max(top - need, 0) + c0; i < count; i += cn) none |= p.free_pages[i];
    if (alloc) {
      for (int r = c0; r < R; r += cn)
        if (s_cu[r + 1] > s_cu[r] && (s_len[r] & (P - 1)))
          none |= p.block_table[(size_t)r * p.table_stride + (s_len[r] >> p.page_shift)];
      for (int r = c0 >> 5; r < R; r += cn >> 5)
#pragma unroll 4
        for (int32_t i = lane; i < s_back[r + 1] - s_back[r]; i += 32)
          none |= p.block_table[(size_t)r * p.table_stride + i];
    }
    if (none < 0) atomicOr(apart ? &s_none : cluster.map_shared_rank(&s_none, 0), 1);
  }
  const int others = apart ? gridDim.x - 1 : gridDim.x;
  const int gn = others * kThreads;
  const int g0 = apart && lead ? 0x7fffffff : (blockIdx.x - (apart ? 1 : 0)) * kThreads + tid;
  for (int32_t i = g0; i < back; i += gn) p.free_pages[count + i] = free_page(count + i);
  for (int32_t i = g0; i < need; i += gn) {
    const int r = find(s_need, i);
    const int32_t held = (int32_t)(((long long)s_len[r] + P - 1) >> p.page_shift);
    p.block_table[(size_t)r * p.table_stride + held + (i - s_need[r])] = free_page(top - 1 - i);
  }
  // Slots, four neighbours a thread: one search, then a walk.  A page taken in
  // this step is computed again rather than read, so no second wait is needed.
  const bool vec = (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0 && (reinterpret_cast<uintptr_t>(p.positions) & 15) == 0;
  for (int64_t t0 = 4 * (int64_t)g0; t0 < p.num_slots; t0 += 4 * (int64_t)gn) {
    int64_t slot[4];
    int32_t pos[4];
    int r = t0 < add ? find(s_cu, (int32_t)t0) : 0;
    int32_t last_page = -1, id = -1;
    int last_r = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + i;
      slot[i] = -1;
      pos[i] = -1;
      if (t < add) {
        while (t >= s_cu[r + 1]) ++r;
        pos[i] = s_len[r] + (int32_t)(t - s_cu[r]);
        const int32_t page = pos[i] >> p.page_shift;
        if (page != last_page || r != last_r) {
          const int32_t held = alloc ? (int32_t)(((long long)s_len[r] + P - 1) >> p.page_shift) : 0x7fffffff;
          id = page < held ? p.block_table[(size_t)r * p.table_stride + page]
                           : free_page(top - 1 - (s_need[r] + page - held));
          last_page = page;
          last_r = r;
        }
        slot[i] = id < 0 ? -1 : ((int64_t)id << p.page_shift) + (pos[i] & (P - 1));
      }
    }
    if (vec && t0 + 4 <= p.num_slots) {
      longlong2* s = reinterpret_cast<longlong2*>(p.slot_map + t0);
      s[0] = make_longlong2(slot[0], slot[1]);
      s[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int i = 0; i < 4 && t0 + i < p.num_slots; ++i) {
        p.slot_map[t0 + i] = slot[i];
        p.positions[t0 + i] = pos[i];
      }
    }
  }
  cluster.sync();
  if (lead && tid == 0) *p.status = code ? code : s_none ? RA_KV4_BAD_PAGE : 0;
}

// ------------------------------------------------------------------ store / load

// Tokens are taken four at a time (Q = 4): value codes of four neighbouring
// slots (the first a multiple of four) share 32-byte sectors, so that a prompt's
// rows move whole sectors.  Few rows go one at a time (Q = 1), to more threads.
// Threads of a block walk (quad, column) pairs, columns first.
struct Columns {
  // columns of a quad; x / n = umulhi(x, magic) for the x < 256 of several quads a
  // block (magic 0: one quad)
  uint32_t n, magic;
};

// Slots of the quad's tokens, -1 where there is none; true if they are four
// neighbours, the first a multiple of four.
template <int Q>
__device__ __forceinline__ bool quad_slots(const Kv4RowsParams& p, int64_t q, int64_t (&slot)[Q]) {
  const int64_t end = p.cache.num_pages << p.cache.page_shift;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    slot[i] = Q * q + i < p.T ? __ldg(p.slots + Q * q + i) : -1;
    if (slot[i] >= end) slot[i] = -1;
  }
  bool neighbours = Q == 4 && slot[0] >= 0 && (slot[0] & 3) == 0;
#pragma unroll
  for (int i = 1; i < Q; ++i) neighbours &= slot[i] == slot[0] + i;
  return neighbours;
}

template <int D>
__device__ __forceinline__ uint8_t* tile_of(const Kv4RowsParams& p, int64_t slot, int head) {
  const int64_t pmask = (int64_t(1) << p.cache.page_shift) - 1;
  return p.cache.pages + kv4_tile_offset<D>(p.cache, slot >> p.cache.page_shift, head, (int)(slot & pmask));
}

// A column is a group of 16 elements: 32 bytes of each of the four rows, of K and
// of V.
template <int D, int Q>
__global__ void __launch_bounds__(256) kv4_store_kernel(const Kv4RowsParams p, const Columns col, int quads_per_block) {
  using L = Kv4Layout<D>;
  const int64_t quads = (p.T + Q - 1) / Q;
  for (int64_t q0 = blockIdx.x * (int64_t)quads_per_block; q0 < quads; q0 += (int64_t)gridDim.x * quads_per_block) {
    for (uint32_t i = threadIdx.x; i < quads_per_block * col.n; i += 256) {
      const uint32_t ql = __umulhi(i, col.magic);
      const int gi = (int)(i - ql * col.n);
      const int64_t q = q0 + ql;
      if (q >= quads) break;
      int64_t slot[Q];
      const bool neighbours = quad_slots<Q>(p, q, slot);
      const int head = gi / L::kGroups, g = gi % L::kGroups;
      uint4 k[Q][2], v[Q][2];
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        if (slot[j] < 0) continue;
        const uint4* ks = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.k) + (Q * q + j) * p.k_stride + gi * 16);
        const uint4* vs = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.v) + (Q * q + j) * p.v_stride + gi * 16);
        k[j][0] = __ldg(ks);
        k[j][1] = __ldg(ks + 1);
        v[j][0] = __ldg(vs);
        v[j][1] = __ldg(vs + 1);
      }
      uint2 vc[Q];
      uint32_t vb[Q];
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        if (slot[j] < 0) continue;
        uint8_t* tile = tile_of<D>(p, slot[j], head);
        const int t = (int)(slot[j] & 15);
        uint2 c;
        const uint32_t b = kv4_round_group(k[j], c);
        *reinterpret_cast<uint2*>(tile + L::k_code(t, g)) = c;
        tile[L::k_scale(t, g)] = (uint8_t)b;
        vb[j] = kv4_round_group(v[j], vc[j]);
        if (!neighbours) {
          *reinterpret_cast<uint32_t*>(tile + L::v_code(t, g, 0)) = vc[j].x;
          *reinterpret_cast<uint32_t*>(tile + L::v_code(t, g, 1)) = vc[j].y;
          tile[L::v_scale(t, g)] = (uint8_t)vb[j];
        }
      }
      if constexpr (Q == 4) {
        if (!neighbours) continue;
        uint8_t* tile = tile_of<D>(p, slot[0], head);
        const int t = (int)(slot[0] & 15);
        if (D == 128) {  // tokens t .. t + 3: 32 bytes
          uint4* dst = reinterpret_cast<uint4*>(tile + L::v_code(t, g, 0));
          dst[0] = make_uint4(vc[0].x, vc[0].y, vc[1].x, vc[1].y);
          dst[1] = make_uint4(vc[2].x, vc[2].y, vc[3].x, vc[3].y);
        } else if (D == 64) {  // two tokens of one half: 8 bytes
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            *reinterpret_cast<uint2*>(tile + L::v_code(t + j, g, 0)) = make_uint2(vc[j].x, vc[j + 1].x);
            *reinterpret_cast<uint2*>(tile + L::v_code(t + j, g, 1)) = make_uint2(vc[j].y, vc[j + 1].y);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<uint2*>(tile + L::v_code(t + j, g, 0)) = vc[j];
        }
        *reinterpret_cast<uint16_t*>(tile + L::v_scale(t, g)) = (uint16_t)(vb[0] | vb[1] << 8);
        *reinterpret_cast<uint16_t*>(tile + L::v_scale(t + 2, g)) = (uint16_t)(vb[2] | vb[3] << 8);
      }
    }
  }
}

// A column is 8 elements: one 16-byte word of each of the four rows, of K and of
// V, so that the lanes of a warp write whole rows.
template <int D, int Q>
__global__ void __launch_bounds__(256) kv4_load_kernel(const Kv4RowsParams p, const Columns col, int quads_per_block) {
  using L = Kv4Layout<D>;
  const int64_t quads = (p.T + Q - 1) / Q;
  const int64_t row = (int64_t)p.cache.Hkv * D;
  for (int64_t q0 = blockIdx.x * (int64_t)quads_per_block; q0 < quads; q0 += (int64_t)gridDim.x * quads_per_block) {
    for (uint32_t i = threadIdx.x; i < quads_per_block * col.n; i += 256) {
      const uint32_t ql = __umulhi(i, col.magic);
      const int ci = (int)(i - ql * col.n);
      const int64_t q = q0 + ql;
      if (q >= quads) break;
      int64_t slot[Q];
      quad_slots<Q>(p, q, slot);
      const int head = ci / (2 * L::kGroups), g = (ci >> 1) % L::kGroups, half = ci & 1;
      uint32_t kc[Q] = {}, vc[Q] = {}, kb[Q] = {}, vb[Q] = {};
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        if (slot[j] < 0) continue;
        const uint8_t* tile = tile_of<D>(p, slot[j], head);
        const int t = (int)(slot[j] & 15);
        kc[j] = __ldg(reinterpret_cast<const uint32_t*>(tile + L::k_code(t, g) + 4 * half));
        vc[j] = __ldg(reinterpret_cast<const uint32_t*>(tile + L::v_code(t, g, half)));
        kb[j] = __ldg(tile + L::k_scale(t, g));
        vb[j] = __ldg(tile + L::v_scale(t, g));
      }
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        if (Q * q + j >= p.T) break;
        const int64_t off = (Q * q + j) * row + ci * 8;
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.k_out) + off), kv4_expand_half(kc[j], kb[j]));
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.v_out) + off), kv4_expand_half(vc[j], vb[j]));
      }
    }
  }
}

// Four tokens a thread where that still fills the GPU (152 SMs x 2048 threads),
// else one: 64 rows of 8 heads (head_dim 128) are stored and read back in 11.4 us
// one by one and in 13.4 by fours, 32768 of them in 81 and 73 us.
template <typename F>
cudaError_t launch_rows(F by_one, F by_four, uint32_t columns, const Kv4RowsParams& p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  const bool four = p.T * columns >= 4 * 152 * 2048;
  const int per_block = columns >= 256 ? 1 : 256 / columns;  // quads: about one column a thread
  const int64_t quads = four ? (p.T + 3) / 4 : p.T;
  const int64_t blocks = std::min<int64_t>((quads + per_block - 1) / per_block, 1 << 20);
  const Columns col{columns, per_block > 1 ? (uint32_t)((uint64_t(1) << 32) / columns + 1) : 0};
  (four ? by_four : by_one)<<<(unsigned)blocks, 256, 0, stream>>>(p, col, per_block);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_tables(const Kv4TablesParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)(4 * p.num_requests + 3) * sizeof(int32_t);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool in_place = p.kv_lens_out == p.kv_lens || (p.free_pages && p.free_count_out == p.free_count);
  // 256 threads take up to four requests each; four slots a thread
  const bool small = p.num_requests <= 1024;
  const int64_t threads = small ? 256 : 1024;
  const int64_t want = std::max<int64_t>(1, (p.num_slots + 4 * threads - 1) / (4 * threads));
  const int64_t most = in_place ? kTablesCluster : small ? 304 : 152;
  const int64_t ctas = std::min(want, most);
  cfg.gridDim = dim3((unsigned)(ctas > kTablesCluster ? ctas + 1 : ctas));
  cfg.blockDim = dim3((unsigned)threads);
  attr[0].val.clusterDim.x = ctas > kTablesCluster ? 1 : cfg.gridDim.x;
  if (small) return cudaLaunchKernelEx(&cfg, kv4_tables_kernel<256>, p);
  static Kv4SmemLimit limit;
  return limit.launch(reinterpret_cast<const void*>(kv4_tables_kernel<1024>),
                      (4 * kKv4MaxRequests + 3) * (int)sizeof(int32_t),
                      [&] { return cudaLaunchKernelEx(&cfg, kv4_tables_kernel<1024>, p); });
}

cudaError_t launch_kv4_store(int D, const Kv4RowsParams& p, cudaStream_t stream) {
  if (D == 64) return launch_rows(kv4_store_kernel<64, 1>, kv4_store_kernel<64, 4>, p.cache.Hkv * 4, p, stream);
  if (D == 128) return launch_rows(kv4_store_kernel<128, 1>, kv4_store_kernel<128, 4>, p.cache.Hkv * 8, p, stream);
  if (D == 256) return launch_rows(kv4_store_kernel<256, 1>, kv4_store_kernel<256, 4>, p.cache.Hkv * 16, p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_load(int D, const Kv4RowsParams& p, cudaStream_t stream) {
  if (D == 64) return launch_rows(kv4_load_kernel<64, 1>, kv4_load_kernel<64, 4>, p.cache.Hkv * 8, p, stream);
  if (D == 128) return launch_rows(kv4_load_kernel<128, 1>, kv4_load_kernel<128, 4>, p.cache.Hkv * 16, p, stream);
  if (D == 256) return launch_rows(kv4_load_kernel<256, 1>, kv4_load_kernel<256, 4>, p.cache.Hkv * 32, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ra
