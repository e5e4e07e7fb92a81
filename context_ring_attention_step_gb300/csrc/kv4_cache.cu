// kv4_cache.cu -- the 4-bit key/value cache around its attention:
//   * tables: pages taken and released, block table, slot map and positions
//     of a step, from the requests' lengths;
//   * store: bf16 rows rounded to 4 bits into the pages;
//   * load: cached rows back as bf16.
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

// One cluster runs the whole step.  Every CTA computes the prefix sums of all
// requests for itself (at most 4096 of them: a few loads a thread), then the
// cluster shares out the pages and the slots.  Nothing is written before every
// CTA has read the lengths and the free count, so the new lengths and the new
// free count may replace the old ones in place.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) kv4_tables_kernel(const Kv4TablesParams p) {
  extern __shared__ int32_t sm[];
  const int R = p.num_requests, P = 1 << p.page_shift;
  int32_t* s_len = sm;                // length before the step
  int32_t* s_cu = sm + R;             // [R + 1] tokens added before request r
  int32_t* s_need = s_cu + R + 1;     // [R + 1] pages taken before request r
  int32_t* s_back = s_need + R + 1;   // [R + 1] pages given back before request r
  __shared__ Counts s_warp[kThreads / 32];
  __shared__ int s_bad;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool alloc = p.free_pages != nullptr;
  const int32_t count = alloc ? *p.free_count : 0;
  if (tid == 0) s_bad = 0;
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
    const long long cap = (long long)p.table_width * P;
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
  const bool lead = cluster.block_rank() == 0;
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
  cluster.sync();  // every CTA has read its inputs; this CTA's prefix sums are in place

  if (lead) {
    for (int r = r0; r < r1; ++r) {
      const int i = r - r0;
      const bool leaves = ok && (i == 0 ? gone[0] : i == 1 ? gone[1] : i == 2 ? gone[2] : gone[3]);
      p.kv_lens_out[r] = leaves ? 0 : s_len[r] + (s_cu[r + 1] - s_cu[r]);
      p.cu_new[r] = s_cu[r];
    }
    if (tid == 0) {
      p.cu_new[R] = add;
      if (alloc) *p.free_count_out = count + back - need;
      *p.status = code;
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
  const int g0 = cluster.block_rank() * kThreads + tid, gn = cluster.num_blocks() * kThreads;
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
}

// ------------------------------------------------------------------ store / load

// One thread a group of 16 elements: 32 bytes of the row.
template <int D>
__global__ void __launch_bounds__(256) kv4_store_kernel(const Kv4RowsParams p) {
  using L = Kv4Layout<D>;
  const int groups = p.cache.Hkv * L::kGroups;
  const int64_t n = p.T * groups;
  const int64_t pmask = (int64_t(1) << p.cache.page_shift) - 1;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / groups;
    const int gi = (int)(i - t * groups);
    const int64_t slot = p.slots[t];
    const int64_t page = slot >> p.cache.page_shift;
    if (slot < 0 || page >= p.cache.num_pages) continue;
    const int head = gi / L::kGroups, g = gi % L::kGroups, tok = (int)(slot & pmask);
    uint8_t* tile = p.cache.pages + kv4_tile_offset<D>(p.cache, page, head, tok);
    const int tt = tok & 15;
    uint2 codes;
    uint32_t sc = kv4_round_group(reinterpret_cast<const uint4*>(
        reinterpret_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride + gi * 16), codes);
    *reinterpret_cast<uint2*>(tile + L::k_code(tt, g)) = codes;
    tile[L::k_scale(tt, g)] = (uint8_t)sc;
    sc = kv4_round_group(reinterpret_cast<const uint4*>(
        reinterpret_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride + gi * 16), codes);
    *reinterpret_cast<uint32_t*>(tile + L::v_code(tt, g, 0)) = codes.x;
    *reinterpret_cast<uint32_t*>(tile + L::v_code(tt, g, 1)) = codes.y;
    tile[L::v_scale(tt, g)] = (uint8_t)sc;
  }
}

template <int D>
__global__ void __launch_bounds__(256) kv4_load_kernel(const Kv4RowsParams p) {
  using L = Kv4Layout<D>;
  const int groups = p.cache.Hkv * L::kGroups;
  const int64_t n = p.T * groups;
  const int64_t pmask = (int64_t(1) << p.cache.page_shift) - 1;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / groups;
    const int gi = (int)(i - t * groups);
    const int64_t slot = p.slots[t];
    const int64_t page = slot >> p.cache.page_shift;
    uint4 ko[2] = {}, vo[2] = {};
    if (slot >= 0 && page < p.cache.num_pages) {
      const int head = gi / L::kGroups, g = gi % L::kGroups, tok = (int)(slot & pmask);
      const uint8_t* tile = p.cache.pages + kv4_tile_offset<D>(p.cache, page, head, tok);
      const int tt = tok & 15;
      kv4_expand_group(*reinterpret_cast<const uint2*>(tile + L::k_code(tt, g)), tile[L::k_scale(tt, g)], ko);
      kv4_expand_group(make_uint2(*reinterpret_cast<const uint32_t*>(tile + L::v_code(tt, g, 0)),
                                  *reinterpret_cast<const uint32_t*>(tile + L::v_code(tt, g, 1))),
                       tile[L::v_scale(tt, g)], vo);
    }
    uint4* kd = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.k_out) + i * 16);
    uint4* vd = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.v_out) + i * 16);
    kd[0] = ko[0];
    kd[1] = ko[1];
    vd[0] = vo[0];
    vd[1] = vo[1];
  }
}

template <typename F>
cudaError_t launch_rows(F kernel, int D, const Kv4RowsParams& p, cudaStream_t stream) {
  const int64_t n = p.T * p.cache.Hkv * (D / 16);
  if (n == 0) return cudaSuccess;
  const int64_t blocks = (n + 255) / 256;
  kernel<<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), 256, 0, stream>>>(p);
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
  if (p.num_slots <= 1024 && p.num_requests <= 256) {
    cfg.gridDim = dim3(attr[0].val.clusterDim.x = 1);
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, kv4_tables_kernel<256>, p);
  }
  static Kv4SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kv4_tables_kernel<1024>),
                                    (4 * kKv4MaxRequests + 3) * (int)sizeof(int32_t));
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(attr[0].val.clusterDim.x = 8);
  cfg.blockDim = dim3(1024);
  return cudaLaunchKernelEx(&cfg, kv4_tables_kernel<1024>, p);
}

cudaError_t launch_kv4_store(int D, const Kv4RowsParams& p, cudaStream_t stream) {
  if (D == 64) return launch_rows(kv4_store_kernel<64>, D, p, stream);
  if (D == 128) return launch_rows(kv4_store_kernel<128>, D, p, stream);
  if (D == 256) return launch_rows(kv4_store_kernel<256>, D, p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_load(int D, const Kv4RowsParams& p, cudaStream_t stream) {
  if (D == 64) return launch_rows(kv4_load_kernel<64>, D, p, stream);
  if (D == 128) return launch_rows(kv4_load_kernel<128>, D, p, stream);
  if (D == 256) return launch_rows(kv4_load_kernel<256>, D, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ra
