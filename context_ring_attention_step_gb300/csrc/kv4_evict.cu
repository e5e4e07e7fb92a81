// kv4_evict.cu -- eviction from the 4-bit cache by accumulated attention weight:
//   * evict: which tokens of every request over its budget go, which kept rows move
//     into their places, and the pages given back;
//   * move: rows copied from slots to slots, bit by bit.
//
// A request of L tokens with budget B keeps its first `sinks`, its last `recent`, and
// of the others those with the largest sums.  A key orders them: the sum's bits (sums
// are no negative numbers, so their bits order like they do), above all of them for the
// protected ones; the B-th largest key is found digit by digit from histograms (11, 11 and 10 bits),
// and of equal keys the lowest indices are taken.  Then kept tokens behind place B (the
// m-th of them) move into the places of dropped ones before it (the m-th): sources and places
// are disjoint, so the rows can move in any order, and no more of them than are dropped.
//
// What has to be read are 4 bytes a token; what takes time are the steps that wait for one
// another: lengths, pages, sums, then for each digit the counts of all, the digit, the tokens with it.  A
// request is one cluster of CTAs: its tokens' keys lie in their shared memory, and the counts
// are added up in that of the first.  One request of 131072 tokens takes 25 us, 64 of 4096
// 13 us, and a request of 500 9 us.
// Rows move in pieces of 4 and 8 bytes, as the cache's tiles hold them: V's pieces of a row lie
// 32 bytes apart, so that a row costs 5 times its bytes: 8192 rows of 8 heads of 128, 8.8 MB, take
// 13.6 us and read 43 MB of sectors.
#include <algorithm>

#include <cooperative_groups.h>

#include "kv4.cuh"
#include "kv4.h"
#include "kv4_walk.cuh"

namespace ra {
namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;
constexpr int kMaxKeys = 40960;  // keys of a CTA in shared memory; the others are made again where they are needed
constexpr uint32_t kProtected = 0xffffffffu;

// Block-wide exclusive prefix sum in thread order; `total` receives the sum.
template <int T>
__device__ __forceinline__ int block_prefix(int x, int* s_sum, int& total) {
  constexpr int W = T / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  __syncthreads();  // (s_sum of the call before was read)
  if (lane == 31) s_sum[warp] = y;
  __syncthreads();
  int before = lane < warp ? s_sum[lane % W] : 0;
  total = lane < W ? s_sum[lane % W] : 0;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    total += __shfl_xor_sync(0xffffffffu, total, d);
  }
  return before + y - x;
}

// What a CTA of a cluster tells the others.
struct Told {
  int bad, equal, holes, movers;
};

// T threads: 512 or 256 (launch_kv4_evict).
template <int T>
__global__ void __launch_bounds__(T, T == 512 ? 2 : 4) kv4_evict_kernel(const Kv4EvictParams p, int keys_held) {
  constexpr int kWarps = T / 32;
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ __align__(16) uint32_t s_hist[kBins];      // of this CTA
  __shared__ __align__(16) uint32_t s_total[3][kBins];  // of the cluster, in its first CTA
  __shared__ int s_sum[kWarps], s_digit[3];             // digit, keys still to take at it, keys with it
  __shared__ Told s_told;
  __shared__ int s_last, s_mine[4];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.page_shift;
  const int64_t pages = p.num_pages;

  const int L = p.kv_lens[r], B = p.budgets[r];
  int code = 0;
  const bool sane = L >= 0 && (long long)L <= min((long long)p.table_width << p.page_shift, (long long)kKv4MaxLength);
  if (!sane) code = RA_KV4_BAD_LENGTH;
  bool cut = sane && B >= 0 && (long long)L > (long long)B + p.slack;
  if (cut && B < (long long)p.sinks + p.recent) {
    code = RA_KV4_BAD_BUDGET;
    cut = false;
  }
  const int32_t* table = p.block_table + (size_t)r * p.table_stride;
  int moves = 0;
  int64_t* src = p.src + (size_t)r * p.max_moves;
  int64_t* dst = p.dst + (size_t)r * p.max_moves;
  if (cut) {
    // this CTA's tokens [t0, t1), and each warp's share of them [w0, w1), in whole 128s: a lane
    // takes four neighbours at a time, which lie on one page
    const int per_cta = (L + C - 1) / C, per_warp = ((per_cta + kWarps - 1) / kWarps + 127) & ~127;
    const int t0 = min(rank * per_warp * kWarps, L), t1 = min(t0 + per_warp * kWarps, L);
    const int w0 = min(t0 + warp * per_warp, t1), w1 = min(w0 + per_warp, t1);
    int bad = 0;
    auto slot_of = [&](int t) -> int64_t {
      return ((int64_t)table[t >> p.page_shift] << p.page_shift) + (t & (P - 1));
    };
    const bool wide = (reinterpret_cast<uintptr_t>(p.weights) & 15) == 0;
    auto make_keys = [&](int t) -> uint4 {
      const int page = table[t >> p.page_shift];
      if ((uint32_t)page >= (uint64_t)pages) {
        bad = 1;
        return make_uint4(0u, 0u, 0u, 0u);
      }
      const float* w = p.weights + ((int64_t)page << p.page_shift) + (t & (P - 1));
      const float4 x = wide ? __ldg(reinterpret_cast<const float4*>(w))
                            : make_float4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
      auto key = [&](int t, float w) -> uint32_t {
        return t < p.sinks || t >= L - p.recent ? kProtected : w > 0.f ? __float_as_uint(w) : 0u;
      };
      return make_uint4(key(t, x.x), key(t + 1, x.y), key(t + 2, x.z), key(t + 3, x.w));
    };
    auto keys_of = [&](int t) -> uint4 {
      return t - t0 + 3 < keys_held ? *reinterpret_cast<const uint4*>(s_keys + (t - t0)) : make_keys(t);
    };
    auto get = [](const uint4& k, int i) { return i == 0 ? k.x : i == 1 ? k.y : i == 2 ? k.z : k.w; };
    for (int i = tid; i < kBins; i += T) s_hist[i] = s_total[0][i] = s_total[1][i] = s_total[2][i] = 0u;
    if (tid == 0) s_told = Told{0, 0, 0, 0};
    if (C > 1) cluster.sync();  // (the others add to the first CTA's bins)
    __syncthreads();
    // add one to a bin for every lane that asks; neighbours often ask for the same one
    auto count = [&](uint32_t* hist, bool in, uint32_t bin) {
      const uint32_t who = __ballot_sync(0xffffffffu, in);
      if (who == 0) return;
      const uint32_t first = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
      if (__all_sync(0xffffffffu, !in || bin == first)) {
        if (lane == 0) atomicAdd(hist + first, (uint32_t)__popc(who));
      } else if (in) {
        atomicAdd(hist + bin, 1u);
      }
    };
    uint32_t* hist = C > 1 ? s_hist : s_total[0];
#pragma unroll 1
    for (int t = w0 + 4 * lane; t - 4 * lane < w1; t += 256) {
      uint4 k[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) k[h] = t + 128 * h < w1 ? make_keys(t + 128 * h) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int u = t + 128 * h;
        if (u < w1 && u - t0 + 3 < keys_held) *reinterpret_cast<uint4*>(s_keys + (u - t0)) = k[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) count(hist, u + i < w1, get(k[h], i) >> 21);
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&s_told.bad, 1);

    // ---- the B-th largest key, and how many of its equals are taken
    uint32_t key = 0u;
    int take = B, equal = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      if (pass > 0) {
        const uint32_t top = shift + (pass == 1 ? 11 : 10);
        if (C == 1) hist = s_total[pass];
        for (int t = w0 + 4 * lane; t - 4 * lane < w1; t += 128) {
          const uint4 k = t < w1 ? keys_of(t) : make_uint4(0u, 0u, 0u, 0u);
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) m |= (t + i < w1 && (get(k, i) >> top) == (key >> top) ? 1u : 0u) << i;
          if (!__any_sync(0xffffffffu, m != 0)) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) count(hist, (m >> i) & 1u, (get(k, i) >> shift) & (pass == 1 ? 2047u : 1023u));
        }
      }
      __syncthreads();
      if (C > 1) {  // this CTA's bins to the cluster's; most are empty
        for (int i = tid; i < kBins; i += T) {
          const uint32_t n = s_hist[i];
          if (n) {
            atomicAdd(cluster.map_shared_rank(&s_total[pass][i], 0), n);
            s_hist[i] = 0u;
          }
        }
        cluster.sync();
      }
      // The first CTA finds the digit for all: 16 that each read its 8 KB of bins took 6 us a pass.
      // Bins from the top: thread i has the kBins / T behind place kBins - (i + 1) kBins / T.
      if (rank == 0) {
        constexpr int kEach = kBins / T;
        const int b0 = kBins - kEach - kEach * tid;
        int n[kEach], sum = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) sum += n[i] = (int)s_total[pass][b0 + i];
        int total;
        int above = block_prefix<T>(sum, s_sum, total);
#pragma unroll
        for (int i = kEach - 1; i >= 0; --i) {
          if (above < take && above + n[i] >= take) {
            s_digit[0] = b0 + i;
            s_digit[1] = take - above;
            s_digit[2] = n[i];
          }
          above += n[i];
        }
      }
      if (C > 1) cluster.sync(); else __syncthreads();
      if (take <= 0) {  // none is kept
        key = kProtected;
        break;
      }
      const int* digit = cluster.map_shared_rank(s_digit, 0);
      key |= (uint32_t)digit[0] << shift;
      take = digit[1];
      equal = digit[2];
      if (equal == take) break;  // all keys that begin with these digits are taken: those from `key` on
    }

    // ---- of equal keys the lowest indices: this warp's first one's rank among them
    int before_equal = 0;
    // sums over the cluster's CTAs of what they told: f(Told) of all of them, and of those before this one
    auto gather = [&](auto f, int& before) {
      int x = lane < C ? f(*cluster.map_shared_rank(&s_told, lane)) : 0;
      before = lane < rank ? x : 0;
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, d);
        before += __shfl_xor_sync(0xffffffffu, before, d);
      }
      return x;
    };
    if (equal != take) {
      int mine = 0;
      for (int t = w0 + 4 * lane; t < w1; t += 128) {
        const uint4 k = keys_of(t);
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += t + i < w1 && get(k, i) == key;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
      int total, others;
      before_equal = __shfl_sync(0xffffffffu, block_prefix<T>(lane == 0 ? mine : 0, s_sum, total), 0);
      if (tid == 0) s_told.equal = total;
      if (C > 1) cluster.sync(); else __syncthreads();
      gather([](const Told& o) { return o.equal; }, others);
      before_equal += others;
    }
    // The warp's tokens in order, 128 at a time: f(t, places, moves), a lane's four from t on:
    // those that are dropped before place B, and those that are kept behind it.
    const uint32_t below = (1u << lane) - 1u;
    auto rank_of = [&](uint32_t m, int& all) {  // bits set in the lanes before; in all
      int n = 0;
      all = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = __ballot_sync(0xffffffffu, (m >> i) & 1u);
        n += __popc(b & below);
        all += __popc(b);
      }
      return n;
    };
    auto walk = [&](auto f) {
      int seen = before_equal;
      for (int t = w0 + 4 * lane; t - 4 * lane < w1; t += 128) {
        const uint4 k = t < w1 ? keys_of(t) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t in = 0, kept = 0, same = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          in |= (t + i < w1 ? 1u : 0u) << i;
          kept |= (get(k, i) > key ? 1u : 0u) << i;
          same |= (get(k, i) == key ? 1u : 0u) << i;
        }
        kept &= in;
        same &= in;
        if (equal == take) {
          kept |= same;
        } else if (__any_sync(0xffffffffu, same != 0)) {
          int all;
          int n = seen + rank_of(same, all);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((same >> i) & 1u) kept |= (n++ < take ? 1u : 0u) << i;
          seen += all;
        }
        const int inside = min(max(B - t, 0), 4);  // of the four, before place B
        const uint32_t first = (1u << inside) - 1u;
        f(t, in & ~kept & first, kept & ~first);
      }
    };
    int holes = 0, movers = 0;  // of this warp
    walk([&](int t, uint32_t h, uint32_t m) {
      holes += __popc(h);
      movers += __popc(m);
    });
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      holes += __shfl_xor_sync(0xffffffffu, holes, d);
      movers += __shfl_xor_sync(0xffffffffu, movers, d);
    }
    int cta_holes, cta_movers;
    int h0 = __shfl_sync(0xffffffffu, block_prefix<T>(lane == 0 ? holes : 0, s_sum, cta_holes), 0);
    int m0 = __shfl_sync(0xffffffffu, block_prefix<T>(lane == 0 ? movers : 0, s_sum, cta_movers), 0);
    if (tid == 0) {
      s_told.holes = cta_holes;
      s_told.movers = cta_movers;
    }
    if (C > 1) cluster.sync(); else __syncthreads();
    if (warp == 0) {
      int holes_before, movers_before, none;
      gather([](const Told& o) { return o.holes; }, holes_before);
      const int all = gather([](const Told& o) { return o.movers; }, movers_before);
      const int wrong = gather([](const Told& o) { return o.bad; }, none);
      if (lane == 0) {
        s_mine[0] = holes_before;
        s_mine[1] = movers_before;
        s_mine[2] = all;
        s_mine[3] = wrong;
      }
    }
    __syncthreads();
    h0 += s_mine[0];
    m0 += s_mine[1];
    moves = s_mine[2];
    bad = s_mine[3];
    if (bad) code = RA_KV4_BAD_PAGE;
    else if (moves > p.max_moves) code = RA_KV4_TOO_MANY_MOVES;
    if (code) {
      cut = false;
      moves = 0;
    } else {
      walk([&](int t, uint32_t h, uint32_t m) {
        if (!__any_sync(0xffffffffu, (h | m) != 0)) return;
        int all_h, all_m;
        int nh = h0 + rank_of(h, all_h), nm = m0 + rank_of(m, all_m);
        h0 += all_h;
        m0 += all_m;
        if (!(h | m)) return;
        const int64_t slot = slot_of(t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((h >> i) & 1u) dst[nh++] = slot + i;
          if ((m >> i) & 1u) src[nm++] = slot + i;
        }
      });
    }
    if (C > 1) cluster.sync();  // no CTA ends while another reads its shared memory
  }
  for (int i = moves + rank * T + tid; i < p.max_moves; i += C * T) src[i] = dst[i] = -1;

  // ---- the call's last CTA: lengths, pages given back, status
  __syncthreads();
  if (tid == 0) {
    if (rank == 0) {
      p.after[r] = cut ? B : L;
      if (code) atomicMax(p.found, code);
    }
    __threadfence();
    s_last = atomicAdd(p.ended, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const int R = p.num_requests;
  const int count0 = p.free_count ? *p.free_count : 0;
  // (the prefix sums of all requests' pages lie where the histograms were)
  int* s_back = reinterpret_cast<int*>(&s_total[0][0]);  // [R + 1], R <= 4096
  const int per = (R + T - 1) / T, r0 = min(tid * per, R), r1 = min(r0 + per, R);
  auto held = [&](int n) { return n > 0 ? (int)(((long long)n + P - 1) >> p.page_shift) : 0; };
  long long back = 0;
  for (int i = r0; i < r1; ++i) {
    const int l = p.kv_lens[i], a = __ldcg(p.after + i);
    if (a < l) back += held(l) - held(a);
  }
  // the sum of all in 64 bits: tables that are not sound may hold more pages than there are
  long long sum = back;
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  __shared__ long long s_pages[kWarps];
  if (lane == 0) s_pages[warp] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < kWarps; ++w) sum += s_pages[w];
  const bool push = p.free_pages != nullptr;
  const bool fits = !push || (count0 >= 0 && count0 + sum <= p.num_free);
  if (!push || !fits) back = sum = 0;
  int total;
  int at = block_prefix<T>((int)back, s_sum, total);
  for (int i = r0; i < r1; ++i) {
    const int l = p.kv_lens[i], a = fits ? __ldcg(p.after + i) : l;
    s_back[i] = at;
    if (push && a < l) at += held(l) - held(a);
  }
  if (tid == 0) s_back[R] = total;
  __syncthreads();
  for (int i = tid; i < total; i += T) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_back[mid] <= i) lo = mid; else hi = mid;
    }
    p.free_pages[count0 + i] = p.block_table[(size_t)lo * p.table_stride + held(__ldcg(p.after + lo)) + (i - s_back[lo])];
  }
  if (!fits)  // nothing is dropped
    for (long long i = tid; i < (long long)R * p.max_moves; i += T) p.src[i] = p.dst[i] = -1;
  __syncthreads();
  for (int i = r0; i < r1; ++i) {
    const int l = p.kv_lens[i], a = fits ? __ldcg(p.after + i) : l;
    p.dropped[i] = a < l ? l - a : 0;
    p.kv_lens_out[i] = a;  // (may be kv_lens)
  }
  if (tid == 0) {
    if (p.free_count_out) *p.free_count_out = count0 + total;
    const int found = atomicExch(p.found, 0);
    *p.status = !fits ? (int)RA_KV4_BAD_FREE_COUNT : found;
    *p.ended = 0;
  }
}

// A thread copies 16 dims of one row and head: K and V codes and scales.
template <int D>
__global__ void __launch_bounds__(256) kv4_move_kernel(const Kv4MoveParams p) {
  using L = Kv4Layout<D>;
  const int64_t end = p.cache.num_pages << p.cache.page_shift;
  const int64_t pmask = (int64_t(1) << p.cache.page_shift) - 1;
  const int columns = p.cache.Hkv * L::kGroups;
  const int64_t n = p.n * columns;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const int64_t m = kv4_div(i, columns);
    const int c = (int)(i - m * columns), head = c / L::kGroups, g = c % L::kGroups;
    const int64_t from = __ldg(p.src + m), to = __ldg(p.dst + m);
    if (from < 0 || to < 0 || from >= end || to >= end) continue;
    const uint8_t* a = p.cache.pages + kv4_tile_offset<D>(p.cache, from >> p.cache.page_shift, head, (int)(from & pmask));
    uint8_t* b = p.cache.pages + kv4_tile_offset<D>(p.cache, to >> p.cache.page_shift, head, (int)(to & pmask));
    const int s = (int)(from & 15), t = (int)(to & 15);
    const uint2 k = *reinterpret_cast<const uint2*>(a + L::k_code(s, g));
    const uint32_t v0 = *reinterpret_cast<const uint32_t*>(a + L::v_code(s, g, 0));
    const uint32_t v1 = *reinterpret_cast<const uint32_t*>(a + L::v_code(s, g, 1));
    const uint8_t ks = a[L::k_scale(s, g)], vs = a[L::v_scale(s, g)];
    *reinterpret_cast<uint2*>(b + L::k_code(t, g)) = k;
    *reinterpret_cast<uint32_t*>(b + L::v_code(t, g, 0)) = v0;
    *reinterpret_cast<uint32_t*>(b + L::v_code(t, g, 1)) = v1;
    b[L::k_scale(t, g)] = ks;
    b[L::v_scale(t, g)] = vs;
    if (p.weights && c == 0) p.weights[to] = p.weights[from];
  }
}

}  // namespace

template <int T>
static cudaError_t launch_evict(const Kv4EvictParams& p, int ctas, int64_t most, cudaStream_t stream) {
  auto kern = kv4_evict_kernel<T>;
  const int64_t share = ((most + ctas - 1) / ctas + T / 32 - 1) / (T / 32);
  const int keys = (int)std::min<int64_t>((share + 127) / 128 * 4 * T, kMaxKeys);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(p.num_requests * ctas));
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = (size_t)keys * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static Kv4SmemLimit limit;
  return limit.launch(reinterpret_cast<const void*>(kern), kMaxKeys * 4, [&] {
    cudaError_t e = ctas > 8 ? cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                    cudaFuncAttributeNonPortableClusterSizeAllowed, 1)
                             : cudaSuccess;
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, p, keys) : e;
  });
}

cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t stream) {
  // CTAs of a request: as many as have 4096 tokens each, while two for every SM are not exceeded.  A cluster's
  // steps cost more than a CTA's, and a CTA that holds many tokens takes longer over them; with 2048 / 4096 / 8192
  // each one request of 4096 takes 13.6 / 12.2 / 12.2 us, of 16384 15 / 16 / 19, four of 16384 16.4 / 16.1 / 21.7,
  // 16 of 32768 32 / 20 / 22 us (and one CTA alone 146 us for 131072).
  const int64_t most = std::min((int64_t)p.table_width << p.page_shift, (int64_t)kKv4MaxLength);
  int ctas = 1;
  while (ctas < kMaxCluster && most > 4096ll * ctas && (int64_t)p.num_requests * ctas * 2 <= 256) ctas *= 2;
  // 512 threads where the requests' CTAs lie two on an SM, 256 where more wait for one: 256 requests of 4096 take
  // 16.5 us with 512 threads and 18.1 with 256, 512 of them 27.5 and 24.3.  (1024: 23 and 41.)
  if (p.num_requests > 304) return launch_evict<256>(p, ctas, most, stream);
  cudaError_t e = launch_evict<512>(p, ctas, most, stream);
  if (e != cudaSuccess && ctas > 8) {  // (a GPU, or a part of one, without 16 free SMs side by side)
    (void)cudaGetLastError();
    e = launch_evict<512>(p, 8, most, stream);
  }
  return e;
}

cudaError_t launch_kv4_move(int D, const Kv4MoveParams& p, cudaStream_t stream) {
  if (p.n == 0) return cudaSuccess;
  const int64_t threads = p.n * p.cache.Hkv * (D / 16);
  const unsigned blocks = (unsigned)std::min<int64_t>((threads + 255) / 256, 1 << 20);
  if (D == 64) kv4_move_kernel<64><<<blocks, 256, 0, stream>>>(p);
  else if (D == 128) kv4_move_kernel<128><<<blocks, 256, 0, stream>>>(p);
  else if (D == 256) kv4_move_kernel<256><<<blocks, 256, 0, stream>>>(p);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace ra
