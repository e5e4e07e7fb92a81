// kv4_weights.cu -- the attention weight that every cached token receives from a
// step's query rows, over the paged 4-bit cache, for requests with few rows.
//
// With x_ij = scale q_i . k_j for the rows i (query tokens x query heads) that see
// key j, and their log-sum-exp known from the attention call,
//   w_j += sum over i of exp(x_ij - lse_i).
// A key's sum needs no other key: there is no running maximum, nothing to merge,
// and a key belongs to one warp for all heads and rows, so the order of its
// additions is fixed.
//
// What has to be read are the codes of the keys: 0.5625 D bytes a token and head
// for 2 D flops and one exponential a row: 128 requests of 4000 tokens on average, 4 rows a head at
// head_dim 128, take 73 us, 4.0 TB/s; a tile and head costs 190 instructions of a warp (a third of them
// the expansion), and the schedulers issue 64 % of the time.  As in kv4_attn.cu keys are the M side
// of the product (16 tokens x 8 rows), a lane's codes are whole words that it
// copies through a ring of its own, and a code expands with one conversion and one
// multiplication; asked for early in registers instead of the ring, the same call took 103 us,
// and with three CTAs on an SM in place of four 78.  A tile is expanded once for all row tiles; those lie in shared
// memory in the order of the operand registers.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "kv4.h"
#include "kv4_mma.cuh"
#include "kv4_walk.cuh"
#include "tc.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int KB = 16 * kWarps;  // keys of one block: a tile a warp
constexpr int kExpandCost = 3;   // expanding a tile, in row tiles

template <int D>
struct WeightsCfg {
  static constexpr int kPerSm = D == 256 ? 2 : 4;      // CTAs on an SM
  static constexpr int kTile = 9 * D;                  // bytes of a tile's keys: codes, then scales
  static constexpr int kSlots = D == 256 ? 6 : 8;      // ring of each warp
  static constexpr int kQTile = 16 * D;                // bytes of eight rows in fp16
  static constexpr int kCap = D == 64 ? 28 : D == 128 ? 8 : 12;  // row tiles in shared memory at once
  static constexpr int kRing = kWarps * kSlots * kTile;
  static constexpr int kSmem = kRing + kCap * (kQTile + 8 * 12);
  static_assert(kSmem <= (220 / kPerSm - 1) * 1024, "CTAs on an SM");
  static_assert(Kv4Layout<D>::kKCodes == 0 && Kv4Layout<D>::kKScales == 8 * D, "keys lie at a tile's start");
};

// Copy a lane's words of a tile's keys: codes from `k`, scales from `s` (the lane's own),
// to the tile's place in the ring (`dst`; at head_dim 64 two lanes share a word of scales,
// and both copy it).
template <int D>
__device__ __forceinline__ void copy_keys(uint32_t dst, const uint8_t* k, const uint8_t* s, int lane) {
  constexpr int kS = Kv4Layout<D>::kKScales;
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * i + 16 * lane), "l"(k + 512 * i) : "memory");
  if (D == 256)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + kS + 8 * lane), "l"(s) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + kS + (D == 64 ? 2 * lane & ~3 : 4 * lane)), "l"(s)
                 : "memory");
}
template <int D>
__device__ __forceinline__ void load_keys(KeyRegs<D>& t, const uint8_t* tile, int lane) {
  using L = Kv4Layout<D>;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) t.k[i] = *reinterpret_cast<const uint4*>(tile + 512 * i + 16 * lane);
  if (D == 64) {
    t.ks[0] = *reinterpret_cast<const uint16_t*>(tile + L::kKScales + 2 * lane);
  } else if (D == 128) {
    t.ks[0] = *reinterpret_cast<const uint32_t*>(tile + L::kKScales + 4 * lane);
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(tile + L::kKScales + 8 * lane);
    t.ks[0] = a.x;
    t.ks[D == 256 ? 1 : 0] = a.y;
  }
}
// A tile's keys as the A operands of its D / 16 products.
template <int D>
__device__ __forceinline__ void expand_keys(const KeyRegs<D>& t, uint32_t (&a)[D / 16][4]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t lo[4], hi[4];
    kv4_code_pairs(k_word<D>(t, 0, i), lo);
    kv4_code_pairs(k_word<D>(t, 1, i), hi);
    const uint32_t sa = k_scale2<D>(t, 0, i >> 1), sb = k_scale2<D>(t, 1, i >> 1);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[2 * i + k][0] = hmul2(lo[2 * k], sa);
      a[2 * i + k][1] = hmul2(hi[2 * k], sb);
      a[2 * i + k][2] = hmul2(lo[2 * k + 1], sa);
      a[2 * i + k][3] = hmul2(hi[2 * k + 1], sb);
    }
  }
}

// What a request asks of this kernel: blocks [i0, i1) of 64 keys, each `cost` places
// of the line of work.
struct Job {
  Kv4Request rq;
  int fresh;  // keys from here on begin at zero
  int i0, i1;
  long long cost;
};
__device__ __forceinline__ Job job_of(const Kv4WeightsParams& p, int r) {
  Job j;
  j.rq = kv4_request<8, KB, false>(p.a, r);
  const int L = j.rq.L;
  const int added = p.new_lens ? min(max(p.new_lens[r], 0), L) : 0;
  j.fresh = L - added;
  j.i0 = j.rq.n > 0 ? 0 : j.fresh / KB;
  j.i1 = (L + KB - 1) / KB;
  if (j.rq.n == 0 && added == 0) j.i0 = j.i1;         // nothing to do
  if (j.rq.n > 0 && j.rq.row_tiles == 0) j.i0 = j.i1;  // the other kernel's
  j.cost = j.rq.n > 0 ? (long long)p.a.cache.Hkv * (j.rq.row_tiles + kExpandCost) : 1;
  return j;
}

template <int D>
__global__ void __launch_bounds__(kThreads, (WeightsCfg<D>::kPerSm)) kv4_weights_kernel(const Kv4WeightsParams wp) {
  using C = WeightsCfg<D>;
  using L = Kv4Layout<D>;
  constexpr int S = C::kSlots;
  const Kv4AttnParams& p = wp.a;
  extern __shared__ __align__(128) uint8_t s_dyn[];
  __shared__ long long s_sum[kWarps], s_found[2];
  __shared__ int s_bad, s_lim_min;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r8 = lane >> 2, c4 = lane & 3;
  const int G = p.Hq / p.cache.Hkv, P = 1 << p.cache.page_shift;
  const uint8_t* ring = s_dyn + warp * S * C::kTile;
  const uint32_t ring_at = smem_u32(ring);
  uint4* s_q = reinterpret_cast<uint4*>(s_dyn + C::kRing);                                // [kCap][D / 32][32]
  float2* s_row = reinterpret_cast<float2*>(s_dyn + C::kRing + C::kCap * C::kQTile);  // [kCap][8] scale, - lse (log2)
  int* s_lim = reinterpret_cast<int*>(s_row + 8 * C::kCap);                      // [kCap][8] keys that the row sees
  if (tid == 0) s_bad = 0;

  int bad = 0;
  auto work = [&](int r) {
    const Job j = job_of(wp, r);
    bad = max(bad, j.rq.bad);
    return (long long)(j.i1 - j.i0) * j.cost;
  };
  int r;
  long long base;
  const Kv4Line line = kv4_cut<kThreads>(p.R, work, s_sum, s_found, r, base);

  // a block belongs to the CTA in whose part it begins
  for (; base < line.end && r < p.R; ++r) {
    const Job job = job_of(wp, r);
    const Kv4Request& rq = job.rq;
    const long long here = base;
    base += (long long)(job.i1 - job.i0) * job.cost;
    const int b0 = job.i0 + (int)kv4_div(max(line.begin - here, 0ll) + job.cost - 1, job.cost);
    const int b1 = min((long long)job.i1, job.i0 + kv4_div(line.end - here + job.cost - 1, job.cost));
    if (b0 >= b1) continue;
    const int32_t* table = p.block_table + (size_t)r * p.table_stride;
    // this warp's tiles of those blocks
    const int e1 = min(b1, (rq.L - 16 * warp + KB - 1) / KB);
    auto page_of = [&](int i) -> int { return i < e1 ? table[(i * KB + 16 * warp) >> p.cache.page_shift] : 0; };

    const int RT = rq.row_tiles, cap_t = min(RT, C::kCap), cap_h = RT == 0 ? 1 : max(1, min(p.cache.Hkv, C::kCap / RT));
    // heads by heads (and, of very many rows, row tiles by row tiles) that fit shared memory
    bool first = true;
    for (int h0 = 0; h0 < (RT == 0 ? 1 : p.cache.Hkv); h0 += cap_h) {
      const int nh = RT == 0 ? 0 : min(cap_h, p.cache.Hkv - h0);
      for (int t0 = 0; t0 == 0 || t0 < RT; t0 += cap_t) {
        const int nt = min(cap_t, RT - t0);
        // ---- query rows: fp16 after a power of two, as in kv4_attn.cu
        __syncthreads();
        if (tid == 0) s_lim_min = 0x7fffffff;
        __syncthreads();
        for (int k = warp; k < nh * nt; k += kWarps) {
          const int head = h0 + k / nt, row = 8 * (t0 + k % nt) + r8;
          const bool valid = row < rq.n * G;
          const int token = rq.b + (valid ? row / G : 0), h = head * G + row % G;
          uint4 w[D / 32];
          if (valid) {
            const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                              (size_t)token * p.q_stride + (size_t)h * D + c4 * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) w[i] = src[i];
          } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = __vmaxu2(mx, word(w[i], j) & 0x7fff7fffu);
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          float up;
          const float down = kv4_row_scale(mx, up);
          auto cvt = [&](uint32_t x) {
            return pack_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
          };
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            s_q[(k * (D / 32) + i) * 32 + lane] = make_uint4(cvt(w[i].x), cvt(w[i].y), cvt(w[i].z), cvt(w[i].w));
          if (c4 == 0) {
            // rows that are none, or have no softmax (lse = -inf: they see no key), see no key here
            const float lse = valid ? wp.lse[(size_t)h * p.Tq + token] : neg_inf();
            const bool dead = lse == neg_inf();
            const int lim = dead ? 0 : kv4_key_limit(p, rq, row);
            s_row[8 * k + r8] = dead ? make_float2(0.f, neg_inf()) : make_float2(p.scale * kLog2e * down, -lse * kLog2e);
            s_lim[8 * k + r8] = lim;
            if (valid) atomicMin(&s_lim_min, lim);
          }
        }
        __syncthreads();
        const int lim_min = s_lim_min;

        // ---- this warp's (tile, head) pairs, S - 1 of them under way in the warp's ring
        const size_t head_bytes = (size_t)L::kBytes << (p.cache.page_shift - 4);
        int ai = b0, ah = 0, page = page_of(b0), page_next = page_of(b0 + 1);
        const uint8_t *kp, *sp;
        auto aim = [&]() {  // at the first head of tile `ai`; a page that is none: somewhere in the cache
          const uint8_t* tile = p.cache.pages + (int64_t)((uint32_t)page < (uint64_t)p.cache.num_pages ? page : 0) * p.page_bytes +
                                h0 * head_bytes + (((ai * KB + 16 * warp) & (P - 1)) >> 4) * L::kBytes;
          kp = tile + 16 * lane;
          sp = tile + L::kKScales + (D == 64 ? 2 * lane & ~3 : (D / 32) * lane);
        };
        aim();
        uint32_t slot_ask = 0;
        auto ask = [&]() {  // (behind the last tile: that again, unused)
          copy_keys<D>(ring_at + slot_ask, kp, sp, lane);
          copy_commit();
          slot_ask = slot_ask == (S - 1) * C::kTile ? 0 : slot_ask + C::kTile;
          if (++ah < nh) {
            kp += head_bytes;
            sp += head_bytes;
          } else if (ai + 1 < e1) {
            ah = 0;
            ++ai;
            page = page_next;
            page_next = page_of(ai + 1);
            aim();
          }
        };
        int i = b0, mine = page;
        float sum0 = 0.f, sum1 = 0.f, old = 0.f;
        float* dst = nullptr;
        // lanes c4 < 2 hand in token r8 + 8 c4 of the tile
        const int off = r8 + 8 * (c4 & 1);
        auto begin = [&]() {
          const bool good = (uint32_t)mine < (uint64_t)p.cache.num_pages;
          if (!good) bad = max(bad, (int)RA_KV4_BAD_PAGE);
          const int out = i * KB + 16 * warp + off;
          dst = good && c4 < 2 && out < rq.L ? wp.weights + ((int64_t)mine << p.cache.page_shift) + (out & (P - 1)) : nullptr;
          const bool fresh = out >= job.fresh;
          old = dst && !(first && fresh) ? *dst : 0.f;
          if (nh == 0 && !fresh) dst = nullptr;
          mine = page_of(i + 1);
          sum0 = sum1 = 0.f;
        };
        auto end = [&]() {
          sum0 += __shfl_xor_sync(0xffffffffu, sum0, 1);
          sum1 += __shfl_xor_sync(0xffffffffu, sum1, 1);
          sum0 += __shfl_xor_sync(0xffffffffu, sum0, 2);
          sum1 += __shfl_xor_sync(0xffffffffu, sum1, 2);
          if (dst) *dst = old + (c4 == 0 ? sum0 : sum1);
        };
        // a tile's keys of one head against all rows of it
        int slot = 0;
        auto products = [&](int hh) {
          const int tok = i * KB + 16 * warp;
          const bool masked = tok + 16 > lim_min;
          copy_wait<S - 2>();
          uint32_t a[D / 16][4];
          KeyRegs<D> keys;
          load_keys<D>(keys, ring + slot, lane);
          slot = slot == (S - 1) * C::kTile ? 0 : slot + C::kTile;
          expand_keys<D>(keys, a);
          ask();
          const uint4* q = s_q + hh * nt * D + lane;
          const float2* rows = s_row + hh * nt * 8 + 2 * c4;
#pragma unroll 1
          for (int t = 0; t < nt; ++t, q += D, rows += 8) {
            float c[2][4] = {}, e[4];
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              const uint4 w = q[32 * j];
              const uint32_t x[2] = {w.x, w.y}, y[2] = {w.z, w.w};
              mma16816(c[0], a[2 * j], x);
              mma16816(c[1], a[2 * j + 1], y);
            }
            const float4 row = *reinterpret_cast<const float4*>(rows);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              e[v] = ex2_approx(fmaf(c[0][v] + c[1][v], v & 1 ? row.z : row.x, v & 1 ? row.w : row.y));
            if (masked) {
              const int2 lim = *reinterpret_cast<const int2*>(s_lim + (hh * nt + t) * 8 + 2 * c4);
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (tok + r8 + 8 * (v >> 1) >= (v & 1 ? lim.y : lim.x)) e[v] = 0.f;
            }
            sum0 += e[0] + e[1];
            sum1 += e[2] + e[3];
          }
        };
        if (nh > 0 && i < e1) {
#pragma unroll
          for (int u = 0; u < S - 1; ++u) ask();
        }
#pragma unroll 1
        for (; i < e1; ++i) {
          begin();
#pragma unroll 1
          for (int hh = 0; hh < nh; ++hh) products(hh);
          end();
        }
        copy_wait<0>();
        first = false;
        if (RT == 0) break;
      }
    }
  }
  if (bad) atomicMax(&s_bad, bad);
  __syncthreads();
  if (tid == 0) kv4_end(p, s_bad);
}

template <int D>
cudaError_t launch(int sms, const Kv4WeightsParams& p, cudaStream_t stream) {
  using C = WeightsCfg<D>;
  auto kern = kv4_weights_kernel<D>;
  static Kv4SmemLimit limit;
  return limit.launch(reinterpret_cast<const void*>(kern), C::kSmem, [&] {
    kern<<<C::kPerSm * sms, kThreads, C::kSmem, stream>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_kv4_weights(int D, int sms, const Kv4WeightsParams& p, cudaStream_t stream) {
  if (D == 64) return launch<64>(sms, p, stream);
  if (D == 128) return launch<128>(sms, p, stream);
  if (D == 256) return launch<256>(sms, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ra
