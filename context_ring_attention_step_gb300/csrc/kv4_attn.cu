// kv4_attn.cu -- attention of packed query rows over the paged 4-bit cache.
//
// With x_ij = scale q_i . k_j over the keys that row i sees,
//   lse_i = ln sum_j exp(x_ij),   o_i = sum_j exp(x_ij - lse_i) v_j,
// in one pass over the keys with a running reference m and a running sum:
// p_ij = 2^(x_ij log2 e - m), l += p, O += p v, and O, l times 2^(m - m') when
// the reference moves.  Partial results over disjoint keys merge the same way.
//
// What has to be read is the cache: 1.125 D bytes a token and head for 4 D
// flops a query row, so a decode step is bound by memory as long as expanding
// the codes costs less than reading them.  Hence:
//   * keys are the M side of the tensor-core product (S^T = K Q^T, and
//     O^T = V^T P^T): 16 tokens a tile against 8 query rows, so that the few
//     rows of a step (query tokens x query heads of a key/value head) waste
//     little of it;
//   * a code expands with one conversion (two codes to fp16 x 2) and one
//     multiplication by its scale.  The product has 6 significant bits and
//     a smallest step of 2^-18: exact in fp16.  Query rows go in as fp16 after
//     scaling by a power of two, which the softmax scale takes back: a bf16
//     number has 8 significant bits, so only elements below 2^-14 of the row's
//     largest lose any (less than 2^-25 of the largest).  P goes in as fp16
//     (half a step: 2^-12); its reference keeps the row's largest P between 2^6
//     and 2^15, so that keys down to 2^-20 of the largest keep all 11 bits;
//   * a tile's bytes lie in the order of the operand registers: a lane's share
//     is whole 16-byte words.  Lanes copy them into a ring in shared memory
//     (cp.async), a few tiles ahead, and read back only what they copied
//     themselves: no barrier and no branch stands between a tile's expansions
//     and its products, which the compiler mixes only inside one basic block;
//   * the work of all requests, 64 keys at a time, is one line that the grid's
//     CTAs cut into equal parts (lengths are on the device: the grid is fixed,
//     and each CTA finds its part from the lengths).  A unit (request, row
//     tile, head) that spans CTAs leaves partial results in the workspace, and
//     the CTA that brings the last one merges them (in the CTAs' order, so the
//     result does not depend on which one that is).
// What bounds it: with long caches the steady state reads 5.4 TB/s (4 x 131072
// tokens, 8 heads, head_dim 128: 604 MB in 112 us).  No pipe is full (ALU 51 %,
// issue 55 % of all cycles over 128 ragged requests): expanding and multiplying a
// 16-token tile alone takes 155 ns of each scheduler, 66 % of what it then takes
// in all, and with 12 warps an SM the fixed latencies between the steps of a tile
// stay in the open.  A single 131072-token
// request (151 MB, 22 us at the measured 6.78 TB/s) takes 41 us: about 7 us until
// the first tiles are there, 25 to 30 of reading, 6 for the two merges.  128
// ragged requests (579 MB): 117 us, 5.0 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "kv4.h"
#include "kv4_walk.cuh"
#include "tc.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
// What beginning a unit costs, in blocks of 64 keys: 128 ragged requests (lognormal
// lengths around 2000) take 172 us with 0, 140 with 4 and 8, 150 with 16.
constexpr int kUnit = 6;
constexpr int kFan = 8;    // partial results merged at once
constexpr int kAlone = 4;  // parts of a unit that one warp merges
constexpr int kThreads = 32 * kWarps;
constexpr int KB = 16 * kWarps;  // keys of one block: a tile a warp
// P's reference: a row's largest P is in (2^6, 2^7] when the reference moves,
// and it moves when a P would pass 2^15.
constexpr float kHeadroom = 7.f;
constexpr float kMaxExp = 15.f;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held one row a quad.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// One warp's tile in registers.
template <int D>
struct TileRegs {
  uint4 k[D / 64], v[D / 64];
  uint32_t ks[D == 256 ? 2 : 1], vs[D == 256 ? 2 : 1];
};

// Asynchronous copies of a lane's own words into its warp's ring; `n` bytes (all
// or none: then zeros) are read.  A lane reads back only what it copied itself, so
// that waiting for its own copies is all the synchronisation there is.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const uint8_t* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const uint8_t* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups are there
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint8_t* tile, bool in, int lane) {
  using L = Kv4Layout<D>;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    copy16(dst + L::kKCodes + 512 * i + 16 * lane, tile + L::kKCodes + 512 * i + 16 * lane, in ? 16 : 0);
    copy16(dst + L::kVCodes + 512 * i + 16 * lane, tile + L::kVCodes + 512 * i + 16 * lane, in ? 16 : 0);
  }
  if (D == 256) {
    copy8(dst + L::kKScales + 8 * lane, tile + L::kKScales + 8 * lane, in ? 8 : 0);
    copy8(dst + L::kVScales + 8 * lane, tile + L::kVScales + 8 * lane, in ? 8 : 0);
  } else {  // at head_dim 64 two lanes share a word, and both copy it
    const int k = D == 64 ? 2 * lane & ~3 : 4 * lane, v = D == 64 ? 4 * ((lane >> 3) * 4 + (lane & 3)) : 4 * lane;
    copy4(dst + L::kKScales + k, tile + L::kKScales + k, in ? 4 : 0);
    copy4(dst + L::kVScales + v, tile + L::kVScales + v, in ? 4 : 0);
  }
}
template <int D>
__device__ __forceinline__ void load_tile(TileRegs<D>& t, const uint8_t* tile, int lane) {
  using L = Kv4Layout<D>;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    t.k[i] = *reinterpret_cast<const uint4*>(tile + L::kKCodes + 512 * i + 16 * lane);
    t.v[i] = *reinterpret_cast<const uint4*>(tile + L::kVCodes + 512 * i + 16 * lane);
  }
  if (D == 64) {
    t.ks[0] = *reinterpret_cast<const uint16_t*>(tile + L::kKScales + 2 * lane);
    t.vs[0] = *reinterpret_cast<const uint32_t*>(tile + L::kVScales + 4 * ((lane >> 3) * 4 + (lane & 3)));
  } else if (D == 128) {
    t.ks[0] = *reinterpret_cast<const uint32_t*>(tile + L::kKScales + 4 * lane);
    t.vs[0] = *reinterpret_cast<const uint32_t*>(tile + L::kVScales + 4 * lane);
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(tile + L::kKScales + 8 * lane);
    const uint2 b = *reinterpret_cast<const uint2*>(tile + L::kVScales + 8 * lane);
    t.ks[0] = a.x; t.ks[D == 256 ? 1 : 0] = a.y;
    t.vs[0] = b.x; t.vs[D == 256 ? 1 : 0] = b.y;
  }
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// Word `i` of the run of K codes that a lane holds for token r + 8 h.
template <int D>
__device__ __forceinline__ uint32_t k_word(const TileRegs<D>& t, int h, int i) {
  if (D == 64) return word(t.k[0], 2 * h + i);
  if (D == 128) return word(t.k[h], i);
  return word(t.k[(2 * h + (i >> 2)) % (D / 64)], i & 3);
}
// Its scale of group g, in both halves.
template <int D>
__device__ __forceinline__ uint32_t k_scale2(const TileRegs<D>& t, int h, int g) {
  if (D == 64) return scale_both(t.ks[0], h);
  if (D == 128) return scale_both(t.ks[0], 2 * h + g);
  return scale_both(t.ks[h % (D == 256 ? 2 : 1)], g);
}
// Word `i` of the run of V codes that a lane holds for token 2c + e + 8 h.
template <int D>
__device__ __forceinline__ uint32_t v_word(const TileRegs<D>& t, int h, int e, int i) {
  if (D == 64) return word(t.v[0], 2 * h + e);
  if (D == 128) return word(t.v[h], 2 * e + i);
  return word(t.v[(2 * h + e) % (D / 64)], i);
}

template <int D, int NT>
struct Acc {
  float o[NT][D / 16][4];
  // the rows' reference (0 while a row has seen no key), the value of x - m that
  // moves it (-inf while the row has seen no key), and the running sum
  float m[NT][2], top[NT][2], l[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = 0.f;
      top[nt][0] = top[nt][1] = neg_inf();
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][d][i] = 0.f;
    }
  }
  __device__ __forceinline__ float ref(int nt, int e) const { return top[nt][e] == neg_inf() ? neg_inf() : m[nt][e]; }
};

// Add the warps' accumulators up in warp 0: all take the rows' largest
// reference, then half of those left hand theirs to the other half, until one is
// left; l, one sum a lane before, becomes the row's.  The buffers of the next call
// are other ones (ml) or are written behind its first barrier (so).
template <int D, int NT>
__device__ __forceinline__ void merge_warps(Acc<D, NT>& acc, float4 (&ml)[kWarps][NT][4], float4* so, int warp,
                                            int lane) {
  constexpr int F = NT * (D / 16);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      acc.l[nt][e] += __shfl_xor_sync(0xffffffffu, acc.l[nt][e], 4);
      acc.l[nt][e] += __shfl_xor_sync(0xffffffffu, acc.l[nt][e], 8);
      acc.l[nt][e] += __shfl_xor_sync(0xffffffffu, acc.l[nt][e], 16);
    }
    if (lane < 4) ml[warp][nt][lane] = make_float4(acc.ref(nt, 0), acc.ref(nt, 1), acc.l[nt][0], acc.l[nt][1]);
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float mm[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = ml[w][nt][lane & 3];
      mm[0] = fmaxf(mm[0], x.x);
      mm[1] = fmaxf(mm[1], x.y);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = ml[w][nt][lane & 3];
      // without a reference: no key (l = 0), or scores that are all NaN (l = NaN, which the row's l becomes)
      l[0] += x.x == neg_inf() ? x.z : x.z * ex2_approx(x.x - mm[0]);
      l[1] += x.y == neg_inf() ? x.w : x.w * ex2_approx(x.y - mm[1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float a = acc.ref(nt, e) == neg_inf() ? 0.f : ex2_approx(acc.ref(nt, e) - mm[e]);
      if (mm[e] != neg_inf()) {
        acc.m[nt][e] = mm[e];
        acc.top[nt][e] = kMaxExp;
      }
      acc.l[nt][e] = l[e];
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        acc.o[nt][d][e] *= a;
        acc.o[nt][d][2 + e] *= a;
      }
    }
  }
#pragma unroll
  for (int n = kWarps; n > 1; n = (n + 1) / 2) {
    const int half = (n + 1) / 2;
    if (n < kWarps) __syncthreads();
    if (warp >= half && warp < n) {
      float4* dst = so + (warp - half) * 32 * F + lane;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
          dst[32 * (nt * (D / 16) + d)] =
              make_float4(acc.o[nt][d][0], acc.o[nt][d][1], acc.o[nt][d][2], acc.o[nt][d][3]);
    }
    __syncthreads();
    if (warp < n - half) {
      const float4* src = so + warp * 32 * F + lane;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const float4 x = src[32 * (nt * (D / 16) + d)];
          acc.o[nt][d][0] += x.x; acc.o[nt][d][1] += x.y; acc.o[nt][d][2] += x.z; acc.o[nt][d][3] += x.w;
        }
    }
  }
}

// A finished unit's rows: O / l and the log-sum-exp, from warp 0's accumulators.
template <int D, int NT>
__device__ __forceinline__ void write_rows(const Kv4AttnParams& p, const Acc<D, NT>& acc, int b, int head, int row0,
                                           int rows, int G, int lane) {
  const int r8 = lane >> 2, c4 = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * nt + 2 * c4 + e;
      if (row >= rows) continue;
      const int token = b + (row0 + row) / G, h = head * G + (row0 + row) % G;
      const float l = acc.l[nt][e], inv = l == 0.f ? 0.f : 1.f / l;
      const size_t off = ((size_t)token * p.Hq + h) * D + r8 * (D / 8);
#pragma unroll
      for (int d = 0; d < D / 16; d += 4) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = acc.o[nt][d + i][e] * inv;
          v[2 * i + 1] = acc.o[nt][d + i][2 + e] * inv;
        }
        if (p.o_is_fp32) {
          float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.o) + off + 2 * d);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.o) + off + 2 * d) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        }
      }
      if (r8 == 0) p.lse[(size_t)h * p.Tq + token] = l == 0.f ? neg_inf() : (acc.m[nt][e] + log2f(l)) * kLn2;
    }
}

// O^T rows of dims whose V is NaN for a token that a row sees (only reached
// where a mask runs through the tile; elsewhere the product carries the NaN).
template <int D, int NT>
__device__ __forceinline__ void add_nan(Acc<D, NT>& acc, uint32_t nan0, uint32_t nan1, int t0, const int (&lim)[NT][2],
                                     int lane) {
  // nanG: bit i set: this lane's token i (2c, 2c+1, 2c+8, 2c+9) is NaN in its dims of group G
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const uint32_t m0 = __shfl_sync(0xffffffffu, nan0, (lane & ~3) + c);
    const uint32_t m1 = __shfl_sync(0xffffffffu, nan1, (lane & ~3) + c);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (t < lim[nt][e])
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
              if (((D == 256 && d >= 8 ? m1 : m0) >> i) & 1) {
                acc.o[nt][d][e] = quiet_nan();
                acc.o[nt][d][2 + e] = quiet_nan();
              }
    }
  }
}

// CTAs of four warps per SM: 128 registers a thread at four, 168 at three, 255 at
// two.  More registers beat more warps as soon as the compiler can use them: at
// head_dim 128 three CTAs take 126 us for 128 ragged requests, four 138, two 138;
// at 16 query rows two take 65 us over 131072 tokens, three 77 (they spill).
__host__ __device__ constexpr int ctas_per_sm(int D, int NT) {
  return D == 64 ? (NT == 1 ? 4 : 3) : D == 128 && NT == 1 ? 3 : 2;
}

template <int D, int NT>
struct AttnCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kPerSm = ctas_per_sm(D, NT);
  static constexpr int kFrag = NT * (D / 16);       // float4 accumulators of a lane
  static constexpr int kMerge = (kWarps / 2) * kFrag * 512;
  static constexpr int kFit = ((220 / kPerSm - 2) * 1024 - kMerge) / (kWarps * Kv4Layout<D>::kBytes);
  static constexpr int kMost = D == 64 ? 6 : D == 128 ? 4 : 3;
  static constexpr int kSlots = kFit > kMost ? kMost : kFit;  // ring of each warp
  static constexpr int kSmem = kSlots * kWarps * Kv4Layout<D>::kBytes + kMerge;
  static_assert(kSlots >= 3, "tiles under way");
  static constexpr int kSlot = (kFrag + NT) * 128;  // floats of a partial result
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (AttnCfg<D, NT>::kPerSm)) kv4_attn_kernel(const Kv4AttnParams p) {
  using C = AttnCfg<D, NT>;
  using L = Kv4Layout<D>;
  constexpr int RT = C::kRows, S = C::kSlots;
  extern __shared__ __align__(128) uint8_t s_dyn[];
  __shared__ __align__(16) float4 s_ml[2][kWarps][NT][4];  // m and l of a warp's rows, for two units in turn
  __shared__ long long s_sum[kWarps];
  __shared__ long long s_found[2];
  __shared__ int s_bad, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r8 = lane >> 2, c4 = lane & 3;
  const int G = p.Hq / p.cache.Hkv;
  uint8_t* ring = s_dyn + warp * S * L::kBytes;
  float4* s_o = reinterpret_cast<float4*>(s_dyn + kWarps * S * L::kBytes);  // [kWarps / 2][kFrag][32]
  if (tid == 0) s_bad = 0;

  int bad = 0;
  Kv4Walk wk;
  const Kv4Line line = kv4_find_part<RT, KB, kUnit, false, kThreads>(p, s_sum, s_found, wk, bad);

  int units = 0;
  while (wk.pos < line.end) {
    wk.enter<RT, KB, kUnit, false>(p, line.end);
    const Kv4Request& rq = wk.rq;
    const int blk0 = wk.blk, head = wk.head;
    const int nb = wk.nb;
    if (nb == 0) {
      wk.leave(line.end);
      continue;
    }
    const int row0 = wk.rt * RT, rows = min(RT, rq.n * G - row0);
    const int lim_min = kv4_key_limit(p, rq, row0), lim_max = wk.t_end;

    // ---- this warp's tiles: keys t0, t0 + KB, ...  S - 1 tiles are under way into
    // the ring while one is worked on, without a branch or a barrier: behind the
    // last tile, and for a page that is not one of the cache, zeros.  A slot is
    // filled again one tile after it was read.
    const int t_stop = min((blk0 + nb) * KB, lim_max);
    const int32_t* table = p.block_table + (size_t)wk.r * p.table_stride;
    const int tiles_mask = (1 << (p.cache.page_shift - 4)) - 1;
    const uint8_t* base = p.cache.pages + ((size_t)head << (p.cache.page_shift - 4)) * L::kBytes;
    auto page_of = [&](int t) -> int { return t < t_stop ? table[t >> p.cache.page_shift] : 0; };
    uint32_t oks = 0;  // bit i: the (i + 1)-th last tile asked for comes from a page of the cache
    auto ask = [&](int slot, int page, int tok) {
      const bool good = (uint32_t)page < (uint64_t)p.cache.num_pages;
      oks = oks << 1 | (good ? 1u : 0u);
      if (!good) bad = max(bad, (int)RA_KV4_BAD_PAGE);
      copy_tile<D>(smem_u32(ring) + slot, base + (int64_t)(good ? page : 0) * p.page_bytes + ((tok >> 4) & tiles_mask) * L::kBytes,
                   good && tok < t_stop, lane);
      copy_commit();
    };
    int t0 = blk0 * KB + 16 * warp;
    int page = page_of(t0 + (S - 1) * KB);
    {
      int pages[S - 1];
#pragma unroll
      for (int i = 0; i < S - 1; ++i) pages[i] = page_of(t0 + i * KB);
#pragma unroll
      for (int i = 0; i < S - 1; ++i) ask(i * L::kBytes, pages[i], t0 + i * KB);
    }

    // ---- query rows: fp16 operands, scales and key limits
    uint32_t qf[NT][D / 16][2];
    float sl2[NT][2];
    int lim[NT][2];
    auto limit = [&](int row) { return kv4_key_limit(p, rq, row); };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + 8 * nt + r8;
      uint4 w[D / 32];
      if (row < row0 + rows) {
        const uint4* src = reinterpret_cast<const uint4*>(
            reinterpret_cast<const __nv_bfloat16*>(p.q) + (size_t)(rq.b + row / G) * p.q_stride +
            (size_t)(head * G + row % G) * D + c4 * (D / 4));
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
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const uint32_t a = word(w[j / 2], 2 * (j & 1)), b = word(w[j / 2], 2 * (j & 1) + 1);
        qf[nt][j][0] = pack_f16x2(__uint_as_float(a << 16) * up, __uint_as_float(a & 0xffff0000u) * up);
        qf[nt][j][1] = pack_f16x2(__uint_as_float(b << 16) * up, __uint_as_float(b & 0xffff0000u) * up);
      }
      const float s = p.scale * kLog2e * down;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sl2[nt][e] = __shfl_sync(0xffffffffu, s, 4 * (2 * c4 + e));
        const int rr = row0 + 8 * nt + 2 * c4 + e;
        lim[nt][e] = rr < row0 + rows ? limit(rr) : lim_max;
      }
    }

    Acc<D, NT> acc;
    acc.clear();

    int slot = 0, slot_ask = (S - 1) * L::kBytes;
#pragma unroll 1
    for (; t0 < t_stop; t0 += KB) {
      copy_wait<S - 2>();
      TileRegs<D> cur;
      load_tile<D>(cur, ring + slot, lane);
      const bool page_ok = (oks >> (S - 2)) & 1;
      ask(slot_ask, page, t0 + (S - 1) * KB);
      slot_ask = slot;
      slot = slot == (S - 1) * L::kBytes ? 0 : slot + L::kBytes;
      page = page_of(t0 + S * KB);

      // S^T = K Q^T
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t lo[4], hi[4];
        kv4_code_pairs(k_word<D>(cur, 0, i), lo);
        kv4_code_pairs(k_word<D>(cur, 1, i), hi);
        const uint32_t sa = k_scale2<D>(cur, 0, i >> 1), sb = k_scale2<D>(cur, 1, i >> 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t a[4] = {hmul2(lo[2 * k], sa), hmul2(hi[2 * k], sb), hmul2(lo[2 * k + 1], sa),
                                 hmul2(hi[2 * k + 1], sb)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a, qf[nt][2 * i + k]);
        }
      }
      // x - m in log2 units, and the mask
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = fmaf(s[nt][i], sl2[nt][i & 1], -acc.m[nt][i & 1]);
      uint32_t nan0 = 0, nan1 = 0;
      const bool masked = t0 + 16 > lim_min || !page_ok;
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!page_ok || t0 + r8 + 8 * (i >> 1) >= lim[nt][i & 1]) s[nt][i] = neg_inf();
        // V of keys that no row sees counts as zero whatever the page holds, and
        // a NaN must not reach the rows that do not see its key through 0 x NaN
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 2 * c4 + (i & 1) + 8 * (i >> 1);
          const bool out = !page_ok || t >= lim_max;
#pragma unroll
          for (int g = 0; g < (D == 256 ? 2 : 1); ++g) {
            const bool nan = ((cur.vs[g] >> (8 * i)) & 0xffu) >= 0xf8u;
            if (nan && !out) (g ? nan1 : nan0) |= 1u << i;
            if (nan || out) cur.vs[g] &= ~(0xffu << (8 * i));
          }
        }
      }
      // does the reference still hold?
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) over |= fmaxf(s[nt][e], s[nt][2 + e]) > acc.top[nt][e];
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mt = fmaxf(s[nt][e], s[nt][2 + e]);
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
            if (mt > acc.top[nt][e]) {
              const float up = ceilf(mt) - kHeadroom;  // the reference moves by this much
              const float alpha = acc.top[nt][e] == neg_inf() ? 0.f : ex2_approx(-up);
              acc.m[nt][e] += up;
              acc.top[nt][e] = kMaxExp;
              acc.l[nt][e] *= alpha;
              s[nt][e] -= up;
              s[nt][2 + e] -= up;
#pragma unroll
              for (int d = 0; d < D / 16; ++d) {
                acc.o[nt][d][e] *= alpha;
                acc.o[nt][d][2 + e] *= alpha;
              }
            }
          }
      }
      // P^T as the B operand
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = ex2_approx(s[nt][i]);
          acc.l[nt][i & 1] += x[i];
        }
        pf[nt][0] = transpose8x8(pack_f16x2(x[0], x[1]));
        pf[nt][1] = transpose8x8(pack_f16x2(x[2], x[3]));
      }
      // O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < (D + 63) / 64; ++i) {
        uint32_t ev[2][4], od[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w0 = v_word<D>(cur, h, 0, i), w1 = v_word<D>(cur, h, 1, i);
          kv4_code_pairs((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), ev[h]);
          kv4_code_pairs(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), od[h]);
        }
        const uint32_t vs = cur.vs[D == 256 ? i >> 1 : 0];
        const uint32_t sa = scale_pair(vs, 0, 1), sb = scale_pair(vs, 2, 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a[4] = {hmul2(ev[0][k], sa), hmul2(od[0][k], sa), hmul2(ev[1][k], sb), hmul2(od[1][k], sb)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(acc.o[nt][4 * i + k], a, pf[nt]);
        }
      }
      if (masked && __any_sync(0xffffffffu, (nan0 | nan1) != 0)) add_nan<D, NT>(acc, nan0, nan1, t0, lim, lane);
    }

    copy_wait<0>();

    // ---- merge the warps; warp 0 then holds the segment's result
    merge_warps<D, NT>(acc, s_ml[units & 1], s_o, warp, lane);
    ++units;
    const bool direct = wk.whole();
    if (direct) {
      if (warp == 0) write_rows<D, NT>(p, acc, rq.b, head, row0, rows, G, lane);
    } else {
      // A partial result; the CTA that brings the last one merges them.
      const int c0 = line.owner(wk.first), parts = line.owner(wk.first + rq.blocks - 1) - c0 + 1;
      auto place = [&](int c) { return 2 * c + (c == c0 ? 1 : 0); };
      auto slot = [&](int i) { return reinterpret_cast<float4*>(p.partials + (size_t)place(c0 + i) * C::kSlot); };
      const int at = blockIdx.x - c0;
      if (warp == 0) {
        float4* dst = slot(at);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          dst[32 * nt + lane] = make_float4(acc.ref(nt, 0), acc.ref(nt, 1), acc.l[nt][0], acc.l[nt][1]);
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
            dst[32 * (NT + nt * (D / 16) + d) + lane] =
                make_float4(acc.o[nt][d][0], acc.o[nt][d][1], acc.o[nt][d][2], acc.o[nt][d][3]);
        }
        __threadfence();
        __syncwarp();
      }
      // the rows' largest reference over `count` partial results, `stride` apart
      auto largest = [&](float (&mm)[NT][2], int from, int count, int stride) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mm[nt][0] = mm[nt][1] = neg_inf();
          for (int i = r8; i < count; i += 8) {
            const float4 ml = __ldcg(slot(from + i * stride) + 32 * nt + lane);
            mm[nt][0] = fmaxf(mm[nt][0], ml.x);
            mm[nt][1] = fmaxf(mm[nt][1], ml.y);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mm[nt][e] = fmaxf(mm[nt][e], __shfl_xor_sync(0xffffffffu, mm[nt][e], d));
        }
      };
      // (0 times an l that is NaN, where every score was NaN, stays NaN)
      auto weight = [](float m, float mm) { return m == neg_inf() ? 0.f : ex2_approx(m - mm); };
      if (parts <= kAlone) {
        // few parts: warp 0's business alone; the others go on meanwhile
        bool is_last = false;
        if (warp == 0 && lane == 0) {
          int* ticket = p.tickets + place(c0);
          is_last = atomicAdd(ticket, 1) == parts - 1;
          if (is_last) *ticket = 0;  // as the next call expects it
        }
        if (__shfl_sync(0xffffffffu, is_last, 0)) {
          __threadfence();
          float mm[NT][2];
          largest(mm, 0, parts, 1);
          acc.clear();
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (mm[nt][e] != neg_inf()) {
                acc.m[nt][e] = mm[nt][e];
                acc.top[nt][e] = kMaxExp;
              }
#pragma unroll 1
          for (int i = 0; i < parts; ++i) {
            const float4* src = slot(i);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float4 ml = __ldcg(src + 32 * nt + lane);
              const float w0 = weight(ml.x, mm[nt][0]), w1 = weight(ml.y, mm[nt][1]);
              acc.l[nt][0] = fmaf(ml.z, w0, acc.l[nt][0]);
              acc.l[nt][1] = fmaf(ml.w, w1, acc.l[nt][1]);
#pragma unroll
              for (int d = 0; d < D / 16; ++d) {
                const float4 x = __ldcg(src + 32 * (NT + nt * (D / 16) + d) + lane);
                acc.o[nt][d][0] = fmaf(x.x, w0, acc.o[nt][d][0]);
                acc.o[nt][d][1] = fmaf(x.y, w1, acc.o[nt][d][1]);
                acc.o[nt][d][2] = fmaf(x.z, w0, acc.o[nt][d][2]);
                acc.o[nt][d][3] = fmaf(x.w, w1, acc.o[nt][d][3]);
              }
            }
          }
          write_rows<D, NT>(p, acc, rq.b, head, row0, rows, G, lane);
        }
      } else {
        // many: by neighbours of kFan, then those; each warp takes a quarter of the columns
        constexpr int DW = D / 64;
        int from = at / kFan * kFan, count = min(kFan, parts - from), stride = 1;
        int* ticket = p.tickets + place(c0 + from);
#pragma unroll 1
        for (;;) {
          __syncthreads();  // the slot is written (and s_last was read)
          if (tid == 0) {
            s_last = atomicAdd(ticket, 1) == count - 1;
            if (s_last) *ticket = 0;
          }
          __syncthreads();
          if (!s_last) break;
          __threadfence();
          float mm[NT][2], l[NT][2];
          largest(mm, from, count, stride);
          float4 o[NT][DW];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int d = 0; d < DW; ++d) o[nt][d] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll 8
          for (int i = 0; i < count; ++i) {
            const float4* src = slot(from + i * stride);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float4 ml = __ldcg(src + 32 * nt + lane);
              const float w0 = weight(ml.x, mm[nt][0]), w1 = weight(ml.y, mm[nt][1]);
              l[nt][0] = fmaf(ml.z, w0, l[nt][0]);
              l[nt][1] = fmaf(ml.w, w1, l[nt][1]);
#pragma unroll
              for (int d = 0; d < DW; ++d) {
                const float4 x = __ldcg(src + 32 * (NT + nt * (D / 16) + warp * DW + d) + lane);
                o[nt][d].x = fmaf(x.x, w0, o[nt][d].x);
                o[nt][d].y = fmaf(x.y, w1, o[nt][d].y);
                o[nt][d].z = fmaf(x.z, w0, o[nt][d].z);
                o[nt][d].w = fmaf(x.w, w1, o[nt][d].w);
              }
            }
          }
          if (stride > 1 || parts <= kFan) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int row = 8 * nt + 2 * c4 + e;
                if (row >= rows) continue;
                const int token = rq.b + (row0 + row) / G, h = head * G + (row0 + row) % G;
                const float sum = l[nt][e], inv = sum == 0.f ? 0.f : 1.f / sum;
                const size_t off = ((size_t)token * p.Hq + h) * D + r8 * (D / 8) + 2 * warp * DW;
#pragma unroll
                for (int d = 0; d < DW; ++d) {
                  const float x = (e ? o[nt][d].y : o[nt][d].x) * inv, y = (e ? o[nt][d].w : o[nt][d].z) * inv;
                  if (p.o_is_fp32)
                    *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.o) + off + 2 * d) = make_float2(x, y);
                  else
                    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.o) + off + 2 * d) = pack_bf16x2(x, y);
                }
                if (warp == 0 && r8 == 0)
                  p.lse[(size_t)h * p.Tq + token] = sum == 0.f ? neg_inf() : (mm[nt][e] + log2f(sum)) * kLn2;
              }
            break;
          }
          float4* dst = slot(from);  // (read above by other warps too: they are done behind the barrier)
          __syncthreads();
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (warp == 0) dst[32 * nt + lane] = make_float4(mm[nt][0], mm[nt][1], l[nt][0], l[nt][1]);
#pragma unroll
            for (int d = 0; d < DW; ++d) dst[32 * (NT + nt * (D / 16) + warp * DW + d) + lane] = o[nt][d];
          }
          __threadfence();
          from = 0;
          count = (parts + kFan - 1) / kFan;
          stride = kFan;
          ticket = p.tickets + 2 * gridDim.x + c0;
        }
      }
    }
    wk.leave(line.end);
  }
  if (bad) atomicMax(&s_bad, bad);
  __syncthreads();
  if (tid == 0) kv4_end(p, s_bad);
}

template <int D, int NT>
cudaError_t launch(int ctas, const Kv4AttnParams& p, cudaStream_t stream) {
  using C = AttnCfg<D, NT>;
  auto kern = kv4_attn_kernel<D, NT>;
  static Kv4SmemLimit limit;
  return limit.launch(reinterpret_cast<const void*>(kern), C::kSmem, [&] {
    kern<<<ctas, kThreads, C::kSmem, stream>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace

Kv4AttnShape kv4_attn_shape(int D, long long rows, int sms) {
  int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 3;
  if (D == 256) nt = 1;
  return Kv4AttnShape{8 * nt, ctas_per_sm(D, nt) * (sms < kKv4MaxSms ? sms : kKv4MaxSms), (size_t)8 * nt * (D + 16)};
}

cudaError_t launch_kv4_attn(int D, const Kv4AttnShape& s, const Kv4AttnParams& p, cudaStream_t stream) {
  const int nt = s.rows / 8;
  if (D == 64 && nt == 1) return launch<64, 1>(s.ctas, p, stream);
  if (D == 64 && nt == 2) return launch<64, 2>(s.ctas, p, stream);
  if (D == 64 && nt == 3) return launch<64, 3>(s.ctas, p, stream);
  if (D == 128 && nt == 1) return launch<128, 1>(s.ctas, p, stream);
  if (D == 128 && nt == 2) return launch<128, 2>(s.ctas, p, stream);
  if (D == 128 && nt == 3) return launch<128, 3>(s.ctas, p, stream);
  if (D == 256 && nt == 1) return launch<256, 1>(s.ctas, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ra
