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
//     is whole 16-byte words, loaded straight into registers;
//   * the work of all requests, 64 keys at a time, is one line that the grid's
//     CTAs cut into equal parts (lengths are on the device: the grid is fixed,
//     and each CTA finds its part from the lengths).  A unit (request, row
//     tile, head) that spans CTAs leaves partial results in the workspace, which
//     a second launch merges.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "kv4.h"
#include "tc.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockKeys = 16 * kWarps;  // keys of one block: a tile a warp
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634f;
// P's reference: a row's largest P is in (2^6, 2^7] when the reference moves,
// and it moves when a P would pass 2^15.
constexpr float kHeadroom = 7.f;
constexpr float kMaxExp = 15.f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Scale byte `i` of a word as fp16 in both halves; bytes i and j in low and high half.
__device__ __forceinline__ uint32_t scale_both(uint32_t w, int i) {
  return __byte_perm(w, 0, 0x0404 | (i << 4) | (i << 12)) >> 1;
}
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, int i, int j) {
  return __byte_perm(w, 0, 0x0404 | (i << 4) | (j << 12)) >> 1;
}

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Four columns of a finished row: O / l, and the row's log-sum-exp with the first.
__device__ __forceinline__ void kv4_write_row(const Kv4AttnParams& p, int token, int h, int D, int d4, float4 v,
                                              float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
  const size_t off = ((size_t)token * p.Hq + h) * D + 4 * d4;
  if (p.o_is_fp32)
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.o) + off) = v;
  else
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.o) + off) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  if (d4 == 0) p.lse[(size_t)h * p.Tq + token] = l == 0.f ? neg_inf() : (m + log2f(l)) * kLn2;
}

// What a CTA knows of a request.
struct Request {
  int b, n, L;     // first query row, query tokens, keys
  int row_tiles;
  int blocks;      // 64-key blocks of each of its units (at least one: empty rows are written too)
  int bad;
};

template <int RT>
__device__ __forceinline__ Request request(const Kv4AttnParams& p, int r) {
  Request q;
  int b = p.cu_q[r], e = p.cu_q[r + 1];
  int L = p.kv_lens[r];
  q.bad = 0;
  if (b < 0 || e < b || e > p.Tq) {
    q.bad = RA_KV4_BAD_OFFSET;
    b = min(max(b, 0), p.Tq);
    e = min(max(e, b), p.Tq);
  }
  const long long cap = (long long)p.table_width << p.cache.page_shift;
  if (L < 0 || L > cap) {
    q.bad = RA_KV4_BAD_LENGTH;
    L = L < 0 ? 0 : (int)cap;
  }
  q.b = b;
  q.n = e - b;
  q.L = L;
  const int G = p.Hq / p.cache.Hkv;
  q.row_tiles = (int)(((long long)q.n * G + RT - 1) / RT);
  q.blocks = max(1, (L + kBlockKeys - 1) / kBlockKeys);
  return q;
}
__device__ __forceinline__ long long request_work(const Request& q, int Hkv) {
  return (long long)q.row_tiles * Hkv * q.blocks;
}

// One warp's tile in registers.
template <int D>
struct TileRegs {
  uint4 k[D / 64], v[D / 64];
  uint32_t ks[D == 256 ? 2 : 1], vs[D == 256 ? 2 : 1];
};

template <int D>
__device__ __forceinline__ void load_tile(TileRegs<D>& t, const uint8_t* tile, int lane) {
  using L = Kv4Layout<D>;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    t.k[i] = ldg_stream(tile + L::kKCodes + 512 * i + 16 * lane);
    t.v[i] = ldg_stream(tile + L::kVCodes + 512 * i + 16 * lane);
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
  float m[NT][2], l[NT][2];
};

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

constexpr int ctas_per_sm(int D, int NT) { return D * NT <= 128 ? 4 : D * NT <= 256 ? 3 : 2; }

template <int D, int NT>
struct AttnCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;  // floats between rows of the merge buffer
  static constexpr int kSmem = kWarps * kRows * (kPitch + 2) * 4;
  static constexpr int kSlot = kRows * (D + 2);  // floats of a partial result: m, l, O
  // CTAs per SM (registers: 32 NT (D / 128) accumulators and half as many query words)
  static constexpr int kPerSm = ctas_per_sm(D, NT);
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (AttnCfg<D, NT>::kPerSm)) kv4_attn_kernel(const Kv4AttnParams p) {
  using C = AttnCfg<D, NT>;
  constexpr int RT = C::kRows;
  extern __shared__ float s_dyn[];
  float* s_o = s_dyn;                               // [kWarps][RT][kPitch]
  float* s_m = s_dyn + kWarps * RT * C::kPitch;     // [kWarps][RT]
  float* s_l = s_m + kWarps * RT;                   // [kWarps][RT]
  __shared__ long long s_sum[kWarps];
  __shared__ long long s_found[2];
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r8 = lane >> 2, c4 = lane & 3;
  const int G = p.Hq / p.cache.Hkv, Hkv = p.cache.Hkv;
  if (tid == 0) s_bad = 0;

  // ---- this CTA's part of the line of work
  long long total = 0;
  int bad = 0;
  for (int r = tid; r < p.R; r += kThreads) {
    const Request q = request<RT>(p, r);
    total += request_work(q, Hkv);
    bad = max(bad, q.bad);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  if (bad) atomicMax(&s_bad, bad);
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += s_sum[w];
  // no part is empty: a unit's partial results then lie in consecutive CTAs
  const long long cut = min((long long)gridDim.x, total);
  const bool idle = blockIdx.x >= cut;
  const long long begin = idle ? 0 : total * blockIdx.x / cut, end = idle ? 0 : total * (blockIdx.x + 1) / cut;
  long long base = 0;  // work before request r
  int r = 0;
  if (begin < end) {
    for (int r0 = 0; r0 < p.R; r0 += kThreads) {
      long long w = r0 + tid < p.R ? request_work(request<RT>(p, r0 + tid), Hkv) : 0;
      long long x = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = x;
      if (tid == 0) s_found[0] = -1;
      __syncthreads();
      long long before = base, chunk = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += s_sum[i];
        chunk += s_sum[i];
      }
      if (begin >= before + x - w && begin < before + x) {
        s_found[0] = r0 + tid;
        s_found[1] = before + x - w;
      }
      __syncthreads();
      if (s_found[0] >= 0) {
        r = (int)s_found[0];
        base = s_found[1];
        break;
      }
      base += chunk;
    }
  }

  Kv4Part part{};
  for (long long pos = begin; pos < end && r < p.R;) {
    const Request rq = request<RT>(p, r);
    const long long work = request_work(rq, Hkv);
    if (pos >= base + work) {  // (requests without rows have no work)
      base += work;
      ++r;
      continue;
    }
    const long long unit = (pos - base) / rq.blocks;
    const int blk0 = (int)(pos - base - unit * rq.blocks);
    const int nb = (int)min((long long)(rq.blocks - blk0), end - pos);
    const int rt = (int)(unit / Hkv), head = (int)(unit - (long long)rt * Hkv);
    const int row0 = rt * RT, rows = min(RT, rq.n * G - row0);

    // ---- query rows: fp16 operands, scales and key limits
    uint32_t qf[NT][D / 16][2];
    float sl2[NT][2];
    int lim[NT][2];
    auto limit = [&](int row) {
      return p.causal ? max(0, min(rq.L, rq.L - rq.n + row / G + 1)) : rq.L;
    };
    const int lim_min = limit(row0), lim_max = limit(row0 + rows - 1);
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
      // a power of two that brings the row's largest element to about 1; a row
      // of zeros or with an infinity or NaN stays as it is
      int ex = (int)(mx >> 7) - 127;
      ex = mx == 0 || mx >= 0x7f80 ? 0 : min(max(ex, -126), 126);
      const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
      const float down = __uint_as_float((uint32_t)(127 + ex) << 23);
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
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      acc.m[nt][0] = acc.m[nt][1] = neg_inf();
      acc.l[nt][0] = acc.l[nt][1] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.o[nt][d][i] = 0.f;
    }

    // ---- this warp's tiles: keys t0, t0 + 64, ...
    const int32_t* table = p.block_table + (size_t)r * p.table_stride;
    int t0 = blk0 * kBlockKeys + 16 * warp;
    const int t_end = min((blk0 + nb) * kBlockKeys, lim_max);
    auto page_of = [&](int t) -> int { return t < t_end ? table[t >> p.cache.page_shift] : 0; };
    auto fetch = [&](TileRegs<D>& t, int page, int tok) {
      // a page id outside the cache: read page 0, and mask the tile
      const int64_t pg = (uint32_t)page < (uint64_t)p.cache.num_pages ? page : 0;
      load_tile<D>(t, p.cache.pages + kv4_tile_offset<D>(p.cache, pg, head, tok & ((1 << p.cache.page_shift) - 1)),
                   lane);
    };
    TileRegs<D> next;
    int page = page_of(t0), page_next = page_of(t0 + kBlockKeys);
    if (t0 < t_end) fetch(next, page, t0);
    for (; t0 < t_end; t0 += kBlockKeys) {
      TileRegs<D> cur = next;
      const bool page_ok = (uint32_t)page < (uint64_t)p.cache.num_pages;
      if (!page_ok) bad = RA_KV4_BAD_PAGE;
      page = page_next;
      if (t0 + kBlockKeys < t_end) fetch(next, page, t0 + kBlockKeys);
      page_next = page_of(t0 + 2 * kBlockKeys);

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
        for (int j = 0; j < 2; ++j) {
          const uint32_t a[4] = {hmul2(lo[2 * j], sa), hmul2(hi[2 * j], sb), hmul2(lo[2 * j + 1], sa),
                                 hmul2(hi[2 * j + 1], sb)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a, qf[nt][2 * i + j]);
        }
      }
      // log2 units and the mask
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] *= sl2[nt][i & 1];
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
        for (int i = 0; i < 4; ++i) over |= s[nt][i] - kMaxExp > acc.m[nt][i & 1];
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mt = fmaxf(s[nt][e], s[nt][2 + e]);
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
            if (mt - kMaxExp > acc.m[nt][e]) {
              const float m_new = ceilf(mt) - kHeadroom;
              const float alpha = ex2_approx(acc.m[nt][e] - m_new);
              acc.m[nt][e] = m_new;
              acc.l[nt][e] *= alpha;
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
          const float m = acc.m[nt][i & 1];
          x[i] = ex2_approx(s[nt][i] - (m == neg_inf() ? 0.f : m));
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
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {hmul2(ev[0][j], sa), hmul2(od[0][j], sa), hmul2(ev[1][j], sb), hmul2(od[1][j], sb)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(acc.o[nt][4 * i + j], a, pf[nt]);
        }
      }
      if (masked && __any_sync(0xffffffffu, (nan0 | nan1) != 0)) add_nan<D, NT>(acc, nan0, nan1, t0, lim, lane);
    }

    // ---- merge the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = acc.l[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (r8 == 0) {
          s_m[warp * RT + 8 * nt + 2 * c4 + e] = acc.m[nt][e];
          s_l[warp * RT + 8 * nt + 2 * c4 + e] = l;
        }
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * nt + 2 * c4 + e;
        float mm = neg_inf();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * RT + row]);
        const float a = acc.m[nt][e] == neg_inf() ? 0.f : ex2_approx(acc.m[nt][e] - mm);
        float* dst = s_o + (warp * RT + row) * C::kPitch + r8 * (D / 8);
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
          *reinterpret_cast<float2*>(dst + 2 * d) = make_float2(acc.o[nt][d][e] * a, acc.o[nt][d][2 + e] * a);
      }
    __syncthreads();
    const bool starts = blk0 == 0, ends = blk0 + nb == rq.blocks;
    const bool direct = starts && ends;
    float* slot = p.partials + ((size_t)blockIdx.x * 2 + (starts ? 1 : 0)) * C::kSlot;
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d4 = i % (D / 4);
      float mm = neg_inf(), l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * RT + row]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = s_m[w * RT + row];
        l += mw == neg_inf() ? 0.f : s_l[w * RT + row] * ex2_approx(mw - mm);
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * RT + row) * C::kPitch + 4 * d4);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      if (direct) {
        kv4_write_row(p, rq.b + (row0 + row) / G, head * G + (row0 + row) % G, D, d4, v, mm, l);
      } else {
        *reinterpret_cast<float4*>(slot + 2 * RT + row * D + 4 * d4) = v;
        if (d4 == 0) {
          slot[row] = mm;
          slot[RT + row] = l;
        }
      }
    }
    if (starts && !ends) {
      part.request = r;
      part.row_tile = rt;
      part.head = head;
      // the CTA that holds the unit's last block
      const long long last = base + (unit + 1) * rq.blocks - 1;
      int c = (int)(last * cut / total);
      while (total * (c + 1) / cut <= last) ++c;
      while (total * c / cut > last) --c;
      part.parts = c - (int)blockIdx.x + 1;
    }
    __syncthreads();  // the merge buffers are free again
    pos += nb;
  }
  if (bad) atomicMax(&s_bad, bad);
  __syncthreads();
  if (tid == 0) {
    part.status = s_bad;
    p.parts[blockIdx.x] = part;
  }
}

// Merge the partial results of the units that span CTAs: block (c, row) the
// unit that CTA c began.  Block (0, 0) also gathers the CTAs' status.
template <int D>
__global__ void __launch_bounds__(256) kv4_merge_kernel(const Kv4AttnParams p, int rt_rows, int ctas) {
  constexpr int V = D / 32;
  __shared__ float s_o[8][D];
  __shared__ float s_l[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int st = 0;
    for (int c = tid; c < ctas; c += 256) st = max(st, p.parts[c].status);
    st = __reduce_max_sync(0xffffffffu, st);
    __shared__ int s_st[8];
    if (lane == 0) s_st[warp] = st;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < 8; ++w) st = max(st, s_st[w]);
      *p.status = st;
    }
  }
  const Kv4Part part = p.parts[blockIdx.x];
  if (part.parts == 0) return;
  const int G = p.Hq / p.cache.Hkv;
  int b = p.cu_q[part.request], e = p.cu_q[part.request + 1];
  b = min(max(b, 0), p.Tq);
  e = min(max(e, b), p.Tq);
  const int row = blockIdx.y, grow = part.row_tile * rt_rows + row;
  if (grow >= (e - b) * G) return;
  const size_t slot_floats = (size_t)rt_rows * (D + 2);
  auto slot = [&](int i) {
    return p.partials + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * slot_floats;
  };
  float mm = neg_inf();
  for (int i = lane; i < part.parts; i += 32) mm = fmaxf(mm, slot(i)[row]);
#pragma unroll
  for (int d = 16; d; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
  float o[V], l = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = 0.f;
  for (int i = warp; i < part.parts; i += 8) {
    const float* s = slot(i);
    const float m = s[row];
    const float a = m == neg_inf() ? 0.f : ex2_approx(m - mm);
    l += m == neg_inf() ? 0.f : s[rt_rows + row] * a;
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] += s[2 * rt_rows + row * D + 32 * j + lane] * a;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) s_o[warp][32 * j + lane] = o[j];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (tid < D / 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(&s_o[w][4 * tid]);
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      l += s_l[w];
    }
    kv4_write_row(p, b + grow / G, part.head * G + grow % G, D, tid, v, mm, l);
  }
}

template <int D, int NT>
cudaError_t launch(int ctas, const Kv4AttnParams& p, cudaStream_t stream) {
  using C = AttnCfg<D, NT>;
  auto kern = kv4_attn_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kThreads, C::kSmem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  kv4_merge_kernel<D><<<dim3(ctas, C::kRows), 256, 0, stream>>>(p, C::kRows, ctas);
  return cudaGetLastError();
}

}  // namespace

Kv4AttnShape kv4_attn_shape(int D, int G, int max_q_len, int sms) {
  const long long rows = (long long)G * max_q_len;
  int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 3;
  if (D == 256) nt = nt > 2 ? 2 : nt;
  return Kv4AttnShape{8 * nt, ctas_per_sm(D, nt) * (sms < kKv4MaxSms ? sms : kKv4MaxSms), (size_t)8 * nt * (D + 2)};
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
  if (D == 256 && nt == 2) return launch<256, 2>(s.ctas, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ra
