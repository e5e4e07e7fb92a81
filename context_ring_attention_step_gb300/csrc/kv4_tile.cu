// kv4_tile.cu -- attention over the paged 4-bit cache for requests with many
// query rows (the next part of a prompt over what is cached), on tcgen05 tensor
// cores.  Formulas as in kv4_attn.cu.
//
// Here the products dominate: 4 D flops a row and key against 1.125 D bytes a
// key.  A CTA takes 256 query rows (tokens x query heads of one key/value head)
// as two 128-row tiles, so that a key tile is expanded once for both; four warps
// expand it from registers into the swizzled shared-memory layout that the
// tensor cores read, ahead of the products.
// Measured: 1024 tokens over 33792 (32 query heads, 8 key/value heads, head_dim
// 128) in 555 us, 1010 TFLOP/s; tensor pipe 41 % of all cycles.  Without the
// expansion (timed once, results wrong) it would be 474 us, the rate of the ring
// forward, where the softmax of one Q tile beside the other's products sets the
// period; the expanding warps share its schedulers and the shared-memory bandwidth.
// A unit of few key tiles costs about 16 us besides them (query rows, first tiles
// and output follow one another): 32 prompts of 256 tokens and 32 heads take 171 us.

// Warp roles (512 threads):
//   warps 0, 1    UMMA issuers of Q tiles 0 and 1 (warp 0 owns tensor memory)
//   warps 4-11    softmax, output and merge of Q tile 0 (4-7) and 1 (8-11); a
//                 thread is a row, and loads it: fp16 after a power of two
//   warps 12-15   cache tiles -> fp16 K and V tiles in a ring of stages
// At head_dim 256, whose O alone takes half of tensor memory, there is one Q tile;
// warps 8-11 expand too.
// Tensor memory (512 columns): S0 [0,128), S1 [128,256), O0, O1 behind them; P
// (fp16) overwrites the first 64 columns of its S and feeds P.V from there.
// Stages hold K(0), V(0), K(1), V(1), ...; both issuers release each of them.
// The CTAs cut the line of work evenly and merge partial results as in
// kv4_attn.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "kv4.h"
#include "kv4_walk.cuh"
#include "tc.cuh"

namespace ra {
namespace {

constexpr int kKeys = 128;
constexpr int kThreads = 512;
constexpr int kFan = 8;  // partial results merged at once
constexpr int kUnit = 1;  // what beginning a unit costs, in blocks of 128 keys
// Polls of a wait for the other Q tile's turn.  In us, for 0, 6, 64 and 4096: one unit of many
// key tiles (1024 tokens over 33792) 575, 548, 545, 542; several short units a CTA (16 parts of
// 280 over 900, 32 / 8 heads) 181, 187, 225, 225: there the two are often a unit apart.
constexpr int kTurnLimit = 6;
constexpr int kSegs = 8;  // segments (and key tiles) that the expanding warps may be ahead, rounded up
// P's reference as in kv4_attn.cu: the row's largest P is in (2^6, 2^7] when it
// moves.  A tile whose P's add up to no more than 2^15 needs no look at its maximum.
constexpr float kHeadroom = 7.f;
constexpr float kMaxExp = 14.f;
constexpr float kSumLimit = 32768.f;

// fp16 x fp16 -> fp32 (formats 0 where idesc_bf16_f32 has 1)
constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int D>
struct TileCfg {
  static constexpr int kQt = D == 256 ? 1 : 2;  // 128-row Q tiles (tensor memory: 128 + D columns each)
  static constexpr int kRows = 128 * kQt;
  static constexpr int kSoft = 4 * kQt;         // softmax warps, then the expanding ones
  static constexpr int kExpand = 12 - kSoft;
  static constexpr int kSubs = 8 / kExpand;     // cache tiles of a key tile that an expanding warp takes
  static constexpr int kTile = 128 * D * 2;  // bytes of one 128-row fp16 tile
  static constexpr int kStages = D == 256 ? 2 : D == 128 ? 5 : 8;
  static constexpr int kQBytes = kQt * kTile;
  static constexpr int kBarOff = kQBytes + kStages * kTile;
  static constexpr int kSmem = kBarOff + 1024 + 1024;  // barriers and notes, alignment slack
  static constexpr int kSlot = kRows * (D + 2);        // floats of a partial result: m, l, O
  static constexpr uint32_t kIdescQK = idesc_f16_f32(128, 128, false);
  static constexpr uint32_t kIdescPV = idesc_f16_f32(128, D, true);
};

// What all roles know of a segment.
struct Segment {
  int k0, row0, rows;  // first key; first row of the unit, rows
  int n;                   // key tiles that some row sees
  int na[2];               // of these, those that a row of Q tile 0 / 1 sees (a prefix)
  int lim_lo[2];           // keys that the tile's first row sees
};

template <int kQt>
__device__ __forceinline__ Segment segment(const Kv4AttnParams& p, const Kv4Walk& wk) {
  constexpr int kRows = 128 * kQt;
  Segment s;
  const int G = p.Hq / p.cache.Hkv;
  s.k0 = wk.blk * kKeys;
  s.row0 = wk.rt * kRows;
  s.rows = min(kRows, wk.rq.n * G - s.row0);
  const auto tiles = [&](int lim) { return max(0, min(wk.nb, (lim - s.k0 + kKeys - 1) / kKeys)); };
  s.n = tiles(wk.t_end);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const bool has = s.rows > 128 * q;
    s.na[q] = has ? tiles(kv4_key_limit(p, wk.rq, s.row0 + min(s.rows, 128 * (q + 1)) - 1)) : 0;
    s.lim_lo[q] = has ? kv4_key_limit(p, wk.rq, s.row0 + 128 * q) : 0;
  }
  return s;
}

// Barrier of the softmax warps / of the expanding warps.
template <int kWarps>
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }
template <int kWarps>
__device__ __forceinline__ void expand_sync() { asm volatile("bar.sync 2, %0;" ::"n"(32 * kWarps) : "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// One lane's share of a 16-token cache tile: K or V codes and scales.
template <int D>
struct Words {
  uint4 w[D / 64];
  uint32_t s, s1;  // scales (s1: the second word, head_dim 256)
};
template <int D>
__device__ __forceinline__ void load_words(Words<D>& t, const uint8_t* tile, bool v, int lane) {
  using L = Kv4Layout<D>;
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    t.w[i] = __ldg(reinterpret_cast<const uint4*>(tile + (v ? L::kVCodes : L::kKCodes) + 512 * i + 16 * lane));
  if (D == 256) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(tile + (v ? L::kVScales : L::kKScales)) + lane);
    t.s = x.x;
    t.s1 = x.y;
  } else if (D == 64)
    t.s = v ? __ldg(reinterpret_cast<const uint32_t*>(tile + L::kVScales) + (lane >> 3) * 4 + (lane & 3))
            : __ldg(reinterpret_cast<const uint16_t*>(tile + L::kKScales) + lane);
  else
    t.s = __ldg(reinterpret_cast<const uint32_t*>(tile + (v ? L::kVScales : L::kKScales)) + lane);
}

// Eight codes times a scale -> 16 bytes of fp16.
__device__ __forceinline__ void expand8(uint32_t addr, uint32_t codes, uint32_t scale2) {
  uint32_t h[4];
  kv4_code_pairs(codes, h);
  st_shared_v4(addr, hmul2(h[0], scale2), hmul2(h[1], scale2), hmul2(h[2], scale2), hmul2(h[3], scale2));
}

// Where a lane writes: byte offsets in a K or V tile of 128-byte-swizzled rows
// (16-byte chunk x of row y at chunk x ^ (y & 7); 64 dims a row, the next 64
// 16 KB on), for cache tile 0; tile `sub` lies 2048 sub bytes on, tokens 8 to 15
// of it 1024.
//   K: lane 4 r + c holds tokens r and r + 8 and dims [c D/4, (c+1) D/4);
//   V: lane 4 r + c holds tokens 2c + e (+ 8) and dims [r D/8, (r+1) D/8).
// The eight lanes of a shared-memory pass should touch eight different chunks.
// At head_dim 128 they do not by themselves: lanes with c >= 2 write their K
// chunks in another order (`turn`: 2 before 0), those with odd r their V chunks.
// (At head_dim 256 they share banks, four lanes K and two V: the one Q tile's
// products leave the time.)
template <int D>
struct Places {
  uint32_t k[D / 32], v[2][D / 64];
  bool k_turn, v_turn;
  __device__ __forceinline__ explicit Places(int lane) {
    const int r = lane >> 2, c = lane & 3;
    k_turn = D == 128 && c >= 2;
    v_turn = D == 128 && (r & 1);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int ch = D == 64 ? 2 * c + i : D == 256 ? i : 4 * (c & 1) + (k_turn ? i ^ 2 : i);
      k[i] = (D == 64 ? 0 : D == 256 ? c * 16384 : (c >> 1) * 16384) + r * 128 + ((ch ^ r) << 4);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int row = 2 * c + e, ch = D == 64 ? r : D == 256 ? 4 * (r & 1) + i : 2 * (r & 3) + (v_turn ? i ^ 1 : i);
        v[e][i] = (D == 64 ? 0 : D == 256 ? (r >> 1) * 16384 : (r >> 2) * 16384) + row * 128 + ((ch ^ row) << 4);
      }
  }
};

// The words of one cache tile into its rows of the K / V tile; `base` is the
// stage's address plus 2048 x the cache tile's number.
template <int D>
__device__ __forceinline__ void expand_k(uint32_t base, const Words<D>& t, const Places<D>& pl) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (D == 64) {
      const uint32_t s = scale_both(t.s, h);
      expand8(base + pl.k[0] + 1024 * h, h ? t.w[0].z : t.w[0].x, s);
      expand8(base + pl.k[1] + 1024 * h, h ? t.w[0].w : t.w[0].y, s);
    } else if (D == 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 w = t.w[(2 * h + (i >> 2)) % (D / 64)];
        expand8(base + pl.k[i % (D / 32)] + 1024 * h, (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w,
                scale_both(h ? t.s1 : t.s, i >> 1));
      }
    } else {
      const uint4 w = t.w[h % (D / 64)];
      const uint32_t s0 = scale_both(t.s, 2 * h), s1 = scale_both(t.s, 2 * h + 1);
      const bool sw = pl.k_turn;
      expand8(base + pl.k[0] + 1024 * h, sw ? w.z : w.x, sw ? s1 : s0);
      expand8(base + pl.k[1] + 1024 * h, sw ? w.w : w.y, sw ? s1 : s0);
      expand8(base + pl.k[D == 128 ? 2 : 0] + 1024 * h, sw ? w.x : w.z, sw ? s0 : s1);
      expand8(base + pl.k[D == 128 ? 3 : 0] + 1024 * h, sw ? w.y : w.w, sw ? s0 : s1);
    }
  }
}
template <int D>
__device__ __forceinline__ void expand_v(uint32_t base, const Words<D>& t, const Places<D>& pl) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = i >> 1, e = i & 1;
    const uint32_t s = scale_both(t.s, i);
    if (D == 64) {
      expand8(base + pl.v[e][0] + 1024 * h, i == 0 ? t.w[0].x : i == 1 ? t.w[0].y : i == 2 ? t.w[0].z : t.w[0].w, s);
    } else if (D == 256) {
      const uint4 w = t.w[i % (D / 64)];
      const uint32_t s1 = scale_both(t.s1, i);
      expand8(base + pl.v[e][0] + 1024 * h, w.x, s);
      expand8(base + pl.v[e][1 % (D / 64)] + 1024 * h, w.y, s);
      expand8(base + pl.v[e][2 % (D / 64)] + 1024 * h, w.z, s1);
      expand8(base + pl.v[e][3 % (D / 64)] + 1024 * h, w.w, s1);
    } else {
      const uint4 w = t.w[h % (D / 64)];
      const uint32_t a = e ? w.z : w.x, b = e ? w.w : w.y;
      expand8(base + pl.v[e][0] + 1024 * h, pl.v_turn ? b : a, s);
      expand8(base + pl.v[e][D == 128 ? 1 : 0] + 1024 * h, pl.v_turn ? a : b, s);
    }
  }
}

// Columns [32 c, 32 c + 32) of a finished row.
__device__ __forceinline__ void write_cols(const Kv4AttnParams& p, size_t off, const float (&v)[32]) {
  if (p.o_is_fp32) {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.o) + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.o) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dst[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                          pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_tile_kernel(const Kv4AttnParams p) {
  using C = TileCfg<D>;
  constexpr int S = C::kStages, kRows = C::kRows, kQt = C::kQt, kGroups = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem), sKV = sQ + C::kQBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  const uint32_t b_q = smem_u32(bars);              // [2] Q tile written (4 warps)
  const uint32_t b_full = smem_u32(bars + 2);       // [S] (4 warps)
  const uint32_t b_empty = smem_u32(bars + 2 + S);  // [S] (2 issuers)
  const uint32_t b_s = smem_u32(bars + 2 + 2 * S);  // [2] S ready / O final (Q tile without a key: once a segment)
  const uint32_t b_p = smem_u32(bars + 4 + 2 * S);  // [2] P written (4 warps)
  const uint32_t b_drain = smem_u32(bars + 6 + 2 * S);  // [2]
  // notes of the expanding warps: the first key of a segment with a NaN in a
  // group of V; the cache tiles of a key tile whose page is not one of the cache
  int* s_nan = reinterpret_cast<int*>(bars + 8 + 2 * S);            // [kSegs][16]
  uint8_t* s_dead = reinterpret_cast<uint8_t*>(s_nan + kSegs * 16);  // [kSegs][8]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_dead + kSegs * 8);
  int* s_int = reinterpret_cast<int*>(tmem_slot + 1);  // abort, bad, last
  volatile uint32_t* s_turns = reinterpret_cast<uint32_t*>(s_int + 3);  // [2] warps' P tiles of Q tile 0 / 1 so far
  // s_int[5]: where a wait was given up
  __shared__ long long s_sum[kThreads / 32], s_found[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.cache.Hkv;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_q + 8 * i, 4);
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 4);
      mbar_init(b_drain + 8 * i, 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(b_full + 8 * i, C::kExpand);
      mbar_init(b_empty + 8 * i, kQt);
    }
    s_int[0] = s_int[1] = s_int[2] = s_int[5] = 0;
    s_turns[0] = s_turns[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  int bad = 0;
  Kv4Walk wk;
  const Kv4Line line = kv4_find_part<kRows, kKeys, kUnit, true, kThreads>(p, s_sum, s_found, wk, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Abort ab{s_int, s_int + 5};
  if (bad) atomicMax(s_int + 1, bad);

  // Register split: 512 threads x 128 at launch = 128 x 40 + 256 x 184 + 128 x 104.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp < kQt && lane == 0) {
      // ---------------------------------------------------------- MMA issuers
      const int qt = warp;
      const uint32_t tS = tmem + qt * 128, tO = tmem + 256 + qt * D;
      const uint64_t d0 = sdesc_sw128(sQ, 0, 1024);
      int stage = 0;
      uint32_t kph = 0, pph = 0, qph = 0;
      bool ok = true;
      auto advance = [&]() { if (++stage == S) { stage = 0; kph ^= 1; } };
      auto qk = [&](int kst) {
        const uint64_t b = opaque(d0);
        const uint64_t dq = sdesc_at(b, (uint32_t)qt * C::kTile, 0);
        const uint64_t dk = sdesc_at(b, (uint32_t)(C::kQBytes + kst * C::kTile), 0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(tS, sdesc_at(dq, off, 16), sdesc_at(dk, off, 16), C::kIdescQK, kk > 0);
        }
      };
      for (; wk.pos < line.end && ok;) {
        wk.enter<kRows, kKeys, kUnit, true>(p, line.end);
        const Segment sg = segment<C::kQt>(p, wk);
        wk.leave(line.end);
        const int na = qt == 0 ? sg.na[0] : sg.na[1];
        if (sg.n == 0) continue;
        if (!(ok = mbar_wait(b_q + 8 * qt, qph, ab, 130))) break;
        qph ^= 1;
        if (!(ok = mbar_wait(b_full + 8 * stage, kph, ab, 131))) break;
        tc_fence_after();
        if (na > 0) qk(stage);
        umma_commit(b_s + 8 * qt);
        umma_commit(b_empty + 8 * stage);
        advance();
        for (int j = 0; j < sg.n; ++j) {
          const int vst = stage;
          if (!(ok = mbar_wait(b_full + 8 * vst, kph, ab, 132))) break;
          tc_fence_after();
          advance();  // stage now holds K of the next tile
          if (j < na) {
            if (!(ok = mbar_wait(b_p + 8 * qt, pph, ab, 133))) break;
            pph ^= 1;
            tc_fence_after();
            const uint64_t dv = sdesc_at(opaque(d0), (uint32_t)(C::kQBytes + vst * C::kTile), 0);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ts(tO, tS + kk * 8, sdesc_at(dv, kk * 2048, 16384), C::kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
            if (j + 1 == na) umma_commit(b_s + 8 * qt);  // O final
          }
          umma_commit(b_empty + 8 * vst);
          if (j + 1 < sg.n) {
            if (!(ok = mbar_wait(b_full + 8 * stage, kph, ab, 134))) break;
            tc_fence_after();
            if (j + 1 < na) { qk(stage); umma_commit(b_s + 8 * qt); }
            umma_commit(b_empty + 8 * stage);
            advance();
          }
        }
      }
      if (!ok) {  // let issued MMAs finish before tensor memory is released
        umma_commit(b_drain + 8 * qt);
        mbar_wait_drain(b_drain + 8 * qt, 0);
      }
    }
  } else if (warp < 4 + C::kSoft) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ------------------------------------------------------------ softmax
    const int qt = (warp - 4) >> 2, row_t = tid - 128 * (1 + qt);  // row within the Q tile
    const uint32_t lane_base = (uint32_t)(warp & 3) * 32;
    const uint32_t tS = tmem_addr(tmem, lane_base, qt * 128), tO = tmem_addr(tmem, lane_base, 256 + qt * D);
    uint32_t sph = 0;
    int seg = 0, tiles = 0;  // segments with key tiles, and key tiles, so far
    uint32_t turns = 0;      // P tiles of the other Q tile in the segments before
    bool ok = true;
    for (; wk.pos < line.end;) {
      wk.enter<kRows, kKeys, kUnit, true>(p, line.end);
      if (wk.nb == 0) {
        wk.leave(line.end);
        continue;
      }
      const Segment sg = segment<C::kQt>(p, wk);
      const int na = qt == 0 ? sg.na[0] : sg.na[1];
      const int na_other = qt == 0 ? sg.na[1] : sg.na[0];
      const int urow = 128 * qt + row_t, row = sg.row0 + urow;  // row of the unit, of the request
      const bool valid = urow < sg.rows;
      const int lim_lo = qt == 0 ? sg.lim_lo[0] : sg.lim_lo[1];
      const int lim = valid ? kv4_key_limit(p, wk.rq, row) : 0x7fffffff;
      const int token = wk.rq.b + row / G, h = wk.head * G + row % G;
      float sl2 = 0.f;
      if (na > 0) {
        // this thread's query row, as fp16 after a power of two, into the Q tile
        // (free: the tile's products of the segment before are done)
        uint4 w[D / 8];
        if (valid) {
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                            (size_t)token * p.q_stride + (size_t)h * D);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) w[i] = src[i];
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          mx = __vmaxu2(mx, __vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu));
          mx = __vmaxu2(mx, __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
        }
        float up;
        sl2 = p.scale * kLog2e * kv4_row_scale(max(mx & 0xffffu, mx >> 16), up);
        // It scales masked scores (-inf) too: not with NaN in a row without keys, and not
        // with a product that underflowed to 0 (2^-126 leaves scores that are as good as 0).
        if (lim == 0) sl2 = 1.f;
        if (sl2 < 0x1p-126f) sl2 = 0x1p-126f;
        auto cvt = [&](uint32_t x) { return pack_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up); };
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          st_shared_v4(sQ + qt * C::kTile + (i >> 3) * 16384 + row_t * 128 + (((i & 7) ^ (row_t & 7)) << 4), cvt(w[i].x),
                       cvt(w[i].y), cvt(w[i].z), cvt(w[i].w));
        fence_proxy_async_smem();
      }
      if (sg.n > 0) {
        // (A Q tile without a key in this segment too: its issuer, and with it the
        // ring of stages, may not leave these warps behind, which still read the
        // notes of the segment before.)
        tc_fence_before();  // this segment's first P.V overwrites the O read before
        __syncwarp();
        if (lane == 0) mbar_arrive(b_q + 8 * qt);
      }
      const uint64_t sl2x2 = f2_pack(sl2, sl2);
      float m_ref = neg_inf(), l_sum = 0.f;
      for (int j = 0; j < na; ++j) {
        if (ok) ok = mbar_wait(b_s + 8 * qt, sph, ab, 140);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        sph ^= 1;
        tc_fence_after();
        uint32_t r[4][32];
        tmem_ld32(tS + 0, r[0]);
        tmem_ld32(tS + 32, r[1]);
        tmem_ld32(tS + 64, r[2]);
        tmem_ld32(tS + 96, r[3]);
        // The two Q tiles take turns (0's tile j after 1's tile j - 1, 1's after 0's
        // tile j), so that one's softmax runs beside the other's products.  A phase's
        // parity cannot tell whether it is the other's turn: at a segment's first
        // tile, and where a Q tile sees no key, nothing holds one back, so the other
        // may be two phases behind or ahead.  The count of its P tiles decides, and
        // the barrier only passes the time until the next one.  The order is for
        // speed alone: a wait that takes too long is given up.
        const int k_other = j - (qt == 0 ? 1 : 0);
        if (k_other >= 0 && k_other < na_other) {
          const uint32_t k = turns + k_other, want = 4 * (k + 1);
          for (int n = 0; n < kTurnLimit && (int32_t)(s_turns[1 - qt] - want) < 0 && !*ab.flag; ++n)
            mbar_try_wait(b_p + 8 * (1 - qt), k & 1u);
          __syncwarp();
        }
        const uint2 dead = *reinterpret_cast<const uint2*>(s_dead + ((tiles + j) & (kSegs - 1)) * 8);
        tmem_ld_wait();
        reg_fence32(r[0]); reg_fence32(r[1]); reg_fence32(r[2]); reg_fence32(r[3]);
        const int kst = sg.k0 + kKeys * j;
        if (kst + kKeys > lim_lo || (dead.x | dead.y)) {
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            const uint32_t d = (c >> 4) < 4 ? dead.x >> (8 * (c >> 4)) : dead.y >> (8 * ((c >> 4) & 3));
            if (kst + c >= lim || (d & 0xffu)) r[c >> 5][c & 31] = __float_as_uint(neg_inf());
          }
        }
        uint64_t nm2 = 0, ls_a = 0, ls_b = 0;
        auto p_tile = [&](float m_use) {
          nm2 = f2_pack(-m_use, -m_use);
          ls_a = ls_b = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t x =
                  f2_fma(f2_pack(__uint_as_float(r[c][2 * i]), __uint_as_float(r[c][2 * i + 1])), sl2x2, nm2);
              float x0, x1;
              f2_unpack(x, x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              pk[i] = pack_f16x2(p0, p1);
              if (i & 1) ls_b = f2_add(ls_b, f2_pack(p0, p1));
              else ls_a = f2_add(ls_a, f2_pack(p0, p1));
            }
            tmem_st16(tS + 16 * c, pk);
          }
        };
        auto tile_sum = [&]() {
          float a0, a1, b0, b1;
          f2_unpack(ls_a, a0, a1);
          f2_unpack(ls_b, b0, b1);
          return (a0 + a1) + (b0 + b1);
        };
        // As in the ring forward: try the reference as it stands; where a tile's P
        // would grow too large (or a row has seen no key), take the maximum, move
        // the reference and redo the tile.
        bool exact = __any_sync(0xffffffffu, m_ref == neg_inf());
        bool rescale = false;
        float alpha = 1.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          if (exact) {
            float mx[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx[k] = neg_inf();
#pragma unroll
            for (int i = 0; i < 16; i += 2)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mx[k] = fmax3(mx[k], __uint_as_float(r[k >> 1][16 * (k & 1) + i]),
                              __uint_as_float(r[k >> 1][16 * (k & 1) + i + 1]));
            const float m_tile = fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], fmax3(mx[5], mx[6], mx[7]))) * sl2;
            rescale = m_tile > m_ref + kMaxExp;
            if (rescale) {
              const float m_new = ceilf(m_tile) - kHeadroom;
              alpha = ex2_approx(m_ref - m_new);
              l_sum *= alpha;
              m_ref = m_new;
            }
          }
          p_tile(m_ref == neg_inf() ? 0.f : m_ref);
          if (exact || !__any_sync(0xffffffffu, !(tile_sum() <= kSumLimit))) break;
          tmem_st_wait();  // the redo overwrites these P stores
          exact = true;
        }
        if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_ld_wait();
            reg_fence32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tO + 32 * c, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          atomicAdd(const_cast<uint32_t*>(s_turns) + qt, 1u);
          mbar_arrive(b_p + 8 * qt);
        }
        l_sum += tile_sum();
      }
      if (sg.n > 0 && ok) {
        ok = mbar_wait(b_s + 8 * qt, sph, ab, 141);  // O final (without a key: the issuer is here as well)
        ok = __all_sync(0xffffffffu, ok);
        sph ^= 1;
        tc_fence_after();
      }

      // After a wait that was given up the rows are not known: NaN, not zero.
      if (!ok) l_sum = quiet_nan();
      // A row whose scores were all NaN has no reference, but a sum that is NaN; with
      // any reference its partial result makes the row NaN.
      if (m_ref == neg_inf() && !(l_sum == 0.f)) m_ref = 0.f;

      // ---- output, or a partial result
      const bool direct = wk.whole();
      const int c0 = direct ? 0 : line.owner(wk.first);
      auto slot = [&](int c) { return p.partials + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * C::kSlot; };
      const float inv = !direct ? 1.f : l_sum == 0.f ? 0.f : 1.f / l_sum;
      const int* nan_key = s_nan + (seg & (kSegs - 1)) * 16;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        __syncwarp();
        if (na > 0 && ok) {
          tmem_ld32(tO + 32 * c, o);
          tmem_ld_wait();
          reg_fence32(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * inv;
        if (na > 0) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (nan_key[2 * c + g] < lim) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[16 * g + i] = quiet_nan();
            }
        }
        if (!valid) continue;
        if (direct) {
          write_cols(p, ((size_t)token * p.Hq + h) * D + 32 * c, v);
        } else if (m_ref != neg_inf()) {
          float4* dst = reinterpret_cast<float4*>(slot(blockIdx.x) + 2 * kRows + urow * D + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      if (direct) {
        if (valid) p.lse[(size_t)h * p.Tq + token] = l_sum == 0.f ? neg_inf() : (m_ref + log2f(l_sum)) * kLn2;
      } else {
        if (valid) {
          slot(blockIdx.x)[urow] = m_ref;
          slot(blockIdx.x)[kRows + urow] = l_sum;
        }
        // Of every kFan neighbours the CTA that brings the last one merges them into
        // the first one's slot, and of those the CTA that brings the last one the unit.
        const int parts = line.owner(wk.first + wk.rq.blocks - 1) - c0 + 1;
        int from = ((int)blockIdx.x - c0) / kFan * kFan, count = min(kFan, parts - from), stride = 1;
        int* ticket = p.tickets + 2 * (c0 + from) + (from == 0 ? 1 : 0);
#pragma unroll 1
        for (;;) {
          __threadfence();
          softmax_sync<C::kSoft>();
          if (tid == 128) {
            s_int[2] = atomicAdd(ticket, 1) == count - 1;
            if (s_int[2]) *ticket = 0;  // as the next call expects it
          }
          softmax_sync<C::kSoft>();
          if (!s_int[2]) break;
          __threadfence();
          const bool done = stride > 1 || parts <= kFan;
          auto part = [&](int i) { return slot(c0 + from + i * stride); };
          // a thread a row: the rows' largest references and their sums, kept in the
          // Q tiles' shared memory (all products of the segment are done)
          float* s_ref = reinterpret_cast<float*>(smem);
          float* s_inv = s_ref + kRows;
          float mm = neg_inf(), l = 0.f;
#pragma unroll 4
          for (int i = 0; i < count; ++i) mm = fmaxf(mm, __ldcg(part(i) + urow));
#pragma unroll 4
          for (int i = 0; i < count; ++i) {
            const float m = __ldcg(part(i) + urow), li = __ldcg(part(i) + kRows + urow);
            l += m == neg_inf() ? 0.f : li * ex2_approx(m - mm);
          }
          s_ref[urow] = mm;
          s_inv[urow] = !done ? 1.f : l == 0.f ? 0.f : 1.f / l;
          if (done && valid) p.lse[(size_t)h * p.Tq + token] = l == 0.f ? neg_inf() : (mm + log2f(l)) * kLn2;
          softmax_sync<C::kSoft>();
          // a warp four rows at once: their weighted sums
          constexpr int V = D / 32, B = 4;
          for (int r0 = warp - 4; r0 < sg.rows; r0 += C::kSoft * B) {
            float acc[B][V] = {}, ref[B];
#pragma unroll
            for (int b = 0; b < B; ++b) ref[b] = s_ref[min(r0 + C::kSoft * b, kRows - 1)];
#pragma unroll 2
            for (int i = 0; i < count; ++i) {
              const float* s = part(i);
#pragma unroll
              for (int b = 0; b < B; ++b) {
                const int rr = min(r0 + C::kSoft * b, sg.rows - 1);
                const float m = __ldcg(s + rr);
                const float wgt = m == neg_inf() ? 0.f : ex2_approx(m - ref[b]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                  const float x = __ldcg(s + 2 * kRows + rr * D + 32 * v + lane);
                  acc[b][v] += m == neg_inf() ? 0.f : x * wgt;  // (a row without keys has no O there)
                }
              }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
              const int rr = r0 + C::kSoft * b;
              if (rr >= sg.rows) break;
              const int grow = sg.row0 + rr, tk = wk.rq.b + grow / G, hh = wk.head * G + grow % G;
#pragma unroll
              for (int v = 0; v < V; ++v) {
                const size_t off = ((size_t)tk * p.Hq + hh) * D + 32 * v + lane;
                const float x = acc[b][v] * s_inv[rr];
                if (!done) part(0)[2 * kRows + rr * D + 32 * v + lane] = x;  // (read by this warp only)
                else if (p.o_is_fp32) reinterpret_cast<float*>(p.o)[off] = x;
                else reinterpret_cast<__nv_bfloat16*>(p.o)[off] = __float2bfloat16_rn(x);
              }
            }
          }
          softmax_sync<C::kSoft>();  // the Q tiles, and the merged slot's m and l, may be written again
          if (done) break;
          if (valid) {
            part(0)[urow] = mm;
            part(0)[kRows + urow] = l;
          }
          from = 0;
          count = (parts + kFan - 1) / kFan;
          stride = kFan;
          ticket = p.tickets + 2 * gridDim.x + c0;
        }
      }
      wk.leave(line.end);
      tiles += sg.n;
      seg += sg.n > 0;
      turns += na_other;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    // ------------------------------------------------------------ expansion
    using L = Kv4Layout<D>;
    constexpr int kSubs = C::kSubs;
    const int dw = warp - 4 - C::kSoft;  // cache tiles kSubs dw ... of every key tile
    const Places<D> places(lane);
    int issued = 0, seg = 0, tiles = 0;
    bool ok = true;
    for (; wk.pos < line.end;) {
      wk.enter<kRows, kKeys, kUnit, true>(p, line.end);
      const Segment sg = segment<C::kQt>(p, wk);
      wk.leave(line.end);
      if (sg.n == 0) continue;
      int* nan_key = s_nan + (seg & (kSegs - 1)) * 16;
      if (dw == 0 && lane < kGroups) nan_key[lane] = 0x7fffffff;
      expand_sync<C::kExpand>();
      const int32_t* table = p.block_table + (size_t)wk.r * p.table_stride;
      const uint8_t* base = p.cache.pages + ((size_t)wk.head << (p.cache.page_shift - 4)) * L::kBytes;
      const int tiles_mask = (1 << (p.cache.page_shift - 4)) - 1;
      // lanes u < kSubs: page ids of this warp's cache tiles of key tile j
      auto lane_page = [&](int j) -> int {
        const int t = sg.k0 + kKeys * j + 16 * (kSubs * dw + lane);
        return lane < kSubs && j < sg.n && t < wk.t_end ? table[t >> p.cache.page_shift] : 0;
      };
      // The words of a key tile are loaded as soon as the registers of the one
      // before are free: the way to memory is covered by a whole tile's products.
      Words<D> k[kSubs], v[kSubs];
      uint32_t dead = 0;  // bit u: cache tile u of key tile j lies on a page that is not one of the cache
      auto fetch = [&](Words<D> (&w)[kSubs], bool is_v, int page, int j) {
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
          const int t = sg.k0 + kKeys * j + 16 * (kSubs * dw + u);
          const int pg = __shfl_sync(0xffffffffu, page, u);
          const bool in = j < sg.n && t < wk.t_end, good = (uint32_t)pg < (uint64_t)p.cache.num_pages;
          if (!is_v) dead = (dead & ~(1u << u)) | (in && !good ? 1u << u : 0u);
          w[u].s = w[u].s1 = 0;
          if (in && good)
            load_words<D>(w[u], base + (int64_t)pg * p.page_bytes + ((t >> 4) & tiles_mask) * L::kBytes, is_v, lane);
        }
      };
      int page = lane_page(0), page_next = lane_page(1);
      fetch(k, false, page, 0);
      fetch(v, true, page, 0);
      for (int j = 0; j < sg.n; ++j) {
        page = page_next;
        page_next = lane_page(j + 2);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const int st = issued % S;
          if (ok) ok = mbar_wait(b_empty + 8 * st, ((issued / S) & 1) ^ 1, ab, 150);
          ok = __all_sync(0xffffffffu, ok);
          ++issued;
          if (!ok) continue;
          const uint32_t dst = sKV + st * C::kTile + 2048 * kSubs * dw;
          if (kind == 0) {
            if (dead) bad = max(bad, (int)RA_KV4_BAD_PAGE);
            if (lane < kSubs) s_dead[((tiles + j) & (kSegs - 1)) * 8 + kSubs * dw + lane] = (dead >> lane) & 1;
#pragma unroll
            for (int u = 0; u < kSubs; ++u) expand_k<D>(dst + 2048 * u, k[u], places);
          } else {
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
              // keys that no row sees, and NaN groups, count as zero; a row that
              // sees a key with a NaN gets it from the notes
              const int t0 = sg.k0 + kKeys * j + 16 * (kSubs * dw + u);
              auto clean = [&](uint32_t& sc, int g) {
                if (!__vcmpgeu4(sc, 0xf8f8f8f8u) && t0 + 16 <= wk.t_end) return;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int t = t0 + 2 * (lane & 3) + (i & 1) + 8 * (i >> 1);
                  if (((sc >> (8 * i)) & 0xffu) >= 0xf8u || t >= wk.t_end) {
                    if (t < wk.t_end) atomicMin(&nan_key[g], t);
                    sc &= ~(0xffu << (8 * i));
                  }
                }
              };
              clean(v[u].s, D == 64 ? lane >> 3 : D == 128 ? lane >> 2 : 2 * (lane >> 2));
              if (D == 256) clean(v[u].s1, 2 * (lane >> 2) + 1);
              expand_v<D>(dst + 2048 * u, v[u], places);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_full + 8 * st);
          fetch(kind == 0 ? k : v, kind == 1, page, j + 1);
        }
      }
      tiles += sg.n;
      ++seg;
    }
    if (bad) atomicMax(s_int + 1, bad);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) kv4_end(p, s_int[5] ? kKv4GaveUp + s_int[5] : s_int[1]);
}

template <int D>
cudaError_t launch(int ctas, const Kv4AttnParams& p, cudaStream_t stream) {
  auto kern = kv4_tile_kernel<D>;
  static Kv4SmemLimit limit;
  return limit.launch(reinterpret_cast<const void*>(kern), TileCfg<D>::kSmem, [&] {
    kern<<<ctas, kThreads, TileCfg<D>::kSmem, stream>>>(p);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_kv4_tile(int D, int ctas, const Kv4AttnParams& p, cudaStream_t stream) {
  if (D == 64) return launch<64>(ctas, p, stream);
  if (D == 128) return launch<128>(ctas, p, stream);
  if (D == 256) return launch<256>(ctas, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ra
