// kv4_wtile.cu -- the attention weight that every cached token receives, for
// requests with many query rows (a prompt's next part, or the last tokens of one
// that look back over it), on tcgen05 tensor cores.  Formulas as in kv4_weights.cu.
//
// Here products and exponentials dominate: 2 D flops and one exponential a row and
// key.  Keys are the rows of S^T = K Q^T, so that a thread owns a key: it adds up
// the exponentials of a row of tensor memory, and nothing is exchanged between
// threads.  A unit is 256 keys (head_dim 256: 128) of one request and head.  The keys lie in
// tensor memory as the products' A operand, expanded once, while the head's query rows stream past,
// 128 (64) at a time, straight from the query tensor (TMA): from shared memory both operands
// would be read at 128 bytes a clock, all there is.  Both are bf16: codes times scales
// have 6 significant bits.
//
// The rows' log-sum-exps come in by a product too: one more step of 16 along K adds 1 times
// - lse / scale, in three bf16 pieces that add up to 24 bits.  Read from shared memory by the
// threads, a value for every column, they would cost four passes a warp for four columns, as much of
// the bandwidth as all else.
//
// Warp roles (896 threads; at head_dim 256 512, with 8 warps for the sums and 4 for the keys):
//   warps 0, 1    UMMA issuers of the two key tiles (warp 0 owns tensor memory): a wait costs one
//                 of them 100 to 200 clocks even where nothing is to be waited for
//   warp 2        the query tiles' log-sum-exps and key limits
//   warp 3        TMA loads of query tiles
//   warps 4-19    exponentials and sums: a thread is a key and half of a tile's rows
//   warps 20-27   cache -> bf16 keys: a thread is a key here too
// Tensor memory (512 columns): the keys (D / 2 columns for 128 of them; at head_dim 256 those of two
// units, 4 to 10 % faster), then a ring of S^T tiles.
//
// 1024 tokens x 32 query heads over 33792 cached, 8 key heads of 128: 246 us, 1135 TFLOP/s; tensor
// cores and exponentials are at work half of that.  128 rows of queries against 256 keys cost 1154
// clocks of the one, 1024 of the other, and about 2050 in all: a summing warp waits for its tile and its
// columns about as long as it sums them, and four warps a scheduler, whose tiles are ready at the same
// time, do not cover that.  64 tokens over 32768: 41 us, of which 13 are start, first keys and the
// merge of blocks whose heads lie in two CTAs; 32 requests of 4096, 512 rows a head: 193 us.
// Measured on the way, the first call: one issuer 290 us, two 257; issuers in strict turns 269; log-sum-exps
// from shared memory 294; tiles of 192 rows 364; a tile in pieces of 32 columns, each summed while the next
// comes, 298.  With 8 summing and 4 expanding warps (168 and 104 registers) it took 254, the other two 44 and
// 232; with 16 and 4 (72, 104; spills) 246, 47 and 215; other splits of the registers of 28 warps 250 to 343.
// (Its 56, 80 and 64 registers are not without spills either: 208 bytes of the 72 at launch at head_dim
// 128, 192 at 64, 84 at 256.)
// A tile with columns that are no rows takes the masked sums, with a limit read for every column: where the
// heads of a group do not divide the tile that is every tile.  The same call at 28 query and 4 key heads takes
// 360 us (679 TFLOP/s), at 40 and 8 451 us (774), at 24 and 8 288 us (728).
// Items (block of keys, head) lie on one line that the CTAs cut evenly; of a block
// whose heads went to several CTAs the one that brings the last sum adds them, in
// the CTAs' order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"
#include "kv4.h"
#include "kv4_walk.cuh"
#include "tc.cuh"

namespace ra {
namespace {

constexpr int kExpandCost = 1;  // expanding a unit's keys, in query tiles
constexpr int kLseStages = 4;

template <int D>
struct WTile {
  static constexpr int kSumWarps = D == 256 ? 8 : 16;
  static constexpr int kExpandWarps = D == 256 ? 4 : 8;
  static constexpr int kThreads = 32 * (4 + kSumWarps + kExpandWarps);
  static constexpr int kKeyTiles = D == 256 ? 1 : 2;  // 128 keys each
  static constexpr int kKeys = 128 * kKeyTiles;
  static constexpr int kN = D == 256 ? 64 : 128;      // query rows of a tile
  static constexpr int kShares = kSumWarps / 4 / kKeyTiles;  // threads that share a key
  static constexpr int kCols = kN / kShares;                 // columns of a thread
  static constexpr int kKCols = D / 2;                // tensor memory columns of 128 keys
  static constexpr int kSRing = D == 256 ? 4 : 3;     // S^T tiles (128 keys x kN rows) in tensor memory
  static constexpr int kSets = D == 256 ? 2 : 1;      // units whose keys lie there (two at 128 or 64: no faster)
  static constexpr int kSOff = kSets * kKeyTiles * kKCols;
  static_assert(kSOff + kSRing * kN <= 512 && (kSets == 1 || kKeyTiles == 1), "tensor memory");
  static constexpr int kQTile = kN * D * 2;
  static constexpr int kQStages = D == 64 ? 8 : 6;
  static constexpr int kOnesOff = kQStages * kQTile;  // the keys' side of the lse's step: 128 rows of 32 bytes
  static constexpr int kLseOff = kOnesOff + 128 * 32;
  static constexpr int kLseTile = 32 * kN;            // the rows' side
  static constexpr int kLimOff = kLseOff + kLseStages * kLseTile;
  static constexpr int kLimStage = 4 * kN + 16;       // limits, the smallest and the largest of them
  static constexpr int kPartOff = kLimOff + kLseStages * kLimStage;
  static constexpr int kBarOff = kPartOff + 4 * kKeys * (kShares - 1);  // (the other threads' sums)
  static constexpr int kSmem = kBarOff + 512 + 1024;  // barriers, alignment slack
  static constexpr uint32_t kIdesc = idesc_bf16_f32(128, kN, false, false);
  static_assert(kLseOff == kOnesOff + 128 * 32 && kOnesOff % 1024 == 0, "descriptors");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int kWarps>
__device__ __forceinline__ void keys_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// One token's keys of one head: the codes in order (8 dims a word), and the scales' bytes.
template <int D>
struct KeyWords {
  uint32_t w[D / 8];
  uint32_t s[D / 64];  // scales of groups 4 i .. 4 i + 3
};
// From the cache tile that holds token t (of 16).  A token's codes are D / 2 bytes in whole words of
// 16 bytes (head_dim 64: of 8), its scales D / 64 of every 4, or neighbouring bytes (Kv4Layout).
template <int D>
__device__ __forceinline__ void load_key(KeyWords<D>& k, const uint8_t* tile, int t) {
  using L = Kv4Layout<D>;
  const int r = t & 7, h = t >> 3;
  if (D == 64) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(tile + (4 * r + g) * 16 + h * 8));
      k.w[2 * g] = x.x;
      k.w[2 * g + 1] = x.y;
    }
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(tile + L::kKScales + 8 * r));  // [group][h]
    k.s[0] = __byte_perm(x.x, x.y, h ? 0x7531 : 0x6420);
  } else if (D == 128) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(tile + h * 512 + (4 * r + c) * 16));
      k.w[4 * c] = x.x;
      k.w[4 * c + 1] = x.y;
      k.w[4 * c + 2] = x.z;
      k.w[(4 * c + 3) % (D / 8)] = x.w;
    }
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(tile + L::kKScales + 16 * r));  // [quarter][h][2]
    k.s[0] = __byte_perm(x.x, x.y, h ? 0x7632 : 0x5410);
    k.s[D == 128 ? 1 : 0] = __byte_perm(x.z, x.w, h ? 0x7632 : 0x5410);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(tile + (2 * h + i) * 512 + (4 * r + c) * 16));
        k.w[(8 * c + 4 * i) % (D / 8)] = x.x;
        k.w[(8 * c + 4 * i + 1) % (D / 8)] = x.y;
        k.w[(8 * c + 4 * i + 2) % (D / 8)] = x.z;
        k.w[(8 * c + 4 * i + 3) % (D / 8)] = x.w;
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(tile + L::kKScales + 32 * r + 16 * i));  // [quarter][h][4]
      k.s[(2 * i) % (D / 64)] = h ? x.y : x.x;
      k.s[(2 * i + 1) % (D / 64)] = h ? x.w : x.z;
    }
  }
}
// Expand them into this thread's row of tensor memory, 32 columns (64 dims) at a time.
template <int D>
__device__ __forceinline__ void expand_key(uint32_t taddr, const KeyWords<D>& k) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    uint32_t o[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 v = kv4_expand_half(k.w[8 * i + j], (k.s[i] >> (8 * (j >> 1))) & 0xffu);
      o[4 * j] = v.x;
      o[4 * j + 1] = v.y;
      o[4 * j + 2] = v.z;
      o[4 * j + 3] = v.w;
    }
    tmem_st32(taddr + 32 * i, o);
  }
}

// How a head's query rows lie in tiles: `tokens` tokens of all G heads of the group, or, of
// large groups, a part of one token's.
struct Tiling {
  int tokens, per_token;  // tokens of a tile; tiles of a token (1 where a tile holds whole tokens)
};
template <int N>
__host__ __device__ __forceinline__ Tiling tiling(int G) {
  return G <= N ? Tiling{N / G, 1} : Tiling{1, (G + N - 1) / N};
}

// What a request asks of this kernel: items (block of keys, head), `cost` places of the
// line each.
struct Job {
  Kv4Request rq;
  int fresh, tiles;  // keys from here on begin at zero; query tiles of a head
  long long items, cost;
};
template <int D>
__device__ __forceinline__ Job job_of(const Kv4WeightsParams& p, int r) {
  using C = WTile<D>;
  Job j;
  j.rq = kv4_request<128, C::kKeys, true>(p.a, r);
  const int L = j.rq.L;
  j.fresh = L - (p.new_lens ? min(max(p.new_lens[r], 0), L) : 0);
  const Tiling t = tiling<C::kN>(p.a.Hq / p.a.cache.Hkv);
  j.tiles = t.per_token > 1 ? j.rq.n * t.per_token : (j.rq.n + t.tokens - 1) / t.tokens;
  const bool mine = j.rq.row_tiles > 0 && L > 0;
  j.items = mine ? (long long)j.rq.blocks * p.a.cache.Hkv : 0;
  j.cost = j.tiles + kExpandCost;
  return j;
}

// A CTA's items, request by request.
template <int D>
struct Walk {
  const Kv4WeightsParams& p;
  const Kv4Line& line;
  int r;
  long long base, here, x0, x1;  // places before the next request; before this one; its items of this CTA
  Job job;
  __device__ __forceinline__ Walk(const Kv4WeightsParams& p_, const Kv4Line& l, int r_, long long base_)
      : p(p_), line(l), r(r_ - 1), base(base_) {}
  __device__ __forceinline__ bool next() {
    while (base < line.end && ++r < p.a.R) {
      job = job_of<D>(p, r);
      here = base;
      base += job.items * job.cost;
      x0 = kv4_div(max(line.begin - here, 0ll) + job.cost - 1, job.cost);
      x1 = min(job.items, kv4_div(line.end - here + job.cost - 1, job.cost));
      if (x0 < x1) return true;
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__((WTile<D>::kThreads), 1)
kv4_wtile_kernel(const Kv4WeightsParams wp, const __grid_constant__ CUtensorMap tq) {
  using C = WTile<D>;
  constexpr int N = C::kN, QS = C::kQStages, LS = kLseStages, kThreads = C::kThreads, kSumWarps = C::kSumWarps;
  const Kv4AttnParams& p = wp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem);
  auto lim_of = [&](int s) { return reinterpret_cast<int*>(smem + C::kLimOff + s * C::kLimStage); };  // [N], then the smallest and the largest
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  const uint32_t b_kfull = smem_u32(bars);            // [2] a tile's keys expanded (4 warps): of a key tile, or of a set
  const uint32_t b_kempty = smem_u32(bars + 2);       // [2]
  const uint32_t b_qfull = smem_u32(bars + 4);        // [QS]
  const uint32_t b_qempty = smem_u32(bars + 12);      // [QS]
  const uint32_t b_lfull = smem_u32(bars + 20);       // [LS]
  const uint32_t b_lempty = smem_u32(bars + 20 + LS); // [LS] (the summing warps and the issuers)
  // S^T tiles: the t-th tile of key tile kt lies in place (kKeyTiles t + kt) % kSRing.  Each key
  // tile has barriers of its own for every place: neither may be two phases behind or ahead of a wait.
  const uint32_t b_sfull = smem_u32(bars + 20 + 2 * LS);   // [2][4] ready
  const uint32_t b_sempty = smem_u32(bars + 28 + 2 * LS);  // [2][4] read (by the warps that sum that key tile)
  const uint32_t b_drain = smem_u32(bars + 36 + 2 * LS);   // [2]
  int* s_int = reinterpret_cast<int*>(bars + 38 + 2 * LS);  // abort, bad, last, where a wait was given up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_int + 4);
  static_assert(QS <= 8 && (38 + 2 * LS) * 8 + 20 <= 512, "barriers");
  __shared__ long long s_sum[kThreads / 32], s_found[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.cache.Hkv, Hkv = p.cache.Hkv, P = 1 << p.cache.page_shift;
  const Tiling tl = tiling<N>(G);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_kfull + 8 * i, 4);
      mbar_init(b_kempty + 8 * i, 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(b_sfull + 8 * i, 1);
      mbar_init(b_sempty + 8 * i, kSumWarps / C::kKeyTiles);
    }
    for (int i = 0; i < QS; ++i) {
      mbar_init(b_qfull + 8 * i, 1);
      mbar_init(b_qempty + 8 * i, C::kKeyTiles);
    }
    for (int i = 0; i < LS; ++i) {
      mbar_init(b_lfull + 8 * i, 1);
      mbar_init(b_lempty + 8 * i, kSumWarps + C::kKeyTiles);
    }
    mbar_init(b_drain, 1);
    mbar_init(b_drain + 8, 1);
    s_int[0] = s_int[1] = s_int[2] = s_int[3] = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 3 && lane == 0) tma_prefetch_desc(&tq);
  // 1, 1, 1, 0 ... in every row of the ones; zeros in the rows of the log-sum-exps, whose
  // first three places are written tile by tile.  (Rows of 32 bytes, 16-byte halves swapped in
  // rows 4 to 7 of every 8.)
  for (int i = tid; i < (128 * 32 + LS * C::kLseTile) / 16; i += kThreads) {
    const bool ones = i < 256 && ((i ^ (i >> 3)) & 1) == 0;
    *reinterpret_cast<uint4*>(smem + C::kOnesOff + 16 * i) =
        ones ? make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  int bad = 0;
  auto work = [&](int i) {
    const Job j = job_of<D>(wp, i);
    bad = max(bad, j.rq.bad);
    return j.items * j.cost;
  };
  int r0;
  long long base0;
  const Kv4Line line = kv4_cut<kThreads>(p.R, work, s_sum, s_found, r0, base0);
  // alone in the call: requests without rows, whose new tokens' sums begin at zero all the same
  if (p.split_rows == 0) {
    for (int r = 0; r < p.R; ++r) {
      const Job j = job_of<D>(wp, r);
      if (j.rq.n > 0) continue;
      for (int t = j.fresh + blockIdx.x * kThreads + tid; t < j.rq.L; t += gridDim.x * kThreads) {
        const int page = p.block_table[(size_t)r * p.table_stride + (t >> p.cache.page_shift)];
        if ((uint32_t)page < (uint64_t)p.cache.num_pages)
          wp.weights[((int64_t)page << p.cache.page_shift) + (t & (P - 1))] = 0.f;
        else
          bad = max(bad, (int)RA_KV4_BAD_PAGE);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Abort ab{s_int, s_int + 3};
  if (bad) atomicMax(s_int + 1, bad);
  Walk<D> wk(wp, line, r0, base0);

  // Register split: 896 threads x 72 at launch = 128 x 56 + 512 x 80 + 256 x 64; head_dim 256: 512 x 128 =
  // 128 x 72 + 256 x 168 + 128 x 104.
  if (warp < 4) {
    if (D == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp < C::kKeyTiles && lane == 0) {
      // ---------------------------------------------------------- MMA issuers
      const int kt = warp;
      const uint64_t d0 = sdesc_sw128(sQ, 0, 1024);
      const uint32_t tK = tmem + kt * C::kKCols;
      const uint64_t d1 = sdesc_sw32(sQ + C::kOnesOff);
      uint32_t g = 0, qs = 0, qph = 0, ls = 0, lph = 0, item = 0;
      bool ok = true;
      while (ok && wk.next()) {
        const int tiles = wk.job.tiles;
        for (long long x = wk.x0; x < wk.x1 && ok; ++x, ++item) {
          const uint32_t set = item % C::kSets;
          if (!(ok = mbar_wait(b_kfull + 8 * (kt + set), (item / C::kSets) & 1, ab, 160))) break;
          for (int t = 0; t < tiles; ++t, ++g) {
            if (!(ok = mbar_wait(b_qfull + 8 * qs, qph, ab, 161))) break;
            if (!(ok = mbar_wait(b_lfull + 8 * ls, lph, ab, 168))) break;
            // the place's last tile: with two key tiles the other one's, one or two before this one
            const uint32_t sb = (C::kKeyTiles * g + kt) % C::kSRing;
            const uint32_t back = C::kKeyTiles == 1 ? C::kSRing : 2 - kt;
            if (g >= back && !(ok = mbar_wait(b_sempty + 8 * (4 * (C::kKeyTiles - 1 - kt) + sb),
                                              ((g - back) / C::kSRing) & 1, ab, 162)))
              break;
            tc_fence_after();
            const uint64_t dq = sdesc_at(opaque(d0), (uint32_t)(qs * C::kQTile), 0);
            const uint32_t tS = tmem + C::kSOff + sb * N;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ts(tS, tK + set * C::kKCols + kk * 8, sdesc_at(dq, (kk >> 2) * (N * 128) + (kk & 3) * 32, 16), C::kIdesc, kk > 0);
            umma_ss(tS, d1, sdesc_at(d1, (uint32_t)(128 * 32 + ls * C::kLseTile), 0), C::kIdesc, 1);
            umma_commit(b_sfull + 8 * (4 * kt + sb));
            umma_commit(b_qempty + 8 * qs);
            umma_commit(b_lempty + 8 * ls);
            if (++qs == QS) { qs = 0; qph ^= 1; }
            if (++ls == LS) { ls = 0; lph ^= 1; }
          }
          if (ok) umma_commit(b_kempty + 8 * (kt + set));
        }
      }
      // Issued MMAs finish before tensor memory is released, and copies land before the CTA's shared memory is
      // given up (below), also where only another role gave a wait up; without that they have by now.
      umma_commit(b_drain + 8 * kt);
      mbar_wait_drain(b_drain + 8 * kt, 0);
    } else if (warp == 3 && lane == 0) {
      // ---------------------------------------------------------- query tiles
      const uint32_t bytes = (uint32_t)(tl.tokens * (tl.per_token > 1 ? N : G)) * D * 2;
      uint32_t g = 0;
      bool ok = true;
      while (ok && wk.next()) {
        const int tiles = wk.job.tiles;
        int head = (int)(wk.x0 % Hkv);
        for (long long x = wk.x0; x < wk.x1 && ok; ++x) {
          int tok = wk.job.rq.b, part = 0;
          for (int t = 0; t < tiles; ++t, ++g) {
            const uint32_t qs = g % QS;
            if (!(ok = mbar_wait(b_qempty + 8 * qs, ((g / QS) & 1) ^ 1, ab, 163))) break;
            mbar_expect_tx(b_qfull + 8 * qs, bytes);
#pragma unroll
            for (int s = 0; s < D / 64; ++s)
              tma_load_3d(sQ + qs * C::kQTile + s * (N * 128), &tq, b_qfull + 8 * qs, 64 * s, head * G + part * N, tok);
            if (++part == tl.per_token) {
              part = 0;
              tok += tl.tokens;
            }
          }
          if (++head == Hkv) head = 0;
        }
      }
      for (uint32_t k = g > QS ? g - QS : 0; k < g; ++k) mbar_wait_drain(b_qfull + 8 * (k % QS), (k / QS) & 1);
    } else if (warp == 2) {
      // ---------------------------------------------------------- log-sum-exps and limits
      constexpr int V = N / 32;
      const float inv_scale = 1.f / p.scale;
      // where this lane's columns lie in a tile: token and head of the group (a tile of a part
      // of one token: head alone), past any of both for columns that are none
      int col_tok[V], col_head[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = lane + 32 * i;
        col_tok[i] = tl.per_token > 1 ? 0 : c / G;
        col_head[i] = tl.per_token > 1 ? c : c - col_tok[i] * G;
        if (tl.per_token == 1 && c >= tl.tokens * G) col_head[i] = 0x40000000;
      }
      // the values of a tile; those of the next one are on their way while they wait for their place
      struct Tile {
        float v[V];
        int lim[V];
      } a, b;
      long long x = 0;
      int head = 0, t = 0, tok0 = 0, part = 0;
      bool any = wk.next();
      if (any) {
        x = wk.x0;
        head = (int)(wk.x0 % Hkv);
      }
      auto load = [&](Tile& o) -> bool {
        if (!any) return false;
        const Kv4Request& rq = wk.job.rq;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int gi = part * N + col_head[i], tok = tok0 + col_tok[i];
          const bool valid = gi < G && tok < rq.n;
          o.v[i] = valid ? __ldg(wp.lse + (size_t)(head * G + gi) * p.Tq + rq.b + tok) : neg_inf();
          o.lim[i] = !valid ? 0 : p.causal ? max(0, min(rq.L, rq.L - rq.n + tok + 1)) : rq.L;
        }
        if (++part == tl.per_token) {
          part = 0;
          tok0 += tl.tokens;
        }
        if (++t == wk.job.tiles) {
          t = part = tok0 = 0;
          if (++head == Hkv) head = 0;
          if (++x == wk.x1 && (any = wk.next())) {
            x = wk.x0;
            head = (int)(wk.x0 % Hkv);
          }
        }
        return true;
      };
      uint32_t ls = 0, lph = 0;
      auto put = [&](Tile& o) -> bool {
        bool ok = mbar_wait(b_lempty + 8 * ls, lph ^ 1, ab, 164);
        if (!(ok = __all_sync(0xffffffffu, ok))) return false;
        int least = 0x7fffffff, most = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // rows that are none, or have no softmax (lse = -inf: they see no key), see no key here
          const bool dead = o.v[i] == neg_inf();
          const int lim = dead ? 0 : o.lim[i];
          const float f = dead ? neg_inf() : -o.v[i] * inv_scale;
          float r1 = f - __bfloat162float(__float2bfloat16_rn(f));
          if (!isfinite(f)) r1 = 0.f;
          const float r2 = r1 - __bfloat162float(__float2bfloat16_rn(r1));
          const int c = lane + 32 * i;
          *reinterpret_cast<uint2*>(smem + C::kLseOff + ls * C::kLseTile + 32 * c + ((c & 4) << 2)) =
              make_uint2(pack_bf16x2(f, r1), pack_bf16x2(r2, 0.f));
          lim_of(ls)[c] = lim;
          least = min(least, lim);
          most = max(most, lim);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) *reinterpret_cast<int2*>(lim_of(ls) + N) = make_int2(least, most);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_lfull + 8 * ls);
        if (++ls == LS) { ls = 0; lph ^= 1; }
        return true;
      };
      bool more = load(a);
      while (more) {
        more = load(b);
        if (!put(a) || !more) break;
        more = load(a);
        if (!put(b)) break;
      }
    }
  } else if (warp < 4 + kSumWarps) {
    if (D == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    // ------------------------------------------------------------ exponentials and sums
    constexpr int NC = C::kCols;
    const int gp = (warp - 4) >> 2, kt = gp % C::kKeyTiles, share = gp / C::kKeyTiles;
    const int key_t = 128 * kt + 32 * (warp & 3) + lane;  // key of the block
    const int col0 = NC * share;
    const uint32_t tS = tmem_addr(tmem, (uint32_t)(warp & 3) * 32, C::kSOff + col0);
    const float c1 = p.scale * kLog2e;
    const uint64_t c2 = f2_pack(c1, c1);
    uint32_t g = 0;  // tiles so far
    bool ok = true;
    float acc = 0.f;
    uint64_t sum_a, sum_b;
    auto columns = [&](const uint32_t (&s)[32]) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float e[4];
        f2_unpack(f2_mul(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2), e[0], e[1]);
        f2_unpack(f2_mul(f2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), c2), e[2], e[3]);
        sum_a = f2_add(sum_a, f2_pack(ex2_approx(e[0]), ex2_approx(e[1])));
        sum_b = f2_add(sum_b, f2_pack(ex2_approx(e[2]), ex2_approx(e[3])));
      }
    };
    auto masked_columns = [&](const uint32_t (&s)[32], const int4* lim, int key) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const int4 l = lim[i / 4];
        const float e0 = ex2_approx(__uint_as_float(s[i]) * c1), e1 = ex2_approx(__uint_as_float(s[i + 1]) * c1);
        const float e2 = ex2_approx(__uint_as_float(s[i + 2]) * c1), e3 = ex2_approx(__uint_as_float(s[i + 3]) * c1);
        sum_a = f2_add(sum_a, f2_pack(key < l.x ? e0 : 0.f, key < l.y ? e1 : 0.f));
        sum_b = f2_add(sum_b, f2_pack(key < l.z ? e2 : 0.f, key < l.w ? e3 : 0.f));
      }
    };
    while (wk.next()) {
      const Job& job = wk.job;
      for (long long x = wk.x0; x < wk.x1; ++x) {
        const int blk = (int)kv4_div(x, Hkv), head = (int)(x - (long long)blk * Hkv);
        const int key = blk * C::kKeys + key_t, key_end = (key & ~127) + 128;
        if (head == 0 || x == wk.x0) acc = 0.f;
        for (int t = 0; t < job.tiles; ++t, ++g) {
          const uint32_t ls = g % LS;
          if (ok) ok = mbar_wait(b_lfull + 8 * ls, (g / LS) & 1, ab, 165);
          const int4* lim = reinterpret_cast<const int4*>(lim_of(ls) + col0);
          const int2 ends = *reinterpret_cast<const int2*>(lim_of(ls) + N);
          const bool whole = key_end <= ends.x, none = key_end - 128 >= ends.y;  // all rows see all keys; none does any
          const uint32_t sb = (C::kKeyTiles * g + kt) % C::kSRing;
          if (ok) ok = mbar_wait(b_sfull + 8 * (4 * kt + sb), (g / C::kSRing) & 1, ab, 166);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          auto release = [&]() {  // all columns are in registers: the S^T tile may be written again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_sempty + 8 * (4 * kt + sb));
          };
          sum_a = sum_b = 0;
          if (none) {
            release();
          } else {
            uint32_t s[32];
#pragma unroll
            for (int c = 0; c < NC / 32; ++c) {
              tmem_ld32(tS + sb * N + 32 * c, s);
              tmem_ld_wait();
              reg_fence32(s);
              if (c == NC / 32 - 1) release();
              if (whole) columns(s);
              else masked_columns(s, lim + 8 * c, key);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(b_lempty + 8 * ls);
          float a0, a1, a2, a3;
          f2_unpack(sum_a, a0, a1);
          f2_unpack(sum_b, a2, a3);
          acc += (a0 + a1) + (a2 + a3);
        }
        if (head + 1 < Hkv && x + 1 < wk.x1) continue;

        // ---- the block's sums (after a wait that was given up: not known)
        if (!ok) acc = quiet_nan();
        float total = acc;
        const bool owner = share == 0;
        if (C::kShares > 1) {
          float* others = reinterpret_cast<float*>(smem + C::kPartOff);
          keys_sync<kSumWarps>();  // (they were read)
          if (!owner) others[(share - 1) * C::kKeys + key_t] = acc;
          keys_sync<kSumWarps>();
#pragma unroll
          for (int i = 1; i < C::kShares; ++i)
            if (owner) total += others[(i - 1) * C::kKeys + key_t];
        }
        const long long first = (long long)blk * Hkv;  // the block's first item
        bool writes = true;
        if (x - head < wk.x0 || head + 1 < Hkv) {
          // Some heads are other CTAs': each CTA that has one leaves its sums, and the one that brings
          // the last adds them.  Items shorter than a part lie in neighbouring CTAs, longer
          // ones in one each.
          const bool single = job.cost > line.size;
          const int c0 = line.owner(wk.here + first * job.cost);
          const int parts = single ? Hkv : line.owner(wk.here + (first + Hkv - 1) * job.cost) - c0 + 1;
          auto slot = [&](int i) {
            const int c = single ? line.owner(wk.here + (first + i) * job.cost) : c0 + i;
            return p.partials + (size_t)(2 * c + (c == c0 ? 1 : 0)) * C::kKeys + key_t;
          };
          const int me = blockIdx.x;
          if (owner) p.partials[(size_t)(2 * me + (me == c0 ? 1 : 0)) * C::kKeys + key_t] = total;
          __threadfence();
          keys_sync<kSumWarps>();
          if (tid == 128) {
            int* ticket = p.tickets + 2 * c0 + 1;
            s_int[2] = atomicAdd(ticket, 1) == parts - 1;
            if (s_int[2]) *ticket = 0;  // as the next call expects it
          }
          keys_sync<kSumWarps>();
          writes = s_int[2];
          keys_sync<kSumWarps>();
          if (writes) {
            __threadfence();
            total = 0.f;
            if (owner)
              for (int i = 0; i < parts; ++i) total += __ldcg(slot(i));
          }
        }
        if (writes && owner && key < job.rq.L) {
          const int page = p.block_table[(size_t)wk.r * p.table_stride + (key >> p.cache.page_shift)];
          if ((uint32_t)page < (uint64_t)p.cache.num_pages) {
            float* dst = wp.weights + ((int64_t)page << p.cache.page_shift) + (key & (P - 1));
            *dst = (key >= job.fresh ? 0.f : *dst) + total;
          } else {
            bad = max(bad, (int)RA_KV4_BAD_PAGE);
          }
        }
      }
    }
    if (bad) atomicMax(s_int + 1, bad);
  } else {
    if (D == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------------ expansion
    // Key tile by key tile: while one is expanded for the next head, the products of this
    // head's last query tile go on with the other.
    constexpr int kGroups = C::kExpandWarps / 4, kT = C::kKeyTiles / kGroups;
    const int kt0 = kGroups == 1 ? 0 : (warp - 4 - kSumWarps) >> 2;
    const int row = 32 * (warp & 3) + lane;  // key of a key tile
    const uint32_t tK = tmem_addr(tmem, (uint32_t)(warp & 3) * 32, 0);
    uint32_t item = 0;
    bool ok = true;
    KeyWords<D> k[kT];
#pragma unroll
    for (int kt = 0; kt < kT; ++kt) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) k[kt].w[i] = 0u;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) k[kt].s[i] = 0u;
    }
    while (ok && wk.next()) {
      const Kv4Request& rq = wk.job.rq;
      const int32_t* table = p.block_table + (size_t)wk.r * p.table_stride;
      // page of this thread's key of a block's key tile, and that key's words of one head; where there is
      // none (no page of the cache, behind the last key) whatever was there: its sum is not used
      auto page_of = [&](int kt, int blk) -> int {
        const int t = blk * C::kKeys + 128 * (kt0 + kt) + row;
        return t < rq.L ? table[t >> p.cache.page_shift] : -1;
      };
      auto fetch = [&](KeyWords<D>& w, int kt, int blk, int head, int page) {
        const int t = (blk * C::kKeys + 128 * (kt0 + kt) + row) & (P - 1);
        if ((uint32_t)page < (uint64_t)p.cache.num_pages)
          load_key<D>(w, p.cache.pages + kv4_tile_offset<D>(p.cache, page, head, t), t & 15);
      };
      int blk = (int)kv4_div(wk.x0, Hkv), head = (int)(wk.x0 - (long long)blk * Hkv);
      int page[kT], page_next[kT];
#pragma unroll
      for (int kt = 0; kt < kT; ++kt) {
        page[kt] = page_of(kt, blk);
        page_next[kt] = page_of(kt, blk + 1);
        fetch(k[kt], kt, blk, head, page[kt]);
      }
      for (long long x = wk.x0; x < wk.x1 && ok; ++x, ++item) {
        if (++head == Hkv) {
          head = 0;
          ++blk;
#pragma unroll
          for (int kt = 0; kt < kT; ++kt) {
            page[kt] = page_next[kt];
            page_next[kt] = page_of(kt, blk + 1);
          }
        }
#pragma unroll
        for (int kt = 0; kt < kT; ++kt) {
          const uint32_t set = item % C::kSets;
          if (ok) ok = mbar_wait(b_kempty + 8 * (kt0 + kt + set), ((item / C::kSets) & 1) ^ 1, ab, 167);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          expand_key<D>(tK + (kt0 + kt + set) * C::kKCols, k[kt]);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_kfull + 8 * (kt0 + kt + set));
          if (x + 1 < wk.x1) fetch(k[kt], kt, blk, head, page[kt]);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) kv4_end(p, s_int[3] ? kKv4GaveUp + s_int[3] : s_int[1]);
}

template <int D>
cudaError_t launch(int ctas, const Kv4WeightsParams& p, const CUtensorMap& tq, cudaStream_t stream) {
  auto kern = kv4_wtile_kernel<D>;
  static Kv4SmemLimit limit;
  return limit.launch(reinterpret_cast<const void*>(kern), WTile<D>::kSmem, [&] {
    kern<<<ctas, WTile<D>::kThreads, WTile<D>::kSmem, stream>>>(p, tq);
    return cudaGetLastError();
  });
}

template <int D>
void box_of(int G, int* heads, int* tokens) {
  const Tiling t = tiling<WTile<D>::kN>(G);
  *heads = t.per_token > 1 ? WTile<D>::kN : G;
  *tokens = t.tokens;
}

}  // namespace

void kv4_wtile_box(int D, int G, int* heads, int* tokens) {
  if (D == 256) box_of<256>(G, heads, tokens);
  else if (D == 128) box_of<128>(G, heads, tokens);
  else box_of<64>(G, heads, tokens);
}

cudaError_t launch_kv4_wtile(int D, int ctas, const Kv4WeightsParams& p, const CUtensorMap& tq, cudaStream_t stream) {
  if (D == 64) return launch<64>(ctas, p, tq, stream);
  if (D == 128) return launch<128>(ctas, p, tq, stream);
  if (D == 256) return launch<256>(ctas, p, tq, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ra
