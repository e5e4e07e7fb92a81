// kv4_wtile.cu -- the attention weight that every cached token receives, for
// requests with many query rows (a prompt's next part, or the last tokens of one
// that look back over it), on tcgen05 tensor cores.  Formulas as in kv4_weights.cu.
//
// Here products and exponentials dominate: 2 D flops and one exponential a row and
// key.  Keys are the rows of S^T = K Q^T, so that a thread owns a key: it adds up
// the exponentials of a row of tensor memory, and nothing is exchanged between
// threads.  A unit is 256 keys (head_dim 256: 128) of one request and head; K stays in
// shared memory, expanded once, while the head's query rows stream past, 128 (64) at a time,
// straight from the query tensor (TMA).  Both are bf16: codes times scales have 6
// significant bits.
//
// Warp roles (512 threads):
//   warp 0        UMMA issuer (owns tensor memory)
//   warp 1        TMA loads of query tiles
//   warps 2, 3    the tiles' log-sum-exps and key limits, tiles in turn
//   warps 4-11    exponentials and sums: a thread is a key; at head_dim 256 warps
//                 4-7 take the first half of a tile's rows and 8-11 the second
//   warps 12-15   cache tiles -> bf16 keys
// Tensor memory (512 columns): two buffers of S^T, 256 columns each.
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

constexpr int kThreads = 512;
constexpr int kExpandCost = 1;  // expanding a unit's keys, in query tiles
constexpr int kLseStages = 8;

template <int D>
struct WTile {
  static constexpr int kKeyTiles = D == 256 ? 1 : 2;  // 128 keys each
  static constexpr int kKeys = 128 * kKeyTiles;
  static constexpr int kN = D == 256 ? 64 : 128;      // query rows of a tile
  static constexpr int kCols = kN * kKeyTiles / 2;    // columns of a thread
  static constexpr int kKTile = 128 * D * 2;
  static constexpr int kKBytes = kKeyTiles * kKTile;  // of one of the two stages
  static constexpr int kQTile = kN * D * 2;
  static constexpr int kQStages = D == 64 ? 4 : 2;
  static constexpr int kQOff = 2 * kKBytes;
  static constexpr int kLseOff = kQOff + kQStages * kQTile;
  static constexpr int kLseStage = 8 * kN + 16;       // - lse (log2), limits, their smallest
  static constexpr int kPartOff = kLseOff + kLseStages * kLseStage;
  static constexpr int kBarOff = kPartOff + 512;      // (half sums of 128 keys: head_dim 256)
  static constexpr int kSmem = kBarOff + 512 + 1024;  // barriers, alignment slack
  static constexpr uint32_t kIdesc = idesc_bf16_f32(128, kN, false, false);
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void keys_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// One lane's share of a 16-token cache tile's keys.
template <int D>
struct Words {
  uint4 w[D / 64];
  uint32_t s, s1;  // scales (s1: the second word, head_dim 256)
};
template <int D>
__device__ __forceinline__ void load_words(Words<D>& t, const uint8_t* tile, int lane) {
  using L = Kv4Layout<D>;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) t.w[i] = __ldg(reinterpret_cast<const uint4*>(tile + L::kKCodes + 512 * i + 16 * lane));
  if (D == 256) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(tile + L::kKScales) + lane);
    t.s = x.x;
    t.s1 = x.y;
  } else if (D == 64) {
    t.s = __ldg(reinterpret_cast<const uint16_t*>(tile + L::kKScales) + lane);
  } else {
    t.s = __ldg(reinterpret_cast<const uint32_t*>(tile + L::kKScales) + lane);
  }
}
// Eight codes and their scale byte (of a word) -> 16 bytes of bf16.
__device__ __forceinline__ void expand8(uint32_t addr, uint32_t codes, uint32_t scales, int i) {
  const uint4 v = kv4_expand_half(codes, (scales >> (8 * i)) & 0xffu);
  st_shared_v4(addr, v.x, v.y, v.z, v.w);
}
// Lane 4 r + c of a cache tile holds tokens r and r + 8 and dims [c D/4, (c+1) D/4).  Where
// its 16-byte chunks go in a tile of 128-byte-swizzled rows (64 dims a row, the next 64
// 16 KB on); cache tile `sub` lies 2048 sub bytes on, tokens 8 to 15 of it 1024.  At
// head_dim 128 lanes with c >= 2 write their chunks in another order (2 before 0), so that
// the eight lanes of a shared-memory pass touch eight different chunks.
template <int D>
struct Places {
  uint32_t k[D / 32];
  bool turn;
  __device__ __forceinline__ explicit Places(int lane) {
    const int r = lane >> 2, c = lane & 3;
    turn = D == 128 && c >= 2;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int ch = D == 64 ? 2 * c + i : D == 256 ? i : 4 * (c & 1) + (turn ? i ^ 2 : i);
      k[i] = (D == 64 ? 0 : D == 256 ? c * 16384 : (c >> 1) * 16384) + r * 128 + ((ch ^ r) << 4);
    }
  }
};
template <int D>
__device__ __forceinline__ void expand_keys(uint32_t base, const Words<D>& t, const Places<D>& pl) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (D == 64) {
      expand8(base + pl.k[0] + 1024 * h, h ? t.w[0].z : t.w[0].x, t.s, h);
      expand8(base + pl.k[1] + 1024 * h, h ? t.w[0].w : t.w[0].y, t.s, h);
    } else if (D == 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 w = t.w[(2 * h + (i >> 2)) % (D / 64)];
        expand8(base + pl.k[i % (D / 32)] + 1024 * h, (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w,
                h ? t.s1 : t.s, i >> 1);
      }
    } else {
      const uint4 w = t.w[h % (D / 64)];
      const bool sw = pl.turn;
      const int a = 2 * h + (sw ? 1 : 0), b = 2 * h + (sw ? 0 : 1);
      expand8(base + pl.k[0] + 1024 * h, sw ? w.z : w.x, t.s, a);
      expand8(base + pl.k[1] + 1024 * h, sw ? w.w : w.y, t.s, a);
      expand8(base + pl.k[D == 128 ? 2 : 0] + 1024 * h, sw ? w.x : w.z, t.s, b);
      expand8(base + pl.k[D == 128 ? 3 : 0] + 1024 * h, sw ? w.y : w.w, t.s, b);
    }
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
__global__ void __launch_bounds__(kThreads, 1)
kv4_wtile_kernel(const Kv4WeightsParams wp, const __grid_constant__ CUtensorMap tq) {
  using C = WTile<D>;
  constexpr int N = C::kN, QS = C::kQStages, LS = kLseStages;
  const Kv4AttnParams& p = wp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sK = smem_u32(smem), sQ = sK + C::kQOff;
  auto lse_of = [&](int s) { return reinterpret_cast<float*>(smem + C::kLseOff + s * C::kLseStage); };
  auto lim_of = [&](int s) { return reinterpret_cast<int*>(lse_of(s) + N); };  // [N], then the smallest
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  const uint32_t b_kfull = smem_u32(bars);            // [2] keys expanded (4 warps)
  const uint32_t b_kempty = smem_u32(bars + 2);       // [2]
  const uint32_t b_qfull = smem_u32(bars + 4);        // [QS]
  const uint32_t b_qempty = smem_u32(bars + 8);       // [QS]
  const uint32_t b_lfull = smem_u32(bars + 12);       // [LS]
  const uint32_t b_lempty = smem_u32(bars + 12 + LS); // [LS] (8 warps)
  const uint32_t b_sfull = smem_u32(bars + 12 + 2 * LS);   // [2] S^T ready
  const uint32_t b_sempty = smem_u32(bars + 14 + 2 * LS);  // [2] (8 warps)
  const uint32_t b_drain = smem_u32(bars + 16 + 2 * LS);
  int* s_int = reinterpret_cast<int*>(bars + 17 + 2 * LS);  // abort, bad, last, where a wait was given up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_int + 4);
  static_assert((17 + 2 * LS) * 8 + 20 <= 512, "barriers");
  __shared__ long long s_sum[kThreads / 32], s_found[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.cache.Hkv, Hkv = p.cache.Hkv, P = 1 << p.cache.page_shift;
  const Tiling tl = tiling<N>(G);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_kfull + 8 * i, 4);
      mbar_init(b_kempty + 8 * i, 1);
      mbar_init(b_sfull + 8 * i, 1);
      mbar_init(b_sempty + 8 * i, 8);
    }
    for (int i = 0; i < QS; ++i) {
      mbar_init(b_qfull + 8 * i, 1);
      mbar_init(b_qempty + 8 * i, 1);
    }
    for (int i = 0; i < LS; ++i) {
      mbar_init(b_lfull + 8 * i, 1);
      mbar_init(b_lempty + 8 * i, 8);
    }
    mbar_init(b_drain, 1);
    s_int[0] = s_int[1] = s_int[2] = s_int[3] = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 1 && lane == 0) tma_prefetch_desc(&tq);
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

  // Register split: 512 threads x 128 at launch = 128 x 64 + 256 x 176 + 128 x 96.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t d0 = sdesc_sw128(sK, 0, 1024);
      uint32_t g = 0, item = 0;
      bool ok = true;
      while (ok && wk.next()) {
        for (long long x = wk.x0; x < wk.x1 && ok; ++x, ++item) {
          const uint32_t ks = item & 1;
          if (!(ok = mbar_wait(b_kfull + 8 * ks, (item >> 1) & 1, ab, 160))) break;
          for (int t = 0; t < wk.job.tiles; ++t, ++g) {
            const uint32_t qs = g % QS, sb = g & 1;
            if (!(ok = mbar_wait(b_qfull + 8 * qs, (g / QS) & 1, ab, 161))) break;
            if (!(ok = mbar_wait(b_sempty + 8 * sb, ((g >> 1) & 1) ^ 1, ab, 162))) break;
            tc_fence_after();
            const uint64_t b = opaque(d0);
            const uint64_t dq = sdesc_at(b, (uint32_t)(C::kQOff + qs * C::kQTile), 0);
#pragma unroll
            for (int kt = 0; kt < C::kKeyTiles; ++kt) {
              const uint64_t dk = sdesc_at(b, (uint32_t)(ks * C::kKBytes + kt * C::kKTile), 0);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_ss(tmem + sb * 256 + kt * 128, sdesc_at(dk, (kk >> 2) * 16384 + (kk & 3) * 32, 16),
                        sdesc_at(dq, (kk >> 2) * (N * 128) + (kk & 3) * 32, 16), C::kIdesc, kk > 0);
            }
            umma_commit(b_sfull + 8 * sb);
            umma_commit(b_qempty + 8 * qs);
          }
          umma_commit(b_kempty + 8 * ks);
        }
      }
      if (!ok) {  // let issued MMAs finish before tensor memory is released
        umma_commit(b_drain);
        mbar_wait_drain(b_drain, 0);
      }
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- query tiles
      const uint32_t bytes = (uint32_t)(tl.tokens * (tl.per_token > 1 ? N : G)) * D * 2;
      uint32_t g = 0;
      bool ok = true;
      while (ok && wk.next()) {
        for (long long x = wk.x0; x < wk.x1 && ok; ++x) {
          const int head = (int)(x % Hkv);
          for (int t = 0; t < wk.job.tiles; ++t, ++g) {
            const uint32_t qs = g % QS;
            if (!(ok = mbar_wait(b_qempty + 8 * qs, ((g / QS) & 1) ^ 1, ab, 163))) break;
            mbar_expect_tx(b_qfull + 8 * qs, bytes);
            const int h = head * G + (t % tl.per_token) * N;
            const int tok = wk.job.rq.b + (tl.per_token > 1 ? t / tl.per_token : t * tl.tokens);
#pragma unroll
            for (int s = 0; s < D / 64; ++s)
              tma_load_3d(sQ + qs * C::kQTile + s * (N * 128), &tq, b_qfull + 8 * qs, 64 * s, h, tok);
          }
        }
      }
      if (!ok)  // copies under way land before the CTA's shared memory is given up
        for (uint32_t k = g > QS ? g - QS : 0; k < g; ++k) mbar_wait_drain(b_qfull + 8 * (k % QS), (k / QS) & 1);
    } else if (warp >= 2) {
      // ---------------------------------------------------------- log-sum-exps and limits
      // (values of the next tile are on their way while this one's wait for their place)
      constexpr int V = N / 32;
      float v[V];
      int lim[V];
      uint32_t g = 0, held = 0;  // `held`: the tile in v and lim
      bool ok = true, have = false;
      auto put = [&]() {
        const uint32_t ls = held % LS;
        ok = mbar_wait(b_lempty + 8 * ls, ((held / LS) & 1) ^ 1, ab, 164);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        int least = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // rows that are none, or have no softmax (lse = -inf: they see no key), see no key here
          const bool dead = v[i] == neg_inf();
          if (dead) lim[i] = 0;
          lse_of(ls)[lane + 32 * i] = dead ? neg_inf() : -v[i] * kLog2e;
          lim_of(ls)[lane + 32 * i] = lim[i];
          least = min(least, lim[i]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) lim_of(ls)[N] = least;
        __syncwarp();
        if (lane == 0) mbar_arrive(b_lfull + 8 * ls);
      };
      while (ok && wk.next()) {
        const Kv4Request& rq = wk.job.rq;
        for (long long x = wk.x0; x < wk.x1 && ok; ++x) {
          const int head = (int)(x % Hkv);
          for (int t = 0; t < wk.job.tiles && ok; ++t, ++g) {
            if ((g & 1) != (uint32_t)(warp - 2)) continue;
            float nv[V];
            int nl[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const int c = lane + 32 * i;
              const int gi = tl.per_token > 1 ? (t % tl.per_token) * N + c : c % G;
              const int tok = tl.per_token > 1 ? t / tl.per_token : t * tl.tokens + c / G;
              const bool valid = gi < G && tok < rq.n && (tl.per_token > 1 || c < tl.tokens * G);
              nv[i] = valid ? __ldg(wp.lse + (size_t)(head * G + gi) * p.Tq + rq.b + tok) : neg_inf();
              nl[i] = valid ? kv4_key_limit(p, rq, tok * G) : 0;
            }
            if (have) put();
#pragma unroll
            for (int i = 0; i < V; ++i) {
              v[i] = nv[i];
              lim[i] = nl[i];
            }
            held = g;
            have = true;
          }
        }
      }
      if (have && ok) put();
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // ------------------------------------------------------------ exponentials and sums
    constexpr int NC = C::kCols;
    const int gp = (warp - 4) >> 2, row = tid - 128 * (1 + gp);
    const int key_t = C::kKeyTiles == 2 ? 128 * gp + row : row;  // key of the block
    const int col0 = C::kKeyTiles == 2 ? 0 : NC * gp;
    const uint32_t tS = tmem_addr(tmem, (uint32_t)(warp & 3) * 32, C::kKeyTiles == 2 ? 128 * gp : col0);
    const float c1 = p.scale * kLog2e;
    const uint64_t c2 = f2_pack(c1, c1);
    uint32_t g = 0;
    bool ok = true;
    float acc = 0.f;
    while (wk.next()) {
      const Job& job = wk.job;
      for (long long x = wk.x0; x < wk.x1; ++x) {
        const int blk = (int)kv4_div(x, Hkv), head = (int)(x - (long long)blk * Hkv);
        const int key = blk * C::kKeys + key_t, key_end = (key & ~127) + 128;
        if (head == 0 || x == wk.x0) acc = 0.f;
        for (int t = 0; t < job.tiles; ++t, ++g) {
          const uint32_t ls = g % LS, sb = g & 1;
          if (ok) ok = mbar_wait(b_lfull + 8 * ls, (g / LS) & 1, ab, 165) && mbar_wait(b_sfull + 8 * sb, (g >> 1) & 1, ab, 166);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          uint32_t s[NC / 32][32];
#pragma unroll
          for (int c = 0; c < NC / 32; ++c) tmem_ld32(tS + sb * 256 + 32 * c, s[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < NC / 32; ++c) reg_fence32(s[c]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_sempty + 8 * sb);
          const float4* nl = reinterpret_cast<const float4*>(lse_of(ls) + col0);
          uint64_t sum_a = 0, sum_b = 0;
          if (key_end <= lim_of(ls)[N]) {
#pragma unroll
            for (int c = 0; c < NC / 32; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 m = nl[8 * c + i];
                float e[4];
                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c][4 * i]), __uint_as_float(s[c][4 * i + 1])), c2, f2_pack(m.x, m.y)), e[0], e[1]);
                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c][4 * i + 2]), __uint_as_float(s[c][4 * i + 3])), c2, f2_pack(m.z, m.w)), e[2], e[3]);
                sum_a = f2_add(sum_a, f2_pack(ex2_approx(e[0]), ex2_approx(e[1])));
                sum_b = f2_add(sum_b, f2_pack(ex2_approx(e[2]), ex2_approx(e[3])));
              }
          } else {
            const int4* lim = reinterpret_cast<const int4*>(lim_of(ls) + col0);
#pragma unroll
            for (int c = 0; c < NC / 32; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 m = nl[8 * c + i];
                const int4 l = lim[8 * c + i];
                const float e0 = ex2_approx(fmaf(__uint_as_float(s[c][4 * i]), c1, m.x));
                const float e1 = ex2_approx(fmaf(__uint_as_float(s[c][4 * i + 1]), c1, m.y));
                const float e2 = ex2_approx(fmaf(__uint_as_float(s[c][4 * i + 2]), c1, m.z));
                const float e3 = ex2_approx(fmaf(__uint_as_float(s[c][4 * i + 3]), c1, m.w));
                sum_a = f2_add(sum_a, f2_pack(key < l.x ? e0 : 0.f, key < l.y ? e1 : 0.f));
                sum_b = f2_add(sum_b, f2_pack(key < l.z ? e2 : 0.f, key < l.w ? e3 : 0.f));
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
        if (C::kKeyTiles == 1) {
          float* half = reinterpret_cast<float*>(smem + C::kPartOff);
          keys_sync();  // (it was read)
          if (gp == 1) half[row] = acc;
          keys_sync();
          if (gp == 0) total += half[row];
        }
        const bool owner = C::kKeyTiles == 2 || gp == 0;
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
          keys_sync();
          if (tid == 128) {
            int* ticket = p.tickets + 2 * c0 + 1;
            s_int[2] = atomicAdd(ticket, 1) == parts - 1;
            if (s_int[2]) *ticket = 0;  // as the next call expects it
          }
          keys_sync();
          writes = s_int[2];
          keys_sync();
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    // ------------------------------------------------------------ expansion
    using L = Kv4Layout<D>;
    constexpr int kSubs = C::kKeys / 64;  // cache tiles of a block that a warp takes
    const int dw = warp - 12;
    const Places<D> places(lane);
    uint32_t item = 0;
    bool ok = true;
    Words<D> k[kSubs];
    while (wk.next()) {
      const Kv4Request& rq = wk.job.rq;
      const int32_t* table = p.block_table + (size_t)wk.r * p.table_stride;
      const int tiles_mask = (1 << (p.cache.page_shift - 4)) - 1;
      // lanes u < kSubs: page ids of this warp's cache tiles of a block
      auto lane_page = [&](int blk) -> int {
        const int t = blk * C::kKeys + 16 * (kSubs * dw + lane);
        return lane < kSubs && t < rq.L ? table[t >> p.cache.page_shift] : -1;
      };
      auto fetch = [&](int blk, int head, int page) {
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
          const int t = blk * C::kKeys + 16 * (kSubs * dw + u);
          const int pg = __shfl_sync(0xffffffffu, page, u);
          if ((uint32_t)pg < (uint64_t)p.cache.num_pages) {  // (else, and behind the last key: whatever was there; its sums are not used)
            const size_t tile = ((size_t)head << (p.cache.page_shift - 4)) + ((t >> 4) & tiles_mask);
            load_words<D>(k[u], p.cache.pages + (int64_t)pg * p.page_bytes + tile * L::kBytes, lane);
          } else {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) k[u].w[i] = make_uint4(0u, 0u, 0u, 0u);
            k[u].s = k[u].s1 = 0;
          }
        }
      };
      int blk = (int)kv4_div(wk.x0, Hkv), head = (int)(wk.x0 - (long long)blk * Hkv);
      int page = lane_page(blk), page_next = lane_page(blk + 1);
      fetch(blk, head, page);
      for (long long x = wk.x0; x < wk.x1; ++x, ++item) {
        const uint32_t ks = item & 1;
        if (ok) ok = mbar_wait(b_kempty + 8 * ks, ((item >> 1) & 1) ^ 1, ab, 167);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
          const int ct = kSubs * dw + u;
          expand_keys<D>(sK + ks * C::kKBytes + (ct >> 3) * C::kKTile + 2048 * (ct & 7), k[u], places);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_kfull + 8 * ks);
        if (++head == Hkv) {
          head = 0;
          ++blk;
          page = page_next;
          page_next = lane_page(blk + 1);
        }
        if (x + 1 < wk.x1) fetch(blk, head, page);
      }
      if (!ok) break;
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
    kern<<<ctas, kThreads, WTile<D>::kSmem, stream>>>(p, tq);
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
