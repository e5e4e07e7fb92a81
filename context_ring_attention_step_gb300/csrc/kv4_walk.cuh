// kv4_walk.cuh -- device helpers shared by the two cache attention kernels: the
// fp16 arithmetic of expanded codes, and the line of work (requests' units of
// key blocks, one after the other) that a grid's CTAs cut into equal parts.
#pragma once

#include "kv4.h"
#include "tc.cuh"

namespace ra {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

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

// The power of two that brings a row whose largest magnitude has the bf16 bits
// `mx` to about 1 (`up`, applied to the row) and its inverse (returned, for the
// softmax scale); 1 for a row of zeros.  A row with an infinity or NaN gets a
// scale of NaN: its scores are infinite or NaN, and a softmax has no value then, even
// where all of them are -inf (which would look like a row without keys).
__device__ __forceinline__ float kv4_row_scale(uint32_t mx, float& up) {
  const int ex = mx == 0 || mx >= 0x7f80 ? 0 : min(max((int)(mx >> 7) - 127, -126), 126);
  up = __uint_as_float((uint32_t)(127 - ex) << 23);
  return mx >= 0x7f80 ? quiet_nan() : __uint_as_float((uint32_t)(127 + ex) << 23);
}

// What a CTA knows of a request.
struct Kv4Request {
  int b, n, L;     // first query row, query tokens, keys
  int row_tiles;
  int blocks;      // blocks of keys of each of its units (at least one: empty rows are written too)
  int bad;
};

// `kTiles`: the kernel of large row tiles, which takes the requests with at
// least split_rows rows; the other one takes those with fewer (split_rows = 0:
// all).  The requests of the other kernel have no row tiles here.
template <int RT, int KB, bool kTiles>
__device__ __forceinline__ Kv4Request kv4_request(const Kv4AttnParams& p, int r) {
  Kv4Request q;
  int b = p.cu_q[r], e = p.cu_q[r + 1];
  int L = p.kv_lens[r];
  q.bad = 0;
  if (b < 0 || e < b || e > p.Tq) {  // the request has no rows
    q.bad = RA_KV4_BAD_OFFSET;
    b = e = 0;
  }
  const long long cap = min((long long)p.table_width << p.cache.page_shift, (long long)kKv4MaxLength);
  if (L < 0 || L > cap) {  // its rows see no key
    q.bad = RA_KV4_BAD_LENGTH;
    L = 0;
  }
  q.b = b;
  q.n = e - b;
  q.L = L;
  const int G = p.Hq / p.cache.Hkv;
  const long long rows = (long long)q.n * G;
  const bool other = p.split_rows > 0 && (kTiles ? rows < p.split_rows : rows >= p.split_rows);
  q.row_tiles = other ? 0 : (int)((rows + RT - 1) / RT);
  q.blocks = max(1, (int)(((long long)L + KB - 1) / KB));
  return q;
}
// A unit's length on the line: its blocks, and before them `KU` places that
// stand for what beginning a unit costs (query rows, first tiles, merge).
template <int KU>
__device__ __forceinline__ long long kv4_request_work(const Kv4Request& q, int Hkv) {
  return (long long)q.row_tiles * Hkv * (q.blocks + KU);
}

__device__ __forceinline__ int kv4_key_limit(const Kv4AttnParams& p, const Kv4Request& q, int row) {
  return p.causal ? max(0, min(q.L, q.L - q.n + row / (p.Hq / p.cache.Hkv) + 1)) : q.L;
}

// Quotient of numbers that hardly ever need 64 bits.
__device__ __forceinline__ long long kv4_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// A place on the line of work, and what a CTA whose part ends at `end` does of
// the unit (r, rt, head) there: blocks [blk, blk + nb), possibly none.
struct Kv4Walk {
  long long pos;    // places before this one
  long long base;   // places before request r
  long long first;  // place of the unit's first block
  int r;
  int rt = 0, head = 0, blk = 0, nb = 0, t_end = 0;  // t_end: keys that some row of the unit sees
  Kv4Request rq;
  // look at the unit that holds pos (pos is inside the line)
  template <int RT, int KB, int KU, bool kTiles>
  __device__ __forceinline__ void enter(const Kv4AttnParams& p, long long end) {
    long long work;
    for (;; ++r) {  // (requests without rows have no work)
      rq = kv4_request<RT, KB, kTiles>(p, r);
      work = kv4_request_work<KU>(rq, p.cache.Hkv);
      if (pos < base + work || r + 1 >= p.R) break;
      base += work;
    }
    const int len = rq.blocks + KU;
    const long long unit = kv4_div(pos - base, len);
    first = base + unit * len + KU;
    rt = (int)kv4_div(unit, p.cache.Hkv);
    head = (int)(unit - (long long)rt * p.cache.Hkv);
    blk = (int)max(pos - first, 0ll);
    nb = (int)max(min(first + rq.blocks, end) - (first + blk), 0ll);
    t_end = kv4_key_limit(p, rq, min((rt + 1) * RT, rq.n * (p.Hq / p.cache.Hkv)) - 1);
  }
  // on to the next unit (or the end of the part)
  __device__ __forceinline__ void leave(long long end) { pos = min(first + rq.blocks, end); }
  // does the part hold all of the unit's blocks?
  __device__ __forceinline__ bool whole() const { return blk == 0 && nb == rq.blocks; }
};

// The line's length and this CTA's part [begin, end) of it.  Of `cut` parts the
// first `rest` have `size` + 1 places, the others `size`.
struct Kv4Line {
  long long total, cut, size, rest, begin, end;
  __device__ __forceinline__ int owner(long long x) const {  // the CTA whose part holds place x
    const long long longer = rest * (size + 1);
    return (int)(x < longer ? kv4_div(x, size + 1) : rest + kv4_div(x - longer, size));
  }
};

// Cut the line for this grid: `work(r)` places for each of R requests.  `r` and `base`
// receive the request that holds the first place of this CTA's part (when it has one) and
// the places before that request.  All threads of the CTA; s_sum has one entry a warp.
template <int kThreads, typename F>
__device__ __forceinline__ Kv4Line kv4_cut(int R, F work, long long* s_sum, long long* s_found, int& r, long long& base) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_found[0] = -1;
  long long mine = 0, total = 0;  // work of request `tid`; of all
  for (int i = tid; i < R; i += kThreads) {
    const long long w = work(i);
    if (i == tid) mine = w;
    total += w;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  Kv4Line line;
  line.total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) line.total += s_sum[w];
  // no part is empty: a unit's blocks, and its partial results, then lie in consecutive CTAs
  line.cut = min((long long)gridDim.x, line.total);
  const bool idle = blockIdx.x >= line.cut;
  line.size = idle ? 0 : kv4_div(line.total, line.cut);
  line.rest = line.total - line.size * line.cut;
  line.begin = idle ? 0 : line.size * blockIdx.x + min((long long)blockIdx.x, line.rest);
  line.end = idle ? 0 : line.begin + line.size + (blockIdx.x < line.rest ? 1 : 0);
  base = 0;
  r = 0;
  if (idle) return line;
  for (int r0 = 0; r0 < R; r0 += kThreads) {
    const long long w = r0 == 0 ? mine : r0 + tid < R ? work(r0 + tid) : 0;
    long long x = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    long long before = base, chunk = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += s_sum[i];
      chunk += s_sum[i];
    }
    if (line.begin >= before + x - w && line.begin < before + x) {
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
  return line;
}

// The same for attention's units; `wk` receives the place where this CTA's part begins.
template <int RT, int KB, int KU, bool kTiles, int kThreads>
__device__ __forceinline__ Kv4Line kv4_find_part(const Kv4AttnParams& p, long long* s_sum, long long* s_found,
                                                 Kv4Walk& wk, int& bad) {
  auto work = [&](int i) {
    const Kv4Request q = kv4_request<RT, KB, kTiles>(p, i);
    bad = max(bad, q.bad);
    return kv4_request_work<KU>(q, p.cache.Hkv);
  };
  const Kv4Line line = kv4_cut<kThreads>(p.R, work, s_sum, s_found, wk.r, wk.base);
  wk.pos = line.begin;
  return line;
}

// One thread of a CTA at its end: the grid's last CTA turns what was found into
// the call's status and leaves the counters as the next call expects them.
__device__ __forceinline__ void kv4_end(const Kv4AttnParams& p, int bad) {
  if (bad) atomicMax(p.found, bad);
  __threadfence();
  if (atomicAdd(p.ended, 1) == (int)gridDim.x - 1) {
    __threadfence();
    const int found = atomicExch(p.found, 0);
    *p.status = p.status_kept ? max(*p.status, found) : found;
    *p.ended = 0;
  }
}

}  // namespace ra
