// rope.cu -- root-mean-square norms of query and key rows for each head and the
// rotation by their positions, in one pass, and the gradients of both.
//
// A row x [D] with weight w [D] at position p:
//   r = (mean x^2 + eps)^(-1/2),  u = r x w   (without the norm u = x),
//   y_a = u_a cos t - u_b sin t,  y_b = u_b cos t + u_a sin t,  t = p f_i,
// for the pairs (a, b) of the first `rot` elements: (i, i + rot/2), or
// (2i, 2i + 1) interleaved; the others are y = u.  With g = dL/dy and h the
// rotation of g by -t,
//   dw = sum over tokens and heads of h r x,   dx = r (h w - r x mean(h w r x)).
//
// Both only move bytes: 4 D a row forward, 6 D backward.  Hence
//   * a row lies on D / 8 lanes, eight elements each: four neighbours and the other
//     elements of their pairs, so that a pair never crosses lanes; the sum of squares is a
//     few shuffles, and nothing passes through shared memory but the angles;
//   * norm weight and angle make one coefficient of the own and one of the other
//     element, taken once a token and used for all its heads: y_a = r (x_a ca + x_b sa).
//     Arithmetic runs on pairs of fp32 numbers (one instruction for two);
//   * the angle is the product of p and the frequency in turns as a 64-bit
//     fixed-point fraction, where whole turns fall out exactly: at position 2^20
//     an fp32 product would be off by 0.03 of a radian.
// Rows at a negative position are no tokens: zero, and without a gradient.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "rope.h"
#include "tc.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs of 8 warps an SM, and rows (of 32 lanes) that a warp has on the way at once.  The grids
// are as many CTAs as run at the same time.  32768 tokens of 40 heads (head_dim 128) take forward
// 131, 106 and 107 us with 2, 3 and 4 CTAs of 4 rows; 65536 tokens backward 551 us as 3 x 1, 478
// as 3 x 2, 395 as 2 x 2, 327 as 2 x 4: what is on the way counts, more than the warps do.
constexpr int kFwdCtas = 3, kFwdRows = 4, kBwdCtas = 2, kBwdRows = 4;

__device__ __forceinline__ uint64_t widen(uint32_t w) {  // two bf16 numbers
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float f2_sum(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return a + b;
}
__device__ __forceinline__ uint64_t f2_both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ uint64_t f2_neg(uint64_t x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ uint64_t f2_swap(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return f2_pack(b, a);
}
__device__ __forceinline__ uint32_t narrow(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return pack_bf16x2(a, b);
}

// A lane's eight elements of a row, as they came: four at `a`, four at `b` (bf16, or fp32).
template <bool kFp32>
struct Vec {
  uint4 w;      // bf16: a in x, y, b in z, w
  uint4 w2;     // fp32: a in w, b here
  typedef typename std::conditional<kFp32, float, __nv_bfloat16>::type T;
  __device__ __forceinline__ void load(const T* a, int b) {  // b: from there to the other four
    if constexpr (kFp32) {
      w = *reinterpret_cast<const uint4*>(a);
      w2 = *reinterpret_cast<const uint4*>(a + b);
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(a + b);
      w = make_uint4(x.x, x.y, y.x, y.y);
    }
  }
  __device__ __forceinline__ void clear() { w = w2 = make_uint4(0u, 0u, 0u, 0u); }
  // fp32 pairs: elements a, a + 1; a + 2, a + 3; the same of b
  __device__ __forceinline__ void get(uint64_t (&x)[4]) const {
    if (kFp32) {
      x[0] = f2_pack(__uint_as_float(w.x), __uint_as_float(w.y));
      x[1] = f2_pack(__uint_as_float(w.z), __uint_as_float(w.w));
      x[2] = f2_pack(__uint_as_float(w2.x), __uint_as_float(w2.y));
      x[3] = f2_pack(__uint_as_float(w2.z), __uint_as_float(w2.w));
    } else {
      x[0] = widen(w.x); x[1] = widen(w.y); x[2] = widen(w.z); x[3] = widen(w.w);
    }
  }
};
__device__ __forceinline__ void store(__nv_bfloat16* a, int b, const uint64_t (&x)[4]) {
  *reinterpret_cast<uint2*>(a) = make_uint2(narrow(x[0]), narrow(x[1]));
  *reinterpret_cast<uint2*>(a + b) = make_uint2(narrow(x[2]), narrow(x[3]));
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = D / 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
template <int D>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int d = D / 16; d; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// Squares of bf16 numbers leave fp32's range below 2^-63 and above 2^63.  Rows whose sum of
// squares comes near its ends (the lower one matters only beside an eps that small) are
// scaled by a power of two first.
__device__ __forceinline__ bool far_out(float ss, float eps) { return !(ss <= 0x1p120f) || (ss < 0x1p-80f && eps < 0x1p-60f); }
// Likewise the sum of h w x (backward): above, products leave the range; below, what was lost of them shows
// beside h w, where the eps is small enough for the row to count at all.
__device__ __forceinline__ bool products_far_out(float dot, float eps) {
  return !(fabsf(dot) <= 0x1p120f) || (fabsf(dot) < 0x1p-90f && eps < 0x1p-30f);
}
// The inverse of the power of two that brings the row's largest magnitude (fp32 bits) to
// [1, 2); 1 for a row that is zero or not finite.  At most 2^60 beside an eps, which is far
// above the squares then and must not overflow when it is scaled along.
__device__ __forceinline__ float row_scale(uint32_t top, float eps) {
  int e = (int)(top >> 23) - 127;
  if (top == 0u || top >= 0x7f800000u) e = 0;
  e = min(max(e, eps > 0.f ? -60 : -126), 126);
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// The row times that power of two, and the power: what a row with a far sum is scaled by.
template <int D>
__device__ __forceinline__ float scale_row(uint64_t (&x)[4], float eps, bool far) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_unpack(x[i], a, b);
    top = max(top, max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
  }
  const float down = row_scale(row_max<D>(top), eps);
  if (!far) return 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_mul(x[i], f2_both(down));
  return down;
}
__device__ __forceinline__ float square_sum(const uint64_t (&x)[4]) {
  uint64_t s = f2_mul(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = f2_fma(x[i], x[i], s);
  return f2_sum(s);
}

// cos and sin of a token's angles, j = 0 .. rot / 2 - 1, by one warp.
__device__ __forceinline__ void angles(const RopeParams& p, int32_t pos, float2* table, int lane) {
  __syncwarp();
#pragma unroll 1
  for (int j = lane; j < p.rot / 2; j += 32) {
    const uint64_t turn = p.turns[j] * (uint64_t)(uint32_t)pos;
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    table[j] = make_float2(c, s);
  }
  __syncwarp();
}

// The elements of a row that a lane holds: a .. a + 3 and b .. b + 3.
//   half layout: the first rot / 8 lanes hold pairs (i, i + rot / 2), the others
//     neighbours behind the rotated part; interleaved: eight neighbours.
template <int D, bool kInter>
struct Lane {
  int a, b;
  bool turns;  // half layout: the lane's elements are rotated
  __device__ __forceinline__ Lane(const RopeParams& p, int lane) {
    const int l = lane % (D / 8);
    turns = !kInter && 8 * l < p.rot;
    a = turns ? 4 * l : 8 * l;
    b = turns ? 4 * l + p.rot / 2 : 8 * l + 4;
  }
  // Cosines and sines of the pairs (half layout: c[0], c[1] for a .. a + 3 and again for
  // b; interleaved: both elements of a pair alike).  Elements that are not rotated: 1 and 0.
  __device__ __forceinline__ void angles_of(const RopeParams& p, const float2* table, uint64_t (&c)[4],
                                            uint64_t (&s)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kInter) {
        const int e = (i < 2 ? a : b - 4) + 2 * i;  // (b = a + 4)
        const float2 t = e < p.rot ? table[e >> 1] : make_float2(1.f, 0.f);
        c[i] = f2_both(t.x);
        s[i] = f2_pack(-t.y, t.y);
      } else if (i < 2) {
        float2 t = make_float2(1.f, 0.f), u = t;
        if (turns) {
          t = table[a + 2 * i];
          u = table[a + 2 * i + 1];
        }
        c[i] = c[i + 2] = f2_pack(t.x, u.x);
        s[i] = f2_pack(-t.y, -u.y);
        s[i + 2] = f2_pack(t.y, u.y);
      }
    }
  }
  // The other elements of the pairs; zero where nothing turns, so that an infinity there
  // does not meet the coefficient 0.
  __device__ __forceinline__ void others(const RopeParams& p, const uint64_t (&x)[4], uint64_t (&o)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kInter) o[i] = a + 2 * i < p.rot ? f2_swap(x[i]) : 0ull;
      else o[i] = turns ? x[i ^ 2] : 0ull;
    }
  }
  __device__ __forceinline__ void weights(const float* w, uint64_t (&v)[4]) const {
    const float4 x = *reinterpret_cast<const float4*>(w + a), y = *reinterpret_cast<const float4*>(w + b);
    v[0] = f2_pack(x.x, x.y);
    v[1] = f2_pack(x.z, x.w);
    v[2] = f2_pack(y.x, y.y);
    v[3] = f2_pack(y.z, y.w);
  }
};

// Both weights as fp32, ones where there is none.
template <int D>
__device__ __forceinline__ void read_weights(const RopeParams& p, float (&w)[2][D]) {
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const void* src = i < D ? p.w[0] : p.w[1];
    const int e = i % D;
    w[i / D][e] = !src      ? 1.f
                  : p.w_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src)[e])
                             : reinterpret_cast<const float*>(src)[e];
  }
  __syncthreads();
}

// Work of one warp at a time: one token, either all of its heads, or, where the tokens
// alone would not fill the GPU, a share of one side's.
struct Item {
  int64_t t;
  int h0[2], h1[2];  // heads of either side
};
template <int RPW>
__device__ __forceinline__ Item item_of(const RopeParams& p, int64_t it) {
  const int n = p.parts[0] + p.parts[1];
  if (n == 0) return Item{it, {0, 0}, {p.H[0], p.H[1]}};
  Item c{it / n, {0, 0}, {0, 0}};
  const int part = (int)(it - c.t * n);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int k = part - (s ? p.parts[0] : 0);
    if (k < 0 || k >= p.parts[s]) continue;
    const int per = ((p.H[s] + RPW - 1) / RPW + p.parts[s] - 1) / p.parts[s] * RPW;
    c.h0[s] = min(k * per, p.H[s]);
    c.h1[s] = min(k * per + per, p.H[s]);
  }
  return c;
}

template <typename T>
__device__ __forceinline__ T* at(const RopeRows& r, int64_t off) { return reinterpret_cast<T*>(r.p) + off; }

// `n` heads of zeros.
template <int D>
__device__ __forceinline__ void zero_heads(__nv_bfloat16* y, int db, int n, int row) {
  const uint64_t z[4] = {};
  for (int h = row; h < n; h += 256 / D) store(y + h * D, db, z);
}

// ------------------------------------------------------------------ forward

// One row (and those of the warp's other lanes) from x to y; `in`: it is one of the heads.
template <int D, bool kInter>
__device__ __forceinline__ void fwd_row(const RopeParams& p, const Lane<D, kInter>& ln, const Vec<false>& v,
                                        const uint64_t (&ca)[4], const uint64_t (&sa)[4], __nv_bfloat16* y, bool in) {
  uint64_t x[4], o[4];
  v.get(x);
  uint64_t r2 = f2_both(1.f);
  if (p.norm) {
    float ss = row_sum<D>(square_sum(x)), e = p.eps;
    const bool far = in && far_out(ss, p.eps);
    if (__any_sync(0xffffffffu, far)) {
      const float down = scale_row<D>(x, p.eps, far);
      const float s2 = row_sum<D>(square_sum(x));
      if (far) {
        ss = s2;
        e = p.eps * down * down;
      }
    }
    r2 = f2_both(rsqrtf(fmaf(ss, 1.f / D, e)));
  }
  ln.others(p, x, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_mul(f2_fma(x[i], ca[i], f2_mul(o[i], sa[i])), r2);
  if (in) store(y, ln.b - ln.a, x);
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, kFwdCtas) rope_fwd_kernel(const RopeParams p) {
  constexpr int RPW = 256 / D, U = kFwdRows;  // rows of a warp at once, and how often before it waits for them
  extern __shared__ float2 s_angles[];
  __shared__ __align__(16) float s_w[2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* table = s_angles + warp * (p.rot / 2);
  const Lane<D, kInter> ln(p, lane);
  const int row = lane / (D / 8), db = ln.b - ln.a;
  const int64_t items = p.T * max(1, p.parts[0] + p.parts[1]);
  read_weights<D>(p, s_w);
  for (int64_t it = blockIdx.x * (int64_t)kWarps + warp; it < items; it += gridDim.x * (int64_t)kWarps) {
    const Item c = item_of<RPW>(p, it);
    const int32_t pos = p.pos[c.t];
    if (pos >= 0 && p.rot > 0) angles(p, pos, table, lane);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int h0 = side ? c.h0[1] : c.h0[0], n = (side ? c.h1[1] : c.h1[0]) - h0;
      if (n <= 0) continue;
      const RopeRows& xr = side ? p.x[1] : p.x[0];
      const RopeRows& yr = side ? p.y[1] : p.y[0];
      const __nv_bfloat16* x = at<__nv_bfloat16>(xr, c.t * xr.stride + h0 * D + ln.a);
      __nv_bfloat16* y = at<__nv_bfloat16>(yr, c.t * yr.stride + h0 * D + ln.a);
      if (pos < 0) {
        zero_heads<D>(y, db, n, row);
        continue;
      }
      uint64_t ca[4], sa[4];  // coefficients of the own and of the pair's other element
      {
        uint64_t w[4], wo[4];
        ln.weights(s_w[side], w);
        ln.others(p, w, wo);
        ln.angles_of(p, table, ca, sa);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ca[i] = f2_mul(ca[i], w[i]);
          sa[i] = f2_mul(sa[i], wo[i]);
        }
      }
      x += row * D;
      y += row * D;
      int h = 0;
#pragma unroll 1
      for (; h + U * RPW <= n; h += U * RPW, x += U * RPW * D, y += U * RPW * D) {
        Vec<false> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u].load(x + u * RPW * D, db);
#pragma unroll
        for (int u = 0; u < U; ++u) fwd_row<D, kInter>(p, ln, v[u], ca, sa, y + u * RPW * D, true);
      }
      if (h < n) {  // the last ones, on the way together too (one after the other, 7 + 1 heads took 101 us for 77)
        Vec<false> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          v[u].clear();
          if (h + u * RPW + row < n) v[u].load(x + u * RPW * D, db);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h + u * RPW < n) fwd_row<D, kInter>(p, ln, v[u], ca, sa, y + u * RPW * D, h + u * RPW + row < n);
      }
    }
  }
}

// ------------------------------------------------------------------ backward

template <int D, bool kInter, bool kFp32, bool kNorm>
__device__ __forceinline__ void bwd_row(const RopeParams& p, const Lane<D, kInter>& ln, const Vec<false>& v,
                                        const Vec<kFp32>& g, const uint64_t (&cs)[4], const uint64_t (&sn)[4],
                                        const uint64_t (&w)[4], uint64_t (&dw)[4], __nv_bfloat16* y, bool in) {
  uint64_t x[4], d[4], o[4];
  g.get(d);
  ln.others(p, d, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = f2_fma(d[i], cs[i], f2_mul(o[i], sn[i]));  // h
  if (kNorm) {
    v.get(x);
    uint64_t hw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) hw[i] = f2_mul(d[i], w[i]);
    auto product = [&]() {
      uint64_t s = f2_mul(hw[0], x[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) s = f2_fma(hw[i], x[i], s);
      return f2_sum(s);
    };
    float ss = row_sum<D>(square_sum(x)), dot = row_sum<D>(product()), e = p.eps, up = 1.f;
    const bool far = in && (far_out(ss, p.eps) || products_far_out(dot, p.eps));
    if (__any_sync(0xffffffffu, far)) {
      // as forward: r is the scaled row's then, and r times the power of two that of the row itself.  h w takes
      // the power, of one above 2^63 that much, and at most 2^-16 where the sum was large; r takes the rest
      const float down = scale_row<D>(x, p.eps, far);
      if (far) {
        const float take = fminf(down, fabsf(dot) <= 0x1p100f ? 0x1p63f : 0x1p-16f);
        e = p.eps * down * down;
        up = down / take;
#pragma unroll
        for (int i = 0; i < 4; ++i) hw[i] = f2_mul(hw[i], f2_both(take));
      }
      const float s2 = row_sum<D>(square_sum(x)), d2 = row_sum<D>(product());
      if (far) {
        ss = s2;
        dot = d2;
      }
    }
    const float r = rsqrtf(fmaf(ss, 1.f / D, e));
    const float mean = dot * r * (1.f / D);  // of h w r x
    const uint64_t r2 = f2_both(r), m2 = f2_both(-mean), rd = f2_both(r * up);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t n = f2_mul(x[i], r2);
      if (in) dw[i] = f2_fma(d[i], n, dw[i]);
      d[i] = f2_mul(f2_fma(n, m2, hw[i]), rd);
    }
  }
  if (in) store(y, ln.b - ln.a, d);
}

template <int D, bool kInter, bool kFp32, bool kNorm>
__global__ void __launch_bounds__(kThreads, kBwdCtas) rope_bwd_kernel(const RopeParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = kBwdRows;
  typedef typename Vec<kFp32>::T G;
  extern __shared__ __align__(16) float2 s_angles[];
  __shared__ __align__(16) float s_w[2][D];
  // a lane's sums of the weights' gradients: in registers for one side of a token only
  __shared__ __align__(16) uint64_t s_dw[2][4][kNorm ? kThreads : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2* table = s_angles + warp * (p.rot / 2);
  const Lane<D, kInter> ln(p, lane);
  const int row = lane / LPR, db = ln.b - ln.a;
  const int64_t items = p.T * max(1, p.parts[0] + p.parts[1]);
  if (kNorm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s_dw[0][i][tid] = s_dw[1][i][tid] = 0ull;
  }
  read_weights<D>(p, s_w);
  for (int64_t it = blockIdx.x * (int64_t)kWarps + warp; it < items; it += gridDim.x * (int64_t)kWarps) {
    const Item c = item_of<RPW>(p, it);
    const int32_t pos = p.pos[c.t];
    uint64_t cs[4], sn[4];
    if (pos >= 0) {
      if (p.rot > 0) angles(p, pos, table, lane);
      ln.angles_of(p, table, cs, sn);
#pragma unroll
      for (int i = 0; i < 4; ++i) sn[i] = f2_neg(sn[i]);  // back, by -t
    }
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int h0 = side ? c.h0[1] : c.h0[0], n = (side ? c.h1[1] : c.h1[0]) - h0;
      if (n <= 0) continue;
      const RopeRows& xr = side ? p.x[1] : p.x[0];
      const RopeRows& gr = side ? p.g[1] : p.g[0];
      const RopeRows& yr = side ? p.y[1] : p.y[0];
      __nv_bfloat16* y = at<__nv_bfloat16>(yr, c.t * yr.stride + h0 * D + ln.a);
      if (pos < 0) {
        zero_heads<D>(y, db, n, row);
        continue;
      }
      y += row * D;
      const __nv_bfloat16* x = at<__nv_bfloat16>(xr, c.t * xr.stride + (h0 + row) * D + ln.a);
      const G* g = at<G>(gr, c.t * gr.stride + (h0 + row) * D + ln.a);
      uint64_t w[4], dw[4] = {};
      ln.weights(s_w[side], w);
      int h = 0;
#pragma unroll 1
      for (; h + U * RPW <= n; h += U * RPW, x += U * RPW * D, g += U * RPW * D, y += U * RPW * D) {
        Vec<false> v[U];
        Vec<kFp32> gv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (kNorm) v[u].load(x + u * RPW * D, db);
          gv[u].load(g + u * RPW * D, db);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          bwd_row<D, kInter, kFp32, kNorm>(p, ln, v[u], gv[u], cs, sn, w, dw, y + u * RPW * D, true);
      }
      if (h < n) {  // the last ones
        Vec<false> v[U];
        Vec<kFp32> gv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          v[u].clear();
          gv[u].clear();
          if (h + u * RPW + row < n) {
            if (kNorm) v[u].load(x + u * RPW * D, db);
            gv[u].load(g + u * RPW * D, db);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h + u * RPW < n)
            bwd_row<D, kInter, kFp32, kNorm>(p, ln, v[u], gv[u], cs, sn, w, dw, y + u * RPW * D, h + u * RPW + row < n);
      }
      if (kNorm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s_dw[side][i][tid] = f2_add(s_dw[side][i][tid], dw[i]);
      }
    }
  }
  if (!kNorm || !p.partials) return;
  // this CTA's sums, always in the same order: the lanes that hold the same elements, warp by warp
  __syncthreads();
  for (int i = tid; i < 2 * D / 2; i += kThreads) {
    const int side = i / (D / 2), j = i % (D / 2) % 4, l = i % (D / 2) / 4;  // pair j of lane l of a row
    uint64_t v = 0ull;
    for (int k = l; k < kThreads; k += LPR) v = f2_add(v, s_dw[side][j][k]);
    const Lane<D, kInter> o(p, l);
    float* dst = p.partials + ((size_t)blockIdx.x * 2 + side) * D + (j < 2 ? o.a : o.b - 4) + 2 * j;
    f2_unpack(v, dst[0], dst[1]);
  }
}

// Sum the CTAs' partial sums, 32 columns a CTA, always in the same order.
__global__ void __launch_bounds__(256) rope_dw_kernel(const float* partials, int ctas, int D, float* dq, float* dk) {
  __shared__ float s[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float v = 0.f;
#pragma unroll 8
  for (int i = k; i < ctas; i += 8) v += partials[(size_t)i * 2 * D + col];
  s[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][threadIdx.x & 31];
    float* dst = col < D ? dq : dk;
    if (dst) dst[col < D ? col : col - D] = v;
  }
}

// CTAs for this many tokens: a token's heads go to one warp (parts 0), or, of fewer tokens than a
// quarter of the warps that run at once (912 forward, 608 backward), to several warps, each with the
// token's angles to make.  Shared out / not, 40 heads of 128, us: forward 256 tokens 4.1 / 7.4, 760 6.4 / 7.6,
// 1024 7.9 / 7.6, 3600 14.2 / 10.7; backward 256 tokens 7.8 / 11.0, 600 11.2 / 11.3, 1024 13.5 / 11.4.
unsigned share_out(RopeParams& p, int D, int sms, int per_sm) {
  const int rows_at_once = 256 / D;
  const int64_t want = (int64_t)sms * per_sm * kWarps;  // warps that run at once
  int64_t items = p.T;
  p.parts[0] = p.parts[1] = 0;
  if (4 * p.T < want) {
    const int g0 = (p.H[0] + rows_at_once - 1) / rows_at_once, g1 = (p.H[1] + rows_at_once - 1) / rows_at_once;
    const int64_t warps = std::max<int64_t>(2, want / std::max<int64_t>(1, p.T));
    const int per = (int)std::max<int64_t>(1, (g0 + g1 + warps - 1) / warps);  // rows (of 32 lanes) of a warp
    p.parts[0] = (g0 + per - 1) / per;
    p.parts[1] = (g1 + per - 1) / per;
    items *= p.parts[0] + p.parts[1];
  }
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + kWarps - 1) / kWarps, (int64_t)sms * per_sm));
}

}  // namespace

cudaError_t launch_rope_fwd(int D, bool interleaved, RopeParams p, int sms, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  const unsigned ctas = share_out(p, D, sms, kFwdCtas);
  const size_t smem = (size_t)kWarps * (p.rot / 2) * sizeof(float2);
  auto go = [&](auto kern) {
    kern<<<ctas, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  };
  if (D == 64) return interleaved ? go(rope_fwd_kernel<64, true>) : go(rope_fwd_kernel<64, false>);
  if (D == 128) return interleaved ? go(rope_fwd_kernel<128, true>) : go(rope_fwd_kernel<128, false>);
  if (D == 256) return interleaved ? go(rope_fwd_kernel<256, true>) : go(rope_fwd_kernel<256, false>);
  return cudaErrorInvalidValue;
}

cudaError_t launch_rope_bwd(int D, bool interleaved, bool g_fp32, RopeParams p, int sms, float* dw[2],
                            cudaStream_t stream) {
  sms = std::min(sms, kRopeMaxCtas / kBwdCtas);
  const unsigned ctas = share_out(p, D, sms, kBwdCtas);
  const size_t smem = (size_t)kWarps * (p.rot / 2) * sizeof(float2);
  auto go = [&](auto kern) {
    kern<<<ctas, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  };
  auto pick = [&](auto inter, auto fp32, auto norm) {
    constexpr bool I = decltype(inter)::value, F = decltype(fp32)::value, N = decltype(norm)::value;
    return D == 64    ? go(rope_bwd_kernel<64, I, F, N>)
           : D == 128 ? go(rope_bwd_kernel<128, I, F, N>)
           : D == 256 ? go(rope_bwd_kernel<256, I, F, N>)
                      : cudaErrorInvalidValue;
  };
  auto with_norm = [&](auto inter, auto fp32) {
    return p.norm ? pick(inter, fp32, std::true_type{}) : pick(inter, fp32, std::false_type{});
  };
  auto with_type = [&](auto inter) {
    return g_fp32 ? with_norm(inter, std::true_type{}) : with_norm(inter, std::false_type{});
  };
  const cudaError_t e = interleaved ? with_type(std::true_type{}) : with_type(std::false_type{});
  if (e != cudaSuccess || !p.partials) return e;
  rope_dw_kernel<<<2 * D / 32, 256, 0, stream>>>(p.partials, (int)ctas, D, dw[0], dw[1]);
  return cudaGetLastError();
}

}  // namespace ra
