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
//   * a row lies on D / 8 lanes, one 16-byte word each; its sum of squares is a
//     few shuffles, and so is the way to the other element of a pair (raw bf16,
//     four words), so nothing passes through shared memory but the angles;
//   * norm weight and angle make one coefficient of the own and one of the other
//     element, taken once a token and used for all its heads:
//     y = r (x cw + x' sw);
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

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight elements of a row as a lane holds them: bf16 (four words) or fp32 (eight).
template <bool kFp32>
struct Vec {
  uint32_t w[kFp32 ? 8 : 4];
  __device__ __forceinline__ void load(const void* p, int64_t off) {
    if (kFp32) {
      const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + off);
      const uint4 a = s[0], b = s[1];
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[kFp32 ? 4 : 0] = b.x; w[kFp32 ? 5 : 0] = b.y; w[kFp32 ? 6 : 0] = b.z; w[kFp32 ? 7 : 0] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + off);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (kFp32 ? 8 : 4); ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float at(int i) const {
    if (kFp32) return __uint_as_float(w[i % (kFp32 ? 8 : 4)]);
    return i & 1 ? hi_f(w[i >> 1]) : lo_f(w[i >> 1]);
  }
  // The other elements of the pairs; zero where an element is not rotated
  // (mask), so that an infinity there does not meet the coefficient 0.
  template <bool kInter>
  __device__ __forceinline__ Vec partner(int from, const uint32_t (&mask)[4]) const {
    Vec r;
#pragma unroll
    for (int i = 0; i < (kFp32 ? 8 : 4); ++i) {
      if (!kInter) r.w[i] = __shfl_sync(0xffffffffu, w[i], from) & mask[kFp32 ? i >> 1 : i];
      else if (kFp32) r.w[i] = w[i ^ 1] & mask[i >> 1];
      else r.w[i] = __byte_perm(w[i], 0, 0x1032) & mask[i % 4];
    }
    return r;
  }
};

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
// The inverse of the power of two that brings the row's largest magnitude (fp32 bits) to
// [1, 2); 1 for a row that is zero or not finite.  At most 2^60 beside an eps, which is far
// above the squares then and must not overflow when it is scaled along.
__device__ __forceinline__ float row_scale(uint32_t top, float eps) {
  int e = (int)(top >> 23) - 127;
  if (top == 0u || top >= 0x7f800000u) e = 0;
  e = min(max(e, eps > 0.f ? -60 : -126), 126);
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// cos and sin of a token's angles, j = 0 .. rot / 2 - 1, by one warp.
__device__ __forceinline__ void angles(const RopeParams& p, int32_t pos, float2* table, int lane) {
  __syncwarp();
  for (int j = lane; j < p.rot / 2; j += 32) {
    const uint64_t turn = p.turns[j] * (uint64_t)(uint32_t)pos;
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    table[j] = make_float2(c, s);
  }
  __syncwarp();
}

// What a lane needs to know of its eight elements.
template <int D, bool kInter>
struct Lane {
  int e0, from;       // first element; lane that holds the pairs' other elements (half layout)
  uint32_t mask[4];   // all ones where a pair of elements (2i, 2i + 1 of the lane) is rotated
  int first;          // angle of element 0 (half layout)
  float sign;         // of the sine, half layout: - for the first half
  __device__ __forceinline__ Lane(const RopeParams& p, int lane) {
    constexpr int LPR = D / 8;
    const int ch = lane % LPR, half = p.rot / 16;
    e0 = 8 * ch;
    from = lane;
    first = 0;
    sign = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) mask[i] = e0 + 2 * i < p.rot ? 0xffffffffu : 0u;
    if (!kInter && e0 < p.rot) {
      from = ch < half ? lane + half : lane - half;
      first = e0 < p.rot / 2 ? e0 : e0 - p.rot / 2;
      sign = ch < half ? -1.f : 1.f;
    }
  }
  // cosine and signed sine of element i
  __device__ __forceinline__ float2 turn(const float2* table, int i) const {
    if (!mask[i >> 1]) return make_float2(1.f, 0.f);
    if (kInter) {
      const float2 t = table[(e0 + i) >> 1];
      return make_float2(t.x, i & 1 ? t.y : -t.y);
    }
    const float2 t = table[first + i];
    return make_float2(t.x, sign * t.y);
  }
};

// Weight of element e (the pair's other element is weighted too).
__device__ __forceinline__ float weight(const RopeParams& p, const void* w, int e) {
  if (!w) return 1.f;
  return p.w_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[e]) : reinterpret_cast<const float*>(w)[e];
}
template <int D, bool kInter>
__device__ __forceinline__ int other(const RopeParams& p, const Lane<D, kInter>& ln, int i) {
  if (!ln.mask[i >> 1]) return ln.e0 + i;
  if (kInter) return ln.e0 + (i ^ 1);
  return ln.e0 + i + (ln.sign < 0.f ? p.rot / 2 : -(p.rot / 2));
}

// Work of one warp at a time: row groups (32 / (D / 8) neighbouring heads, one pass of the
// lanes) of one token.  Either all of its heads, the queries' first, or, where the tokens
// alone would not fill the GPU, a share of one side's.
struct Item {
  int64_t t;
  int side, h, h1;  // side and first head; end of the heads on this side
  bool both;        // goes on to the keys
};
template <int RPW>
__device__ __forceinline__ Item item_of(const RopeParams& p, int64_t it) {
  const int n = p.parts[0] + p.parts[1];
  if (n == 0) return Item{it, 0, 0, p.H[0], true};
  const int64_t t = it / n;
  int part = (int)(it - t * n);
  const int side = part >= p.parts[0];
  if (side) part -= p.parts[0];
  const int H = side ? p.H[1] : p.H[0], parts = side ? p.parts[1] : p.parts[0];
  const int per = ((H + RPW - 1) / RPW + parts - 1) / parts * RPW;
  return Item{t, side, min(part * per, H), min((part + 1) * per, H), false};
}
// On by n heads; false at the end.
__device__ __forceinline__ bool advance(const RopeParams& p, Item& c, int n) {
  c.h += n;
  if (c.h < c.h1) return true;
  if (!c.both || c.side) return false;
  c.side = 1;
  c.h = 0;
  c.h1 = p.H[1];
  return true;
}

// ------------------------------------------------------------------ forward

template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  extern __shared__ float2 s_angles[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* table = s_angles + warp * (p.rot / 2);
  const Lane<D, kInter> ln(p, lane);
  const int row = lane / LPR;
  const int64_t items = p.T * max(1, p.parts[0] + p.parts[1]);
  for (int64_t it = blockIdx.x * (int64_t)kWarps + warp; it < items; it += gridDim.x * (int64_t)kWarps) {
    Item c = item_of<RPW>(p, it);
    const int32_t pos = p.pos[c.t];
    auto load = [&](Vec<false> (&v)[U], const Item& at) {
      const RopeRows x = at.side ? p.x[1] : p.x[0];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = at.h + u * RPW + row;
        if (h < at.h1 && pos >= 0) v[u].load(x.p, at.t * x.stride + (int64_t)h * D + ln.e0);
        else v[u].clear();
      }
    };
    Vec<false> next[U];
    load(next, c);  // on the way while the angles are taken
    if (pos >= 0 && p.rot > 0) angles(p, pos, table, lane);
    float cw[8], sw[8];
    int side = -1;
#pragma unroll 1
    for (bool more = true; more;) {
      if (c.side != side) {
        side = c.side;
        const void* w = side ? p.w[1] : p.w[0];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 a = pos >= 0 ? ln.turn(table, i) : make_float2(0.f, 0.f);
          cw[i] = a.x * weight(p, w, ln.e0 + i);
          sw[i] = a.y * weight(p, w, other(p, ln, i));
        }
      }
      Vec<false> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = next[u];
      const Item at = c;
      more = advance(p, c, U * RPW);
      if (more) load(next, c);
      const RopeRows y = side ? p.y[1] : p.y[0];
      const int64_t yo = at.t * y.stride + ln.e0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at.h + u * RPW >= at.h1) break;
        const int h = at.h + u * RPW + row;
        float r = 1.f;
        if (p.norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[u].at(i), v[u].at(i), ss);
          ss = row_sum<D>(ss);
          r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
          const bool far = h < at.h1 && far_out(ss, p.eps);
          if (__any_sync(0xffffffffu, far)) {
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[u].at(i)) & 0x7fffffffu);
            const float down = row_scale(row_max<D>(top), p.eps);
            float s2 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s2 = fmaf(v[u].at(i) * down, v[u].at(i) * down, s2);
            s2 = row_sum<D>(s2);
            if (far) r = rsqrtf(fmaf(s2, 1.f / D, p.eps * down * down)) * down;
          }
        }
        const Vec<false> o = v[u].template partner<kInter>(ln.from, ln.mask);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (r first: the row times its coefficients alone may overflow, or lose small numbers)
          const float a = fmaf(v[u].at(2 * i) * r, cw[2 * i], o.at(2 * i) * r * sw[2 * i]);
          const float b = fmaf(v[u].at(2 * i + 1) * r, cw[2 * i + 1], o.at(2 * i + 1) * r * sw[2 * i + 1]);
          w[i] = pos >= 0 ? pack_bf16x2(a, b) : 0u;
        }
        if (h < at.h1)
          *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(y.p) + yo + (int64_t)h * D) =
              make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// ------------------------------------------------------------------ backward

template <int D, bool kInter, bool kFp32>
__global__ void __launch_bounds__(kThreads, 2) rope_bwd_kernel(const RopeParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 2;
  extern __shared__ float2 s_angles[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* table = s_angles + warp * (p.rot / 2);
  const Lane<D, kInter> ln(p, lane);
  const int row = lane / LPR;
  const int64_t items = p.T * max(1, p.parts[0] + p.parts[1]);
  float dwq[8], dwk[8];  // sums of the weights' gradients
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;

  for (int64_t it = blockIdx.x * (int64_t)kWarps + warp; it < items; it += gridDim.x * (int64_t)kWarps) {
    Item c = item_of<RPW>(p, it);
    const int32_t pos = p.pos[c.t];
    auto load = [&](Vec<false> (&v)[U], Vec<kFp32> (&g)[U], const Item& at) {
      const RopeRows x = at.side ? p.x[1] : p.x[0], gr = at.side ? p.g[1] : p.g[0];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = at.h + u * RPW + row;
        const bool in = h < at.h1 && pos >= 0;
        if (in && p.norm) v[u].load(x.p, at.t * x.stride + (int64_t)h * D + ln.e0);
        else v[u].clear();
        if (in) g[u].load(gr.p, at.t * gr.stride + (int64_t)h * D + ln.e0);
        else g[u].clear();
      }
    };
    Vec<false> v_next[U];
    Vec<kFp32> g_next[U];
    load(v_next, g_next, c);
    if (pos >= 0 && p.rot > 0) angles(p, pos, table, lane);
    float cs[8], sn[8];  // of the rotation by -t
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = pos >= 0 ? ln.turn(table, i) : make_float2(0.f, 0.f);
      cs[i] = a.x;
      sn[i] = -a.y;
    }
    float w[8];
    int side = -1;
#pragma unroll 1
    for (bool more = true; more;) {
      if (c.side != side) {
        side = c.side;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = weight(p, side ? p.w[1] : p.w[0], ln.e0 + i);
      }
      Vec<false> v[U];
      Vec<kFp32> g[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = v_next[u];
        g[u] = g_next[u];
      }
      const Item at = c;
      more = advance(p, c, U * RPW);
      if (more) load(v_next, g_next, c);
      const RopeRows y = side ? p.y[1] : p.y[0];
      const int64_t yo = at.t * y.stride + ln.e0;
      float dw[8] = {};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at.h + u * RPW >= at.h1) break;
        const Vec<kFp32> o = g[u].template partner<kInter>(ln.from, ln.mask);
        const int h = at.h + u * RPW + row;
        const bool in = h < at.h1 && pos >= 0;
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(g[u].at(i), cs[i], o.at(i) * sn[i]);
        if (p.norm) {
          float ss = 0.f, dot = 0.f, down = 1.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(v[u].at(i), v[u].at(i), ss);
            dot = fmaf(d[i] * w[i], v[u].at(i), dot);
          }
          ss = row_sum<D>(ss);
          dot = row_sum<D>(dot);
          float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
          const bool far = in && far_out(ss, p.eps);
          if (__any_sync(0xffffffffu, far)) {
            // as forward; the row itself is scaled (`down`), and r is the scaled row's
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[u].at(i)) & 0x7fffffffu);
            const float dn = row_scale(row_max<D>(top), p.eps);
            float s2 = 0.f, d2 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float xs = v[u].at(i) * dn;
              s2 = fmaf(xs, xs, s2);
              d2 = fmaf(d[i] * w[i], xs, d2);
            }
            s2 = row_sum<D>(s2);
            d2 = row_sum<D>(d2);
            if (far) {
              r = rsqrtf(fmaf(s2, 1.f / D, p.eps * dn * dn));
              dot = d2;
              down = dn;
            }
          }
          const float mean = dot * r * (1.f / D);  // of h w r x
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float n = v[u].at(i) * down * r;
            if (in) dw[i] = fmaf(d[i], n, dw[i]);
            d[i] = fmaf(-n, mean, d[i] * w[i]) * r * down;
          }
        }
        if (h < at.h1) {
          uint4 out = make_uint4(0u, 0u, 0u, 0u);
          if (pos >= 0)
            out = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[4], d[5]),
                             pack_bf16x2(d[6], d[7]));
          *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(y.p) + yo + (int64_t)h * D) = out;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dwq[i] += side ? 0.f : dw[i];
        dwk[i] += side ? dw[i] : 0.f;
      }
    }
  }
  if (!p.partials) return;
  // this CTA's sums, in a fixed order: rows of a warp, then the warps
  __shared__ float s_dw[kWarps][D];
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = side ? dwk[i] : dwq[i];
#pragma unroll
      for (int d = LPR; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      if (row == 0) s_dw[warp][ln.e0 + i] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += s_dw[k][e];
      p.partials[((size_t)blockIdx.x * 2 + side) * D + e] = v;
    }
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

// A token's heads on one warp (parts 0) where the tokens alone fill the GPU, else each side's
// shared out over some.
int64_t share_out(RopeParams& p, int D, int sms) {
  const int rows_at_once = 256 / D;
  const int64_t want = (int64_t)sms * 32;  // warps
  p.parts[0] = p.parts[1] = 0;
  if (p.T >= want) return p.T;
  const int g0 = (p.H[0] + rows_at_once - 1) / rows_at_once, g1 = (p.H[1] + rows_at_once - 1) / rows_at_once;
  const int64_t warps = std::max<int64_t>(2, want / std::max<int64_t>(1, p.T));
  const int per = (int)std::max<int64_t>(1, (g0 + g1 + warps - 1) / warps);  // row groups of a warp
  p.parts[0] = (g0 + per - 1) / per;
  p.parts[1] = (g1 + per - 1) / per;
  return p.T * (p.parts[0] + p.parts[1]);
}

}  // namespace

cudaError_t launch_rope_fwd(int D, bool interleaved, RopeParams p, int sms, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  const int64_t items = share_out(p, D, sms);
  const unsigned ctas = (unsigned)std::min<int64_t>((items + kWarps - 1) / kWarps, (int64_t)sms * 8);
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
  const int64_t items = share_out(p, D, sms);
  const unsigned ctas = (unsigned)std::max<int64_t>(
      1, std::min<int64_t>({(items + kWarps - 1) / kWarps, (int64_t)sms * 4, (int64_t)kRopeMaxCtas}));
  const size_t smem = (size_t)kWarps * (p.rot / 2) * sizeof(float2);
  auto go = [&](auto kern) {
    kern<<<ctas, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  };
  auto pick = [&](auto inter) {
    constexpr bool I = decltype(inter)::value;
    if (D == 64) return g_fp32 ? go(rope_bwd_kernel<64, I, true>) : go(rope_bwd_kernel<64, I, false>);
    if (D == 128) return g_fp32 ? go(rope_bwd_kernel<128, I, true>) : go(rope_bwd_kernel<128, I, false>);
    if (D == 256) return g_fp32 ? go(rope_bwd_kernel<256, I, true>) : go(rope_bwd_kernel<256, I, false>);
    return cudaErrorInvalidValue;
  };
  cudaError_t e = interleaved ? pick(std::true_type{}) : pick(std::false_type{});
  if (e != cudaSuccess || !p.partials) return e;
  rope_dw_kernel<<<2 * D / 32, 256, 0, stream>>>(p.partials, (int)ctas, D, dw[0], dw[1]);
  return cudaGetLastError();
}

}  // namespace ra
