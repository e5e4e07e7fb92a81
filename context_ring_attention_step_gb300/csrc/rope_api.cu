// rope_api.cu -- C entry points of the norms with rotation: argument checks and
// launches.  Nothing here allocates or synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/ring_attn.h"
#include "ring_attn_internal.h"
#include "rope.h"

namespace {

using ra::aligned;

ra_status fail(ra_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return ra::set_last_error(st, buf);
}
ra_status cuda_fail(cudaError_t e, const char* what) { return fail(RA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

ra_status check_head_dim(int32_t D) {
  return D == 64 || D == 128 || D == 256 ? RA_OK : fail(RA_ERR_UNSUPPORTED, "head_dim %d: 64, 128 or 256", D);
}

// T rows of `row` bytes, `stride` bytes apart.
struct Span {
  const void* p;
  int64_t stride, row, T;
  const char* name;
  size_t bytes() const { return T > 0 ? (size_t)((T - 1) * stride + row) : 0; }
};
// Do two sets of rows share a byte?  Slices of one fused tensor lie between one
// another without doing so: rows the same distance apart are compared within it.
bool share_bytes(const Span& a, const Span& b) {
  if (!ra::overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
  if (a.T < 2 || b.T < 2 || a.stride != b.stride) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t s = (uintptr_t)a.stride;
  const uintptr_t d = y >= x ? (y - x) % s : (s - (x - y) % s) % s;  // b's rows begin d bytes behind a's (modulo the distance)
  return d < (uintptr_t)a.row || d + (uintptr_t)b.row > s;
}

ra_status check_shape(const ra_norm_rope* r, ra::RopeParams* p) {
  if (!r) return fail(RA_ERR_INVALID_ARG, "shape is NULL");
  ra_status rs = check_head_dim(r->head_dim);
  if (rs != RA_OK) return rs;
  if (r->num_tokens < 0 || r->num_tokens > 0x7fffffff)
    return fail(RA_ERR_INVALID_ARG, "num_tokens %lld outside [0, 2^31)", (long long)r->num_tokens);
  if (r->num_q_heads < 1 || r->num_q_heads > 65536 || r->num_kv_heads < 1 || r->num_kv_heads > 65536)
    return fail(RA_ERR_INVALID_ARG, "num_q_heads %d, num_kv_heads %d outside [1, 65536]", r->num_q_heads, r->num_kv_heads);
  if (r->rotary_dim < 0 || r->rotary_dim > r->head_dim || r->rotary_dim % (r->interleaved ? 2 : 8))
    return fail(RA_ERR_UNSUPPORTED, "rotary_dim %d: a multiple of %d up to head_dim %d", r->rotary_dim,
                r->interleaved ? 2 : 8, r->head_dim);
  if (r->norm && !(r->eps >= 0.f && std::isfinite(r->eps))) return fail(RA_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!r->norm && (r->q_weight || r->k_weight)) return fail(RA_ERR_INVALID_ARG, "weights need the norm");
  if (r->num_tokens > 0 && !r->positions) return fail(RA_ERR_INVALID_ARG, "positions is NULL");
  if (r->rotary_dim > 0 && !r->turns) return fail(RA_ERR_INVALID_ARG, "turns is NULL");
  if (!aligned(r->positions, 4) || !aligned(r->turns, 8) || !aligned(r->q_weight, r->weights_bf16 ? 2 : 4) ||
      !aligned(r->k_weight, r->weights_bf16 ? 2 : 4))
    return fail(RA_ERR_INVALID_ARG, "positions must be 4-byte, turns 8-byte aligned, the weights to their type");
  p->T = r->num_tokens;
  p->H[0] = r->num_q_heads;
  p->H[1] = r->num_kv_heads;
  p->rot = r->rotary_dim;
  p->norm = r->norm != 0;
  p->w_bf16 = r->weights_bf16 != 0;
  p->eps = r->eps;
  p->pos = r->positions;
  p->turns = r->turns;
  p->w[0] = r->q_weight;
  p->w[1] = r->k_weight;
  return RA_OK;
}

// Rows [T, heads, D] of elements of `size` bytes.
ra_status check_rows(const char* name, const void* ptr, int64_t stride, int64_t T, int32_t heads, int32_t D, int size,
                     ra::RopeRows* rows, Span* span) {
  const int64_t row = (int64_t)heads * D;
  if (T > 0 && !ptr) return fail(RA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(ptr, 16)) return fail(RA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (T > 1 && (stride < row || stride % (16 / size) || stride > (int64_t(1) << 31)))
    return fail(RA_ERR_INVALID_ARG, "%s: row stride %lld: a multiple of %d elements, at least %lld", name,
                (long long)stride, 16 / size, (long long)row);
  *rows = ra::RopeRows{const_cast<void*>(ptr), T > 1 ? stride : row};
  *span = Span{ptr, rows->stride * size, row * size, T, name};
  return RA_OK;
}

Span flat(const void* p, size_t bytes, const char* name) { return Span{p, (int64_t)bytes, (int64_t)bytes, 1, name}; }

// What a call only reads besides its rows.
struct Reads {
  Span s[4];
};
Reads reads_of(const ra_norm_rope* r) {
  const size_t w = (size_t)r->head_dim * (r->weights_bf16 ? 2 : 4);
  return Reads{{flat(r->positions, (size_t)r->num_tokens * 4, "positions"),
                flat(r->turns, (size_t)r->rotary_dim * 4, "turns"), flat(r->q_weight, w, "q_weight"),
                flat(r->k_weight, w, "k_weight")}};
}
ra_status over(const Span& a, const Span& b) { return fail(RA_ERR_INVALID_ARG, "%s lies over %s", a.name, b.name); }

}  // namespace

extern "C" {

ra_status ra_rope_turns(int32_t rotary_dim, double base, const double* inv_freq, uint64_t* turns) {
  if (rotary_dim < 0 || rotary_dim % 2 || rotary_dim > 65536)
    return fail(RA_ERR_INVALID_ARG, "rotary_dim %d: an even number", rotary_dim);
  if (rotary_dim > 0 && !turns) return fail(RA_ERR_INVALID_ARG, "NULL output");
  if (!inv_freq && !(base > 0.0 && std::isfinite(base))) return fail(RA_ERR_INVALID_ARG, "base must be finite and positive");
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    const double f = inv_freq ? inv_freq[i] : std::pow(base, -2.0 * i / rotary_dim);
    if (!(std::fabs(f) <= 6.2832)) return fail(RA_ERR_INVALID_ARG, "inv_freq[%d] is not a number within 2 pi", i);
    double t = f / 6.283185307179586476925286766559;
    t -= std::floor(t);  // positions are whole numbers: whole turns fall out
    t = std::ldexp(t, 64);
    turns[i] = t < 18446744073709551616.0 ? (uint64_t)t : 0u;
  }
  return RA_OK;
}

ra_status ra_qk_norm_rope_fwd(const ra_norm_rope* r, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  ra::RopeParams p{};
  ra_status rs = check_shape(r, &p);
  if (rs != RA_OK) return rs;
  const int32_t D = r->head_dim;
  Span in[2], out[2];
  if ((rs = check_rows("q", q, q_stride, p.T, p.H[0], D, 2, &p.x[0], &in[0])) != RA_OK ||
      (rs = check_rows("k", k, k_stride, p.T, p.H[1], D, 2, &p.x[1], &in[1])) != RA_OK ||
      (rs = check_rows("q_out", q_out, q_out_stride, p.T, p.H[0], D, 2, &p.y[0], &out[0])) != RA_OK ||
      (rs = check_rows("k_out", k_out, k_out_stride, p.T, p.H[1], D, 2, &p.y[1], &out[1])) != RA_OK)
    return rs;
  if (p.T == 0) return RA_OK;
  const Reads reads = reads_of(r);
  if (share_bytes(out[0], out[1])) return over(out[0], out[1]);
  for (int s = 0; s < 2; ++s) {
    for (int i = 0; i < 2; ++i) {  // in place: a row is read before it is written, by the same warp
      const bool in_place = s == i && out[s].p == in[i].p && out[s].stride == in[i].stride;
      if (!in_place && share_bytes(out[s], in[i])) return over(out[s], in[i]);
    }
    for (const Span& x : reads.s)
      if (share_bytes(out[s], x)) return over(out[s], x);
  }
  int sms = 0;
  cudaError_t e = ra::sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  e = ra::launch_rope_fwd(D, r->interleaved != 0, p, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "norm and rotation launch");
}

ra_status ra_qk_norm_rope_workspace_bytes(int32_t head_dim, size_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "NULL output");
  ra_status rs = check_head_dim(head_dim);
  if (rs != RA_OK) return rs;
  *bytes = (size_t)ra::kRopeMaxCtas * 2 * head_dim * sizeof(float);
  return RA_OK;
}

ra_status ra_qk_norm_rope_bwd(const ra_norm_rope* r, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* gq, int64_t gq_stride, const void* gk, int64_t gk_stride, int32_t g_is_fp32,
                              void* dq, int64_t dq_stride, void* dk, int64_t dk_stride, float* dq_weight,
                              float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  ra::RopeParams p{};
  ra_status rs = check_shape(r, &p);
  if (rs != RA_OK) return rs;
  const int32_t D = r->head_dim;
  const int gs = g_is_fp32 ? 4 : 2;
  Span in[4], out[4];
  if ((rs = check_rows("q", q, q_stride, p.T, p.H[0], D, 2, &p.x[0], &in[0])) != RA_OK ||
      (rs = check_rows("k", k, k_stride, p.T, p.H[1], D, 2, &p.x[1], &in[1])) != RA_OK ||
      (rs = check_rows("gq", gq, gq_stride, p.T, p.H[0], D, gs, &p.g[0], &in[2])) != RA_OK ||
      (rs = check_rows("gk", gk, gk_stride, p.T, p.H[1], D, gs, &p.g[1], &in[3])) != RA_OK ||
      (rs = check_rows("dq", dq, dq_stride, p.T, p.H[0], D, 2, &p.y[0], &out[0])) != RA_OK ||
      (rs = check_rows("dk", dk, dk_stride, p.T, p.H[1], D, 2, &p.y[1], &out[1])) != RA_OK)
    return rs;
  if ((dq_weight && !r->q_weight) || (dk_weight && !r->k_weight))
    return fail(RA_ERR_INVALID_ARG, "a weight's gradient needs the weight");
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return fail(RA_ERR_INVALID_ARG, "dq_weight, dk_weight must be 4-byte aligned");
  out[2] = flat(dq_weight, (size_t)D * 4, "dq_weight");
  out[3] = flat(dk_weight, (size_t)D * 4, "dk_weight");
  const bool sums = dq_weight || dk_weight;
  if (sums) {
    size_t need = 0;
    ra_qk_norm_rope_workspace_bytes(D, &need);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need)
      return fail(RA_ERR_WORKSPACE, "workspace of %zu bytes: need %zu, 256-byte aligned", workspace ? workspace_bytes : 0, need);
    p.partials = reinterpret_cast<float*>(workspace);
  }
  const Reads reads = reads_of(r);
  const Span ws = flat(sums ? workspace : nullptr, workspace_bytes, "workspace");
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (share_bytes(out[i], out[j])) return over(out[i], out[j]);
    for (const Span& x : in)
      if (share_bytes(out[i], x)) return over(out[i], x);
    for (const Span& x : reads.s)
      if (share_bytes(out[i], x)) return over(out[i], x);
    if (share_bytes(out[i], ws)) return over(out[i], ws);
  }
  for (const Span& x : in)
    if (share_bytes(ws, x)) return over(ws, x);
  for (const Span& x : reads.s)
    if (share_bytes(ws, x)) return over(ws, x);
  if (p.T == 0 && !sums) return RA_OK;
  int sms = 0;
  cudaError_t e = ra::sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  float* dw[2] = {dq_weight, dk_weight};
  e = ra::launch_rope_bwd(D, r->interleaved != 0, g_is_fp32 != 0, p, sms, dw, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "norm and rotation backward launch");
}

}  // extern "C"
