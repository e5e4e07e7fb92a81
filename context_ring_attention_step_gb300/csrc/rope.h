// rope.h -- norms of queries and keys with the position rotation: parameter
// blocks and launch wrappers shared by the kernels (rope.cu) and the C entry
// points (rope_api.cu).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/ring_attn.h"

namespace ra {

// Rows [T, H, D], the heads of a row dense, `stride` elements between rows.
struct RopeRows {
  void* p;
  int64_t stride;
};

struct RopeParams {
  int64_t T;
  int32_t H[2];      // query heads, key heads
  int32_t rot;       // rotated elements of a row (the first ones)
  int32_t norm, w_bf16;
  float eps;
  const int32_t* pos;
  const uint64_t* turns;  // [rot / 2] turns per position, in 2^-64
  const void* w[2];       // [D], null: ones
  RopeRows x[2];          // bf16
  RopeRows y[2];          // forward: results; backward: gradients of x
  RopeRows g[2];          // backward: gradients of the results, bf16 or fp32
  int32_t parts[2];       // a token's heads are shared out over so many warps
  float* partials;        // backward: [CTAs][2][D] sums of the weights' gradients, or null
};

constexpr int kRopeMaxCtas = 320;  // of a backward pass: what its workspace holds
cudaError_t launch_rope_fwd(int D, bool interleaved, RopeParams p, int sms, cudaStream_t stream);
cudaError_t launch_rope_bwd(int D, bool interleaved, bool g_fp32, RopeParams p, int sms, float* dw[2],
                            cudaStream_t stream);

}  // namespace ra
