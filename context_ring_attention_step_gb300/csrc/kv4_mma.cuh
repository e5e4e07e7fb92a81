// kv4_mma.cuh -- what the kernels for few query rows share: the m16n8k16 product,
// a warp's asynchronous copies, and a tile's keys as operand registers.
#pragma once

#include "kv4.h"
#include "kv4_walk.cuh"

namespace ra {

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

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


__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// The keys of one warp's tile in registers.
template <int D>
struct KeyRegs {
  uint4 k[D / 64];
  uint32_t ks[D == 256 ? 2 : 1];
};

// Word `i` of the run of K codes that a lane holds for token r + 8 h.
template <int D>
__device__ __forceinline__ uint32_t k_word(const KeyRegs<D>& t, int h, int i) {
  if (D == 64) return word(t.k[0], 2 * h + i);
  if (D == 128) return word(t.k[h], i);
  return word(t.k[(2 * h + (i >> 2)) % (D / 64)], i & 3);
}
// Its scale of group g, in both halves.
template <int D>
__device__ __forceinline__ uint32_t k_scale2(const KeyRegs<D>& t, int h, int g) {
  if (D == 64) return scale_both(t.ks[0], h);
  if (D == 128) return scale_both(t.ks[0], 2 * h + g);
  return scale_both(t.ks[h % (D == 256 ? 2 : 1)], g);
}

}  // namespace ra
