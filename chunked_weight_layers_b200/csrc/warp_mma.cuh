// Warp-level matrix and asynchronous-copy wrappers.
//
// Fragments of mma.m16n8k16 (lane = 4·g + q): A holds rows g, g + 8 and columns 2q, 2q + 1,
// 2q + 8, 2q + 9; B holds rows (k) 2q, 2q + 1, 2q + 8, 2q + 9 of column g; D holds rows g (0, 1)
// and g + 8 (2, 3), columns 2q, 2q + 1.
#pragma once

#include "common.cuh"

namespace ttt {
namespace wm {

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 bf16 matrices, fragments as above, to the rows that the lanes 0 .. 7, 8 .. 15, ... name.
__device__ __forceinline__ void stsm(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float2 unpack(uint32_t x) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
}

}  // namespace wm
}  // namespace ttt
