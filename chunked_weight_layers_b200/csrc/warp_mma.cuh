// Warp-level tensor-core and asynchronous-copy wrappers for kernels on 64-wide bf16 tiles with
// 128-byte rows and the 128-byte swizzle (16-byte chunk index XOR row % 8).
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

__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// A fragment of rows row0 .. row0 + 15, columns col0 .. col0 + 15 of a tile stored [row][col].
__device__ __forceinline__ void frag_a(uint32_t tile, int row0, int col0, int lane, uint32_t (&a)[4]) {
  ldsm(tile + swz128_bf16(row0 + (lane & 15), col0 + 8 * (lane >> 4)), a);
}

// A fragment whose rows are the tile's columns: rows (tile columns) col0 .. col0 + 15, k (tile
// rows) row0 .. row0 + 15.
__device__ __forceinline__ void frag_a_t(uint32_t tile, int row0, int col0, int lane, uint32_t (&a)[4]) {
  const int mi = lane >> 3, ri = lane & 7;
  ldsm_t(tile + swz128_bf16(row0 + 8 * (mi >> 1) + ri, col0 + 8 * (mi & 1)), a);
}

// B fragments of columns (tile rows) row0 .. row0 + 15, k (tile columns) col0 .. col0 + 15: the
// tile is stored [n][k]. b[0], b[1] for n-tile row0 .. +7; b[2], b[3] for row0 + 8 .. +15.
__device__ __forceinline__ void frag_b(uint32_t tile, int row0, int col0, int lane, uint32_t (&b)[4]) {
  const int mi = lane >> 3, ri = lane & 7;
  ldsm(tile + swz128_bf16(row0 + 8 * (mi >> 1) + ri, col0 + 8 * (mi & 1)), b);
}

// B fragments of k (tile rows) row0 .. row0 + 15, columns (tile columns) col0 .. col0 + 15: the
// tile is stored [k][n]. b[0], b[1] for n-tile col0 .. +7; b[2], b[3] for col0 + 8 .. +15.
__device__ __forceinline__ void frag_b_t(uint32_t tile, int row0, int col0, int lane, uint32_t (&b)[4]) {
  const int mi = lane >> 3, ri = lane & 7;
  ldsm_t(tile + swz128_bf16(row0 + 8 * (mi & 1) + ri, col0 + 8 * (mi >> 1)), b);
}

// Asynchronous copy of 16 bytes to shared memory, or 16 zero bytes when !valid (src is not read).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float2 unpack(uint32_t x) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
}

// x ⊙ (w0, w1) as the sum of two bf16 pairs: hi the product rounded, lo what the rounding left
// (the sum is the product to 2^-17 of its size).
__device__ __forceinline__ void scale_split(uint32_t x, float w0, float w1, uint32_t& hi, uint32_t& lo) {
  const float2 f = unpack(x);
  const float p0 = f.x * w0, p1 = f.y * w1;
  hi = pack_bf16(p0, p1);
  const float2 h = unpack(hi);
  lo = pack_bf16(p0 - h.x, p1 - h.y);
}

}  // namespace wm
}  // namespace ttt
