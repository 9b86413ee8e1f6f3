// Gated feed-forward block, the producer of the In-Place scan's keys: Z = act(G) ⊙ U with
// G = X·Wgᵀ and U = X·Wuᵀ, and its gradients.
//
// Mathematics. X [T, d], Wg and Wu [f, d], Z [T, f]; act is SiLU, x·σ(x), or GELU, x·Φ(x).
// Backward from dZ and the kept G and U: dG = dZ ⊙ U ⊙ act'(G), dU = dZ ⊙ act(G),
// dX = dG·Wg + dU·Wu, dWg = dGᵀ·X, dWu = dUᵀ·X. All products take bf16 operands and sum in fp32;
// dG and dU are rounded to bf16 once, since they are operands of the products after them.
//
// What bounds it: the tensor cores from some hundreds of tokens on, the weights' bytes below that.
//
// k_ffn_pair is one persistent GEMM on SM pairs (tcgen05, cta_group::2, 256 x 256 accumulators, two
// of them in TMEM so that one tile's epilogue runs under the next tile's products), in three forms:
//   FWD  rows: tokens; columns: 128 of Wg's rows (loaded by the first CTA) and the same 128 of
//        Wu's (by the second), so every thread of the epilogue finds g and u of one output in
//        its own TMEM lane and no pre-activation goes through memory. A, B K-major.
//        Tiles take 128 columns of f, or fewer where that fills the SM pairs' last round better
//        (columns_of).
//   DX   rows: tokens; columns: 256 of d; the sum runs over dG·Wg and then dU·Wu in the same
//        accumulator. A K-major, B MN-major.
//   DW   rows: 256 of f, gate tiles and then up tiles; columns: 256 of d; the sum runs over the
//        tokens. A, B MN-major: X, dG and dU are read as they lie, nothing is transposed.
// The pairs take whole tiles in rounds; DX and DW cut the sums of the tiles left for a last, unfilled
// round into as many parts as there are pairs, whose fp32 results a small launch adds in order.
// Sizes need not be multiples of the tiles: TMA reads zeros past the ends, stores are clipped.
//
// k_ffn_few takes up to 16 tokens, where the weights' bytes are all that counts, and k_ffn_rows some tens of
// tokens against wide weights: see there.
//
// Measured (B200), d 2560, f 9728: forward over 8192 tokens 550 us at full clocks (1480 TFLOP/s, 88 % of a
// large library product's rate), 620 to 640 us once the card runs at its power limit; over one token 17 us
// (5.8 TB/s). Backward over 4096 tokens 690 to 750 us at the power limit; at full clocks 57 us for the
// activation's part, 256 for dX (1590 TFLOP/s), 264 for the weights' gradients and 10 for the joins.
// 777 tokens, d 1000, f 2744, keeping G and U: 19 us (450 TFLOP/s: two rounds of tiles of 16 k-blocks, whose
// first loads and epilogues take half of it).
#include <algorithm>

#include "internal.h"
#include "tc_common.cuh"
#include "tc_pair.cuh"
#include "warp_mma.cuh"

namespace ttt {

namespace {

constexpr int FM = 128, FK = 64;            // rows per CTA, k-block
constexpr int kTileM = 256, kTileN = 256;   // of a pair
constexpr int kHalf = FM * FK * 2;          // 16 KB: a CTA's part of A, and of B, in one stage
constexpr int kFStages = 6;
constexpr int kFEpi = 8;
constexpr int kFThreads = (2 + kFEpi) * 32;
constexpr int kFTmem = 512;

enum : int { FWD = 0, DX = 1, DW = 2 };

struct __align__(1024) FfnSmem {
  uint8_t ring[kFStages][2 * kHalf];
  uint8_t out[kFEpi][32 * 64];  // a warp's 32 rows x 32 bf16 columns on their way out
  uint64_t full[kFStages], empty[kFStages];
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  int abort;
};

struct FfnArgs {
  int M, N;           // rows and columns of the result (FWD: T, f; DX: T, d; DW: f, d)
  int kblocks;        // k-blocks of one product (DX: of each of the two)
  int tiles_m, tiles_n;
  int cols;           // FWD: columns of f in a tile, a multiple of 8 up to 128
  int rows;           // FWD, DX: tokens of a tile that each CTA takes, a multiple of 8 up to 128 (DW: 128)
  int whole;          // tiles whose sum one pair makes alone: the first of the order
  int splits, per_split;  // parts of the sums of the tiles after them, and k-blocks of a part
  int act;
  __nv_bfloat16 *z, *g, *u;  // FWD: outputs (g and u or null); DX: z = dX; DW: g = dWg, u = dWu
  float* part;               // [tiles after the whole ones][splits][256][256]
  DevStatus status;
  int stall;                 // a k-block of every pair that is never loaded (tests), or -1
};

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// Φ(x) = 1 − erfc(x/√2)/2, erfc by the rational approximation 7.1.26 of Abramowitz and Stegun
// (|error| <= 1.5e-7), from the side where it is small. erff took the forward epilogue over.
__device__ __forceinline__ float normal_cdf(float x) {
  const float z = fabsf(x) * 0.70710678118654752f;
  const float t = __fdividef(1.f, fmaf(0.3275911f, z, 1.f));
  const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
  const float tail = 0.5f * p * __expf(-z * z);
  return x < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float act_of(float x, int act) {
  return act == TTT_ACT_SILU ? x * sigmoid(x) : x * normal_cdf(x);
}

// A warp's 32 rows (one a lane) of 32 bf16 values out to rows row0 .., columns col0 .. of `out` (row
// length ld), clipped to `rows` and `cols` (a multiple of 8): through shared memory, so that four
// lanes write 64 bytes of one row and not each lane its own row.
__device__ __forceinline__ void store_tile(uint8_t* stage, int lane, const float (&v)[32], __nv_bfloat16* out, size_t ld, int row0,
                                           int rows, int col0, int cols) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                   pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]));
  __syncwarp();
  const int c = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    if (row0 + r < rows && col0 + 8 * c < cols)
      *reinterpret_cast<uint4*>(out + (size_t)(row0 + r) * ld + col0 + 8 * c) =
          *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
  __syncwarp();
}

// What unit u of the order is: tile (m, n) and k-blocks k0 .. k1. The order keeps the running tiles
// on few rows and columns at once (L2): blocks of eight row tiles, down the rows first. After the
// whole tiles come the parts of the others.
struct Unit {
  int m, n, k0, k1, part;  // part: index of the part's result, -1 for a whole tile
};

__device__ __forceinline__ Unit unit_at(const FfnArgs& a, int u, int total_k) {
  Unit r;
  int t = u;
  r.k0 = 0;
  r.k1 = total_k;
  r.part = -1;
  if (u >= a.whole) {
    r.part = u - a.whole;
    t = a.whole + r.part / a.splits;
    r.k0 = (r.part % a.splits) * a.per_split;
    r.k1 = min(total_k, r.k0 + a.per_split);
  }
  const int block = t / (8 * a.tiles_n), m0 = 8 * block, rows = min(8, a.tiles_m - m0);
  const int at = t - block * 8 * a.tiles_n;
  r.m = m0 + at % rows;
  r.n = at / rows;
  return r;
}

__host__ __device__ inline int units_of(const FfnArgs& a) { return a.whole + (a.tiles_m * a.tiles_n - a.whole) * a.splits; }

// FWD: tmA0 = X, tmB0 = Wg, tmB1 = Wu. DX: tmA0 = dG, tmA1 = dU, tmB0 = Wg, tmB1 = Wu.
// DW: tmA0 = dG, tmA1 = dU, tmB0 = X.
template <int MODE>
__global__ void __launch_bounds__(kFThreads, 1)
    k_ffn_pair(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
               const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1, const FfnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  FfnSmem& sm = *reinterpret_cast<FfnSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)pair::rank();
  const int npairs = gridDim.x / 2, me = blockIdx.x / 2;
  const int units = units_of(a);
  const int total_k = MODE == DX ? 2 * a.kblocks : a.kblocks;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.tfull[i], 1);
      mbar_init(&sm.tempty[i], 2 * kFEpi);  // the epilogue warps of both CTAs
    }
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) pair::alloc(&sm.tmem, kFTmem);
  tc::fence_before();
  __syncthreads();
  pair::sync();  // both CTAs' barriers exist before either arrives remotely
  tc::fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int* abort = &sm.abort;
  const int bcols = MODE == FWD ? a.cols : FM;  // columns of B that each CTA loads

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmA0);
      tma_prefetch_desc(&tmB0);
      uint32_t it = 0;
      bool ok = true;
      for (int t = me; t < units && ok; t += npairs) {
        const Unit un = unit_at(a, t, total_k);
        const int m = un.m, n = un.n;
        for (int kb = un.k0; kb < un.k1; ++kb, ++it) {
          const int s = it % kFStages;
          if (*abort || (it >= (uint32_t)kFStages && !mbar_wait(&sm.empty[s], ((it / kFStages) - 1) & 1, a.status, abort))) {
            ok = false;
            break;
          }
          if ((int)it == a.stall) continue;
          uint8_t *sa = sm.ring[s], *sb = sa + kHalf;
          // Both CTAs' loads complete on the first CTA's barrier, which expects the bytes of both.
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * (a.rows + bcols) * FK * 2);
          const uint32_t bar = pair::in_first(&sm.full[s]);
          if constexpr (MODE == FWD) {
            pair::load_2d(sa, &tmA0, bar, kb * FK, (2 * m + rank) * a.rows);
            pair::load_2d(sb, rank ? &tmB1 : &tmB0, bar, kb * FK, n * a.cols);
          } else if constexpr (MODE == DX) {
            const bool up = kb >= a.kblocks;
            const int k = (up ? kb - a.kblocks : kb) * FK;
            pair::load_2d(sa, up ? &tmA1 : &tmA0, bar, k, (2 * m + rank) * a.rows);
            for (int j = 0; j < 2; ++j)
              pair::load_2d(sb + j * (kHalf / 2), up ? &tmB1 : &tmB0, bar, n * kTileN + rank * FM + 64 * j, k);
          } else {
            const int half_m = a.tiles_m / 2;
            const bool up = m >= half_m;
            const int row = (up ? m - half_m : m) * kTileM + rank * FM;
            for (int j = 0; j < 2; ++j) {
              pair::load_2d(sa + j * (kHalf / 2), up ? &tmA1 : &tmA0, bar, row + 64 * j, kb * FK);
              pair::load_2d(sb + j * (kHalf / 2), &tmB0, bar, n * kTileN + rank * FM + 64 * j, kb * FK);
            }
          }
        }
      }
      // Nothing may still land in, or arrive at, this CTA's shared memory when it exits.
      const uint32_t first = it > (uint32_t)kFStages ? it - kFStages : 0;
      if (!*abort) {
        for (uint32_t k = first; k < it; ++k) mbar_wait(&sm.empty[k % kFStages], (k / kFStages) & 1, a.status, nullptr);
      } else {
        // A stage may never complete (its partner's half missing): wait 50 us, far beyond the
        // latency of a load.
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 50000) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = tc::idesc_bf16(kTileM, 2 * bcols, MODE == DW, MODE != FWD);
      // K-major operands step along their rows, MN-major ones (64 columns a box, 8192 bytes) down them.
      const uint32_t da = tc::desc_of(sm.ring[0], MODE == DW ? 8192 : 16), db = tc::desc_of(sm.ring[0] + kHalf, MODE == FWD ? 16 : 8192);
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int t = me; t < units && ok; t += npairs) {
        const Unit un = unit_at(a, t, total_k);
        const int acc = tcount & 1;
        if (tcount >= 2 && !mbar_wait<true>(&sm.tempty[acc], ((tcount >> 1) - 1) & 1, a.status, abort)) {
          ok = false;
          break;
        }
        tc::fence_after();
        for (int kb = un.k0; kb < un.k1; ++kb, ++it) {
          const int s = it % kFStages;
          if (!mbar_wait<true>(&sm.full[s], (it / kFStages) & 1, a.status, abort)) {
            ok = false;
            break;
          }
          tc::fence_after();
          const uint32_t ad = da + s * (2 * kHalf >> 4), bd = db + s * (2 * kHalf >> 4);
#pragma unroll
          for (int kk = 0; kk < FK / 16; ++kk)
            pair::mma(tmem + acc * kTileN, tc::desc_at(ad, kk * (MODE == DW ? 2048 : 32)), tc::desc_at(bd, kk * (MODE == FWD ? 32 : 2048)),
                      idesc, (kb != un.k0 || kk != 0));
          pair::commit(&sm.empty[s]);
        }
        if (!ok) break;
        pair::commit(&sm.tfull[acc]);
        ++tcount;
      }
      // The last commit covers every MMA issued before it: wait for it before TMEM is freed.
      if (ok && tcount > 0)
        mbar_wait(&sm.tfull[(tcount - 1) & 1], ((tcount - 1) >> 1) & 1, a.status, nullptr);
      else if (!ok && it > 0)
        mbar_wait(&sm.empty[(it - 1) % kFStages], ((it - 1) / kFStages) & 1, a.status, nullptr);
    }
  } else {
    const int lq = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter; every other 32 columns
    uint8_t* stage = sm.out[warp - 2];
    uint32_t tcount = 0;
    for (int t = me; t < units; t += npairs) {
      const Unit un = unit_at(a, t, total_k);
      const int acc = tcount & 1;
      const bool ok = mbar_wait(&sm.tfull[acc], (tcount >> 1) & 1, a.status, nullptr);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::fence_after();
      const uint32_t tb = tmem + ((uint32_t)(lq * 32) << 16) + (uint32_t)(acc * kTileN);
      int row0 = (2 * un.m + rank) * a.rows + lq * 32, row_end = min(a.M, (2 * un.m + rank + 1) * a.rows);
      if constexpr (MODE == FWD) {
        const int col_end = min(a.N, (un.n + 1) * a.cols);
#pragma unroll 1
        for (int c = half * 32; c < a.cols; c += 64) {
          const int col = un.n * a.cols + c;
          uint32_t rg[32], ru[32];
          tc::ld32(tb + c, rg);
          tc::ld32(tb + a.cols + c, ru);
          tc::wait_ld();
          float g[32], u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            g[i] = __uint_as_float(rg[i]);
            u[i] = __uint_as_float(ru[i]);
          }
          if (a.g != nullptr) {
            store_tile(stage, lane, g, a.g, a.N, row0, row_end, col, col_end);
            store_tile(stage, lane, u, a.u, a.N, row0, row_end, col, col_end);
          }
          if (a.act == TTT_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) g[i] = g[i] * sigmoid(g[i]) * u[i];
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) g[i] = g[i] * normal_cdf(g[i]) * u[i];
          }
          store_tile(stage, lane, g, a.z, a.N, row0, row_end, col, col_end);
        }
      } else {
        __nv_bfloat16* out = a.z;
        if constexpr (MODE == DW) {
          const int half_m = a.tiles_m / 2;
          out = un.m >= half_m ? a.u : a.g;
          row0 -= un.m >= half_m ? half_m * kTileM : 0;
          row_end = a.M;
        }
#pragma unroll 1
        for (int c = half * 32; c < kTileN; c += 64) {
          uint32_t r[32];
          tc::ld32(tb + c, r);
          tc::wait_ld();
          if (un.part >= 0) {
            uint4* p = reinterpret_cast<uint4*>(a.part + ((size_t)un.part * kTileM + rank * FM + lq * 32 + lane) * kTileN + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          } else {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            store_tile(stage, lane, v, out, a.N, row0, row_end, un.n * kTileN + c, a.N);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) pair::arrive(pair::in_first(&sm.tempty[acc]));
      ++tcount;
    }
  }
  tc::fence_before();
  __syncthreads();
  // Neither CTA exits, or frees TMEM, while the other may still arrive on its barriers or the MMAs
  // may still write its TMEM.
  pair::sync();
  tc::fence_after();
  if (warp == 1) pair::dealloc(tmem, kFTmem);
}

// The tiles made in parts: the sums of their parts, in order, as bf16. grid (32, tiles after the whole
// ones), eight values a thread, eight rows a CTA.
template <int MODE>
__global__ void __launch_bounds__(256) k_ffn_join(const FfnArgs a) {
  const Unit un = unit_at(a, a.whole + blockIdx.y * a.splits, 0);
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), c = (threadIdx.x & 31) * 8;
  __nv_bfloat16* out = a.z;
  int row = (2 * un.m + r / FM) * a.rows + r % FM;
  if (r % FM >= a.rows) return;
  if (MODE == DW) {
    const int half_m = a.tiles_m / 2;
    out = un.m >= half_m ? a.u : a.g;
    row -= un.m >= half_m ? half_m * kTileM : 0;
  }
  const int col = un.n * kTileN + c;
  if (row >= a.M || col >= a.N) return;
  const float* p = a.part + ((size_t)blockIdx.y * a.splits * kTileM + r) * kTileN + c;
  float v[8] = {};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s, p += kTileM * kTileN) {
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
  *reinterpret_cast<uint4*>(out + (size_t)row * a.N + col) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// dG = dZ ⊙ U ⊙ act'(G), dU = dZ ⊙ act(G) over n elements (a multiple of 8), eight a thread: HBM
// bound, ten bytes an element.
template <int ACT>
__global__ void __launch_bounds__(256) k_ffn_act_bwd(const __nv_bfloat16* __restrict__ dz, const __nv_bfloat16* __restrict__ g,
                                                     const __nv_bfloat16* __restrict__ u, __nv_bfloat16* __restrict__ dg,
                                                     __nv_bfloat16* __restrict__ du, size_t n) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const uint4 Z = *reinterpret_cast<const uint4*>(dz + i), G = *reinterpret_cast<const uint4*>(g + i),
              U = *reinterpret_cast<const uint4*>(u + i);
  const uint32_t z4[4] = {Z.x, Z.y, Z.z, Z.w}, g4[4] = {G.x, G.y, G.z, G.w}, u4[4] = {U.x, U.y, U.z, U.w};
  uint32_t a4[4], b4[4];
  auto one = [](float z, float x, float y, float& da, float& db) {
    float act, slope;
    if constexpr (ACT == TTT_ACT_SILU) {
      const float s = sigmoid(x);
      act = x * s;
      slope = s * fmaf(x, 1.f - s, 1.f);
    } else {
      const float p = normal_cdf(x);
      act = x * p;
      slope = fmaf(x * 0.3989422804014327f, __expf(-0.5f * x * x), p);
    }
    da = z * y * slope;
    db = z * act;
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 zf = wm::unpack(z4[j]), gf = wm::unpack(g4[j]), uf = wm::unpack(u4[j]);
    float a0, b0, a1, b1;
    one(zf.x, gf.x, uf.x, a0, b0);
    one(zf.y, gf.y, uf.y, a1, b1);
    a4[j] = pack_bf16(a0, a1);
    b4[j] = pack_bf16(b0, b1);
  }
  *reinterpret_cast<uint4*>(dg + i) = make_uint4(a4[0], a4[1], a4[2], a4[3]);
  *reinterpret_cast<uint4*>(du + i) = make_uint4(b4[0], b4[1], b4[2], b4[3]);
}

// ---- up to 16 tokens -------------------------------------------------------------------------

// The weights' bytes bound it, so they go from HBM straight into the registers that the tensor
// cores read (mma.sync: with at most 16 columns its rate is far from counting), with no stage in
// shared memory and no barrier on the way. A CTA of four warps takes eight rows of Wg and the same
// eight of Wu as the 16 rows of one product, so a thread ends with g and u of the same outputs; warp
// w takes every fourth 32-wide slice of the sum, the next slices' loads in flight while it works on
// these, and the warps' results are added in order at the end. A lane's 16-byte load holds eight
// consecutive k of one row; the products' k slots are filled in that order for the weights and for X
// alike, which a sum does not mind. NT: token blocks of eight; MT: such blocks of rows a CTA, two for the two
// blocks of tokens, since every CTA reads all of X (9 x 5120 x 5120: 23 us against 31 with one). The CTAs
// an SM must hold leave room for the loads to go ahead of the products: left to itself the compiler took few
// registers and 22 us for one token of 5120 x 5120, so 17.4; six CTAs: 18.6; for two blocks of rows three:
// 23, five: 27.
constexpr int kFewWarps = 4;

__device__ __forceinline__ uint4 load_once(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <int NT, int MT>
__global__ void __launch_bounds__(32 * kFewWarps, MT == 1 ? 5 : 3) k_ffn_few(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ Wg,
                                                            const __nv_bfloat16* __restrict__ Wu, int T, int d, int f, int act,
                                                            __nv_bfloat16* __restrict__ z, __nv_bfloat16* __restrict__ gout,
                                                            __nv_bfloat16* __restrict__ uout) {
  __shared__ float part[kFewWarps][2][8 * NT][8 * MT + 1];  // [warp][gate, up][token][row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int f0 = blockIdx.x * 8 * MT, blocks = min(MT, (f - f0) / 8);  // f is a multiple of 8
  const int steps = (d + 31) / 32;
  constexpr int UN = 2;  // slices in flight: more take registers from the warps that hide the latency (4: 22 us, 2: 17)
  const __nv_bfloat16* pg = Wg + (size_t)(f0 + g) * d + 8 * q;
  const __nv_bfloat16* pu = Wu + (size_t)(f0 + g) * d + 8 * q;
  const __nv_bfloat16* px = X + (size_t)g * d + 8 * q;
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 wg[2][UN][MT], wu[2][UN][MT];
  auto fetch = [&](int st, uint4 (&G)[UN][MT], uint4 (&U)[UN][MT]) {
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = (st + kFewWarps * i) * 32;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bool in = k + 8 * q < d && m < blocks;
        G[i][m] = in ? load_once(pg + (size_t)(8 * m) * d + k) : none;
        U[i][m] = in ? load_once(pu + (size_t)(8 * m) * d + k) : none;
      }
    }
  };
  float acc[MT][NT][4] = {};
  auto work = [&](int st, const uint4 (&G)[UN][MT], const uint4 (&U)[UN][MT]) {
    uint4 x[UN][NT];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = (st + kFewWarps * i) * 32;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        x[i][nt] = k + 8 * q < d && 8 * nt + g < T ? *reinterpret_cast<const uint4*>(px + (size_t)(8 * nt) * d + k) : none;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint32_t a0[4] = {G[i][m].x, U[i][m].x, G[i][m].y, U[i][m].y}, a1[4] = {G[i][m].z, U[i][m].z, G[i][m].w, U[i][m].w};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          wm::mma(acc[m][nt], a0, x[i][nt].x, x[i][nt].y);
          wm::mma(acc[m][nt], a1, x[i][nt].z, x[i][nt].w);
        }
      }
  };
  constexpr int kStep = kFewWarps * UN;
  fetch(warp, wg[0], wu[0]);
  for (int st = warp; st < steps; st += 2 * kStep) {
    fetch(st + kStep, wg[1], wu[1]);  // past the end: zeros, no loads
    work(st, wg[0], wu[0]);
    fetch(st + 2 * kStep, wg[0], wu[0]);
    work(st + kStep, wg[1], wu[1]);
  }
  // A lane holds row g of the gate (0, 1) and of up (2, 3) for tokens 2q, 2q + 1 of each block.
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[warp][e >> 1][8 * nt + 2 * q + (e & 1)][8 * m + g] = acc[m][nt][e];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * MT * 64; i += 32 * kFewWarps) {
    const int r = i % (8 * MT), t = i / (8 * MT);
    if (t >= T || r >= 8 * blocks) continue;
    float sg = 0.f, su = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      sg += part[w][0][t][r];
      su += part[w][1][t][r];
    }
    const size_t at = (size_t)t * f + f0 + r;
    if (gout != nullptr) {
      gout[at] = __float2bfloat16_rn(sg);
      uout[at] = __float2bfloat16_rn(su);
    }
    z[at] = __float2bfloat16_rn(act_of(sg, act) * su);
  }
}

// ---- some tens of tokens ---------------------------------------------------------------------

// Few tokens leave the pairs' 256 rows nearly empty, and their products cost as much as full ones; so here
// the weights are the rows. A CTA takes `rows` rows of Wg and the same of Wu against all T tokens (up
// to 160 columns), two accumulators of 128 lanes (those past `rows` hold what the products make of the next
// bytes of the ring, and are not looked at), so that an epilogue thread finds g and u of its row in its own
// lane. One tile a CTA, as many rows as spread f evenly over the SMs: bound by the weights' bytes, which
// pass once, and for more tokens by X's, which every CTA reads from L2. 17 x 4096 x 14336: 40 us (5.9 TB/s),
// 17 x 8192 x 28672: 148 us (6.3), 17 x 2560 x 9728: 20.5 us (4.9; the launch's ends are a fifth of it).
struct RowsArgs {
  int T, f, kblocks, rows, cols, stages;  // cols: T rounded up to 16
  int act;
  __nv_bfloat16 *z, *g, *u;  // g and u or null
  DevStatus status;
  int stall;  // a k-block that is never loaded (tests), or -1
};

constexpr int kRowsMaxStages = 8, kRowsEpi = 16, kRowsThreads = (3 + kRowsEpi) * 32;
constexpr int kRowsSlack = kHalf;       // what the last stage's products read past its rows
constexpr int kRowsRing = 200 * 1024;

struct RowsSync {
  uint64_t full[kRowsMaxStages], empty[kRowsMaxStages], done;
  uint32_t tmem;
  int abort;
};

// Bytes of a CTA's rows of one weight in a stage, and of a stage: whole groups of eight rows.
__host__ __device__ inline int rows_part(int rows) { return (rows + 7) / 8 * 8 * FK * 2; }
__host__ __device__ inline int rows_stage(int rows, int cols) { return 2 * rows_part(rows) + cols * FK * 2; }

// Eight consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Columns of two tokens, one row a lane, to out[token][row]: each lane a pair of rows of one token.
__device__ __forceinline__ void store_tokens(__nv_bfloat16* out, float a, float b, int t, int lane, int T, size_t ld, bool in) {
  const bool odd = lane & 1;
  const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
  if (in && t + odd < T) *reinterpret_cast<uint32_t*>(out + (size_t)(t + odd) * ld - odd) = odd ? pack_bf16(got, b) : pack_bf16(a, got);
}

__global__ void __launch_bounds__(kRowsThreads, 1)
    k_ffn_rows(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmU,
               const RowsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ RowsSync sm;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, f0 = blockIdx.x * a.rows;
  const int part = rows_part(a.rows), stage = rows_stage(a.rows, a.cols);
  const uint32_t up = a.cols <= 128 ? 128 : 256;  // TMEM column of the second accumulator
  volatile int* abort = &sm.abort;
  auto load = [&](int kb, int s) {
    if (kb == a.stall) return;
    uint8_t* p = ring + s * stage;
    mbar_arrive_expect_tx(&sm.full[s], (2 * a.rows + a.cols) * FK * 2);
    tma_load_2d(p, &tmG, &sm.full[s], kb * FK, f0);
    tma_load_2d(p + part, &tmU, &sm.full[s], kb * FK, f0);
    tma_load_2d(p + 2 * part, &tmX, &sm.full[s], kb * FK, 0);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 2);
    }
    mbar_init(&sm.done, 2);
    sm.abort = 0;
    fence_barrier_init();
    for (int kb = 0; kb < min(a.stages, a.kblocks); ++kb) load(kb, kb);
  }
  __syncwarp();
  if (warp == 1) tc::alloc(&sm.tmem, 2 * up);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sm.tmem;
  if (warp == 0) {
    if (lane == 0) {
      // The stage and the parity of its round are counted, not divided out of kb: with the divisions a
      // k-block took 930 cycles whatever its size.
      int kb = min(a.stages, a.kblocks);
      uint32_t s = 0, round = 0;
      for (; kb < a.kblocks; ++kb) {
        if (*abort || !mbar_wait(&sm.empty[s], round & 1, a.status, abort)) break;
        load(kb, s);
        if (++s == (uint32_t)a.stages) s = 0, ++round;
      }
      // Nothing may still land in this CTA's shared memory when it exits.
      for (int k = max(0, kb - a.stages); k < kb; ++k) mbar_wait(&sm.full[k % a.stages], (k / a.stages) & 1, a.status, nullptr);
    }
  } else if (warp <= 2) {
    // One thread issues the gate's products, another up's: beside the products (47 cycles each) a k-block
    // costs the issuing thread some 400 cycles.
    if (lane == 0) {
      const bool second = warp == 2;
      const uint32_t idesc = tc::idesc_bf16(128, a.cols, 0, 0), acc = tmem + (second ? up : 0), skip = second ? part >> 4 : 0;
      const uint32_t first = tc::desc_of(ring);
      bool ok = true;
      uint32_t s = 0, round = 0;
      for (int kb = 0; kb < a.kblocks; ++kb) {
        if (!(ok = mbar_wait(&sm.full[s], round & 1, a.status, abort))) break;
        tc::fence_after();
        const uint32_t dw = first + s * (stage >> 4) + skip, dx = first + s * (stage >> 4) + (2 * part >> 4);
#pragma unroll
        for (int kk = 0; kk < FK / 16; ++kk) tc::mma(acc, tc::desc_at(dw, kk * 32), tc::desc_at(dx, kk * 32), idesc, kb != 0 || kk != 0);
        tc::commit(&sm.empty[s]);
        if (++s == (uint32_t)a.stages) s = 0, ++round;
      }
      tc::commit(&sm.done);  // of all products, so that TMEM can be freed
      if (!ok) *abort = 1;
    }
  }
  __syncwarp();
  if (warp >= 3) {
    const int q = warp & 3, r = 32 * q + lane;
    const bool in = r < a.rows && f0 + r < a.f;
    const bool ok = mbar_wait(&sm.done, 0, a.status, nullptr);
    tc::fence_after();
    if (__all_sync(0xffffffffu, ok) && *abort == 0 && 32 * q < a.rows) {
      const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16);
      const size_t at = (size_t)f0 + r;
#pragma unroll 1
      for (int c = 8 * ((warp - 3) >> 2); c < a.cols; c += 8 * (kRowsEpi / 4)) {
        uint32_t g[8], u[8];
        ld8(tb + c, g);
        ld8(tb + up + c, u);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float g0 = __uint_as_float(g[i]), g1 = __uint_as_float(g[i + 1]), u0 = __uint_as_float(u[i]), u1 = __uint_as_float(u[i + 1]);
          if (a.g != nullptr) {
            store_tokens(a.g + at, g0, g1, c + i, lane, a.T, a.f, in);
            store_tokens(a.u + at, u0, u1, c + i, lane, a.T, a.f, in);
          }
          store_tokens(a.z + at, act_of(g0, a.act) * u0, act_of(g1, a.act) * u1, c + i, lane, a.T, a.f, in);
        }
      }
    }
  } else if (warp == 1) {
    mbar_wait(&sm.done, 0, a.status, nullptr);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::dealloc(tmem, 2 * up);
}

// ---- host ------------------------------------------------------------------------------------

constexpr size_t kFfnSmem = sizeof(FfnSmem) + 1024;
static_assert(kFfnSmem <= 232448, "k_ffn_pair exceeds the 227 KB of shared memory per block");

ttt_status map_bf16(CUtensorMap* m, const void* base, int64_t inner, int64_t outer, uint32_t box_in, uint32_t box_out) {
  const uint64_t dims[2] = {(uint64_t)inner, (uint64_t)outer};
  const uint64_t strides[1] = {(uint64_t)inner * 2};
  const uint32_t box[2] = {box_in, box_out};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int pairs_of(int num_sms) { return std::max(1, num_sms / 2); }

// k_ffn_rows takes up to 160 tokens where the pairs would need a second round of tiles, which costs them as
// much as the first (f above 9472 on 148 SMs): 17 x 2560 x 9728: 20.5 us against 31, 128 tokens: 27 against 31,
// 192: 35 against 33; 17 x 8192 x 28672: 148 against 278. In one round the pairs are as fast or faster (17 x 2048
// x 7168: 17.3 against 17.6, 128 tokens: 18.7 against 22.8). Against k_ffn_few it needs more than 8 tokens and
// long rows: 16 x 4096 x 14336: 41 us against 52, 16 x 512 x 28672: 16.8 against 15.2; with 8 tokens 2560 x 9728:
// 20.0 against 18.1, 2048 x 16384: 24.6 against 23.0, 4096 x 14336: 40.4 against 41.4, 8192 x 28672: 144 against 147.
bool takes_rows(int64_t T, int d, int f, int num_sms) {
  return f > FM * pairs_of(num_sms) && T <= 160 && T > (d >= 1024 ? 8 : 16);
}

// Tokens of a tile that each CTA of the pair takes: the fewest, in steps of eight, that cover them in this
// many tiles, rather than 128 and the rest past the end (17 x 2560 x 9728: 31 us instead of 42; 777 x 1000 x
// 2744: 16.4 instead of 17.3).
int rows_of(int64_t T, int tiles_m) { return 8 * cdiv(T, 16 * (int64_t)tiles_m); }

// Columns of f in a forward tile. The pairs take `rounds` tiles each; a k-block of a tile costs the
// loads of its rows and c columns a CTA (about three cycles each) or the products (4·c cycles), and a tile
// some 1500 cycles besides. The fewest cycles win: 777 x 1000 x 2744 takes two rounds of 80 columns instead of
// two of 128.
int columns_of(int tiles_m, int rows, int f, int kblocks, int num_sms) {
  int best = kTileN / 2;
  double least = 0;
  for (int c = kTileN / 2; c >= 32; c -= 8) {
    const int rounds = cdiv((int64_t)tiles_m * cdiv(f, c), pairs_of(num_sms));
    const double cost = (double)rounds * (kblocks * std::max(4.0 * c, 3.0 * (rows + c)) + 1500);
    if (c == kTileN / 2 || cost < least) {
      best = c;
      least = cost;
    }
  }
  return best;
}

// DX and DW: whole tiles in full rounds, and the sums of the tiles left cut so that their parts make
// at most one more (4096 tokens, d 2560, f 9728: DX's 160 tiles take 2 rounds and a sixth of one
// instead of 3).
void plan_parts(FfnArgs& a, int total_k, int num_sms) {
  const int tiles = a.tiles_m * a.tiles_n, pairs = pairs_of(num_sms), rest = tiles % pairs;
  a.whole = tiles;
  a.splits = 1;
  a.per_split = total_k;
  if (rest == 0) return;
  const int splits = std::min(pairs / rest, total_k / 8);
  if (splits < 2) return;
  a.per_split = cdiv(total_k, splits);
  a.splits = cdiv(total_k, a.per_split);  // none empty
  a.whole = tiles - rest;
}

void plan_dx(FfnArgs& a, int64_t T, int d, int f, int num_sms) {
  a.M = (int)T;
  a.N = d;
  a.kblocks = cdiv(f, FK);
  a.tiles_m = cdiv(T, kTileM);
  a.rows = rows_of(T, a.tiles_m);
  a.tiles_n = cdiv(d, kTileN);
  plan_parts(a, 2 * a.kblocks, num_sms);
}

void plan_dw(FfnArgs& a, int64_t T, int d, int f, int num_sms) {
  a.M = f;
  a.N = d;
  a.kblocks = cdiv(T, FK);
  a.tiles_m = 2 * cdiv(f, kTileM);
  a.rows = FM;
  a.tiles_n = cdiv(d, kTileN);
  plan_parts(a, a.kblocks, num_sms);
}

size_t part_bytes(const FfnArgs& a) {
  return (size_t)(a.tiles_m * a.tiles_n - a.whole) * a.splits * kTileM * kTileN * sizeof(float);
}

template <int MODE>
ttt_status launch_pair(const CUtensorMap& A0, const CUtensorMap& A1, const CUtensorMap& B0, const CUtensorMap& B1, FfnArgs& a,
                       int num_sms, cudaStream_t s) {
  TTT_CUDA(cudaFuncSetAttribute(k_ffn_pair<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFfnSmem));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)std::min(units_of(a), pairs_of(num_sms)));
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = kFfnSmem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  TTT_CUDA(cudaLaunchKernelEx(&cfg, k_ffn_pair<MODE>, A0, A1, B0, B1, a));
  if constexpr (MODE != FWD) {
    const int rest = a.tiles_m * a.tiles_n - a.whole;
    if (rest > 0) {
      k_ffn_join<MODE><<<dim3(kTileM / 8, rest), 256, 0, s>>>(a);
      TTT_CUDA(cudaGetLastError());
    }
  }
  return TTT_OK;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

ttt_status gated_ffn(const void* X, const void* Wg, const void* Wu, int64_t T, int d, int f, int act, void* Z, void* G, void* U,
                     const DevStatus& status, int num_sms, cudaStream_t s) {
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16*>(X), *wg = static_cast<const __nv_bfloat16*>(Wg),
                      *wu = static_cast<const __nv_bfloat16*>(Wu);
  __nv_bfloat16 *z = static_cast<__nv_bfloat16*>(Z), *g = static_cast<__nv_bfloat16*>(G), *u = static_cast<__nv_bfloat16*>(U);
  const bool by_rows = takes_rows(T, d, f, num_sms);
  if (T <= 16 && !by_rows) {
    const int threads = 32 * kFewWarps;
    if (T <= 8)
      k_ffn_few<1, 1><<<f / 8, threads, 0, s>>>(x, wg, wu, (int)T, d, f, act, z, g, u);
    else
      k_ffn_few<2, 2><<<cdiv(f, 16), threads, 0, s>>>(x, wg, wu, (int)T, d, f, act, z, g, u);
    TTT_CUDA(cudaGetLastError());
    return TTT_OK;
  }
  if (by_rows) {
    RowsArgs a = {};
    a.T = (int)T;
    a.f = f;
    a.kblocks = cdiv(d, FK);
    const int rounds = cdiv(f, (int64_t)FM * num_sms);
    a.rows = 2 * cdiv(f, (int64_t)2 * rounds * num_sms);
    a.cols = 16 * cdiv(T, 16);
    a.stages = std::min(kRowsMaxStages, kRowsRing / rows_stage(a.rows, a.cols));
    a.act = act;
    a.z = z;
    a.g = g;
    a.u = u;
    a.status = status;
    a.stall = op_stall(a.kblocks > 1);
    CUtensorMap tx, tg, tu;
    TTT_TRY(map_bf16(&tx, X, d, T, FK, a.cols));
    TTT_TRY(map_bf16(&tg, Wg, d, f, FK, a.rows));
    TTT_TRY(map_bf16(&tu, Wu, d, f, FK, a.rows));
    const int smem = a.stages * rows_stage(a.rows, a.cols) + kRowsSlack + 1024;
    TTT_CUDA(cudaFuncSetAttribute(k_ffn_rows, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsRing + kRowsSlack + 1024));
    k_ffn_rows<<<cdiv(f, a.rows), kRowsThreads, smem, s>>>(tx, tg, tu, a);
    TTT_CUDA(cudaGetLastError());
    return TTT_OK;
  }
  FfnArgs a = {};
  a.M = (int)T;
  a.N = f;
  a.kblocks = cdiv(d, FK);
  a.tiles_m = cdiv(T, kTileM);
  a.rows = rows_of(T, a.tiles_m);
  a.cols = columns_of(a.tiles_m, a.rows, f, a.kblocks, num_sms);
  a.tiles_n = cdiv(f, a.cols);
  a.whole = a.tiles_m * a.tiles_n;
  a.splits = 1;
  CUtensorMap tx, tg, tu;
  TTT_TRY(map_bf16(&tx, X, d, T, FK, a.rows));
  TTT_TRY(map_bf16(&tg, Wg, d, f, FK, a.cols));
  TTT_TRY(map_bf16(&tu, Wu, d, f, FK, a.cols));
  a.per_split = a.kblocks;
  a.act = act;
  a.z = z;
  a.g = g;
  a.u = u;
  a.status = status;
  a.stall = op_stall(a.kblocks > 1);
  return launch_pair<FWD>(tx, tx, tg, tu, a, num_sms, s);
}

size_t gated_ffn_backward_workspace(int64_t T, int d, int f, int num_sms) {
  FfnArgs x = {}, w = {};
  plan_dx(x, T, d, f, num_sms);
  plan_dw(w, T, d, f, num_sms);
  return 2 * round256((size_t)T * f * 2) + std::max(part_bytes(x), part_bytes(w));
}

ttt_status gated_ffn_backward(const void* dZ, const void* X, const void* Wg, const void* Wu, const void* G, const void* U,
                              int64_t T, int d, int f, int act, void* dX, void* dWg, void* dWu, void* ws,
                              const DevStatus& status, int num_sms, cudaStream_t s) {
  const size_t n = (size_t)T * f;
  uint8_t* w = static_cast<uint8_t*>(ws);
  __nv_bfloat16* dg = reinterpret_cast<__nv_bfloat16*>(w);
  __nv_bfloat16* du = reinterpret_cast<__nv_bfloat16*>(w + round256(n * 2));
  float* part = reinterpret_cast<float*>(w + 2 * round256(n * 2));
  const unsigned blocks = (unsigned)((n / 8 + 255) / 256);
  const __nv_bfloat16 *z = static_cast<const __nv_bfloat16*>(dZ), *g = static_cast<const __nv_bfloat16*>(G),
                      *u = static_cast<const __nv_bfloat16*>(U);
  if (act == TTT_ACT_SILU)
    k_ffn_act_bwd<TTT_ACT_SILU><<<blocks, 256, 0, s>>>(z, g, u, dg, du, n);
  else
    k_ffn_act_bwd<TTT_ACT_GELU><<<blocks, 256, 0, s>>>(z, g, u, dg, du, n);
  TTT_CUDA(cudaGetLastError());
  FfnArgs a = {};
  a.status = status;
  a.stall = op_stall(dX != nullptr || (dWg != nullptr && T > FK));
  a.part = part;
  CUtensorMap A0, A1, B0, B1;
  if (dX != nullptr) {
    plan_dx(a, T, d, f, num_sms);
    TTT_TRY(map_bf16(&A0, dg, f, T, FK, a.rows));
    TTT_TRY(map_bf16(&A1, du, f, T, FK, a.rows));
    TTT_TRY(map_bf16(&B0, Wg, d, f, 64, FK));
    TTT_TRY(map_bf16(&B1, Wu, d, f, 64, FK));
    a.z = static_cast<__nv_bfloat16*>(dX);
    TTT_TRY(launch_pair<DX>(A0, A1, B0, B1, a, num_sms, s));
  }
  if (dWg != nullptr) {
    TTT_TRY(map_bf16(&A0, dg, f, T, 64, FK));
    TTT_TRY(map_bf16(&A1, du, f, T, 64, FK));
    TTT_TRY(map_bf16(&B0, X, d, T, 64, FK));
    plan_dw(a, T, d, f, num_sms);
    a.g = static_cast<__nv_bfloat16*>(dWg);
    a.u = static_cast<__nv_bfloat16*>(dWu);
    TTT_TRY(launch_pair<DW>(A0, A1, B0, B0, a, num_sms, s));
  }
  return TTT_OK;
}

}  // namespace ttt
