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
//   DX   rows: tokens; columns: 256 of d; the sum runs over dG·Wg and then dU·Wu in the same
//        accumulator. A K-major, B MN-major. With fewer tiles than SM pairs the sum is cut into
//        parts, whose fp32 results a second launch adds in order.
//   DW   rows: 256 of f, gate tiles and then up tiles; columns: 256 of d; the sum runs over the
//        tokens. A, B MN-major: X, dG and dU are read as they lie, nothing is transposed.
// Sizes need not be multiples of the tiles: TMA reads zeros past the ends, stores are clipped.
//
// k_ffn_few takes up to 32 tokens, where the weights' bytes are all that counts: see there.
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
  uint64_t full[kFStages], empty[kFStages];
  uint64_t tfull[2], tempty[2];
  uint32_t tmem;
  int abort;
};

struct FfnArgs {
  int M, N;           // rows and columns of the result (FWD: T, f; DX: T, d; DW: f, d)
  int kblocks;        // k-blocks of one product (DX: of each of the two)
  int tiles_m, tiles_n, splits, per_split;
  int act;
  __nv_bfloat16 *z, *g, *u;  // FWD: outputs (g and u or null); DX: z = dX; DW: g = dWg, u = dWu
  float* part;               // DX with splits > 1: [splits][M][N]
  DevStatus status;
};

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * (1.f + erff(x * 0.70710678118654752f)); }

__device__ __forceinline__ float act_of(float x, int act) {
  return act == TTT_ACT_SILU ? x * sigmoid(x) : x * normal_cdf(x);
}

// Stores 32 bf16 values of one row, clipped to ncols (a multiple of 8).
__device__ __forceinline__ void store32(__nv_bfloat16* row, int col0, int ncols, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col0 + 8 * i < ncols)
      *reinterpret_cast<uint4*>(row + col0 + 8 * i) =
          make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                     pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
}

// Tile t of the order that keeps the running tiles on few rows and columns at once (L2): blocks of
// eight row tiles, down the rows first.
__device__ __forceinline__ void tile_at(const FfnArgs& a, int t, int& m, int& n, int& split) {
  const int per = a.tiles_m * a.tiles_n;
  split = t / per;
  t %= per;
  const int block = t / (8 * a.tiles_n), m0 = 8 * block, rows = min(8, a.tiles_m - m0);
  const int r = t - block * 8 * a.tiles_n;
  m = m0 + r % rows;
  n = r / rows;
}

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
  const int ntiles = a.tiles_m * a.tiles_n * a.splits;
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
  auto k_range = [&](int split, int& k0, int& k1) {
    k0 = split * a.per_split;
    k1 = min(total_k, k0 + a.per_split);
  };

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmA0);
      tma_prefetch_desc(&tmB0);
      uint32_t it = 0;
      bool ok = true;
      for (int t = me; t < ntiles && ok; t += npairs) {
        int m, n, split, k0, k1;
        tile_at(a, t, m, n, split);
        k_range(split, k0, k1);
        for (int kb = k0; kb < k1; ++kb, ++it) {
          const int s = it % kFStages;
          if (*abort || (it >= (uint32_t)kFStages && !mbar_wait(&sm.empty[s], ((it / kFStages) - 1) & 1, a.status, abort))) {
            ok = false;
            break;
          }
          uint8_t *sa = sm.ring[s], *sb = sa + kHalf;
          // Both CTAs' loads complete on the first CTA's barrier, which expects the bytes of both.
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 4 * kHalf);
          const uint32_t bar = pair::in_first(&sm.full[s]);
          if constexpr (MODE == FWD) {
            pair::load_2d(sa, &tmA0, bar, kb * FK, m * kTileM + rank * FM);
            pair::load_2d(sb, rank ? &tmB1 : &tmB0, bar, kb * FK, n * (kTileN / 2));
          } else if constexpr (MODE == DX) {
            const bool up = kb >= a.kblocks;
            const int k = (up ? kb - a.kblocks : kb) * FK;
            pair::load_2d(sa, up ? &tmA1 : &tmA0, bar, k, m * kTileM + rank * FM);
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
      constexpr uint32_t idesc = tc::idesc_bf16(kTileM, kTileN, MODE == DW, MODE != FWD);
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int t = me; t < ntiles && ok; t += npairs) {
        int m, n, split, k0, k1;
        tile_at(a, t, m, n, split);
        k_range(split, k0, k1);
        const int acc = tcount & 1;
        if (tcount >= 2 && !mbar_wait<true>(&sm.tempty[acc], ((tcount >> 1) - 1) & 1, a.status, abort)) {
          ok = false;
          break;
        }
        tc::fence_after();
        for (int kb = k0; kb < k1; ++kb, ++it) {
          const int s = it % kFStages;
          if (!mbar_wait<true>(&sm.full[s], (it / kFStages) & 1, a.status, abort)) {
            ok = false;
            break;
          }
          tc::fence_after();
          const uint32_t a0 = smem_u32(sm.ring[s]), b0 = a0 + kHalf;
#pragma unroll
          for (int kk = 0; kk < FK / 16; ++kk) {
            const uint64_t ad = MODE == DW ? tc::smem_desc(a0 + kk * 2048, 8192, 1024) : tc::smem_desc(a0 + kk * 32, 16, 1024);
            const uint64_t bd = MODE == FWD ? tc::smem_desc(b0 + kk * 32, 16, 1024) : tc::smem_desc(b0 + kk * 2048, 8192, 1024);
            pair::mma(tmem + acc * kTileN, ad, bd, idesc, (kb != k0 || kk != 0));
          }
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
    const int lq = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter, half of the columns
    uint32_t tcount = 0;
    for (int t = me; t < ntiles; t += npairs) {
      int m, n, split;
      tile_at(a, t, m, n, split);
      const int acc = tcount & 1;
      const bool ok = mbar_wait(&sm.tfull[acc], (tcount >> 1) & 1, a.status, nullptr);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::fence_after();
      const uint32_t tb = tmem + ((uint32_t)(lq * 32) << 16) + (uint32_t)(acc * kTileN);
      int row = m * kTileM + rank * FM + lq * 32 + lane;
      if constexpr (MODE == FWD) {
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          const int c = half * 64 + j * 32, col = n * (kTileN / 2) + c;
          uint32_t rg[32], ru[32];
          tc::ld32(tb + c, rg);
          tc::ld32(tb + kTileN / 2 + c, ru);
          tc::wait_ld();
          float g[32], u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            g[i] = __uint_as_float(rg[i]);
            u[i] = __uint_as_float(ru[i]);
          }
          if (row < a.M) {
            const size_t at = (size_t)row * a.N;
            if (a.g != nullptr) {
              store32(a.g + at, col, a.N, g);
              store32(a.u + at, col, a.N, u);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) g[i] = act_of(g[i], a.act) * u[i];
            store32(a.z + at, col, a.N, g);
          }
        }
      } else {
        __nv_bfloat16* out = a.z;
        int mrow = row;
        if constexpr (MODE == DW) {
          const int half_m = a.tiles_m / 2;
          out = m >= half_m ? a.u : a.g;
          mrow = m >= half_m ? row - half_m * kTileM : row;
        }
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          const int c = half * 128 + j * 32, col = n * kTileN + c;
          uint32_t r[32];
          tc::ld32(tb + c, r);
          tc::wait_ld();
          if (mrow < a.M) {
            if (MODE == DX && a.splits > 1) {
              float* p = a.part + ((size_t)split * a.M + mrow) * a.N + col;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (col + 4 * i < a.N)
                  *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            } else {
              float v[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
              store32(out + (size_t)mrow * a.N, col, a.N, v);
            }
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

// out = Σ over the parts, in order, as bf16; eight values a thread.
__global__ void __launch_bounds__(256) k_ffn_join(const float* __restrict__ part, int splits, size_t n, __nv_bfloat16* __restrict__ out) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float v[8] = {};
  for (int s = 0; s < splits; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(part + s * n + i), y = *reinterpret_cast<const float4*>(part + s * n + i + 4);
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
  *reinterpret_cast<uint4*>(out + i) =
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

// ---- up to 32 tokens -------------------------------------------------------------------------

// The weights' bytes bound it, so they go from HBM straight into the registers that the tensor
// cores read (mma.sync: with at most 32 columns its rate is far from counting), with no stage in
// shared memory and no barrier on the way. A CTA of eight warps takes 16 rows of Wg and the same 16
// of Wu; warp w takes every eighth 32-wide slice of the sum, and the warps' results are added in
// order at the end. A lane's 16-byte load holds eight consecutive k of one row; the products' k
// slots are filled in that order for the weights and for X alike, which a sum does not mind.
// NT: token blocks of eight.
template <int NT>
__global__ void __launch_bounds__(256) k_ffn_few(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ Wg,
                                                 const __nv_bfloat16* __restrict__ Wu, int T, int d, int f, int act,
                                                 __nv_bfloat16* __restrict__ z, __nv_bfloat16* __restrict__ gout,
                                                 __nv_bfloat16* __restrict__ uout) {
  __shared__ float part[8][2][NT][8][17];  // [warp][gate, up][token block][token][row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int f0 = blockIdx.x * 16;
  const int steps = (d + 31) / 32;
  float ag[NT][4] = {}, au[NT][4] = {};
  const bool lo = f0 + g < f, hi = f0 + g + 8 < f;
  const __nv_bfloat16* pg = Wg + (size_t)(f0 + (lo ? g : 0)) * d + 8 * q;
  const __nv_bfloat16* pu = Wu + (size_t)(f0 + (lo ? g : 0)) * d + 8 * q;
  const size_t down = hi ? (size_t)8 * d : 0;
  const uint4 none = make_uint4(0, 0, 0, 0);
  constexpr int UN = NT == 1 ? 4 : 2;
  for (int st = warp; st < steps; st += 8 * UN) {
    uint4 wg[UN][2], wu[UN][2], x[UN][NT];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = (st + 8 * i) * 32;
      const bool in = k + 8 * q < d;
      wg[i][0] = in && lo ? __ldcs(reinterpret_cast<const uint4*>(pg + k)) : none;
      wg[i][1] = in && hi ? __ldcs(reinterpret_cast<const uint4*>(pg + down + k)) : none;
      wu[i][0] = in && lo ? __ldcs(reinterpret_cast<const uint4*>(pu + k)) : none;
      wu[i][1] = in && hi ? __ldcs(reinterpret_cast<const uint4*>(pu + down + k)) : none;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        x[i][nt] = in && 8 * nt + g < T ? *reinterpret_cast<const uint4*>(X + (size_t)(8 * nt + g) * d + k + 8 * q) : none;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const uint32_t a0[4] = {wg[i][0].x, wg[i][1].x, wg[i][0].y, wg[i][1].y}, a1[4] = {wg[i][0].z, wg[i][1].z, wg[i][0].w, wg[i][1].w};
      const uint32_t b0[4] = {wu[i][0].x, wu[i][1].x, wu[i][0].y, wu[i][1].y}, b1[4] = {wu[i][0].z, wu[i][1].z, wu[i][0].w, wu[i][1].w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        wm::mma(ag[nt], a0, x[i][nt].x, x[i][nt].y);
        wm::mma(ag[nt], a1, x[i][nt].z, x[i][nt].w);
        wm::mma(au[nt], b0, x[i][nt].x, x[i][nt].y);
        wm::mma(au[nt], b1, x[i][nt].z, x[i][nt].w);
      }
    }
  }
  // A lane holds rows g, g + 8 (of the 16) and tokens 2q, 2q + 1 of each block.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      part[warp][0][nt][2 * q + (e & 1)][g + 8 * (e >> 1)] = ag[nt][e];
      part[warp][1][nt][2 * q + (e & 1)][g + 8 * (e >> 1)] = au[nt][e];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 128; i += 256) {
    const int r = i & 15, t = i >> 4;
    if (t >= T || f0 + r >= f) continue;
    float sg = 0.f, su = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      sg += part[w][0][t >> 3][t & 7][r];
      su += part[w][1][t >> 3][t & 7][r];
    }
    const size_t at = (size_t)t * f + f0 + r;
    if (gout != nullptr) {
      gout[at] = __float2bfloat16_rn(sg);
      uout[at] = __float2bfloat16_rn(su);
    }
    z[at] = __float2bfloat16_rn(act_of(sg, act) * su);
  }
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

template <int MODE>
ttt_status launch_pair(const CUtensorMap& A0, const CUtensorMap& A1, const CUtensorMap& B0, const CUtensorMap& B1, FfnArgs& a,
                       int num_sms, cudaStream_t s) {
  TTT_CUDA(cudaFuncSetAttribute(k_ffn_pair<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFfnSmem));
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n * a.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(tiles, std::max(1, num_sms / 2)));
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
  return TTT_OK;
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Parts of dX's sum: as many as give every SM pair a tile, each of at least 16 k-blocks.
int dx_splits(int64_t T, int d, int f, int num_sms) {
  const int64_t tiles = (int64_t)cdiv(T, kTileM) * cdiv(d, kTileN), pairs = std::max(1, num_sms / 2);
  const int64_t kb = 2 * (int64_t)cdiv(f, FK);
  return (int)std::max<int64_t>(1, std::min<int64_t>(pairs / std::max<int64_t>(1, tiles), kb / 16));
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

ttt_status gated_ffn(const void* X, const void* Wg, const void* Wu, int64_t T, int d, int f, int act, void* Z, void* G, void* U,
                     int32_t* status, int num_sms, cudaStream_t s) {
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16*>(X), *wg = static_cast<const __nv_bfloat16*>(Wg),
                      *wu = static_cast<const __nv_bfloat16*>(Wu);
  __nv_bfloat16 *z = static_cast<__nv_bfloat16*>(Z), *g = static_cast<__nv_bfloat16*>(G), *u = static_cast<__nv_bfloat16*>(U);
  if (T <= 32) {
    const int grid = cdiv(f, 16);
    if (T <= 8)
      k_ffn_few<1><<<grid, 256, 0, s>>>(x, wg, wu, (int)T, d, f, act, z, g, u);
    else if (T <= 16)
      k_ffn_few<2><<<grid, 256, 0, s>>>(x, wg, wu, (int)T, d, f, act, z, g, u);
    else
      k_ffn_few<4><<<grid, 256, 0, s>>>(x, wg, wu, (int)T, d, f, act, z, g, u);
    TTT_CUDA(cudaGetLastError());
    return TTT_OK;
  }
  CUtensorMap tx, tg, tu;
  TTT_TRY(map_bf16(&tx, X, d, T, FK, FM));
  TTT_TRY(map_bf16(&tg, Wg, d, f, FK, FM));
  TTT_TRY(map_bf16(&tu, Wu, d, f, FK, FM));
  FfnArgs a = {};
  a.M = (int)T;
  a.N = f;
  a.kblocks = cdiv(d, FK);
  a.tiles_m = cdiv(T, kTileM);
  a.tiles_n = cdiv(f, kTileN / 2);
  a.splits = 1;
  a.per_split = a.kblocks;
  a.act = act;
  a.z = z;
  a.g = g;
  a.u = u;
  a.status = DevStatus{status, kWaitLimitNs};
  return launch_pair<FWD>(tx, tx, tg, tu, a, num_sms, s);
}

size_t gated_ffn_backward_workspace(int64_t T, int d, int f, int num_sms) {
  const int splits = dx_splits(T, d, f, num_sms);
  return 2 * round256((size_t)T * f * 2) + (splits > 1 ? (size_t)splits * T * d * 4 : 0);
}

ttt_status gated_ffn_backward(const void* dZ, const void* X, const void* Wg, const void* Wu, const void* G, const void* U,
                              int64_t T, int d, int f, int act, void* dX, void* dWg, void* dWu, void* ws, int32_t* status,
                              int num_sms, cudaStream_t s) {
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
  a.status = DevStatus{status, kWaitLimitNs};
  CUtensorMap A0, A1, B0, B1;
  if (dX != nullptr) {
    TTT_TRY(map_bf16(&A0, dg, f, T, FK, FM));
    TTT_TRY(map_bf16(&A1, du, f, T, FK, FM));
    TTT_TRY(map_bf16(&B0, Wg, d, f, 64, FK));
    TTT_TRY(map_bf16(&B1, Wu, d, f, 64, FK));
    a.M = (int)T;
    a.N = d;
    a.kblocks = cdiv(f, FK);
    a.tiles_m = cdiv(T, kTileM);
    a.tiles_n = cdiv(d, kTileN);
    a.splits = dx_splits(T, d, f, num_sms);
    a.per_split = cdiv(2 * a.kblocks, a.splits);
    a.splits = cdiv(2 * a.kblocks, a.per_split);  // none empty
    a.z = static_cast<__nv_bfloat16*>(dX);
    a.part = part;
    TTT_TRY(launch_pair<DX>(A0, A1, B0, B1, a, num_sms, s));
    if (a.splits > 1) {
      const size_t nx = (size_t)T * d;
      k_ffn_join<<<(unsigned)((nx / 8 + 255) / 256), 256, 0, s>>>(part, a.splits, nx, a.z);
      TTT_CUDA(cudaGetLastError());
    }
  }
  if (dWg != nullptr) {
    TTT_TRY(map_bf16(&A0, dg, f, T, 64, FK));
    TTT_TRY(map_bf16(&A1, du, f, T, 64, FK));
    TTT_TRY(map_bf16(&B0, X, d, T, 64, FK));
    a.M = f;
    a.N = d;
    a.kblocks = cdiv(T, FK);
    a.tiles_m = 2 * cdiv(f, kTileM);
    a.tiles_n = cdiv(d, kTileN);
    a.splits = 1;
    a.per_split = a.kblocks;
    a.g = static_cast<__nv_bfloat16*>(dWg);
    a.u = static_cast<__nv_bfloat16*>(dWu);
    TTT_TRY(launch_pair<DW>(A0, A1, B0, B0, a, num_sms, s));
  }
  return TTT_OK;
}

}  // namespace ttt
