// Gated linear recurrence on 64 x 64 per-head states: the fast weight with a forget gate and the
// Hebbian update, S_t = e^{g_t}·S_{t-1} + k_tᵀ·v_t, o_t = scale · q_t·S_t, its gradients, and its
// one-token form.
//
// Mathematics. Tokens are taken in chunks of 64. With b_i the sum of the chunk's gates up to and
// with token i, S the state before the chunk and w_j = e^{b_64 - b_j}:
//   O  = scale · [ e^{b_i}·(Q·S)_i + Σ_{j <= i} e^{b_i - b_j}·(q_i·k_j)·v_j ]
//   S' = e^{b_64}·S + (w ⊙ K)ᵀ·V
// so a chunk is four 64 x 64 x 64 products, and only S goes from chunk to chunk. Backward, with
// dS' the gradient of the state after the chunk and u_i = scale·e^{b_i}:
//   dQ = u ⊙ (dO·Sᵀ) + A·K,      A_ij = scale·e^{b_i - b_j}·(do_i·v_j)  (j <= i)
//   dK = w ⊙ (V·dS'ᵀ) + Aᵀ·Q
//   dV = w ⊙ (K·dS') + Pᵀ·dO,    P_ij = scale·e^{b_i - b_j}·(q_i·k_j)  (j <= i)
//   dS = e^{b_64}·dS' + (u ⊙ Q)ᵀ·dO
//   dg_t = e^{b_64}·<S, dS'> + Σ_{i >= t} q_i·(u_i·S·do_i) + Σ_{j < t} k_j·(w_j·dS'·v_j)
//          + Σ_{i >= t > j} A_ij·(q_i·k_j)
// (the gate of token t scales every path from before t to t or after). Each chunk's dg starts
// from the states, not from the chunk after it, so rounding does not add up along the sequence.
//
// Precision. The products run on the tensor cores with bf16 operands and fp32 sums. S and dS stay
// in fp32 registers. Where a product's result is a bf16 output, one factor is rounded to bf16
// (P, A, or the copy of S); where it feeds a fp32 output (the states and dg), the rounded factor
// is kept as a sum of two bf16 numbers (2^-17 of its size), at the price of a second product.
// The gates are summed in base-2 units; one below -150 (its factor is 0 in fp32, as for -inf,
// which starts a new document) counts as -150, so that differences of sums stay finite.
//
// Where there are fewer (sequence, head) pairs than the SMs hold CTAs, the sequence is cut into
// segments: the states that the segments add are found first, combined in order, and then every
// segment runs from its own start.
#include <algorithm>

#include "internal.h"
#include "warp_mma.cuh"

namespace ttt {

namespace {

constexpr int kC = 64;               // tokens per chunk
constexpr int kD = 64;               // head width
constexpr int kTile = kC * 128;      // bytes of a [64][64] bf16 tile
constexpr int kState = kD * kD;      // elements of a state
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinGate = -150.f;   // base-2 units: 2^-150 is 0 in fp32
constexpr float kGoneGate = -104.f;  // a gate below kMinGate / kLog2e

struct Rows {  // bf16 [batch, heads, tokens, 64] with strides in elements
  const __nv_bfloat16* p;
  int64_t sb, sh, st;
};

struct GsArgs {
  int heads, nchunk, nseg, per_seg;  // per_seg: chunks of a segment
  int64_t T;
  float scale;
  Rows q, k, v, dout;
  const float* g;
  int64_t gb, gh, gt;
  __nv_bfloat16* o;                   // forward outputs
  int64_t ob, oh, ot;
  const float* start;                 // [pairs][nseg or 1][64][64] states the segments start from, or null (zero)
  float* end;                         // final state [pairs][64][64] (the last segment's), or null
  float* local;                       // what each segment adds [pairs][nseg][64][64]
  float* seg_decay;                   // sums of the segments' gates, base-2 units [pairs][nseg]
  __nv_bfloat16* ckpt;                // state before every chunk, as two bf16 planes [pairs][nchunk][2][64][64]
  __nv_bfloat16 *dq, *dk, *dv;        // dense [pairs][T][64]
  float* dg;                          // dense [pairs][T]
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of a chunk's gates up to and with each token, base-2 units, into b[64] (one copy per warp;
// the calling warp's lanes hold the raw gates of tokens lane and lane + 32).
__device__ __forceinline__ void gate_sums(float g0, float g1, float* b, int lane) {
  float x0 = g0 * kLog2e, x1 = g1 * kLog2e;
  x0 = x0 < kMinGate ? kMinGate : x0;  // NaN stays
  x1 = x1 < kMinGate ? kMinGate : x1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y0 = __shfl_up_sync(0xffffffffu, x0, o), y1 = __shfl_up_sync(0xffffffffu, x1, o);
    if (lane >= o) {
      x0 += y0;
      x1 += y1;
    }
  }
  x1 += __shfl_sync(0xffffffffu, x0, 31);
  __syncwarp();
  b[lane] = x0;
  b[lane + 32] = x1;
  __syncwarp();
}

__device__ __forceinline__ void load_gates(const GsArgs& a, const float* gp, int64_t t0, int lane, float& g0, float& g1) {
  g0 = t0 + lane < a.T ? gp[(t0 + lane) * a.gt] : 0.f;
  g1 = t0 + lane + 32 < a.T ? gp[(t0 + lane + 32) * a.gt] : 0.f;
}

// Asynchronous copy of tokens t0 .. t0 + 63 of one (sequence, head) into a tile (rows past T zero).
template <int THREADS>
__device__ __forceinline__ void load_rows(uint32_t tile, const __nv_bfloat16* base, int64_t st, int64_t t0, int64_t T) {
#pragma unroll
  for (int i = threadIdx.x; i < kC * 8; i += THREADS) {
    const int r = i >> 3, c = i & 7;
    const bool ok = t0 + r < T;
    wm::cp16(tile + r * 128 + ((c ^ (r & 7)) << 4), base + (ok ? (t0 + r) * st : 0) + 8 * c, ok);
  }
}

// S += (w ⊙ X)ᵀ·Y for this warp's rows 16·warp .. +15 of S: X and Y tiles of 64 tokens, the
// weighted X as two bf16 terms.
__device__ __forceinline__ void add_outer(float (&S)[8][4], uint32_t X, uint32_t Y, const float (&w)[16], int row0, int lane) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint32_t x[4], hi[4], lo[4];
    wm::frag_a_t(X, 16 * ks, row0, lane, x);
    // Registers 0, 1 hold tokens 16·ks + 2q, + 1 and registers 2, 3 those 8 later.
    wm::scale_split(x[0], w[4 * ks], w[4 * ks + 1], hi[0], lo[0]);
    wm::scale_split(x[1], w[4 * ks], w[4 * ks + 1], hi[1], lo[1]);
    wm::scale_split(x[2], w[4 * ks + 2], w[4 * ks + 3], hi[2], lo[2]);
    wm::scale_split(x[3], w[4 * ks + 2], w[4 * ks + 3], hi[3], lo[3]);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t y[4];
      wm::frag_b_t(Y, 16 * ks, 16 * np, lane, y);
      wm::mma(S[2 * np], hi, y[0], y[1]);
      wm::mma(S[2 * np + 1], hi, y[2], y[3]);
      wm::mma(S[2 * np], lo, y[0], y[1]);
      wm::mma(S[2 * np + 1], lo, y[2], y[3]);
    }
  }
}

// A thread's part of a [64][64] fp32 state: rows row0 + g, + 8, columns 8·nt + 2q, + 1.
__device__ __forceinline__ void load_state(float (&S)[8][4], const float* p, int row0, int lane) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = p == nullptr ? make_float2(0.f, 0.f)
                                    : *reinterpret_cast<const float2*>(p + (row0 + g + 8 * h) * kD + 8 * nt + 2 * q);
      S[nt][2 * h] = x.x;
      S[nt][2 * h + 1] = x.y;
    }
}

__device__ __forceinline__ void store_state(const float (&S)[8][4], float* p, int row0, int lane) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2*>(p + (row0 + g + 8 * h) * kD + 8 * nt + 2 * q) = make_float2(S[nt][2 * h], S[nt][2 * h + 1]);
}

// ---- states --------------------------------------------------------------------------------

struct __align__(1024) StateSmem {
  uint8_t X[2][kTile], Y[2][kTile];
  float b[4][kC];
};

// Runs the state alone over a segment, 128 threads, warp w rows 16w .. 16w + 15 of the state.
// Forward: X = K, Y = V, weights w; REV: from the last chunk to the first, X = Q, Y = dO, weights
// u. CKPT: writes the state before every chunk (forward). grid: pairs · nseg.
template <bool REV, bool CKPT>
__global__ void __launch_bounds__(128, 4) k_gs_state(const GsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  StateSmem& sm = *reinterpret_cast<StateSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int pair = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int64_t bi = pair / a.heads, hi_ = pair % a.heads;
  const Rows& rx = REV ? a.q : a.k;
  const Rows& ry = REV ? a.dout : a.v;
  const __nv_bfloat16* X = rx.p + bi * rx.sb + hi_ * rx.sh;
  const __nv_bfloat16* Y = ry.p + bi * ry.sb + hi_ * ry.sh;
  const float* gp = a.g + bi * a.gb + hi_ * a.gh;
  const int c0 = seg * a.per_seg, c1 = min(a.nchunk, c0 + a.per_seg), n = c1 - c0;
  auto chunk_at = [&](int i) { return REV ? c1 - 1 - i : c0 + i; };
  auto load = [&](int i) {
    const int64_t t0 = (int64_t)chunk_at(i) * kC;
    load_rows<128>(smem_u32(sm.X[i & 1]), X, rx.st, t0, a.T);
    load_rows<128>(smem_u32(sm.Y[i & 1]), Y, ry.st, t0, a.T);
    wm::cp_commit();
  };
  float S[8][4];
  load_state(S, a.start != nullptr ? a.start + (size_t)blockIdx.x * kState : nullptr, 16 * warp, lane);
  float decay = 0.f, g0 = 0.f, g1 = 0.f;
  if (n > 0) {
    load(0);
    load_gates(a, gp, (int64_t)chunk_at(0) * kC, lane, g0, g1);
  }
  for (int i = 0; i < n; ++i) {
    gate_sums(g0, g1, sm.b[warp], lane);
    if constexpr (CKPT) {
      __nv_bfloat16* hp = a.ckpt + ((size_t)pair * a.nchunk + chunk_at(i)) * 2 * kState;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = (16 * warp + g + 8 * h) * kD + 8 * nt + 2 * q;
          const uint32_t hi = pack_bf16(S[nt][2 * h], S[nt][2 * h + 1]);
          const float2 f = wm::unpack(hi);
          *reinterpret_cast<uint32_t*>(hp + at) = hi;
          *reinterpret_cast<uint32_t*>(hp + kState + at) = pack_bf16(S[nt][2 * h] - f.x, S[nt][2 * h + 1] - f.y);
        }
    }
    wm::cp_wait<0>();
    __syncthreads();
    if (i + 1 < n) {
      load(i + 1);
      load_gates(a, gp, (int64_t)chunk_at(i + 1) * kC, lane, g0, g1);
    }
    const float* b = sm.b[warp];
    const float bC = b[kC - 1];
    float w[16];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = b[16 * ks + 2 * q + (e & 1) + 8 * (e >> 1)];
        w[4 * ks + e] = REV ? a.scale * exp2_fast(x) : exp2_fast(bC - x);
      }
    const float keep = exp2_fast(bC);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[nt][e] *= keep;
    add_outer(S, smem_u32(sm.X[i & 1]), smem_u32(sm.Y[i & 1]), w, 16 * warp, lane);
    decay += bC;
  }
  if (a.local != nullptr) {
    store_state(S, a.local + (size_t)blockIdx.x * kState, 16 * warp, lane);
    if (threadIdx.x == 0) a.seg_decay[blockIdx.x] = decay;
  }
}

// The states the segments start from, in place of what they add: start[s + 1] =
// 2^decay[s]·start[s] + local[s], from `first` (or zero); REV: start[s − 1] from start[s].
// grid (pairs, 64·64 / 4 / 128), one float4 a thread.
template <bool REV>
__global__ void __launch_bounds__(128) k_gs_combine(float* local, const float* __restrict__ decay,
                                                    const float* __restrict__ first, int nseg) {
  const int at = (blockIdx.y * 128 + threadIdx.x) * 4;
  const size_t pair = blockIdx.x;
  float4 s = first != nullptr ? *reinterpret_cast<const float4*>(first + pair * kState + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  float* p = local + pair * nseg * kState + at;
  const float* d = decay + pair * nseg;
#pragma unroll 4
  for (int i = 0; i < nseg; ++i) {
    const int seg = REV ? nseg - 1 - i : i;
    float4* at_seg = reinterpret_cast<float4*>(p + (size_t)seg * kState);
    const float4 x = *at_seg;
    const float f = exp2_fast(d[seg]);
    *at_seg = s;
    s.x = fmaf(f, s.x, x.x);
    s.y = fmaf(f, s.y, x.y);
    s.z = fmaf(f, s.z, x.z);
    s.w = fmaf(f, s.w, x.w);
  }
}

// ---- forward -------------------------------------------------------------------------------

struct __align__(1024) OutSmem {
  uint8_t Q[2][kTile], K[2][kTile], V[2][kTile];
  uint8_t S[2][kTile];  // bf16 copy of the state before the chunk
  float b[4][kC];
};

// 128 threads; warp w holds rows 16w .. 16w + 15 of the state and of each chunk's outputs.
// grid: pairs · nseg.
__global__ void __launch_bounds__(128, 3) k_gs_out(const GsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  OutSmem& sm = *reinterpret_cast<OutSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int pair = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int64_t bi = pair / a.heads, hi_ = pair % a.heads;
  const __nv_bfloat16* Q = a.q.p + bi * a.q.sb + hi_ * a.q.sh;
  const __nv_bfloat16* K = a.k.p + bi * a.k.sb + hi_ * a.k.sh;
  const __nv_bfloat16* V = a.v.p + bi * a.v.sb + hi_ * a.v.sh;
  __nv_bfloat16* O = a.o + bi * a.ob + hi_ * a.oh;
  const float* gp = a.g + bi * a.gb + hi_ * a.gh;
  const int c0 = seg * a.per_seg, c1 = min(a.nchunk, c0 + a.per_seg);
  const int row0 = 16 * warp;
  auto load = [&](int c) {
    const int64_t t0 = (int64_t)c * kC;
    load_rows<128>(smem_u32(sm.Q[c & 1]), Q, a.q.st, t0, a.T);
    load_rows<128>(smem_u32(sm.K[c & 1]), K, a.k.st, t0, a.T);
    load_rows<128>(smem_u32(sm.V[c & 1]), V, a.v.st, t0, a.T);
    wm::cp_commit();
  };
  float S[8][4];
  load_state(S, a.start != nullptr ? a.start + (size_t)blockIdx.x * kState : nullptr, row0, lane);
  float g0 = 0.f, g1 = 0.f;
  if (c0 < c1) {
    load(c0);
    load_gates(a, gp, (int64_t)c0 * kC, lane, g0, g1);
  }
  for (int c = c0; c < c1; ++c) {
    const int64_t t0 = (int64_t)c * kC;
    gate_sums(g0, g1, sm.b[warp], lane);
    uint8_t* Ss = sm.S[c & 1];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<uint32_t*>(Ss + swz128_bf16(row0 + g + 8 * h, 8 * nt + 2 * q)) =
            pack_bf16(S[nt][2 * h], S[nt][2 * h + 1]);
    wm::cp_wait<0>();
    __syncthreads();  // the chunk's rows and the state's copy are visible; the other buffers are free
    if (c + 1 < c1) {
      load(c + 1);
      load_gates(a, gp, t0 + kC, lane, g0, g1);
    }
    const uint32_t Qs = smem_u32(sm.Q[c & 1]), Ks = smem_u32(sm.K[c & 1]), Vs = smem_u32(sm.V[c & 1]);
    const float* b = sm.b[warp];
    uint32_t qa[4][4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) wm::frag_a(Qs, row0, 16 * ks, lane, qa[ks]);
    const float bi0 = b[row0 + g], bi1 = b[row0 + g + 8];

    // u ⊙ (Q·S).
    float o[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
    const uint32_t Sa = smem_u32(Ss);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t y[4];
        wm::frag_b_t(Sa, 16 * ks, 16 * np, lane, y);
        wm::mma(o[2 * np], qa[ks], y[0], y[1]);
        wm::mma(o[2 * np + 1], qa[ks], y[2], y[3]);
      }
    const float u0 = a.scale * exp2_fast(bi0), u1 = a.scale * exp2_fast(bi1);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      o[nt][0] *= u0;
      o[nt][1] *= u0;
      o[nt][2] *= u1;
      o[nt][3] *= u1;
    }

    // P·V over blocks of 16 keys, up to this warp's own tokens.
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      if (kb > warp) break;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t y[4];
        wm::frag_b(Ks, 16 * kb, 16 * ks, lane, y);
        wm::mma(s[0], qa[ks], y[0], y[1]);
        wm::mma(s[1], qa[ks], y[2], y[3]);
      }
      uint32_t pa[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int j = 16 * kb + 8 * nt + 2 * q;
        const float2 bj = *reinterpret_cast<const float2*>(b + j);
        const int i0 = row0 + g;
        const float p0 = j <= i0 ? a.scale * s[nt][0] * exp2_fast(bi0 - bj.x) : 0.f;
        const float p1 = j + 1 <= i0 ? a.scale * s[nt][1] * exp2_fast(bi0 - bj.y) : 0.f;
        const float p2 = j <= i0 + 8 ? a.scale * s[nt][2] * exp2_fast(bi1 - bj.x) : 0.f;
        const float p3 = j + 1 <= i0 + 8 ? a.scale * s[nt][3] * exp2_fast(bi1 - bj.y) : 0.f;
        pa[2 * nt] = pack_bf16(p0, p1);
        pa[2 * nt + 1] = pack_bf16(p2, p3);
      }
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t y[4];
        wm::frag_b_t(Vs, 16 * kb, 16 * np, lane, y);
        wm::mma(o[2 * np], pa, y[0], y[1]);
        wm::mma(o[2 * np + 1], pa, y[2], y[3]);
      }
    }

    // S ← e^{b_64}·S + (w ⊙ K)ᵀ·V.
    {
      const float bC = b[kC - 1];
      float w[16];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * ks + e] = exp2_fast(bC - b[16 * ks + 2 * q + (e & 1) + 8 * (e >> 1)]);
      const float keep = exp2_fast(bC);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] *= keep;
      add_outer(S, Ks, Vs, w, row0, lane);
    }

    // Outputs through this warp's own rows of the query tile (no other warp reads them).
    __syncwarp();
    uint8_t* Qt = sm.Q[c & 1];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<uint32_t*>(Qt + swz128_bf16(row0 + g + 8 * h, 8 * nt + 2 * q)) =
            pack_bf16(o[nt][2 * h], o[nt][2 * h + 1]);
    __syncwarp();
#pragma unroll
    for (int i = lane; i < 128; i += 32) {
      const int r = row0 + (i >> 3), x = i & 7;
      if (t0 + r < a.T)
        *reinterpret_cast<uint4*>(O + (t0 + r) * a.ot + 8 * x) =
            *reinterpret_cast<const uint4*>(Qt + r * 128 + ((x ^ (r & 7)) << 4));
    }
  }
  if (a.end != nullptr && seg == a.nseg - 1) store_state(S, a.end + (size_t)pair * kState, row0, lane);
}

// ---- backward ------------------------------------------------------------------------------

struct __align__(1024) BwdSmem {
  uint8_t Q[2][kTile], K[2][kTile], V[2][kTile], G[2][kTile];  // G: dO
  uint8_t S[2][kTile];   // the state before the chunk: rounded, and what the rounding left
  uint8_t dS[2][kTile];  // the gradient of the state after the chunk, the same way
  float b[8][kC];
  float rows[kC];        // Σ_j A_ij·(q_i·k_j) over j < i, plus q_i·(u_i·S·do_i)
  float cols[kC];        // Σ_i A_ij·(q_i·k_j) over i > j
  float past[kC];        // k_j·(w_j·dS'·v_j)
  float dot[4];          // parts of e^{b_64}·<S, dS'>
};

// 256 threads, from the segment's last chunk to its first. Warps 0 .. 3 take rows of queries (dQ,
// the rows' part of dg) and carry dS; warps 4 .. 7 take rows of keys (dK, dV, their part of dg).
// grid: pairs · nseg.
__global__ void __launch_bounds__(256, 2) k_gs_bwd(const GsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  BwdSmem& sm = *reinterpret_cast<BwdSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int pair = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int64_t bi = pair / a.heads, hi_ = pair % a.heads;
  const __nv_bfloat16* Q = a.q.p + bi * a.q.sb + hi_ * a.q.sh;
  const __nv_bfloat16* K = a.k.p + bi * a.k.sb + hi_ * a.k.sh;
  const __nv_bfloat16* V = a.v.p + bi * a.v.sb + hi_ * a.v.sh;
  const __nv_bfloat16* G = a.dout.p + bi * a.dout.sb + hi_ * a.dout.sh;
  const float* gp = a.g + bi * a.gb + hi_ * a.gh;
  const __nv_bfloat16* ckpt = a.ckpt + (size_t)pair * a.nchunk * 2 * kState;
  const size_t out0 = (size_t)pair * a.T * kD;
  const int c0 = seg * a.per_seg, c1 = min(a.nchunk, c0 + a.per_seg);
  const bool query_side = warp < 4;
  const int row0 = 16 * (warp & 3);

  auto load = [&](int c) {
    const int64_t t0 = (int64_t)c * kC;
    load_rows<256>(smem_u32(sm.Q[c & 1]), Q, a.q.st, t0, a.T);
    load_rows<256>(smem_u32(sm.K[c & 1]), K, a.k.st, t0, a.T);
    load_rows<256>(smem_u32(sm.V[c & 1]), V, a.v.st, t0, a.T);
    load_rows<256>(smem_u32(sm.G[c & 1]), G, a.dout.st, t0, a.T);
  };
  auto load_ckpt = [&](int c) {
    load_rows<256>(smem_u32(sm.S[0]), ckpt + (size_t)c * 2 * kState, kD, 0, kD);
    load_rows<256>(smem_u32(sm.S[1]), ckpt + (size_t)c * 2 * kState + kState, kD, 0, kD);
  };
  float dS[8][4];
  load_state(dS, a.start != nullptr && query_side ? a.start + (size_t)blockIdx.x * kState : nullptr, row0, lane);
  float g0 = 0.f, g1 = 0.f;
  if (c0 < c1) {
    load(c1 - 1);
    load_ckpt(c1 - 1);
    wm::cp_commit();
    load_gates(a, gp, (int64_t)(c1 - 1) * kC, lane, g0, g1);
  }
  for (int c = c1 - 1; c >= c0; --c) {
    const int64_t t0 = (int64_t)c * kC;
    const float raw0 = g0, raw1 = g1;
    gate_sums(g0, g1, sm.b[warp], lane);
    if (query_side) {
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = swz128_bf16(row0 + g + 8 * h, 8 * nt + 2 * q);
          const uint32_t hi = pack_bf16(dS[nt][2 * h], dS[nt][2 * h + 1]);
          const float2 f = wm::unpack(hi);
          *reinterpret_cast<uint32_t*>(sm.dS[0] + at) = hi;
          *reinterpret_cast<uint32_t*>(sm.dS[1] + at) = pack_bf16(dS[nt][2 * h] - f.x, dS[nt][2 * h + 1] - f.y);
        }
    }
    wm::cp_wait<0>();
    __syncthreads();
    if (c > c0) {
      load(c - 1);
      load_gates(a, gp, t0 - kC, lane, g0, g1);
    }
    const int buf = c & 1;
    const uint32_t Qs = smem_u32(sm.Q[buf]), Ks = smem_u32(sm.K[buf]), Vs = smem_u32(sm.V[buf]), Gs = smem_u32(sm.G[buf]);
    const float* b = sm.b[warp];
    const float bC = b[kC - 1];
    const float br0 = b[row0 + g], br1 = b[row0 + g + 8];
    float x1[8][4];  // dQ, or dK
    float x2[8][4];  // dV (key side)
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x1[nt][e] = x2[nt][e] = 0.f;

    if (query_side) {
      uint32_t ga[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) wm::frag_a(Gs, row0, 16 * ks, lane, ga[ks]);
      // u ⊙ (dO·Sᵀ), with S as two terms.
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t Sa = smem_u32(sm.S[half]);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
          for (int np = 0; np < 4; ++np) {
            uint32_t y[4];
            wm::frag_b(Sa, 16 * np, 16 * ks, lane, y);
            wm::mma(x1[2 * np], ga[ks], y[0], y[1]);
            wm::mma(x1[2 * np + 1], ga[ks], y[2], y[3]);
          }
      }
      const float u0 = a.scale * exp2_fast(br0), u1 = a.scale * exp2_fast(br1);
      float r0 = 0.f, r1 = 0.f, dot = 0.f;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        x1[nt][0] *= u0;
        x1[nt][1] *= u0;
        x1[nt][2] *= u1;
        x1[nt][3] *= u1;
        const uint32_t at0 = swz128_bf16(row0 + g, 8 * nt + 2 * q), at1 = swz128_bf16(row0 + g + 8, 8 * nt + 2 * q);
        const float2 q0 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.Q[buf] + at0));
        const float2 q1 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.Q[buf] + at1));
        r0 = fmaf(q0.x, x1[nt][0], fmaf(q0.y, x1[nt][1], r0));
        r1 = fmaf(q1.x, x1[nt][2], fmaf(q1.y, x1[nt][3], r1));
        const float2 h0 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.S[0] + at0));
        const float2 h1 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.S[0] + at1));
        const float2 l0 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.S[1] + at0));
        const float2 l1 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.S[1] + at1));
        dot = fmaf(h0.x + l0.x, dS[nt][0], fmaf(h0.y + l0.y, dS[nt][1], dot));
        dot = fmaf(h1.x + l1.x, dS[nt][2], fmaf(h1.y + l1.y, dS[nt][3], dot));
      }
      uint32_t qa[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) wm::frag_a(Qs, row0, 16 * ks, lane, qa[ks]);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb > (warp & 3)) break;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t y[4];
          wm::frag_b(Ks, 16 * kb, 16 * ks, lane, y);
          wm::mma(s[0], qa[ks], y[0], y[1]);
          wm::mma(s[1], qa[ks], y[2], y[3]);
          wm::frag_b(Vs, 16 * kb, 16 * ks, lane, y);
          wm::mma(d[0], ga[ks], y[0], y[1]);
          wm::mma(d[1], ga[ks], y[2], y[3]);
        }
        uint32_t pa[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int j = 16 * kb + 8 * nt + 2 * q, i0 = row0 + g;
          const float2 bj = *reinterpret_cast<const float2*>(b + j);
          const float a0 = j <= i0 ? a.scale * d[nt][0] * exp2_fast(br0 - bj.x) : 0.f;
          const float a1 = j + 1 <= i0 ? a.scale * d[nt][1] * exp2_fast(br0 - bj.y) : 0.f;
          const float a2 = j <= i0 + 8 ? a.scale * d[nt][2] * exp2_fast(br1 - bj.x) : 0.f;
          const float a3 = j + 1 <= i0 + 8 ? a.scale * d[nt][3] * exp2_fast(br1 - bj.y) : 0.f;
          r0 += (j < i0 ? a0 * s[nt][0] : 0.f) + (j + 1 < i0 ? a1 * s[nt][1] : 0.f);
          r1 += (j < i0 + 8 ? a2 * s[nt][2] : 0.f) + (j + 1 < i0 + 8 ? a3 * s[nt][3] : 0.f);
          pa[2 * nt] = pack_bf16(a0, a1);
          pa[2 * nt + 1] = pack_bf16(a2, a3);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t y[4];
          wm::frag_b_t(Ks, 16 * kb, 16 * np, lane, y);
          wm::mma(x1[2 * np], pa, y[0], y[1]);
          wm::mma(x1[2 * np + 1], pa, y[2], y[3]);
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        r0 += __shfl_xor_sync(0xffffffffu, r0, o);
        r1 += __shfl_xor_sync(0xffffffffu, r1, o);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (q == 0) {
        sm.rows[row0 + g] = r0;
        sm.rows[row0 + g + 8] = r1;
      }
      const float keep = exp2_fast(bC);
      if (lane == 0) sm.dot[warp] = keep * dot;
      // dS ← e^{b_64}·dS' + (u ⊙ Q)ᵀ·dO.
      float w[16];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * ks + e] = a.scale * exp2_fast(b[16 * ks + 2 * q + (e & 1) + 8 * (e >> 1)]);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) dS[nt][e] *= keep;
      add_outer(dS, Qs, Gs, w, row0, lane);
    } else {
      uint32_t ka[4][4], va[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        wm::frag_a(Ks, row0, 16 * ks, lane, ka[ks]);
        wm::frag_a(Vs, row0, 16 * ks, lane, va[ks]);
      }
      // w ⊙ (V·dS'ᵀ), with dS' as two terms, and w ⊙ (K·dS').
      const uint32_t dSa = smem_u32(sm.dS[0]), dSb = smem_u32(sm.dS[1]);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t y[4];
          wm::frag_b(dSa, 16 * np, 16 * ks, lane, y);
          wm::mma(x1[2 * np], va[ks], y[0], y[1]);
          wm::mma(x1[2 * np + 1], va[ks], y[2], y[3]);
          wm::frag_b(dSb, 16 * np, 16 * ks, lane, y);
          wm::mma(x1[2 * np], va[ks], y[0], y[1]);
          wm::mma(x1[2 * np + 1], va[ks], y[2], y[3]);
          wm::frag_b_t(dSa, 16 * ks, 16 * np, lane, y);
          wm::mma(x2[2 * np], ka[ks], y[0], y[1]);
          wm::mma(x2[2 * np + 1], ka[ks], y[2], y[3]);
        }
      const float w0 = exp2_fast(bC - br0), w1 = exp2_fast(bC - br1);
      float p0 = 0.f, p1 = 0.f, m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        x1[nt][0] *= w0;
        x1[nt][1] *= w0;
        x1[nt][2] *= w1;
        x1[nt][3] *= w1;
        x2[nt][0] *= w0;
        x2[nt][1] *= w0;
        x2[nt][2] *= w1;
        x2[nt][3] *= w1;
        const float2 k0 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.K[buf] + swz128_bf16(row0 + g, 8 * nt + 2 * q)));
        const float2 k1 = wm::unpack(*reinterpret_cast<const uint32_t*>(sm.K[buf] + swz128_bf16(row0 + g + 8, 8 * nt + 2 * q)));
        p0 = fmaf(k0.x, x1[nt][0], fmaf(k0.y, x1[nt][1], p0));
        p1 = fmaf(k1.x, x1[nt][2], fmaf(k1.y, x1[nt][3], p1));
      }
      // Blocks of 16 queries from this warp's own tokens on: rows j (keys), columns i (queries).
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        if (ib < (warp & 3)) continue;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t y[4];
          wm::frag_b(Qs, 16 * ib, 16 * ks, lane, y);
          wm::mma(s[0], ka[ks], y[0], y[1]);
          wm::mma(s[1], ka[ks], y[2], y[3]);
          wm::frag_b(Gs, 16 * ib, 16 * ks, lane, y);
          wm::mma(d[0], va[ks], y[0], y[1]);
          wm::mma(d[1], va[ks], y[2], y[3]);
        }
        uint32_t pa[4], aa[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int i = 16 * ib + 8 * nt + 2 * q, j0 = row0 + g;
          const float2 bq = *reinterpret_cast<const float2*>(b + i);
          const float e0 = i >= j0 ? a.scale * exp2_fast(bq.x - br0) : 0.f;
          const float e1 = i + 1 >= j0 ? a.scale * exp2_fast(bq.y - br0) : 0.f;
          const float e2 = i >= j0 + 8 ? a.scale * exp2_fast(bq.x - br1) : 0.f;
          const float e3 = i + 1 >= j0 + 8 ? a.scale * exp2_fast(bq.y - br1) : 0.f;
          const float a0 = e0 * d[nt][0], a1 = e1 * d[nt][1], a2 = e2 * d[nt][2], a3 = e3 * d[nt][3];
          m0 += (i > j0 ? a0 * s[nt][0] : 0.f) + (i + 1 > j0 ? a1 * s[nt][1] : 0.f);
          m1 += (i > j0 + 8 ? a2 * s[nt][2] : 0.f) + (i + 1 > j0 + 8 ? a3 * s[nt][3] : 0.f);
          aa[2 * nt] = pack_bf16(a0, a1);
          aa[2 * nt + 1] = pack_bf16(a2, a3);
          pa[2 * nt] = pack_bf16(e0 * s[nt][0], e1 * s[nt][1]);
          pa[2 * nt + 1] = pack_bf16(e2 * s[nt][2], e3 * s[nt][3]);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t y[4];
          wm::frag_b_t(Qs, 16 * ib, 16 * np, lane, y);
          wm::mma(x1[2 * np], aa, y[0], y[1]);
          wm::mma(x1[2 * np + 1], aa, y[2], y[3]);
          wm::frag_b_t(Gs, 16 * ib, 16 * np, lane, y);
          wm::mma(x2[2 * np], pa, y[0], y[1]);
          wm::mma(x2[2 * np + 1], pa, y[2], y[3]);
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        p0 += __shfl_xor_sync(0xffffffffu, p0, o);
        p1 += __shfl_xor_sync(0xffffffffu, p1, o);
        m0 += __shfl_xor_sync(0xffffffffu, m0, o);
        m1 += __shfl_xor_sync(0xffffffffu, m1, o);
      }
      if (q == 0) {
        sm.past[row0 + g] = p0;
        sm.past[row0 + g + 8] = p1;
        sm.cols[row0 + g] = m0;
        sm.cols[row0 + g + 8] = m1;
      }
    }
    __syncthreads();  // every tile of this chunk has been read; rows, cols, past and dot are visible
    if (c > c0) {
      load_ckpt(c - 1);
      wm::cp_commit();
    }
    // Gradients out through the tiles just read (this warp's own rows of Q, or of K and V).
    auto put = [&](uint8_t* tile, const float (&x)[8][4], __nv_bfloat16* out) {
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint32_t*>(tile + swz128_bf16(row0 + g + 8 * h, 8 * nt + 2 * q)) =
              pack_bf16(x[nt][2 * h], x[nt][2 * h + 1]);
      __syncwarp();
#pragma unroll
      for (int i = lane; i < 128; i += 32) {
        const int r = row0 + (i >> 3), y = i & 7;
        if (t0 + r < a.T)
          *reinterpret_cast<uint4*>(out + out0 + (t0 + r) * kD + 8 * y) =
              *reinterpret_cast<const uint4*>(tile + r * 128 + ((y ^ (r & 7)) << 4));
      }
    };
    if (query_side) {
      put(sm.Q[buf], x1, a.dq);
    } else {
      put(sm.K[buf], x1, a.dk);
      put(sm.V[buf], x2, a.dv);
    }
    if (warp == 7) {
      // dg over the chunk: sums over the tokens from t on of (rows − cols), sums over those before
      // t of past.
      float s0 = sm.rows[lane] - sm.cols[lane], s1 = sm.rows[lane + 32] - sm.cols[lane + 32];
      const float f0 = sm.past[lane], f1 = sm.past[lane + 32];
      float c0_ = f0, c1_ = f1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y0 = __shfl_down_sync(0xffffffffu, s0, o), y1 = __shfl_down_sync(0xffffffffu, s1, o);
        const float z0 = __shfl_up_sync(0xffffffffu, c0_, o), z1 = __shfl_up_sync(0xffffffffu, c1_, o);
        if (lane + o < 32) {
          s0 += y0;
          s1 += y1;
        }
        if (lane >= o) {
          c0_ += z0;
          c1_ += z1;
        }
      }
      s0 += __shfl_sync(0xffffffffu, s1, 0);
      const float first = __shfl_sync(0xffffffffu, c0_, 31);
      const float all = (sm.dot[0] + sm.dot[1]) + (sm.dot[2] + sm.dot[3]);
      const float d0 = all + s0 + (c0_ - f0), d1 = all + s1 + (first + (c1_ - f1));
      float* dg = a.dg + (size_t)pair * a.T;
      // Where the gate's factor is 0 in fp32 so is its derivative.
      if (t0 + lane < a.T) dg[t0 + lane] = raw0 < kGoneGate ? 0.f : d0;
      if (t0 + lane + 32 < a.T) dg[t0 + lane + 32] = raw1 < kGoneGate ? 0.f : d1;
    }
  }
  if (a.end != nullptr && seg == 0 && query_side) store_state(dS, a.end + (size_t)pair * kState, row0, lane);
}

// ---- one token -----------------------------------------------------------------------------

// S ← e^g·S + kᵀ·v in place, o = scale · q·S: one CTA of 128 threads per (sequence, head), each
// thread four columns of eight rows, all its loads in flight at once.
__global__ void __launch_bounds__(128) k_gs_step(const GsArgs a, float* __restrict__ state) {
  __shared__ float4 part[8][16];
  const int pair = blockIdx.x, cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int64_t bi = pair / a.heads, hi = pair % a.heads;
  float4* S = reinterpret_cast<float4*>(state + (size_t)pair * kState) + cg;
  float4 s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = S[(rg + 8 * i) * 16];
  const __nv_bfloat16* q = a.q.p + bi * a.q.sb + hi * a.q.sh;
  const __nv_bfloat16* k = a.k.p + bi * a.k.sb + hi * a.k.sh;
  const __nv_bfloat16* v = a.v.p + bi * a.v.sb + hi * a.v.sh;
  const float e = expf(a.g[bi * a.gb + hi * a.gh]);
  const uint2 vv = *reinterpret_cast<const uint2*>(v + 4 * cg);
  const float2 v0 = wm::unpack(vv.x), v1 = wm::unpack(vv.y);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float kr = __bfloat162float(k[rg + 8 * i]), qr = a.scale * __bfloat162float(q[rg + 8 * i]);
    s[i].x = fmaf(e, s[i].x, kr * v0.x);
    s[i].y = fmaf(e, s[i].y, kr * v0.y);
    s[i].z = fmaf(e, s[i].z, kr * v1.x);
    s[i].w = fmaf(e, s[i].w, kr * v1.y);
    S[(rg + 8 * i) * 16] = s[i];
    o.x = fmaf(qr, s[i].x, o.x);
    o.y = fmaf(qr, s[i].y, o.y);
    o.z = fmaf(qr, s[i].z, o.z);
    o.w = fmaf(qr, s[i].w, o.w);
  }
  part[rg][cg] = o;
  __syncthreads();
  if (threadIdx.x < 16) {
    float4 t = part[0][cg];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const float4 x = part[i][cg];
      t.x += x.x;
      t.y += x.y;
      t.z += x.z;
      t.w += x.w;
    }
    uint2 y;
    y.x = pack_bf16(t.x, t.y);
    y.y = pack_bf16(t.z, t.w);
    *reinterpret_cast<uint2*>(a.o + bi * a.ob + hi * a.oh + 4 * cg) = y;
  }
}

// ---- host ----------------------------------------------------------------------------------

// Segments of a sequence: as many as fill the GPU (`slots` CTAs at once) when there are fewer
// (sequence, head) pairs than that, each of at least four chunks.
int segments(int64_t pairs, int nchunk, int slots) {
  if (pairs >= slots) return 1;
  const int most = std::max(1, nchunk / 4);
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, slots / pairs));
}

struct Plan {
  int nchunk, nseg, per_seg;
};

Plan plan_for(const ttt_gated_scan_desc* d, int num_sms, int per_sm) {
  Plan p;
  p.nchunk = (int)((d->tokens + kC - 1) / kC);
  p.nseg = segments((int64_t)d->batch * d->heads, p.nchunk, num_sms * per_sm);
  p.per_seg = (p.nchunk + p.nseg - 1) / p.nseg;
  p.nseg = (p.nchunk + p.per_seg - 1) / p.per_seg;  // none empty
  return p;
}

constexpr int kOutPerSm = 3, kBwdPerSm = 2;  // resident CTAs the kernels are built for

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <class K>
ttt_status raise_smem(K* fn, size_t bytes) {
  TTT_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  return TTT_OK;
}

constexpr size_t kStateSmem = sizeof(StateSmem) + 1024, kOutSmem = sizeof(OutSmem) + 1024, kBwdSmem = sizeof(BwdSmem) + 1024;
static_assert(2 * (kBwdSmem + 1024) <= 233472, "two CTAs of k_gs_bwd do not fit an SM");

Rows rows_of(const void* p, const ttt_strides& s) {
  return Rows{static_cast<const __nv_bfloat16*>(p), s.batch, s.head, s.token};
}

GsArgs base_args(const ttt_gated_scan_desc* d, const void* q, const void* k, const void* v, const float* g) {
  GsArgs a = {};
  a.heads = d->heads;
  a.T = d->tokens;
  a.scale = d->scale;
  a.q = rows_of(q, d->q);
  a.k = rows_of(k, d->k);
  a.v = rows_of(v, d->v);
  a.g = g;
  a.gb = d->g.batch;
  a.gh = d->g.head;
  a.gt = d->g.token;
  a.nseg = 1;
  return a;
}

// The states that the segments start from, into a.local (which every later launch reads as start).
template <bool REV>
ttt_status segment_starts(GsArgs a, const float* first, int64_t pairs, cudaStream_t s) {
  a.start = nullptr;
  TTT_TRY(raise_smem(k_gs_state<REV, false>, kStateSmem));
  k_gs_state<REV, false><<<(unsigned)(pairs * a.nseg), 128, kStateSmem, s>>>(a);
  TTT_CUDA(cudaGetLastError());
  k_gs_combine<REV><<<dim3((unsigned)pairs, kState / 4 / 128), 128, 0, s>>>(a.local, a.seg_decay, first, a.nseg);
  TTT_CUDA(cudaGetLastError());
  return TTT_OK;
}

}  // namespace

size_t gated_scan_workspace(const ttt_gated_scan_desc* d, bool backward, int num_sms) {
  const size_t pairs = (size_t)d->batch * d->heads;
  const Plan p = plan_for(d, num_sms, backward ? kBwdPerSm : kOutPerSm);
  const size_t seg = p.nseg > 1 ? round256(pairs * p.nseg * kState * 4) + round256(pairs * p.nseg * 4) : 0;
  return seg + (backward ? round256(pairs * p.nchunk * 2 * kState * 2) : 0);
}

ttt_status gated_scan(const ttt_gated_scan_desc* d, const void* q, const void* k, const void* v, const float* g,
                      const float* S0, void* o, float* S_end, void* ws, int num_sms, cudaStream_t s) {
  const int64_t pairs = (int64_t)d->batch * d->heads;
  const Plan p = plan_for(d, num_sms, kOutPerSm);
  GsArgs a = base_args(d, q, k, v, g);
  a.nchunk = p.nchunk;
  a.nseg = p.nseg;
  a.per_seg = p.per_seg;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.ob = d->o.batch;
  a.oh = d->o.head;
  a.ot = d->o.token;
  a.start = S0;
  if (p.nseg > 1) {
    a.local = static_cast<float*>(ws);
    a.seg_decay = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round256((size_t)pairs * p.nseg * kState * 4));
    TTT_TRY(segment_starts<false>(a, S0, pairs, s));
    a.start = a.local;
  }
  a.end = S_end;
  TTT_TRY(raise_smem(k_gs_out, kOutSmem));
  k_gs_out<<<(unsigned)(pairs * p.nseg), 128, kOutSmem, s>>>(a);
  TTT_CUDA(cudaGetLastError());
  return TTT_OK;
}

ttt_status gated_scan_backward(const ttt_gated_scan_desc* d, const void* dout, const void* q, const void* k,
                               const void* v, const float* g, const float* S0, const float* dS_end, void* dq, void* dk,
                               void* dv, float* dg, float* dS0, void* ws, int num_sms, cudaStream_t s) {
  const int64_t pairs = (int64_t)d->batch * d->heads;
  const Plan p = plan_for(d, num_sms, kBwdPerSm);
  GsArgs a = base_args(d, q, k, v, g);
  a.nchunk = p.nchunk;
  a.nseg = p.nseg;
  a.per_seg = p.per_seg;
  a.dout = rows_of(dout, d->o);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.ckpt = reinterpret_cast<__nv_bfloat16*>(w);
  w += round256((size_t)pairs * p.nchunk * 2 * kState * 2);
  float* local = reinterpret_cast<float*>(w);
  float* decay = reinterpret_cast<float*>(w + round256((size_t)pairs * p.nseg * kState * 4));
  if (p.nseg > 1) {
    a.local = local;
    a.seg_decay = decay;
    TTT_TRY(segment_starts<false>(a, S0, pairs, s));
  }
  // The state before every chunk.
  a.start = p.nseg > 1 ? local : S0;
  a.local = nullptr;
  TTT_TRY(raise_smem(k_gs_state<false, true>, kStateSmem));
  k_gs_state<false, true><<<(unsigned)(pairs * p.nseg), 128, kStateSmem, s>>>(a);
  TTT_CUDA(cudaGetLastError());
  if (p.nseg > 1) {
    a.local = local;
    TTT_TRY(segment_starts<true>(a, dS_end, pairs, s));
    a.local = nullptr;
  }
  a.start = p.nseg > 1 ? local : dS_end;
  a.end = dS0;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.dg = dg;
  TTT_TRY(raise_smem(k_gs_bwd, kBwdSmem));
  k_gs_bwd<<<(unsigned)(pairs * p.nseg), 256, kBwdSmem, s>>>(a);
  TTT_CUDA(cudaGetLastError());
  return TTT_OK;
}

ttt_status gated_scan_step(const ttt_gated_scan_desc* d, const void* q, const void* k, const void* v, const float* g,
                           float* state, void* o, cudaStream_t s) {
  GsArgs a = base_args(d, q, k, v, g);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.ob = d->o.batch;
  a.oh = d->o.head;
  k_gs_step<<<(unsigned)((int64_t)d->batch * d->heads), 128, 0, s>>>(a, state);
  TTT_CUDA(cudaGetLastError());
  return TTT_OK;
}

}  // namespace ttt
