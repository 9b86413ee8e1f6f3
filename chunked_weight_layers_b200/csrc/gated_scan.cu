// Gated linear recurrence on 64 x 64 per-head states: the fast weight with a forget gate and the
// Hebbian update, S_t = e^{g_t}·S_{t-1} + k_tᵀ·v_t, o_t = scale · q_t·S_t, its gradients, and its
// one-token form.
//
// Mathematics. Tokens are taken in chunks of 128. With b_i the sum of the chunk's gates up to and
// with token i, S the state before the chunk and w_j = e^{b_128 - b_j}:
//   O  = scale · [ e^{b_i}·(Q·S)_i + Σ_{j <= i} e^{b_i - b_j}·(q_i·k_j)·v_j ]
//   S' = e^{b_128}·S + (w ⊙ K)ᵀ·V
// so a chunk is four products, and only S goes from chunk to chunk. Backward, with dS' the gradient of
// the state after the chunk and u_i = scale·e^{b_i}:
//   dQ = u ⊙ (dO·Sᵀ) + A·K,      A_ij = scale·e^{b_i - b_j}·(do_i·v_j)  (j <= i)
//   dK = w ⊙ (V·dS'ᵀ) + Aᵀ·Q
//   dV = w ⊙ (K·dS') + Pᵀ·dO,    P_ij = scale·e^{b_i - b_j}·(q_i·k_j)  (j <= i)
//   dS = e^{b_128}·dS' + (u ⊙ Q)ᵀ·dO
//   dg_t = e^{b_128}·<S, dS'> + Σ_{i >= t} q_i·(u_i·S·do_i) + Σ_{j < t} k_j·(w_j·dS'·v_j)
//          + Σ_{i >= t > j} A_ij·(q_i·k_j)
// (the gate of token t scales every path from before t to t or after). Each chunk's dg starts
// from the states, not from the chunk after it, so rounding does not add up along the sequence.
//
// Precision. The products run on the tensor cores (tcgen05) with bf16 operands and fp32 sums. S and
// dS stay in fp32 registers. Where a product's result is a bf16 output, one factor is rounded to bf16
// (P, A, or the copy of S); where it feeds a fp32 output (the states and dg), the factor is kept as a sum of
// three bf16 numbers, which is all of its fp32 value, at the price of as many products: the states come out
// within 3e-7 and dg within 6e-7 in two norms (1.1e-6 for gates of -30), about as from products in fp32 (with two
// numbers 2.5e-6 and 5e-6, and 5 to 7 % less time). The gates are summed in base-2 units; one below -150 (its factor is 0 in
// fp32, as for -inf, which starts a new document) counts as -150, so that differences of sums stay
// finite.
//
// Where there are fewer (sequence, head) pairs than the SMs hold CTAs, the sequence is cut into
// segments: the states that the segments add are found first (k_gs_segment), combined in order, and
// then every segment runs from its own start.
//
// What bounds it (B200): latency, no unit is near its limit (of the time, tensor pipe 17 to 29 %, HBM 26 to 50 %,
// the counters' fullest SM unit 30 to 47 %). Forward: a chunk's chain of scores, their weights, P·V and outputs
// beside that of the state; seven chunks take 26.8 us in a CTA alone on the GPU, 29.0 in one on every SM and
// 41.0 in two, whose TMEM leaves no room for a third. The pass over K and V for the segments' starts and the launches'
// first and last microseconds come on top (8 x 12 heads x 2048 tokens: 18 + 33 us, which overlap to 45, where
// the bytes need 16). Backward: one CTA an SM, whose chunk passes through one set of tiles in shared memory (49 us
// for seven in a CTA alone, 58 in one on every SM); the next chunk's tiles come when its last product has read
// these. 4 x 16 heads x 8192 tokens: 64 us for what the segments add, 49 for the state before every chunk, 207 to 217
// for the rest, where the bytes need 74. The state before every chunk is kept in pieces of eight columns, all rows of
// a piece after each other: a warp then writes whole sectors, where rows of 128 bytes took 15 us more.
#include <algorithm>

#include "f32x2.cuh"
#include "internal.h"
#include "tc_common.cuh"
#include "warp_mma.cuh"

namespace ttt {

namespace {

constexpr int kD = 64;               // head width
constexpr int kTile = kD * 128;      // bytes of a [64][64] bf16 tile
constexpr int kState = kD * kD;      // elements of a state
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinGate = -150.f;   // base-2 units: 2^-150 is 0 in fp32
constexpr float kGoneGate = -104.f;  // a gate below kMinGate / kLog2e

struct Rows {  // bf16 [batch, heads, 64], strides in elements
  const __nv_bfloat16* p;
  int64_t sb, sh;
};

struct GsArgs {
  int heads, nchunk, nseg, per_seg;  // per_seg: chunks of a segment
  int64_t T;
  float scale;
  const float* g;
  int64_t gb, gh, gt;
  const float* start;                 // [pairs][nseg or 1][64][64] states the segments start from, or null (zero)
  float* end;                         // final state [pairs][64][64] (the last segment's), or null
  int few;                            // start holds one state a pair: the CTAs add the segments' on their own
  float* local[2];                    // what each segment adds [pairs][nseg][64][64], forward and in reverse
  float* seg_decay[2];                // sums of the segments' gates, base-2 units [pairs][nseg]
  __nv_bfloat16* ckpt;                // state before every chunk, as three bf16 terms [pairs][nchunk][3][8 pieces][64 rows][8]
  float* dg;                          // dense [pairs][T]
  DevStatus status;
  int stall;                          // a chunk of every segment that is never loaded (tests), or -1
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- states --------------------------------------------------------------------------------

// The states the segments start from, in place of what they add: start[s + 1] =
// 2^decay[s]·start[s] + local[s], from `first` (or zero); in reverse start[s − 1] from start[s]. One element
// a thread, 16 segments' loads in flight. grid (pairs, 64·64 / 128, directions).
__global__ void __launch_bounds__(128) k_gs_combine(const GsArgs a, const float* first_fwd, const float* first_rev) {
  constexpr int kAhead = 16;
  const int at = blockIdx.y * 128 + threadIdx.x, rev = blockIdx.z, nseg = a.nseg;
  const size_t pair = blockIdx.x;
  const float* first = rev ? first_rev : first_fwd;
  float* p = a.local[rev] + pair * nseg * kState + at;
  const float* d = a.seg_decay[rev] + pair * nseg;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = first != nullptr ? first[pair * kState + at] : 0.f;
  for (int i0 = 0; i0 < nseg; i0 += kAhead) {
    float x[kAhead], f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int seg = rev ? nseg - 1 - (i0 + i) : i0 + i;
      const bool in = i0 + i < nseg;
      x[i] = in ? p[(size_t)seg * kState] : 0.f;
      f[i] = in ? d[seg] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int seg = rev ? nseg - 1 - (i0 + i) : i0 + i;
      if (i0 + i < nseg) p[(size_t)seg * kState] = s;
      s = fmaf(exp2_fast(f[i]), s, x[i]);
    }
  }
}

// ---- tensor-core (tcgen05) chunks of 128 tokens ------------------------------------------------

constexpr int kL = 128;                   // tokens per chunk
constexpr int kLTile = kL * 128;          // bytes of a [128][64] bf16 tile with 128-byte rows

// A chunk's gates, made by one warp a chunk ahead. A decay between two tokens is a difference of sums from
// the chunk's start, which gates that both sums hold (150 for each document's start before the two) can make far
// longer than itself; so the sums are made in 64 bits and kept as two fp32 numbers.
struct __align__(16) Gates {
  float b[kL];    // sum from the chunk's start up to and with token t
  float lo[kL];   // what the rounding of b left
  float end[kL];  // 2^(sum of the gates after t to the end of t's block of 32)
  float w[kL];    // 2^(sum of the gates after t to the chunk's end)
  float total;    // sum of all
};

// Asynchronous copy of a chunk's raw gates to shared memory by one warp (zeros past T): they are asked
// for two chunks ahead, and registers that wait for them would be stored away at once.
__device__ __forceinline__ void fetch_gates(const GsArgs& a, const float* gp, int64_t t0, float* raw, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + lane + 32 * i;
    const bool ok = t < a.T;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(raw + lane + 32 * i)), "l"(gp + (ok ? t * a.gt : 0)),
                 "r"(ok ? 4 : 0)
                 : "memory");
  }
  wm::cp_commit();
}

// From the raw gates of the last fetch_gates of this warp, or of the one before (another). Sum: float makes no
// lo, for decays from or to the chunk's ends alone (double cost k_gs_segment 3 us of 18; for k_gs_out, sums as pairs
// of fp32 numbers cost 1 us more than double).
template <class Sum>
__device__ __forceinline__ void make_gates(const float* raw, Gates& s, int lane, bool another = false) {
  if (another)
    wm::cp_wait<1>();
  else
    wm::cp_wait<0>();
  __syncwarp();
  const float4 r = *reinterpret_cast<const float4*>(raw + 4 * lane);
  float x[4] = {r.x, r.y, r.z, r.w};
  Sum pre[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] *= kLog2e;
    x[i] = x[i] < kMinGate ? kMinGate : x[i];  // NaN stays
  }
  pre[0] = x[0];
#pragma unroll
  for (int i = 1; i < 4; ++i) pre[i] = pre[i - 1] + x[i];
  // Inclusive sums over the lanes up to this one, from this one on, and from it to the end of its eight.
  Sum up = pre[3];
  float down = (float)pre[3], seg = down;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum u = __shfl_up_sync(0xffffffffu, up, o);
    const float d = __shfl_down_sync(0xffffffffu, down, o);
    if (lane >= o) up += u;
    if (lane + o < 32) down += d;
    if (o < 8) {
      const float e = __shfl_down_sync(0xffffffffu, seg, o);
      if ((lane & 7) + o < 8) seg += e;
    }
  }
  // The neighbours' sums are those without this lane (a subtraction would cancel).
  Sum base = __shfl_up_sync(0xffffffffu, up, 1);
  float after = __shfl_down_sync(0xffffffffu, down, 1), after8 = __shfl_down_sync(0xffffffffu, seg, 1);
  if (lane == 0) base = 0;
  if (lane == 31) after = 0.f;
  if ((lane & 7) == 7) after8 = 0.f;
  float b[4], lo[4], w[4], e[4], suf = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Sum sum = base + pre[i];
    b[i] = (float)sum;
    if constexpr (sizeof(Sum) == 8) lo[i] = (float)(sum - b[i]);
  }
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    w[i] = exp2_fast(after + suf);
    e[i] = exp2_fast(after8 + suf);
    suf += x[i];
  }
  *reinterpret_cast<float4*>(s.b + 4 * lane) = make_float4(b[0], b[1], b[2], b[3]);
  if constexpr (sizeof(Sum) == 8) *reinterpret_cast<float4*>(s.lo + 4 * lane) = make_float4(lo[0], lo[1], lo[2], lo[3]);
  *reinterpret_cast<float4*>(s.w + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<float4*>(s.end + 4 * lane) = make_float4(e[0], e[1], e[2], e[3]);
  if (lane == 31) s.total = (float)up;
  __syncwarp();  // the raw gates have been read
}

// Two fp32 values as three bf16 terms: each the rounded rest of those before.
__device__ __forceinline__ void terms_of(F2 p, uint32_t& a, uint32_t& b, uint32_t& c) {
  const F2 minus = f2(-1.f, -1.f);
  a = to_bf16(p);
  p = fma2(from_bf16(a), minus, p);
  b = to_bf16(p);
  c = to_bf16(fma2(from_bf16(b), minus, p));
}

// A 16-byte piece of a row, weighted, as three bf16 terms.
__device__ __forceinline__ void weigh(const uint4& x, F2 w, uint4 (&t)[3]) {
  terms_of(mul(from_bf16(x.x), w), t[0].x, t[1].x, t[2].x);
  terms_of(mul(from_bf16(x.y), w), t[0].y, t[1].y, t[2].y);
  terms_of(mul(from_bf16(x.z), w), t[0].z, t[1].z, t[2].z);
  terms_of(mul(from_bf16(x.w), w), t[0].w, t[1].w, t[2].w);
}

using tc::desc_at;
using tc::desc_of;

// XWᵀ·Y over 128 tokens into 64 TMEM columns, XW one of three terms (a tile); the least come first. Both
// operands MN-major. The 64 rows lie in the first 16 lanes of each warp's 32.
__device__ __forceinline__ void outer_mma(uint32_t tmem_d, uint32_t x, uint32_t y, bool first) {
#pragma unroll
  for (int kk = 0; kk < kL / 16; ++kk)
    tc::mma(tmem_d, desc_at(x, kk * 2048), desc_at(y, kk * 2048), tc::idesc_bf16(64, 64, 1, 1), !first || kk != 0);
}

// Of two bf16 values at columns 0 and 1: both where the row is 1 or more, the first where it is 0, none
// before.
__device__ __forceinline__ uint32_t causal(uint32_t pair, int row) {
  uint32_t keep;
  asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(keep) : "r"(max(row + 1, 0) * 16));
  return pair & keep;
}

// All N threads of the CTA, from wherever their halves or groups are.
template <int N>
__device__ __forceinline__ void cta_sync() {
  asm volatile("bar.sync 0, %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// A group of four warps holds a state, half a row a thread as 16 pairs: the row of its TMEM lane in the warp's
// first 16, columns 0 .. 31 in threads 0 .. 15 of the warp and 32 .. 63 in the others.
__device__ __forceinline__ int row_of(int id) { return 16 * (id >> 5) + (id & 15); }
__device__ __forceinline__ int half_of(int id) { return (id >> 4) & 1; }
// Where the thread's half row is in a [64][64] fp32 state.
__device__ __forceinline__ int half_row(int id) { return row_of(id) * kD + 32 * half_of(id); }

// S ← keep·S + what outer_mma left in TMEM (tmem: the warp's lanes).
__device__ __forceinline__ void take_sums(F2 (&S)[16], uint32_t tmem, float keep) {
  const F2 k = f2(keep, keep);
  uint32_t d[32];
  tc::ld_half32(tmem, d);
  tc::wait_ld();
#pragma unroll
  for (int c = 0; c < 16; ++c) S[c] = fma2(k, S[c], f2u(d[2 * c], d[2 * c + 1]));
}

// A half row between registers and global memory (null: zeros).
__device__ __forceinline__ void load_row(F2 (&S)[16], const float* p) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float4 x = p != nullptr ? reinterpret_cast<const float4*>(p)[c] : make_float4(0.f, 0.f, 0.f, 0.f);
    S[2 * c] = f2(x.x, x.y);
    S[2 * c + 1] = f2(x.z, x.w);
  }
}

__device__ __forceinline__ void store_row(const F2 (&S)[16], float* p) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float2 x = split(S[2 * c]), y = split(S[2 * c + 1]);
    reinterpret_cast<float4*>(p)[c] = make_float4(x.x, x.y, y.x, y.y);
  }
}

// The thread's half row of the state that a segment starts from. With few segments: what those before it add
// (REV: those after it), in order, onto the pair's state.
template <bool REV>
__device__ __forceinline__ void load_start(F2 (&S)[16], const GsArgs& a, int pair, int seg, int id) {
  load_row(S, a.start != nullptr ? a.start + (size_t)(a.few ? pair : pair * a.nseg + seg) * kState + half_row(id) : nullptr);
  if (!a.few) return;
  for (int i = REV ? a.nseg - 1 : 0; REV ? i > seg : i < seg; i += REV ? -1 : 1) {
    const size_t at = (size_t)pair * a.nseg + i;
    const float f = exp2_fast(a.seg_decay[REV][at]);
    const F2 ff = f2(f, f);
    const ulonglong2* x = reinterpret_cast<const ulonglong2*>(a.local[REV] + at * kState + half_row(id));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const ulonglong2 y = x[c];
      S[2 * c] = fma2(ff, S[2 * c], F2{y.x});
      S[2 * c + 1] = fma2(ff, S[2 * c + 1], F2{y.y});
    }
  }
}

// Launched beside the end of the launch before it (programmatic dependent launch): until before_results()
// returns, only what was there before that launch may be read, and nothing written. may_follow(): the
// next launch's CTAs may start where there is room.
__device__ __forceinline__ void before_results() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void may_follow() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The thread's half row, rounded to bf16, into a [64][64] tile.
__device__ __forceinline__ void put_state_row(uint8_t* tile, const F2 (&S)[16], int id) {
  const int r = row_of(id);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(tile + r * 128 + (((4 * half_of(id) + c) ^ (r & 7)) << 4)) =
        make_uint4(to_bf16(S[4 * c]), to_bf16(S[4 * c + 1]), to_bf16(S[4 * c + 2]), to_bf16(S[4 * c + 3]));
}

// TMA copies of a [128 tokens][64] tile of one (sequence, head): rows past the last token read as
// zeros and are not written.
__device__ __forceinline__ void tma_load_tile(void* dst, const CUtensorMap* map, uint64_t* bar, int t, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(t), "r"(h), "r"(b)
      : "memory");
}

// Brings the tile into L2.
__device__ __forceinline__ void tma_prefetch_tile(const CUtensorMap* map, int t, int h, int b) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global [%0, {%1, %2, %3, %4}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(0),
               "r"(t), "r"(h), "r"(b)
               : "memory");
}

// The same for consecutive bytes (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_store_tile(const CUtensorMap* map, const void* src, int t, int h, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(0), "r"(t), "r"(h), "r"(b)
               : "memory");
}

// A tensor map of [batch, heads, tokens, 64] rows, and where its (sequence, head) coordinates count (a
// dimension with stride 0 is one element for the map).
struct Tiles {
  CUtensorMap map;
  int head, batch;  // 0 or 1: factors of the coordinates
};

// After a wait that ran out, copies may still be on their way into this CTA's shared memory: 50 us, far
// beyond the latency of a TMA load, before it may exit.
__device__ __forceinline__ void let_land(const volatile int* abort) {
  if (*abort) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 50000) __nanosleep(1000);
  }
}

struct __align__(1024) SegSmem {
  uint8_t X[2][kLTile];  // X; once weighed, the first term of w ⊙ X
  uint8_t Y[2][kLTile];
  uint8_t L[2][kLTile];  // the second and third terms
  Gates gates[4];
  __align__(16) float raw[2][kL];
  uint64_t full[2], ready[2], done[2], gated[4], read[4];
  uint32_t tmem;
  int abort;
};

constexpr int kSegThreads = 320;

// Runs the state alone over a segment. Forward: X = K, Y = V, weights w; in reverse, from the last chunk to
// the first: X = Q, Y = dO, weights scale·2^b. Warps 0 .. 7 weigh half a row of X a thread while the tensor
// cores take the tile before; warps 4 .. 7 then add the sums of the chunk before (two sets of TMEM columns) to
// half a row of the state each. Warp 8 asks for the tiles and issues the products, warp 9 makes the gates: in a
// weighing warp both held up the next chunk's weighing (8 x 12 heads x 2048 tokens: 19.5 us against 17.9). A chunk
// takes some 3000 cycles, of which the 24 products' instructions take 1900 with two CTAs at it. CKPT: writes the
// state before every chunk, as three bf16 planes (forward). grid (pairs · nseg, directions).
struct SegTiles {
  Tiles x[2], y[2];
};

template <bool CKPT>
__global__ void __launch_bounds__(kSegThreads, 2) k_gs_segment(const __grid_constant__ SegTiles tiles, const GsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  SegSmem& sm = *reinterpret_cast<SegSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, id = tid & 127;
  const int pair = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const bool rev = blockIdx.y != 0;
  const Tiles &tx = tiles.x[blockIdx.y], &ty = tiles.y[blockIdx.y];
  may_follow();
  if (!CKPT && seg == (rev ? 0 : a.nseg - 1)) return;  // no segment starts from what this one adds
  const int c0 = seg * a.per_seg, c1 = min(a.nchunk, c0 + a.per_seg), n = c1 - c0;
  auto chunk_of = [&](int i) { return rev ? c1 - 1 - i : c0 + i; };
  const int bi = pair / a.heads, hi_ = pair % a.heads;
  const float* gp = a.g + bi * a.gb + hi_ * a.gh;
  auto load = [&](int i) {
    if (!CKPT && i == a.stall) return;
    uint64_t* bar = &sm.full[i & 1];
    mbar_arrive_expect_tx(bar, 2 * kLTile);
    tma_load_tile(sm.X[i & 1], &tx.map, bar, chunk_of(i) * kL, hi_ * tx.head, bi * tx.batch);
    tma_load_tile(sm.Y[i & 1], &ty.map, bar, chunk_of(i) * kL, hi_ * ty.head, bi * ty.batch);
  };
  if (tid == 256) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.ready[i], 8);  // the weighing warps
      mbar_init(&sm.done[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.gated[i], 1);
      mbar_init(&sm.read[i], 4);
    }
    sm.abort = 0;
    fence_barrier_init();
    load(0);
    if (n > 1) load(1);
  }
  if (warp == 9) fetch_gates(a, gp, (int64_t)chunk_of(0) * kL, sm.raw[0], lane);
  if (warp == 4) tc::alloc(&sm.tmem, 128);
  tc::fence_before();
  cta_sync<kSegThreads>();
  tc::fence_after();
  const uint32_t tm = sm.tmem;
  if (warp == 8) {
    const uint32_t dx = desc_of(sm.X[0]), dl = desc_of(sm.L[0]), dy = desc_of(sm.Y[0]);
    for (int i = 0; i < n; ++i) {
      const int ph = i & 1;
      if (i > 0) {
        mbar_wait(&sm.done[ph ^ 1], ((i - 1) >> 1) & 1, a.status, &sm.abort);
        if (lane == 0 && i + 1 < n) load(i + 1);  // the tiles of the chunk before have been read
        __syncwarp();
      }
      // The chunk is weighed, and the sums two chunks back have been taken. (An mbarrier, whose waits end: at a named
      // barrier, warps that a wait run out has let go ahead would arrive out of turn, and this one wait for good.)
      mbar_wait(&sm.ready[ph], (i >> 1) & 1, a.status, &sm.abort);
      if (lane == 0) {
        tc::fence_after();
        const uint32_t d = tm + 64 * ph, y = dy + ph * (kLTile >> 4);
        outer_mma(d, dl + (kLTile >> 4), y, true);
        outer_mma(d, dl, y, false);
        outer_mma(d, dx + ph * (kLTile >> 4), y, false);
        tc::commit(&sm.done[ph]);
      }
      __syncwarp();
    }
  } else if (warp == 9) {
    for (int i = 0; i < n; ++i) {
      if (i + 1 < n) fetch_gates(a, gp, (int64_t)chunk_of(i + 1) * kL, sm.raw[(i + 1) & 1], lane);
      if (i > 3) mbar_wait(&sm.read[i & 3], ((i >> 2) - 1) & 1, a.status, &sm.abort);
      make_gates<float>(sm.raw[i & 1], sm.gates[i & 3], lane, i + 1 < n);
      if (lane == 0) mbar_arrive(&sm.gated[i & 3]);
    }
  } else {
    // Half a row of chunk i's X: its first term in place, the others beside once the products of the chunk before
    // have read theirs.
    const int first = 4 * (tid >> 7);
    auto weigh_chunk = [&](int i) {
      const int ph = i & 1;
      const Gates& gt = sm.gates[i & 3];
      mbar_wait(&sm.gated[i & 3], (i >> 2) & 1, a.status, &sm.abort);
      const float w = rev ? a.scale * exp2_fast(gt.b[id]) : gt.w[id];
      mbar_wait(&sm.full[ph], (i >> 1) & 1, a.status, &sm.abort);
      uint4 t[4][3];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4* x = reinterpret_cast<uint4*>(sm.X[ph] + id * 128 + (((first + c) ^ (id & 7)) << 4));
        weigh(*x, f2(w, w), t[c]);
        *x = t[c][0];
      }
      if (i > 0) mbar_wait(&sm.done[ph ^ 1], ((i - 1) >> 1) & 1, a.status, &sm.abort);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t at = id * 128 + (((first + c) ^ (id & 7)) << 4);
        *reinterpret_cast<uint4*>(sm.L[0] + at) = t[c][1];
        *reinterpret_cast<uint4*>(sm.L[1] + at) = t[c][2];
      }
      fence_proxy_async_smem();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ready[ph]);
    };
    if (warp < 4) {
      for (int i = 0; i < n; ++i) weigh_chunk(i);
    } else {
      const uint32_t tmem = tm + ((uint32_t)((warp & 3) * 32) << 16);
      F2 S[16];
      if (CKPT) {
        before_results();
        load_start<false>(S, a, pair, seg, id);
      } else {
        load_row(S, nullptr);
      }
      float decay = 0.f;
      for (int i = 0; i <= n; ++i) {
        if (i < n) weigh_chunk(i);
        if (i > 0) {
          const int last = (i - 1) & 1;
          mbar_wait(&sm.done[last], ((i - 1) >> 1) & 1, a.status, &sm.abort);
          tc::fence_after();
          const float total = sm.gates[(i - 1) & 3].total;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.read[(i - 1) & 3]);
          take_sums(S, tmem + 64 * last, exp2_fast(total));
          decay += total;
        }
        if (CKPT && i < n) {
          uint4* p = reinterpret_cast<uint4*>(a.ckpt + ((size_t)pair * a.nchunk + chunk_of(i)) * 3 * kState) + 256 * half_of(id) + row_of(id);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t t[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) terms_of(S[4 * c + e], t[0][e], t[1][e], t[2][e]);
#pragma unroll
            for (int k = 0; k < 3; ++k) p[64 * c + k * (kState / 8)] = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
          }
        }
      }
      if (!CKPT) {
        store_row(S, a.local[rev] + (size_t)blockIdx.x * kState + half_row(id));
        if (id == 0) a.seg_decay[rev][blockIdx.x] = decay;
      }
    }
  }
  tc::fence_before();
  cta_sync<kSegThreads>();
  tc::fence_after();
  if (warp == 4) {
    let_land(&sm.abort);
    __syncwarp();
    tc::dealloc(sm.tmem, 128);
  }
}

struct __align__(1024) OutSmem {
  uint8_t Q[kLTile], K[kLTile];
  uint8_t V[2][kLTile];    // a chunk's V; after its products its outputs on their way out
  uint8_t W[2][kLTile];    // the weighted K's second and third terms; the first takes K's place
  uint8_t S[kTile];        // bf16 copy of the state before the chunk
  Gates gates[2];
  __align__(16) float raw[2][kL];
  uint64_t qk, v[2];             // loads
  uint64_t scores, outs, added;  // Q·Kᵀ and Q·S; P·V; (w ⊙ K)ᵀ·V
  uint32_t tmem;
  int abort;
};

// TMEM columns of k_gs_out: the scores, whose first half P then takes and whose second half P·V; Q·S;
// the state's sums.
constexpr int kColP = 0, kColO = 64, kColQS = 128, kColD = 192, kOutCols = 256;

// 256 threads, two CTAs an SM, so that one's products and loads run under the other's arithmetic.
// Threads 0 .. 127 take a row of the chunk's outputs each: Q·Kᵀ comes from TMEM, is weighted, rounded
// and put back as the first operand of P·V without passing through shared memory. Threads 128 .. 255
// weigh K and carry the state, half a row each: the second and third terms go to buffers of their own and into the
// tensor cores before the scores are done, the first into K's place when they are. Tiles come and go by TMA:
// the next chunk's Q when the scores are done, its K when the state's sums are, V into the other of two buffers.
// grid: pairs · nseg.
__global__ void __launch_bounds__(256, 2)
    k_gs_out(const __grid_constant__ Tiles tq, const __grid_constant__ Tiles tk, const __grid_constant__ Tiles tv,
             const __grid_constant__ Tiles to, const GsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  OutSmem& sm = *reinterpret_cast<OutSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, id = tid & 127;
  const bool rows_side = tid < 128;
  const int pair = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int bi = pair / a.heads, hi_ = pair % a.heads;
  const float* gp = a.g + bi * a.gb + hi_ * a.gh;
  const int c0 = seg * a.per_seg, c1 = min(a.nchunk, c0 + a.per_seg), n = c1 - c0;
  auto load_q = [&](int i) {
    mbar_arrive_expect_tx(&sm.qk, 2 * kLTile);
    tma_load_tile(sm.Q, &tq.map, &sm.qk, (c0 + i) * kL, hi_ * tq.head, bi * tq.batch);
  };
  auto load_k = [&](int i) { tma_load_tile(sm.K, &tk.map, &sm.qk, (c0 + i) * kL, hi_ * tk.head, bi * tk.batch); };
  auto load_v = [&](int i) {
    if (i == a.stall) return;
    mbar_arrive_expect_tx(&sm.v[i & 1], kLTile);
    tma_load_tile(sm.V[i & 1], &tv.map, &sm.v[i & 1], (c0 + i) * kL, hi_ * tv.head, bi * tv.batch);
  };
  if (tid == 128) {
    mbar_init(&sm.qk, 1);
    mbar_init(&sm.v[0], 1);
    mbar_init(&sm.v[1], 1);
    mbar_init(&sm.scores, 1);
    mbar_init(&sm.outs, 1);
    mbar_init(&sm.added, 1);
    sm.abort = 0;
    fence_barrier_init();
    load_q(0);
    load_k(0);
    load_v(0);
  }
  if (warp == 0) tc::alloc(&sm.tmem, kOutCols);
  // The two halves run loops of their own, so that the state's registers are not held through the other
  // half's work; barrier 0 ends each chunk for both.
  if (rows_side) {
    tc::fence_before();
    cta_sync<256>();
    tc::fence_after();
    const uint32_t tm = sm.tmem, tmem = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t dq = desc_of(sm.Q), dk = desc_of(sm.K), dv = desc_of(sm.V[0]), ds = desc_of(sm.S);
    for (int i = 0; i < n; ++i) {
      const int ph = i & 1;
      const Gates& gt = sm.gates[ph];
      if (tid == 0) {
        mbar_wait(&sm.qk, ph, a.status, &sm.abort);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)
          tc::mma(tm, desc_at(dq, kk * 32), desc_at(dk, kk * 32), tc::idesc_bf16(128, 128, 0, 0), kk != 0);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)
          tc::mma(tm + kColQS, desc_at(dq, kk * 32), desc_at(ds, kk * 2048), tc::idesc_bf16(128, 64, 0, 1), kk != 0);
        tc::commit(&sm.scores);
        if (i + 1 < n) {
          bulk_wait_read<0>();  // the outputs two chunks back have left the buffer
          load_v(i + 1);
        }
      }
      __syncwarp();
      const float bi_ = gt.b[id], lo_ = gt.lo[id];
      const float u = a.scale * exp2_fast(bi_);
      mbar_wait(&sm.scores, ph, a.status, &sm.abort);
      tc::fence_after();
      // P over blocks of 32 keys: before this warp's own tokens the decay is a product of the key's to
      // its block's end and the query's from there; in its own block one exponential each; none after.
      uint32_t sc[32], p[16];
      tc::ld32(tmem, sc);
      for (int jb = 0; jb < warp; ++jb) {
        const float f = a.scale * exp2_fast((bi_ - gt.b[32 * jb + 31]) + (lo_ - gt.lo[32 * jb + 31]));
        const F2 ff = f2(f, f);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(gt.end + 32 * jb + 4 * c);
          p[2 * c] = to_bf16(mul(mul(ff, F2{e.x}), f2u(sc[4 * c], sc[4 * c + 1])));
          p[2 * c + 1] = to_bf16(mul(mul(ff, F2{e.y}), f2u(sc[4 * c + 2], sc[4 * c + 3])));
        }
        tc::ld32(tmem + 32 * (jb + 1), sc);
        tc::st16(tmem + kColP + 16 * jb, p);
      }
      {
        const F2 bb = f2(bi_, bi_), ll = f2(lo_, lo_), one = f2(-1.f, -1.f), sl = f2(a.scale, a.scale);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const ulonglong2 bj = *reinterpret_cast<const ulonglong2*>(gt.b + 32 * warp + 4 * c);
          const ulonglong2 lj = *reinterpret_cast<const ulonglong2*>(gt.lo + 32 * warp + 4 * c);
          const float2 x = split(add(fma2(one, F2{bj.x}, bb), fma2(one, F2{lj.x}, ll)));
          const float2 y = split(add(fma2(one, F2{bj.y}, bb), fma2(one, F2{lj.y}, ll)));
          p[2 * c] = causal(to_bf16(mul(mul(sl, f2(exp2_fast(x.x), exp2_fast(x.y))), f2u(sc[4 * c], sc[4 * c + 1]))), lane - 4 * c);
          p[2 * c + 1] =
              causal(to_bf16(mul(mul(sl, f2(exp2_fast(y.x), exp2_fast(y.y))), f2u(sc[4 * c + 2], sc[4 * c + 3]))), lane - 4 * c - 2);
        }
        tc::st16(tmem + kColP + 16 * warp, p);
#pragma unroll
        for (int c = 0; c < 16; ++c) p[c] = 0;
        for (int jb = warp + 1; jb < 4; ++jb) tc::st16(tmem + kColP + 16 * jb, p);
      }
      tc::wait_st();
      tc::fence_before();
      group_sync(1);
      if (tid == 0) {
        tc::fence_after();
        mbar_wait(&sm.v[ph], (i >> 1) & 1, a.status, &sm.abort);
        const uint32_t v = dv + ph * (kLTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kL / 16; ++kk)
          tc::mma_a_tmem(tm + kColO, tm + kColP + 8 * kk, desc_at(v, kk * 2048), tc::idesc_bf16(128, 64, 0, 1), kk != 0);
        tc::commit(&sm.outs);
      }
      __syncwarp();
      mbar_wait(&sm.added, ph, a.status, &sm.abort);
      mbar_wait(&sm.outs, ph, a.status, &sm.abort);  // both products of V are done: its buffer is free
      tc::fence_after();
      uint8_t* row = sm.V[ph] + id * 128;
      const F2 uu = f2(u, u);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t x[32], y[32];
        tc::ld32(tmem + kColO + 32 * half, x);
        tc::ld32(tmem + kColQS + 32 * half, y);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 8 * c + 2 * e;
            w[e] = to_bf16(fma2(uu, f2u(y[j], y[j + 1]), f2u(x[j], x[j + 1])));
          }
          *reinterpret_cast<uint4*>(row + (((4 * half + c) ^ (id & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      tc::fence_before();
      cta_sync<256>();
      tc::fence_after();
      if (tid == 0) {
        tma_store_tile(&to.map, sm.V[ph], (c0 + i) * kL, hi_, bi);
        bulk_commit();
      }
    }
    if (tid == 0) bulk_wait_read<0>();
  } else {
    F2 S[16];
    if (warp == 7) {
      fetch_gates(a, gp, (int64_t)c0 * kL, sm.raw[0], lane);
      make_gates<double>(sm.raw[0], sm.gates[0], lane);
      if (n > 1) fetch_gates(a, gp, (int64_t)(c0 + 1) * kL, sm.raw[1], lane);
    }
    before_results();
    load_start<false>(S, a, pair, seg, id);
    put_state_row(sm.S, S, id);
    fence_proxy_async_smem();
    tc::fence_before();
    cta_sync<256>();
    tc::fence_after();
    const uint32_t tm = sm.tmem, tmem = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t dk = desc_of(sm.K), dv = desc_of(sm.V[0]), dw = desc_of(sm.W[0]);
    for (int i = 0; i < n; ++i) {
      const int ph = i & 1;
      const Gates& gt = sm.gates[ph];
      mbar_wait(&sm.qk, ph, a.status, &sm.abort);
      uint4 top[8];
      {
        const F2 w = f2(gt.w[id], gt.w[id]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t at = id * 128 + ((c ^ (id & 7)) << 4);
          uint4 t[3];
          weigh(*reinterpret_cast<const uint4*>(sm.K + at), w, t);
          top[c] = t[0];
          *reinterpret_cast<uint4*>(sm.W[0] + at) = t[1];
          *reinterpret_cast<uint4*>(sm.W[1] + at) = t[2];
        }
      }
      fence_proxy_async_smem();
      tc::fence_before();
      group_sync(2);
      const uint32_t v = dv + ph * (kLTile >> 4);
      if (id == 0) {
        tc::fence_after();
        mbar_wait(&sm.v[ph], (i >> 1) & 1, a.status, &sm.abort);
        outer_mma(tm + kColD, dw + (kLTile >> 4), v, true);
        outer_mma(tm + kColD, dw, v, false);
      }
      __syncwarp();
      mbar_wait(&sm.scores, ph, a.status, &sm.abort);  // Q, K and the state's copy have been read
      if (id == 0 && i + 1 < n) load_q(i + 1);
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(sm.K + id * 128 + ((c ^ (id & 7)) << 4)) = top[c];
      fence_proxy_async_smem();
      group_sync(2);
      if (id == 0) {
        outer_mma(tm + kColD, dk, v, false);
        tc::commit(&sm.added);
      }
      __syncwarp();
      mbar_wait(&sm.added, ph, a.status, &sm.abort);
      if (id == 0 && i + 1 < n) load_k(i + 1);
      __syncwarp();
      tc::fence_after();
      take_sums(S, tmem + kColD, exp2_fast(gt.total));
      put_state_row(sm.S, S, id);
      if (warp == 7 && i + 1 < n) {
        make_gates<double>(sm.raw[ph ^ 1], sm.gates[ph ^ 1], lane);
        if (i + 2 < n) fetch_gates(a, gp, (int64_t)(c0 + i + 2) * kL, sm.raw[ph], lane);
      }
      fence_proxy_async_smem();
      tc::fence_before();
      cta_sync<256>();
      tc::fence_after();
    }
    if (a.end != nullptr && seg == a.nseg - 1) store_row(S, a.end + (size_t)pair * kState + half_row(id));
  }
  __syncthreads();
  if (warp == 0) {
    let_land(&sm.abort);
    __syncwarp();
    tc::dealloc(sm.tmem, kOutCols);
  }
}

// ---- backward ------------------------------------------------------------------------------

struct __align__(1024) BwdSmem {
  uint8_t Q[kLTile], K[kLTile], V[kLTile], G[kLTile];  // G: dO
  uint8_t S[3][kTile];    // the state before the chunk, three terms, [8 pieces][64 rows][16 bytes] each
  uint8_t dS[2][kTile];   // the gradient of the state after the chunk, first two terms
  uint8_t W[2][kLTile];   // u ⊙ Q, first two terms; then dV and dK on their way out
  uint8_t P[2][kLTile];   // P and A, 128 queries x 128 keys, in halves of 64 keys; P[1]'s first 64 rows, the queries
                          // before its keys, are not read: they hold the third term of dS
  uint8_t A[2][kLTile];
  uint8_t out[kLTile];    // u ⊙ Q, third term; then dQ on its way out
  Gates gates[2];
  __align__(16) float raw[3][kL];
  __align__(16) float rows[2][kL];  // Σ_j A_ij·(q_i·k_j) over j < i, per half of the keys
  __align__(16) float far[kL];      // q_i·(u_i·S·do_i)
  __align__(16) float cols[4][kL];  // Σ_i A_ij·(q_i·k_j) over i > j, per 32 queries
  __align__(16) float past[kL];     // k_j·(w_j·dS'·v_j)
  float dot[4];                     // parts of e^{b_128}·<S, dS'>
  uint64_t in, scores, inter, added, grads, sent;
  uint32_t tmem;
  int abort;
};

// TMEM columns of k_gs_bwd: Q·Kᵀ and dO·Vᵀ, whose place dQ, dV and dK take once they have been read; the
// products with the states; the state's sums.
constexpr int kColSc = 0, kColDp = 128, kColDq = 64, kColDv = 128, kColDk = 192, kColDqi = 256, kColDki = 320, kColDvi = 384,
              kColDs = 448;

// f · (64 columns of TMEM), and its product with row r of a tile.
__device__ __forceinline__ float scaled_row(F2 (&x)[32], uint32_t tmem, float f, const uint8_t* tile, int r) {
  const F2 ff = f2(f, f);
  F2 d = f2(0.f, 0.f);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t y[32];
    tc::ld32(tmem + 32 * half, y);
    tc::wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 t = *reinterpret_cast<const uint4*>(tile + r * 128 + (((4 * half + c) ^ (r & 7)) << 4));
      const uint32_t tw[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 8 * c + 2 * e;
        const F2 z = mul(ff, f2u(y[j], y[j + 1]));
        x[16 * half + 4 * c + e] = z;
        d = fma2(from_bf16(tw[e]), z, d);
      }
    }
  }
  const float2 s = split(d);
  return s.x + s.y;
}

// x + (64 columns of TMEM), rounded, into row r of a tile.
__device__ __forceinline__ void finish_row(const F2 (&x)[32], uint32_t tmem, uint8_t* tile, int r) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t y[32];
    tc::ld32(tmem + 32 * half, y);
    tc::wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = to_bf16(add(x[16 * half + 4 * c + e], f2u(y[8 * c + 2 * e], y[8 * c + 2 * e + 1])));
      *reinterpret_cast<uint4*>(tile + r * 128 + (((4 * half + c) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// dS as three bf16 terms into the tiles.
__device__ __forceinline__ void put_ds(BwdSmem& sm, const F2 (&S)[16], int id) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t at = row_of(id) * 128 + (((4 * half_of(id) + c) ^ (id & 7)) << 4);
    uint32_t t[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) terms_of(S[4 * c + e], t[0][e], t[1][e], t[2][e]);
    *reinterpret_cast<uint4*>(sm.dS[0] + at) = make_uint4(t[0][0], t[0][1], t[0][2], t[0][3]);
    *reinterpret_cast<uint4*>(sm.dS[1] + at) = make_uint4(t[1][0], t[1][1], t[1][2], t[1][3]);
    *reinterpret_cast<uint4*>(sm.P[1] + at) = make_uint4(t[2][0], t[2][1], t[2][2], t[2][3]);
  }
}

// Half a row (16-byte pieces c0 .. c0 + 3) of u ⊙ Q, as three bf16 terms, by groups 2 and 3 together.
__device__ __forceinline__ void weigh_half(BwdSmem& sm, const GsArgs& a, int id, int c0, float u, int ph, bool later) {
  mbar_wait(&sm.in, ph, a.status, &sm.abort);
  if (later) mbar_wait(&sm.sent, ph ^ 1, a.status, &sm.abort);  // the last chunk's gradients have left the buffers
#pragma unroll
  for (int c = c0; c < c0 + 4; ++c) {
    const uint32_t at = id * 128 + ((c ^ (id & 7)) << 4);
    uint4 t[3];
    weigh(*reinterpret_cast<const uint4*>(sm.Q + at), f2(u, u), t);
    *reinterpret_cast<uint4*>(sm.W[0] + at) = t[0];
    *reinterpret_cast<uint4*>(sm.W[1] + at) = t[1];
    *reinterpret_cast<uint4*>(sm.out + at) = t[2];
  }
  fence_proxy_async_smem();
  asm volatile("bar.sync 2, 256;" ::: "memory");
}

struct BwdTiles {
  Tiles q, k, v, g, dq, dk, dv;
};

// Descriptor of a K-major operand as S lies: pieces of 16 bytes of all 64 rows after each other.
__device__ __forceinline__ uint64_t pieces_at(const void* tile, int bytes) {
  constexpr uint64_t high = (uint64_t)((128u >> 4) | (1u << 14)) << 32;  // 128 bytes from eight rows to the next, no swizzle
  return high | (desc_of(tile, kD * 16) + (uint32_t)(bytes >> 4));       // 1024 from piece to piece
}

// From the segment's last chunk to its first: 512 threads in four groups of 128, one CTA an SM; thread
// `id` of a group holds row `id` of what the group reads from TMEM.
//   group 0  the scores of keys 0 .. 63: P, A and their sums; dQ
//   group 1  the same for keys 64 .. 127; dV
//   group 2  weighs Q (half of each row); carries dS, half a row a thread; dg
//   group 3  weighs Q (the other half); dK
// A chunk takes 12 000 cycles, of which the threads' own accesses hold shared memory for 3900 (counted) and the
// products and copies for a part that no counter shows. The next chunk's tiles are asked for when the last product
// has read these, and come while the gradients are rounded and sent out. grid: pairs · nseg.
__global__ void __launch_bounds__(512, 1) k_gs_bwd(const __grid_constant__ BwdTiles tm_, const GsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  BwdSmem& sm = *reinterpret_cast<BwdSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, id = tid & 127, group = tid >> 7;
  const int pair = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int bi = pair / a.heads, hi_ = pair % a.heads;
  const float* gp = a.g + bi * a.gb + hi_ * a.gh;
  const int c0 = seg * a.per_seg, c1 = min(a.nchunk, c0 + a.per_seg), n = c1 - c0;
  const __nv_bfloat16* states = a.ckpt + (size_t)pair * a.nchunk * 3 * kState;
  auto load = [&](int i) {
    if (i == a.stall) return;
    const int t = (c1 - 1 - i) * kL;
    mbar_arrive_expect_tx(&sm.in, 4 * kLTile + 3 * kTile);
    tma_load_tile(sm.Q, &tm_.q.map, &sm.in, t, hi_ * tm_.q.head, bi * tm_.q.batch);
    tma_load_tile(sm.K, &tm_.k.map, &sm.in, t, hi_ * tm_.k.head, bi * tm_.k.batch);
    tma_load_tile(sm.G, &tm_.g.map, &sm.in, t, hi_ * tm_.g.head, bi * tm_.g.batch);
    tma_load_tile(sm.V, &tm_.v.map, &sm.in, t, hi_ * tm_.v.head, bi * tm_.v.batch);
    bulk_load(sm.S, states + (size_t)(c1 - 1 - i) * 3 * kState, 3 * kTile, &sm.in);
  };
  auto prefetch = [&](int i) {
    const int t = (c1 - 1 - i) * kL;
    tma_prefetch_tile(&tm_.q.map, t, hi_ * tm_.q.head, bi * tm_.q.batch);
    tma_prefetch_tile(&tm_.k.map, t, hi_ * tm_.k.head, bi * tm_.k.batch);
    tma_prefetch_tile(&tm_.g.map, t, hi_ * tm_.g.head, bi * tm_.g.batch);
    tma_prefetch_tile(&tm_.v.map, t, hi_ * tm_.v.head, bi * tm_.v.batch);
    bulk_prefetch(states + (size_t)(c1 - 1 - i) * 3 * kState, 3 * kTile);
  };
  if (tid == 0) {
    mbar_init(&sm.in, 1);
    mbar_init(&sm.scores, 1);
    mbar_init(&sm.inter, 1);
    mbar_init(&sm.added, 1);
    mbar_init(&sm.grads, 1);
    mbar_init(&sm.sent, 3);
    sm.abort = 0;
    fence_barrier_init();
    before_results();  // the states before the chunks
    load(0);
  }
  if (warp == 4) tc::alloc(&sm.tmem, 512);
  // Keys after a query's block of 32 never get a score: zero once.
  for (int i = tid; i < 2 * kLTile / 16; i += 512) {
    if (i < kLTile / 16 || i >= (kLTile + kTile) / 16) reinterpret_cast<uint4*>(sm.P[0])[i] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(sm.A[0])[i] = make_uint4(0, 0, 0, 0);
  }
  for (int i = tid; i < 4 * kL; i += 512) (&sm.cols[0][0])[i] = 0.f;
  for (int i = tid; i < 2 * kL; i += 512) (&sm.rows[0][0])[i] = 0.f;
  // Group 2 runs a loop of its own, so that dS's registers are not held through the others' work; barrier
  // 0 joins all groups twice a chunk.
  if (group == 2) {
    F2 S[16];  // half a row of dS
    before_results();
    load_start<true>(S, a, pair, seg, id);
    put_ds(sm, S, id);
    if (warp == 11) {
      fetch_gates(a, gp, (int64_t)(c1 - 1) * kL, sm.raw[0], lane);
      make_gates<double>(sm.raw[0], sm.gates[0], lane);
      if (n > 1) fetch_gates(a, gp, (int64_t)(c1 - 2) * kL, sm.raw[1], lane);
    }
    fence_proxy_async_smem();
    tc::fence_before();
    cta_sync<512>();
    tc::fence_after();
    const uint32_t tm = sm.tmem, tmem = tm + ((uint32_t)((warp & 3) * 32) << 16);
    for (int i = 0; i < n; ++i) {
      const int ph = i & 1, chunk = c1 - 1 - i;
      const Gates& gt = sm.gates[ph];
      // The next chunk's tiles have no room here yet: they come to L2 meanwhile (loaded from HBM when this
      // chunk is done they took 6500 cycles of the chunk's 12000, all SMs asking at once).
      if (id == 32 && i + 1 < n) prefetch(i + 1);
      __syncwarp();
      weigh_half(sm, a, id, 0, a.scale * exp2_fast(gt.b[id]), ph, i > 0);
      if (id == 0) {
        outer_mma(tm + kColDs, desc_of(sm.out), desc_of(sm.G), true);
        outer_mma(tm + kColDs, desc_of(sm.W[1]), desc_of(sm.G), false);
        outer_mma(tm + kColDs, desc_of(sm.W[0]), desc_of(sm.G), false);
        tc::commit(&sm.added);
      }
      __syncwarp();
      const float keep = exp2_fast(gt.total);
      F2 d = f2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t at = (64 * (4 * half_of(id) + c) + row_of(id)) * 16;
        const uint4 x = *reinterpret_cast<const uint4*>(sm.S[0] + at), y = *reinterpret_cast<const uint4*>(sm.S[1] + at),
                    z = *reinterpret_cast<const uint4*>(sm.S[2] + at);
        d = fma2(S[4 * c], add(from_bf16(x.x), add(from_bf16(y.x), from_bf16(z.x))), d);
        d = fma2(S[4 * c + 1], add(from_bf16(x.y), add(from_bf16(y.y), from_bf16(z.y))), d);
        d = fma2(S[4 * c + 2], add(from_bf16(x.z), add(from_bf16(y.z), from_bf16(z.z))), d);
        d = fma2(S[4 * c + 3], add(from_bf16(x.w), add(from_bf16(y.w), from_bf16(z.w))), d);
      }
      const float2 dd = split(d);
      float dot = dd.x + dd.y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (lane == 0) sm.dot[warp & 3] = keep * dot;
      mbar_wait(&sm.added, ph, a.status, &sm.abort);
      tc::fence_after();
      take_sums(S, tmem + kColDs, keep);
      mbar_wait(&sm.inter, ph, a.status, &sm.abort);  // dS' has been read
      put_ds(sm, S, id);
      fence_proxy_async_smem();
      if (warp == 11 && i + 1 < n) {
        make_gates<double>(sm.raw[(i + 1) % 3], sm.gates[ph ^ 1], lane);
        if (i + 2 < n) fetch_gates(a, gp, (int64_t)(chunk - 2) * kL, sm.raw[(i + 2) % 3], lane);
      }
      tc::fence_before();
      cta_sync<512>();
      tc::fence_after();
      if (warp == 8) {
        // dg over the chunk, four tokens a lane: sums over the tokens from t on of (rows − cols), sums over
        // those before t of past.
        float4 s = *reinterpret_cast<const float4*>(sm.rows[0] + 4 * lane);
        const float4 s1 = *reinterpret_cast<const float4*>(sm.rows[1] + 4 * lane), f = *reinterpret_cast<const float4*>(sm.far + 4 * lane),
                     p = *reinterpret_cast<const float4*>(sm.past + 4 * lane), raw = *reinterpret_cast<const float4*>(sm.raw[i % 3] + 4 * lane);
        s.x += s1.x + f.x, s.y += s1.y + f.y, s.z += s1.z + f.z, s.w += s1.w + f.w;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 c = *reinterpret_cast<const float4*>(sm.cols[q] + 4 * lane);
          s.x -= c.x, s.y -= c.y, s.z -= c.z, s.w -= c.w;
        }
        s.z += s.w, s.y += s.z, s.x += s.y;
        float after = s.x, before = (p.x + p.y) + (p.z + p.w);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, after, o), z = __shfl_up_sync(0xffffffffu, before, o);
          if (lane + o < 32) after += y;
          if (lane >= o) before += z;
        }
        after = __shfl_down_sync(0xffffffffu, after, 1);
        before = __shfl_up_sync(0xffffffffu, before, 1);
        const float all = (sm.dot[0] + sm.dot[1]) + (sm.dot[2] + sm.dot[3]);
        const float base = all + (lane == 31 ? 0.f : after) + (lane == 0 ? 0.f : before);
        const float v[4] = {base + s.x, base + s.y + p.x, base + s.z + (p.x + p.y), base + s.w + (p.x + p.y + p.z)};
        const float g[4] = {raw.x, raw.y, raw.z, raw.w};
        const int64_t t0 = (int64_t)chunk * kL + 4 * lane;
        float* dg = a.dg + (size_t)pair * a.T + t0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (t0 + q < a.T) dg[q] = g[q] < kGoneGate ? 0.f : v[q];  // where the gate's factor is 0 in fp32 so is its derivative
      }
      tc::fence_before();
      cta_sync<512>();
      tc::fence_after();
    }
    if (a.end != nullptr && seg == 0) store_row(S, a.end + (size_t)pair * kState + half_row(id));
  } else {
    fence_proxy_async_smem();
    tc::fence_before();
    cta_sync<512>();
    tc::fence_after();
    const uint32_t tm = sm.tmem, tmem = tm + ((uint32_t)((warp & 3) * 32) << 16);
    for (int i = 0; i < n; ++i) {
      const int ph = i & 1, chunk = c1 - 1 - i;
      const Gates& gt = sm.gates[ph];
      const float mine = gt.b[id];
      if (i > 0 && id == 32) {
        bulk_wait_read<0>();  // the last chunk's gradient has left the buffer
        mbar_arrive(&sm.sent);
      }
      if (group < 2) {
        // Warp 4 has no scores to weigh (its queries come before group 1's keys): it issues the products,
        // which holds it for as long as they run.
        if (tid == 128) {
          const uint32_t dq = desc_of(sm.Q), dk = desc_of(sm.K), dv = desc_of(sm.V), dg = desc_of(sm.G),
                         dd = desc_of(sm.dS[0]), d3 = desc_of(sm.P[1]);
          mbar_wait(&sm.in, ph, a.status, &sm.abort);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc::mma(tm + kColSc, desc_at(dq, kk * 32), desc_at(dk, kk * 32), tc::idesc_bf16(128, 128, 0, 0), kk != 0);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc::mma(tm + kColDp, desc_at(dg, kk * 32), desc_at(dv, kk * 32), tc::idesc_bf16(128, 128, 0, 0), kk != 0);
          tc::commit(&sm.scores);
#pragma unroll
          for (int kk = 0; kk < 12; ++kk)
            tc::mma(tm + kColDqi, desc_at(dg, (kk & 3) * 32), pieces_at(sm.S, kk * 2048), tc::idesc_bf16(128, 64, 0, 0), kk != 0);
#pragma unroll
          for (int kk = 0; kk < 12; ++kk)
            tc::mma(tm + kColDki, desc_at(dv, (kk & 3) * 32), kk < 8 ? desc_at(dd, (kk >> 2) * kTile + (kk & 3) * 32) : desc_at(d3, (kk & 3) * 32),
                    tc::idesc_bf16(128, 64, 0, 0), kk != 0);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc::mma(tm + kColDvi, desc_at(dk, kk * 32), desc_at(dd, kk * 2048), tc::idesc_bf16(128, 64, 0, 1), kk != 0);
          tc::commit(&sm.inter);
        }
        __syncwarp();
        // Blocks of 32 keys up to this warp's own 32 queries (before them the decay is a product of the
        // key's to its block's end and the query's from there), 16 keys at a time as matrix fragments: a
        // lane holds four queries and four keys, so a key's sum over the warp's queries takes four
        // exchanges for 16 keys, where whole rows in a lane would take 16.
        const int w = warp & 3, fg = lane >> 2, fq = lane & 3;
        float br[4], lr[4];
        F2 sum[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          br[r] = gt.b[32 * w + 8 * r + fg];
          lr[r] = gt.lo[32 * w + 8 * r + fg];
          sum[r] = f2(0.f, 0.f);
        }
        mbar_wait(&sm.scores, ph, a.status, &sm.abort);
        tc::fence_after();
        const uint32_t row = 32 * w + (lane & 15), Pt = smem_u32(sm.P[group]), At = smem_u32(sm.A[group]);
#pragma unroll 1
        for (int blk = 0; blk < 2; ++blk) {
          const int jb = 2 * group + blk;
          if (jb > w) break;
          uint32_t s[2][2][8], d[2][2][8];  // [16 keys][16 queries]
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tc::ld_frag16(tmem + ((uint32_t)(16 * h) << 16) + kColSc + 32 * jb + 16 * sub, s[sub][h]);
              tc::ld_frag16(tmem + ((uint32_t)(16 * h) << 16) + kColDp + 32 * jb + 16 * sub, d[sub][h]);
            }
          F2 dec[2][2][4];  // the decays, scaled: [16 keys][8 keys][queries]
          // A token's own pair would drop out of dg, being in its row's and its column's sum alike, but only up to
          // rounding: its decay is 1, and in a head that forgets fast the pairs that dg is made of are lost beside it
          // (gates of -12: dg off by 4e-2, without the own pairs 7e-7).
          const bool own_first = jb == w && fg == 2 * fq, own_second = jb == w && fg == 2 * fq + 1;
          if (jb < w) {
            const float end = gt.b[32 * jb + 31], lend = gt.lo[32 * jb + 31];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float f = a.scale * exp2_fast((br[r] - end) + (lr[r] - lend));
#pragma unroll
              for (int c = 0; c < 4; ++c)
                dec[c >> 1][c & 1][r] = mul(f2(f, f), *reinterpret_cast<const F2*>(gt.end + 32 * jb + 8 * c + 2 * fq));
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 b = *reinterpret_cast<const float2*>(gt.b + 32 * jb + 8 * c + 2 * fq);
              const float2 lo = *reinterpret_cast<const float2*>(gt.lo + 32 * jb + 8 * c + 2 * fq);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int own = 8 * (r - c) + fg - 2 * fq;  // the query's place after the pair's first key
                dec[c >> 1][c & 1][r] = f2(own >= 0 ? a.scale * exp2_fast((br[r] - b.x) + (lr[r] - lo.x)) : 0.f,
                                           own > 0 ? a.scale * exp2_fast((br[r] - b.y) + (lr[r] - lo.y)) : 0.f);
              }
            }
          }
          tc::wait_ld();
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            F2 col[2];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                uint32_t* sp = &s[sub][r >> 1][4 * n + 2 * (r & 1)];
                uint32_t* dp = &d[sub][r >> 1][4 * n + 2 * (r & 1)];
                const F2 sc = f2u(sp[0], sp[1]), at = mul(dec[sub][n][r], f2u(dp[0], dp[1]));
                sp[0] = to_bf16(mul(dec[sub][n][r], sc));
                dp[0] = to_bf16(at);
                F2 m = mul(at, sc);
                if (r == 2 * sub + n) {  // the eight queries and the eight keys are the same tokens
                  const float2 f = split(m);
                  m = f2(own_first ? 0.f : f.x, own_second ? 0.f : f.y);
                }
                sum[r] = add(sum[r], m);
                col[n] = r == 0 ? m : add(col[n], m);
              }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t at = (row + 16 * h) * 128 + (((4 * blk + 2 * sub + (lane >> 4)) ^ (row & 7)) << 4);
              wm::stsm(Pt + at, s[sub][h][0], s[sub][h][2], s[sub][h][4], s[sub][h][6]);
              wm::stsm(At + at, d[sub][h][0], d[sub][h][2], d[sub][h][4], d[sub][h][6]);
            }
            // Halves of the four keys to halves of the lanes, twice, and the last two added up.
            const float2 c0 = split(col[0]), c1 = split(col[1]);
            const bool up = (lane & 16) != 0, odd = (lane & 8) != 0;
            const float x = (up ? c1.x : c0.x) + __shfl_xor_sync(0xffffffffu, up ? c0.x : c1.x, 16);
            const float y = (up ? c1.y : c0.y) + __shfl_xor_sync(0xffffffffu, up ? c0.y : c1.y, 16);
            float z = (odd ? y : x) + __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
            z += __shfl_xor_sync(0xffffffffu, z, 4);
            if ((lane & 4) == 0) sm.cols[w][32 * jb + 16 * sub + (up ? 8 : 0) + 2 * fq + (odd ? 1 : 0)] = z;
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float2 f = split(sum[r]);
          float x = f.x + f.y;
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          if (fq == 0) sm.rows[group][32 * w + 8 * r + fg] = x;
        }
        fence_proxy_async_smem();
        tc::fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tid == 128) {
          tc::fence_after();
          // The first 64 queries have no part in the gradients of keys 64 .. 127: A's zeros there stand in for P's.
          const uint32_t dp = desc_of(sm.P[0], kLTile), dp_early = desc_of(sm.P[0], 3 * kLTile), da = desc_of(sm.A[0], kLTile), dak = desc_of(sm.A[0]), dq = desc_of(sm.Q),
                         dk = desc_of(sm.K), dg = desc_of(sm.G);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma(tm + kColDq, desc_at(dak, (kk >> 2) * kLTile + (kk & 3) * 32), desc_at(dk, kk * 2048), tc::idesc_bf16(128, 64, 0, 1), kk != 0);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma(tm + kColDv, desc_at(kk < 4 ? dp_early : dp, kk * 2048), desc_at(dg, kk * 2048), tc::idesc_bf16(128, 64, 1, 1), kk != 0);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma(tm + kColDk, desc_at(da, kk * 2048), desc_at(dq, kk * 2048), tc::idesc_bf16(128, 64, 1, 1), kk != 0);
          tc::commit(&sm.grads);
        }
        __syncwarp();
      } else {
        weigh_half(sm, a, id, 4, a.scale * exp2_fast(mine), ph, i > 0);
      }
      mbar_wait(&sm.in, ph, a.status, &sm.abort);  // this thread reads Q or K itself
      mbar_wait(&sm.inter, ph, a.status, &sm.abort);
      tc::fence_after();
      F2 x[32];  // the gradient's part from beyond the chunk
      const float dot = scaled_row(x, tmem + (group == 0 ? kColDqi : group == 1 ? kColDvi : kColDki),
                                   group == 0 ? a.scale * exp2_fast(mine) : gt.w[id], group == 0 ? sm.Q : sm.K, id);
      if (group == 0) {
        sm.far[id] = dot;
      }
      if (group == 3) sm.past[id] = dot;
      tc::fence_before();
      cta_sync<512>();  // the chunk's tiles have been read but by the products still running
      tc::fence_after();
      mbar_wait(&sm.grads, ph, a.status, &sm.abort);
      tc::fence_after();
      if (tid == 128 && i + 1 < n) load(i + 1);
      __syncwarp();
      uint8_t* stage = group == 0 ? sm.out : group == 1 ? sm.W[0] : sm.W[1];
      finish_row(x, tmem + (group == 0 ? kColDq : group == 1 ? kColDv : kColDk), stage, id);
      fence_proxy_async_smem();
      group_sync(4 + group);
      if (id == 32) {
        tma_store_tile(group == 0 ? &tm_.dq.map : group == 1 ? &tm_.dv.map : &tm_.dk.map, stage, chunk * kL, hi_, bi);
        bulk_commit();
      }
      tc::fence_before();
      cta_sync<512>();
      tc::fence_after();
    }
    if (id == 32) bulk_wait_read<0>();
  }
  __syncthreads();
  if (warp == 4) {
    let_land(&sm.abort);
    __syncwarp();
    tc::dealloc(sm.tmem, 512);
  }
}

// ---- one token -----------------------------------------------------------------------------

// S ← e^g·S + kᵀ·v in place, o = scale · q·S: one CTA of 128 threads per (sequence, head), each
// thread four columns of eight rows, all its loads in flight at once. Bound by the states' bytes: 64 x 16
// heads, 5.0 us for 34 MB (some of it from L2).
struct StepArgs {
  Rows q, k, v;
  const float* g;
  int64_t gb, gh;
  __nv_bfloat16* o;
  int64_t ob, oh;
  int heads;
  float scale;
};

__global__ void __launch_bounds__(128) k_gs_step(const StepArgs a, float* __restrict__ state) {
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
// (sequence, head) pairs than that, each of at least four chunks. A whole round of CTAs more costs nearly what a
// full one does, and this rule does not look at it: 148, 149 and 296 pairs of 8192 tokens take 219, 254 and 319
// us, 297 take 464; backward, whose main kernel holds one CTA an SM, 638, 848, 1043 and 1330. The same sequences
// cut otherwise (before the states had three terms): 96 pairs of 2048 tokens 44.8, 47.6, 41.0 (taken) and 52.8 us
// with one to four segments; 4 pairs of 65511 76, 60 and 58 with 37, 64 and 74 (taken); backward 64 pairs of 8192
// 300, 342, 304 (taken), 339 and 335 with 2, 3, 4, 5 and 8.
int segments(int64_t pairs, int nchunk, int slots) {
  if (pairs >= slots) return 1;
  const int most = std::max(1, nchunk / 4);
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, slots / pairs));
}

constexpr int kPerSm = 2;  // resident CTAs of k_gs_segment and k_gs_out, which the plan fills

struct Plan {
  int nchunk, nseg, per_seg;
};

Plan plan_for(const ttt_gated_scan_desc* d, int num_sms) {
  Plan p;
  p.nchunk = (int)((d->tokens + kL - 1) / kL);
  p.nseg = segments((int64_t)d->batch * d->heads, p.nchunk, num_sms * kPerSm);
  p.per_seg = (p.nchunk + p.nseg - 1) / p.nseg;
  p.nseg = (p.nchunk + p.per_seg - 1) / p.per_seg;  // none empty
  return p;
}


// Up to so many segments the outputs' CTAs add up the states before theirs on their own (16 KB each from
// L2), which saves a launch of some 8 us; beyond it one launch combines them in order.
constexpr int kFewSegments = 8;

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <class K>
ttt_status raise_smem(K* fn, size_t bytes) {
  TTT_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  return TTT_OK;
}

constexpr size_t kSegSmem = sizeof(SegSmem) + 1024, kOutSmem = sizeof(OutSmem) + 1024, kBwdSmem = sizeof(BwdSmem) + 1024;
static_assert(kBwdSmem <= 232448, "k_gs_bwd exceeds the 227 KB of shared memory per block");
static_assert(2 * (kOutSmem + 1024) <= 233472, "two CTAs of k_gs_out do not fit an SM");
static_assert(2 * (kSegSmem + 1024) <= 233472, "two CTAs of k_gs_segment do not fit an SM");

// Launches fn so that it may start beside the end of the launch before it on the stream.
template <class... P, class... A>
ttt_status launch_after(void (*fn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  TTT_CUDA(cudaLaunchKernelEx(&cfg, fn, args...));
  return TTT_OK;
}

Rows rows_of(const void* p, const ttt_strides& s) {
  return Rows{static_cast<const __nv_bfloat16*>(p), s.batch, s.head};
}

GsArgs base_args(const ttt_gated_scan_desc* d, const float* g) {
  GsArgs a = {};
  a.heads = d->heads;
  a.T = d->tokens;
  a.scale = d->scale;
  a.g = g;
  a.gb = d->g.batch;
  a.gh = d->g.head;
  a.gt = d->g.token;
  a.nseg = 1;
  return a;
}

}  // namespace

size_t gated_scan_workspace(const ttt_gated_scan_desc* d, bool backward, int num_sms) {
  const size_t pairs = (size_t)d->batch * d->heads;
  const Plan p = plan_for(d, num_sms);
  const size_t seg = p.nseg > 1 ? 2 * (round256(pairs * p.nseg * kState * 4) + round256(pairs * p.nseg * 4)) : 0;
  return (backward ? seg : seg / 2) + (backward ? round256(pairs * p.nchunk * 3 * kState * 2) : 0);
}

// The tensor map of [batch, heads, tokens, 64] rows in tiles of 128 tokens.
static ttt_status tiles_of(Tiles* t, const void* p, const ttt_strides& s, const ttt_gated_scan_desc* d) {
  const uint64_t n[3] = {(uint64_t)d->tokens, (uint64_t)d->heads, (uint64_t)d->batch};
  const int64_t st[3] = {s.token, s.head, s.batch};
  uint64_t dims[4] = {kD, 1, 1, 1}, strides[3];
  for (int i = 0; i < 3; ++i) {
    // A stride of 0 (one row for all) is a dimension of one element; its stride is then never used.
    const bool one = st[i] == 0;
    dims[i + 1] = one ? 1 : n[i];
    strides[i] = one ? kD * 2 : (uint64_t)st[i] * 2;
    if (strides[i] >= ((uint64_t)1 << 40)) return fail(TTT_ERR_UNSUPPORTED, "a stride of 2^39 elements or more");
  }
  t->head = s.head != 0;
  t->batch = s.batch != 0;
  const uint32_t box[4] = {kD, kL, 1, 1};
  return encode_tmap(&t->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

ttt_status gated_scan(const ttt_gated_scan_desc* d, const void* q, const void* k, const void* v, const float* g,
                      const float* S0, void* o, float* S_end, void* ws, const DevStatus& status, int num_sms,
                      cudaStream_t s) {
  const int64_t pairs = (int64_t)d->batch * d->heads;
  const Plan p = plan_for(d, num_sms);
  GsArgs a = base_args(d, g);
  a.nchunk = p.nchunk;
  a.nseg = p.nseg;
  a.per_seg = p.per_seg;
  a.status = status;
  a.stall = op_stall(p.per_seg > 1);
  a.start = S0;
  a.end = S_end;
  Tiles tq, tk, tv, to;
  TTT_TRY(tiles_of(&tq, q, d->q, d));
  TTT_TRY(tiles_of(&tk, k, d->k, d));
  TTT_TRY(tiles_of(&tv, v, d->v, d));
  TTT_TRY(tiles_of(&to, o, d->o, d));
  TTT_TRY(raise_smem(k_gs_out, kOutSmem));
  const dim3 grid((unsigned)(pairs * p.nseg));
  if (p.nseg == 1) {
    k_gs_out<<<grid, 256, kOutSmem, s>>>(tq, tk, tv, to, a);
    TTT_CUDA(cudaGetLastError());
    return TTT_OK;
  }
  a.local[0] = static_cast<float*>(ws);
  a.seg_decay[0] = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round256((size_t)pairs * p.nseg * kState * 4));
  SegTiles t = {{tk, tk}, {tv, tv}};
  TTT_TRY(raise_smem(k_gs_segment<false>, kSegSmem));
  k_gs_segment<false><<<grid, kSegThreads, kSegSmem, s>>>(t, a);
  TTT_CUDA(cudaGetLastError());
  // The last segment may write S_end before others have read S0: then not on their own.
  a.few = p.nseg <= kFewSegments && S_end != S0;
  if (!a.few) {
    TTT_TRY(launch_after(k_gs_combine, dim3((unsigned)pairs, kState / 128, 1), 128, 0, s, a, S0, S0));
    a.start = a.local[0];
  }
  return launch_after(k_gs_out, grid, 256, kOutSmem, s, tq, tk, tv, to, a);
}

ttt_status gated_scan_backward(const ttt_gated_scan_desc* d, const void* dout, const void* q, const void* k,
                               const void* v, const float* g, const float* S0, const float* dS_end, void* dq, void* dk,
                               void* dv, float* dg, float* dS0, void* ws, const DevStatus& status, int num_sms,
                               cudaStream_t s) {
  const int64_t pairs = (int64_t)d->batch * d->heads;
  const Plan p = plan_for(d, num_sms);
  GsArgs a = base_args(d, g);
  a.nchunk = p.nchunk;
  a.nseg = p.nseg;
  a.per_seg = p.per_seg;
  a.status = status;
  a.stall = op_stall(p.per_seg > 1);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.ckpt = reinterpret_cast<__nv_bfloat16*>(w);
  w += round256((size_t)pairs * p.nchunk * 3 * kState * 2);
  const size_t local_bytes = round256((size_t)pairs * p.nseg * kState * 4), decay_bytes = round256((size_t)pairs * p.nseg * 4);
  for (int i = 0; i < 2; ++i) {
    a.local[i] = reinterpret_cast<float*>(w + i * (local_bytes + decay_bytes));
    a.seg_decay[i] = reinterpret_cast<float*>(w + i * (local_bytes + decay_bytes) + local_bytes);
  }
  BwdTiles t;
  TTT_TRY(tiles_of(&t.q, q, d->q, d));
  TTT_TRY(tiles_of(&t.k, k, d->k, d));
  TTT_TRY(tiles_of(&t.v, v, d->v, d));
  TTT_TRY(tiles_of(&t.g, dout, d->o, d));
  const ttt_strides dense = {(int64_t)d->heads * d->tokens * kD, d->tokens * kD, kD};
  TTT_TRY(tiles_of(&t.dq, dq, dense, d));
  TTT_TRY(tiles_of(&t.dk, dk, dense, d));
  TTT_TRY(tiles_of(&t.dv, dv, dense, d));
  const dim3 grid((unsigned)(pairs * p.nseg));
  TTT_TRY(raise_smem(k_gs_segment<false>, kSegSmem));
  TTT_TRY(raise_smem(k_gs_segment<true>, kSegSmem));
  TTT_TRY(raise_smem(k_gs_bwd, kBwdSmem));
  const SegTiles both = {{t.k, t.q}, {t.v, t.g}};
  a.start = S0;
  if (p.nseg > 1) {
    // What the segments add in both directions at once.
    k_gs_segment<false><<<dim3(grid.x, 2), kSegThreads, kSegSmem, s>>>(both, a);
    TTT_CUDA(cudaGetLastError());
    a.few = p.nseg <= kFewSegments && dS0 != dS_end;
    if (!a.few) {
      TTT_TRY(launch_after(k_gs_combine, dim3((unsigned)pairs, kState / 128, 2), 128, 0, s, a, S0, dS_end));
      a.start = a.local[0];
    }
    // The state before every chunk.
    TTT_TRY(launch_after(k_gs_segment<true>, grid, kSegThreads, kSegSmem, s, both, a));
  } else {
    k_gs_segment<true><<<grid, kSegThreads, kSegSmem, s>>>(both, a);
    TTT_CUDA(cudaGetLastError());
  }
  a.start = p.nseg > 1 && !a.few ? a.local[1] : dS_end;
  a.end = dS0;
  a.dg = dg;
  return launch_after(k_gs_bwd, grid, 512, kBwdSmem, s, t, a);
}

ttt_status gated_scan_step(const ttt_gated_scan_desc* d, const void* q, const void* k, const void* v, const float* g,
                           float* state, void* o, cudaStream_t s) {
  const StepArgs a = {rows_of(q, d->q), rows_of(k, d->k), rows_of(v, d->v), g, d->g.batch, d->g.head, static_cast<__nv_bfloat16*>(o),
                      d->o.batch, d->o.head, d->heads, d->scale};
  k_gs_step<<<(unsigned)((int64_t)d->batch * d->heads), 128, 0, s>>>(a, state);
  TTT_CUDA(cudaGetLastError());
  return TTT_OK;
}

}  // namespace ttt
