// Norm of each query and key head with the rotary position in the same pass, and its gradients.
//
// Mathematics. For one head's row x of width D: n = x·r with r = (Σx²/D + ε)^-1/2 (RMS), (Σx² +
// ε)^-1/2 (L2) or 1; y = w ⊙ n (gain w, RMS only); the first `rot` values are then rotated in
// pairs by the angle position · freq_i, magnitude m: (y1, y2) → m·(y1·cos − y2·sin, y2·cos + y1·sin).
// A pair is (i, i + rot/2) (half layout) or (2i, 2i + 1) (interleaved). Backward: the rotation
// turned back gives dy; dw = Σ dy ⊙ n over all rows; with e = w ⊙ dy, dx = r·(e − n·c·Σ e·n), c = 1/D
// (RMS), 1 (L2), 0 (none).
//
// What bounds it: HBM, each row read once and written once. A group of 8, 16 or 32 lanes takes one
// token and walks over its heads with 16-byte loads, eight values a lane, so the cosines and sines
// of the token are computed once, in the lanes that use them, and kept in registers: no table is
// read and no position is out of its range. The angle is reduced in 64 bits (turns = position ·
// freq / 2π less the nearest whole number: off by 2^-53 of the turns, where 32 bits would be
// off by 0.004 turns at position 100000), then sine and cosine in 32 bits. All sums are fp32;
// outputs are rounded once. The gains' gradients are summed per CTA, then over the CTAs in a
// second launch in a fixed order (no atomics: the same bits every time).
//
// Measured (B200; the copy rate is 6.45 TB/s): 8 x 2048 tokens of 24 heads of 64: 22 us, 4.5 TB/s; 32768
// tokens of 40 heads of 128, half of each rotated: 126 us, 5.3 TB/s. Backward, 4 x 8192 tokens of 32 heads of
// 64 with the gains' gradients: 85 us, 4.7 TB/s (two CTAs an SM for its registers, so fewer loads in flight).
// 32 tokens of 32 heads: 4 us, nearly all of it the launch's. In fp32 the three take 49 (4.2 TB/s), 279 (4.8) and,
// backward, 141 us (5.7). The registers of four CTAs an SM (two backward) leave some on the stack: 76 to 84
// bytes a thread in bf16 forward, 154 to 188 in fp32 both ways; none in bf16 backward.
#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"

namespace ttt {

namespace {

constexpr int kThreadsQK = 256;

struct QkSide {
  const void* x;   // rows, strides in elements
  const void* dy;  // backward: gradients of the outputs
  void* y;         // outputs, or gradients of the inputs
  int64_t xb, xh, xt, yb, yh, yt, gb, gh, gt;  // x, y and dy
  const float* w;
  int heads;
};

struct QkArgs {
  QkSide side[2];
  int width, rot, norm;
  float eps, magnitude;
  int64_t tokens, items;  // items: batch · tokens · splits
  int splits, heads_per;  // a token's heads in `splits` parts of heads_per
  const int64_t* positions;
  int64_t position0, positions_stride;
  const double* freqs;
  float* partial;  // backward: [CTAs][2][width]
};

// The kernels were bound by instruction issue (185 a row and warp with scalar arithmetic, 34 us over 8
// x 2048 tokens of 24 heads of 64, where the bytes need 16), so all of a row's arithmetic is in
// pairs.

// Eight values of a row as they lie in memory, and as four pairs. partner(): the eight values that
// are rotated with this lane's: the other lane's, or the same with each pair swapped.
template <class T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  template <bool HALF>
  __device__ __forceinline__ void partner(F2 (&v)[4], bool in, int lane) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x = HALF ? __shfl_sync(0xffffffffu, w[i], lane) : w[i];
      x = in ? x : 0u;  // the coefficient there is 0, and 0 times an infinity is NaN
      const float lo = __uint_as_float(x << 16), hi = __uint_as_float(x & 0xffff0000u);
      v[i] = HALF ? f2(lo, hi) : f2(hi, lo);
    }
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const F2 (&v)[4]) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = split(v[i]);
      o[i] = pack_bf16(f.x, f.y);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
  }
};
template <>
struct Raw<float> {
  float w[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.f;
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(w[2 * i], w[2 * i + 1]);
  }
  template <bool HALF>
  __device__ __forceinline__ void partner(F2 (&v)[4], bool in, int lane) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = HALF ? __shfl_sync(0xffffffffu, w[2 * i], lane) : w[2 * i + 1];
      float y = HALF ? __shfl_sync(0xffffffffu, w[2 * i + 1], lane) : w[2 * i];
      v[i] = f2(in ? x : 0.f, in ? y : 0.f);
    }
  }
  __device__ __forceinline__ static void store(float* p, const F2 (&v)[4]) {
    const float2 a = split(v[0]), b = split(v[1]), c = split(v[2]), d = split(v[3]);
    reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
  }
};

__device__ __forceinline__ float sum_of_squares(const F2 (&v)[4]) {
  F2 s = mul(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(v[i], v[i], s);
  const float2 f = split(s);
  return f.x + f.y;
}

// Sum over the group of L lanes.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A lane's rotation: its value i becomes own[i]·value + other[i]·partner. Lanes past the rotated part
// hold own = 1 and other = 0.
struct Turn {
  F2 own[4], other[4];
  bool in;
  int partner;  // half layout: the lane of the other values of the pairs
};

// BACK: turned back (the sines' sign).
template <bool HALF, bool BACK>
__device__ __forceinline__ Turn make_turn(const QkArgs& a, int64_t pos, int lane_in, int lane) {
  Turn t;
  const int lanes_rot = a.rot / 8, half = a.rot / 16;
  const bool in = lane_in < lanes_rot;
  const bool first = lane_in < half;
  t.in = in;
  t.partner = HALF && in ? lane + (first ? half : -half) : lane;
  // Half layout: both lanes of a pair of lanes need the same eight angles; each makes four of them.
  const int at = HALF ? 8 * (first ? lane_in : lane_in - half) + (first ? 0 : 4) : 4 * lane_in;
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
    if (in) {
      double turns = (double)pos * (a.freqs[at + i] * 0.15915494309189533577);
      turns -= rint(turns);
      sincospif(2.f * (float)turns, &s[i], &c[i]);
      c[i] *= a.magnitude;
      s[i] *= BACK ? -a.magnitude : a.magnitude;
    }
  }
  if constexpr (HALF) {
    const float sign = first ? -1.f : 1.f;
    float cc[8], ss[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float co = __shfl_sync(0xffffffffu, c[i], t.partner), so = __shfl_sync(0xffffffffu, s[i], t.partner);
      cc[i] = first ? c[i] : co;
      ss[i] = sign * (first ? s[i] : so);
      cc[i + 4] = first ? co : c[i];
      ss[i + 4] = sign * (first ? so : s[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.own[i] = f2(cc[2 * i], cc[2 * i + 1]);
      t.other[i] = f2(ss[2 * i], ss[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.own[i] = f2(c[i], c[i]);
      t.other[i] = f2(-s[i], s[i]);
    }
  }
  return t;
}

// The group's token and its part of the heads.
template <int L>
struct Item {
  int64_t b, t;
  int h0, h1;
  bool valid;
  __device__ __forceinline__ Item(const QkArgs& a, int64_t item) {
    valid = item < a.items;
    const int64_t rows = a.items / a.splits, i = valid ? item : 0;
    const int64_t row = i % rows;
    const int part = (int)(i / rows);
    b = row / a.tokens;
    t = row % a.tokens;
    h0 = part * a.heads_per;
    h1 = valid ? min(a.side[0].heads + a.side[1].heads, h0 + a.heads_per) : h0;
  }
};

// A group walks over its part of the heads in batches of one side, with the loads of a batch in
// flight at once: four heads forward, four (of two rows each) backward. The first batch is on its way
// while the angles are made.
constexpr int kFly = 4, kFlyBack = 4;

// One side's heads of the item, and the batches that the longest walk in the warp takes (all lanes
// take part in the shuffles).
template <int FLY>
struct Walk {
  int h0, h1, n;
  template <int L>
  __device__ __forceinline__ Walk(const QkArgs& a, const Item<L>& it, int sd) {
    const int base = sd ? a.side[0].heads : 0;
    h0 = max(it.h0 - base, 0);
    h1 = min(it.h1 - base, a.side[sd].heads);
    n = __reduce_max_sync(0xffffffffu, max(0, h1 - h0 + FLY - 1) / FLY);
  }
};

// The gains of a lane's eight values (1 without).
__device__ __forceinline__ void load_gain(const QkSide& S, bool live, int lane_in, Raw<float>& w) {
  if (S.w != nullptr && live) {
    w.load(S.w + 8 * lane_in);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w.w[j] = 1.f;
  }
}

// grid: items / groups per CTA. y = r·(own·w·x + other·w'·x'), x' and w' the partner's.
template <class T, int L, bool HALF>
__global__ void __launch_bounds__(kThreadsQK, 4) k_qk_norm_rope(const QkArgs a) {
  const int lane = threadIdx.x & 31, lane_in = threadIdx.x % L;
  const Item<L> it(a, (int64_t)blockIdx.x * (kThreadsQK / L) + threadIdx.x / L);
  const bool live = it.valid && 8 * lane_in < a.width;
  const float inv = a.norm == TTT_NORM_RMS ? 1.f / a.width : 1.f;
  const int64_t pos = !it.valid ? 0 : a.positions != nullptr ? a.positions[it.b * a.positions_stride + it.t] : a.position0 + it.t;
  Turn turn;
  bool made = false;
#pragma unroll 1
  for (int sd = 0; sd < 2; ++sd) {
    const Walk<kFly> wk(a, it, sd);
    if (wk.n == 0) continue;
    const QkSide& S = a.side[sd];
    const T* x = static_cast<const T*>(S.x) + it.b * S.xb + it.t * S.xt + 8 * lane_in + wk.h0 * S.xh;
    T* y = static_cast<T*>(S.y) + it.b * S.yb + it.t * S.yt + 8 * lane_in + wk.h0 * S.yh;
    int left = live ? wk.h1 - wk.h0 : 0;
    Raw<T> raw[kFly];
    auto fetch = [&](int n) {
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        if (u < n)
          raw[u].load(x + u * S.xh);
        else
          raw[u].zero();
      }
      x += kFly * S.xh;
    };
    fetch(left);
    if (!made) {
      turn = make_turn<HALF, false>(a, pos, lane_in, lane);
      made = true;
    }
    F2 A[4], B[4];
    {
      Raw<float> w;
      F2 own[4], other[4];
      load_gain(S, live, lane_in, w);
      w.get(own);
      w.template partner<HALF>(other, true, turn.partner);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        A[i] = mul(turn.own[i], own[i]);
        B[i] = mul(turn.other[i], other[i]);
      }
    }
#pragma unroll 1
    for (int b = 0; b < wk.n; ++b) {
      F2 v[kFly][4];
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        F2 p[4], q[4];
        raw[u].get(p);
        raw[u].template partner<HALF>(q, turn.in, turn.partner);
        float r = 1.f;
        if (a.norm != TTT_NORM_NONE) r = rsqrtf(fmaf(group_sum<L>(sum_of_squares(p)), inv, a.eps));
        const F2 rr = f2(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = mul(rr, fma2(q[i], B[i], mul(p[i], A[i])));
        if (u < left) Raw<T>::store(y + u * S.yh, v[u]);
      }
      y += kFly * S.yh;
      left -= kFly;
      if (b + 1 < wk.n) fetch(left);
    }
  }
}

// The gradients of the inputs, and the gains' gradients summed over what the CTA takes. Grid-stride
// over the items.
template <class T, int L, bool HALF>
__global__ void __launch_bounds__(kThreadsQK, 2) k_qk_norm_rope_bwd(const QkArgs a) {
  constexpr int kGroups = kThreadsQK / L;
  __shared__ float part[kGroups][8 * L];
  const int lane = threadIdx.x & 31, lane_in = threadIdx.x % L, group = threadIdx.x / L;
  const float inv = a.norm == TTT_NORM_RMS ? 1.f / a.width : 1.f;
  F2 dw[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[0][i] = dw[1][i] = f2(0.f, 0.f);
  const int64_t step = (int64_t)gridDim.x * kGroups;
  for (int64_t at = (int64_t)blockIdx.x * kGroups; at < a.items; at += step) {
    const Item<L> it(a, at + group);
    const bool live = it.valid && 8 * lane_in < a.width;
    const int64_t pos = !it.valid ? 0 : a.positions != nullptr ? a.positions[it.b * a.positions_stride + it.t] : a.position0 + it.t;
    Turn turn;
    bool made = false;
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) {
      const Walk<kFlyBack> wk(a, it, sd);
      if (wk.n == 0) continue;
      const QkSide& S = a.side[sd];
      const T* x = static_cast<const T*>(S.x) + it.b * S.xb + it.t * S.xt + 8 * lane_in + wk.h0 * S.xh;
      const T* g = static_cast<const T*>(S.dy) + it.b * S.gb + it.t * S.gt + 8 * lane_in + wk.h0 * S.gh;
      T* y = static_cast<T*>(S.y) + it.b * S.yb + it.t * S.yt + 8 * lane_in + wk.h0 * S.yh;
      int left = live ? wk.h1 - wk.h0 : 0;
      Raw<T> gr[kFlyBack], xr[kFlyBack];
      auto fetch = [&](int n) {
#pragma unroll
        for (int u = 0; u < kFlyBack; ++u) {
          if (u < n)
            gr[u].load(g + u * S.gh);
          else
            gr[u].zero();
          if (u < n && a.norm != TTT_NORM_NONE)
            xr[u].load(x + u * S.xh);
          else
            xr[u].zero();
        }
        g += kFlyBack * S.gh;
        x += kFlyBack * S.xh;
      };
      fetch(left);
      if (!made) {
        turn = make_turn<HALF, true>(a, pos, lane_in, lane);
        made = true;
      }
      F2 w[4];
      {
        Raw<float> wr;
        load_gain(S, live, lane_in, wr);
        wr.get(w);
      }
#pragma unroll 1
      for (int b = 0; b < wk.n; ++b) {
#pragma unroll
        for (int u = 0; u < kFlyBack; ++u) {
          F2 e[4], o[4];
          gr[u].get(e);
          gr[u].template partner<HALF>(o, turn.in, turn.partner);
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = fma2(o[i], turn.other[i], mul(e[i], turn.own[i]));
          if (a.norm != TTT_NORM_NONE) {
            F2 n[4];
            xr[u].get(n);
            const float size = fmaf(group_sum<L>(sum_of_squares(n)), inv, a.eps);
            const float r = u < left ? rsqrtf(size) : 0.f;  // a slot past the heads adds nothing
            const F2 rr = f2(r, r);
            F2 d = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              n[i] = mul(n[i], rr);
              dw[sd][i] = fma2(e[i], n[i], dw[sd][i]);
              e[i] = mul(e[i], w[i]);
              d = fma2(e[i], n[i], d);
            }
            const float2 ds = split(d);
            const float dot = -group_sum<L>(ds.x + ds.y) * inv;
            const F2 dd = f2(dot, dot);
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = mul(rr, fma2(dd, n[i], e[i]));
          }
          if (u < left) Raw<T>::store(y + u * S.yh, e);
        }
        y += kFlyBack * S.yh;
        left -= kFlyBack;
        if (b + 1 < wk.n) fetch(left);
      }
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int sd = 0; sd < 2; ++sd) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = split(dw[sd][i]);
      part[group][8 * lane_in + 2 * i] = f.x;
      part[group][8 * lane_in + 2 * i + 1] = f.y;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.width; j += kThreadsQK) {
      float s = 0.f;
#pragma unroll 8
      for (int gi = 0; gi < kGroups; ++gi) s += part[gi][j];
      a.partial[((size_t)blockIdx.x * 2 + sd) * a.width + j] = s;
    }
  }
}

// Sums over the CTAs: one CTA of 128 threads per value, grid (width, 2).
__global__ void __launch_bounds__(128) k_qk_gain_sum(const float* __restrict__ partial, int n, int width, float* dwq, float* dwk) {
  const int j = blockIdx.x, sd = blockIdx.y;
  float* out = sd ? dwk : dwq;
  if (out == nullptr) return;
  __shared__ double warp_sum[4];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 128) s += (double)partial[((size_t)i * 2 + sd) * width + j];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[j] = (float)((warp_sum[0] + warp_sum[1]) + (warp_sum[2] + warp_sum[3]));
}

template <class T, int L, bool HALF>
void launch(const QkArgs& a, bool back, int blocks, cudaStream_t s) {
  if (back)
    k_qk_norm_rope_bwd<T, L, HALF><<<blocks, kThreadsQK, 0, s>>>(a);
  else
    k_qk_norm_rope<T, L, HALF><<<blocks, kThreadsQK, 0, s>>>(a);
}

template <class T, int L>
void launch(const QkArgs& a, bool half, bool back, int blocks, cudaStream_t s) {
  if (half)
    launch<T, L, true>(a, back, blocks, s);
  else
    launch<T, L, false>(a, back, blocks, s);
}

template <class T>
void launch(const QkArgs& a, int L, bool half, bool back, int blocks, cudaStream_t s) {
  if (L == 8)
    launch<T, 8>(a, half, back, blocks, s);
  else if (L == 16)
    launch<T, 16>(a, half, back, blocks, s);
  else
    launch<T, 32>(a, half, back, blocks, s);
}

int lanes_of(int width) { return width <= 64 ? 8 : width <= 128 ? 16 : 32; }

int64_t groups_per_block(int width) { return kThreadsQK / lanes_of(width); }

// Resident CTAs of the backward kernel (its registers allow two).
constexpr int kBwdCtasPerSm = 2;

// Parts of a token's heads: one, unless the tokens alone give the GPU fewer than 512 threads an SM.
// Backward, where CTAs walk over several items each, two parts of six heads or more if that saves half a
// round out of five or fewer: 4 x 8192 tokens (four rounds, or seven of half the size) of 12, 16, 24, 32 and 48
// heads of 64 take 46.6, 49.6, 67.0, 83.2 and 122.6 us in two, 48.9, 51.9, 71.1, 89.4 and 128.7 in one, 10000 of
// 32 heads 37.0 against 43.3, 21000 of 24 heads of 128 (five rounds) 85.7 against 89.3. Two are slower over more
// rounds (60000 tokens, seven: 16 heads of 64 83.8 against 81.1; 146000, 16: 193 against 186), with as many
// (2 x 4096 tokens of 16 heads of 128: 31.5 against 30.3) and with few heads (30000 tokens of 8 of 128: 54.7
// against 50.5).
int splits_of(const ttt_qk_desc* d, bool back, int num_sms) {
  const int64_t rows = (int64_t)d->batch * d->tokens, heads = (int64_t)d->q_heads + d->k_heads;
  const int64_t want = (int64_t)num_sms * 512 / lanes_of(d->width);
  const int64_t splits = std::max<int64_t>(1, std::min(heads, want / std::max<int64_t>(1, rows)));
  if (!back || splits > 1 || heads < 12) return (int)splits;
  const int64_t round = groups_per_block(d->width) * num_sms * kBwdCtasPerSm;
  const int64_t one = (rows + round - 1) / round, two = (2 * rows + round - 1) / round;
  return one <= 5 && two < 2 * one ? 2 : 1;
}

int64_t bwd_blocks(int64_t items, int width, int num_sms) {
  const int64_t g = groups_per_block(width);
  return std::max<int64_t>(1, std::min<int64_t>((items + g - 1) / g, (int64_t)num_sms * kBwdCtasPerSm));
}

QkSide side_of(const void* x, const ttt_strides& xs, const void* dy, const ttt_strides& gs, void* y, const ttt_strides& ys,
               const float* w, int heads) {
  return QkSide{x, dy, y, xs.batch, xs.head, xs.token, ys.batch, ys.head, ys.token, gs.batch, gs.head, gs.token, w, heads};
}

QkArgs args_of(const ttt_qk_desc* d, bool back, const int64_t* positions, const double* freqs, int num_sms) {
  QkArgs a = {};
  a.width = d->width;
  a.rot = d->rot;
  a.norm = d->norm;
  a.eps = d->eps;
  a.magnitude = d->magnitude;
  a.tokens = d->tokens;
  const int heads = d->q_heads + d->k_heads;
  const int splits = splits_of(d, back, num_sms);
  a.heads_per = (heads + splits - 1) / splits;
  a.splits = (heads + a.heads_per - 1) / a.heads_per;
  a.items = (int64_t)d->batch * d->tokens * a.splits;
  a.positions = positions;
  a.position0 = d->position0;
  a.positions_stride = d->positions_stride;
  a.freqs = freqs;
  return a;
}

void run(const QkArgs& a, const ttt_qk_desc* d, bool back, int64_t blocks, cudaStream_t s) {
  const bool half = d->layout == TTT_ROPE_HALF;
  if (d->io_dtype == TTT_F32)
    launch<float>(a, lanes_of(d->width), half, back, (int)blocks, s);
  else
    launch<__nv_bfloat16>(a, lanes_of(d->width), half, back, (int)blocks, s);
}

}  // namespace

size_t qk_norm_rope_workspace(const ttt_qk_desc* d, int num_sms) {
  return (size_t)num_sms * kBwdCtasPerSm * 2 * d->width * sizeof(float);
}

ttt_status qk_norm_rope(const ttt_qk_desc* d, const void* q, const void* k, const float* qw, const float* kw,
                        const int64_t* positions, const double* freqs, void* qo, void* ko, int num_sms, cudaStream_t s) {
  QkArgs a = args_of(d, false, positions, freqs, num_sms);
  a.side[0] = side_of(q, d->q, nullptr, d->q, qo, d->q_out, qw, d->q_heads);
  a.side[1] = side_of(k, d->k, nullptr, d->k, ko, d->k_out, kw, d->k_heads);
  const int64_t g = groups_per_block(d->width), blocks = (a.items + g - 1) / g;
  if (blocks > 0x7fffffff) return fail(TTT_ERR_UNSUPPORTED, "too many tokens for one call");
  run(a, d, false, blocks, s);
  TTT_CUDA(cudaGetLastError());
  return TTT_OK;
}

ttt_status qk_norm_rope_backward(const ttt_qk_desc* d, const void* dqo, const void* dko, const void* q, const void* k,
                                 const float* qw, const float* kw, const int64_t* positions, const double* freqs, void* dq,
                                 void* dk, float* dqw, float* dkw, void* ws, int num_sms, cudaStream_t s) {
  QkArgs a = args_of(d, true, positions, freqs, num_sms);
  a.side[0] = side_of(q, d->q, dqo, d->q_out, dq, d->q_grad, qw, d->q_heads);
  a.side[1] = side_of(k, d->k, dko, d->k_out, dk, d->k_grad, kw, d->k_heads);
  const bool gains = dqw != nullptr || dkw != nullptr;
  a.partial = gains ? static_cast<float*>(ws) : nullptr;
  const int64_t blocks = bwd_blocks(a.items, d->width, num_sms);
  run(a, d, true, blocks, s);
  TTT_CUDA(cudaGetLastError());
  if (gains) {
    k_qk_gain_sum<<<dim3(d->width, 2), 128, 0, s>>>(a.partial, (int)blocks, d->width, dqw, dkw);
    TTT_CUDA(cudaGetLastError());
  }
  return TTT_OK;
}

}  // namespace ttt
