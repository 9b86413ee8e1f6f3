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
#include <algorithm>

#include "common.cuh"
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

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the group of L lanes.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A lane's rotation: half layout, cosine and sine of its eight values; interleaved, of its four
// pairs. Lanes past the rotated part hold the identity.
struct Turn {
  float c[8], s[8];
  bool in;      // whether this lane's values are rotated
  int partner;  // half layout: the lane of the other values of the pairs
  float sign;   // half layout: −1 in the lanes of the pairs' first values, +1 in the others
};

template <bool HALF>
__device__ __forceinline__ Turn make_turn(const QkArgs& a, int64_t pos, int lane_in, int lane) {
  Turn t;
  const int lanes_rot = a.rot / 8, half = a.rot / 16;
  const bool in = lane_in < lanes_rot;
  const bool first = lane_in < half;
  t.in = in;
  t.partner = HALF && in ? lane + (first ? half : -half) : lane;
  t.sign = first ? -1.f : 1.f;
#pragma unroll
  for (int i = 0; i < (HALF ? 8 : 4); ++i) {
    t.c[i] = 1.f;
    t.s[i] = 0.f;
    if (in) {
      const int at = HALF ? 8 * (first ? lane_in : lane_in - half) + i : 4 * lane_in + i;
      double turns = (double)pos * (a.freqs[at] * 0.15915494309189533577);
      turns -= rint(turns);
      float sn, cs;
      sincospif(2.f * (float)turns, &sn, &cs);
      t.c[i] = cs * a.magnitude;
      t.s[i] = sn * a.magnitude;
    }
  }
  return t;
}

// Rotates a lane's eight values; BACK turns the rotation back. Every lane of the warp takes part.
template <bool HALF, bool BACK>
__device__ __forceinline__ void rotate(float (&v)[8], const Turn& t) {
  if constexpr (HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, v[i], t.partner);
      if (t.in) v[i] = fmaf(v[i], t.c[i], other * (BACK ? -t.sign : t.sign) * t.s[i]);
    }
  } else if (t.in) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1], s = BACK ? -t.s[i] : t.s[i];
      v[2 * i] = fmaf(x, t.c[i], -(y * s));
      v[2 * i + 1] = fmaf(y, t.c[i], x * s);
    }
  }
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

// grid: items / groups per CTA.
template <class T, int L, bool HALF>
__global__ void __launch_bounds__(kThreadsQK) k_qk_norm_rope(const QkArgs a) {
  const int lane = threadIdx.x & 31, lane_in = threadIdx.x % L;
  const Item<L> it(a, (int64_t)blockIdx.x * (kThreadsQK / L) + threadIdx.x / L);
  const int64_t pos = !it.valid ? 0 : a.positions != nullptr ? a.positions[it.b * a.positions_stride + it.t] : a.position0 + it.t;
  const Turn turn = make_turn<HALF>(a, pos, lane_in, lane);
  const bool live = it.valid && 8 * lane_in < a.width;
  const float inv = a.norm == TTT_NORM_RMS ? 1.f / a.width : 1.f;
  float w[8];
  int wside = -1;
  // The trip count is the same for every group of the warp: all its lanes take part in the shuffles.
  for (int i = 0; i < a.heads_per; ++i) {
    const int h = it.h0 + i;
    const bool ok = live && h < it.h1;
    const int sd = h >= a.side[0].heads ? 1 : 0;
    const QkSide& S = a.side[sd];
    const int64_t hh = h - (sd ? a.side[0].heads : 0);
    float v[8];
    if (ok) {
      load8<T>(static_cast<const T*>(S.x) + it.b * S.xb + hh * S.xh + it.t * S.xt + 8 * lane_in, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    if (a.norm != TTT_NORM_NONE) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
      const float r = rsqrtf(fmaf(group_sum<L>(ss), inv, a.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= r;
      if (S.w != nullptr && ok) {
        if (wside != sd) {
          load8<float>(S.w + 8 * lane_in, w);
          wside = sd;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= w[j];
      }
    }
    rotate<HALF, false>(v, turn);
    if (ok) store8<T>(static_cast<T*>(S.y) + it.b * S.yb + hh * S.yh + it.t * S.yt + 8 * lane_in, v);
  }
}

// The gradients of the inputs, and the gains' gradients summed over what the CTA takes. Grid-stride
// over the items.
template <class T, int L, bool HALF>
__global__ void __launch_bounds__(kThreadsQK) k_qk_norm_rope_bwd(const QkArgs a) {
  constexpr int kGroups = kThreadsQK / L;
  __shared__ float part[kGroups][8 * L];
  const int lane = threadIdx.x & 31, lane_in = threadIdx.x % L, group = threadIdx.x / L;
  const float inv = a.norm == TTT_NORM_RMS ? 1.f / a.width : 1.f;
  float dw[2][8] = {};
  const int64_t step = (int64_t)gridDim.x * kGroups;
  for (int64_t base = (int64_t)blockIdx.x * kGroups; base < a.items; base += step) {
    const Item<L> it(a, base + group);
    const int64_t pos = !it.valid ? 0 : a.positions != nullptr ? a.positions[it.b * a.positions_stride + it.t] : a.position0 + it.t;
    const Turn turn = make_turn<HALF>(a, pos, lane_in, lane);
    const bool live = it.valid && 8 * lane_in < a.width;
    for (int i = 0; i < a.heads_per; ++i) {
      const int h = it.h0 + i;
      const bool ok = live && h < it.h1;
      const int sd = h >= a.side[0].heads ? 1 : 0;
      const QkSide& S = a.side[sd];
      const int64_t hh = h - (sd ? a.side[0].heads : 0);
      float e[8], n[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = n[j] = 0.f;
      if (ok) {
        load8<T>(static_cast<const T*>(S.dy) + it.b * S.gb + hh * S.gh + it.t * S.gt + 8 * lane_in, e);
        if (a.norm != TTT_NORM_NONE)
          load8<T>(static_cast<const T*>(S.x) + it.b * S.xb + hh * S.xh + it.t * S.xt + 8 * lane_in, n);
      }
      rotate<HALF, true>(e, turn);
      if (a.norm != TTT_NORM_NONE) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(n[j], n[j], ss);
        const float r = rsqrtf(fmaf(group_sum<L>(ss), inv, a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] *= r;
        if (S.w != nullptr && ok) {
          float w[8];
          load8<float>(S.w + 8 * lane_in, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = e[j] * n[j];
            dw[0][j] += sd ? 0.f : d;
            dw[1][j] += sd ? d : 0.f;
            e[j] *= w[j];
          }
        }
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = fmaf(e[j], n[j], dot);
        dot = group_sum<L>(dot) * inv;
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = r * fmaf(-dot, n[j], e[j]);
      }
      if (ok) store8<T>(static_cast<T*>(S.y) + it.b * S.yb + hh * S.yh + it.t * S.yt + 8 * lane_in, e);
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int sd = 0; sd < 2; ++sd) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) part[group][8 * lane_in + j] = dw[sd][j];
    __syncthreads();
    for (int j = threadIdx.x; j < a.width; j += kThreadsQK) {
      float s = 0.f;
#pragma unroll 8
      for (int gi = 0; gi < kGroups; ++gi) s += part[gi][j];
      a.partial[((size_t)blockIdx.x * 2 + sd) * a.width + j] = s;
    }
  }
}

// Sums over the CTAs: one warp per value, grid (width, 2).
__global__ void __launch_bounds__(32) k_qk_gain_sum(const float* __restrict__ partial, int n, int width, float* dwq, float* dwk) {
  const int j = blockIdx.x, sd = blockIdx.y;
  float* out = sd ? dwk : dwq;
  if (out == nullptr) return;
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 32) s += (double)partial[((size_t)i * 2 + sd) * width + j];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x == 0) out[j] = (float)s;
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

// Parts of a token's heads: one, unless the tokens alone give the GPU fewer than 512 threads an SM.
int splits_of(const ttt_qk_desc* d, int num_sms) {
  const int64_t rows = (int64_t)d->batch * d->tokens, heads = (int64_t)d->q_heads + d->k_heads;
  const int64_t want = (int64_t)num_sms * 512 / lanes_of(d->width);
  return (int)std::max<int64_t>(1, std::min(heads, want / std::max<int64_t>(1, rows)));
}

constexpr int kBwdCtasPerSm = 4;

int64_t bwd_blocks(int64_t items, int width, int num_sms) {
  const int64_t g = groups_per_block(width);
  return std::max<int64_t>(1, std::min<int64_t>((items + g - 1) / g, (int64_t)num_sms * kBwdCtasPerSm));
}

QkSide side_of(const void* x, const ttt_strides& xs, const void* dy, const ttt_strides& gs, void* y, const ttt_strides& ys,
               const float* w, int heads) {
  return QkSide{x, dy, y, xs.batch, xs.head, xs.token, ys.batch, ys.head, ys.token, gs.batch, gs.head, gs.token, w, heads};
}

QkArgs args_of(const ttt_qk_desc* d, const int64_t* positions, const double* freqs, int num_sms) {
  QkArgs a = {};
  a.width = d->width;
  a.rot = d->rot;
  a.norm = d->norm;
  a.eps = d->eps;
  a.magnitude = d->magnitude;
  a.tokens = d->tokens;
  const int heads = d->q_heads + d->k_heads;
  a.heads_per = (heads + splits_of(d, num_sms) - 1) / splits_of(d, num_sms);
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
  QkArgs a = args_of(d, positions, freqs, num_sms);
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
  QkArgs a = args_of(d, positions, freqs, num_sms);
  a.side[0] = side_of(q, d->q, dqo, d->q_out, dq, d->q_grad, qw, d->q_heads);
  a.side[1] = side_of(k, d->k, dko, d->k_out, dk, d->k_grad, kw, d->k_heads);
  const bool gains = dqw != nullptr || dkw != nullptr;
  a.partial = gains ? static_cast<float*>(ws) : nullptr;
  const int64_t blocks = bwd_blocks(a.items, d->width, num_sms);
  run(a, d, true, blocks, s);
  TTT_CUDA(cudaGetLastError());
  if (gains) {
    k_qk_gain_sum<<<dim3(d->width, 2), 32, 0, s>>>(a.partial, (int)blocks, d->width, dqw, dkw);
    TTT_CUDA(cudaGetLastError());
  }
  return TTT_OK;
}

}  // namespace ttt
