// C entry points of the operators around the scans: argument checks, the device's SM count, and
// dispatch. What each call means is documented in include/ttt.h.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <nvtx3/nvToolsExt.h>

#include "internal.h"

namespace ttt {

namespace {

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

bool aligned(const void* p, uintptr_t n = 16) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

ttt_status need(const void* p, const char* name) {
  if (p == nullptr || !aligned(p)) return fail(TTT_ERR_INVALID_ARG, "%s must be a 16-byte aligned device pointer", name);
  return TTT_OK;
}

ttt_status optional(const void* p, const char* name) {
  if (!aligned(p)) return fail(TTT_ERR_INVALID_ARG, "%s must be a 16-byte aligned device pointer or NULL", name);
  return TTT_OK;
}

constexpr int kMaxDevices = 64;

// SMs of the current device, or 0 without one (read once per device).
int current_sms() {
  static std::atomic<int> sms[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return 0;
  }
  int n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

ttt_status need_device(int* sms) {
  *sms = current_sms();
  if (*sms == 0) return fail(TTT_ERR_CUDA, "no usable CUDA device is current");
  return TTT_OK;
}

// Where kernels of calls without a status word of their own report: code and site, one pair a device.
__device__ int g_op_status[2];
std::atomic<int*> g_op_words[kMaxDevices];

std::atomic<uint64_t> g_op_limit{kWaitLimitNs};
std::atomic<int> g_op_inject{0};

// The device's pair, of the current device (found once per device).
ttt_status op_words(int** out) {
  int dev = -1;
  TTT_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return fail(TTT_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  *out = g_op_words[dev].load(std::memory_order_acquire);
  if (*out != nullptr) return TTT_OK;
  void* p = nullptr;
  TTT_CUDA(cudaGetSymbolAddress(&p, g_op_status));
  *out = static_cast<int*>(p);
  g_op_words[dev].store(*out, std::memory_order_release);
  return TTT_OK;
}

ttt_status check_workspace(const void* ws, size_t have, size_t want) {
  if (want == 0) return TTT_OK;
  if (ws == nullptr || !aligned(ws, 256)) return fail(TTT_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
  if (have < want) return fail(TTT_ERR_INVALID_ARG, "workspace holds %zu bytes, the call needs %zu", have, want);
  return TTT_OK;
}

constexpr int64_t kMaxStride = (int64_t)1 << 48;

ttt_status check_strides(const ttt_strides& s, int unit, const char* name) {
  const int64_t v[3] = {s.batch, s.head, s.token};
  for (int64_t x : v)
    if (x < 0 || x > kMaxStride || x % unit != 0)
      return fail(TTT_ERR_INVALID_ARG, "%s: strides must be non-negative%s", name,
                  unit > 1 ? " and whole 16-byte steps" : "");
  return TTT_OK;
}

// Rows of `width` elements at these strides must not overlap.
ttt_status check_output(const ttt_strides& s, int64_t batch, int64_t heads, int64_t tokens, int64_t width, int unit,
                        const char* name) {
  TTT_TRY(check_strides(s, unit, name));
  struct D {
    int64_t stride, n;
  } d[3] = {{s.batch, batch}, {s.head, heads}, {s.token, tokens}};
  std::sort(d, d + 3, [](const D& a, const D& b) { return a.stride < b.stride; });
  double extent = (double)width;
  for (const D& x : d) {
    if (x.n <= 1) continue;
    if ((double)x.stride < extent) return fail(TTT_ERR_INVALID_ARG, "%s: its rows would overlap at these strides", name);
    extent += (double)x.stride * (double)(x.n - 1);
  }
  return TTT_OK;
}

ttt_status check_qk(const ttt_qk_desc* d) {
  if (d == nullptr) return fail(TTT_ERR_INVALID_ARG, "desc is NULL");
  if (d->io_dtype != TTT_BF16 && d->io_dtype != TTT_F32)
    return fail(TTT_ERR_UNSUPPORTED, "queries and keys: io_dtype must be BF16 or F32");
  if (d->batch < 0 || d->tokens < 0 || d->q_heads < 0 || d->k_heads < 0 || (d->q_heads == 0 && d->k_heads == 0))
    return fail(TTT_ERR_INVALID_ARG, "batch and tokens must be non-negative and one of q_heads, k_heads positive");
  if ((int64_t)d->q_heads + d->k_heads > (1 << 20)) return fail(TTT_ERR_UNSUPPORTED, "more than 2^20 heads");
  if (d->tokens > ((int64_t)1 << 40)) return fail(TTT_ERR_UNSUPPORTED, "more than 2^40 tokens");
  if (d->width < 8 || d->width > 256 || d->width % 8 != 0)
    return fail(TTT_ERR_UNSUPPORTED, "head width must be a multiple of 8 from 8 to 256");
  if (d->rot < 0 || d->rot > d->width || d->rot % 16 != 0)
    return fail(TTT_ERR_UNSUPPORTED, "rot must be a multiple of 16 from 0 to the head width");
  if (d->norm != TTT_NORM_NONE && d->norm != TTT_NORM_RMS && d->norm != TTT_NORM_L2)
    return fail(TTT_ERR_INVALID_ARG, "unknown norm %d", d->norm);
  if (d->layout != TTT_ROPE_HALF && d->layout != TTT_ROPE_INTERLEAVED)
    return fail(TTT_ERR_INVALID_ARG, "unknown rotary layout %d", d->layout);
  if (!(d->eps >= 0.f)) return fail(TTT_ERR_INVALID_ARG, "eps must not be negative");
  if (d->positions_stride != 0 && d->positions_stride < d->tokens)
    return fail(TTT_ERR_INVALID_ARG, "positions_stride must be 0 or at least the tokens of a sequence");
  return TTT_OK;
}

ttt_status check_weights(const ttt_qk_desc* d, const float* qw, const float* kw, const double* freqs) {
  TTT_TRY(optional(qw, "q_weight"));
  TTT_TRY(optional(kw, "k_weight"));
  if ((qw != nullptr || kw != nullptr) && d->norm != TTT_NORM_RMS)
    return fail(TTT_ERR_INVALID_ARG, "q_weight and k_weight belong to the RMS norm");
  if ((d->rot > 0) != (freqs != nullptr) || !aligned(freqs, 8))
    return fail(TTT_ERR_INVALID_ARG, "freqs must be an 8-byte aligned device pointer where rot > 0, and NULL otherwise");
  return TTT_OK;
}

ttt_status check_scan(const ttt_gated_scan_desc* d) {
  if (d == nullptr) return fail(TTT_ERR_INVALID_ARG, "desc is NULL");
  if (d->batch < 1 || d->heads < 1 || d->tokens < 0)
    return fail(TTT_ERR_INVALID_ARG, "batch and heads must be positive and tokens non-negative");
  if ((int64_t)d->batch * d->heads > (1 << 24)) return fail(TTT_ERR_UNSUPPORTED, "batch times heads above 2^24");
  if (d->tokens > ((int64_t)1 << 30)) return fail(TTT_ERR_UNSUPPORTED, "more than 2^30 tokens");
  const struct {
    const ttt_strides* s;
    const char* name;
  } in[4] = {{&d->q, "q"}, {&d->k, "k"}, {&d->v, "v"}, {&d->o, "o"}};
  for (const auto& x : in) {
    TTT_TRY(check_strides(*x.s, 8, x.name));
    if (x.s->token == 0 && d->tokens > 1) return fail(TTT_ERR_UNSUPPORTED, "%s: one row for all tokens (token stride 0)", x.name);
    for (int64_t v : {x.s->batch, x.s->head, x.s->token})
      if (v >= (int64_t)1 << 39) return fail(TTT_ERR_UNSUPPORTED, "%s: a stride of 2^39 elements or more", x.name);
  }
  TTT_TRY(check_strides(d->g, 1, "g"));
  return TTT_OK;
}

ttt_status check_scan_inputs(const void* q, const void* k, const void* v, const float* g) {
  TTT_TRY(need(q, "q"));
  TTT_TRY(need(k, "k"));
  TTT_TRY(need(v, "v"));
  if (g == nullptr || !aligned(g, 4)) return fail(TTT_ERR_INVALID_ARG, "g must be a 4-byte aligned device pointer");
  return TTT_OK;
}

ttt_status check_ffn(int64_t T, int32_t d, int32_t f, int32_t act) {
  if (T < 0) return fail(TTT_ERR_INVALID_ARG, "T must be non-negative");
  if (act != TTT_ACT_SILU && act != TTT_ACT_GELU) return fail(TTT_ERR_INVALID_ARG, "unknown activation %d", act);
  if (T > (1 << 24)) return fail(TTT_ERR_UNSUPPORTED, "T must be at most 2^24");
  if (d < 8 || f < 8 || d % 8 != 0 || f % 8 != 0 || d > (1 << 20) || f > (1 << 20))
    return fail(TTT_ERR_UNSUPPORTED, "d and f must be multiples of 8 from 8 to 2^20");
  return TTT_OK;
}

ttt_status check_status(const int32_t* status) {
  if (!aligned(status, 4)) return fail(TTT_ERR_INVALID_ARG, "status must be a 4-byte aligned device pointer or NULL");
  return TTT_OK;
}

cudaStream_t cs(ttt_stream s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

ttt_status op_status(int32_t* callers, DevStatus* out) {
  *out = DevStatus{callers, g_op_limit.load(std::memory_order_relaxed)};
  if (callers == nullptr) {
    TTT_TRY(op_words(&out->word));
    out->site = out->word + 1;
  }
  return TTT_OK;
}

int op_stall(bool can) { return can && g_op_inject.load(std::memory_order_relaxed) != 0 && g_op_inject.exchange(0) != 0 ? 1 : -1; }

}  // namespace ttt

using namespace ttt;

extern "C" ttt_status ttt_qk_norm_rope(const ttt_qk_desc* d, const void* q, const void* k, const float* qw, const float* kw,
                                       const int64_t* positions, const double* freqs, void* qo, void* ko,
                                       ttt_stream stream) {
  Range range("ttt_qk_norm_rope");
  TTT_TRY(check_qk(d));
  if (d->batch == 0 || d->tokens == 0) return TTT_OK;
  TTT_TRY(check_weights(d, qw, kw, freqs));
  if (!aligned(positions, 8)) return fail(TTT_ERR_INVALID_ARG, "positions must be an 8-byte aligned device pointer or NULL");
  const int unit = d->io_dtype == TTT_F32 ? 4 : 8;
  const struct {
    int heads;
    const void *x, *y;
    const ttt_strides *xs, *ys;
    const char* name;
  } side[2] = {{d->q_heads, q, qo, &d->q, &d->q_out, "q"}, {d->k_heads, k, ko, &d->k, &d->k_out, "k"}};
  for (const auto& s : side) {
    if ((s.heads == 0) != (s.x == nullptr) || (s.heads == 0) != (s.y == nullptr))
      return fail(TTT_ERR_INVALID_ARG, "%s and its output must be given exactly where it has heads", s.name);
    if (s.heads == 0) continue;
    TTT_TRY(need(s.x, s.name));
    TTT_TRY(need(s.y, s.name));
    TTT_TRY(check_strides(*s.xs, unit, s.name));
    TTT_TRY(check_output(*s.ys, d->batch, s.heads, d->tokens, d->width, unit, s.name));
  }
  int sms;
  TTT_TRY(need_device(&sms));
  return qk_norm_rope(d, q, k, qw, kw, positions, freqs, qo, ko, sms, cs(stream));
}

extern "C" size_t ttt_qk_norm_rope_workspace(const ttt_qk_desc* d) {
  return check_qk(d) == TTT_OK && current_sms() > 0 ? qk_norm_rope_workspace(d, current_sms()) : 0;
}

extern "C" ttt_status ttt_qk_norm_rope_backward(const ttt_qk_desc* d, const void* dqo, const void* dko, const void* q,
                                                const void* k, const float* qw, const float* kw, const int64_t* positions,
                                                const double* freqs, void* dq, void* dk, float* dqw, float* dkw, void* ws,
                                                size_t ws_bytes, ttt_stream stream) {
  Range range("ttt_qk_norm_rope_backward");
  TTT_TRY(check_qk(d));
  if ((dqw != nullptr && qw == nullptr) || (dkw != nullptr && kw == nullptr))
    return fail(TTT_ERR_INVALID_ARG, "the gradient of a weight that was not given");
  TTT_TRY(optional(dqw, "dq_weight"));
  TTT_TRY(optional(dkw, "dk_weight"));
  TTT_TRY(optional(qw, "q_weight"));
  TTT_TRY(optional(kw, "k_weight"));
  if (d->batch == 0 || d->tokens == 0) {
    if (dqw != nullptr) TTT_CUDA(cudaMemsetAsync(dqw, 0, sizeof(float) * d->width, cs(stream)));
    if (dkw != nullptr) TTT_CUDA(cudaMemsetAsync(dkw, 0, sizeof(float) * d->width, cs(stream)));
    return TTT_OK;
  }
  TTT_TRY(check_weights(d, qw, kw, freqs));
  if (!aligned(positions, 8)) return fail(TTT_ERR_INVALID_ARG, "positions must be an 8-byte aligned device pointer or NULL");
  const int unit = d->io_dtype == TTT_F32 ? 4 : 8;
  const bool norm = d->norm != TTT_NORM_NONE;
  const struct {
    int heads;
    const void *x, *dy, *dx;
    const ttt_strides *xs, *gs, *ys;
    const char* name;
  } side[2] = {{d->q_heads, q, dqo, dq, &d->q, &d->q_out, &d->q_grad, "q"},
               {d->k_heads, k, dko, dk, &d->k, &d->k_out, &d->k_grad, "k"}};
  for (const auto& s : side) {
    if ((s.heads == 0) != (s.dy == nullptr) || (s.heads == 0) != (s.dx == nullptr) || (s.heads == 0 && s.x != nullptr))
      return fail(TTT_ERR_INVALID_ARG, "%s and its gradients must be given exactly where it has heads", s.name);
    if (s.heads == 0) continue;
    if (norm) {
      TTT_TRY(need(s.x, s.name));
      TTT_TRY(check_strides(*s.xs, unit, s.name));
    }
    TTT_TRY(need(s.dy, s.name));
    TTT_TRY(need(s.dx, s.name));
    TTT_TRY(check_strides(*s.gs, unit, s.name));
    TTT_TRY(check_output(*s.ys, d->batch, s.heads, d->tokens, d->width, unit, s.name));
  }
  int sms;
  TTT_TRY(need_device(&sms));
  if (dqw != nullptr || dkw != nullptr) TTT_TRY(check_workspace(ws, ws_bytes, qk_norm_rope_workspace(d, sms)));
  return qk_norm_rope_backward(d, dqo, dko, q, k, qw, kw, positions, freqs, dq, dk, dqw, dkw, ws, sms, cs(stream));
}

extern "C" ttt_status ttt_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double trained,
                                           double beta_fast, double beta_slow, double* freqs, float* magnitude) {
  if (freqs == nullptr) return fail(TTT_ERR_INVALID_ARG, "freqs is NULL");
  if (rot < 2 || rot % 2 != 0) return fail(TTT_ERR_INVALID_ARG, "rot must be a positive even number");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(TTT_ERR_INVALID_ARG, "base must be above 1");
  if (!(factor >= 1.0) || !std::isfinite(factor)) return fail(TTT_ERR_INVALID_ARG, "factor must be at least 1");
  if (scaling < TTT_ROPE_SCALE_NONE || scaling > TTT_ROPE_SCALE_YARN)
    return fail(TTT_ERR_INVALID_ARG, "unknown rotary scaling %d", scaling);
  float m = 1.f;
  if (scaling == TTT_ROPE_SCALE_NTK) {
    if (rot == 2) return fail(TTT_ERR_INVALID_ARG, "NTK scaling needs rot above 2");
    base *= std::pow(factor, (double)rot / (rot - 2));
  }
  for (int i = 0; i < rot / 2; ++i) freqs[i] = std::pow(base, -2.0 * i / rot);
  if (scaling == TTT_ROPE_SCALE_LINEAR)
    for (int i = 0; i < rot / 2; ++i) freqs[i] /= factor;
  if (scaling == TTT_ROPE_SCALE_YARN) {
    if (!(trained > 0.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(trained) || !std::isfinite(beta_fast))
      return fail(TTT_ERR_INVALID_ARG, "YaRN needs trained > 0 and beta_fast > beta_slow > 0");
    // The pair that turns n times within the trained length: base^(-2i/rot)·trained = 2π·n.
    auto pair_of = [&](double n) { return rot * std::log(trained / (n * 2.0 * M_PI)) / (2.0 * std::log(base)); };
    const double lo = std::max(std::floor(pair_of(beta_fast)), 0.0), hi = std::min(std::ceil(pair_of(beta_slow)), rot - 1.0);
    for (int i = 0; i < rot / 2; ++i) {
      const double ramp = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      freqs[i] = freqs[i] / factor * ramp + freqs[i] * (1.0 - ramp);
    }
    m = (float)(0.1 * std::log(factor) + 1.0);
  }
  if (magnitude != nullptr) *magnitude = m;
  return TTT_OK;
}

extern "C" size_t ttt_gated_scan_workspace(const ttt_gated_scan_desc* d) {
  return check_scan(d) == TTT_OK && d->tokens > 0 && current_sms() > 0 ? gated_scan_workspace(d, false, current_sms()) : 0;
}

extern "C" size_t ttt_gated_scan_backward_workspace(const ttt_gated_scan_desc* d) {
  return check_scan(d) == TTT_OK && d->tokens > 0 && current_sms() > 0 ? gated_scan_workspace(d, true, current_sms()) : 0;
}

extern "C" ttt_status ttt_gated_scan(const ttt_gated_scan_desc* d, const void* q, const void* k, const void* v,
                                     const float* g, const float* S0, void* o, float* S_end, void* ws, size_t ws_bytes,
                                     int32_t* status, ttt_stream stream) {
  Range range("ttt_gated_scan");
  TTT_TRY(check_scan(d));
  TTT_TRY(optional(S0, "S0"));
  TTT_TRY(optional(S_end, "S_end"));
  TTT_TRY(check_status(status));
  if (d->tokens == 0) {
    if (status != nullptr) TTT_CUDA(cudaMemsetAsync(status, 0, sizeof(int32_t), cs(stream)));
    const size_t bytes = (size_t)d->batch * d->heads * 64 * 64 * sizeof(float);
    if (S_end != nullptr && S0 == nullptr) TTT_CUDA(cudaMemsetAsync(S_end, 0, bytes, cs(stream)));
    if (S_end != nullptr && S0 != nullptr && S_end != S0)
      TTT_CUDA(cudaMemcpyAsync(S_end, S0, bytes, cudaMemcpyDeviceToDevice, cs(stream)));
    return TTT_OK;
  }
  TTT_TRY(check_scan_inputs(q, k, v, g));
  TTT_TRY(need(o, "o"));
  TTT_TRY(check_output(d->o, d->batch, d->heads, d->tokens, 64, 8, "o"));
  int sms;
  TTT_TRY(need_device(&sms));
  TTT_TRY(check_workspace(ws, ws_bytes, gated_scan_workspace(d, false, sms)));
  if (status != nullptr) TTT_CUDA(cudaMemsetAsync(status, 0, sizeof(int32_t), cs(stream)));
  DevStatus report;
  TTT_TRY(op_status(status, &report));
  return gated_scan(d, q, k, v, g, S0, o, S_end, ws, report, sms, cs(stream));
}

extern "C" ttt_status ttt_gated_scan_backward(const ttt_gated_scan_desc* d, const void* d_o, const void* q, const void* k,
                                              const void* v, const float* g, const float* S0, const float* dS_end, void* dq,
                                              void* dk, void* dv, float* dg, float* dS0, void* ws, size_t ws_bytes,
                                              int32_t* status, ttt_stream stream) {
  Range range("ttt_gated_scan_backward");
  TTT_TRY(check_scan(d));
  TTT_TRY(optional(S0, "S0"));
  TTT_TRY(optional(dS_end, "dS_end"));
  TTT_TRY(optional(dS0, "dS0"));
  TTT_TRY(check_status(status));
  if (d->tokens == 0) {
    if (status != nullptr) TTT_CUDA(cudaMemsetAsync(status, 0, sizeof(int32_t), cs(stream)));
    const size_t bytes = (size_t)d->batch * d->heads * 64 * 64 * sizeof(float);
    if (dS0 != nullptr && dS_end == nullptr) TTT_CUDA(cudaMemsetAsync(dS0, 0, bytes, cs(stream)));
    if (dS0 != nullptr && dS_end != nullptr && dS0 != dS_end)
      TTT_CUDA(cudaMemcpyAsync(dS0, dS_end, bytes, cudaMemcpyDeviceToDevice, cs(stream)));
    return TTT_OK;
  }
  TTT_TRY(check_scan_inputs(q, k, v, g));
  TTT_TRY(need(d_o, "d_o"));
  TTT_TRY(need(dq, "dq"));
  TTT_TRY(need(dk, "dk"));
  TTT_TRY(need(dv, "dv"));
  TTT_TRY(need(dg, "dg"));
  int sms;
  TTT_TRY(need_device(&sms));
  TTT_TRY(check_workspace(ws, ws_bytes, gated_scan_workspace(d, true, sms)));
  if (status != nullptr) TTT_CUDA(cudaMemsetAsync(status, 0, sizeof(int32_t), cs(stream)));
  DevStatus report;
  TTT_TRY(op_status(status, &report));
  return gated_scan_backward(d, d_o, q, k, v, g, S0, dS_end, dq, dk, dv, dg, dS0, ws, report, sms, cs(stream));
}

extern "C" ttt_status ttt_gated_scan_step(const ttt_gated_scan_desc* d, const void* q, const void* k, const void* v,
                                          const float* g, float* S, void* o, ttt_stream stream) {
  Range range("ttt_gated_scan_step");
  TTT_TRY(check_scan(d));
  if (d->tokens != 1) return fail(TTT_ERR_INVALID_ARG, "a step takes one token");
  TTT_TRY(check_scan_inputs(q, k, v, g));
  TTT_TRY(need(S, "S"));
  TTT_TRY(need(o, "o"));
  TTT_TRY(check_output(d->o, d->batch, d->heads, 1, 64, 8, "o"));
  int sms;
  TTT_TRY(need_device(&sms));
  return gated_scan_step(d, q, k, v, g, S, o, cs(stream));
}

extern "C" ttt_status ttt_gated_ffn(const void* X, const void* Wg, const void* Wu, int64_t T, int32_t d, int32_t f, int32_t act,
                                    void* Z, void* G, void* U, int32_t* status, ttt_stream stream) {
  Range range("ttt_gated_ffn");
  TTT_TRY(check_ffn(T, d, f, act));
  TTT_TRY(check_status(status));
  int sms;
  if (T > 0) {
    TTT_TRY(need(X, "X"));
    TTT_TRY(need(Wg, "Wg"));
    TTT_TRY(need(Wu, "Wu"));
    TTT_TRY(need(Z, "Z"));
    TTT_TRY(optional(G, "G"));
    TTT_TRY(optional(U, "U"));
    if ((G == nullptr) != (U == nullptr)) return fail(TTT_ERR_INVALID_ARG, "G and U are kept together or not at all");
    TTT_TRY(need_device(&sms));
  }
  if (status != nullptr) TTT_CUDA(cudaMemsetAsync(status, 0, sizeof(int32_t), cs(stream)));
  if (T == 0) return TTT_OK;
  DevStatus report;
  TTT_TRY(op_status(status, &report));
  return gated_ffn(X, Wg, Wu, T, d, f, act, Z, G, U, report, sms, cs(stream));
}

extern "C" size_t ttt_gated_ffn_backward_workspace(int64_t T, int32_t d, int32_t f) {
  return check_ffn(T, d, f, TTT_ACT_SILU) == TTT_OK && T > 0 && current_sms() > 0
             ? gated_ffn_backward_workspace(T, d, f, current_sms())
             : 0;
}

extern "C" ttt_status ttt_gated_ffn_backward(const void* dZ, const void* X, const void* Wg, const void* Wu, const void* G,
                                             const void* U, int64_t T, int32_t d, int32_t f, int32_t act, void* dX, void* dWg,
                                             void* dWu, void* ws, size_t ws_bytes, int32_t* status, ttt_stream stream) {
  Range range("ttt_gated_ffn_backward");
  TTT_TRY(check_ffn(T, d, f, act));
  TTT_TRY(check_status(status));
  TTT_TRY(optional(dX, "dX"));
  TTT_TRY(optional(dWg, "dWg"));
  TTT_TRY(optional(dWu, "dWu"));
  if ((dWg == nullptr) != (dWu == nullptr)) return fail(TTT_ERR_INVALID_ARG, "dWg and dWu are made together or not at all");
  int sms;
  if (T > 0) {
    TTT_TRY(need(dZ, "dZ"));
    TTT_TRY(need(G, "G"));
    TTT_TRY(need(U, "U"));
    if (dWg != nullptr) TTT_TRY(need(X, "X"));
    if (dX != nullptr) {
      TTT_TRY(need(Wg, "Wg"));
      TTT_TRY(need(Wu, "Wu"));
    }
    TTT_TRY(need_device(&sms));
    TTT_TRY(check_workspace(ws, ws_bytes, gated_ffn_backward_workspace(T, d, f, sms)));
  }
  if (status != nullptr) TTT_CUDA(cudaMemsetAsync(status, 0, sizeof(int32_t), cs(stream)));
  if (T == 0) {
    if (dWg != nullptr) {
      TTT_CUDA(cudaMemsetAsync(dWg, 0, (size_t)f * d * 2, cs(stream)));
      TTT_CUDA(cudaMemsetAsync(dWu, 0, (size_t)f * d * 2, cs(stream)));
    }
    return TTT_OK;
  }
  DevStatus report;
  TTT_TRY(op_status(status, &report));
  return gated_ffn_backward(dZ, X, Wg, Wu, G, U, T, d, f, act, dX, dWg, dWu, ws, report, sms, cs(stream));
}

extern "C" ttt_status ttt_operators_set_option(int32_t option, int64_t value) {
  switch (option) {
    case TTT_OPT_WAIT_LIMIT_NS:
      if (value < 1000000 || value > 60000000000ll)
        return fail(TTT_ERR_INVALID_ARG, "TTT_OPT_WAIT_LIMIT_NS of the operators must lie in [1e6, 6e10] (got %lld)", (long long)value);
      g_op_limit.store((uint64_t)value);
      return TTT_OK;
    case TTT_OPT_INJECT_STALL:
      if (value != 0 && value != 1) return fail(TTT_ERR_INVALID_ARG, "TTT_OPT_INJECT_STALL must be 0 or 1");
      g_op_inject.store((int)value);
      return TTT_OK;
    default:
      return fail(TTT_ERR_INVALID_ARG, "option %d is not one of the operators'", option);
  }
}

extern "C" ttt_status ttt_operators_poll(void) {
  int sms, *words;
  TTT_TRY(need_device(&sms));
  TTT_TRY(op_words(&words));
  TTT_CUDA(cudaDeviceSynchronize());
  int v[2] = {0, 0};
  TTT_CUDA(cudaMemcpy(v, words, sizeof(v), cudaMemcpyDeviceToHost));
  if (v[0] == 0) return TTT_OK;
  TTT_CUDA(cudaMemset(words, 0, sizeof(v)));
  return fail(TTT_ERR_TIMEOUT, "a bounded device-side wait ran out (mbarrier at shared offset 0x%x)", v[1] & 0xFFFF);
}
