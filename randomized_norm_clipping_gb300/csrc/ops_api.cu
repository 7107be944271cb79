// libdprc C ABI of the operators around the norm path (the embedding, dropout,
// the linear map, normalisation, rotary positions, attention): argument checks,
// then the launchers.

#include <algorithm>

#include <cuda_runtime.h>
#include <stdint.h>

#include "dprc.h"
#include "internal.h"

using namespace dprc;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxOpWidth = int64_t(1) << 20;
constexpr int64_t kMaxSamples = 65535;

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool finite_f(float x) { return x > -__builtin_inff() && x < __builtin_inff(); }
bool known(dprc_dtype dt) { return dt == DPRC_F32 || dt == DPRC_BF16; }
dprc_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DPRC_OK : DPRC_ERR_CUDA; }

dprc_status check_plan(int64_t N, int64_t V, const void* plan, size_t plan_bytes) {
  if (!plan || plan_bytes < embed_plan_bytes(N, V)) return DPRC_ERR_WORKSPACE;
  return aligned(plan) ? DPRC_OK : DPRC_ERR_ALIGN;
}

dprc_status check_embed(const void* G, dprc_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d,
                        float scale, const void* out, const void* plan, size_t plan_bytes,
                        const void* ws, size_t ws_bytes) {
  if (!known(dt)) return DPRC_ERR_DTYPE;
  if (B < 1 || B > kMaxSamples || T < 0 || T > kMaxTokens / B) return DPRC_ERR_SHAPE;
  if (V < 1 || V > kMaxVocab || d < 1 || d > kMaxOpWidth) return DPRC_ERR_SHAPE;
  if (!finite_f(scale)) return DPRC_ERR_SHAPE;
  if (!out || (T > 0 && !G)) return DPRC_ERR_NULL;
  if (!aligned(G) || !aligned(out)) return DPRC_ERR_ALIGN;
  const dprc_status st = check_plan(B * T, V, plan, plan_bytes);
  if (st != DPRC_OK) return st;
  if (!ws || ws_bytes < embed_norm_ws_bytes(dt, B * T, d)) return DPRC_ERR_WORKSPACE;
  return aligned(ws) ? DPRC_OK : DPRC_ERR_ALIGN;
}

dprc_status check_linear(dprc_dtype dt, int64_t M, int64_t K, int64_t N, int act, double p) {
  if (!known(dt)) return DPRC_ERR_DTYPE;
  if (M < 0 || M > kMaxTokens || K < 1 || K > kMaxOpWidth || N < 1 || N > kMaxOpWidth)
    return DPRC_ERR_SHAPE;
  // block counts of the launches stay below 2^31
  if ((M + 63) / 64 * ((N + 255) / 256) > (int64_t(1) << 30)) return DPRC_ERR_SHAPE;
  if (act < DPRC_ACT_NONE || act > DPRC_ACT_SILU) return DPRC_ERR_SHAPE;
  if (!(p >= 0.0) || !(p <= 1.0)) return DPRC_ERR_SHAPE;
  return DPRC_OK;
}

constexpr int64_t kMaxNormWidth = 16384;
constexpr int64_t kMaxHeadWidth = 128;
constexpr int64_t kMaxRotWidth = 4096;
constexpr int64_t kMaxPositions = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40;

dprc_status check_layernorm(dprc_dtype dt, int64_t B, int64_t T, int64_t d) {
  if (!known(dt)) return DPRC_ERR_DTYPE;
  if (B < 1 || B > kMaxSamples || T < 0 || T > kMaxTokens / B) return DPRC_ERR_SHAPE;
  return d < 1 || d > kMaxNormWidth ? DPRC_ERR_SHAPE : DPRC_OK;
}

bool strides_ok(const int64_t* s) {
  for (int k = 0; k < 3; ++k)
    if (s[k] < 0 || s[k] > kMaxStride) return false;
  return true;
}

// Whether rows of D elements at these strides (of B, T and H of them) lie apart, so that each
// element of a result has one writer: every axis steps over all that lies within.
bool apart(const int64_t* s, int64_t B, int64_t T, int64_t H, int64_t D) {
  const int64_t n[3] = {B, T, H};
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return s[a] < s[b]; });
  __int128 span = D;
  for (const int k : order) {
    if (n[k] < 2) continue;
    if (s[k] < span) return false;
    span += static_cast<__int128>(n[k] - 1) * s[k];
  }
  return true;
}

// An array of elements of `size` bytes, from an address of its own type's alignment on.
bool element_aligned(const void* p, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0;
}
size_t size_of(dprc_dtype dt) { return dt == DPRC_F32 ? 4 : 2; }

dprc_status check_attention(const dprc_attention_args* a) {
  if (!a) return DPRC_ERR_NULL;
  if (!known(a->dtype)) return DPRC_ERR_DTYPE;
  if (a->B < 1 || a->Tq < 0 || a->Tq > kMaxPositions || a->Tk < 0 || a->Tk > kMaxPositions)
    return DPRC_ERR_SHAPE;
  if (a->H < 1 || a->Hkv < 1 || a->H % a->Hkv != 0 || a->D < 1 || a->D > kMaxHeadWidth)
    return DPRC_ERR_SHAPE;
  // grids and row numbers stay in range
  if (a->Hkv > kMaxSamples || a->B > kMaxSamples / a->Hkv) return DPRC_ERR_SHAPE;
  if (a->H / a->Hkv > 4096 || a->Tq * (a->H / a->Hkv) > (int64_t(1) << 28)) return DPRC_ERR_SHAPE;
  if (a->Tq * (a->H / a->Hkv) / 16 + a->Tk / 16 > (int64_t(1) << 30) / (a->B * a->Hkv))
    return DPRC_ERR_SHAPE;
  if (!finite_f(a->scale) || !finite_f(a->cap) || a->cap < 0.f) return DPRC_ERR_SHAPE;
  if (!strides_ok(a->q_stride) || !strides_ok(a->k_stride) || !strides_ok(a->v_stride))
    return DPRC_ERR_SHAPE;
  return DPRC_OK;
}

dprc_status check_attention_inputs(const dprc_attention_args* a) {
  if ((a->Tq > 0 && !a->Q) || (a->Tk > 0 && (!a->K || !a->V))) return DPRC_ERR_NULL;
  const size_t e = size_of(a->dtype);
  if (!element_aligned(a->Q, e) || !element_aligned(a->K, e) || !element_aligned(a->V, e) ||
      !element_aligned(a->slopes, 4) || !element_aligned(a->docs, 4) ||
      !element_aligned(a->prefix, 4) || !element_aligned(a->lengths, 4) ||
      !element_aligned(a->first, 4))
    return DPRC_ERR_ALIGN;
  return DPRC_OK;
}

AttentionCall attention_call(const dprc_attention_args* a) {
  AttentionCall c;
  c.Q = a->Q;
  c.K = a->K;
  c.V = a->V;
  for (int k = 0; k < 3; ++k) {
    c.qs[k] = a->q_stride[k];
    c.ks[k] = a->k_stride[k];
    c.vs[k] = a->v_stride[k];
  }
  c.dtype = a->dtype;
  c.B = a->B;
  c.Tq = a->Tq;
  c.Tk = a->Tk;
  c.H = a->H;
  c.Hkv = a->Hkv;
  c.D = a->D;
  c.scale = a->scale;
  // (cap tanh(s / cap) is s to a half step while s < 2^-12 cap)
  c.cap = a->cap < 0x1p60f ? a->cap : 0.f;
  c.causal = a->causal != 0;
  c.slopes = a->slopes;
  c.docs = a->docs;
  c.prefix = a->prefix;
  c.lengths = a->lengths;
  c.first = a->first;
  return c;
}

}  // namespace

extern "C" {

size_t dprc_embed_plan_bytes(int64_t N, int64_t V) {
  if (N < 0 || N > kMaxTokens || V < 1 || V > kMaxVocab) return 0;
  return embed_plan_bytes(N, V);
}

size_t dprc_embed_workspace_bytes(dprc_dtype dtype, int64_t B, int64_t T, int64_t d) {
  if (!known(dtype) || B < 1 || B > kMaxSamples || T < 0 || T > kMaxTokens / B) return 0;
  if (d < 1 || d > kMaxOpWidth) return 0;
  return embed_norm_ws_bytes(dtype, B * T, d);
}

dprc_status dprc_embed_lookup(const void* W, dprc_dtype dtype, const void* tokens,
                              int token_bytes, int64_t N, int64_t V, int64_t d, float scale,
                              void* out, void* stream) {
  DPRC_NVTX_RANGE();
  if (!known(dtype) || (token_bytes != 4 && token_bytes != 8)) return DPRC_ERR_DTYPE;
  if (N < 0 || N > kMaxTokens || V < 1 || V > kMaxVocab || d < 1 || d > kMaxOpWidth)
    return DPRC_ERR_SHAPE;
  if (!finite_f(scale)) return DPRC_ERR_SHAPE;
  if (!W || (N > 0 && (!tokens || !out))) return DPRC_ERR_NULL;
  if (!aligned(W) || !aligned(tokens) || !aligned(out)) return DPRC_ERR_ALIGN;
  if (N == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  return from_cuda(launch_embed_lookup(W, dtype, tokens, token_bytes, N, V, d, scale, out,
                                       static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_embed_plan(const void* tokens, int token_bytes, int64_t N, int64_t V, void* plan,
                            size_t plan_bytes, void* stream) {
  DPRC_NVTX_RANGE();
  if (token_bytes != 4 && token_bytes != 8) return DPRC_ERR_DTYPE;
  if (N < 0 || N > kMaxTokens || V < 1 || V > kMaxVocab) return DPRC_ERR_SHAPE;
  if (N > 0 && !tokens) return DPRC_ERR_NULL;
  if (!aligned(tokens)) return DPRC_ERR_ALIGN;
  const dprc_status st = check_plan(N, V, plan, plan_bytes);
  if (st != DPRC_OK) return st;
  if (N == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  return from_cuda(launch_embed_plan(tokens, token_bytes, N, V, plan,
                                     static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_embed_norm(const void* G, dprc_dtype dtype, int64_t B, int64_t T, int64_t V,
                            int64_t d, float scale, const void* plan, size_t plan_bytes, float* n,
                            int accumulate, void* ws, size_t ws_bytes, void* stream) {
  DPRC_NVTX_RANGE();
  const dprc_status st =
      check_embed(G, dtype, B, T, V, d, scale, n, plan, plan_bytes, ws, ws_bytes);
  if (st != DPRC_OK) return st;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  EmbedCall c;
  c.G = G;
  c.dtype = dtype;
  c.B = B;
  c.T = T;
  c.V = V;
  c.d = d;
  c.scale = scale;
  c.plan = plan;
  c.accumulate = accumulate != 0;
  return from_cuda(launch_embed_norm(c, n, ws, static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_embed_grad(const void* G, dprc_dtype dtype, const float* c, int64_t B, int64_t T,
                            int64_t V, int64_t d, float scale, const void* plan,
                            size_t plan_bytes, void* dW, int accumulate, void* ws,
                            size_t ws_bytes, void* stream) {
  DPRC_NVTX_RANGE();
  const dprc_status st =
      check_embed(G, dtype, B, T, V, d, scale, dW, plan, plan_bytes, ws, ws_bytes);
  if (st != DPRC_OK) return st;
  if (!aligned(c)) return DPRC_ERR_ALIGN;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  EmbedCall e;
  e.G = G;
  e.dtype = dtype;
  e.B = B;
  e.T = T;
  e.V = V;
  e.d = d;
  e.scale = scale;
  e.plan = plan;
  e.accumulate = accumulate != 0;
  return from_cuda(launch_embed_grad(e, c, dW, ws, static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_dropout(const void* x, const void* residual, dprc_dtype dtype, int64_t N,
                         uint64_t first_element, double p, uint64_t seed, uint64_t step, void* y,
                         void* stream) {
  DPRC_NVTX_RANGE();
  if (!known(dtype)) return DPRC_ERR_DTYPE;
  if (N < 0 || !(p >= 0.0) || !(p <= 1.0)) return DPRC_ERR_SHAPE;
  if (static_cast<uint64_t>(N) > ~uint64_t(0) - first_element) return DPRC_ERR_SHAPE;
  if (N > 0 && (!x || !y)) return DPRC_ERR_NULL;
  if (!aligned(x) || !aligned(residual) || !aligned(y)) return DPRC_ERR_ALIGN;
  if (N == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  return from_cuda(launch_dropout(x, residual, dtype, N, first_element, p, seed, step, y,
                                  static_cast<cudaStream_t>(stream)));
}

size_t dprc_linear_workspace_bytes(dprc_dtype dtype, int64_t M, int64_t K, int64_t N, int grad) {
  if (check_linear(dtype, M, K, N, DPRC_ACT_NONE, 0.0) != DPRC_OK) return 0;
  return grad ? linear_grad_ws_bytes(dtype, M, K, N) : linear_ws_bytes(dtype, M, K, N);
}

dprc_status dprc_linear(const void* X, const void* W, const void* bias, const void* residual,
                        dprc_dtype dtype, int64_t M, int64_t K, int64_t N, dprc_act act, double p,
                        uint64_t seed, uint64_t step, void* Z, void* Y, void* ws, size_t ws_bytes,
                        void* stream) {
  DPRC_NVTX_RANGE();
  const dprc_status st = check_linear(dtype, M, K, N, act, p);
  if (st != DPRC_OK) return st;
  if (!W || (M > 0 && (!X || !Y))) return DPRC_ERR_NULL;
  if (!aligned(X) || !aligned(W) || !aligned(bias) || !aligned(residual) || !aligned(Z) ||
      !aligned(Y))
    return DPRC_ERR_ALIGN;
  if (!ws || ws_bytes < linear_ws_bytes(dtype, M, K, N)) return DPRC_ERR_WORKSPACE;
  if (!aligned(ws)) return DPRC_ERR_ALIGN;
  if (M == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  LinearCall c;
  c.X = X;
  c.W = W;
  c.bias = bias;
  c.res = residual;
  c.dtype = dtype;
  c.M = M;
  c.K = K;
  c.N = N;
  c.act = act;
  c.p = p;
  c.seed = seed;
  c.step = step;
  c.Z = Z;
  c.Y = Y;
  return from_cuda(launch_linear(c, ws, static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_linear_grad(const void* dY, const void* X, const void* W, const void* Z,
                             dprc_dtype dtype, int64_t M, int64_t K, int64_t N, dprc_act act,
                             double p, uint64_t seed, uint64_t step, void* dX, void* dW, void* db,
                             void* dZ, void* ws, size_t ws_bytes, void* stream) {
  DPRC_NVTX_RANGE();
  const dprc_status st = check_linear(dtype, M, K, N, act, p);
  if (st != DPRC_OK) return st;
  if (!dX && !dW && !db && !dZ) return DPRC_ERR_NULL;
  if (M > 0 && (!dY || (act != DPRC_ACT_NONE && !Z) || (dW && !X) || (dX && !W)))
    return DPRC_ERR_NULL;
  if (!aligned(dY) || !aligned(X) || !aligned(W) || !aligned(Z) || !aligned(dX) || !aligned(dW) ||
      !aligned(db) || !aligned(dZ))
    return DPRC_ERR_ALIGN;
  if (!ws || ws_bytes < linear_grad_ws_bytes(dtype, M, K, N)) return DPRC_ERR_WORKSPACE;
  if (!aligned(ws)) return DPRC_ERR_ALIGN;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  LinearGradCall c;
  c.dY = dY;
  c.X = X;
  c.W = W;
  c.Z = Z;
  c.dtype = dtype;
  c.M = M;
  c.K = K;
  c.N = N;
  c.act = act;
  c.p = p;
  c.seed = seed;
  c.step = step;
  c.dX = dX;
  c.dW = dW;
  c.db = db;
  c.dZ = dZ;
  return from_cuda(launch_linear_grad(c, ws, static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_layernorm(const void* X, const void* weight, const void* bias, dprc_dtype dtype,
                           int64_t B, int64_t T, int64_t d, float eps, int center, void* Y,
                           float* stats, void* stream) {
  DPRC_NVTX_RANGE();
  const dprc_status st = check_layernorm(dtype, B, T, d);
  if (st != DPRC_OK) return st;
  if (!finite_f(eps) || eps < 0.f) return DPRC_ERR_SHAPE;
  if (T > 0 && (!X || !Y)) return DPRC_ERR_NULL;
  if (!aligned(X) || !aligned(weight) || !aligned(bias) || !aligned(Y) || !aligned(stats))
    return DPRC_ERR_ALIGN;
  if (T == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  LayernormCall c;
  c.X = X;
  c.weight = weight;
  c.bias = bias;
  c.dtype = dtype;
  c.B = B;
  c.T = T;
  c.d = d;
  c.eps = eps;
  c.center = center != 0;
  c.Y = Y;
  c.stats = stats;
  return from_cuda(launch_layernorm(c, static_cast<cudaStream_t>(stream)));
}

size_t dprc_layernorm_workspace_bytes(int64_t B, int64_t T, int64_t d, int norms) {
  if (check_layernorm(DPRC_F32, B, T, d) != DPRC_OK) return 0;
  return layernorm_grad_ws_bytes(B, T, d, norms);
}

dprc_status dprc_layernorm_grad(const void* dY, const void* X, const float* stats,
                                const void* weight, dprc_dtype dtype, int64_t B, int64_t T,
                                int64_t d, int center, void* dX, void* dW, void* db, float* n,
                                int norm_of_bias, int accumulate, const float* c, void* ws,
                                size_t ws_bytes, void* stream) {
  DPRC_NVTX_RANGE();
  const dprc_status st = check_layernorm(dtype, B, T, d);
  if (st != DPRC_OK) return st;
  if (!dX && !dW && !db && !n) return DPRC_ERR_NULL;
  if (T > 0 && (!dY || !X || !stats)) return DPRC_ERR_NULL;
  if (!aligned(dY) || !aligned(X) || !aligned(stats) || !aligned(weight) || !aligned(dX) ||
      !aligned(dW) || !aligned(db) || !element_aligned(n, 4) || !element_aligned(c, 4))
    return DPRC_ERR_ALIGN;
  if (!ws || ws_bytes < layernorm_grad_ws_bytes(B, T, d, n != nullptr)) return DPRC_ERR_WORKSPACE;
  if (!aligned(ws)) return DPRC_ERR_ALIGN;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  LayernormGradCall g;
  g.dY = dY;
  g.X = X;
  g.weight = weight;
  g.stats = stats;
  g.c = c;
  g.dtype = dtype;
  g.B = B;
  g.T = T;
  g.d = d;
  g.center = center != 0;
  g.norm_of_bias = norm_of_bias != 0;
  g.accumulate = accumulate != 0;
  g.dX = dX;
  g.dW = dW;
  g.db = db;
  g.n = n;
  return from_cuda(launch_layernorm_grad(g, ws, static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_rotary(const void* X, const int64_t* x_stride, dprc_dtype dtype, int64_t B,
                        int64_t T, int64_t H, int64_t D, const void* positions,
                        int position_bytes, int axes, const int64_t* sections,
                        const double* freqs, int interleaved, int inverse, void* out,
                        const int64_t* out_stride, void* stream) {
  DPRC_NVTX_RANGE();
  if (!known(dtype) || (position_bytes != 4 && position_bytes != 8)) return DPRC_ERR_DTYPE;
  if (B < 0 || T < 0 || H < 1 || D < 1 || D > kMaxRotWidth || H > kMaxSamples)
    return DPRC_ERR_SHAPE;
  if (B > 0 && T > kMaxTokens / B) return DPRC_ERR_SHAPE;
  if (axes < 1 || axes > kMaxRotAxes) return DPRC_ERR_SHAPE;
  if (!sections || !x_stride || !out_stride) return DPRC_ERR_NULL;
  if (!strides_ok(x_stride) || !strides_ok(out_stride)) return DPRC_ERR_SHAPE;
  int64_t pairs = 0;
  for (int k = 0; k < axes; ++k) {
    if (sections[k] < 0 || sections[k] > D) return DPRC_ERR_SHAPE;
    pairs += sections[k];
  }
  if (2 * pairs > D || !apart(out_stride, B, T, H, D)) return DPRC_ERR_SHAPE;
  if (B * T > 0 && (!X || !out || (pairs > 0 && (!positions || !freqs)))) return DPRC_ERR_NULL;
  const size_t e = size_of(dtype);
  if (!element_aligned(X, e) || !element_aligned(out, e) ||
      !element_aligned(positions, position_bytes) || !element_aligned(freqs, 8))
    return DPRC_ERR_ALIGN;
  if (B * T == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  RotaryCall c;
  c.X = X;
  c.dtype = dtype;
  c.B = B;
  c.T = T;
  c.H = H;
  c.D = D;
  c.pairs = pairs;
  for (int k = 0; k < 3; ++k) {
    c.xs[k] = x_stride[k];
    c.os[k] = out_stride[k];
  }
  c.positions = positions;
  c.position_bytes = position_bytes;
  c.axes = axes;
  for (int k = 0; k < axes; ++k) c.sections[k] = sections[k];
  c.freqs = freqs;
  c.interleaved = interleaved != 0;
  c.inverse = inverse != 0;
  c.out = out;
  return from_cuda(launch_rotary(c, static_cast<cudaStream_t>(stream)));
}

size_t dprc_attention_workspace_bytes(const dprc_attention_args* a, int grad) {
  if (check_attention(a) != DPRC_OK) return 0;
  const AttentionCall c = attention_call(a);
  return grad ? attention_grad_ws_bytes(c) : attention_ws_bytes(c);
}

dprc_status dprc_attention(const dprc_attention_args* a, void* out, float* lse, void* ws,
                           size_t ws_bytes, void* stream) {
  DPRC_NVTX_RANGE();
  dprc_status st = check_attention(a);
  if (st == DPRC_OK) st = check_attention_inputs(a);
  if (st != DPRC_OK) return st;
  if (a->Tq > 0 && !out) return DPRC_ERR_NULL;
  if (!aligned(out) || !element_aligned(lse, 4)) return DPRC_ERR_ALIGN;
  const AttentionCall c = attention_call(a);
  if (!ws || ws_bytes < attention_ws_bytes(c)) return DPRC_ERR_WORKSPACE;
  if (!aligned(ws)) return DPRC_ERR_ALIGN;
  if (a->Tq == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  return from_cuda(launch_attention(c, out, lse, ws, static_cast<cudaStream_t>(stream)));
}

dprc_status dprc_attention_grad(const dprc_attention_args* a, const void* dO,
                                const int64_t* do_stride, const void* O, const int64_t* o_stride,
                                const float* lse, void* dQ, const int64_t* dq_stride, void* dK,
                                const int64_t* dk_stride, void* dV, const int64_t* dv_stride,
                                void* ws, size_t ws_bytes, void* stream) {
  DPRC_NVTX_RANGE();
  dprc_status st = check_attention(a);
  if (st == DPRC_OK) st = check_attention_inputs(a);
  if (st != DPRC_OK) return st;
  if (!dQ && !dK && !dV) return DPRC_ERR_NULL;
  if ((dQ && !dq_stride) || (dK && !dk_stride) || (dV && !dv_stride)) return DPRC_ERR_NULL;
  if ((dQ && !strides_ok(dq_stride)) || (dK && !strides_ok(dk_stride)) ||
      (dV && !strides_ok(dv_stride)))
    return DPRC_ERR_SHAPE;
  if ((dQ && !apart(dq_stride, a->B, a->Tq, a->H, a->D)) ||
      (dK && !apart(dk_stride, a->B, a->Tk, a->Hkv, a->D)) ||
      (dV && !apart(dv_stride, a->B, a->Tk, a->Hkv, a->D)))
    return DPRC_ERR_SHAPE;
  if (a->Tq > 0 && (!dO || !O || !lse || !do_stride || !o_stride)) return DPRC_ERR_NULL;
  if (a->Tq > 0 && (!strides_ok(do_stride) || !strides_ok(o_stride))) return DPRC_ERR_SHAPE;
  const size_t e = size_of(a->dtype);
  if (!element_aligned(dO, e) || !element_aligned(O, e) || !element_aligned(lse, 4) ||
      !element_aligned(dQ, e) || !element_aligned(dK, e) || !element_aligned(dV, e))
    return DPRC_ERR_ALIGN;
  AttentionGradCall g;
  g.f = attention_call(a);
  if (!ws || ws_bytes < attention_grad_ws_bytes(g.f)) return DPRC_ERR_WORKSPACE;
  if (!aligned(ws)) return DPRC_ERR_ALIGN;
  if (a->Tq == 0 && a->Tk == 0) return DPRC_OK;
  if (!device_supported()) return DPRC_ERR_DEVICE;
  g.dO = dO;
  g.O = O;
  g.lse = lse;
  g.dQ = dQ;
  g.dK = dK;
  g.dV = dV;
  for (int k = 0; k < 3; ++k) {
    if (a->Tq > 0) {
      g.dos[k] = do_stride[k];
      g.os[k] = o_stride[k];
    }
    if (dQ) g.dqs[k] = dq_stride[k];
    if (dK) g.dks[k] = dk_stride[k];
    if (dV) g.dvs[k] = dv_stride[k];
  }
  return from_cuda(launch_attention_grad(g, ws, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
