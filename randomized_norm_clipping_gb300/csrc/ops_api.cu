// libdprc C ABI of the operators around the norm path (the embedding, dropout,
// the linear map): argument checks, then the launchers.

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

}  // extern "C"
