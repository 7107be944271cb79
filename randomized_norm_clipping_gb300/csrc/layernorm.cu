// Layer normalisation and its form without the mean (RMS), forward and
// backward, with the per-sample norms of its parameters' gradients.
//
//   y  = w xh + b,  xh = (x - mu) r,  r = (mean((x - mu)^2) + eps)^(-1/2)
//   dx = r (g - mean(g) - xh mean(g xh)),  g = dy w     (without mean(g) for RMS)
//   W_i = sum_t dy_it xh_it,  b_i = sum_t dy_it         (of sample i)
//   n_i = ||W_i||^2 (+ ||b_i||^2),  dw = sum_i c_i W_i,  db = sum_i c_i b_i
//
// Bound by bytes: each pass reads its tensors once; a row's values stay in the
// registers of the threads that share it, and the sums over rows in those of the
// threads that own a column.
//
// A row is shared by G threads (a power of two), each of which holds up to kNv
// accesses of kE elements: 16 bytes where the width allows, else single
// elements.  Up to 32 threads sum by shuffles; more through shared memory.

#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "vec.cuh"

namespace dprc {
namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWide = 512;  // threads of a CTA of the backward pass on wide rows
constexpr int kMaxWarps = kLnWide / 32;

// Sums of kN values over the G threads of a row, the same in all of them.  The
// order is fixed.  buf: [2][kMaxWarps][kN], the halves in turn, so that one
// barrier is enough.
template <int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], int G, float* buf, int& turn) {
  const int lim = G < 32 ? G : 32;
  for (int o = 1; o < lim; o <<= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (G <= 32) return;
  const int warp = threadIdx.x >> 5, per = G >> 5;
  float* b = buf + (turn & 1) * kMaxWarps * kN;
  ++turn;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) b[warp * kN + i] = v[i];
  __syncthreads();
  const int w0 = warp / per * per;
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = 0.f;
  for (int w = 0; w < per; ++w)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += b[(w0 + w) * kN + i];
}

// The variance is summed of the differences from the mean, in registers: no
// cancellation of large means.  What the mean lost in its rounding is the mean of
// those differences, and taken off them too: two values that agree to a half
// step of each other still come out at full accuracy.
template <typename T, int kE, int kNv>
__global__ void __launch_bounds__(kLnThreads)
    layernorm_kernel(const T* x, const T* w, const T* b, long long rows, int d, int G, float eps,
                     int center, T* y, float2* stats) {
  __shared__ float buf[2 * kMaxWarps * 2];
  pdl_launch_dependents();
  pdl_wait();
  int turn = 0;
  const int t = threadIdx.x & (G - 1);
  const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / G) + threadIdx.x / G;
  const bool mine = row < rows;
  const T* xr = x + (mine ? row : 0) * d;
  Raw<T, kE> raw[kNv];
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const int c = (k * G + t) * kE;
    if (mine && c < d) raw[k].load(xr + c); else raw[k].zero();
  }
  const float inv = 1.f / static_cast<float>(d);
  float mean = 0.f;
  if (center) {
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      float v[kE];
      raw[k].get(v);
#pragma unroll
      for (int e = 0; e < kE; ++e) s[0] += v[e];
    }
    row_sum<1>(s, G, buf, turn);
    mean = s[0] * inv;
  }
  float q[2] = {0.f, 0.f};  // sums of the differences (what the mean's rounding left) and squares
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const int c = (k * G + t) * kE;
    if (c < d) {
      float v[kE];
      raw[k].get(v);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        q[0] += v[e] - mean;
        q[1] = fmaf(v[e] - mean, v[e] - mean, q[1]);
      }
    }
  }
  row_sum<2>(q, G, buf, turn);
  const float left = center ? q[0] * inv : 0.f;
  const float rstd = 1.f / sqrtf(fmaxf(q[1] * inv - left * left, 0.f) + eps);
  if (!mine) return;
  if (stats != nullptr && t == 0) stats[row] = make_float2(mean + left, rstd);
  T* yr = y + row * d;
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const int c = (k * G + t) * kE;
    if (c >= d) continue;
    float v[kE], g[kE];
    raw[k].get(v);
#pragma unroll
    for (int e = 0; e < kE; ++e) v[e] = (v[e] - mean - left) * rstd;
    if (w != nullptr) {
      Raw<T, kE> u;
      u.load(w + c);
      u.get(g);
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] *= g[e];
    }
    if (b != nullptr) {
      Raw<T, kE> u;
      u.load(b + c);
      u.get(g);
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] += g[e];
    }
    store_row<kE>(yr + c, v);
  }
}

struct LnGradArgs {
  const float2* stats;
  const float* c;        // factors of the samples' rows, or null: 1
  long long rows;        // of a sample (blockIdx.y)
  long long per_chunk;   // rows of a CTA
  long long T;           // rows of a sample of c
  int d, G, center, sums;
  float* part;           // [samples][chunks][2][d]
};

// kRows rows of a group at a time, so that one round of sums serves them.
// kReload: a row's values are read again (from L1) after the sums, not kept.
template <typename T, int kE, int kNv, int kRows, bool kReload>
__global__ void __launch_bounds__(kReload ? kLnWide : kLnThreads)
    layernorm_grad_kernel(const T* dy, const T* x, const T* w, T* dx, const LnGradArgs a) {
  __shared__ float buf[2 * kMaxWarps * 2 * kRows];
  __shared__ float fold[kReload ? 1 : kLnThreads];
  pdl_launch_dependents();
  pdl_wait();
  int turn = 0;
  const int d = a.d, G = a.G;
  const int t = threadIdx.x & (G - 1), groups = blockDim.x / G, grp = threadIdx.x / G;
  const long long base = blockIdx.y * a.rows;  // the sample's first row
  const long long r0 = blockIdx.x * a.per_chunk;
  const long long r1 = min(r0 + a.per_chunk, a.rows);
  const float inv = 1.f / static_cast<float>(d);
  float wsum[kNv * kE], bsum[kNv * kE];
#pragma unroll
  for (int i = 0; i < kNv * kE; ++i) wsum[i] = bsum[i] = 0.f;

  for (long long rr = r0; rr < r1; rr += groups * kRows) {  // the same for a CTA
    Raw<T, kE> xv[kRows][kNv], gv[kRows][kNv];
    float2 st[kRows];
    float s[2 * kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const long long r = rr + grp * kRows + j;
      const bool mine = r < r1;
      const long long row = base + (mine ? r : r0);
      st[j] = mine ? ld_once(a.stats + row) : make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        const int c = (k * G + t) * kE;
        if (mine && c < d) {
          xv[j][k].load(x + row * d + c);
          gv[j][k].load(dy + row * d + c);
        } else {
          xv[j][k].zero();
          gv[j][k].zero();
        }
      }
    }
    if (dx != nullptr) {
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        s[2 * j] = s[2 * j + 1] = 0.f;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
          const int c = (k * G + t) * kE;
          if (c >= d) continue;
          float xf[kE], gf[kE], wf[kE];
          xv[j][k].get(xf);
          gv[j][k].get(gf);
          if (w != nullptr) {
            Raw<T, kE> u;
            u.load(w + c);
            u.get(wf);
          }
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const float g = w != nullptr ? gf[e] * wf[e] : gf[e];
            s[2 * j] += g;
            s[2 * j + 1] = fmaf(g, (xf[e] - st[j].x) * st[j].y, s[2 * j + 1]);
          }
        }
      }
      row_sum<2 * kRows>(s, G, buf, turn);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const long long r = rr + grp * kRows + j;
      if (r >= r1) continue;
      const long long row = base + r;
      const float mg = a.center ? s[2 * j] * inv : 0.f, mh = s[2 * j + 1] * inv;
      const float f = a.c != nullptr ? a.c[row / a.T] : 1.f;
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        const int c = (k * G + t) * kE;
        if (c >= d) continue;
        float xf[kE], gf[kE], wf[kE], out[kE];
        if constexpr (kReload) {
          Raw<T, kE> u;
          u.load(x + row * d + c);
          u.get(xf);
          u.load(dy + row * d + c);
          u.get(gf);
        } else {
          xv[j][k].get(xf);
          gv[j][k].get(gf);
        }
        if (w != nullptr) {
          Raw<T, kE> u;
          u.load(w + c);
          u.get(wf);
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const float xh = (xf[e] - st[j].x) * st[j].y;
          const float g = w != nullptr ? gf[e] * wf[e] : gf[e];
          out[e] = (g - mg - xh * mh) * st[j].y;
          const float gc = gf[e] * f;
          wsum[k * kE + e] = fmaf(gc, xh, wsum[k * kE + e]);
          bsum[k * kE + e] += gc;
        }
        if (dx != nullptr) store_row<kE>(dx + row * d + c, out);
      }
    }
  }
  if (!a.sums) return;
  // the groups of the CTA in order
  float* part = a.part + (blockIdx.y * static_cast<long long>(gridDim.x) + blockIdx.x) * 2 * d;
#pragma unroll
  for (int i = 0; i < 2 * kNv * kE; ++i) {
    float v = i < kNv * kE ? wsum[i < kNv * kE ? i : 0] : bsum[i < kNv * kE ? 0 : i - kNv * kE];
    if (!kReload && groups > 1) {
      __syncthreads();
      fold[threadIdx.x] = v;
      __syncthreads();
      if (grp != 0) continue;
      for (int q = 1; q < groups; ++q) v += fold[q * G + t];
    }
    const int m = i % (kNv * kE), c = ((m / kE) * G + t) * kE + m % kE;
    if (c < d && DPRC_IN(c >= 0)) part[(i < kNv * kE ? 0 : d) + c] = v;
  }
}

constexpr int kFinWarps = 8;

// The samples' sums over their chunks, 32 columns of the weight's (blockIdx.y 0)
// or the bias's a CTA: their squares, and the sum over the samples times c.  A
// warp takes every eighth chunk of a sample (few samples) or every eighth sample.
template <typename T>
__global__ void __launch_bounds__(32 * kFinWarps)
    layernorm_finish_kernel(const float* part, const float* c, int B, int chunks, int d, T* dw,
                            T* db, float* npart, int norm_parts) {
  __shared__ float sm[2][kFinWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane, which = blockIdx.y;
  const bool in = col < d;
  const float* p = part + which * static_cast<long long>(d) + (in ? col : 0);
  const long long step = 2ll * d;
  const bool norm = npart != nullptr && which < norm_parts;
  float* np = npart + (which * static_cast<long long>(gridDim.x) + blockIdx.x) * B;
  float total = 0.f;
  const auto chunk_sum = [&](long long i, int first, int stride) {
    float s = 0.f;
    const float* q = p + i * chunks * step;
    int k = first;
    for (; k + 3 * stride < chunks; k += 4 * stride) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = ld_l2(q + (k + u * stride) * step);
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; k < chunks; k += stride) s += ld_l2(q + k * step);
    return in ? s : 0.f;
  };
  const auto finish = [&](long long i, float s) {
    total = fmaf(c != nullptr ? ld_l2(c + i) : 1.f, s, total);
    if (norm) {
      float q = s * s;
      for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      if (lane == 0) np[i] = q;
    }
  };
  if (B < 8 * kFinWarps) {
    for (int i = 0; i < B; ++i) {
      sm[i & 1][warp][lane] = chunk_sum(i, warp, kFinWarps);
      __syncthreads();
      if (warp == i % kFinWarps) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kFinWarps; ++w) s += sm[i & 1][w][lane];
        finish(i, s);
      }
    }
  } else {
    for (int i = warp; i < B; i += kFinWarps) finish(i, chunk_sum(i, 0, 1));
  }
  __syncthreads();
  sm[0][warp][lane] = total;
  __syncthreads();
  if (warp == 0 && in) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kFinWarps; ++w) s += sm[0][w][lane];
    T* out = which == 0 ? dw : db;
    if (out != nullptr) out[col] = T(s);
  }
}

// n_i (+)= the sum of its parts in a fixed order, a warp a sample.
__global__ void __launch_bounds__(256)
    layernorm_norm_kernel(const float* npart, int parts, int B, float* n, int accumulate) {
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= B) return;
  float s = 0.f;
  for (int k = lane; k < parts; k += 32) s += ld_l2(npart + static_cast<long long>(k) * B + i);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) n[i] = accumulate ? n[i] + s : s;
}

int pow2_at_least(int64_t v, int lo, int hi) {
  int g = lo;
  while (g < v && g < hi) g *= 2;
  return g;
}

template <typename T>
bool whole_vectors(int64_t d) {
  return d % kVec16<T> == 0;
}

// Chunks of rows: as many CTAs as are resident twice over, at least 8 rows each.
struct LnPlan {
  int64_t samples, rows, chunks, per_chunk;
};
LnPlan plan_grad(int64_t B, int64_t T, bool by_sample) {
  LnPlan p;
  p.samples = by_sample ? B : 1;
  p.rows = by_sample ? T : B * T;
  const int64_t want = std::max<int64_t>(1, 4 * 152 / p.samples);
  p.per_chunk = std::max<int64_t>(16, (p.rows + want - 1) / want);
  p.chunks = std::max<int64_t>(1, (p.rows + p.per_chunk - 1) / p.per_chunk);
  return p;
}

template <typename T>
cudaError_t forward(const LayernormCall& c, cudaStream_t s) {
  const int64_t rows = c.B * c.T, d = c.d;
  const T* x = static_cast<const T*>(c.X);
  const T* w = static_cast<const T*>(c.weight);
  const T* b = static_cast<const T*>(c.bias);
  T* y = static_cast<T*>(c.Y);
  constexpr int kV = kVec16<T>;
  const bool vec = whole_vectors<T>(d);
  const int e = vec ? kV : 1;
  const int64_t acc = (d + e - 1) / e;  // accesses of a row
  // a warp or less a row while its share fits 64 registers, else a CTA
  const int G = acc * e <= 32 * 64 ? pow2_at_least(acc, 8, 32) : kLnThreads;
  const int64_t nv = (acc + G - 1) / G;
  const int64_t per = kLnThreads / G;
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per));
  float2* st = reinterpret_cast<float2*>(c.stats);
  const auto go = [&](auto kernel) {
    return launch_after(kernel, grid, kLnThreads, 1, s, 0, x, w, b, static_cast<long long>(rows),
                        static_cast<int>(d), G, c.eps, c.center, y, st);
  };
  if (vec) {
    if (nv <= 1) return go(layernorm_kernel<T, kV, 1>);
    if (nv <= 2) return go(layernorm_kernel<T, kV, 2>);
    if (nv <= 4) return go(layernorm_kernel<T, kV, 4>);
    if (nv <= 8) return go(layernorm_kernel<T, kV, 8>);
    if constexpr (kV == 4) return go(layernorm_kernel<T, kV, 16>);
  }
  if (nv <= 4) return go(layernorm_kernel<T, 1, 4>);
  if (nv <= 16) return go(layernorm_kernel<T, 1, 16>);
  return go(layernorm_kernel<T, 1, 64>);
}

template <typename T>
cudaError_t backward(const LayernormGradCall& c, void* ws, cudaStream_t s) {
  const bool by_sample = c.n != nullptr;
  const LnPlan p = plan_grad(c.B, c.T, by_sample);
  const int64_t d = c.d;
  constexpr int kV = kVec16<T>;
  const bool vec = whole_vectors<T>(d);
  const int e = vec ? kV : 1;
  const int64_t acc = (d + e - 1) / e;
  const bool sums = c.dW != nullptr || c.db != nullptr || by_sample;
  LnGradArgs a;
  a.stats = reinterpret_cast<const float2*>(c.stats);
  a.c = by_sample ? nullptr : c.c;  // (by sample, the finishing step takes it)
  a.rows = p.rows;
  a.per_chunk = p.per_chunk;
  a.T = std::max<int64_t>(1, c.T);
  a.d = static_cast<int>(d);
  a.center = c.center;
  a.sums = sums;
  a.part = static_cast<float*>(ws);
  // columns of a thread: up to 16 in registers with their rows; wide rows have
  // 512 threads, 32 columns each, and are read again behind the sums
  const bool wide = acc * e > kLnThreads * 16;
  a.G = wide ? kLnWide : pow2_at_least(acc, 8, kLnThreads);
  const int threads = wide ? kLnWide : kLnThreads;
  const int64_t nv = (acc + a.G - 1) / a.G;
  const dim3 grid(static_cast<unsigned>(p.chunks), static_cast<unsigned>(p.samples));
  const auto go = [&](auto kernel) {
    return launch_after(kernel, grid, threads, 1, s, 0, static_cast<const T*>(c.dY),
                        static_cast<const T*>(c.X), static_cast<const T*>(c.weight),
                        static_cast<T*>(c.dX), a);
  };
  cudaError_t err;
  if (vec) {
    if (wide) err = go(layernorm_grad_kernel<T, kV, 32 / kV, 1, true>);
    else if (nv <= 1) err = go(layernorm_grad_kernel<T, kV, 1, 2, false>);
    else if (nv <= 2) err = go(layernorm_grad_kernel<T, kV, 2, 2, false>);
    else err = go(layernorm_grad_kernel<T, kV, 16 / kV, 2, false>);
  } else {
    if (wide) err = go(layernorm_grad_kernel<T, 1, 32, 1, true>);
    else if (nv <= 4) err = go(layernorm_grad_kernel<T, 1, 4, 2, false>);
    else err = go(layernorm_grad_kernel<T, 1, 16, 2, false>);
  }
  if (err != cudaSuccess || !sums) return err;
  const int tiles = static_cast<int>((d + 31) / 32);
  float* npart = by_sample ? a.part + p.samples * p.chunks * 2 * d : nullptr;
  const int parts = c.norm_of_bias ? 2 : 1;
  const float* cf = by_sample ? c.c : nullptr;
  const int which = c.db != nullptr || (by_sample && c.norm_of_bias) ? 2 : 1;
  err = launch_after(layernorm_finish_kernel<T>, dim3(tiles, which), 32 * kFinWarps, 1, s, 0,
                     static_cast<const float*>(a.part), cf, static_cast<int>(p.samples),
                     static_cast<int>(p.chunks), static_cast<int>(d), static_cast<T*>(c.dW),
                     static_cast<T*>(c.db), npart, parts);
  if (err != cudaSuccess || !by_sample) return err;
  return launch_after(layernorm_norm_kernel, dim3(static_cast<unsigned>((c.B + 7) / 8)), 256, 1, s,
                      0, static_cast<const float*>(npart), tiles * parts, static_cast<int>(c.B),
                      c.n, c.accumulate);
}

}  // namespace

size_t layernorm_grad_ws_bytes(int64_t B, int64_t T, int64_t d, int with_norms) {
  const LnPlan p = plan_grad(B, T, with_norms != 0);
  const size_t part = static_cast<size_t>(p.samples) * p.chunks * 2 * d * 4;
  const size_t np = with_norms ? static_cast<size_t>((d + 31) / 32) * 2 * B * 4 : 0;
  return part + np + 16;
}

cudaError_t launch_layernorm(const LayernormCall& c, cudaStream_t s) {
  return c.dtype == DPRC_F32 ? forward<float>(c, s) : forward<__nv_bfloat16>(c, s);
}

cudaError_t launch_layernorm_grad(const LayernormGradCall& c, void* ws, cudaStream_t s) {
  return c.dtype == DPRC_F32 ? backward<float>(c, ws, s) : backward<__nv_bfloat16>(c, ws, s);
}

cudaError_t read_device_error_layernorm(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

}  // namespace dprc
