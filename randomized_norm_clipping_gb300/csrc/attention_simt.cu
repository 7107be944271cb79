// Attention on the CUDA cores, in fp32: fp32 inputs, and bf16 ones whose widths
// or strides the tensor copies do not take.  The same sums as the tensor-core kernels
// (attention_tc.cu), in tiles of rows and 64 keys.
//
// A CTA has 16 groups of 16 threads.  A group has kR rows of the tile (4, or fewer where
// that leaves SMs idle); a thread forms kR x 4 products of rows and keys (keys 16 apart,
// so that a warp reads whole lines of banks), four of the width at a time, then the
// same rows times four of every 64 columns of the values.  A row's weights are written and
// read by one group, so a warp's step orders them.  Bound by fp32 operations and the loads of
// shared memory that feed them.  Measured, fp32, causal, 2 x 1024 tokens of 16 heads of 64
// over 4: 176 us forward, 1.08 ms backward.  (Eight groups of eight rows read less
// shared memory, but two warps a scheduler did not cover its latency: the gradient of
// 2 x 1024 tokens, 16 heads of 64, took 1.66 ms.)

#include <algorithm>

#include "attention.cuh"
#include "vec.cuh"

namespace dprc {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;
constexpr int kN = 64;
constexpr int kPad = 4;

__device__ __forceinline__ float4 four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const float* p) {
  return ld_once(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = ld_once(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}

// Rows of width D from src(r) (null: zeros) into dst [kRows][kD + kPad], zeros behind n
// rows and D columns.  vec: rows are whole accesses of four.
template <typename T, int kRows, int kD, typename Src>
__device__ __forceinline__ void load_tile(float* dst, int n, int D, bool vec, Src src) {
  constexpr int kLanes = kD / 4, kStep = kThreads / kLanes;
  const int c = (threadIdx.x % kLanes) * 4;
#pragma unroll 4
  for (int r = threadIdx.x / kLanes; r < kRows; r += kStep) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const T* p = r < n ? src(r) : nullptr;
    if (p != nullptr && DPRC_IN(n <= kRows && (!vec || reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0))) {
      if (vec) {
        if (c < D) v = load4(p + c);
      } else {
        if (c < D) v.x = to_f32<T>(ld_once(p + c));
        if (c + 1 < D) v.y = to_f32<T>(ld_once(p + c + 1));
        if (c + 2 < D) v.z = to_f32<T>(ld_once(p + c + 2));
        if (c + 3 < D) v.w = to_f32<T>(ld_once(p + c + 3));
      }
    }
    *reinterpret_cast<float4*>(dst + r * (kD + kPad) + c) = v;
  }
}

// acc[i][j] += row i of a times row 16 j of b, over the width (rows kD + kPad apart).
template <int kR, int kC, int kD>
__device__ __forceinline__ void dots(const float* a, const float* b, int D, float (&acc)[kR][kC]) {
#pragma unroll(kR <= 2 ? 4 : 2)
  for (int d = 0; d < D; d += 4) {
    float4 y[kC];
#pragma unroll
    for (int j = 0; j < kC; ++j) y[j] = four(b + j * 16 * (kD + kPad) + d);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const float4 x = four(a + i * (kD + kPad) + d);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        acc[i][j] = fmaf(x.x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x.y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x.z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x.w, y[j].w, acc[i][j]);
      }
    }
  }
}

// kR weights from p.
template <int kR>
__device__ __forceinline__ void load_weights(const float* p, float (&w)[kR]) {
  if constexpr (kR >= 4) {
#pragma unroll
    for (int i = 0; i < kR; i += 4) {
      const float4 v = four(p + i);
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  } else if constexpr (kR == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *p;
  }
}
template <int kR>
__device__ __forceinline__ void store_weights(float* p, const float (&w)[kR]) {
  if constexpr (kR >= 4) {
#pragma unroll
    for (int i = 0; i < kR; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else if constexpr (kR == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(w[0], w[1]);
  } else {
    *p = w[0];
  }
}

// acc[i][4 q ..] += sum over n terms of weight i (wt [n][kW]) and columns 64 q + 4 tx of v.
template <int kR, int kO, int kD, int kW>
__device__ __forceinline__ void add_rows(const float* wt, const float* v, int n,
                                         float (&acc)[kR][4 * kO]) {
#pragma unroll(kR <= 2 ? 8 : 4)
  for (int j = 0; j < n; ++j) {
    float w[kR];
    load_weights<kR>(wt + j * kW, w);
#pragma unroll
    for (int q = 0; q < kO; ++q) {
      const float4 y = four(v + j * (kD + kPad) + q * 64);
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        acc[i][4 * q] = fmaf(w[i], y.x, acc[i][4 * q]);
        acc[i][4 * q + 1] = fmaf(w[i], y.y, acc[i][4 * q + 1]);
        acc[i][4 * q + 2] = fmaf(w[i], y.z, acc[i][4 * q + 2]);
        acc[i][4 * q + 3] = fmaf(w[i], y.w, acc[i][4 * q + 3]);
      }
    }
  }
}

__device__ __forceinline__ float half_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ int block_max(int v, int* sm) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) v = max(v, sm[w]);
  __syncthreads();
  return v;
}

// The score of a product z = q k scale, and the cap's slope by z.
__device__ __forceinline__ float capped(const AttnArgs& a, float z, float* slope) {
  if (a.cap <= 0.f) {
    *slope = 1.f;
    return z;
  }
  const float t = tanhf(z / a.cap);  // (1 - 2 / (1 + exp) is off by 2^-24 cap: too much of large caps)
  *slope = 1.f - t * t;
  return t * a.cap;
}

// Whether any row with documents in [lo, hi] may see a key of this span.
__device__ __forceinline__ bool span_meets(const AttnArgs& a, int b, int tile, int lo, int hi) {
  if (a.docs == nullptr) return true;
  const DocSpan s = a.spans[static_cast<long long>(b) * ((a.Tk + kDocSpan - 1) / kDocSpan) + tile];
  return s.lo <= hi && lo <= s.hi;
}

template <int kD, int kR>
constexpr int kFwdSmem =
    4 * ((kGroups * kR + 2 * kN) * (kD + kPad) + kN * (kGroups * kR + kPad) + kN + 8);

template <typename T, int kD, int kR>
__global__ void __launch_bounds__(kThreads) attention_simt_kernel(const AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int kM = kGroups * kR;          // rows of the tile
  constexpr int kO = kD / 64;         // fours of the values' columns of a thread
  constexpr int kRow = kD + kPad;
  float* qs = sm;                     // [kM][kRow]
  float* ks = qs + kM * kRow;         // [kN][kRow]
  float* vs = ks + kN * kRow;         // [kN][kRow]
  float* pt = vs + kN * kRow;         // [kN][kM + kPad]
  int* kdoc = reinterpret_cast<int*>(pt + kN * (kM + kPad));  // [kN]
  int* red = kdoc + kN;               // [8]
  pdl_launch_dependents();
  pdl_wait();
  const int bhs = a.B * a.Hkv, bh = blockIdx.x % bhs, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  const int rows = a.Tq * a.G;
  const int p0 = (gridDim.x / bhs - 1 - blockIdx.x / bhs) * kM;  // (the longest rows first)
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const T* Q = static_cast<const T*>(a.Q) + b * a.qb;
  const T* K = static_cast<const T*>(a.K) + b * a.kb + hk * a.kh;
  const T* V = static_cast<const T*>(a.V) + b * a.vb + hk * a.vh;
  const bool vec = a.vec != 0;

  load_tile<T, kM, kD>(qs, min(kM, rows - p0), a.D, vec, [&](int r) {
    const int p = p0 + r, t = p / a.G;
    return Q + t * a.qt + (hk * a.G + p - t * a.G) * a.qh;
  });
  RowSees see[kR];
  float slope[kR];
  int top = 0, dlo = 0x7fffffff, dhi = -1;
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int p = p0 + ty * kR + i, t = p / a.G;
    see[i].pos = see[i].lim = 0;
    see[i].doc = -1;
    slope[i] = 0.f;
    if (p < rows) {
      see[i] = attn_row(a, b, t, keys, first);
      if (a.slopes != nullptr) slope[i] = a.slopes[hk * a.G + p - t * a.G];
    }
    top = max(top, see[i].lim);
    if (see[i].doc >= 0) {
      dlo = min(dlo, see[i].doc);
      dhi = max(dhi, see[i].doc);
    }
  }
  top = block_max(top, red);
  dhi = block_max(dhi, red);
  dlo = ~block_max(~dlo, red);

  float m[kR], l[kR], o[kR][4 * kO];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * kO; ++c) o[i][c] = 0.f;
  }
  // keys of no document may hold anything: their values are not read
  const auto key_is = [&](int j) {
    return a.docs == nullptr || a.docs[static_cast<long long>(b) * a.Tk + j] >= 0;
  };
  const int t0 = blockIdx.z * a.per_split;
  const int t1 = min(t0 + a.per_split, (top + kN - 1) / kN);
  for (int tile = t0; tile < t1; ++tile) {
    if (!span_meets(a, b, tile, dlo, dhi)) continue;  // the same for the CTA
    const int j0 = tile * kN;
    const int n = min(kN, min(keys, top) - j0);  // keys that no row sees are not read
    __syncthreads();
    load_tile<T, kN, kD>(ks, n, a.D, vec, [&](int r) { return K + (j0 + r) * a.kt; });
    load_tile<T, kN, kD>(vs, n, a.D, vec, [&](int r) -> const T* {
      return key_is(j0 + r) ? V + (j0 + r) * a.vt : nullptr;
    });
    if (a.docs != nullptr && threadIdx.x < kN)
      kdoc[threadIdx.x] = j0 + static_cast<int>(threadIdx.x) < a.Tk
                              ? a.docs[static_cast<long long>(b) * a.Tk + j0 + threadIdx.x] : -1;
    __syncthreads();
    float s[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    dots<kR, 4, kD>(qs + ty * kR * kRow, ks + tx * kRow, a.D, s);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float top_s = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = tx + 16 * j, key = j0 + col;
        float unused;
        float z = capped(a, s[i][j] * a.scale, &unused);
        z -= slope[i] * fabsf(static_cast<float>(see[i].pos - key));
        const bool ok = key < see[i].lim && (a.docs == nullptr || kdoc[col] == see[i].doc);
        s[i][j] = ok ? z : -INFINITY;
        top_s = fmaxf(top_s, s[i][j]);
      }
      const float mn = fmaxf(m[i], half_max(top_s));
      const float at = mn == -INFINITY ? 0.f : mn;  // (a row that has seen nothing yet)
      const float f = expf(m[i] - at);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = expf(s[i][j] - at);
        sum += s[i][j];
      }
      l[i] = l[i] * f + half_sum(sum);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < 4 * kO; ++c) o[i][c] *= f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float w[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) w[i] = s[i][j];
      store_weights<kR>(pt + (tx + 16 * j) * (kM + kPad) + ty * kR, w);
    }
    __syncwarp();  // (a row's weights are written and read by one half warp)
    add_rows<kR, kO, kD, kM + kPad>(pt + ty * kR, vs + tx * 4, n, o);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int p = p0 + ty * kR + i, t = p / a.G, h = hk * a.G + p - t * a.G;
    if (p >= rows) continue;
    if (a.splits > 1) {
      const long long at = (static_cast<long long>(blockIdx.z) * bhs + bh) * rows + p;
#pragma unroll
      for (int c = 0; c < 4 * kO; ++c) {
        const int col = (c / 4) * 64 + tx * 4 + c % 4;
        if (col < a.D) a.part[at * a.D + col] = o[i][c];
      }
      if (tx == 0) a.part_stats[at] = make_float2(m[i] * kLog2e, l[i]);
      continue;
    }
    const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
    T* out = static_cast<T*>(a.out) + ((static_cast<long long>(b) * a.Tq + t) * a.H + h) * a.D;
#pragma unroll
    for (int c = 0; c < 4 * kO; ++c) {
      const int col = (c / 4) * 64 + tx * 4 + c % 4;
      if (col < a.D) out[col] = T(o[i][c] * inv);
    }
    if (a.lse != nullptr && tx == 0)
      a.lse[(static_cast<long long>(b) * a.H + h) * a.Tq + t] = m[i] + logf(l[i]);
  }
}

// ---------------------------------------------------------------------------
// Gradient.  With s the score, t the tanh of the cap and P = exp(s - lse):
//   dV = P^T dO,  dS = P (dO V^T - delta) (1 - t^2) scale,  dQ = dS K,  dK = dS^T Q
// delta = sum of dO O over a row (attention.cu).  Two kernels, which form P twice and
// so need neither sums from several CTAs in an order nor partial results.
// ---------------------------------------------------------------------------
template <int kD, int kR>
constexpr int kDqSmem = 4 * ((2 * kGroups * kR + 2 * kN) * (kD + kPad) + kN * (kGroups * kR + kPad) + kN + 8);
// rows of a step of the keys' kernel
constexpr int kMB = 64;
template <int kD, int kR>
constexpr int kDkvSmem =
    4 * ((2 * kGroups * kR + 2 * kMB) * (kD + kPad) + 2 * kMB * (kGroups * kR + kPad) + 6 * kMB + 8);

template <typename T, int kD, int kR>
__global__ void __launch_bounds__(kThreads) attention_dq_simt_kernel(const AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int kM = kGroups * kR, kO = kD / 64, kRow = kD + kPad, kW = kM + kPad;
  float* qs = sm;                        // [kM][kRow]
  float* os = qs + kM * kRow;
  float* ks = os + kM * kRow;            // [kN][kRow]
  float* vs = ks + kN * kRow;
  float* st = vs + kN * kRow;            // [kN][kW]
  int* kdoc = reinterpret_cast<int*>(st + kN * kW);
  int* red = kdoc + kN;
  pdl_launch_dependents();
  pdl_wait();
  const int bhs = a.B * a.Hkv, bh = blockIdx.x % bhs, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  const int rows = a.Tq * a.G;
  const int p0 = (gridDim.x / bhs - 1 - blockIdx.x / bhs) * kM;  // (the longest rows first)
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const T* Q = static_cast<const T*>(a.Q) + b * a.qb;
  const T* K = static_cast<const T*>(a.K) + b * a.kb + hk * a.kh;
  const T* V = static_cast<const T*>(a.V) + b * a.vb + hk * a.vh;
  const T* dO = static_cast<const T*>(a.dO) + b * a.dob;
  const bool vec = a.vec != 0;
  RowSees see[kR];
  float slope[kR], lse[kR], delta[kR];
  int top = 0, dlo = 0x7fffffff, dhi = -1;
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int p = p0 + ty * kR + i, t = p / a.G, h = hk * a.G + p - t * a.G;
    see[i].pos = see[i].lim = 0;
    see[i].doc = -1;
    slope[i] = lse[i] = delta[i] = 0.f;
    if (p < rows) {
      see[i] = attn_row(a, b, t, keys, first);
      if (a.slopes != nullptr) slope[i] = a.slopes[h];
      const long long at = (static_cast<long long>(b) * a.H + h) * a.Tq + t;
      lse[i] = a.lse_in[at];
      delta[i] = a.delta[at];
    }
    top = max(top, see[i].lim);
    if (see[i].doc >= 0) {
      dlo = min(dlo, see[i].doc);
      dhi = max(dhi, see[i].doc);
    }
  }
  top = block_max(top, red);
  dhi = block_max(dhi, red);
  dlo = ~block_max(~dlo, red);
  // (rows that see nothing may hold anything: their products are masked)
  load_tile<T, kM, kD>(qs, min(kM, rows - p0), a.D, vec, [&](int r) {
    const int p = p0 + r, t = p / a.G;
    return Q + t * a.qt + (hk * a.G + p - t * a.G) * a.qh;
  });
  load_tile<T, kM, kD>(os, min(kM, rows - p0), a.D, vec, [&](int r) {
    const int p = p0 + r, t = p / a.G;
    return dO + t * a.dot + (hk * a.G + p - t * a.G) * a.doh;
  });
  float dq[kR][4 * kO];
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int c = 0; c < 4 * kO; ++c) dq[i][c] = 0.f;
  const auto key_is = [&](int j) {  // keys of no document may hold anything
    return a.docs == nullptr || a.docs[static_cast<long long>(b) * a.Tk + j] >= 0;
  };
  const int t1 = (top + kN - 1) / kN;
  for (int tile = 0; tile < t1; ++tile) {
    if (!span_meets(a, b, tile, dlo, dhi)) continue;
    const int j0 = tile * kN;
    const int n = min(kN, min(keys, top) - j0);
    __syncthreads();
    load_tile<T, kN, kD>(ks, n, a.D, vec, [&](int r) -> const T* {
      return key_is(j0 + r) ? K + (j0 + r) * a.kt : nullptr;
    });
    load_tile<T, kN, kD>(vs, n, a.D, vec, [&](int r) { return V + (j0 + r) * a.vt; });
    if (a.docs != nullptr && threadIdx.x < kN)
      kdoc[threadIdx.x] = j0 + static_cast<int>(threadIdx.x) < a.Tk
                              ? a.docs[static_cast<long long>(b) * a.Tk + j0 + threadIdx.x] : -1;
    __syncthreads();
    float s[kR][4], dp[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
    dots<kR, 4, kD>(qs + ty * kR * kRow, ks + tx * kRow, a.D, s);
    dots<kR, 4, kD>(os + ty * kR * kRow, vs + tx * kRow, a.D, dp);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = tx + 16 * j, key = j0 + col;
      float w[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        float sl;
        float z = capped(a, s[i][j] * a.scale, &sl);
        z -= slope[i] * fabsf(static_cast<float>(see[i].pos - key));
        const bool ok = key < see[i].lim && (a.docs == nullptr || kdoc[col] == see[i].doc);
        w[i] = ok ? expf(z - lse[i]) * (dp[i][j] - delta[i]) * sl * a.scale : 0.f;
      }
      store_weights<kR>(st + col * kW + ty * kR, w);
    }
    __syncwarp();
    add_rows<kR, kO, kD, kW>(st + ty * kR, ks + tx * 4, n, dq);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int p = p0 + ty * kR + i, t = p / a.G, h = hk * a.G + p - t * a.G;
    if (p >= rows) continue;
    T* out = static_cast<T*>(a.dQ) + b * a.dqb + t * a.dqt + h * a.dqh;
#pragma unroll
    for (int c = 0; c < 4 * kO; ++c) {
      const int col = (c / 4) * 64 + tx * 4 + c % 4;
      if (col < a.D) out[col] = T(dq[i][c]);
    }
  }
}

// A thread's "rows" are keys here, and its columns rows of queries.
template <typename T, int kD, int kR>
__global__ void __launch_bounds__(kThreads) attention_dkv_simt_kernel(const AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int kM = kGroups * kR, kO = kD / 64, kRow = kD + kPad, kW = kM + kPad;
  float* ks = sm;                          // [kM][kRow]
  float* vs = ks + kM * kRow;
  float* qs = vs + kM * kRow;              // [kMB][kRow]
  float* os = qs + kMB * kRow;
  float* pt = os + kMB * kRow;             // [kMB][kW]
  float* st = pt + kMB * kW;
  float* rlse = st + kMB * kW;             // of the step's rows
  float* rdel = rlse + kMB;
  float* rslope = rdel + kMB;
  int* rpos = reinterpret_cast<int*>(rslope + kMB);
  int* rlim = rpos + kMB;
  int* rdoc = rlim + kMB;
  pdl_launch_dependents();
  pdl_wait();
  const int bhs = a.B * a.Hkv, bh = blockIdx.x % bhs, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  const int rows = a.Tq * a.G;
  const int j0 = blockIdx.x / bhs * kM;  // (the first keys have the most rows)
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const T* Q = static_cast<const T*>(a.Q) + b * a.qb;
  const T* K = static_cast<const T*>(a.K) + b * a.kb + hk * a.kh;
  const T* V = static_cast<const T*>(a.V) + b * a.vb + hk * a.vh;
  const T* dO = static_cast<const T*>(a.dO) + b * a.dob;
  const bool vec = a.vec != 0;
  const int n = max(0, min(kM, keys - j0));
  const int* docs = a.docs != nullptr ? a.docs + static_cast<long long>(b) * a.Tk : nullptr;
  DocSpan span = {0, 0, 0, 0};
  if (docs != nullptr)
    span = a.spans[static_cast<long long>(b) * ((a.Tk + kDocSpan - 1) / kDocSpan) + j0 / kDocSpan];
  // (keys that nobody sees may hold anything: their products are masked)
  load_tile<T, kM, kD>(ks, n, a.D, vec, [&](int r) { return K + (j0 + r) * a.kt; });
  load_tile<T, kM, kD>(vs, n, a.D, vec, [&](int r) { return V + (j0 + r) * a.vt; });
  int kdoc[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i)
    kdoc[i] = docs != nullptr ? (ty * kR + i < n ? docs[j0 + ty * kR + i] : -2) : 0;
  float dk[kR][4 * kO], dv[kR][4 * kO];
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int c = 0; c < 4 * kO; ++c) dk[i][c] = dv[i][c] = 0.f;
  // the first token that may see a key of this tile
  int tok0 = 0;
  if (a.causal && (a.prefix == nullptr || a.prefix[b] <= j0)) tok0 = max(0, min(a.Tq, j0 - first));
  for (int p0 = tok0 * a.G / kMB * kMB; p0 < rows && n > 0; p0 += kMB) {
    if (p0 / kMB % a.row_splits != static_cast<int>(blockIdx.z)) continue;  // another CTA's
    __syncthreads();
    int any = 0;
    if (threadIdx.x < kMB) {
      const int p = p0 + threadIdx.x, t = p / a.G, h = hk * a.G + p - t * a.G;
      RowSees r = {0, 0, -1};
      float lse = 0.f, del = 0.f, slope = 0.f;
      if (p < rows) {
        r = attn_row(a, b, t, keys, first);
        const long long at = (static_cast<long long>(b) * a.H + h) * a.Tq + t;
        lse = a.lse_in[at];
        // (a document behind its sample's length: the position sees keys, the query none)
        if (lse == -INFINITY) r.lim = 0;
        del = a.delta[at];
        if (a.slopes != nullptr) slope = a.slopes[h];
      }
      rlse[threadIdx.x] = lse;
      rdel[threadIdx.x] = del;
      rslope[threadIdx.x] = slope;
      rpos[threadIdx.x] = r.pos;
      rlim[threadIdx.x] = r.lim;
      rdoc[threadIdx.x] = r.doc;
      any = r.lim > j0 && (docs == nullptr || (r.doc >= span.lo && r.doc <= span.hi));
    }
    if (!__syncthreads_or(any)) continue;
    // rows that see nothing are not read: they are summed over
    const int nr = min(kMB, rows - p0);
    load_tile<T, kMB, kD>(qs, nr, a.D, vec, [&](int r) -> const T* {
      const int p = p0 + r, t = p / a.G;
      return rlim[r] > 0 ? Q + t * a.qt + (hk * a.G + p - t * a.G) * a.qh : nullptr;
    });
    load_tile<T, kMB, kD>(os, nr, a.D, vec, [&](int r) -> const T* {
      const int p = p0 + r, t = p / a.G;
      return rlim[r] > 0 ? dO + t * a.dot + (hk * a.G + p - t * a.G) * a.doh : nullptr;
    });
    __syncthreads();
    float s[kR][4], dp[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
    dots<kR, 4, kD>(ks + ty * kR * kRow, qs + tx * kRow, a.D, s);
    dots<kR, 4, kD>(vs + ty * kR * kRow, os + tx * kRow, a.D, dp);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = tx + 16 * j;
      float w[kR], u[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int key = j0 + ty * kR + i;
        float sl;
        float z = capped(a, s[i][j] * a.scale, &sl);
        z -= rslope[r] * fabsf(static_cast<float>(rpos[r] - key));
        const bool ok = key < rlim[r] && (docs == nullptr || kdoc[i] == rdoc[r]);
        w[i] = ok ? expf(z - rlse[r]) : 0.f;
        u[i] = ok ? w[i] * (dp[i][j] - rdel[r]) * sl * a.scale : 0.f;
      }
      store_weights<kR>(pt + r * kW + ty * kR, w);
      store_weights<kR>(st + r * kW + ty * kR, u);
    }
    __syncwarp();
    add_rows<kR, kO, kD, kW>(pt + ty * kR, os + tx * 4, nr, dv);
    add_rows<kR, kO, kD, kW>(st + ty * kR, qs + tx * 4, nr, dk);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int key = j0 + ty * kR + i;
    if (key >= a.Tk) continue;
    if (a.row_splits > 1) {
      float* part = a.key_part +
                    ((static_cast<long long>(blockIdx.z) * bhs + bh) * a.Tk + key) * 2 * a.D;
#pragma unroll
      for (int c = 0; c < 4 * kO; ++c) {
        const int col = (c / 4) * 64 + tx * 4 + c % 4;
        if (col >= a.D) continue;
        part[col] = dk[i][c];
        part[a.D + col] = dv[i][c];
      }
      continue;
    }
    T* k = static_cast<T*>(a.dK) + b * a.dkb + key * a.dkt + hk * a.dkh;
    T* v = static_cast<T*>(a.dV) + b * a.dvb + key * a.dvt + hk * a.dvh;
#pragma unroll
    for (int c = 0; c < 4 * kO; ++c) {
      const int col = (c / 4) * 64 + tx * 4 + c % 4;
      if (col >= a.D) continue;
      if (a.dK != nullptr) k[col] = T(dk[i][c]);
      if (a.dV != nullptr) v[col] = T(dv[i][c]);
    }
  }
}

// Rows of a group: four, or two where the tiles would not fill the SMs twice; one for few rows.
int rows_of_group(long long rows, long long heads, bool one) {
  const auto ctas = [&](int r) { return (rows + kGroups * r - 1) / (kGroups * r) * heads; };
  if (one && rows <= 16) return 1;
  return ctas(4) >= 304 ? 4 : 2;
}

template <typename T, int kD, int kR>
cudaError_t forward(const AttnArgs& a, cudaStream_t s) {
  constexpr int bytes = kFwdSmem<kD, kR>;
  const cudaError_t e = allow_smem<attention_simt_kernel<T, kD, kR>>(bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.Tq * a.G + kGroups * kR - 1) / (kGroups * kR) * (a.B * a.Hkv), 1, a.splits);
  return launch_after(attention_simt_kernel<T, kD, kR>, grid, kThreads, 1, s, bytes, a);
}

template <typename T, int kD>
cudaError_t forward_rows(const AttnArgs& a, cudaStream_t s) {
  switch (attention_simt_rows(a.Tq * a.G, a.B * a.Hkv)) {
    case 16: return forward<T, kD, 1>(a, s);
    case 32: return forward<T, kD, 2>(a, s);
  }
  return forward<T, kD, 4>(a, s);
}

template <typename T, int kD, int kR>
cudaError_t rows_grad(const AttnArgs& a, cudaStream_t s) {
  constexpr int bytes = kDqSmem<kD, kR>;
  const cudaError_t e = allow_smem<attention_dq_simt_kernel<T, kD, kR>>(bytes);
  if (e != cudaSuccess) return e;
  return launch_after(attention_dq_simt_kernel<T, kD, kR>,
                      dim3((a.Tq * a.G + kGroups * kR - 1) / (kGroups * kR) * (a.B * a.Hkv)), kThreads, 1, s,
                      bytes, a);
}
template <typename T, int kD, int kR>
cudaError_t keys_grad(const AttnArgs& a, cudaStream_t s) {
  constexpr int bytes = kDkvSmem<kD, kR>;
  const cudaError_t e = allow_smem<attention_dkv_simt_kernel<T, kD, kR>>(bytes);
  if (e != cudaSuccess) return e;
  return launch_after(attention_dkv_simt_kernel<T, kD, kR>,
                      dim3((a.Tk + kGroups * kR - 1) / (kGroups * kR) * (a.B * a.Hkv), 1, a.row_splits),
                      kThreads, 1, s, bytes, a);
}

template <typename T, int kD>
cudaError_t backward(const AttnArgs& a, cudaStream_t s) {
  if (a.dQ != nullptr) {
    const cudaError_t e = rows_of_group(a.Tq * a.G, a.B * a.Hkv, false) == 4
                              ? rows_grad<T, kD, 4>(a, s) : rows_grad<T, kD, 2>(a, s);
    if (e != cudaSuccess) return e;
  }
  if (a.dK == nullptr && a.dV == nullptr) return cudaSuccess;
  return rows_of_group(a.Tk, a.B * a.Hkv, false) == 4 ? keys_grad<T, kD, 4>(a, s)
                                                      : keys_grad<T, kD, 2>(a, s);
}

// Whether rows of the three (gradient: four) tensors are whole accesses of four.
template <typename T>
bool fours(const AttnArgs& a) {
  const long long all = a.D | a.qb | a.qt | a.qh | a.kb | a.kt | a.kh | a.vb | a.vt | a.vh |
                        a.dob | a.dot | a.doh;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.Q) | reinterpret_cast<uintptr_t>(a.K) |
                       reinterpret_cast<uintptr_t>(a.V) | reinterpret_cast<uintptr_t>(a.dO);
  return all % 4 == 0 && at % (4 * sizeof(T)) == 0;
}

}  // namespace

int attention_simt_rows(long long rows, long long heads) {
  return kGroups * rows_of_group(rows, heads, true);
}

int attention_simt_keys(long long keys, long long heads) {
  return kGroups * rows_of_group(keys, heads, false);
}

cudaError_t launch_attention_simt(const AttnArgs& args, dprc_dtype dt, cudaStream_t s) {
  AttnArgs a = args;
  if (dt == DPRC_F32) {
    a.vec = fours<float>(a);
    return a.D > 64 ? forward_rows<float, 128>(a, s) : forward_rows<float, 64>(a, s);
  }
  a.vec = fours<__nv_bfloat16>(a);
  return a.D > 64 ? forward_rows<__nv_bfloat16, 128>(a, s) : forward_rows<__nv_bfloat16, 64>(a, s);
}

cudaError_t launch_attention_grad_simt(const AttnArgs& args, dprc_dtype dt, cudaStream_t s) {
  AttnArgs a = args;
  if (dt == DPRC_F32) {
    a.vec = fours<float>(a);
    return a.D > 64 ? backward<float, 128>(a, s) : backward<float, 64>(a, s);
  }
  a.vec = fours<__nv_bfloat16>(a);
  return a.D > 64 ? backward<__nv_bfloat16, 128>(a, s) : backward<__nv_bfloat16, 64>(a, s);
}

cudaError_t read_device_error_attention_simt(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

}  // namespace dprc
