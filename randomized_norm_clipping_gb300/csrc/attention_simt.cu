// Attention on the CUDA cores, in fp32: fp32 inputs, and bf16 ones whose widths
// or strides the tensor copies do not take.  The same sums as the tensor-core kernels
// (attention_tc.cu), in tiles of 64 rows and 64 keys.
//
// A CTA of 128 threads holds kM rows (64, or 16 where a sample has few); a thread
// has kM / 8 rows and four keys of the product, then the same rows and four columns
// in sixteen of the values' width.  The rows' statistics are kept by the sixteen
// threads that share them, so the sums over keys are shuffles.  Bound by the
// shared memory's reads for the products: 12 floats read for 32 products (64 rows).

#include <algorithm>

#include "attention.cuh"

namespace dprc {
namespace {

constexpr int kThreads = 128;
constexpr int kN = 64;
constexpr int kPad = 4;

// rows [n] of width D from src (row stride rs, null rows are zero) into dst:
// transposed [kD][n + kPad], or as they are [n][kD + kPad].
template <typename T, int kRowsMax, int kD, bool kTrans, typename Src>
__device__ __forceinline__ void load_tile(float* dst, int n, int D, Src src) {
  for (int i = threadIdx.x; i < kRowsMax * kD; i += kThreads) {
    const int r = i / kD, c = i - r * kD;
    float v = 0.f;
    if (r < n && c < D) {
      const T* p = src(r);
      if (p != nullptr) v = to_f32<T>(ld_once(p + c));
    }
    if (kTrans) dst[c * (kRowsMax + kPad) + r] = v;
    else dst[r * (kD + kPad) + c] = v;
  }
}

template <int kD>
struct FwdSmem {
  template <int kM>
  static constexpr int bytes() {
    return 4 * (kD * (kM + kPad) + kD * (kN + kPad) + kN * (kD + kPad) + kN * (kM + kPad)) +
           4 * (kM * 4 + kN);
  }
};

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
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = max(max(sm[0], sm[1]), max(sm[2], sm[3]));
  __syncthreads();
  return v;
}

// Whether any row with documents in [lo, hi] may see a key of this span.
__device__ __forceinline__ bool span_meets(const AttnArgs& a, int b, int tile, int lo, int hi) {
  if (a.docs == nullptr) return true;
  const DocSpan s = a.spans[static_cast<long long>(b) * ((a.Tk + kDocSpan - 1) / kDocSpan) + tile];
  return s.lo <= hi && lo <= s.hi;
}

// Products of kR rows (from at, [kD][stride as]) and kC columns (from bt): acc += .
template <int kR, int kC>
__device__ __forceinline__ void dot_step(const float* at, const float* bt, float (&acc)[kR][kC]) {
  float x[kR], y[kC];
#pragma unroll
  for (int i = 0; i < kR; i += (kR >= 4 ? 4 : 2)) {
    if constexpr (kR >= 4) {
      const float4 v = *reinterpret_cast<const float4*>(at + i);
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(at + i);
      x[i] = v.x; x[i + 1] = v.y;
    }
  }
#pragma unroll
  for (int j = 0; j < kC; j += (kC >= 4 ? 4 : 2)) {
    if constexpr (kC >= 4) {
      const float4 v = *reinterpret_cast<const float4*>(bt + j);
      y[j] = v.x; y[j + 1] = v.y; y[j + 2] = v.z; y[j + 3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(bt + j);
      y[j] = v.x; y[j + 1] = v.y;
    }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int j = 0; j < kC; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
}

template <typename T, int kD, int kM>
__global__ void __launch_bounds__(kThreads) attention_simt_kernel(const AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int kR = kM / 8;          // rows of a thread
  constexpr int kO = kD / 64;         // fours of the values' columns of a thread
  float* qt = sm;                              // [kD][kM + kPad]
  float* kt = qt + kD * (kM + kPad);           // [kD][kN + kPad]
  float* vs = kt + kD * (kN + kPad);           // [kN][kD + kPad]
  float* pt = vs + kN * (kD + kPad);           // [kN][kM + kPad]
  int* kdoc = reinterpret_cast<int*>(pt + kN * (kM + kPad));  // [kN]
  int* red = kdoc + kN;                        // [4]
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y / a.Hkv, hk = blockIdx.y - b * a.Hkv;
  const int rows = a.Tq * a.G, p0 = blockIdx.x * kM;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const T* Q = static_cast<const T*>(a.Q) + b * a.qb;
  const T* K = static_cast<const T*>(a.K) + b * a.kb + hk * a.kh;
  const T* V = static_cast<const T*>(a.V) + b * a.vb + hk * a.vh;

  load_tile<T, kM, kD, true>(qt, min(kM, rows - p0), a.D, [&](int r) {
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
    load_tile<T, kN, kD, true>(kt, n, a.D, [&](int r) { return K + (j0 + r) * a.kt; });
    load_tile<T, kN, kD, false>(vs, n, a.D, [&](int r) -> const T* {
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
#pragma unroll 4
    for (int d = 0; d < a.D; ++d)
      dot_step<kR, 4>(qt + d * (kM + kPad) + ty * kR, kt + d * (kN + kPad) + tx * 4, s);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float top_s = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx * 4 + j;
        float unused;
        float z = attn_capped(a, s[i][j] * a.scale, &unused);
        z -= slope[i] * fabsf(static_cast<float>(see[i].pos - key));
        const bool ok = key < see[i].lim && (a.docs == nullptr || kdoc[tx * 4 + j] == see[i].doc);
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
        pt[(tx * 4 + j) * (kM + kPad) + ty * kR + i] = s[i][j];
      }
      l[i] = l[i] * f + half_sum(sum);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < 4 * kO; ++c) o[i][c] *= f;
    }
    __syncwarp();  // (a row's weights are written and read by one half warp)
#pragma unroll 2
    for (int j = 0; j < n; ++j) {
#pragma unroll
      for (int q = 0; q < kO; ++q) {
        float acc[kR][4];
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] = o[i][q * 4 + c];
        dot_step<kR, 4>(pt + j * (kM + kPad) + ty * kR, vs + j * (kD + kPad) + q * 64 + tx * 4, acc);
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][q * 4 + c] = acc[i][c];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int p = p0 + ty * kR + i, t = p / a.G, h = hk * a.G + p - t * a.G;
    if (p >= rows) continue;
    if (a.splits > 1) {
      const long long at = (static_cast<long long>(blockIdx.z) * a.B * a.Hkv + blockIdx.y) * rows + p;
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
constexpr int kMB = 32;  // rows of a step of the keys' kernel

template <int kD>
constexpr int kDqSmem = 4 * (4 * kD * (kN + kPad) + kN * (kD + kPad) + kN * (kN + kPad) + kN + 8);
template <int kD>
constexpr int kDkvSmem =
    4 * (2 * kD * (kN + kPad) + 2 * kD * (kMB + kPad) + 2 * kMB * (kD + kPad) + 2 * kMB * (kN + kPad) + 6 * kMB + 8);

template <typename T, int kD>
__global__ void __launch_bounds__(kThreads) attention_dq_simt_kernel(const AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int kR = 8, kO = kD / 64, kS = kN + kPad;
  float* qt = sm;
  float* ot = qt + kD * kS;
  float* kt = ot + kD * kS;
  float* vt = kt + kD * kS;
  float* ks = vt + kD * kS;              // [kN][kD + kPad]
  float* st = ks + kN * (kD + kPad);     // [kN][kS]
  int* kdoc = reinterpret_cast<int*>(st + kN * kS);
  int* red = kdoc + kN;
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y / a.Hkv, hk = blockIdx.y - b * a.Hkv;
  const int rows = a.Tq * a.G, p0 = blockIdx.x * kN;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const T* Q = static_cast<const T*>(a.Q) + b * a.qb;
  const T* K = static_cast<const T*>(a.K) + b * a.kb + hk * a.kh;
  const T* V = static_cast<const T*>(a.V) + b * a.vb + hk * a.vh;
  const T* dO = static_cast<const T*>(a.dO);
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
  // rows that see nothing: what stands in them is not read
  const auto row_of = [&](int r, int& t, int& h) {
    const int p = p0 + r;
    t = p / a.G;
    h = hk * a.G + p - t * a.G;
    return attn_row(a, b, t, keys, first).lim > 0;
  };
  load_tile<T, kN, kD, true>(qt, min(kN, rows - p0), a.D, [&](int r) -> const T* {
    int t, h;
    return row_of(r, t, h) ? Q + t * a.qt + h * a.qh : nullptr;
  });
  load_tile<T, kN, kD, true>(ot, min(kN, rows - p0), a.D, [&](int r) -> const T* {
    int t, h;
    return row_of(r, t, h) ? dO + b * a.dob + t * a.dot + h * a.doh : nullptr;
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
    const auto k_row = [&](int r) -> const T* {
      return key_is(j0 + r) ? K + (j0 + r) * a.kt : nullptr;
    };
    load_tile<T, kN, kD, true>(kt, n, a.D, k_row);
    load_tile<T, kN, kD, false>(ks, n, a.D, k_row);
    load_tile<T, kN, kD, true>(vt, n, a.D, [&](int r) { return V + (j0 + r) * a.vt; });
    if (a.docs != nullptr && threadIdx.x < kN)
      kdoc[threadIdx.x] = j0 + static_cast<int>(threadIdx.x) < a.Tk
                              ? a.docs[static_cast<long long>(b) * a.Tk + j0 + threadIdx.x] : -1;
    __syncthreads();
    float s[kR][4], dp[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = dp[i][j] = 0.f;
#pragma unroll 2
    for (int d = 0; d < a.D; ++d) {
      dot_step<kR, 4>(qt + d * kS + ty * kR, kt + d * kS + tx * 4, s);
      dot_step<kR, 4>(ot + d * kS + ty * kR, vt + d * kS + tx * 4, dp);
    }
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx * 4 + j;
        float sl;
        float z = attn_capped(a, s[i][j] * a.scale, &sl);
        z -= slope[i] * fabsf(static_cast<float>(see[i].pos - key));
        const bool ok = key < see[i].lim && (a.docs == nullptr || kdoc[tx * 4 + j] == see[i].doc);
        const float ds = expf(z - lse[i]) * (dp[i][j] - delta[i]) * sl * a.scale;
        st[(tx * 4 + j) * kS + ty * kR + i] = ok ? ds : 0.f;
      }
    __syncwarp();
    for (int j = 0; j < n; ++j) {
#pragma unroll
      for (int q = 0; q < kO; ++q) {
        float acc[kR][4];
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] = dq[i][q * 4 + c];
        dot_step<kR, 4>(st + j * kS + ty * kR, ks + j * (kD + kPad) + q * 64 + tx * 4, acc);
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) dq[i][q * 4 + c] = acc[i][c];
      }
    }
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

template <typename T, int kD>
__global__ void __launch_bounds__(kThreads) attention_dkv_simt_kernel(const AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int kR = 8, kO = kD / 64, kS = kN + kPad, kSB = kMB + kPad;
  float* kt = sm;                          // [kD][kS]
  float* vt = kt + kD * kS;
  float* qt = vt + kD * kS;                // [kD][kSB]
  float* ot = qt + kD * kSB;
  float* qs = ot + kD * kSB;               // [kMB][kD + kPad]
  float* os = qs + kMB * (kD + kPad);
  float* pt = os + kMB * (kD + kPad);      // [kMB][kS]
  float* st = pt + kMB * kS;
  float* rlse = st + kMB * kS;             // of the step's rows
  float* rdel = rlse + kMB;
  float* rslope = rdel + kMB;
  int* rpos = reinterpret_cast<int*>(rslope + kMB);
  int* rlim = rpos + kMB;
  int* rdoc = rlim + kMB;
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y / a.Hkv, hk = blockIdx.y - b * a.Hkv;
  const int rows = a.Tq * a.G, j0 = blockIdx.x * kN;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const T* Q = static_cast<const T*>(a.Q) + b * a.qb;
  const T* K = static_cast<const T*>(a.K) + b * a.kb + hk * a.kh;
  const T* V = static_cast<const T*>(a.V) + b * a.vb + hk * a.vh;
  const T* dO = static_cast<const T*>(a.dO);
  const int n = max(0, min(kN, keys - j0));
  const int* docs = a.docs != nullptr ? a.docs + static_cast<long long>(b) * a.Tk : nullptr;
  DocSpan span = {0, 0, 0, 0};
  if (docs != nullptr)
    span = a.spans[static_cast<long long>(b) * ((a.Tk + kDocSpan - 1) / kDocSpan) + blockIdx.x];
  // keys of no document may hold anything
  const auto key_is = [&](int r) { return docs == nullptr || docs[j0 + r] >= 0; };
  load_tile<T, kN, kD, true>(kt, n, a.D, [&](int r) -> const T* {
    return key_is(r) ? K + (j0 + r) * a.kt : nullptr;
  });
  load_tile<T, kN, kD, true>(vt, n, a.D, [&](int r) -> const T* {
    return key_is(r) ? V + (j0 + r) * a.vt : nullptr;
  });
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
    const auto q_row = [&](int r) -> const T* {
      const int p = p0 + r, t = p / a.G;
      return rlim[r] > 0 ? Q + t * a.qt + (hk * a.G + p - t * a.G) * a.qh : nullptr;
    };
    const auto o_row = [&](int r) -> const T* {
      const int p = p0 + r, t = p / a.G, h = hk * a.G + p - t * a.G;
      return rlim[r] > 0 ? dO + b * a.dob + t * a.dot + h * a.doh : nullptr;
    };
    const int nr = min(kMB, rows - p0);
    load_tile<T, kMB, kD, true>(qt, nr, a.D, q_row);
    load_tile<T, kMB, kD, true>(ot, nr, a.D, o_row);
    load_tile<T, kMB, kD, false>(qs, nr, a.D, q_row);
    load_tile<T, kMB, kD, false>(os, nr, a.D, o_row);
    __syncthreads();
    float s[kR][2], dp[kR][2];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) s[i][j] = dp[i][j] = 0.f;
#pragma unroll 2
    for (int d = 0; d < a.D; ++d) {
      dot_step<kR, 2>(kt + d * kS + ty * kR, qt + d * kSB + tx * 2, s);
      dot_step<kR, 2>(vt + d * kS + ty * kR, ot + d * kSB + tx * 2, dp);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = tx * 2 + j;
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int key = j0 + ty * kR + i;
        float sl;
        float z = attn_capped(a, s[i][j] * a.scale, &sl);
        z -= rslope[r] * fabsf(static_cast<float>(rpos[r] - key));
        const bool ok = key < rlim[r] && (docs == nullptr || kdoc[i] == rdoc[r]);
        const float p = ok ? expf(z - rlse[r]) : 0.f;
        pt[r * kS + ty * kR + i] = p;
        st[r * kS + ty * kR + i] = ok ? p * (dp[i][j] - rdel[r]) * sl * a.scale : 0.f;
      }
    }
    __syncwarp();
    for (int r = 0; r < nr; ++r) {
#pragma unroll
      for (int q = 0; q < kO; ++q) {
        float acc[kR][4];
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] = dv[i][q * 4 + c];
        dot_step<kR, 4>(pt + r * kS + ty * kR, os + r * (kD + kPad) + q * 64 + tx * 4, acc);
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            dv[i][q * 4 + c] = acc[i][c];
            acc[i][c] = dk[i][q * 4 + c];
          }
        dot_step<kR, 4>(st + r * kS + ty * kR, qs + r * (kD + kPad) + q * 64 + tx * 4, acc);
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) dk[i][q * 4 + c] = acc[i][c];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int key = j0 + ty * kR + i;
    if (key >= a.Tk) continue;
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


template <typename T, int kD, int kM>
cudaError_t forward(const AttnArgs& a, cudaStream_t s) {
  constexpr int bytes = FwdSmem<kD>::template bytes<kM>();
  cudaError_t e = allow_smem<attention_simt_kernel<T, kD, kM>>(bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.Tq * a.G + kM - 1) / kM, a.B * a.Hkv, a.splits);
  return launch_after(attention_simt_kernel<T, kD, kM>, grid, kThreads, 1, s, bytes, a);
}

template <typename T, int kD>
cudaError_t backward(const AttnArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.dQ != nullptr) {
    if ((e = allow_smem<attention_dq_simt_kernel<T, kD>>(kDqSmem<kD>)) != cudaSuccess) return e;
    e = launch_after(attention_dq_simt_kernel<T, kD>, dim3((a.Tq * a.G + kN - 1) / kN, a.B * a.Hkv),
                     kThreads, 1, s, kDqSmem<kD>, a);
    if (e != cudaSuccess) return e;
  }
  if (a.dK == nullptr && a.dV == nullptr) return e;
  if ((e = allow_smem<attention_dkv_simt_kernel<T, kD>>(kDkvSmem<kD>)) != cudaSuccess) return e;
  return launch_after(attention_dkv_simt_kernel<T, kD>, dim3((a.Tk + kN - 1) / kN, a.B * a.Hkv),
                      kThreads, 1, s, kDkvSmem<kD>, a);
}

}  // namespace

int attention_simt_rows(int rows) { return rows <= 16 ? 16 : 64; }

cudaError_t launch_attention_simt(const AttnArgs& a, dprc_dtype dt, cudaStream_t s) {
  const bool few = attention_simt_rows(a.Tq * a.G) == 16, wide = a.D > 64;
  using bf16 = __nv_bfloat16;
  if (dt == DPRC_F32) {
    if (few) return wide ? forward<float, 128, 16>(a, s) : forward<float, 64, 16>(a, s);
    return wide ? forward<float, 128, 64>(a, s) : forward<float, 64, 64>(a, s);
  }
  if (few) return wide ? forward<bf16, 128, 16>(a, s) : forward<bf16, 64, 16>(a, s);
  return wide ? forward<bf16, 128, 64>(a, s) : forward<bf16, 64, 64>(a, s);
}

cudaError_t launch_attention_grad_simt(const AttnArgs& a, dprc_dtype dt, cudaStream_t s) {
  const bool wide = a.D > 64;
  using bf16 = __nv_bfloat16;
  if (dt == DPRC_F32) return wide ? backward<float, 128>(a, s) : backward<float, 64>(a, s);
  return wide ? backward<bf16, 128>(a, s) : backward<bf16, 64>(a, s);
}

cudaError_t read_device_error_attention_simt(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

}  // namespace dprc
