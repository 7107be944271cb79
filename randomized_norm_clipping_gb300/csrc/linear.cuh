// The linear map's epilogue and the plan of its products, shared by the
// kernels of linear.cu and linear_gemm.cu.
#pragma once

#include "common.cuh"
#include "dropout.cuh"
#include "internal.h"

namespace dprc {

// What happens to 8 neighbouring outputs of a product:
//   z = v + bias;  Z = z (kept for the gradient);  y = res + drop(act(z)).
struct LinearEpi {
  long long M = 0;
  int N = 0;
  int vec = 0;               // 1: N is a multiple of 8, 16-byte accesses; 2: bf16 rows of whole
                             // 32 bytes, and accesses of as many where a thread has them
  int act = DPRC_ACT_NONE;
  const void* bias = nullptr;  // [N]
  const void* res = nullptr;   // [M][N]
  void* Z = nullptr;           // [M][N]
  void* Y = nullptr;           // [M][N]
  DropArgs drop;
};

// sigmoid; kFast: the hardware exponential and reciprocal (a few ulp of fp32,
// far below the rounding of a bf16 result).
template <bool kFast>
__device__ __forceinline__ float sigmoid_f(float x) {
  if (kFast) return __fdividef(1.f, 1.f + __expf(-x));
  return 1.f / (1.f + expf(-x));
}

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// gelu(z) = z (1 + tanh u) / 2 = z sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3)
template <bool kFast>
__device__ __forceinline__ void act_value8(float* z, int act) {
  if (act == DPRC_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] *= sigmoid_f<kFast>(z[e]);
  } else if (act == DPRC_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      z[e] *= sigmoid_f<kFast>(kGelu2C * fmaf(kGeluA * z[e] * z[e], z[e], z[e]));
  } else if (act == DPRC_ACT_RELU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = z[e] <= 0.f ? 0.f : z[e];  // NaN stays
  }
}

// g *= act'(z)
template <bool kFast>
__device__ __forceinline__ void act_slope8(float* g, const float* z, int act) {
  if (act == DPRC_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sigmoid_f<kFast>(z[e]);
      g[e] *= fmaf(z[e] * s, 1.f - s, s);
    }
  } else if (act == DPRC_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = z[e] * z[e];
      const float s = sigmoid_f<kFast>(kGelu2C * fmaf(kGeluA * q, z[e], z[e]));
      // (where s (1 - s) has underflowed the slope is s, however large z^2)
      const float b = z[e] * s * (1.f - s);
      g[e] *= b == 0.f ? s : fmaf(b, kGelu2C * fmaf(3.f * kGeluA, q, 1.f), s);
    }
  } else if (act == DPRC_ACT_RELU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= z[e] > 0.f ? 1.f : (z[e] <= 0.f ? 0.f : z[e]);
  }
}

__device__ __forceinline__ void ld8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(u[e] << 16);
    v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void st8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float* v) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    u[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// cnt (1..8) values at p, by 16-byte accesses where vec.
template <typename T>
__device__ __forceinline__ void ld_n(const T* p, int cnt, bool vec, float* v) {
  if (vec) {
    ld8(p, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < cnt ? to_f32<T>(p[e]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void st_n(T* p, int cnt, bool vec, const float* v) {
  if (vec) {
    st8(p, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) st1(p + e, v[e]);
}

// Drops elements e0 .. e0 + 7 of a tensor (dropout.cuh); e0 of any residue.
__device__ __forceinline__ void drop8_at(float* v, uint64_t e0, const DropArgs& d,
                                         const RoundKeys& rk) {
  const uint4 w0 = philox_block(e0 >> 3, d.step, rk);
  if ((e0 & 7) == 0) {
    drop8(v, w0, d.thr, d.keep);
    return;
  }
  const uint4 w1 = philox_block((e0 >> 3) + 1, d.step, rk);
  uint32_t keep = 0;
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    keep |= (drop_keep(w0, h, d.thr) ? 1u : 0u) << h;
    keep |= (drop_keep(w1, h, d.thr) ? 1u : 0u) << (h + 8);
  }
  keep >>= static_cast<int>(e0 & 7);
#pragma unroll
  for (int h = 0; h < 8; ++h) v[h] = ((keep >> h) & 1u) ? v[h] * d.keep : 0.f;
}

// 16 bf16 values as one 32-byte access (sm_100 and later): a whole sector, where
// two accesses of 16 bytes go to L2 as two halves of one.
__device__ __forceinline__ void ld16_raw(const __nv_bfloat16* p, uint32_t* u) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]),
                 "=r"(u[6]), "=r"(u[7])
               : "l"(p));
}
__device__ __forceinline__ void ld16_bf16(const __nv_bfloat16* p, float* v) {
  uint32_t u[8];
  ld16_raw(p, u);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[2 * e] = __uint_as_float(u[e] << 16);
    v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void st16_bf16(__nv_bfloat16* p, const float* v) {
  uint32_t u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    u[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// kG groups of 8 neighbouring values of a row from p on (column n of N), to or
// from memory, by the widest access that vec allows.
template <typename T, int kG>
__device__ __forceinline__ void row_ld(const T* p, int n, int N, int vec, float* v) {
  if constexpr (sizeof(T) == 2 && kG % 2 == 0) {
    if (vec == 2) {
#pragma unroll
      for (int g = 0; g < kG; g += 2)
        if (n + 8 * g < N) ld16_bf16(p + 8 * g, v + 8 * g);
      return;
    }
  }
#pragma unroll
  for (int g = 0; g < kG; ++g)
    if (n + 8 * g < N) ld_n<T>(p + 8 * g, min(8, N - n - 8 * g), vec != 0, v + 8 * g);
}
template <typename T, int kG>
__device__ __forceinline__ void row_st(T* p, int n, int N, int vec, const float* v) {
  if constexpr (sizeof(T) == 2 && kG % 2 == 0) {
    if (vec == 2) {
#pragma unroll
      for (int g = 0; g < kG; g += 2)
        if (n + 8 * g < N) st16_bf16(p + 8 * g, v + 8 * g);
      return;
    }
  }
#pragma unroll
  for (int g = 0; g < kG; ++g)
    if (n + 8 * g < N) st_n<T>(p + 8 * g, min(8, N - n - 8 * g), vec != 0, v + 8 * g);
}

// Outputs (m, n0 .. n0 + 8 kG) from the fp32 sums v; the residual first, so
// that it is on its way while the rest is computed.  kReady: the bias is in v,
// and the residual, if there is one, in `ready` (bf16 pairs as they are stored).
template <typename T, int kG, bool kReady = false>
__device__ __forceinline__ void linear_out(const LinearEpi& e, long long m, int n0, float* v,
                                           const RoundKeys& rk,
                                           const uint32_t* ready = nullptr) {
  constexpr bool kFast = sizeof(T) == 2;
  const long long base = m * e.N + n0;
  if (!DPRC_IN(m < e.M && n0 < e.N)) return;
  float r[kG * 8];
  if (!kReady && e.res != nullptr) row_ld<T, kG>(static_cast<const T*>(e.res) + base, n0, e.N, e.vec, r);
  if (!kReady && e.bias != nullptr) {
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int cnt = min(8, e.N - n0 - 8 * g);
      if (cnt <= 0) continue;
      float b[8];
      ld_n<T>(static_cast<const T*>(e.bias) + n0 + 8 * g, cnt, e.vec != 0, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * g + j] += b[j];
    }
  }
  if (e.Z != nullptr) row_st<T, kG>(static_cast<T*>(e.Z) + base, n0, e.N, e.vec, v);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    act_value8<kFast>(v + 8 * g, e.act);
    if (e.drop.thr != 0) drop8_at(v + 8 * g, static_cast<uint64_t>(base + 8 * g), e.drop, rk);
  }
  if (e.res != nullptr) {
    if constexpr (kReady) {
#pragma unroll
      for (int j = 0; j < 4 * kG; ++j) {
        v[2 * j] += __uint_as_float(ready[j] << 16);
        v[2 * j + 1] += __uint_as_float(ready[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8 * kG; ++j) v[j] += r[j];
    }
  }
  row_st<T, kG>(static_cast<T*>(e.Y) + base, n0, e.N, e.vec, v);
}

// v: lane l holds kN columns of row l.  After it lane l holds column l mod kN of
// the kN rows from l - l mod kN on: log2(kN) exchanges between lanes and
// registers that differ in one bit.
template <int kN>
__device__ __forceinline__ void warp_transpose(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 1; b < kN; b *= 2) {
    const bool up = (lane & b) != 0;
#pragma unroll
    for (int r = 0; r < kN; ++r) {
      if (r & b) continue;
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[r] : v[r + b], b);
      v[r] = up ? got : v[r];
      v[r + b] = up ? v[r + b] : got;
    }
  }
}

// The values of warp_transpose to or from [M][N] at (m, n), rows m .. m + kN - 1
// of one column: kN lanes side by side in a row.
template <typename T, int kN>
__device__ __forceinline__ void column_st(T* p, long long m, int n, long long M, int N,
                                          const float* v) {
  p += m * N + n;
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (n < N && m + i < M) st1(p + static_cast<long long>(i) * N, v[i]);
}

// linear_out for 32 rows of a warp, lane l's row m, where rows are not whole
// 16-byte accesses: bias, activation and dropout as there, then the warp turns
// its 32 x kN values so that a store has kN neighbouring elements of a row, and
// not one of each of 32 rows: 6609 x 475 x 2466 bf16 178 -> 53 us, with GELU,
// dropout and Z 328 -> 105.  Every lane of the warp takes part, rows past M too.
template <typename T, int kN>
__device__ __forceinline__ void linear_out_odd(const LinearEpi& e, long long m, int n0, float* v,
                                               const RoundKeys& rk) {
  constexpr bool kFast = sizeof(T) == 2;
  const int lane = threadIdx.x & 31;
  const long long mt = m - lane + (lane & ~(kN - 1));  // what the lane holds turned
  const int nt = n0 + (lane & (kN - 1));
  float r[kN];
  if (e.res != nullptr) {
    const T* p = static_cast<const T*>(e.res) + mt * e.N + nt;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      r[i] = nt < e.N && mt + i < e.M ? to_f32<T>(p[static_cast<long long>(i) * e.N]) : 0.f;
  }
  if (e.bias != nullptr) {
    const float b = nt < e.N ? to_f32<T>(static_cast<const T*>(e.bias)[nt]) : 0.f;
#pragma unroll
    for (int t = 0; t < kN; ++t) v[t] += __shfl_sync(0xffffffffu, b, t);
  }
  if (e.Z != nullptr) {
    float z[kN];
#pragma unroll
    for (int t = 0; t < kN; ++t) z[t] = v[t];
    warp_transpose<kN>(z);
    column_st<T, kN>(static_cast<T*>(e.Z), mt, nt, e.M, e.N, z);
  }
#pragma unroll
  for (int g = 0; g < kN / 8; ++g) {
    act_value8<kFast>(v + 8 * g, e.act);
    if (e.drop.thr != 0)
      drop8_at(v + 8 * g, static_cast<uint64_t>(m * e.N + n0 + 8 * g), e.drop, rk);
  }
  warp_transpose<kN>(v);
  if (e.res != nullptr) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += r[i];
  }
  column_st<T, kN>(static_cast<T*>(e.Y), mt, nt, e.M, e.N, v);
}

// ---------------------------------------------------------------------------
// One product D [rows][cols] = sum over the contraction of A(row, .) B(col, .).
// An operand is bf16 planes [planes][dim][ld]: one plane for bf16 data; fp32
// data is three planes whose sum is the value to 24 bits (x = x0 + x1 + x2,
// each the rounding of what is left), and a product of two such values is the
// six plane products whose size is above 2^-24 of it.
// K-major: the contraction runs along a stored row; otherwise (MN-major) the
// rows or columns of D do.
// ---------------------------------------------------------------------------
struct GemmOperand {
  const void* data = nullptr;
  bool mn_major = false;
  int64_t ld = 0;           // elements between stored rows
  int64_t plane = 0;        // elements between planes
};

struct GemmShape {
  int64_t rows = 0, cols = 0, K = 0;
  int planes = 1;           // 1 (bf16) or 3 (fp32)
  bool transposed = false;  // D is stored [cols][rows] (the tokens are cols)
};

// How a product is cut: tiles of 128 x tn, the contraction in `split` shares
// whose fp32 partial sums a second kernel adds.
struct GemmPlan {
  int tn = 256;
  bool pair = false;        // 256 x 256 tiles on CTA pairs
  bool join = false;        // the shares of a tile are a cluster: no partial sums in memory
  int split = 1;
  int64_t units = 0;        // contraction units of 64
  int64_t per = 0;          // units of a share
  int64_t ldpart = 0;       // row stride of a partial result
  size_t part_bytes = 0;
  double cost = 0.0;        // estimated cycles
};

GemmPlan plan_gemm(const GemmShape& g);
// D into epi (split == 1) or the partial sums into `part`.  T of the epilogue's
// tensors: dt.  beside: runs beside the kernel before it (launch.cuh).
cudaError_t launch_gemm(const GemmShape& g, const GemmPlan& p, const GemmOperand& A,
                        const GemmOperand& B, dprc_dtype dt, const LinearEpi& epi, void* part,
                        bool beside, cudaStream_t s);

// The whole map for a few tokens on the CUDA cores (linear_few.cu).
cudaError_t launch_linear_few(const void* X, const void* W, dprc_dtype dt, int64_t M, int64_t K,
                              int64_t N, const LinearEpi& epi, cudaStream_t s);

// Two products in one launch (no shares), the longer contraction first;
// gemm_together: whether that is estimated to be faster than one by one.
struct GemmTask {
  const GemmShape* shape = nullptr;
  const GemmPlan* plan = nullptr;
  GemmOperand A, B;
  LinearEpi epi;
};
bool gemm_together(const GemmShape& g0, const GemmPlan& p0, const GemmShape& g1,
                   const GemmPlan& p1);
cudaError_t launch_gemm_two(const GemmTask& t0, const GemmTask& t1, dprc_dtype dt,
                            cudaStream_t s);

}  // namespace dprc
