// Dropout from the library's Philox stream, with an optional residual:
//   y_i = r_i + (x_i / (1 - p) or 0)
// with the mask of dropout.cuh for the element first_element + i.  The mask
// is never stored: the backward pass is the same call on the gradient, with
// the same (seed, step) and no residual.
//
// Bound by bytes: it reads x (and r) and writes y once.  8 x 4096 x 2048 bf16 with
// a residual, calls in turn on one stream: 58.2 us, 6.92 TB/s (60.5 with each
// launch behind the full end of the one before).

#include "common.cuh"
#include "dropout.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dprc {
namespace {

constexpr int kDropThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* v) {
  const float4 a = ld_stream(reinterpret_cast<const float4*>(p));
  const float4 b = ld_stream(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint4 a = ld_stream(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(u[e] << 16);
    v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    u[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A thread takes 8 consecutive elements, aligned in memory.  kShift: the
// offset first_element is no multiple of 8, so they span two blocks (twice the
// generator's work); else they are one block.
template <typename T, bool kRes, bool kShift>
__global__ void __launch_bounds__(kDropThreads)
    dropout_kernel(const T* x, const T* res, long long n, uint64_t first, const DropArgs a,
                   T* y) {
  const RoundKeys rk = round_keys(a.seed);
  pdl_launch_dependents();
  pdl_wait();
  const long long nvec = n / 8;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const int sh = static_cast<int>(first & 7);
  for (long long j = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; j < nvec;
       j += stride) {
    float v[8], r[8];
    load8<T>(x + 8 * j, v);
    if (kRes) load8<T>(res + 8 * j, r);
    const uint64_t q = (first >> 3) + static_cast<uint64_t>(j);
    const uint4 w0 = philox_block(q, a.step, rk);
    if constexpr (!kShift) {
      drop8(v, w0, a.thr, a.keep);
    } else {
      const uint4 w1 = philox_block(q + 1, a.step, rk);
      uint32_t keep = 0;  // bit h: half h of the 16 halves is kept
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        keep |= (drop_keep(w0, h, a.thr) ? 1u : 0u) << h;
        keep |= (drop_keep(w1, h, a.thr) ? 1u : 0u) << (h + 8);
      }
      keep >>= sh;
#pragma unroll
      for (int h = 0; h < 8; ++h) v[h] = ((keep >> h) & 1u) ? v[h] * a.keep : 0.f;
    }
    if (kRes) {
#pragma unroll
      for (int h = 0; h < 8; ++h) v[h] += r[h];
    }
    store8(y + 8 * j, v);
  }
  // the last n mod 8 elements, one thread each
  if (blockIdx.x == 0 && threadIdx.x < n - nvec * 8) {
    const long long i = nvec * 8 + threadIdx.x;
    const uint64_t e = first + static_cast<uint64_t>(i);
    const uint4 w = philox_block(e >> 3, a.step, rk);
    float v = drop_keep(w, static_cast<int>(e & 7), a.thr) ? to_f32<T>(x[i]) * a.keep : 0.f;
    if (kRes) v += to_f32<T>(res[i]);
    put(y + i, v);
  }
}

template <typename T>
cudaError_t launch_dropout_t(const T* x, const T* res, int64_t n, uint64_t first,
                             const DropArgs& a, T* y, cudaStream_t s) {
  int64_t ctas = (n / 8 + kDropThreads - 1) / kDropThreads;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 64;
  ctas = ctas < 1 ? 1 : ctas > cap ? cap : ctas;
  const bool shift = (first & 7) != 0;
  auto* kernel = res != nullptr
                     ? (shift ? dropout_kernel<T, true, true> : dropout_kernel<T, true, false>)
                     : (shift ? dropout_kernel<T, false, true> : dropout_kernel<T, false, false>);
  return launch_after(kernel, dim3(static_cast<unsigned>(ctas)), kDropThreads, 1, s, 0, x, res,
                      static_cast<long long>(n), first, a, y);
}

}  // namespace

cudaError_t launch_dropout(const void* x, const void* res, dprc_dtype dt, int64_t n,
                           uint64_t first, double p, uint64_t seed, uint64_t step, void* y,
                           cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const DropArgs a = drop_args(p, seed, step);
  if (dt == DPRC_F32)
    return launch_dropout_t(static_cast<const float*>(x), static_cast<const float*>(res), n,
                            first, a, static_cast<float*>(y), s);
  using bf16 = __nv_bfloat16;
  return launch_dropout_t(static_cast<const bf16*>(x), static_cast<const bf16*>(res), n, first, a,
                          static_cast<bf16*>(y), s);
}

}  // namespace dprc
