// The linear map for a few tokens (a decoding step): Y = res + drop(act(X W^T + b))
// with X [M][K], M small, on the CUDA cores.
//
// The weights are read once, at their own width, and that is the bound: with M
// tokens there are M multiply-adds per weight, below what the cores do while
// the weights arrive up to some eight tokens.  The tensor-core path
// (linear_gemm.cu) pays for its start and the sum of its shares and, for fp32, a
// pass that writes the weights' three planes; here the cores start at once.
//
// A warp takes kFeat features (rows of W) and up to kTok tokens: a lane reads
// one 16-byte access of each row and of each token per step, lanes side by
// side along K, and keeps kFeat x kTok sums (pairs, for the two-wide fp32
// multiply-add).  X comes through L1, which holds it.  The warps of a CTA
// share a feature group's K range `ksplit` ways where there are too few
// features to fill the GPU, and add up through shared memory.  More tokens
// than kTok: another row of CTAs, whose weights come from L2.

#include "launch.cuh"
#include "linear.cuh"

namespace dprc {
namespace {

constexpr int kFeat = 4;
constexpr int kFewWarps = 8;

struct FewArgs {
  const void* X;
  const void* W;
  long long M;
  int K, N, ksplit;
  LinearEpi epi;
};

__device__ __forceinline__ unsigned long long few_pair(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void few_fma2(unsigned long long& acc, unsigned long long a,
                                         unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ float few_sum(unsigned long long a) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
  return lo + hi;
}

// The pairs of one access: 16 bytes, or one element (kVec false) as a pair
// with zero.
template <typename T, bool kVec>
struct FewAccess {
  static constexpr int kElems = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
  static constexpr int kPairs = kVec ? kElems / 2 : 1;
  uint4 raw;
  __device__ __forceinline__ void load(const T* p, bool in) {
    if constexpr (kVec) {
      raw = in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
    } else {
      raw.x = in ? __float_as_uint(to_f32<T>(*p)) : 0u;
    }
  }
  // A weight, read once: not kept in L1, which is X's (fp32, 2048 x 8192, four
  // tokens: 29.5 us with both in L1, 22 so, 16.5 with four steps at a time; 18.9 with
  // .cg loads instead).
  __device__ __forceinline__ void load_once(const T* p, bool in) {
    if constexpr (kVec) {
      raw = in ? ld_once(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
    } else {
      load(p, in);
    }
  }
  __device__ __forceinline__ void pairs(unsigned long long* v) const {
    if constexpr (!kVec) {
      v[0] = few_pair(__uint_as_float(raw.x), 0.f);
    } else if constexpr (sizeof(T) == 4) {
      v[0] = few_pair(__uint_as_float(raw.x), __uint_as_float(raw.y));
      v[1] = few_pair(__uint_as_float(raw.z), __uint_as_float(raw.w));
    } else {
      const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = few_pair(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
    }
  }
};

// One output: z = sum + bias, Z, act, drop, residual, Y.
template <typename T>
__device__ __forceinline__ void few_out(const LinearEpi& e, long long m, int n, float v) {
  const long long at = m * e.N + n;
  if (!DPRC_IN(m < e.M && n < e.N)) return;
  float x[8] = {v, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (e.bias != nullptr) x[0] += to_f32<T>(static_cast<const T*>(e.bias)[n]);
  if (e.Z != nullptr) st1(static_cast<T*>(e.Z) + at, x[0]);
  act_value8<sizeof(T) == 2>(x, e.act);
  if (e.drop.thr != 0) {
    const RoundKeys rk = round_keys(e.drop.seed);
    const uint4 w = philox_block(static_cast<uint64_t>(at) >> 3, e.drop.step, rk);
    x[0] = drop_keep(w, static_cast<int>(at & 7), e.drop.thr) ? x[0] * e.drop.keep : 0.f;
  }
  if (e.res != nullptr) x[0] += to_f32<T>(static_cast<const T*>(e.res)[at]);
  st1(static_cast<T*>(e.Y) + at, x[0]);
}

template <typename T, bool kVec, int kTok>
__global__ void __launch_bounds__(32 * kFewWarps) linear_few_kernel(const FewArgs a) {
  using Access = FewAccess<T, kVec>;
  constexpr int kVals = kFeat * kTok;  // sums of a warp
  static_assert(kVals <= 32 && (kVals & (kVals - 1)) == 0, "one lane per sum");
  __shared__ float s_sum[kFewWarps][kVals];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = kFewWarps / a.ksplit;  // feature groups of the CTA
  const int group = warp / a.ksplit, share = warp % a.ksplit;
  const int n0 = (static_cast<int>(blockIdx.x) * groups + group) * kFeat;
  const long long m0 = static_cast<long long>(blockIdx.y) * kTok;

  // this warp's part of K, in whole steps of 32 accesses
  constexpr int kStep = 32 * Access::kElems;
  const int steps = (a.K + kStep - 1) / kStep;
  const int per = (steps + a.ksplit - 1) / a.ksplit;
  const int k_lo = min(share * per * kStep, a.K), k_hi = min((share + 1) * per * kStep, a.K);

  const T* w[kFeat];
  const T* x[kTok];
#pragma unroll
  for (int f = 0; f < kFeat; ++f)
    w[f] = static_cast<const T*>(a.W) + static_cast<long long>(min(n0 + f, a.N - 1)) * a.K;
#pragma unroll
  for (int t = 0; t < kTok; ++t)
    x[t] = static_cast<const T*>(a.X) + min(m0 + t, a.M - 1) * a.K;

  unsigned long long acc[kFeat][kTok];
#pragma unroll
  for (int f = 0; f < kFeat; ++f)
#pragma unroll
    for (int t = 0; t < kTok; ++t) acc[f][t] = 0ull;

  // (the loads of two steps together, of four where an access is only four
  // values: fp32 with 2, 4, 8 tokens 16.3, 22, 31.5 us by twos and 15.7, 16.5,
  // 28.1 by fours, bf16 9.7, 10.2, 19.7 and 9.1, 16.3, 20.5; four features and
  // not two: what a step waits for is X from L1, and two features read it twice
  // as often: 32 us and not 20 us for 8 tokens, 2048 x 8192 bf16)
  constexpr int kAhead = kVec && sizeof(T) == 4 ? 4 : 2;
#pragma unroll kAhead
  for (int k = k_lo + lane * Access::kElems; k - lane * Access::kElems < k_hi; k += kStep) {
    const bool in = k < k_hi;
    Access wa[kFeat];
#pragma unroll
    for (int f = 0; f < kFeat; ++f) wa[f].load_once(w[f] + k, in);
    unsigned long long wp[kFeat][Access::kPairs];
#pragma unroll
    for (int f = 0; f < kFeat; ++f) wa[f].pairs(wp[f]);
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      Access xa;
      xa.load(x[t] + k, in);
      unsigned long long xp[Access::kPairs];
      xa.pairs(xp);
#pragma unroll
      for (int f = 0; f < kFeat; ++f)
#pragma unroll
        for (int i = 0; i < Access::kPairs; ++i) few_fma2(acc[f][t], wp[f][i], xp[i]);
    }
  }

  // Every sum over the lanes, all at once: lanes h apart share the sums out
  // between them; what is left is one sum per 32 / kVals lanes.
  float v[kVals];
#pragma unroll
  for (int f = 0; f < kFeat; ++f)
#pragma unroll
    for (int t = 0; t < kTok; ++t) v[t * kFeat + f] = few_sum(acc[f][t]);
  int h = 16;
#pragma unroll
  for (int n = kVals / 2; n > 0; n >>= 1, h >>= 1) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float give = up ? v[r] : v[r + n];
      const float keep = up ? v[r + n] : v[r];
      v[r] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  for (; h > 0; h >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], h);
  constexpr int kEach = 32 / kVals;  // lanes that hold the same sum
  const int mine = lane / kEach;     // its index
  if (a.ksplit > 1) {
    if (lane % kEach == 0) s_sum[warp][mine] = v[0];
    __syncthreads();
    if (share != 0) return;
    v[0] = 0.f;
    for (int s = 0; s < a.ksplit; ++s) v[0] += s_sum[warp + s][mine];
  }
  const int n = n0 + mine % kFeat;
  const long long m = m0 + mine / kFeat;
  if (lane % kEach == 0 && n < a.N && m < a.M) few_out<T>(a.epi, m, n, v[0]);
}

template <typename T, bool kVec>
cudaError_t launch_few_t(const FewArgs& a, int tok, cudaStream_t s) {
  const int groups = kFewWarps / a.ksplit;
  const int per = groups * kFeat;
  const dim3 grid(static_cast<unsigned>((a.N + per - 1) / per),
                  static_cast<unsigned>((a.M + tok - 1) / tok));
  auto* kernel = tok == 1   ? linear_few_kernel<T, kVec, 1>
                 : tok == 2 ? linear_few_kernel<T, kVec, 2>
                 : tok == 4 ? linear_few_kernel<T, kVec, 4>
                            : linear_few_kernel<T, kVec, 8>;
  return launch_after(kernel, grid, 32 * kFewWarps, 1, s, 0, a);
}

}  // namespace

cudaError_t read_device_error_linear_few(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

cudaError_t launch_linear_few(const void* X, const void* W, dprc_dtype dt, int64_t M, int64_t K,
                              int64_t N, const LinearEpi& epi, cudaStream_t s) {
  FewArgs a;
  a.X = X;
  a.W = W;
  a.M = M;
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.epi = epi;
  const int tok = M > 4 ? 8 : M > 2 ? 4 : static_cast<int>(M);
  const int elems = 16 / (dt == DPRC_F32 ? 4 : 2);
  const bool vec = K % elems == 0;
  // warps for all SMs (16 each) before whole K ranges per warp, while a share
  // keeps a few steps
  const int64_t steps = (K + 32 * (vec ? elems : 1) - 1) / (32 * (vec ? elems : 1));
  const int64_t warps = (N + kFeat - 1) / kFeat * ((M + tok - 1) / tok);
  a.ksplit = 1;
  while (a.ksplit < kFewWarps && warps * a.ksplit < 16 * int64_t(device_sm_count()) &&
         steps >= 4 * a.ksplit)
    a.ksplit *= 2;
  using bf16 = __nv_bfloat16;
  if (dt == DPRC_F32)
    return vec ? launch_few_t<float, true>(a, tok, s) : launch_few_t<float, false>(a, tok, s);
  return vec ? launch_few_t<bf16, true>(a, tok, s) : launch_few_t<bf16, false>(a, tok, s);
}

}  // namespace dprc
