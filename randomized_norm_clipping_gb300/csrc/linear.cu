// The linear map with its epilogue, and its gradient: operand preparation, the
// elementwise part of the gradient, the sums of partial products, and the
// order of the launches.  The products themselves are in linear_gemm.cu.
//
//   Z = X W^T + b,  Y = res + drop(act(Z))
//   dZ = drop(dY) act'(Z),  dX = dZ W,  dW = dZ^T X,  db = sum_m dZ
//
// Operands reach the tensor cores as they are stored when they are bf16 with
// rows of a multiple of 16 bytes.  fp32 operands are split into three bf16
// planes, and rows of another length are copied to a padded pitch, by one
// streaming pass before the product.

#include "launch.cuh"
#include "linear.cuh"

#include <algorithm>

namespace dprc {
namespace {

// ---------------------------------------------------------------------------
// Operand preparation: src [rows][cols] into bf16 planes [P][rows][ld], P = 3
// for fp32, 1 for bf16.  Up to two operands per launch (blockIdx.y).
// ---------------------------------------------------------------------------
struct PackJob {
  const void* src = nullptr;
  __nv_bfloat16* dst = nullptr;
  long long rows = 0;
  int cols = 0, ld = 0;
  long long plane = 0;
};
struct PackArgs {
  PackJob job[2];
  int beside = 0;  // runs beside the kernel before (launch.cuh)
};

__device__ __forceinline__ uint4 pack_bf16x8(const __nv_bfloat16* h) {
  return *reinterpret_cast<const uint4*>(h);
}

// x = x0 + x1 + x2, each the bf16 rounding of what is left (the first one
// towards zero where rounding to nearest would leave bf16's range).  An
// infinity or NaN is its first plane alone.
__device__ __forceinline__ void split3(float x, __nv_bfloat16* p) {
  p[0] = __float2bfloat16_rn(x);
  if (isinf(__bfloat162float(p[0]))) p[0] = __float2bfloat16_rz(x);
  const float r0 = __bfloat162float(p[0]);
  const float r = isfinite(r0) ? x - r0 : 0.f;
  p[1] = __float2bfloat16_rn(r);
  p[2] = __float2bfloat16_rn(r - __bfloat162float(p[1]));
}

template <typename T>
__device__ __forceinline__ void store_planes(__nv_bfloat16* dst, long long plane, const float* v) {
  if constexpr (sizeof(T) == 2) {
    st8(dst, v);
  } else {
    __align__(16) __nv_bfloat16 h[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      __nv_bfloat16 t[3];
      split3(v[e], t);
      h[0][e] = t[0];
      h[1][e] = t[1];
      h[2][e] = t[2];
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint4*>(dst + p * plane) = pack_bf16x8(h[p]);
  }
}

// One value, not through L1: a kernel beside another one reads what was written
// before both.
__device__ __forceinline__ float ld1_l2(const float* p) { return ld_l2(p); }
__device__ __forceinline__ float ld1_l2(const __nv_bfloat16* p) {
  const unsigned short u = ld_l2(reinterpret_cast<const unsigned short*>(p));
  return __uint_as_float(static_cast<uint32_t>(u) << 16);
}
__device__ __forceinline__ void ld8_l2(const float* p, float* v) {
  const float4 a = ld_l2(reinterpret_cast<const float4*>(p));
  const float4 b = ld_l2(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ld8_l2(const __nv_bfloat16* p, float* v) {
  const uint4 a = ld_l2(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(u[e] << 16);
    v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}

// Rows of whole 16-byte accesses: eight values a thread.  Others: a warp reads 256
// values of a row side by side and turns them in shared memory into eight a lane
// (the map 16384 x 2049 x 2048 bf16 202 -> 160 us).
template <typename T>
__global__ void __launch_bounds__(256) linear_pack_kernel(const PackArgs a) {
  __shared__ float4 s_row[8][64];
  beside_begin(a.beside != 0);
  const PackJob& j = a.job[blockIdx.y];
  const T* src = static_cast<const T*>(j.src);
  const int groups = j.ld / 8;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (j.cols % 8 == 0) {
    const long long total = j.rows * groups;
    for (long long i = first; i < total; i += stride) {
      const long long row = i / groups;
      const int c = static_cast<int>(i - row * groups) * 8;
      float v[8];
      ld8_l2(src + row * j.cols + c, v);
      store_planes<T>(j.dst + row * j.ld + c, j.plane, v);
    }
  } else {
    const int lane = threadIdx.x & 31;
    float4* const mine = s_row[threadIdx.x >> 5];
    const int chunks = (j.ld + 255) / 256;
    const long long total = j.rows * chunks;
    for (long long i = first >> 5; i < total; i += stride >> 5) {
      const long long row = i / chunks;
      const int c0 = static_cast<int>(i - row * chunks) * 256;
      const T* p = src + row * j.cols;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + 32 * e + lane;
        v[e] = c < j.cols ? ld1_l2(p + c) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) reinterpret_cast<float*>(mine)[32 * e + lane] = v[e];
      __syncwarp();
      const float4 x = mine[2 * lane], y = mine[2 * lane + 1];
      __syncwarp();
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
      if (c0 + 8 * lane < j.ld) store_planes<T>(j.dst + row * j.ld + c0 + 8 * lane, j.plane, v);
    }
  }
  beside_end(a.beside != 0);
}

// ---------------------------------------------------------------------------
// dZ = drop(dY) act'(Z), elementwise in fp32, rounded once to bf16 (or split
// into planes) for the products; and its column sums, which take the unrounded
// values.  A CTA takes a block of rows of 256 columns; its 8 warps take every 8th
// row, and their column sums are added in warp order.  The rounding of dZ to
// bf16 is the product's operand type: relative 2^-9 per element, as the
// rounding of the results.
// ---------------------------------------------------------------------------
constexpr int kDzWarps = 8;
constexpr int kDzAhead = 2;

// Eight values as they are stored, so that rows on their way cost few registers.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void raw_ld(const T* p, int cnt, bool vec, Raw8<T>& r) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      r.v[i] = ld_stream(reinterpret_cast<const uint4*>(p) + i);
  } else {
    T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < cnt ? p[i] : static_cast<T>(0.f);
  }
}
__device__ __forceinline__ void raw_get(const Raw8<float>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.v[i].x);
    v[4 * i + 1] = __uint_as_float(r.v[i].y);
    v[4 * i + 2] = __uint_as_float(r.v[i].z);
    v[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
__device__ __forceinline__ void raw_get(const Raw8<__nv_bfloat16>& r, float* v) {
  const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(u[e] << 16);
    v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}

struct DzArgs {
  const void* dY;
  const void* Z;
  long long M;
  int N, vec, act, rows;  // rows of a CTA
  DropArgs drop;
  __nv_bfloat16* planes;  // or null
  long long plane;
  int ldp;
  void* dZ;               // the caller's, or null
  float* colsum;          // [row blocks][N], or null
};

template <typename T>
__global__ void __launch_bounds__(32 * kDzWarps, 4) linear_dz_kernel(const DzArgs a) {
  __shared__ float s_sum[kDzWarps][256];
  beside_begin(false);
  constexpr bool kFast = sizeof(T) == 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ncb = (a.N + 255) / 256;
  const int rb = static_cast<int>(blockIdx.x / ncb), cb = static_cast<int>(blockIdx.x % ncb);
  const int n0 = cb * 256 + lane * 8;
  const int cnt = min(8, a.N - n0);
  const long long m0 = static_cast<long long>(rb) * a.rows;
  const RoundKeys rk = round_keys(a.drop.seed);
  const bool vec = a.vec != 0;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (cnt > 0) {
#pragma unroll 1
    for (int r0 = warp; r0 < a.rows; r0 += kDzWarps * kDzAhead) {
      Raw8<T> g8[kDzAhead], z8[kDzAhead];
#pragma unroll
      for (int u = 0; u < kDzAhead; ++u) {
        const long long m = m0 + r0 + u * kDzWarps;
        if (r0 + u * kDzWarps >= a.rows || m >= a.M) continue;
        raw_ld(static_cast<const T*>(a.dY) + m * a.N + n0, cnt, vec, g8[u]);
        if (a.act != DPRC_ACT_NONE)
          raw_ld(static_cast<const T*>(a.Z) + m * a.N + n0, cnt, vec, z8[u]);
      }
#pragma unroll
      for (int u = 0; u < kDzAhead; ++u) {
        const long long m = m0 + r0 + u * kDzWarps;
        if (r0 + u * kDzWarps >= a.rows || m >= a.M) continue;
        float g[8], z[8];
        raw_get(g8[u], g);
        if (a.drop.thr != 0) drop8_at(g, static_cast<uint64_t>(m * a.N + n0), a.drop, rk);
        if (a.act != DPRC_ACT_NONE) {
          raw_get(z8[u], z);
          act_slope8<kFast>(g, z, a.act);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = e < cnt ? g[e] : 0.f;
        if (a.colsum != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += g[e];
        }
        if (a.dZ != nullptr) st_n<T>(static_cast<T*>(a.dZ) + m * a.N + n0, cnt, vec, g);
        if (a.planes != nullptr && DPRC_IN(m < a.M && n0 + 8 <= a.ldp))
          store_planes<T>(a.planes + m * a.ldp + n0, a.plane, g);
      }
    }
  }
  if (a.colsum == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) s_sum[warp][lane * 8 + e] = sum[e];
  __syncthreads();
  const int c = cb * 256 + threadIdx.x;
  if (c < a.N) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kDzWarps; ++w) t += s_sum[w][threadIdx.x];
    a.colsum[static_cast<long long>(rb) * a.N + c] = t;
  }
}

// dZ without the column sums, where its rows are whole 16-byte accesses: then
// [M][N] is one run of groups of 8, and threads with little state stream it at
// 0.98 of the copy rate (16384 x 8192 bf16, SiLU: 121 us; the kernel above 139,
// with dropout 197 against 122).
template <typename T, bool kDrop>
__global__ void __launch_bounds__(256) linear_dz_flat_kernel(const DzArgs a) {
  beside_begin(false);
  constexpr bool kFast = sizeof(T) == 2;
  const long long groups = a.M * (a.N / 8);
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const RoundKeys rk = round_keys(a.drop.seed);
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < groups;
       i += stride) {
    Raw8<T> g8, z8;
    raw_ld(static_cast<const T*>(a.dY) + 8 * i, 8, true, g8);
    if (a.act != DPRC_ACT_NONE) raw_ld(static_cast<const T*>(a.Z) + 8 * i, 8, true, z8);
    float g[8], z[8];
    raw_get(g8, g);
    if (kDrop)
      drop8(g, philox_block(static_cast<uint64_t>(i), a.drop.step, rk), a.drop.thr, a.drop.keep);
    if (a.act != DPRC_ACT_NONE) {
      raw_get(z8, z);
      act_slope8<kFast>(g, z, a.act);
    }
    if (a.dZ != nullptr) st8(static_cast<T*>(a.dZ) + 8 * i, g);
    if (a.planes != nullptr) store_planes<T>(a.planes + 8 * i, a.plane, g);
  }
}

// db[n] = sum over the row blocks, 32 columns and 8 shares per CTA.
template <typename T>
__global__ void __launch_bounds__(256)
    linear_db_kernel(const float* colsum, int nblocks, int N, T* db, int beside) {
  __shared__ float s_sum[8][32];
  beside_begin(beside != 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  const int share = (nblocks + 7) / 8;
  const int b0 = warp * share, b1 = min(b0 + share, nblocks);
  float t = 0.f;
  if (c < N) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) t += ld_l2(colsum + static_cast<long long>(b) * N + c);
  }
  s_sum[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && c < N) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += s_sum[w][lane];
    st1(db + c, s);
  }
  beside_end(beside != 0);
}

// ---------------------------------------------------------------------------
// The shares of a product added in order, then the epilogue: 8 outputs a thread.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
    linear_finish_kernel(const float* part, long long ldpart, long long stride, int split,
                         const LinearEpi e) {
  pdl_launch_dependents();
  pdl_wait();
  const int groups = (e.N + 7) / 8;
  const long long total = e.M * groups;
  const RoundKeys rk = round_keys(e.drop.seed);
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += step) {
    const long long m = i / groups;
    const int n = static_cast<int>(i - m * groups) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const float* p = part + m * ldpart + n;
#pragma unroll 4
    for (int s = 0; s < split; ++s) {
      const float4 a = ld_l2(reinterpret_cast<const float4*>(p + s * stride));
      const float4 b = ld_l2(reinterpret_cast<const float4*>(p + s * stride) + 1);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    linear_out<T, 1>(e, m, n, v, rk);
  }
}

size_t up1k(size_t x) { return (x + 1023) / 1024 * 1024; }
int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }

unsigned stride_grid(int64_t threads) {
  int64_t ctas = (threads + 255) / 256;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 32;
  return static_cast<unsigned>(ctas < 1 ? 1 : ctas > cap ? cap : ctas);
}

cudaError_t launch_pack(dprc_dtype dt, const PackJob* jobs, int n, bool beside, cudaStream_t s) {
  PackArgs a;
  a.beside = beside;
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    a.job[i] = jobs[i];
    const int64_t warps = jobs[i].rows * ((jobs[i].ld + 255) / 256);
    most = std::max<int64_t>(
        most, jobs[i].cols % 8 == 0 ? jobs[i].rows * (jobs[i].ld / 8) : 32 * warps);
  }
  const dim3 grid(stride_grid(most), n);
  return dt == DPRC_F32 ? launch_after(linear_pack_kernel<float>, grid, 256, 1, s, 0, a)
                        : launch_after(linear_pack_kernel<__nv_bfloat16>, grid, 256, 1, s, 0, a);
}

// The sum of a product's shares, where it is in shares, and the epilogue.
cudaError_t launch_finish(const GemmShape& g, const GemmPlan& p, dprc_dtype dt,
                          const LinearEpi& epi, const void* part, cudaStream_t s) {
  if (p.part_bytes == 0) return cudaSuccess;
  const unsigned grid = stride_grid(epi.M * ((epi.N + 7) / 8));
  const long long stride = (g.transposed ? g.cols : g.rows) * p.ldpart;
  const float* sums = static_cast<const float*>(part);
  const long long ld = p.ldpart;
  return dt == DPRC_F32 ? launch_after(linear_finish_kernel<float>, grid, 256, 1, s, 0, sums, ld,
                                       stride, p.split, epi)
                        : launch_after(linear_finish_kernel<__nv_bfloat16>, grid, 256, 1, s, 0,
                                       sums, ld, stride, p.split, epi);
}

// At most this many tokens take the tile's columns and the weights its lanes
// (linear_gemm.cu); with more, the tokens fill half a tile's lanes or more.
constexpr int64_t kFewTokens = 64;

// Whether the forward map of M tokens runs on the CUDA cores (linear_few.cu).
// Measured with the weights in turn in L2 and memory (us, CUDA cores / tensor
// cores): bf16 2048 x 8192 M = 1 6.9 / 10.0, M = 4 10.1 / 10.2, M = 8 19.7 / 10.2;
// 2048 x 512 M = 16 3.1 / 5.6, M = 32 5.6 / 6.3, M = 64 10.3 / 7.0; fp32
// 2048 x 8192 M = 8 28 / 72, M = 24 51 / 67, M = 32 63 / 67, M = 64 111 / 71;
// 8192 x 2048 M = 32 70 / 68; 2048 x 512 M = 64 11.3 / 17.9.  The cores' time grows with N K M, the other's with N K: they
// cross where N K (M - m) is a constant.
bool few_tokens(dprc_dtype dt, int64_t M, int64_t K, int64_t N) {
  if (M > kFewTokens) return false;
  const int64_t nk = N * K;
  return dt == DPRC_F32 ? nk * (M - 26) <= 100000000 : nk * (M - 2) <= 32000000;
}

// LinearEpi::vec for rows of N elements at these addresses (null: not used).
int row_access(dprc_dtype dt, int64_t N, const void* a, const void* b, const void* c) {
  if (N % 8 != 0) return 0;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                        reinterpret_cast<uintptr_t>(c);
  return dt == DPRC_BF16 && N % 16 == 0 && all % 32 == 0 ? 2 : 1;
}

// Sizes and workspace of a forward call.
struct LinearPlan {
  bool few = false, pack = false;
  int planes = 1;
  int64_t ld = 0;
  GemmShape g;
  GemmPlan p;
  size_t x_off = 0, w_off = 0, part_off = 0, total = 0;
};

LinearPlan linear_plan(dprc_dtype dt, int64_t M, int64_t K, int64_t N) {
  LinearPlan l;
  l.few = few_tokens(dt, M, K, N);
  if (l.few) {
    l.total = 1024;  // none; a call without a workspace stays an error
    return l;
  }
  l.planes = dt == DPRC_F32 ? 3 : 1;
  l.pack = dt == DPRC_F32 || K % 8 != 0;
  l.ld = l.pack ? up8(K) : K;
  l.g.transposed = M <= kFewTokens;
  l.g.rows = l.g.transposed ? N : M;
  l.g.cols = l.g.transposed ? M : N;
  l.g.K = K;
  l.g.planes = l.planes;
  l.p = plan_gemm(l.g);
  size_t off = 0;
  if (l.pack) {
    l.x_off = off;
    off = up1k(off + static_cast<size_t>(l.planes) * M * l.ld * 2);
    l.w_off = off;
    off = up1k(off + static_cast<size_t>(l.planes) * N * l.ld * 2);
  }
  l.part_off = off;
  off = up1k(off + l.p.part_bytes);
  l.total = off > 0 ? off : 1024;
  return l;
}

// Sizes and workspace of a gradient call.
struct LinearGradPlan {
  bool pack = false;
  int planes = 1;
  int64_t ldk = 0, ldn = 0, nblocks = 0;
  int dz_rows = 64;
  GemmShape gx, gw;
  GemmPlan px, pw;
  bool together = false;    // dX and dW in one launch
  size_t dz_off = 0, x_off = 0, w_off = 0, sum_off = 0, part_off = 0, total = 0;
};

LinearGradPlan linear_grad_plan(dprc_dtype dt, int64_t M, int64_t K, int64_t N) {
  LinearGradPlan l;
  if (M == 0) {
    l.total = 1024;  // no product runs; a call without a workspace stays an error
    return l;
  }
  l.planes = dt == DPRC_F32 ? 3 : 1;
  l.pack = dt == DPRC_F32 || K % 8 != 0;
  l.ldk = l.pack ? up8(K) : K;
  l.ldn = up8(N);
  // rows of a CTA: 64 while that fills the GPU twice, at least one per warp
  l.dz_rows = 64;
  while (l.dz_rows > kDzWarps &&
         (M + l.dz_rows - 1) / l.dz_rows * ((N + 255) / 256) < 4 * int64_t(device_sm_count()))
    l.dz_rows /= 2;
  l.nblocks = (M + l.dz_rows - 1) / l.dz_rows;
  l.gx.transposed = M <= kFewTokens;
  l.gx.rows = l.gx.transposed ? K : M;
  l.gx.cols = l.gx.transposed ? M : K;
  l.gx.K = N;
  l.gx.planes = l.planes;
  l.px = plan_gemm(l.gx);
  l.gw.rows = N;
  l.gw.cols = K;
  l.gw.K = M;
  l.gw.planes = l.planes;
  l.pw = plan_gemm(l.gw);
  const bool w_first = M >= N;
  l.together = w_first ? gemm_together(l.gw, l.pw, l.gx, l.px)
                       : gemm_together(l.gx, l.px, l.gw, l.pw);
  size_t off = 0;
  l.dz_off = off;
  off = up1k(off + static_cast<size_t>(l.planes) * M * l.ldn * 2);
  if (l.pack) {
    l.x_off = off;
    off = up1k(off + static_cast<size_t>(l.planes) * M * l.ldk * 2);
    l.w_off = off;
    off = up1k(off + static_cast<size_t>(l.planes) * N * l.ldk * 2);
  }
  l.sum_off = off;
  off = up1k(off + static_cast<size_t>(l.nblocks) * N * 4);
  // the two products run one after the other on the stream and share this
  l.part_off = off;
  off = up1k(off + std::max(l.px.part_bytes, l.pw.part_bytes));
  l.total = off > 0 ? off : 1024;
  return l;
}

}  // namespace

cudaError_t read_device_error_linear_prep(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

size_t linear_ws_bytes(dprc_dtype dt, int64_t M, int64_t K, int64_t N) {
  return linear_plan(dt, M, K, N).total;
}
size_t linear_grad_ws_bytes(dprc_dtype dt, int64_t M, int64_t K, int64_t N) {
  return linear_grad_plan(dt, M, K, N).total;
}

cudaError_t launch_linear(const LinearCall& c, void* ws, cudaStream_t s) {
  if (c.M == 0) return cudaSuccess;
  const LinearPlan l = linear_plan(c.dtype, c.M, c.K, c.N);
  LinearEpi epi;
  epi.M = c.M;
  epi.N = static_cast<int>(c.N);
  epi.vec = row_access(c.dtype, c.N, c.res, c.Z, c.Y);
  epi.act = c.act;
  epi.bias = c.bias;
  epi.res = c.res;
  epi.Z = c.Z;
  epi.Y = c.Y;
  epi.drop = drop_args(c.p, c.seed, c.step);
  if (l.few) return launch_linear_few(c.X, c.W, c.dtype, c.M, c.K, c.N, epi, s);

  char* w = static_cast<char*>(ws);
  cudaError_t e = cudaSuccess;
  GemmOperand x, wt;
  x.data = c.X;
  wt.data = c.W;
  x.ld = wt.ld = l.ld;
  x.plane = c.M * l.ld;
  wt.plane = c.N * l.ld;
  if (l.pack) {
    PackJob jobs[2];
    const void* src[2] = {c.X, c.W};
    const int64_t rows[2] = {c.M, c.N};
    const size_t off[2] = {l.x_off, l.w_off};
    for (int i = 0; i < 2; ++i) {
      jobs[i].src = src[i];
      jobs[i].dst = reinterpret_cast<__nv_bfloat16*>(w + off[i]);
      jobs[i].rows = rows[i];
      jobs[i].cols = static_cast<int>(c.K);
      jobs[i].ld = static_cast<int>(l.ld);
      jobs[i].plane = rows[i] * l.ld;
    }
    e = launch_pack(c.dtype, jobs, 2, false, s);
    if (e != cudaSuccess) return e;
    x.data = jobs[0].dst;
    wt.data = jobs[1].dst;
  }
  void* part = w + l.part_off;
  e = launch_gemm(l.g, l.p, l.g.transposed ? wt : x, l.g.transposed ? x : wt, c.dtype, epi, part,
                  false, s);
  return e == cudaSuccess ? launch_finish(l.g, l.p, c.dtype, epi, part, s) : e;
}

cudaError_t launch_linear_grad(const LinearGradCall& c, void* ws, cudaStream_t s) {
  const int elem = c.dtype == DPRC_F32 ? 4 : 2;
  if (c.M == 0) {  // no tokens: nothing to add up
    cudaError_t e = cudaSuccess;
    if (c.dW != nullptr) e = cudaMemsetAsync(c.dW, 0, static_cast<size_t>(c.N) * c.K * elem, s);
    if (e == cudaSuccess && c.db != nullptr)
      e = cudaMemsetAsync(c.db, 0, static_cast<size_t>(c.N) * elem, s);
    return e;
  }
  const LinearGradPlan l = linear_grad_plan(c.dtype, c.M, c.K, c.N);
  char* w = static_cast<char*>(ws);
  const DropArgs drop = drop_args(c.p, c.seed, c.step);
  const bool products = c.dX != nullptr || c.dW != nullptr;
  const bool direct = c.dtype == DPRC_BF16 && c.N % 8 == 0;  // TMA reads [M][N] as it is
  const bool same = c.act == DPRC_ACT_NONE && drop.thr == 0;  // dZ = dY
  cudaError_t e = cudaSuccess;

  GemmOperand dz;
  dz.ld = l.ldn;
  dz.plane = c.M * l.ldn;
  __nv_bfloat16* planes = nullptr;
  if (same && direct) {
    dz.data = c.dY;
  } else if (direct && c.dZ != nullptr) {
    dz.data = c.dZ;
  } else if (products) {
    planes = reinterpret_cast<__nv_bfloat16*>(w + l.dz_off);
    dz.data = planes;
  }
  const bool dz_runs = planes != nullptr || c.dZ != nullptr || c.db != nullptr;
  if (dz_runs) {
    DzArgs a;
    a.dY = c.dY;
    a.Z = c.Z;
    a.M = c.M;
    a.N = static_cast<int>(c.N);
    a.vec = c.N % 8 == 0;
    a.act = c.act;
    a.rows = l.dz_rows;
    a.drop = drop;
    a.planes = planes;
    a.plane = dz.plane;
    a.ldp = static_cast<int>(l.ldn);
    a.dZ = c.dZ;
    a.colsum = c.db != nullptr ? reinterpret_cast<float*>(w + l.sum_off) : nullptr;
    const unsigned grid = static_cast<unsigned>((c.N + 255) / 256 * l.nblocks);
    using bf16 = __nv_bfloat16;
    if (c.db == nullptr && a.vec) {
      const int64_t groups = c.M * (c.N / 8);
      const unsigned flat = static_cast<unsigned>(
          std::min<int64_t>((groups + 255) / 256, int64_t(device_sm_count()) * 64));
      auto* kernel = c.dtype == DPRC_F32
                         ? (drop.thr != 0 ? linear_dz_flat_kernel<float, true>
                                          : linear_dz_flat_kernel<float, false>)
                         : (drop.thr != 0 ? linear_dz_flat_kernel<bf16, true>
                                          : linear_dz_flat_kernel<bf16, false>);
      e = launch_after(kernel, dim3(flat), 256, 1, s, 0, a);
    } else {
      auto* kernel = c.dtype == DPRC_F32 ? linear_dz_kernel<float> : linear_dz_kernel<bf16>;
      e = launch_after(kernel, dim3(grid), 32 * kDzWarps, 1, s, 0, a);
    }
    if (e != cudaSuccess) return e;
  }
  const auto finish_db = [&](bool beside) {
    if (c.db == nullptr) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>((c.N + 31) / 32));
    const float* cs = reinterpret_cast<const float*>(w + l.sum_off);
    const int nb = static_cast<int>(l.nblocks), N = static_cast<int>(c.N);
    return c.dtype == DPRC_F32
               ? launch_after(linear_db_kernel<float>, grid, 256, 1, s, 0, cs, nb, N,
                              static_cast<float*>(c.db), int{beside})
               : launch_after(linear_db_kernel<__nv_bfloat16>, grid, 256, 1, s, 0, cs, nb, N,
                              static_cast<__nv_bfloat16*>(c.db), int{beside});
  };
  if (!products) return finish_db(false);

  // What does not depend on one another runs side by side (launch.cuh): the
  // packing beside dZ, the second product beside the first where that one is
  // not in shares, db beside the last product.  fp32, M = 1001, K = 517,
  // N = 263, GELU, dropout and db: 38 us one by one, 28 us so (bf16 38 and 23).

  GemmOperand x, wt;
  x.data = c.X;
  wt.data = c.W;
  x.ld = wt.ld = l.ldk;
  x.plane = c.M * l.ldk;
  wt.plane = c.N * l.ldk;
  if (l.pack) {
    PackJob jobs[2];
    int n = 0;
    if (c.dW != nullptr) {
      jobs[n].src = c.X;
      jobs[n].dst = reinterpret_cast<__nv_bfloat16*>(w + l.x_off);
      jobs[n].rows = c.M;
      x.data = jobs[n++].dst;
    }
    if (c.dX != nullptr) {
      jobs[n].src = c.W;
      jobs[n].dst = reinterpret_cast<__nv_bfloat16*>(w + l.w_off);
      jobs[n].rows = c.N;
      wt.data = jobs[n++].dst;
    }
    for (int i = 0; i < n; ++i) {
      jobs[i].cols = static_cast<int>(c.K);
      jobs[i].ld = static_cast<int>(l.ldk);
      jobs[i].plane = jobs[i].rows * l.ldk;
    }
    e = launch_pack(c.dtype, jobs, n, dz_runs, s);
    if (e != cudaSuccess) return e;
  }
  GemmTask tx, tw;
  tx.shape = &l.gx;
  tx.plan = &l.px;
  GemmOperand wm = wt;
  wm.mn_major = true;
  tx.A = l.gx.transposed ? wm : dz;
  tx.B = l.gx.transposed ? dz : wm;
  tw.shape = &l.gw;
  tw.plan = &l.pw;
  tw.A = dz;
  tw.B = x;
  tw.A.mn_major = tw.B.mn_major = true;
  tx.epi.N = tw.epi.N = static_cast<int>(c.K);
  tx.epi.vec = row_access(c.dtype, c.K, c.dX, nullptr, nullptr);
  tw.epi.vec = row_access(c.dtype, c.K, c.dW, nullptr, nullptr);
  tx.epi.M = c.M;
  tx.epi.Y = c.dX;
  tw.epi.M = c.N;
  tw.epi.Y = c.dW;
  if (c.dX != nullptr && c.dW != nullptr && l.together) {
    const bool w_first = l.gw.K >= l.gx.K;
    e = launch_gemm_two(w_first ? tw : tx, w_first ? tx : tw, c.dtype, s);
    return e == cudaSuccess ? finish_db(true) : e;
  }
  const bool x_shares = l.px.part_bytes > 0, w_shares = l.pw.part_bytes > 0;
  const GemmTask* order[2] = {&tx, &tw};
  if (x_shares && !w_shares) std::swap(order[0], order[1]);
  const GemmTask* last = order[order[1]->epi.Y != nullptr];
  bool beside = false;
  for (const GemmTask* t : order) {
    if (t->epi.Y == nullptr) continue;
    void* part = w + l.part_off;
    e = launch_gemm(*t->shape, *t->plan, t->A, t->B, c.dtype, t->epi, part, beside, s);
    if (e == cudaSuccess && t == last) e = finish_db(true);
    if (e == cudaSuccess) e = launch_finish(*t->shape, *t->plan, c.dtype, t->epi, part, s);
    if (e != cudaSuccess) return e;
    beside = t->plan->part_bytes == 0;
  }
  return cudaSuccess;
}

}  // namespace dprc
