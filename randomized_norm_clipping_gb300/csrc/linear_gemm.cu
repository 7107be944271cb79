// The products of the linear map and of its gradient on the tensor cores
// (tcgen05, bf16 operands, fp32 accumulation in TMEM), with the map's
// epilogue.
//
//   Y  = res + drop(act(X W^T + b))    A = X  K-major,  B = W  K-major
//   dX = dZ W                          A = dZ K-major,  B = W  MN-major
//   dW = dZ^T X                        A = dZ MN-major, B = X  MN-major
//
// Persistent CTAs, one per SM, walk units of work: a 128 x kTn tile of D and
// one share of its contraction.  Warp 0 copies operand tiles by TMA into a
// ring of 64-deep stages; one thread of warp 1 issues the MMAs; the other
// warps read the finished accumulator and run the epilogue.  The accumulator
// is double buffered, so a tile's epilogue runs under the next tile's MMAs.
//
// Few tokens: the weights' rows take the 128 lanes of the tile and the tokens
// its kTn columns (16 to 64), so the weights stream through once and the
// tokens cost what they are; D is then stored transposed, by partial sums.
//
// Tiles are walked in blocks of kGroupRows row tiles, all columns of a block
// before the next, so the tiles in flight at one time share their operands in
// L2.

#include <atomic>

#include "linear.cuh"

namespace dprc {
namespace {

constexpr int kTm = 128;
constexpr int kTk = 64;
constexpr int kRing = 192 * 1024;
constexpr int kGroupRows = 16;

template <int kTn>
struct GemmCfg {
  static constexpr int kA = kTm * kTk * 2;
  static constexpr int kB = kTn * kTk * 2;
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = kRing / kStage < 10 ? kRing / kStage : 10;
  static constexpr int kEpiWarps = kTn >= 64 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kCols = kTn / (kEpiWarps / 4);  // columns per epilogue warp
  static constexpr int kTmem = 2 * kTn;
  static constexpr int kSmem = kStages * kStage + 1024 + 512;
};

struct GemmArgs {
  long long rows;
  int cols;
  int mt, nt;               // tiles
  int split;
  int units, per_split;     // contraction units, and of one share
  int npairs;               // plane products per 64 of the contraction (1 or 6)
  int a_mn, b_mn;
  int transposed;
  float* part;              // partial sums, or null: the epilogue
  long long ldpart, part_stride;
  LinearEpi epi;
};

// Plane products of fp32 operands, by size: 1, 2^-8 (2), 2^-16 (3).
__device__ __forceinline__ void plane_pair(int i, int& a, int& b) {
  a = i == 0 || i == 1 || i == 3 ? 0 : i == 5 ? 2 : 1;
  b = i == 0 || i == 2 || i == 5 ? 0 : i == 3 ? 2 : 1;
}

struct GemmUnit {
  int m, n, split, u0, u1;
};

__device__ __forceinline__ GemmUnit gemm_unit(const GemmArgs& a, long long w) {
  GemmUnit g;
  const long long tile = w / a.split;
  g.split = static_cast<int>(w - tile * a.split);
  const long long per_group = static_cast<long long>(kGroupRows) * a.nt;
  const int grp = static_cast<int>(tile / per_group);
  const int rem = static_cast<int>(tile - grp * per_group);
  const int gr = min(kGroupRows, a.mt - grp * kGroupRows);
  g.n = rem / gr;
  g.m = grp * kGroupRows + rem - g.n * gr;
  g.u0 = g.split * a.per_split;
  g.u1 = min(g.u0 + a.per_split, a.units);
  return g;
}

template <int kTn, typename T>
__global__ void __launch_bounds__(GemmCfg<kTn>::kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const GemmArgs a) {
  using Cfg = GemmCfg<kTn>;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * Cfg::kStage);
  uint64_t* empty = full + kStages;
  uint64_t* accf = empty + kStages;  // [2]
  uint64_t* acce = accf + 2;         // [2]
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long nwork = static_cast<long long>(a.mt) * a.nt * a.split;
  const long long mine = nwork > blockIdx.x ? (nwork - 1 - blockIdx.x) / gridDim.x + 1 : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], Cfg::kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0 && mine > 0) {
      long long it = 0;
      bool ok = true;
      for (long long j = 0; j < mine && ok; ++j) {
        const GemmUnit g = gemm_unit(a, blockIdx.x + j * gridDim.x);
        for (int u = g.u0; u < g.u1; ++u, ++it) {
          const int s = static_cast<int>(it % kStages);
          const uint32_t ph = static_cast<uint32_t>(it / kStages) & 1;
          if (!mbar_wait_lim(&empty[s], ph ^ 1, DPRC_DEVERR_PIPE_EMPTY, kWaitLimitNs, abort_flag)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          int pa = 0, pb = 0, kb = u;
          if (a.npairs > 1) {
            kb = u / a.npairs;
            plane_pair(u - kb * a.npairs, pa, pb);
          }
          uint8_t* sa = ring + s * Cfg::kStage;
          uint8_t* sb = sa + Cfg::kA;
          mbar_arrive_expect_tx(&full[s], Cfg::kStage);
          if (a.a_mn) {
#pragma unroll
            for (int h = 0; h < kTm / 64; ++h)
              tma_load_3d(sa + h * (kTk * 128), &map_a, &full[s], g.m * kTm + h * 64, kb * kTk, pa);
          } else {
            tma_load_3d(sa, &map_a, &full[s], kb * kTk, g.m * kTm, pa);
          }
          if (a.b_mn) {
#pragma unroll
            for (int h = 0; h < (kTn + 63) / 64; ++h)
              tma_load_3d(sb + h * (kTk * 128), &map_b, &full[s], g.n * kTn + h * 64, kb * kTk, pb);
          } else {
            tma_load_3d(sb, &map_b, &full[s], kb * kTk, g.n * kTn, pb);
          }
        }
      }
      // let the copies this thread issued land before the CTA can exit
      for (long long k = it - 1; k >= 0 && k >= it - kStages; --k)
        mbar_wait(&full[k % kStages], (k / kStages) & 1, DPRC_DEVERR_PIPE_FULL);
    }
  } else if (warp == 1) {
    if (lane == 0 && mine > 0) {
      const uint32_t idesc = make_idesc_bf16(kTm, kTn, a.a_mn != 0, a.b_mn != 0);
      // K-major, 128-byte swizzle: 8-row atoms 1 KB apart (SBO), a K = 16 step
      // is 32 B along the row.  MN-major: a K = 16 step is 16 rows of 128 B,
      // 64-wide atoms along M or N one 8 KB box apart (LBO).
      const uint32_t a_lbo = a.a_mn ? kTk * 128 : 16, a_step = a.a_mn ? 2048 : 32;
      const uint32_t b_lbo = a.b_mn ? kTk * 128 : 16, b_step = a.b_mn ? 2048 : 32;
      long long it = 0;
      bool ok = true, issued = false;
      for (long long j = 0; j < mine && ok; ++j) {
        const GemmUnit g = gemm_unit(a, blockIdx.x + j * gridDim.x);
        const int abuf = static_cast<int>(j & 1);
        if (!mbar_wait_lim(&acce[abuf], static_cast<uint32_t>((j >> 1) & 1) ^ 1, DPRC_DEVERR_ACCUM,
                           kWaitLimitNs, abort_flag)) {
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        for (int u = g.u0; u < g.u1; ++u, ++it) {
          const int s = static_cast<int>(it % kStages);
          const uint32_t ph = static_cast<uint32_t>(it / kStages) & 1;
          if (!mbar_wait_lim(&full[s], ph, DPRC_DEVERR_PIPE_FULL, kWaitLimitNs, abort_flag)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(ring + s * Cfg::kStage);
          const uint32_t sb = sa + Cfg::kA;
#pragma unroll
          for (int kk = 0; kk < kTk / 16; ++kk) {
            const uint64_t ad = make_sdesc(sa + kk * a_step, a_lbo, 1024, kSwz128);
            const uint64_t bd = make_sdesc(sb + kk * b_step, b_lbo, 1024, kSwz128);
            umma_bf16(tmem + abuf * kTn, ad, bd, idesc, (u == g.u0 && kk == 0) ? 0u : 1u);
          }
          umma_commit(&empty[s]);
          issued = true;
        }
        if (ok) umma_commit(&accf[abuf]);
      }
      if (issued) umma_drain(drain, kWaitLimitNs);
    }
  } else {
    const int ew = warp - 2;
    const int q = warp & 3;  // TMEM lane quadrant this warp may read
    const int c_lo = (ew >> 2) * Cfg::kCols;
    const RoundKeys rk = round_keys(a.epi.drop.seed);
    bool ok = true;
    for (long long j = 0; j < mine; ++j) {
      const GemmUnit g = gemm_unit(a, blockIdx.x + j * gridDim.x);
      const int abuf = static_cast<int>(j & 1);
      bool live = ok && mbar_wait_lim(&accf[abuf], static_cast<uint32_t>((j >> 1) & 1),
                                      DPRC_DEVERR_ACCUM, kWaitLimitNs, abort_flag) &&
                  *abort_flag == 0;
      live = __all_sync(0xffffffffu, live);
      if (!live) ok = false;
      tc_fence_after();
      if (live) {
        const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + abuf * kTn + c_lo;
        const long long row = static_cast<long long>(g.m) * kTm + q * 32 + lane;
        constexpr int kStep = Cfg::kCols < 32 ? Cfg::kCols : 32;
#pragma unroll 1
        for (int c0 = 0; c0 < Cfg::kCols; c0 += kStep) {
          const int col = g.n * kTn + c_lo + c0;
          if (col >= a.cols) break;  // uniform over the warp
          float v[kStep];
          tmem_ld_cols<kStep>(tb + c0, v);
          if (row < a.rows) {
            if (a.transposed) {
              float* out = a.part + g.split * a.part_stride + row;
#pragma unroll
              for (int t = 0; t < kStep; ++t)
                if (col + t < a.cols) out[(col + t) * a.ldpart] = v[t];
            } else if (a.part != nullptr) {
              float* out = a.part + g.split * a.part_stride + row * a.ldpart + col;
#pragma unroll
              for (int t = 0; t < kStep; t += 4)
                if (col + t < a.cols && DPRC_IN(col + t + 4 <= a.ldpart))
                  *reinterpret_cast<float4*>(out + t) =
                      make_float4(v[t], v[t + 1], v[t + 2], v[t + 3]);
            } else {
              linear_out<T, kStep / 8>(a.epi, row, col, v, rk);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[abuf]);
    }
  }

  __syncwarp();  // reconverge each warp before the CTA barrier
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmem);
  }
}

template <int kTn, typename T>
cudaError_t launch_gemm_t(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& a,
                          cudaStream_t s) {
  using Cfg = GemmCfg<kTn>;
  constexpr int kMaxDev = 64;
  static std::atomic<int> done[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(linear_gemm_kernel<kTn, T>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDev) done[dev].store(1, std::memory_order_release);
  }
  const long long work = static_cast<long long>(a.mt) * a.nt * a.split;
  const long long grid = work < device_sm_count() ? work : device_sm_count();
  linear_gemm_kernel<kTn, T>
      <<<static_cast<unsigned>(grid), Cfg::kThreads, Cfg::kSmem, s>>>(ma, mb, a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gemm_tn(int tn, const CUtensorMap& ma, const CUtensorMap& mb,
                           const GemmArgs& a, cudaStream_t s) {
  switch (tn) {
    case 16: return launch_gemm_t<16, T>(ma, mb, a, s);
    case 32: return launch_gemm_t<32, T>(ma, mb, a, s);
    case 64: return launch_gemm_t<64, T>(ma, mb, a, s);
    case 128: return launch_gemm_t<128, T>(ma, mb, a, s);
    default: return launch_gemm_t<256, T>(ma, mb, a, s);
  }
}

// Tensor map of an operand's tiles: a box is 64 of the contraction by
// `tile` rows (K-major) or 64 rows by 64 of the contraction (MN-major).
bool operand_map(CUtensorMap* map, const GemmOperand& o, int64_t dim, int64_t K, int planes,
                 int tile) {
  if (o.mn_major)
    return make_tmap_3d_bf16(map, o.data, dim, K, planes, o.ld, planes > 1 ? o.plane : o.ld * K,
                             64, kTk, 128);
  return make_tmap_3d_bf16(map, o.data, K, dim, planes, o.ld, planes > 1 ? o.plane : o.ld * dim,
                           kTk, tile, 128);
}

}  // namespace

cudaError_t read_device_error_linear(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

GemmPlan plan_gemm(const GemmShape& g) {
  GemmPlan p;
  p.units = (g.K + kTk - 1) / kTk * (g.planes > 1 ? 6 : 1);
  const int sms = device_sm_count();
  const int64_t mt = (g.rows + kTm - 1) / kTm;
  // Candidates: the tile widths and contraction shares; the cost of one is its
  // waves of units (in cycles: a 64-deep step of a 128 x tn tile takes about
  // 2 tn cycles on the tensor core and no less than 192 to copy in), plus
  // what a unit costs outside its MMAs, plus the partial sums' way out and in.
  const int wide[] = {256, 128, 64};
  const int few[] = {16, 32, 64};
  double best = 1e300;
  for (int i = 0; i < 3; ++i) {
    int tn = g.transposed ? few[i] : wide[i];
    if (g.transposed && i < 2 && g.cols > tn) continue;
    const int64_t nt = (g.cols + tn - 1) / tn;
    const int64_t tiles = mt * nt;
    const int64_t max_split = p.units < 4 ? 1 : (p.units / 4 < 64 ? p.units / 4 : 64);
    for (int64_t want = 1; want <= max_split; ++want) {
      const int64_t per = (p.units + want - 1) / want;
      const int64_t split = (p.units + per - 1) / per;
      if (split != want) continue;
      const int64_t waves = (tiles * split + sms - 1) / sms;
      const double step = tn >= 96 ? 2.0 * tn : 192.0;
      double cost = static_cast<double>(waves) * (per * step + 200.0) + 2.0 * tn * 4.0;
      const bool partial = split > 1 || g.transposed;
      if (partial)  // written and read through L2 at some 5 KB a cycle, and a launch
        cost += 3000.0 + static_cast<double>(split) * g.rows * g.cols * 8.0 / 5000.0;
      if (cost < best) {
        best = cost;
        p.tn = tn;
        p.split = static_cast<int>(split);
      }
      if (tiles * split >= 4 * static_cast<int64_t>(sms)) break;
    }
  }
  if (p.split > 1 || g.transposed) {
    const int64_t out_rows = g.transposed ? g.cols : g.rows;
    const int64_t out_cols = g.transposed ? g.rows : g.cols;
    p.ldpart = (out_cols + 7) / 8 * 8;
    p.part_bytes = static_cast<size_t>(p.split) * out_rows * p.ldpart * 4;
  }
  return p;
}

cudaError_t launch_gemm(const GemmShape& g, const GemmPlan& p, const GemmOperand& A,
                        const GemmOperand& B, dprc_dtype dt, const LinearEpi& epi, void* part,
                        cudaStream_t s) {
  if (B.mn_major && p.tn < 64) return cudaErrorInvalidValue;  // its boxes are 64 wide
  CUtensorMap ma, mb;
  if (!operand_map(&ma, A, g.rows, g.K, g.planes, kTm)) return cudaErrorInvalidValue;
  if (!operand_map(&mb, B, g.cols, g.K, g.planes, p.tn)) return cudaErrorInvalidValue;
  GemmArgs a;
  a.rows = g.rows;
  a.cols = static_cast<int>(g.cols);
  a.mt = static_cast<int>((g.rows + kTm - 1) / kTm);
  a.nt = static_cast<int>((g.cols + p.tn - 1) / p.tn);
  a.split = p.split;
  a.units = static_cast<int>(p.units);
  a.per_split = static_cast<int>((p.units + p.split - 1) / p.split);
  a.npairs = g.planes > 1 ? 6 : 1;
  a.a_mn = A.mn_major;
  a.b_mn = B.mn_major;
  a.transposed = g.transposed;
  a.part = p.part_bytes > 0 ? static_cast<float*>(part) : nullptr;
  a.ldpart = p.ldpart;
  a.part_stride = (g.transposed ? g.cols : g.rows) * p.ldpart;
  a.epi = epi;
  return dt == DPRC_F32 ? launch_gemm_tn<float>(p.tn, ma, mb, a, s)
                        : launch_gemm_tn<__nv_bfloat16>(p.tn, ma, mb, a, s);
}

}  // namespace dprc
