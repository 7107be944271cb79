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
// tokens cost what they are; D is then stored transposed, by partial sums in
// memory or in the shared memory of a cluster (GemmPlan::join).
//
// Tiles are walked in groups of row tiles, all columns of a group before the
// next: as many rows as make a group about one wave where there are few
// columns (then each row of A comes from memory once), eight otherwise, so the
// tiles in flight at one time share their operands in L2.

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "launch.cuh"
#include "linear.cuh"

namespace dprc {
namespace {

constexpr int kTm = 128;
constexpr int kTk = 64;
constexpr int kRing = 216 * 1024;

// Accumulators of a set, and sets (the pair's fp32 set takes all of TMEM).
template <typename T>
constexpr int kAccs = sizeof(T) == 4 ? 2 : 1;
template <typename T>
constexpr int kPairSets = sizeof(T) == 4 ? 1 : 2;

// Planes of an operand.  A stage holds all planes of its 64 of the contraction,
// so that the six plane products read what was copied once.
template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;

template <int kTn, typename T>
struct GemmCfg {
  static constexpr int kA = kTm * kTk * 2;   // of a plane
  static constexpr int kB = kTn * kTk * 2;
  static constexpr int kStage = kPlanes<T> * (kA + kB);
  static constexpr int kFit = kRing / kStage;
  static constexpr int kStages = kFit < 2 ? 2 : kFit < 10 ? kFit : 10;
  static constexpr int kEpiWarps = kTn >= 64 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kCols = kTn / (kEpiWarps / 4);  // columns per epilogue warp
  // the sums a CTA gives its cluster (GemmPlan::join), [kTn][kTm] behind the barriers
  static constexpr bool kJoin = sizeof(T) == 2 && kTn <= 32;
  static constexpr int kSmem = kStages * kStage + 1024 + 512 + (kJoin ? kTn * kTm * 4 : 0);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// One thread's bounded wait for a phase of a barrier of this CTA: like
// mbar_wait_lim, but each try may suspend the thread for up to kSuspendNs, and a
// warp waits with one lane (wait_warp).  Warps that poll take issue slots and
// shared memory from the thread that feeds the tensor core: eight epilogue warps
// polling with all lanes made it 703,000 cycles and not 478,000 for
// 16384 x 2048 x 8192, one lane each without the hint 363 us and not 324.  (One
// polling warp and a hardware barrier for the others: 336 us.)
constexpr uint32_t kSuspendNs = 20000;

__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, int code,
                                          const volatile int* abort) {
  if (try_wait_long(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    if (try_wait_long(bar, parity)) return true;
    if (abort != nullptr && *abort != 0) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(code);
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int code,
                                          const volatile int* abort) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_long(bar, parity, code, abort) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

struct GemmArgs {
  long long rows;
  int cols;
  int mt, nt, group;        // tiles, and row tiles per group
  int split;
  int units, per_split;     // contraction units of 64, and of one share
  int a_mn, b_mn;
  int transposed;
  int join;                 // the shares of a tile are a cluster, which adds them up
  float* part;              // partial sums, or null: the epilogue
  long long ldpart, part_stride;
  int beside;               // runs beside the kernel before (launch.cuh)
  LinearEpi epi;
};

// Plane products of fp32 operands, by size: 1, 2^-8 (2), 2^-16 (3).
template <typename T>
constexpr int kProducts = sizeof(T) == 4 ? 6 : 1;

__device__ __forceinline__ constexpr int plane_a(int i) {
  return i == 0 || i == 1 || i == 3 ? 0 : i == 5 ? 2 : 1;
}
__device__ __forceinline__ constexpr int plane_b(int i) {
  return i == 0 || i == 2 || i == 5 ? 0 : i == 3 ? 2 : 1;
}

struct GemmUnit {
  int m, n, split, u0, u1;
};

// The stages of a ring in turn, with the parity of the current round.  (Stage
// and parity from a running 64-bit count, as quotient and remainder, cost the
// copying and the issuing thread a tenth of the kernel's time: they are the
// serial path that every stage passes.)
template <int kStages>
struct RingPos {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++s == kStages) {
      s = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ GemmUnit gemm_unit(const GemmArgs& a, int w) {
  GemmUnit g;
  const int tile = a.split == 1 ? w : w / a.split;
  g.split = w - tile * a.split;
  const int per_group = a.group * a.nt;
  const int grp = tile / per_group;
  const int rem = tile - grp * per_group;
  const int gr = min(a.group, a.mt - grp * a.group);
  g.n = rem / gr;
  g.m = grp * a.group + rem - g.n * gr;
  g.u0 = g.split * a.per_split;
  g.u1 = min(g.u0 + a.per_split, a.units);
  return g;
}

// kN finished sums of one row, the first of them column col of D: through the
// epilogue, or to the partial sums.  kOdd: bf16 rows of D that may be no whole
// 16-byte accesses (a lane's eight fp32 values are a whole 32-byte sector without
// turning: 4097 x 1001 x 1001 with GELU, dropout and Z 114 us, turned 129).
template <typename T, int kN, bool kOdd>
__device__ __forceinline__ void gemm_emit(const GemmArgs& a, int split, long long row, int col,
                                          float* v, const RoundKeys& rk) {
  if (col >= a.cols) return;  // the same for a warp
  if constexpr (kOdd) {
    if (a.part == nullptr && a.epi.vec == 0) {
      linear_out_odd<T, kN>(a.epi, row, col, v, rk);
      return;
    }
  }
  if (row >= a.rows) return;
  if (a.transposed) {
    float* out = a.part + split * a.part_stride + row;
#pragma unroll
    for (int t = 0; t < kN; ++t)
      if (col + t < a.cols) out[(col + t) * a.ldpart] = v[t];
  } else if (a.part != nullptr) {
    float* out = a.part + split * a.part_stride + row * a.ldpart + col;
#pragma unroll
    for (int t = 0; t < kN; t += 4)
      if (col + t < a.cols && DPRC_IN(col + t + 4 <= a.ldpart))
        *reinterpret_cast<float4*>(out + t) = make_float4(v[t], v[t + 1], v[t + 2], v[t + 3]);
  } else {
    linear_out<T, kN / 8>(a.epi, row, col, v, rk);
  }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Accumulators.  bf16: one per tile, two sets in turn, so that a tile's
// epilogue runs under the next tile's MMAs.  fp32: the tensor core's additions
// truncate, which showed over a contraction's six plane products per step
// (2.2e-6 of the result at K = 1001, where a plain fp32 product has 5.4e-7).
// So the first plane product, which makes the result's size, has an
// accumulator of its own, the five others, 2^-8 of it and less, a second one,
// and every kAccUnits units (512 of the contraction) the epilogue warps add
// both to sums in registers: 1.7e-7 (1001 x 517 x 263; the plain product 4.1e-7).
template <typename T>
constexpr int kAccUnits = sizeof(T) == 4 ? 8 : 1 << 30;

// Set `count` of kSets accumulator sets.
template <int kSets>
struct AccPos {
  int set = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++set == kSets) {
      set = 0;
      parity ^= 1u;
    }
  }
};

// gemm_collect for bf16 outputs whose rows are whole 32 bytes: the bias (two
// columns a lane) and the residual's first kAhead steps are on their way before
// the accumulator is finished, later ones kAhead steps ahead.  A load of the
// epilogue queues behind the operand tiles that are in flight into the SM, some
// 2 us: 16384 x 2048 x 8192 with bias and residual took 571,000 cycles with the
// loads where they are needed, 499,000 so (475,000 without either); with dropout
// too 406 and 369 us, 16384 x 1024 x 1024 63 and 53 us (three steps ahead: 387
// and 62, for want of registers).
template <int kCols, int kAcc, int kSets, typename Release>
__device__ __forceinline__ bool gemm_collect_ahead(const GemmArgs& a, uint32_t tmem, long long row,
                                                   int col0, const RoundKeys& rk, uint64_t* accf,
                                                   AccPos<kSets>& pos,
                                                   const volatile int* abort_flag, bool ok,
                                                   Release release) {
  using T = __nv_bfloat16;
  constexpr int kStep = 16, kAhead = 2;
  static_assert(kCols == 64, "a lane holds the bias of two columns");
  const LinearEpi& e = a.epi;
  const int lane = threadIdx.x & 31;
  const bool mine = row < a.rows;
  const T* res = static_cast<const T*>(e.res) + (mine ? row : 0) * e.N + col0;
  uint32_t ahead[kAhead][8];
  const auto fetch = [&](uint32_t* u, int c) {
    if (mine && c < kCols && col0 + c < a.cols) ld16_raw(res + c, u);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) fetch(ahead[s], s * kStep);
  uint32_t bias = 0;
  if (e.bias != nullptr && col0 + 2 * lane < a.cols)
    bias = ld_l2(reinterpret_cast<const uint32_t*>(static_cast<const T*>(e.bias) + col0) + lane);
  ok = ok && wait_warp(&accf[pos.set], pos.parity, DPRC_DEVERR_ACCUM, abort_flag);
  tc_fence_after();
  if (ok) {
#pragma unroll 1
    for (int c0 = 0; c0 < kCols; c0 += kStep) {
      if (col0 + c0 >= a.cols) break;  // uniform over the warp
      float v[kStep];
      tmem_ld_cols<kStep>(tmem + pos.set * kAcc + c0, v);
      if (e.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < kStep / 2; ++j) {
          const uint32_t b = __shfl_sync(0xffffffffu, bias, c0 / 2 + j);
          v[2 * j] += __uint_as_float(b << 16);
          v[2 * j + 1] += __uint_as_float(b & 0xFFFF0000u);
        }
      }
      if (mine) linear_out<T, kStep / 8, true>(e, row, col0 + c0, v, rk, ahead[0]);
#pragma unroll
      for (int s = 0; s + 1 < kAhead; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) ahead[s][j] = ahead[s + 1][j];
      fetch(ahead[kAhead - 1], c0 + kAhead * kStep);
    }
  }
  release(pos.set);
  pos.next();
  return ok;
}

// The sums of one unit of work for this thread's row (TMEM lane), kCols of
// them from column tmem of each accumulator on (kAcc columns apart), first
// column col0 of D.  `release(set)` frees a set.
// emit(N, c, v): takes the N sums v from column c of them on.
template <typename T, int kCols, int kAcc, int kSets, typename Release, typename Emit>
__device__ __forceinline__ bool gemm_collect(const GemmArgs& a, const GemmUnit& g, uint32_t tmem,
                                             int col0, uint64_t* accf, AccPos<kSets>& pos,
                                             const volatile int* abort_flag, bool ok,
                                             Release release, Emit emit) {
  if constexpr (sizeof(T) == 2) {
    constexpr int kStep = kCols < 16 ? kCols : 16;
    ok = ok && wait_warp(&accf[pos.set], pos.parity, DPRC_DEVERR_ACCUM, abort_flag);
    tc_fence_after();
    if (ok) {
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += kStep) {
        if (col0 + c0 >= a.cols) break;  // uniform over the warp
        float v[kStep];
        tmem_ld_cols<kStep>(tmem + pos.set * kAcc + c0, v);
        emit(std::integral_constant<int, kStep>{}, c0, v);
      }
    }
    release(pos.set);
    pos.next();
  } else {
    constexpr int kStep = 16;
    float acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
    for (int u = g.u0; u < g.u1; u += kAccUnits<T>) {
      ok = ok && wait_warp(&accf[pos.set], pos.parity, DPRC_DEVERR_ACCUM, abort_flag);
      tc_fence_after();
      if (ok) {
        const uint32_t t0 = tmem + pos.set * 2 * kAcc;
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += kStep) {
          float v[kStep], w[kStep];
          tmem_ld_cols<kStep>(t0 + c0, v);
          tmem_ld_cols<kStep>(t0 + kAcc + c0, w);
#pragma unroll
          for (int t = 0; t < kStep; ++t) acc[c0 + t] += v[t] + w[t];
        }
      }
      release(pos.set);
      pos.next();
    }
    if (ok) {
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 8) emit(std::integral_constant<int, 8>{}, c0, acc + c0);
    }
  }
  return ok;
}

// Matrix descriptors of an operand's K = 16 steps.  K-major, 128-byte swizzle:
// 8-row atoms 1 KB apart (SBO), a step is 32 B along the row.  MN-major: a step
// is 16 rows of 128 B, 64-wide atoms along M or N one 8 KB box apart (LBO).
// The address field (bits 0..13, in 16 bytes) has room for all of shared
// memory, so stages and steps are added to it.
struct StepDesc {
  uint64_t base;
  uint32_t step;
  __device__ __forceinline__ StepDesc(uint32_t addr, bool mn)
      : base(make_sdesc(addr, mn ? kTk * 128 : 16, 1024, kSwz128)), step(mn ? 2048 / 16 : 32 / 16) {}
  __device__ __forceinline__ uint64_t at(uint32_t bytes) const { return base + (bytes >> 4); }
};

template <int kTn, typename T>
__global__ void __launch_bounds__(GemmCfg<kTn, T>::kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const GemmArgs a) {
  using Cfg = GemmCfg<kTn, T>;
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
  float* sums = reinterpret_cast<float*>(ring + kStages * Cfg::kStage + 512);  // kJoin

  if (Cfg::kJoin && a.join && cluster_nctarank() != static_cast<uint32_t>(a.split)) {
    if (threadIdx.x == 0) record_error(DPRC_DEVERR_LAUNCH);  // no peers to read from
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nwork = a.mt * a.nt * a.split;  // the host checks that it fits
  const int first = static_cast<int>(blockIdx.x), stride = static_cast<int>(gridDim.x);
  const int mine = nwork > first ? (nwork - 1 - first) / stride + 1 : 0;

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
    tmem_alloc(tmem_slot, 2 * kAccs<T> * kTn);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // all of the above overlaps the end of the kernel before
  beside_begin(a.beside != 0);

  if (warp == 0) {
    if (lane == 0 && mine > 0) {
      RingPos<kStages> pos;
      long long issued = 0;
      bool ok = true;
      const bool a_mn = a.a_mn != 0, b_mn = a.b_mn != 0;
      for (int j = 0; j < mine && ok; ++j) {
        const GemmUnit g = gemm_unit(a, first + j * stride);
        const int row = g.m * kTm, col = g.n * kTn;
        for (int u = g.u0; u < g.u1; ++u, pos.next()) {
          const int s = pos.s;
          if (!wait_long(&empty[s], pos.parity ^ 1, DPRC_DEVERR_PIPE_EMPTY, abort_flag)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          const int k = u * kTk;
          uint8_t* sa = ring + s * Cfg::kStage;
          uint8_t* sb = sa + kPlanes<T> * Cfg::kA;
          mbar_arrive_expect_tx(&full[s], Cfg::kStage);
#pragma unroll
          for (int p = 0; p < kPlanes<T>; ++p, sa += Cfg::kA, sb += Cfg::kB) {
            if (a_mn) {
#pragma unroll
              for (int h = 0; h < kTm / 64; ++h)
                tma_load_3d(sa + h * (kTk * 128), &map_a, &full[s], row + h * 64, k, p);
            } else {
              tma_load_3d(sa, &map_a, &full[s], k, row, p);
            }
            if (b_mn) {
#pragma unroll
              for (int h = 0; h < (kTn + 63) / 64; ++h)
                tma_load_3d(sb + h * (kTk * 128), &map_b, &full[s], col + h * 64, k, p);
            } else {
              tma_load_3d(sb, &map_b, &full[s], k, col, p);
            }
          }
          ++issued;
        }
      }
      // let the copies this thread issued land before the CTA can exit
      for (long long k = issued - 1; k >= 0 && k >= issued - kStages; --k)
        mbar_wait(&full[k % kStages], (k / kStages) & 1, DPRC_DEVERR_PIPE_FULL);
    }
  } else if (warp == 1) {
    if (lane == 0 && mine > 0) {
      const uint32_t idesc = make_idesc_bf16(kTm, kTn, a.a_mn != 0, a.b_mn != 0);
      const StepDesc da(smem_u32(ring), a.a_mn != 0), db(smem_u32(ring) + kPlanes<T> * Cfg::kA, a.b_mn != 0);
      RingPos<kStages> pos;
      AccPos<2> set;
      bool ok = true, issued = false;
      for (int j = 0; j < mine && ok; ++j) {
        const GemmUnit g = gemm_unit(a, first + j * stride);
        for (int c0 = g.u0, c1; c0 < g.u1 && ok; c0 = c1, set.next()) {
          c1 = g.u1 - c0 < kAccUnits<T> ? g.u1 : c0 + kAccUnits<T>;
          if (!wait_long(&acce[set.set], set.parity ^ 1, DPRC_DEVERR_ACCUM, abort_flag)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t acc = tmem + set.set * kAccs<T> * kTn;
          for (int u = c0; u < c1; ++u, pos.next()) {
            const int s = pos.s;
            if (!wait_long(&full[s], pos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag)) {
              *abort_flag = 1;
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = da.at(s * Cfg::kStage), bd = db.at(s * Cfg::kStage);
#pragma unroll
            for (int i = 0; i < kProducts<T>; ++i) {
              // the first product in one accumulator, the small ones in the other
              const uint32_t d = acc + (i == 0 ? 0 : kTn);
              const uint64_t ai = ad + plane_a(i) * (Cfg::kA >> 4), bi = bd + plane_b(i) * (Cfg::kB >> 4);
#pragma unroll
              for (int kk = 0; kk < kTk / 16; ++kk)
                umma_bf16(d, ai + kk * da.step, bi + kk * db.step, idesc,
                   (u == c0 && i <= 1 && kk == 0) ? 0u : 1u);
            }
            umma_commit(&empty[s]);
            issued = true;
          }
          if (ok) umma_commit(&accf[set.set]);
        }
      }
      if (issued) umma_drain(drain, kWaitLimitNs);
    }
  } else {
    const int ew = warp - 2;
    const int q = warp & 3;  // TMEM lane quadrant this warp may read
    const int c_lo = (ew >> 2) * Cfg::kCols;
    const RoundKeys rk = round_keys(a.epi.drop.seed);
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + c_lo;
    const auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[buf]);
    };
    AccPos<2> pos;
    bool ok = true;
    for (int j = 0; j < mine; ++j) {
      const GemmUnit g = gemm_unit(a, first + j * stride);
      const long long row = static_cast<long long>(g.m) * kTm + q * 32 + lane;
      const int col = g.n * kTn + c_lo;
      const auto emit = [&](auto n, int c, float* v) {
        constexpr int kN = decltype(n)::value;
        if constexpr (Cfg::kJoin) {
          if (a.join) {
#pragma unroll
            for (int t = 0; t < kN; ++t) sums[(c_lo + c + t) * kTm + q * 32 + lane] = v[t];
            return;
          }
        }
        gemm_emit<T, kN, kTn >= 64 && sizeof(T) == 2>(a, g.split, row, col + c, v, rk);
      };
      ok = gemm_collect<T, Cfg::kCols, kTn, 2>(a, g, tb, col, accf, pos, abort_flag, ok, release,
                                               emit);
    }
  }

  __syncwarp();  // reconverge each warp before the CTA barrier
  tc_fence_before();
  if constexpr (Cfg::kJoin) {
    if (a.join) {
      // each CTA of the cluster adds up its part of the tile's outputs, the
      // shares in order
      cluster_sync_all();
      const GemmUnit g = gemm_unit(a, first);
      const RoundKeys rk = round_keys(a.epi.drop.seed);
      const int total = a.cols * (kTm / 8), each = (total + a.split - 1) / a.split;
      const int end = min((g.split + 1) * each, total);
      for (int i = g.split * each + static_cast<int>(threadIdx.x); i < end; i += Cfg::kThreads) {
        const int t = i / (kTm / 8), f = i % (kTm / 8) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < a.split; ++s) {
          const uint32_t from = map_to_rank(sums + t * kTm + f, s);
          const float4 x = ld_cluster_f4(from), y = ld_cluster_f4(from + 16);
          v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
          v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
        }
        const long long n = static_cast<long long>(g.m) * kTm + f;
        if (n < a.rows) linear_out<T, 1>(a.epi, t, static_cast<int>(n), v, rk);
      }
      __syncwarp();
      cluster_sync_all();  // nobody leaves while its sums are read
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kAccs<T> * kTn);
  }
  beside_end(a.beside != 0);
}

// Allows a kernel its shared memory, once per device; kTag: one per kernel.
template <int kTag, typename F>
cudaError_t set_smem_once(F* kernel, int bytes) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> done[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDev && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDev) done[dev].store(1, std::memory_order_release);
  return e;
}

// ---------------------------------------------------------------------------
// CTA pairs: two SMs on one 256 x 256 tile (cta_group::2).  Each CTA of a pair
// holds 128 rows of A and 128 columns of B of a stage, and the accumulator of
// its 128 rows; the leader (rank 0) issues the MMAs, which read both CTAs'
// shared memory.  A stage is 32 KB per SM instead of 48 KB for the same MMA
// time, which is what the single-CTA tile was bound by: copies into shared
// memory.
//
// Barriers: full[s] lives in the leader and counts both CTAs' bytes; empty[s]
// and accf[b] are signalled in both CTAs by the leader's commits; acce[b] lives
// in the leader and counts both CTAs' epilogue warps.
// ---------------------------------------------------------------------------
constexpr int kPairTile = 256;
constexpr double kPairStep = 600.0;  // cycles of a 64-deep step
constexpr int kPairA = kTm * kTk * 2;
// bf16: seven stages of 32 KB; fp32: two of 96 KB, which feed 24 MMAs each.
template <typename T>
constexpr int kPairStageBytes = kPlanes<T> * 2 * kPairA;
template <typename T>
constexpr int kPairRing = sizeof(T) == 4 ? 2 : 7;
// Epilogue warps: fp32 keeps its sums in registers, 64 columns a warp.
template <typename T>
constexpr int kPairEpiWarps = 16;
template <typename T>
constexpr int kPairSmem = kPairRing<T> * kPairStageBytes<T> + 1024 + 512;

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once every MMA issued so
// far by this thread has completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// A tile copy whose bytes count on the barrier at `bar` (shared::cluster
// address, in either CTA of the pair).
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// One or two products in a launch.  The first one's units go round the pairs;
// those that got one unit more of them (the first `extra` pairs) take the
// first extra * a_units units of the second product, the other pairs the rest,
// a_units chosen on the host so that both finish together.
struct GemmBatch {
  GemmArgs p[2];
  int n0, n1;  // units
  int extra, a_units;
};

struct PairWork {
  int mine0, mine1;
  int first0, step0, first1, step1;
  __device__ __forceinline__ int at(int j) const {
    return j < mine0 ? first0 + j * step0 : first1 + (j - mine0) * step1;
  }
};

__device__ __forceinline__ PairWork pair_work(const GemmBatch& b, int me, int pairs) {
  PairWork w;
  w.first0 = me;
  w.step0 = pairs;
  w.mine0 = b.n0 > me ? (b.n0 - 1 - me) / pairs + 1 : 0;
  const int cut = min(b.extra * b.a_units, b.n1);
  const bool ahead = me < b.extra;
  w.first1 = ahead ? me : cut + me - b.extra;
  w.step1 = ahead ? b.extra : pairs - b.extra;
  const int end = ahead ? cut : b.n1;
  w.mine1 = end > w.first1 ? (end - 1 - w.first1) / w.step1 + 1 : 0;
  return w;
}

// Arrives on a barrier of either CTA of the pair.  Relaxed: what it announces
// is that this warp's TMEM loads have completed (tcgen05.wait::ld); a release at
// cluster scope would first wait for the tile's global stores (41 and not 36 us
// at 16384 x 1024 x 1024).
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// The pair's epilogues are instantiations of their own, since two in one kernel
// cost the plain one registers (16384 x 1024 x 1024: 33 -> 35 to 40 us): rows of
// whole 16-byte accesses and fp32, bf16 with a residual (loaded ahead), other bf16.
enum PairEpilogue { kWholeRows, kResidual, kOddRows };
template <typename T, PairEpilogue kEpilogue>
__global__ void __launch_bounds__(64 + 32 * kPairEpiWarps<T>, 1) __cluster_dims__(2, 1, 1)
    linear_gemm_pair_kernel(const __grid_constant__ CUtensorMap map_a0,
                            const __grid_constant__ CUtensorMap map_b0,
                            const __grid_constant__ CUtensorMap map_a1,
                            const __grid_constant__ CUtensorMap map_b1,
                            const __grid_constant__ GemmBatch batch) {
  constexpr int kEpi = kPairEpiWarps<T>;
  constexpr int kStages = kPairRing<T>, kStage = kPairStageBytes<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align_1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * kStage);
  uint64_t* empty = full + kStages;
  uint64_t* accf = empty + kStages;  // [2]
  uint64_t* acce = accf + 2;             // [2]
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (cluster_nctarank() != 2) {  // a launch of another shape has no peer to address
    if (threadIdx.x == 0) record_error(DPRC_DEVERR_LAUNCH);
    return;
  }
  const int pairs = static_cast<int>(gridDim.x) / 2, me = static_cast<int>(blockIdx.x) / 2;
  const PairWork work = pair_work(batch, me, pairs);
  const int mine = work.mine0 + work.mine1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 2 * kEpi);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_a0);
    tma_prefetch_desc(&map_b0);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // all of the above overlaps the end of the kernel before
  beside_begin(batch.p[0].beside != 0);

  if (warp == 0) {
    if (lane == 0 && mine > 0) {
      RingPos<kStages> pos;
      long long issued = 0;
      bool ok = true;
      const uint32_t full0 = map_to_rank(full, 0);
      for (int j = 0; j < mine && ok; ++j) {
        const GemmArgs& a = batch.p[j >= work.mine0];
        const CUtensorMap* map_a = j >= work.mine0 ? &map_a1 : &map_a0;
        const CUtensorMap* map_b = j >= work.mine0 ? &map_b1 : &map_b0;
        const GemmUnit g = gemm_unit(a, work.at(j));
        const int row = g.m * kPairTile + rank * kTm, col = g.n * kPairTile + rank * kTm;
        const bool a_mn = a.a_mn != 0, b_mn = a.b_mn != 0;
        for (int u = g.u0; u < g.u1; ++u, pos.next()) {
          const int s = pos.s;
          if (!wait_long(&empty[s], pos.parity ^ 1, DPRC_DEVERR_PIPE_EMPTY, abort_flag)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          const int k = u * kTk;
          uint8_t* sa = ring + s * kStage;
          uint8_t* sb = sa + kPlanes<T> * kPairA;
          const uint32_t bar = full0 + s * 8;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStage);
#pragma unroll
          for (int p = 0; p < kPlanes<T>; ++p, sa += kPairA, sb += kPairA) {
            if (a_mn) {
              tma_load_3d_pair(sa, map_a, bar, row, k, p);
              tma_load_3d_pair(sa + kTk * 128, map_a, bar, row + 64, k, p);
            } else {
              tma_load_3d_pair(sa, map_a, bar, k, row, p);
            }
            if (b_mn) {
              tma_load_3d_pair(sb, map_b, bar, col, k, p);
              tma_load_3d_pair(sb + kTk * 128, map_b, bar, col + 64, k, p);
            } else {
              tma_load_3d_pair(sb, map_b, bar, k, col, p);
            }
          }
          ++issued;
        }
      }
      // let both CTAs' copies land before either can exit (the closing
      // cluster barrier holds the other one)
      if (rank == 0)
        for (long long k = issued - 1; k >= 0 && k >= issued - kStages; --k)
          mbar_wait(&full[k % kStages], (k / kStages) & 1, DPRC_DEVERR_PIPE_FULL);
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0 && mine > 0) {
      RingPos<kStages> pos;
      AccPos<kPairSets<T>> set;
      bool ok = true, issued = false;
      for (int j = 0; j < mine && ok; ++j) {
        const GemmArgs& a = batch.p[j >= work.mine0];
        const uint32_t idesc = make_idesc_bf16(kPairTile, kPairTile, a.a_mn != 0, a.b_mn != 0);
        const StepDesc da(smem_u32(ring), a.a_mn != 0);
        const StepDesc db(smem_u32(ring) + kPlanes<T> * kPairA, a.b_mn != 0);
        const GemmUnit g = gemm_unit(a, work.at(j));
        for (int c0 = g.u0, c1; c0 < g.u1 && ok; c0 = c1, set.next()) {
          c1 = g.u1 - c0 < kAccUnits<T> ? g.u1 : c0 + kAccUnits<T>;
          if (!wait_long(&acce[set.set], set.parity ^ 1, DPRC_DEVERR_ACCUM, abort_flag)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t acc = tmem + set.set * kAccs<T> * kPairTile;
          for (int u = c0; u < c1; ++u, pos.next()) {
            const int s = pos.s;
            if (!wait_long(&full[s], pos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag)) {
              *abort_flag = 1;
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = da.at(s * kStage), bd = db.at(s * kStage);
#pragma unroll
            for (int i = 0; i < kProducts<T>; ++i) {
              // the first product in one accumulator, the small ones in the other
              const uint32_t d = acc + (i == 0 ? 0 : kPairTile);
              const uint64_t ai = ad + plane_a(i) * (kPairA >> 4), bi = bd + plane_b(i) * (kPairA >> 4);
#pragma unroll
              for (int kk = 0; kk < kTk / 16; ++kk)
                umma_bf16_pair(d, ai + kk * da.step, bi + kk * db.step, idesc,
                   (u == c0 && i <= 1 && kk == 0) ? 0u : 1u);
            }
            umma_commit_pair(&empty[s]);
            issued = true;
          }
          if (ok) umma_commit_pair(&accf[set.set]);
        }
      }
      if (issued) {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_u32(drain))
            : "memory");
        mbar_wait_lim(drain, 0, DPRC_DEVERR_ACCUM, kWaitLimitNs, nullptr);
      }
    }
  } else {
    const int ew = warp - 2;
    const int q = warp & 3;  // TMEM lane quadrant this warp may read
    constexpr int kCols = kPairTile / (kEpi / 4);
    const int c_lo = (ew >> 2) * kCols;
    const RoundKeys rk = round_keys(batch.p[0].epi.drop.seed);  // a pair of problems drops nothing
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + c_lo;
    const uint32_t acce0 = map_to_rank(acce, 0);
    const auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(acce0 + buf * 8);
    };
    AccPos<kPairSets<T>> pos;
    bool ok = true;
    for (int j = 0; j < mine; ++j) {
      const GemmArgs& a = batch.p[j >= work.mine0];
      const GemmUnit g = gemm_unit(a, work.at(j));
      const long long row = static_cast<long long>(g.m) * kPairTile + rank * kTm + q * 32 + lane;
      const int col = g.n * kPairTile + c_lo;
      if constexpr (kEpilogue == kResidual)
        ok = gemm_collect_ahead<kCols, kPairTile>(a, tb, row, col, rk, accf, pos, abort_flag, ok,
                                                  release);
      else
        ok = gemm_collect<T, kCols, kPairTile, kPairSets<T>>(
            a, g, tb, col, accf, pos, abort_flag, ok, release, [&](auto n, int c, float* v) {
              gemm_emit<T, decltype(n)::value, kEpilogue == kOddRows>(a, g.split, row, col + c, v, rk);
            });
    }
  }

  __syncwarp();  // reconverge each warp before the cluster barrier
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  beside_end(batch.p[0].beside != 0);
}

template <typename T, PairEpilogue kEpilogue>
cudaError_t launch_gemm_pair_t(const CUtensorMap* maps, const GemmBatch& batch, cudaStream_t s) {
  auto* kernel = linear_gemm_pair_kernel<T, kEpilogue>;
  const cudaError_t e = set_smem_once<sizeof(T) * 4 + kEpilogue>(kernel, kPairSmem<T>);
  if (e != cudaSuccess) return e;
  const long long pairs =
      std::min<long long>(static_cast<long long>(batch.n0) + batch.n1, device_sm_count() / 2);
  return launch_after(kernel, dim3(static_cast<unsigned>(2 * pairs)), 64 + 32 * kPairEpiWarps<T>, 1,
                      s, kPairSmem<T>, maps[0], maps[1], maps[2], maps[3], batch);
}

template <typename T>
cudaError_t launch_gemm_pair(const CUtensorMap* maps, const GemmBatch& batch, cudaStream_t s) {
  const GemmArgs& a = batch.p[0];  // two products have rows of one length
  if constexpr (sizeof(T) == 2) {
    if (a.part == nullptr && a.epi.vec == 0)
      return launch_gemm_pair_t<T, kOddRows>(maps, batch, s);
    if (batch.n1 == 0 && a.part == nullptr && a.epi.vec == 2 && a.epi.res != nullptr)
      return launch_gemm_pair_t<T, kResidual>(maps, batch, s);
  }
  return launch_gemm_pair_t<T, kWholeRows>(maps, batch, s);
}

// How the second product's units are dealt (GemmBatch), and the busiest pair's
// load: units of u0 and u1 steps.
long long deal_units(long long n0, int u0, long long n1, int u1, long long pairs, int& extra,
                     int& a_units) {
  extra = static_cast<int>(n0 % pairs);
  const long long base = n0 / pairs;
  a_units = 0;
  long long best = -1;
  for (int a = 0; a <= (extra > 0 ? 4096 : 0); ++a) {
    const long long rest = std::max<long long>(n1 - static_cast<long long>(extra) * a, 0);
    const long long b = (rest + pairs - extra - 1) / (pairs - extra);
    const long long load = std::max((base + 1) * u0 * (extra > 0) + static_cast<long long>(a) * u1,
                                    base * u0 + b * u1);
    if (best < 0 || load < best) {
      best = load;
      a_units = a;
    }
    if (rest == 0) break;
  }
  return best;
}

template <int kTn, typename T>
cudaError_t launch_gemm_t(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& a,
                          cudaStream_t s) {
  using Cfg = GemmCfg<kTn, T>;
  cudaError_t e = set_smem_once<kTn * 8 + sizeof(T)>(linear_gemm_kernel<kTn, T>, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  const long long work = static_cast<long long>(a.mt) * a.nt * a.split;
  const long long grid = work < device_sm_count() ? work : device_sm_count();
  return launch_after(linear_gemm_kernel<kTn, T>, dim3(static_cast<unsigned>(grid)), Cfg::kThreads,
                      a.join ? a.split : 1, s, Cfg::kSmem, ma, mb, a);
}

template <typename T>
cudaError_t launch_gemm_tn(int tn, const CUtensorMap& ma, const CUtensorMap& mb,
                           const GemmArgs& a, cudaStream_t s) {
  switch (tn) {
    case 16: return launch_gemm_t<16, T>(ma, mb, a, s);
    case 32: return launch_gemm_t<32, T>(ma, mb, a, s);
    case 64: return launch_gemm_t<64, T>(ma, mb, a, s);
    case 128: return launch_gemm_t<128, T>(ma, mb, a, s);
    default:
      if constexpr (sizeof(T) == 2) return launch_gemm_t<256, T>(ma, mb, a, s);
      return cudaErrorInvalidValue;
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
  p.units = (g.K + kTk - 1) / kTk;
  if (p.units == 0) return p;  // nothing to cut (prepare_gemm refuses it)
  const int sms = device_sm_count();
  // Candidates: the tile shapes and contraction shares; the cost of one is its
  // waves of units (in cycles of a 64-deep step, measured: the pair's step runs
  // at the tensor core's rate, the single CTA's steps at that of the copies
  // into shared memory), plus what a unit costs outside its MMAs, plus the
  // partial sums' way out and in.
  struct Shape {
    int tm, tn, ctas;
    double step;
  };
  const Shape wide[] = {{256, 256, 2, kPairStep}, {128, 256, 1, 632.0}, {128, 128, 1, 450.0},
                        {128, 64, 1, 260.0}};
  const Shape few[] = {{128, 16, 1, 200.0}, {128, 32, 1, 210.0}, {128, 64, 1, 260.0}};
  const Shape* shapes = g.transposed ? few : wide;
  const int nshapes = g.transposed ? 3 : 4;
  const double products = g.planes > 1 ? 6.0 : 1.0;
  const int64_t least = g.planes > 1 ? 1 : 4;  // units of a share
  double best = 1e300;
  for (int i = 0; i < nshapes; ++i) {
    const Shape& sh = shapes[i];
    if (g.transposed && i < 2 && g.cols > sh.tn) continue;
    if (g.planes > 1 && sh.tn == 256 && sh.ctas == 1) continue;  // 128 sums a thread
    const int64_t tiles = (g.rows + sh.tm - 1) / sh.tm * ((g.cols + sh.tn - 1) / sh.tn);
    const int64_t slots = sms / sh.ctas;
    const int64_t max_split = std::max<int64_t>(1, std::min<int64_t>(p.units / least, 64));
    for (int64_t want : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64}) {
      if (want > max_split) break;
      const int64_t per = (p.units + want - 1) / want;
      const int64_t split = (p.units + per - 1) / per;
      if (split != want) continue;
      const int64_t waves = (tiles * split + slots - 1) / slots;
      double cost = static_cast<double>(waves) * (per * sh.step * products + 200.0) + 8.0 * sh.tn;
      // Few tokens: a tile's shares as a cluster that adds them up through shared
      // memory, where all tiles run at once.  How many clusters that is depends on
      // the GPCs: 32 clusters of 4 do (4096 x 4096, 8 tokens: 10.2 us, by partial
      // sums 10.7), 16 of 8 do not (8192 x 2048: 18.2, by partial sums 11.2).
      const int64_t at_once = split <= 2 ? sms : split == 4 ? sms * 7 / 8 : split == 8 ? sms / 2 : 0;
      const bool join =
          g.transposed && g.planes == 1 && sh.tn <= 32 && tiles * split <= at_once;
      const bool partial = !join && (split > 1 || g.transposed);
      if (join) cost += 1500.0;
      if (partial)  // written and read through L2 at some 5 KB a cycle, and a launch
        cost += 3000.0 + static_cast<double>(split) * g.rows * g.cols * 8.0 / 5000.0;
      if (cost < best) {
        best = cost;
        p.cost = cost;
        p.tn = sh.tn;
        p.join = join;
        p.pair = sh.ctas == 2;
        p.split = static_cast<int>(split);
        p.per = per;
      }
      if (tiles * split >= 4 * static_cast<int64_t>(sms)) break;
    }
  }
  if (!p.join && (p.split > 1 || g.transposed)) {
    const int64_t out_rows = g.transposed ? g.cols : g.rows;
    const int64_t out_cols = g.transposed ? g.rows : g.cols;
    p.ldpart = (out_cols + 7) / 8 * 8;
    p.part_bytes = static_cast<size_t>(p.split) * out_rows * p.ldpart * 4;
  }
  return p;
}

namespace {
long long unit_count(const GemmArgs& a) {
  return static_cast<long long>(a.mt) * a.nt * a.split;
}

cudaError_t prepare_gemm(const GemmShape& g, const GemmPlan& p, const GemmOperand& A,
                         const GemmOperand& B, const LinearEpi& epi, void* part, CUtensorMap* maps,
                         GemmArgs& a) {
  if (B.mn_major && p.tn < 64) return cudaErrorInvalidValue;  // its boxes are 64 wide
  if (p.per < 1) return cudaErrorInvalidValue;                // no work: the waits would run out
  const int tile_m = p.pair ? kPairTile : kTm, tile_n = p.pair ? kPairTile : p.tn;
  if (!operand_map(&maps[0], A, g.rows, g.K, g.planes, kTm)) return cudaErrorInvalidValue;
  if (!operand_map(&maps[1], B, g.cols, g.K, g.planes, p.pair ? kTm : p.tn))
    return cudaErrorInvalidValue;
  a.rows = g.rows;
  a.cols = static_cast<int>(g.cols);
  a.mt = static_cast<int>((g.rows + tile_m - 1) / tile_m);
  a.nt = static_cast<int>((g.cols + tile_n - 1) / tile_n);
  const int wave = device_sm_count() / (p.pair ? 2 : 1);
  a.group = std::max(8, (wave + a.nt - 1) / a.nt);
  a.split = p.split;
  a.units = static_cast<int>(p.units);
  a.per_split = static_cast<int>(p.per);
  a.a_mn = A.mn_major;
  a.b_mn = B.mn_major;
  a.transposed = g.transposed;
  a.join = p.join;
  a.part = p.part_bytes > 0 ? static_cast<float*>(part) : nullptr;
  a.ldpart = p.ldpart;
  a.part_stride = (g.transposed ? g.cols : g.rows) * p.ldpart;
  a.beside = 0;
  a.epi = epi;
  return unit_count(a) < (int64_t(1) << 30) ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gemm(const GemmShape& g, const GemmPlan& p, const GemmOperand& A,
                        const GemmOperand& B, dprc_dtype dt, const LinearEpi& epi, void* part,
                        bool beside, cudaStream_t s) {
  CUtensorMap maps[4];
  if (p.pair) {
    GemmBatch batch;
    const cudaError_t e = prepare_gemm(g, p, A, B, epi, part, maps, batch.p[0]);
    if (e != cudaSuccess) return e;
    batch.p[0].beside = beside;
    batch.p[1] = batch.p[0];
    maps[2] = maps[0];
    maps[3] = maps[1];
    batch.n0 = static_cast<int>(unit_count(batch.p[0]));
    batch.n1 = batch.extra = batch.a_units = 0;
    return dt == DPRC_F32 ? launch_gemm_pair<float>(maps, batch, s)
                          : launch_gemm_pair<__nv_bfloat16>(maps, batch, s);
  }
  GemmArgs a;
  const cudaError_t e = prepare_gemm(g, p, A, B, epi, part, maps, a);
  if (e != cudaSuccess) return e;
  a.beside = beside;
  return dt == DPRC_F32 ? launch_gemm_tn<float>(p.tn, maps[0], maps[1], a, s)
                        : launch_gemm_tn<__nv_bfloat16>(p.tn, maps[0], maps[1], a, s);
}

// The cheaper of two products one after the other and both in one launch.
bool gemm_together(const GemmShape& g0, const GemmPlan& p0, const GemmShape& g1,
                   const GemmPlan& p1) {
  if (g0.transposed || g1.transposed) return false;
  const auto tiles = [](const GemmShape& g) {
    return (g.rows + kPairTile - 1) / kPairTile * ((g.cols + kPairTile - 1) / kPairTile);
  };
  if (tiles(g0) + tiles(g1) < device_sm_count() / 2) return false;  // shares fill the GPU better
  int extra, a_units;
  const long long load =
      deal_units(tiles(g0), static_cast<int>(p0.units), tiles(g1), static_cast<int>(p1.units),
                 device_sm_count() / 2, extra, a_units);
  return load * kPairStep * (g0.planes > 1 ? 6.0 : 1.0) + 2048.0 < p0.cost + p1.cost;
}

cudaError_t launch_gemm_two(const GemmTask& t0, const GemmTask& t1, dprc_dtype dt,
                            cudaStream_t s) {
  CUtensorMap maps[4];
  GemmBatch batch;
  const GemmTask* t[2] = {&t0, &t1};
  for (int i = 0; i < 2; ++i) {
    GemmPlan p;
    p.pair = true;
    p.units = p.per = t[i]->plan->units;
    const cudaError_t e = prepare_gemm(*t[i]->shape, p, t[i]->A, t[i]->B, t[i]->epi, nullptr,
                                       maps + 2 * i, batch.p[i]);
    if (e != cudaSuccess) return e;
  }
  batch.n0 = static_cast<int>(unit_count(batch.p[0]));
  batch.n1 = static_cast<int>(unit_count(batch.p[1]));
  const long long pairs = std::min<long long>(static_cast<long long>(batch.n0) + batch.n1, device_sm_count() / 2);
  deal_units(batch.n0, batch.p[0].units, batch.n1, batch.p[1].units, pairs, batch.extra,
             batch.a_units);
  return dt == DPRC_F32 ? launch_gemm_pair<float>(maps, batch, s)
                        : launch_gemm_pair<__nv_bfloat16>(maps, batch, s);
}

}  // namespace dprc
