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
// threads that own a column.  Measured, bf16: forward 16384 x 2048 29 us (0.68 of the copy
// rate), x 2049 94 (accesses of rows at any element of
// theirs); gradient with norms and weights 61 (201 MB in 30 us at the copy rate; the join of
// the chunks and the norms' sum are 10 of it), x 2049 143; 2048 x 16384 96, x 16383 166.
//
// A row is shared by G threads (a power of two), each of which holds up to kNv
// accesses of kE elements, 16 bytes.  Up to 32 threads sum by shuffles; more through
// shared memory.

#include <algorithm>
#include <type_traits>

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
  const int lane = threadIdx.x & 31;
  if (G >= 32 && kN == 2) {
    // the upper half of the lanes sums the second value, so that one shuffle serves both
    const bool upper = (lane & 16) != 0;
    const float give = upper ? v[0] : v[1];
    float keep = upper ? v[kN - 1] : v[0];
    keep += __shfl_xor_sync(0xffffffffu, give, 16);
    for (int o = 8; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
    const float other = __shfl_xor_sync(0xffffffffu, keep, 16);
    v[0] = upper ? other : keep;
    v[kN - 1] = upper ? keep : other;
  } else {
    const int lim = G < 32 ? G : 32;
    for (int o = 1; o < lim; o <<= 1)
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (G <= 32) return;
  const int warp = threadIdx.x >> 5, per = G >> 5;
  float* b = buf + (turn & 1) * kMaxWarps * kN;
  ++turn;
  if (lane == 0)
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

// A row's accesses.  A width that is no multiple of kE puts the rows at any element of
// a 16-byte access: the accesses stay whole and lie `shift` elements ahead of the row, so
// that the first and the last hold elements of its neighbours, which are masked; only
// what would reach behind the tensor is read element by element.  kOdd: such widths.
template <typename T, int kE, bool kOdd>
struct RowAccess {
  int d, shift;
  long long end;  // elements of the tensor
  __device__ __forceinline__ RowAccess(int d, long long row, long long rows)
      : d(d), shift(kOdd ? static_cast<int>(row * d % kE) : 0), end(rows * d) {}
  // the first column of access v
  __device__ __forceinline__ int col(int v) const { return v * kE - shift; }
  __device__ __forceinline__ bool any(int c) const { return c < d; }
  __device__ __forceinline__ bool whole(int c) const { return !kOdd || (c >= 0 && c + kE <= d); }
  __device__ __forceinline__ void load(Raw<T, kE>& r, const T* p, long long row, int c) const {
    const long long at = row * d + c;
    if (!kOdd || at + kE <= end) {
      r.load(p + at);
    } else {
      T* e = reinterpret_cast<T*>(&r);
      for (int i = 0; i < kE; ++i) e[i] = at + i < end ? ld_once(p + at + i) : T(0.f);
    }
  }
  __device__ __forceinline__ void store(T* p, long long row, int c, const float* v) const {
    T* out = p + row * d + c;
    if (!DPRC_IN(row >= 0 && (row + 1) * d <= end)) return;
    if (whole(c)) {
      store_row<kE>(out, v);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (c + e >= 0 && c + e < d) store_row<1>(out + e, v + e);
    }
  }
  // parameters of the columns, `none` where there are none
  __device__ __forceinline__ void param(float* v, const T* p, int c, float none) const {
    if (p == nullptr) {
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] = none;
    } else if constexpr (kOdd) {
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] = c + e >= 0 && c + e < d ? to_f32<T>(p[c + e]) : 0.f;
    } else {
      Raw<T, kE> u;
      u.a = *reinterpret_cast<const decltype(u.a)*>(p + c);
      u.get(v);
    }
  }
};

// The variance is summed of the differences from the mean, in registers: no
// cancellation of large means.  What the mean lost in its rounding is the mean of
// those differences, and taken off them too: two values that agree to a half
// step of each other still come out at full accuracy.
template <typename T, int kE, int kNv, bool kOdd>
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
  const RowAccess<T, kE, kOdd> at(d, mine ? row : 0, rows);
  Raw<T, kE> raw[kNv];
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const int c = at.col(k * G + t);
    if (mine && at.any(c)) at.load(raw[k], x, row, c); else raw[k].zero();
  }
  const auto values = [&](int k, float* v, float none) {  // of access k, `none` outside the row
    const int c = at.col(k * G + t);
    raw[k].get(v);
    if (!at.whole(c)) {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (c + e < 0 || c + e >= d) v[e] = none;
    }
  };
  const float inv = 1.f / static_cast<float>(d);
  float mean = 0.f;
  if (center) {
    F2 sum = f2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      float v[kE];
      values(k, v, 0.f);
#pragma unroll
      for (int e = 0; e < kE; e += 2) sum = add2(sum, f2(v[e], v[e + 1]));
    }
    float s[1], u;
    split(sum, s[0], u);
    s[0] += u;
    row_sum<1>(s, G, buf, turn);
    mean = s[0] * inv;
  }
  const F2 off = f2(-mean, -mean);
  F2 q0 = f2(0.f, 0.f), q1 = q0;  // of the differences (what the mean's rounding left), squares
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    if (at.any(at.col(k * G + t))) {
      float v[kE];
      values(k, v, mean);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const F2 dm = add2(f2(v[e], v[e + 1]), off);
        q0 = add2(q0, dm);
        q1 = fma2(dm, dm, q1);
      }
    }
  }
  float q[2], u;
  split(q0, q[0], u);
  q[0] += u;
  split(q1, q[1], u);
  q[1] += u;
  row_sum<2>(q, G, buf, turn);
  const float left = center ? q[0] * inv : 0.f;
  const float rstd = 1.f / sqrtf(fmaxf(q[1] * inv - left * left, 0.f) + eps);
  if (!mine) return;
  if (stats != nullptr && t == 0) stats[row] = make_float2(mean + left, rstd);
  const F2 rs2 = f2(rstd, rstd), left2 = f2(-left, -left);
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const int c = at.col(k * G + t);
    if (!at.any(c)) continue;
    // y = (x - mean) r w + (b - left r w)
    float v[kE], wv[kE], bv[kE];
    raw[k].get(v);
    at.param(wv, w, c, 1.f);
    at.param(bv, b, c, 0.f);
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const F2 rw = mul2(f2(wv[e], wv[e + 1]), rs2);
      const F2 y2 = fma2(add2(f2(v[e], v[e + 1]), off), rw, fma2(left2, rw, f2(bv[e], bv[e + 1])));
      split(y2, v[e], v[e + 1]);
    }
    at.store(y, row, c, v);
  }
}

struct LnGradArgs {
  const float2* stats;
  const float* c;        // factors of the samples' rows, or null: 1
  long long rows;        // of a sample (blockIdx.y)
  long long per_chunk;   // rows of a chunk
  long long T;           // rows of a sample of c
  long long all;         // rows of the tensor
  int d, G, center, sums;
  int classes;           // CTAs of a chunk (odd widths: rows of one shift have a CTA of their own)
  float* part;           // [samples][CTAs][2][d]
};

// Wide rows: a CTA of 512 threads takes a row at a time and reads the next one before it
// sums.  The sums over rows stand in shared memory, each column's where its thread alone
// adds to it.  A CTA's rows are kE apart where the width is odd, so that they have the
// same shift and a thread the same columns.
template <typename T, int kE, int kNv, bool kOdd>
__global__ void __launch_bounds__(kLnWide)
    layernorm_grad_kernel(const T* dy, const T* x, const T* w, T* dx, const LnGradArgs a) {
  constexpr int kC = kNv * kE;
  __shared__ float buf[2 * kMaxWarps * 2];
  extern __shared__ __align__(16) float sums[];  // [2][kC / 2][512] pairs
  pdl_launch_dependents();
  pdl_wait();
  int turn = 0;
  const int d = a.d, G = kLnWide, t = threadIdx.x;
  const long long base = blockIdx.y * a.rows;  // the sample's first row
  const int chunk = blockIdx.x / a.classes, cls = blockIdx.x - chunk * a.classes;
  const long long r0 = chunk * a.per_chunk;
  const long long r1 = min(r0 + a.per_chunk, a.rows);
  const int stride = kOdd ? kE : 1;
  const long long first = r0 + cls;
  const RowAccess<T, kE, kOdd> at(d, base + first, a.all);
  const float inv = 1.f / static_cast<float>(d);
  F2* wsum = reinterpret_cast<F2*>(sums) + t;
  F2* bsum = wsum + kC / 2 * kLnWide;
#pragma unroll
  for (int i = 0; i < kC / 2; ++i) wsum[i * kLnWide] = bsum[i * kLnWide] = f2(0.f, 0.f);
  Raw<T, kE> xv[kNv], gv[kNv];
  float2 st = make_float2(0.f, 0.f);
  const auto fetch = [&](long long q) {
    if (q >= r1) return;
    st = ld_once(a.stats + base + q);
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = at.col(k * G + t);
      if (at.any(c)) {
        at.load(xv[k], x, base + q, c);
        at.load(gv[k], dy, base + q, c);
      }
    }
  };
  // x - mu and dy of an access in pairs, 0 outside the row
  const auto values = [&](const Raw<T, kE>& xr, const Raw<T, kE>& gr, float mu, int c, F2* dm,
                          F2* g) {
    float u[kE], v[kE];
    xr.get(u);
    gr.get(v);
    if (!at.whole(c)) {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (c + e < 0 || c + e >= d) {
          u[e] = mu;
          v[e] = 0.f;
        }
    }
    const F2 m = f2(-mu, -mu);
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) {
      dm[e] = add2(f2(u[2 * e], u[2 * e + 1]), m);
      g[e] = f2(v[2 * e], v[2 * e + 1]);
    }
  };
  // the weights of access k, read again (from L1)
  const auto weights = [&](int k, F2* w2) {
    float u[kE];
    at.param(u, w, at.col(k * G + t), 1.f);
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) w2[e] = f2(u[2 * e], u[2 * e + 1]);
  };
  fetch(first);
  for (long long r = first; r < r1; r += stride) {  // (the same for the CTA)
    F2 dm[kC / 2], g[kC / 2];  // x - mu, dy
    const float2 sc = st;
    F2 s0 = f2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = at.col(k * G + t);
      if (!at.any(c)) continue;
      values(xv[k], gv[k], sc.x, c, &dm[k * kE / 2], &g[k * kE / 2]);
      F2 w2[kE / 2];
      weights(k, w2);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        const int i = k * kE / 2 + e;
        const F2 gw = mul2(g[i], w2[e]);
        s0 = add2(s0, gw);
        s1 = fma2(gw, dm[i], s1);
      }
    }
    float s[2], u;
    split(s0, s[0], u);
    s[0] += u;
    split(s1, s[1], u);
    s[1] += u;
    fetch(r + stride);  // the next row is on its way while this one is summed
    if (dx != nullptr) row_sum<2>(s, G, buf, turn);
    // dx = r g + (x - mu) (-r^3 mean(g (x - mu))) - r mean(g)
    // (r by r: r^3 leaves fp32's range where a deviation is above 10^13 or below 10^-12)
    const float rs = sc.y, f = a.c != nullptr ? a.c[(base + r) / a.T] : 1.f;
    const float along = -rs * (rs * (rs * (s[1] * inv)));
    const float rest = a.center ? -rs * (s[0] * inv) : 0.f;
    const F2 rs2 = f2(rs, rs), along2 = f2(along, along), rest2 = f2(rest, rest);
    const F2 fr2 = f2(f * rs, f * rs), f22 = f2(f, f);
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      const int c = at.col(k * G + t);
      if (!at.any(c)) continue;
      float out[kE];
      F2 w2[kE / 2];
      weights(k, w2);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        const int i = k * kE / 2 + e;
        const F2 o = fma2(dm[i], along2, fma2(mul2(g[i], w2[e]), rs2, rest2));
        split(o, out[2 * e], out[2 * e + 1]);
        wsum[i * kLnWide] = fma2(mul2(g[i], fr2), dm[i], wsum[i * kLnWide]);
        bsum[i * kLnWide] = fma2(g[i], f22, bsum[i * kLnWide]);
      }
      if (dx != nullptr) at.store(dx, base + r, c, out);
    }
  }
  if (!a.sums) return;
  float* part = a.part + (blockIdx.y * static_cast<long long>(gridDim.x) + blockIdx.x) * 2 * d;
#pragma unroll
  for (int i = 0; i < kC / 2; ++i) {
    float wv[2], bv[2];
    split(wsum[i * kLnWide], wv[0], wv[1]);
    split(bsum[i * kLnWide], bv[0], bv[1]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = at.col(2 * i / kE * G + t) + (2 * i + q) % kE;
      if (c < 0 || c >= d) continue;
      part[c] = wv[q];
      part[d + c] = bv[q];
    }
  }
}

// Rows of up to 4096 elements: blocks of rows of both tensors come by bulk copies into a
// ring of stages in shared memory, several blocks ahead, so that the memory always has
// enough to do; the registers hold a block's values and the columns' sums.  A block
// starts at any element (odd widths): its copy starts at the 16 bytes before, and what it
// leaves of the tensor's last bytes is read element by element.  Odd widths are taken
// an element an access (kE = 1), neighbouring threads neighbouring columns.
constexpr int kRingBytes = 96 * 1024;
constexpr int kMaxRing = 8;
constexpr int kRingMost = 112 * 1024;  // what a CTA may take, two to an SM

struct RingPlan {
  int rows, stages, bytes;  // rows of a block; bytes of a tensor's block in a stage
};
__host__ __device__ inline RingPlan ring_plan(int d, int size, int G, int rows) {
  RingPlan p;
  p.rows = kLnThreads / G * rows;
  p.bytes = (p.rows * d * size + 15) / 16 * 16 + 16;
  p.stages = kRingBytes / (2 * p.bytes);
  p.stages = p.stages < 2 ? 2 : p.stages > kMaxRing ? kMaxRing : p.stages;
  return p;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, int bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

template <typename T, int kE, int kNv, int kRows>
__global__ void __launch_bounds__(kLnThreads, 2)
    layernorm_grad_ring_kernel(const T* dy, const T* x, const T* w, T* dx, const LnGradArgs a) {
  constexpr int kC = kNv * kE;
  static_assert(kC % 2 == 0, "pairs");
  __shared__ float buf[2 * kMaxWarps * 2 * kRows];
  __shared__ uint64_t full[kMaxRing];
  extern __shared__ __align__(16) uint8_t ring_raw[];
  const int d = a.d, G = a.G;
  const RingPlan plan = ring_plan(d, sizeof(T), G, kRows);
  uint8_t* ring = ring_raw;  // [stages][x, dy][bytes]; at the end the groups' sums [2][d]
  float* sums = reinterpret_cast<float*>(ring_raw);
  if (threadIdx.x == 0) {
    for (int s = 0; s < plan.stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  __syncthreads();
  pdl_wait();
  int turn = 0;
  const int t = threadIdx.x & (G - 1), groups = kLnThreads / G, grp = threadIdx.x / G;
  const long long base = blockIdx.y * a.rows;  // the sample's first row
  const long long r0 = blockIdx.x * a.per_chunk;
  const long long r1 = min(r0 + a.per_chunk, a.rows);
  const int blocks = r1 > r0 ? static_cast<int>((r1 - r0 + plan.rows - 1) / plan.rows) : 0;
  const long long end = a.all * d;  // elements of a tensor
  constexpr int kU = 16 / static_cast<int>(sizeof(T));
  // block k: its first element, and the whole 16 bytes that the copies bring
  const auto first_of = [&](int k) { return (base + r0 + static_cast<long long>(k) * plan.rows) * d; };
  const auto copied = [&](int k, long long& from) {  // elements
    const long long e0 = first_of(k);
    const long long e1 = min(e0 + static_cast<long long>(plan.rows) * d, (base + r1) * d);
    from = e0 / kU * kU;
    return static_cast<int>(min((e1 + kU - 1) / kU * kU, end / kU * kU) - from);
  };
  const auto issue = [&](int k, int s) {
    long long from;
    const int n = copied(k, from);
    const int bytes = n * static_cast<int>(sizeof(T));
    uint8_t* to = ring + s * 2 * plan.bytes;
    mbar_arrive_expect_tx(&full[s], 2 * (bytes > 0 ? bytes : 0));
    if (bytes > 0) {
      bulk_load(to, x + from, bytes, &full[s]);
      bulk_load(to + plan.bytes, dy + from, bytes, &full[s]);
    }
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < plan.stages && k < blocks; ++k) issue(k, k);
  const float inv = 1.f / static_cast<float>(d);
  F2 w2[kC / 2], wsum[kC / 2], bsum[kC / 2];
  const auto col = [&](int f) { return (f / kE * G + t) * kE + f % kE; };
#pragma unroll
  for (int i = 0; i < kC / 2; ++i) {
    float u[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = col(2 * i + q);
      u[q] = c < d ? (w != nullptr ? to_f32<T>(w[c]) : 1.f) : 0.f;
    }
    w2[i] = f2(u[0], u[1]);
    wsum[i] = bsum[i] = f2(0.f, 0.f);
  }
  // (running values: an index formed anew for each block took a third of the instructions)
  int left = static_cast<int>(r1 - r0) - grp;  // rows from the group's on
  const float2* sp = a.stats + base + r0 + grp;
  T* dxp = dx != nullptr ? dx + (base + r0 + grp) * d + t * kE : nullptr;
  const long long dx_step = static_cast<long long>(plan.rows) * d;
  float2 ahead[kRows];
  const auto stats_of = [&]() {
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      ahead[j] = j * groups < left ? ld_once(sp + j * groups) : make_float2(0.f, 0.f);
  };
  stats_of();
  int s = 0;
  uint32_t round = 0;
  for (int k = 0; k < blocks; ++k) {
    long long from = 0;
    int n = 0, shift = 0;
    if constexpr (kE == 1) {
      n = copied(k, from);
      shift = static_cast<int>(first_of(k) - from);
    }
    const T* xs = reinterpret_cast<const T*>(ring + s * 2 * plan.bytes);
    const T* gs = reinterpret_cast<const T*>(ring + s * 2 * plan.bytes + plan.bytes);
    const int have = left;
    float2 st[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) st[j] = ahead[j];
    sp += plan.rows;
    left -= plan.rows;
    stats_of();  // the next block's are on their way while this one is taken
    // (a copy that was started ends; a wait that runs out is recorded)
    mbar_wait(&full[s], round, DPRC_DEVERR_PIPE_FULL);
    F2 dm[kRows][kC / 2], g[kRows][kC / 2];  // x - mu, dy
    float sum[2 * kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int lr = j * groups + grp;
      const bool mine = j * groups < have;
      F2 s0 = f2(0.f, 0.f), s1 = s0;
      float xv[kC], gv[kC];
#pragma unroll
      for (int v = 0; v < kNv; ++v) {
        const int c = (v * G + t) * kE, at = shift + lr * d + c;
        if (mine && c < d) {
          if (!DPRC_IN(at >= 0 && (at + kE) * static_cast<int>(sizeof(T)) <= plan.bytes)) {
#pragma unroll
            for (int e = 0; e < kE; ++e) xv[v * kE + e] = gv[v * kE + e] = 0.f;
          } else if constexpr (kE == 1) {
            // the tensor's last bytes, which the copies leave, are read where they are
            xv[v] = to_f32<T>(at < n ? xs[at] : x[from + at]);
            gv[v] = to_f32<T>(at < n ? gs[at] : dy[from + at]);
          } else {
            Raw<T, kE> u;
            u.a = *reinterpret_cast<const decltype(u.a)*>(xs + at);
            u.get(xv + v * kE);
            u.a = *reinterpret_cast<const decltype(u.a)*>(gs + at);
            u.get(gv + v * kE);
          }
        } else {
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            xv[v * kE + e] = st[j].x;
            gv[v * kE + e] = 0.f;
          }
        }
      }
      const F2 mu = f2(-st[j].x, -st[j].x);
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) {
        dm[j][i] = add2(f2(xv[2 * i], xv[2 * i + 1]), mu);
        g[j][i] = f2(gv[2 * i], gv[2 * i + 1]);
        const F2 gw = mul2(g[j][i], w2[i]);
        s0 = add2(s0, gw);
        s1 = fma2(gw, dm[j][i], s1);
      }
      float u;
      split(s0, sum[2 * j], u);
      sum[2 * j] += u;
      split(s1, sum[2 * j + 1], u);
      sum[2 * j + 1] += u;
    }
    row_sum<2 * kRows>(sum, G, buf, turn);
    if (G <= 32) __syncthreads();  // (else the sums' barrier)
    // everyone has read the stage
    if (threadIdx.x == 0 && k + plan.stages < blocks) issue(k + plan.stages, s);
    if (++s == plan.stages) {
      s = 0;
      round ^= 1u;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (j * groups >= have) continue;
      // dx = r g + (x - mu) (-r^3 mean(g (x - mu))) - r mean(g)
      // (r by r: r^3 leaves fp32's range where a deviation is above 10^13 or below 10^-12)
      float f = 1.f;
      if (a.c != nullptr)
        f = a.c[(base + r0 + static_cast<long long>(k) * plan.rows + j * groups + grp) / a.T];
      const float rs = st[j].y;
      const float along = -rs * (rs * (rs * (sum[2 * j + 1] * inv)));
      const float rest = a.center ? -rs * (sum[2 * j] * inv) : 0.f;
      const F2 rs2 = f2(rs, rs), along2 = f2(along, along), rest2 = f2(rest, rest);
      const F2 fr2 = f2(f * rs, f * rs), f22 = f2(f, f);
      float out[kC];
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) {
        const F2 o = fma2(dm[j][i], along2, fma2(mul2(g[j][i], w2[i]), rs2, rest2));
        split(o, out[2 * i], out[2 * i + 1]);
        wsum[i] = fma2(mul2(g[j][i], fr2), dm[j][i], wsum[i]);
        bsum[i] = fma2(g[j][i], f22, bsum[i]);
      }
      if (dx != nullptr) {
#pragma unroll
        for (int v = 0; v < kNv; ++v) {
          const int c = (v * G + t) * kE;
          if (c < d) store_row<kE>(dxp + j * groups * d + v * G * kE, out + v * kE);
        }
      }
    }
    if (dx != nullptr) dxp += dx_step;
  }
  if (!a.sums) return;
  float* part = a.part + (blockIdx.y * static_cast<long long>(gridDim.x) + blockIdx.x) * 2 * d;
  // the groups of the CTA in order, each adding its columns
  for (int q = 0; q < groups; ++q) {
    __syncthreads();
    if (grp != q) continue;
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) {
      float wv[2], bv[2];
      split(wsum[i], wv[0], wv[1]);
      split(bsum[i], bv[0], bv[1]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = col(2 * i + u);
        if (c >= d) continue;
        if (q > 0) {
          wv[u] += sums[c];
          bv[u] += sums[d + c];
        }
        float* out = q + 1 < groups ? sums : part;
        out[c] = wv[u];
        out[d + c] = bv[u];
      }
    }
  }
}

constexpr int kFinWarps = 32;

// The samples' sums over their chunks, 32 columns of the weight's (blockIdx.y 0)
// or the bias's a CTA: their squares, and the sum over the samples times c.  A warp
// takes every 32nd chunk of a sample (few samples) or every 32nd sample.
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
  if (B < 2 * kFinWarps) {
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

// Chunks of rows: as many CTAs as are resident (two to an SM), at least 16 rows each.
// Odd widths: up to `classes` CTAs a chunk.
struct LnPlan {
  int64_t samples, rows, chunks, per_chunk;
};
LnPlan plan_grad(int64_t B, int64_t T, bool by_sample, int64_t classes) {
  LnPlan p;
  p.samples = by_sample ? B : 1;
  p.rows = by_sample ? T : B * T;
  const int64_t want = std::max<int64_t>(1, 2 * 152 / (p.samples * classes));
  p.per_chunk = std::max<int64_t>(16 * classes, (p.rows + want - 1) / want);
  p.chunks = std::max<int64_t>(1, (p.rows + p.per_chunk - 1) / p.per_chunk);
  return p;
}

// Threads of a row and accesses of a thread.  Up to 4096 elements (16 a thread): the ring,
// of accesses of 16 bytes or of an element; wider: accesses of 16 bytes, shifted (one more)
// where the width is odd.
struct RowShape {
  bool odd, wide;
  int G;
  int64_t nv;
};
template <typename T>
RowShape grad_shape(int64_t d) {
  constexpr int kV = kVec16<T>;
  RowShape r;
  r.odd = !whole_vectors<T>(d);
  r.wide = d > kLnThreads * 16;
  int64_t acc = r.odd && !r.wide ? d : (d + kV - 1) / kV;
  if (r.wide && r.odd) ++acc;
  // 16 elements a thread: the sums of a row, whose operations a thread has whatever its
  // share, are spread over fewer threads
  r.G = r.wide ? kLnWide : pow2_at_least((acc * (r.odd ? 1 : kV) + 15) / 16, 8, kLnThreads);
  r.nv = (acc + r.G - 1) / r.G;
  return r;
}
template <typename T>
int64_t grad_classes(int64_t d) {
  const RowShape r = grad_shape<T>(d);
  return r.odd && r.wide ? kVec16<T> : 1;
}

template <typename T>
cudaError_t forward(const LayernormCall& c, cudaStream_t s) {
  const int64_t rows = c.B * c.T, d = c.d;
  const T* x = static_cast<const T*>(c.X);
  const T* w = static_cast<const T*>(c.weight);
  const T* b = static_cast<const T*>(c.bias);
  T* y = static_cast<T*>(c.Y);
  constexpr int kV = kVec16<T>;
  const bool odd = !whole_vectors<T>(d);
  const int64_t acc = (d + kV - 1) / kV + (odd ? 1 : 0);  // accesses of a row (a shift adds one)
  // a warp or less a row while its share fits 64 registers, else a CTA
  const int G = acc * kV <= 32 * 64 ? pow2_at_least(acc, 8, 32) : kLnThreads;
  const int64_t nv = (acc + G - 1) / G;
  const int64_t per = kLnThreads / G;
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per));
  float2* st = reinterpret_cast<float2*>(c.stats);
  const auto go = [&](auto kernel) {
    return launch_after(kernel, grid, kLnThreads, 1, s, 0, x, w, b, static_cast<long long>(rows),
                        static_cast<int>(d), G, c.eps, c.center, y, st);
  };
  const auto by_odd = [&](auto n) {
    constexpr int kN = decltype(n)::value;
    return odd ? go(layernorm_kernel<T, kV, kN, true>) : go(layernorm_kernel<T, kV, kN, false>);
  };
  if (nv <= 1) return by_odd(std::integral_constant<int, 1>{});
  if (nv <= 2) return by_odd(std::integral_constant<int, 2>{});
  if (nv <= 4) return by_odd(std::integral_constant<int, 4>{});
  if (nv <= 8) return by_odd(std::integral_constant<int, 8>{});
  // (an odd width of nearly 16384 has one access more)
  if constexpr (kV == 4) return by_odd(std::integral_constant<int, 17>{});
  else return go(layernorm_kernel<T, kV, 9, true>);
}

template <typename T>
cudaError_t backward(const LayernormGradCall& c, void* ws, cudaStream_t s) {
  const bool by_sample = c.n != nullptr;
  const int64_t d = c.d, classes = grad_classes<T>(d);
  const RowShape shape = grad_shape<T>(d);
  const LnPlan p = plan_grad(c.B, c.T, by_sample, classes);
  constexpr int kV = kVec16<T>;
  const bool sums = c.dW != nullptr || c.db != nullptr || by_sample;
  LnGradArgs a;
  a.stats = reinterpret_cast<const float2*>(c.stats);
  a.c = by_sample ? nullptr : c.c;  // (by sample, the finishing step takes it)
  a.rows = p.rows;
  a.per_chunk = p.per_chunk;
  a.T = std::max<int64_t>(1, c.T);
  a.all = c.B * c.T;
  a.d = static_cast<int>(d);
  a.G = shape.G;
  a.center = c.center;
  a.sums = sums;
  a.classes = static_cast<int>(classes);
  a.part = static_cast<float*>(ws);
  const dim3 grid(static_cast<unsigned>(p.chunks * classes), static_cast<unsigned>(p.samples));
  const auto go = [&](auto kernel, int threads, size_t smem) {
    return launch_after(kernel, grid, threads, 1, s, smem, static_cast<const T*>(c.dY),
                        static_cast<const T*>(c.X), static_cast<const T*>(c.weight),
                        static_cast<T*>(c.dX), a);
  };
  const auto ring = [&](auto e, auto n) {
    constexpr int kE = decltype(e)::value, kN = decltype(n)::value, kR = kE * kN <= 4 ? 2 : 1;
    const RingPlan rp = ring_plan(static_cast<int>(d), sizeof(T), shape.G, kR);
    const int bytes = std::max<int>(rp.stages * 2 * rp.bytes, 2 * static_cast<int>(d) * 4);
    const cudaError_t err = allow_smem<layernorm_grad_ring_kernel<T, kE, kN, kR>>(kRingMost);
    return err != cudaSuccess
        ? err : go(layernorm_grad_ring_kernel<T, kE, kN, kR>, kLnThreads, bytes);
  };
  const auto wide_of = [&](auto n, auto o) {
    constexpr int kN = decltype(n)::value, bytes = 2 * kN * kV * kLnWide * 4;
    constexpr bool kO = decltype(o)::value;
    const cudaError_t e = allow_smem<layernorm_grad_kernel<T, kV, kN, kO>>(bytes);
    return e != cudaSuccess ? e : go(layernorm_grad_kernel<T, kV, kN, kO>, kLnWide, bytes);
  };
  const auto wide = [&](auto n) {
    return shape.odd ? wide_of(n, std::true_type{}) : wide_of(n, std::false_type{});
  };
  cudaError_t err;
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, kV> vec{};
  if (shape.wide) {
    constexpr int kUnit = 8 / kV;  // accesses of eight elements
    if (shape.nv <= 2 * kUnit) err = wide(std::integral_constant<int, 2 * kUnit>{});
    else if (shape.nv <= 3 * kUnit) err = wide(std::integral_constant<int, 3 * kUnit>{});
    else if (shape.nv <= 4 * kUnit) err = wide(std::integral_constant<int, 4 * kUnit>{});
    else err = wide_of(std::integral_constant<int, 4 * kUnit + 1>{}, std::true_type{});  // (a shift's)
  } else if (shape.odd) {
    if (shape.nv <= 2) err = ring(one, std::integral_constant<int, 2>{});
    else if (shape.nv <= 4) err = ring(one, std::integral_constant<int, 4>{});
    else if (shape.nv <= 8) err = ring(one, std::integral_constant<int, 8>{});
    else err = ring(one, std::integral_constant<int, 16>{});
  } else if (shape.nv <= 1) {
    err = ring(vec, std::integral_constant<int, 1>{});
  } else if (shape.nv <= 2) {
    err = ring(vec, std::integral_constant<int, 2>{});
  } else {
    err = ring(vec, std::integral_constant<int, 16 / kV>{});
  }
  if (err != cudaSuccess || !sums) return err;
  const int tiles = static_cast<int>((d + 31) / 32);
  const int64_t ctas = p.chunks * classes;
  float* npart = by_sample ? a.part + p.samples * ctas * 2 * d : nullptr;
  const int parts = c.norm_of_bias ? 2 : 1;
  const float* cf = by_sample ? c.c : nullptr;
  const int which = c.db != nullptr || (by_sample && c.norm_of_bias) ? 2 : 1;
  err = launch_after(layernorm_finish_kernel<T>, dim3(tiles, which), 32 * kFinWarps, 1, s, 0,
                     static_cast<const float*>(a.part), cf, static_cast<int>(p.samples),
                     static_cast<int>(ctas), static_cast<int>(d), static_cast<T*>(c.dW),
                     static_cast<T*>(c.db), npart, parts);
  if (err != cudaSuccess || !by_sample) return err;
  return launch_after(layernorm_norm_kernel, dim3(static_cast<unsigned>((c.B + 7) / 8)), 256, 1, s,
                      0, static_cast<const float*>(npart), tiles * parts, static_cast<int>(c.B),
                      c.n, c.accumulate);
}

}  // namespace

size_t layernorm_grad_ws_bytes(int64_t B, int64_t T, int64_t d, int with_norms) {
  size_t part = 0;
  for (const int64_t classes : {grad_classes<float>(d), grad_classes<__nv_bfloat16>(d)}) {
    const LnPlan p = plan_grad(B, T, with_norms != 0, classes);
    part = std::max(part, static_cast<size_t>(p.samples) * p.chunks * classes * 2 * d * 4);
  }
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
