// The embedding of a DP-SGD-RC step: lookup, the sorted token order that its
// gradient is taken in, the exact per-sample squared norm of that gradient and
// the clipped gradient itself.
//
// The weight W [V][d] of an embedding gets, from sample i, the gradient
//   dW_i[v] = s * sum over t with tok_it = v of G_it      (G the gradient of the output)
// so  ||dW_i||^2 = s^2 sum_v || sum_{t: tok_it = v} G_it ||^2   and
//     sum_i c_i dW_i[v] = s sum_i c_i sum_{t: tok_it = v} G_it.
// Both are sums over groups of equal tokens.  The tokens are sorted once,
// stably, with their positions (dprc_embed_plan); a group is then a run of
// consecutive entries, a token's entries of one sample are a run inside it,
// and one pass over the rows of G in that order gives either result with no
// atomics: every sum has one fixed order, so results repeat bitwise.
//
// What bounds them: bytes.  The lookup writes N d values, the norm reads them
// once, the gradient reads them once and writes all V rows.

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dprc {
namespace {

// ---------------------------------------------------------------------------
// Accesses of AW bytes (16, 8, 4 or 2) to rows whose pitch is a multiple of AW.
// ---------------------------------------------------------------------------
template <int AW>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}

// The AW / sizeof(T) values of one access as fp32.
template <typename T, int AW>
__device__ __forceinline__ void unpack(const typename Raw<AW>::type& raw, float* v) {
  constexpr int VE = AW / static_cast<int>(sizeof(T));
  if constexpr (sizeof(T) == 4) {
    const float* f = reinterpret_cast<const float*>(&raw);
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = f[e];
  } else if constexpr (VE == 1) {
    v[0] = bf16_bits_to_f32(raw);
  } else {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
  }
}

template <typename T, int AW>
__device__ __forceinline__ typename Raw<AW>::type pack(const float* v) {
  constexpr int VE = AW / static_cast<int>(sizeof(T));
  typename Raw<AW>::type raw;
  if constexpr (sizeof(T) == 4) {
    float* f = reinterpret_cast<float*>(&raw);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = v[e];
  } else if constexpr (VE == 1) {
    raw = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
  } else {
    uint32_t* u = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      u[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return raw;
}

// Two fp32 operations in one instruction (sm_100 and later).
__device__ __forceinline__ unsigned long long pair(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float pair_sum(unsigned long long a) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
  return lo + hi;
}

// Sum of squares of n values (n a power of two), in up to four chains.
template <int n>
__device__ __forceinline__ float square_sum(const float* v) {
  if constexpr (n == 1) {
    return v[0] * v[0];
  } else {
    unsigned long long s[2] = {0ull, 0ull};
#pragma unroll
    for (int e = 0; e < n; e += 2) {
      const unsigned long long x = pair(v[e], v[e + 1]);
      s[(e >> 1) & 1] = fma2(x, x, s[(e >> 1) & 1]);
    }
    return pair_sum(s[0]) + pair_sum(s[1]);
  }
}

// A token as a sort key: ids outside [0, V) become V, the last key.  A
// negative id means "no token"; one of V or more is a mistake of the caller
// and is recorded in the device error word.
template <typename TOK>
__device__ __forceinline__ uint32_t token_key(TOK t, int V) {
  if (t >= 0 && t < static_cast<TOK>(V)) return static_cast<uint32_t>(t);
  if (t >= 0) record_error(DPRC_DEVERR_TOKEN);
  return static_cast<uint32_t>(V);
}

// ---------------------------------------------------------------------------
// Lookup.  A unit is up to 4 accesses per lane of one row; `lanes` lanes (a
// power of two) share a row, so narrow rows do not idle most of a warp.
// Bound by bytes: 4 x 4096 tokens of 2048 bf16 with repeats 16.6 us in turn on
// one stream (13.9 at the copy rate), 18.5 behind the full end of the kernel
// before; eight accesses a lane 18.6.
// ---------------------------------------------------------------------------
constexpr int kLookupUnroll = 4;

template <typename T, int AW, typename TOK>
__global__ void __launch_bounds__(256)
    embed_lookup_kernel(const T* W, const TOK* tokens, long long N, int V, long long d,
                        float scale, T* out, int lanes, int units_per_row) {
  using R = typename Raw<AW>::type;
  constexpr int VE = AW / static_cast<int>(sizeof(T));
  pdl_launch_dependents();
  pdl_wait();
  const int nvec = static_cast<int>(d / VE);
  const int sub = threadIdx.x & (lanes - 1);
  const long long groups = static_cast<long long>(gridDim.x) * (blockDim.x / lanes);
  const long long units = N * units_per_row;
  for (long long u = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / lanes;
       u < units; u += groups) {
    const long long row = u / units_per_row;
    const int v0 = static_cast<int>(u - row * units_per_row) * lanes * kLookupUnroll + sub;
    const uint32_t key = token_key(tokens[row], V);
    const bool have = key < static_cast<uint32_t>(V);
    const R* src = reinterpret_cast<const R*>(W + static_cast<long long>(have ? key : 0) * d);
    R* dst = reinterpret_cast<R*>(out + row * d);
    R raw[kLookupUnroll];
#pragma unroll
    for (int j = 0; j < kLookupUnroll; ++j) {
      const int v = v0 + j * lanes;
      if (have && v < nvec) raw[j] = src[v];
    }
#pragma unroll
    for (int j = 0; j < kLookupUnroll; ++j) {
      const int v = v0 + j * lanes;
      if (v >= nvec) continue;
      float f[VE];
      if (have) {
        unpack<T, AW>(raw[j], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] *= scale;
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = 0.f;
      }
      if (DPRC_IN(row < N)) __stcs(dst + v, pack<T, AW>(f));
    }
  }
}

// ---------------------------------------------------------------------------
// The order, up to kRankMax tokens: an entry's place is the number of entries
// that come before it, keys_j < key_i or equal with j < i, counted by
// comparison.  Every CTA holds all keys in shared memory, a warp counts for
// four entries, its lanes over the keys.  N^2 comparisons over the whole GPU
// take less than the barriers of a radix sort: 2.3 us for 512 tokens, 4.4 us
// for 3000.
// ---------------------------------------------------------------------------
constexpr int kRankMax = 8192;
constexpr int kRankWarps = 8;
constexpr int kRankPer = 4;  // entries of a warp

template <typename TOK>
__global__ void __launch_bounds__(32 * kRankWarps)
    token_rank_kernel(const TOK* tokens, int N, int V, uint32_t* key_out, int* pos_out) {
  extern __shared__ __align__(16) uint32_t s_key[];  // [N rounded up to 128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int padded = (N + 127) / 128 * 128;
  pdl_launch_dependents();
  pdl_wait();
  // (loads first: the error word's atomic keeps them from being moved up)
  for (int j0 = threadIdx.x; j0 < padded; j0 += 8 * 32 * kRankWarps) {
    TOK t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u * 32 * kRankWarps;
      t[u] = j < N ? ld_l2(tokens + j) : TOK(0);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u * 32 * kRankWarps;
      if (j < padded) s_key[j] = j < N ? token_key(t[u], V) : 0xFFFFFFFFu;  // before no entry
    }
  }
  __syncthreads();
  const int i0 = (static_cast<int>(blockIdx.x) * kRankWarps + warp) * kRankPer;
  if (i0 >= N) return;
  uint32_t k[kRankPer];
  int count[kRankPer];
#pragma unroll
  for (int e = 0; e < kRankPer; ++e) {
    k[e] = s_key[min(i0 + e, N - 1)];
    count[e] = 0;
  }
  // blocks of 128 keys: all before the warp's entries, the one that holds
  // them (kRankPer divides 128), all after
  const int own = i0 / 128, nb = padded / 128;
  const uint4* keys = reinterpret_cast<const uint4*>(s_key) + lane;
  auto add = [&](int block, uint32_t equal) {
    const uint4 x = keys[block * 32];
#pragma unroll
    for (int e = 0; e < kRankPer; ++e) {
      const uint32_t bound = k[e] + equal;
      count[e] += (x.x < bound) + (x.y < bound) + (x.z < bound) + (x.w < bound);
    }
  };
#pragma unroll 4
  for (int b = 0; b < own; ++b) add(b, 1u);
  {
    const uint4 x = keys[own * 32];
    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int j = own * 128 + lane * 4 + c;
#pragma unroll
      for (int e = 0; e < kRankPer; ++e) count[e] += v[c] < k[e] + (j < i0 + e ? 1u : 0u);
    }
  }
#pragma unroll 4
  for (int b = own + 1; b < nb; ++b) add(b, 0u);
#pragma unroll
  for (int e = 0; e < kRankPer; ++e) {
    const int at = __reduce_add_sync(0xffffffffu, count[e]);
    if (lane == e && i0 + e < N && DPRC_IN(at >= 0 && at < N)) {
      key_out[at] = k[e];
      pos_out[at] = i0 + e;
    }
  }
}

// ---------------------------------------------------------------------------
// The order of more tokens: a stable radix sort, least significant digit
// first: a launch that counts the first digit, then one a digit.
//
// A CTA owns a contiguous tile.  token_count_kernel counts its digits;
// token_scatter_kernel adds up the counts (over digits, then tiles, then the
// tile's warps: the order of a stable sort) and moves the entries: an entry's
// rank among its warp's equal digits is the count so far plus the equal digits
// in lower lanes.  It also counts the next digit by the tiles the entries go to
// (whole numbers: the order of the additions changes nothing; with a counting
// launch a digit 16384 tokens took 11.2 us and not 10.9, 65536 19.8 and not
// 18.8, and the caller's time for the launch; 11.1 and 19.2 with coherent loads,
// launch.cuh).  Keys have as many bits as V (the
// key of "no token") needs, in digits of at most 10 bits.
//
// Launches and not barriers inside one launch: one cluster of 8 CTAs, with the
// hardware's cluster barrier between the steps, took 44 us for 65536 tokens
// (its 8 SMs' scattered stores alone 18 us), these launches 19.2 us.
// ---------------------------------------------------------------------------
constexpr int kSortWarps = 8;
constexpr int kSortThreads = 32 * kSortWarps;
constexpr int kSortBatch = 4;   // entries of a lane that are loaded together
constexpr int kSortMaxBits = 10;
constexpr int kSortTile = kSortThreads * kSortBatch;
constexpr int kSortMaxTiles = 128;

struct SortArgs {
  int N, per;        // entries; of one warp
  int V, shift, bits;
  const int* pos_in;       // null in the first pass
  uint32_t* key_out;
  int* pos_out;
  int* counts;       // [tiles][digits]
  int* next;         // the next digit's, null in the last pass
  int passes;
};

// kSortBatch keys, `step` entries apart from i0 on (0 past hi): all loads
// before the first use.  TOK uint32_t: keys; else tokens.
template <typename TOK>
__device__ __forceinline__ void sort_keys(const TOK* src, int V, int i0, int step, int hi,
                                          uint32_t* k) {
  TOK t[kSortBatch];
#pragma unroll
  for (int j = 0; j < kSortBatch; ++j) t[j] = i0 + j * step < hi ? ld_l2(src + i0 + j * step) : TOK(0);
#pragma unroll
  for (int j = 0; j < kSortBatch; ++j) {
    if constexpr (sizeof(TOK) == 4 && TOK(-1) > TOK(0))
      k[j] = t[j];
    else
      k[j] = token_key(t[j], V);
  }
}

// The lanes with this lane's digit, one vote per bit (the match instruction
// took 2 us a step here: it loops over the distinct values).  Bits above the
// digit are zero in every lane and change nothing.
__device__ __forceinline__ uint32_t equal_lanes(uint32_t digit, bool live) {
  uint32_t same = __ballot_sync(0xffffffffu, live);
#pragma unroll
  for (int bit = 0; bit < kSortMaxBits; ++bit) {
    const uint32_t v = __ballot_sync(0xffffffffu, (digit >> bit) & 1u);
    same &= ~(v ^ (0u - ((digit >> bit) & 1u)));
  }
  return same;
}

template <typename TOK>
__global__ void __launch_bounds__(kSortThreads)
    token_count_kernel(const TOK* src, const SortArgs a) {
  __shared__ int s_hist[1 << kSortMaxBits];
  pdl_launch_dependents();
  const int nd = 1 << a.bits;
  for (int d = threadIdx.x; d < nd; d += kSortThreads) s_hist[d] = 0;
  __syncthreads();
  pdl_wait();
  const int lo = static_cast<int>(blockIdx.x) * kSortWarps * a.per;
  const int hi = min(lo + kSortWarps * a.per, a.N);
  for (int i0 = lo; i0 < hi; i0 += kSortTile) {
    uint32_t k[kSortBatch];
    sort_keys(src, a.V, i0 + static_cast<int>(threadIdx.x), kSortThreads, hi, k);
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j) {
      const int i = i0 + j * kSortThreads + threadIdx.x;
      if (i < hi) atomicAdd(&s_hist[(k[j] >> a.shift) & (nd - 1)], 1);  // whole numbers: any order
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < nd; d += kSortThreads)
    a.counts[blockIdx.x * nd + d] = s_hist[d];
  for (int p = 1; p < a.passes; ++p)  // the other digits' counts start at zero
    for (int d = threadIdx.x; d < nd; d += kSortThreads)
      a.counts[(p * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x)) * nd + d] = 0;
}

template <typename TOK>
__global__ void __launch_bounds__(kSortThreads)
    token_scatter_kernel(const TOK* src, const SortArgs a) {
  extern __shared__ int s_dyn[];
  __shared__ int s_scan[kSortWarps];
  pdl_launch_dependents();
  const int nd = 1 << a.bits;
  int* const s_hist = s_dyn;                     // [warps][digits]
  int* const s_all = s_hist + kSortWarps * nd;   // [digits], all tiles
  int* const s_base = s_all + nd;                // [digits], lower tiles; then the start
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t lt = (1u << lane) - 1u;
  const int lo = min((static_cast<int>(blockIdx.x) * kSortWarps + warp) * a.per, a.N);
  const int hi = min(lo + a.per, a.N);
  int* const hist = s_hist + warp * nd;
  for (int i = threadIdx.x; i < kSortWarps * nd; i += kSortThreads) s_hist[i] = 0;
  __syncthreads();
  pdl_wait();

  // this warp's digits
  for (int i0 = lo; i0 < hi; i0 += 32 * kSortBatch) {
    uint32_t k[kSortBatch];
    sort_keys(src, a.V, i0 + lane, 32, hi, k);
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j)
      if (i0 + j * 32 + lane < hi) atomicAdd(&hist[(k[j] >> a.shift) & (nd - 1)], 1);
  }
  // all tiles' counts of each digit, and the lower tiles' share: two
  // neighbouring digits a thread
  for (int d = 2 * threadIdx.x; d < nd; d += 2 * kSortThreads) {
    int2 total = make_int2(0, 0), before = make_int2(0, 0);
    const int tiles = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
    for (int t0 = 0; t0 < tiles; t0 += 16) {
      int2 v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        v[u] = t0 + u < tiles ? ld_l2(reinterpret_cast<const int2*>(a.counts + (t0 + u) * nd + d))
                              : make_int2(0, 0);
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        total.x += v[u].x;
        total.y += v[u].y;
        before.x += t0 + u < me ? v[u].x : 0;
        before.y += t0 + u < me ? v[u].y : 0;
      }
    }
    s_all[d] = total.x;
    s_all[d + 1] = total.y;
    s_base[d] = before.x;
    s_base[d + 1] = before.y;
  }
  __syncthreads();
  // scan over the digits, dpt neighbours a thread
  const int dpt = (nd + kSortThreads - 1) / kSortThreads;
  const int d0 = threadIdx.x * dpt;
  int total = 0;
  for (int j = 0; j < dpt; ++j) total += d0 + j < nd ? s_all[d0 + j] : 0;
  int incl = total;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int base = incl - total + __reduce_add_sync(0xffffffffu, lane < warp ? s_scan[lane] : 0);
  for (int j = 0; j < dpt && d0 + j < nd; ++j) {
    int run = s_base[d0 + j] + base;
    base += s_all[d0 + j];
    // hist[w][d] becomes where warp w's entries of digit d start
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = s_hist[w * nd + d0 + j];
      s_hist[w * nd + d0 + j] = run;
      run += c;
    }
  }
  __syncthreads();

  for (int i0 = lo; i0 < hi; i0 += 32 * kSortBatch) {
    uint32_t k[kSortBatch];
    int p[kSortBatch];
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j) {
      const int i = i0 + j * 32 + lane;
      p[j] = i < hi && a.pos_in != nullptr ? ld_l2(a.pos_in + i) : i;
    }
    sort_keys(src, a.V, i0 + lane, 32, hi, k);
#pragma unroll
    for (int j = 0; j < kSortBatch; ++j) {
      if (i0 + j * 32 >= hi) break;  // uniform over the warp
      const bool live = i0 + j * 32 + lane < hi;
      const uint32_t digit = live ? (k[j] >> a.shift) & (nd - 1) : 0u;
      const uint32_t same = equal_lanes(digit, live);
      const int at = live ? hist[digit] + __popc(same & lt) : 0;
      __syncwarp();
      if (live && (same & lt) == 0) hist[digit] += __popc(same);
      __syncwarp();
      // (tokens that another stream changes meanwhile would not be where they were counted)
      if (live && DPRC_IN(at >= 0 && at < a.N) && at < a.N) {
        a.key_out[at] = k[j];
        a.pos_out[at] = p[j];
        if (a.next != nullptr)
          atomicAdd(&a.next[at / (kSortWarps * a.per) * nd + ((k[j] >> (a.shift + a.bits)) & (nd - 1))], 1);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The pass over G in sorted order.
//
// A CTA takes kRange = 16 consecutive entries of the order (a range) and up to
// 256 accesses of their rows' columns, one per thread, and adds up rows in fp32
// registers, run by run.  A run of up to 16 entries belongs whole to the CTA
// whose range holds its first entry (which then reads past its range), so most
// results need no second step.  A longer run is cut at the ranges' ends: each
// piece leaves its partial sum in the workspace and embed_long_kernel adds a
// run's pieces in order.  A range holds at most two such pieces: one that
// covers its first entry (slot 0) and one that begins later and reaches past
// its end (slot 1).
//
// The entries' runs come from comparing neighbours in a window of 32 entries
// before the range and 64 after its first entry; bit masks of run starts then
// answer every question about a run's extent.
//
// Rows are read kBatch at a time into registers, all of a batch before one is
// used: with 256 threads of 16 bytes that is 32 KB in flight per CTA and four
// CTAs per SM.  (All 31 rows of a CTA in one unrolled loop took 27 us where
// this takes 17 us on 4 x 4096 tokens of 2048 bf16: its code did not fit
// the instruction cache.)  One warp works out the runs for the CTA.
// ---------------------------------------------------------------------------
constexpr int kRange = 16;
constexpr int kMaxRows = 2 * kRange;   // rows of a CTA, at most 31
constexpr int kSegThreads = 256;
constexpr int kBatch = 8;

struct SegArgs {
  const uint32_t* key;
  const int* pos;
  int N;              // entries
  int T;              // tokens per sample
  unsigned long long t_inv;  // for pos / T
  int V;
  long long d;
  int nblk;           // column blocks
  int nranges;
  float scale;
  // norm: squared sums by original position [N][nblk]; grad: the weights
  float* sq;
  const float* c;     // per-sample factors or null
  int accumulate;
  float* part;        // [nranges][2][dpad] partial sums of long runs
  long long dpad;
  int* long_at;       // [nranges]: bits 0..1: 0, or 1 + slot of the long run that begins here;
                      // bit 2: a long run reaches from here into the next range; bits 4..7:
                      // the entry of the range that the run beginning here begins with
  // grad: rows no token names
  long long zero_units;
  int zero_chunks;    // of kZeroBytes, of a row
};

// Sample of a position: pos / T by a multiplication (Lemire, Kaser and Kurz,
// "Faster remainder by direct computation", 2019: exact for 32-bit operands
// with t_inv = ceil(2^64 / T); T = 1 has t_inv = 0).
__device__ __forceinline__ int sample_of(const SegArgs& a, int pos) {
  return a.t_inv == 0 ? pos
                      : static_cast<int>(__umul64hi(a.t_inv, static_cast<unsigned long long>(pos)));
}

// Position of sorted entry i.  A plan is memory of the caller's: one that is not
// what dprc_embed_plan wrote (read on another stream before it was written, say)
// gives wrong sums, but no access outside the tensors.
__device__ __forceinline__ int plan_pos(const SegArgs& a, long long i) {
  return static_cast<int>(min(static_cast<uint32_t>(ld_l2(a.pos + i)), static_cast<uint32_t>(a.N - 1)));
}

// Rows of a range: lane l holds row l (l < rows).
struct RangeRows {
  uint32_t key;    // its token
  int pos;         // its position
  int rows;
  uint32_t E;      // bit r: row r ends a run or a piece of one
  uint32_t L;      // bit r: row r belongs to a long run
  int slot;        // slot of the piece that starts at row 0 (the others are slot 1)
  uint32_t none;   // bit j: entry j of the range holds no token
};

template <bool kNorm>
__device__ __forceinline__ RangeRows range_rows(const SegArgs& a, int range, bool tell) {
  using u64 = unsigned long long;
  const int lane = threadIdx.x & 31;
  const int a0 = range * kRange;
  const int R = min(a.N - a0, kRange);
  const uint32_t V = static_cast<uint32_t>(a.V);
  // Run starts: S0 bit j = entry a0 - 32 + j, M bit j = entry a0 + j; entries
  // past the last token count as starts (they end the run before them).
  // (kNorm) runs are equal (token, sample) pairs, otherwise equal tokens.  The
  // window's first entry counts as no start: a run from there on is long.
  uint32_t kw[3], st[3], nt[3];
  int pw[3];
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    const int i = a0 - 32 + w * 32 + lane;
    const bool in = i >= 0 && i < a.N;
    kw[w] = in ? min(ld_l2(a.key + i), V) : V;
    pw[w] = in ? plan_pos(a, i) : 0;
  }
  uint32_t klast = kw[0];
  int slast = 0;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    const int i = a0 - 32 + w * 32 + lane;
    const int smp = kNorm ? sample_of(a, pw[w]) : 0;
    uint32_t kp = __shfl_up_sync(0xffffffffu, kw[w], 1);
    int sp = kNorm ? __shfl_up_sync(0xffffffffu, smp, 1) : 0;
    if (lane == 0) {
      kp = w == 0 ? kw[0] : klast;
      sp = w == 0 ? smp : slast;
    }
    klast = __shfl_sync(0xffffffffu, kw[w], 31);
    if (kNorm) slast = __shfl_sync(0xffffffffu, smp, 31);
    const bool none = kw[w] >= V;
    st[w] = __ballot_sync(0xffffffffu,
                          i >= 0 && (none || i == 0 || kp != kw[w] || (kNorm && sp != smp)));
    nt[w] = __ballot_sync(0xffffffffu, none);
  }
  const uint32_t S0 = st[0];
  const u64 M = st[1] | static_cast<u64>(st[2]) << 32;
  const uint32_t inside = (1u << R) - 1u;
  RangeRows q;
  q.none = nt[1] & inside;
  // entries of the range that hold a token come first
  const int Rt = q.none == 0 ? R : __ffs(static_cast<int>(q.none)) - 1;

  // Rows [first, last) of the window are this CTA's.  A row ends a run where
  // the next entry starts one, or where a long run is cut; rows below head or
  // from tail on belong to long runs.
  int first = 0, last = 0, head = 0, tail = 32;
  u64 E = M >> 1;
  int flags = 0;
  if (Rt > 0 && (M & 1) == 0) {
    // the range begins inside a run
    const int e = M == 0 ? 64 : __ffsll(static_cast<long long>(M)) - 1;
    const int before = S0 == 0 ? 64 : 32 - (31 - __clz(S0));
    if (before + e > kRange) {
      head = last = min(e, R);
      if (e > R) flags |= 4;
      E |= 1ull << (head - 1);
    } else {
      first = last = e;
    }
  }
  const uint32_t S = st[1] & ((1u << Rt) - 1u);  // starts in the range
  if (S != 0) {
    const int o = 31 - __clz(S);  // only the last run can leave the range
    const u64 rest = M >> (o + 1);
    const int len = rest == 0 ? 64 : __ffsll(static_cast<long long>(rest));
    if (len > kRange) {
      flags |= 4 | (o == 0 ? 1 : 2) | o << 4;
      tail = o;
      last = R;
      E |= 1ull << (R - 1);
    } else {
      last = o + len;
    }
  }
  if (tell && lane == 0 && DPRC_IN(range < a.nranges)) a.long_at[range] = flags;
  q.rows = last - first;  // <= 31
  q.E = static_cast<uint32_t>(E >> first) & ((1u << q.rows) - 1u);
  const uint32_t hm = (1u << head) - 1u, tm = tail >= 32 ? 0u : ~((1u << tail) - 1u);
  q.L = (hm | tm) >> first;  // first > 0 only where head is 0
  q.slot = first == 0 ? 0 : 1;
  const int o = first + lane;
  const uint32_t k1 = __shfl_sync(0xffffffffu, kw[1], o & 31);
  const uint32_t k2 = __shfl_sync(0xffffffffu, kw[2], o & 31);
  const int p1 = __shfl_sync(0xffffffffu, pw[1], o & 31);
  const int p2 = __shfl_sync(0xffffffffu, pw[2], o & 31);
  q.key = o < 32 ? k1 : k2;
  q.pos = o < 32 ? p1 : p2;
  return q;
}

// What a CTA knows of its range.
struct RangeShared {
  int pos[kMaxRows];
  uint32_t key[kMaxRows];
  float w[kMaxRows];               // grad: the row's factor
  float q[kSegThreads / 32][kMaxRows];  // norm: each warp's part of a row's square
  uint32_t E, L, none;
  int rows, slot;
};

template <typename T, int AW, bool kNorm>
__device__ __forceinline__ void segment_range(const SegArgs& a, const T* G, T* dW, int range,
                                              int blk, RangeShared& s) {
  using RawT = typename Raw<AW>::type;
  constexpr int VE = AW / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    const RangeRows q = range_rows<kNorm>(a, range, blk == 0);
    s.pos[lane] = q.pos;
    s.key[lane] = q.key;
    if (!kNorm && a.c != nullptr && lane < q.rows) s.w[lane] = ld_l2(a.c + sample_of(a, q.pos));
    if (lane == 0) {
      s.E = q.E;
      s.L = q.L;
      s.none = q.none;
      s.rows = q.rows;
      s.slot = q.slot;
    }
  }
  __syncthreads();
  const int rows = s.rows;
  const uint32_t E = s.E, L = s.L;

  const int nvec = static_cast<int>(a.d / VE);
  const int v = blk * kSegThreads + threadIdx.x;  // this thread's access of a row
  const bool mine = v < nvec;
  const RawT* const col = reinterpret_cast<const RawT*>(G) + (mine ? v : 0);
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.f;

#pragma unroll 1
  for (int base = 0; base < rows; base += kBatch) {
    RawT raw[kBatch];
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      raw[r] = RawT{};
      if (base + r < rows && DPRC_IN(s.pos[base + r] >= 0 && s.pos[base + r] < a.N))
        raw[r] = ld_stream(col + static_cast<long long>(s.pos[base + r]) * nvec);
    }
    // bits of the batch's rows: ends of runs, ends of long runs' pieces, starts
    const uint32_t Eb = E >> base, Pb = (E & L) >> base;
    const uint32_t Bb = base == 0 ? (E << 1) | 1u : E >> (base - 1);
    float sum[kNorm ? kBatch : 1];
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      // A run's first row takes the sums from zero: a mask and not a branch,
      // which would cost more than the eight additions (rows past the last are
      // zero and end no run)
      float f[VE];
      unpack<T, AW>(raw[r], f);
      const uint32_t keep = ((Bb >> r) & 1u) - 1u;
      const float w = !kNorm && a.c != nullptr ? s.w[(base + r) & (kMaxRows - 1)] : 1.f;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float old = __uint_as_float(__float_as_uint(acc[e]) & keep);
        acc[e] = kNorm ? old + f[e] : fmaf(w, f[e], old);
      }
      if (kNorm) {
        const float q = square_sum<VE>(acc);
        sum[r] = mine && ((Eb >> r) & 1u) ? q : 0.f;
      }
      if (kNorm ? (Pb >> r) & 1u : (Eb >> r) & 1u) {
        if ((Pb >> r) & 1u) {
          // a piece of a long run: the one over the range's first entry is slot 0
          const int slot = s.slot == 0 && (E & ((1u << (base + r)) - 1u)) == 0 ? 0 : 1;
          float* out = a.part + (static_cast<long long>(range) * 2 + slot) * a.dpad +
                       static_cast<long long>(v) * VE;
          if (mine) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
              if (DPRC_IN(static_cast<long long>(v) * VE + e < a.dpad)) out[e] = acc[e];
          }
          if (kNorm) sum[r] = 0.f;
        } else if (!kNorm) {
          const uint32_t k = s.key[base + r];
          RawT* out = reinterpret_cast<RawT*>(dW) + static_cast<long long>(k) * nvec + v;
          if (mine && DPRC_IN(k < static_cast<uint32_t>(a.V))) {
            if (a.accumulate) {
              unpack<T, AW>(*out, f);
#pragma unroll
              for (int e = 0; e < VE; ++e) f[e] = fmaf(a.scale, acc[e], f[e]);
            } else {
#pragma unroll
              for (int e = 0; e < VE; ++e) f[e] = a.scale * acc[e];
            }
            __stcs(out, pack<T, AW>(f));
          }
        }
      }
    }
    if constexpr (kNorm) {
      // the batch's squares over the warp's lanes, all at once: lanes h apart
      // share the rows out between them, which leaves lane l with row l >> 2
#pragma unroll
      for (int h = 16, n = kBatch / 2; n > 0; h >>= 1, n >>= 1) {
        const bool up = (lane & h) != 0;
#pragma unroll
        for (int r = 0; r < n; ++r) {
          const float give = up ? sum[r] : sum[r + n];
          const float keep = up ? sum[r + n] : sum[r];
          sum[r] = keep + __shfl_xor_sync(0xffffffffu, give, h);
        }
      }
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
      if ((lane & 3) == 0) s.q[warp][base + (lane >> 2)] = sum[0];
    }
  }

  if constexpr (kNorm) {
    __syncthreads();
    if (warp == 0) {
      // every entry is written once: by the CTA that took its row (a run's
      // square stands at its last row, zero at the others), or here if it
      // holds no token
      float t = 0.f;
      const int nw = blockDim.x >> 5;
      if (lane < rows) {
        for (int w = 0; w < nw; ++w) t += s.q[w][lane];
        const int p = s.pos[lane];
        if (DPRC_IN(p >= 0 && p < a.N)) a.sq[static_cast<long long>(p) * a.nblk + blk] = t;
      }
      if ((s.none >> lane) & 1u)
        a.sq[static_cast<long long>(plan_pos(a, range * kRange + lane)) * a.nblk + blk] = 0.f;
    }
  }
}

// First entry >= v in the sorted keys.
__device__ __forceinline__ long long lower_bound(const uint32_t* key, long long N, uint32_t v) {
  long long lo = 0, hi = N;
  while (lo < hi) {
    const long long m = (lo + hi) >> 1;
    if (key[m] < v) lo = m + 1; else hi = m;
  }
  return lo;
}

// Rows of dW that no token names are zero: kZeroBytes of 32 rows per warp, one
// search per lane.  (Whole rows per warp left too few warps where rows are long:
// gradients of 8361 rows of 6688 bf16 54 us and not 26, 51463 of 5216 173 and
// not 102.)
constexpr int kZeroBytes = 4096;
template <typename T, int AW>
__device__ __forceinline__ void zero_rows(const SegArgs& a, T* dW, long long unit) {
  using RawT = typename Raw<AW>::type;
  constexpr int VE = AW / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31;
  const long long v0 = unit / a.zero_chunks * 32, v = v0 + lane;
  const int chunk = static_cast<int>(unit % a.zero_chunks);
  bool absent = false;
  if (v < a.V) {
    const long long i = lower_bound(a.key, a.N, static_cast<uint32_t>(v));
    absent = i >= a.N || a.key[i] != static_cast<uint32_t>(v);
  }
  uint32_t todo = __ballot_sync(0xffffffffu, absent);
  const long long nvec = a.d / VE;
  float z[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) z[e] = 0.f;
  const RawT zero = pack<T, AW>(z);
  while (todo != 0) {
    const int j = __ffs(static_cast<int>(todo)) - 1;
    todo &= todo - 1;
    RawT* row = reinterpret_cast<RawT*>(dW + (v0 + j) * a.d);
    const long long x0 = static_cast<long long>(chunk) * (kZeroBytes / AW);
    const long long x1 = x0 + kZeroBytes / AW < nvec ? x0 + kZeroBytes / AW : nvec;
    for (long long x = x0 + lane; x < x1; x += 32)
      if (DPRC_IN(v0 + j < a.V)) __stcs(row + x, zero);
  }
}

template <typename T, int AW, bool kNorm>
__global__ void __launch_bounds__(kSegThreads, 4)
    embed_segment_kernel(const SegArgs a, const T* G, T* dW) {
  __shared__ RangeShared s_range;
  pdl_launch_dependents();
  pdl_wait();
  const long long units = static_cast<long long>(a.nranges) * a.nblk;
  if (blockIdx.x < units) {
    const int range = static_cast<int>(blockIdx.x / a.nblk);
    segment_range<T, AW, kNorm>(a, G, dW, range, static_cast<int>(blockIdx.x) - range * a.nblk,
                                s_range);
  } else if (!kNorm) {
    const long long u = (blockIdx.x - units) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (u < a.zero_units) zero_rows<T, AW>(a, dW, u);
  }
}

// ---------------------------------------------------------------------------
// Long runs: the pieces of a run added in order.  A CTA looks at kLongRanges
// ranges (blockIdx.x) and one block of kLongCols columns (blockIdx.y).  Its
// warps deal the long runs that begin there among them; runs of more than
// kLongAlone pieces are shared by all: the warps take contiguous shares of the
// pieces, and the shares are added in warp order.  Where a run ends is read off
// the ranges' flags, 32 at a time.
// ---------------------------------------------------------------------------
constexpr int kLongWarps = 8;
constexpr int kLongRanges = 32;
constexpr int kLongCols = 128;  // 4 per lane
constexpr int kLongAlone = 16;

// Pieces [p0, p1) of the run that begins in `range`, added.
__device__ __forceinline__ float4 add_pieces(const SegArgs& a, long long range, int slot,
                                             long long p0, long long p1, long long col) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (long long p = p0; p < p1; ++p) {
    const long long row = (range + p) * 2 + (p == 0 ? slot : 0);
    if (DPRC_IN(range + p < a.nranges && col + 3 < a.dpad)) {
      const float4 v = ld_l2(reinterpret_cast<const float4*>(a.part + row * a.dpad + col));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  return s;
}

// What becomes of a long run's sums over one block of columns (a warp's).
template <typename T, bool kNorm>
__device__ __forceinline__ void finish_run(const SegArgs& a, T* dW, long long range, int first,
                                           long long col, float4 s) {
  const float f[4] = {s.x, s.y, s.z, s.w};
  if (kNorm) {
    // columns past d hold whatever the workspace held
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < a.d) q = fmaf(f[e], f[e], q);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
    // The run's rows hold zeros in a.sq.  It has at least kRange + 1 of them, and
    // there are at most kRange times as many of these column blocks as of
    // a.sq's, so each block's square gets a place of its own among the first.
    if ((threadIdx.x & 31) == 0) {
      const int at = static_cast<int>(range) * kRange + first + static_cast<int>(blockIdx.y) % kRange;
      const int blk = static_cast<int>(blockIdx.y) / kRange;
      if (DPRC_IN(at < a.N && blk < a.nblk))
        a.sq[static_cast<long long>(plan_pos(a, min(at, a.N - 1))) * a.nblk + blk] = q;
    }
  } else {
    // (the run reaches past `range`)
    const uint32_t k = min(ld_l2(a.key + (range + 1) * kRange - 1), static_cast<uint32_t>(a.V - 1));
    T* out = dW + static_cast<long long>(k) * a.d;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (col + e < a.d && DPRC_IN(k < static_cast<uint32_t>(a.V))) {
        const float prev = a.accumulate ? to_f32<T>(out[col + e]) : 0.f;
        const float v = fmaf(a.scale, f[e], prev);
        if constexpr (sizeof(T) == 4)
          out[col + e] = v;
        else
          out[col + e] = __float2bfloat16_rn(v);
      }
    }
  }
}

template <typename T, bool kNorm>
__global__ void __launch_bounds__(32 * kLongWarps)
    embed_long_kernel(const SegArgs a, T* dW) {
  __shared__ float4 s_sum[kLongWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rbase = static_cast<long long>(blockIdx.x) * kLongRanges;
  const long long col = static_cast<long long>(blockIdx.y) * kLongCols + lane * 4;  // < dpad
  const int f0 = rbase + lane < a.nranges ? a.long_at[rbase + lane] : 0;
  uint32_t todo = __ballot_sync(0xffffffffu, (f0 & 3) != 0);
  // a run ends in the first range after its own from which no long run reaches
  // on, or in which another begins
  const uint32_t stop0 = __ballot_sync(0xffffffffu, (f0 & 4) == 0 || (f0 & 3) == 2);
  for (int turn = 0; todo != 0; todo &= todo - 1, ++turn) {
    const int j = __ffs(static_cast<int>(todo)) - 1;
    const int fj = __shfl_sync(0xffffffffu, f0, j);
    const int slot = (fj & 3) - 1, first = fj >> 4;
    const long long range = rbase + j;
    long long end = rbase + 32;
    const uint32_t here = j == 31 ? 0u : stop0 & ~((2u << j) - 1u);
    if (here != 0) {
      end = rbase + __ffs(static_cast<int>(here)) - 1;
    } else {
      while (true) {
        const int f = end + lane < a.nranges ? a.long_at[end + lane] : 0;
        const uint32_t stop = __ballot_sync(0xffffffffu, (f & 4) == 0 || (f & 3) == 2);
        if (stop != 0) {
          end += __ffs(static_cast<int>(stop)) - 1;
          break;
        }
        end += 32;
      }
    }
    const long long pieces = end - range + 1;
    if (pieces <= kLongAlone) {
      if (turn % kLongWarps == warp)
        finish_run<T, kNorm>(a, dW, range, first, col, add_pieces(a, range, slot, 0, pieces, col));
    } else {  // the same for every warp
      const long long share = (pieces + kLongWarps - 1) / kLongWarps;
      const long long p0 = warp * share;
      s_sum[warp][lane] = add_pieces(a, range, slot, p0, min(p0 + share, pieces), col);
      __syncthreads();
      if (turn % kLongWarps == warp) {
        float4 s = s_sum[0][lane];
        for (int w = 1; w < kLongWarps; ++w) {
          const float4 v = s_sum[w][lane];
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
        finish_run<T, kNorm>(a, dW, range, first, col, s);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// n_i (+)= s^2 (sum of sample i's squares), its positions' squares of every
// column block in a fixed order.  A sample's sum is split over the CTAs of a
// cluster, which add their parts in rank order.  Rank 0's shared memory takes the
// parts, so no CTA stores its own before every CTA has started: each arrives at the
// cluster's barrier first and waits for it after its loads, which hide it.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    embed_norm_finish_kernel(const SegArgs a, float* n) {
  __shared__ float s_warp[8];
  __shared__ float s_cta[8];
  cluster_arrive();
  pdl_wait();
  const uint32_t rank = cluster_ctarank(), cl = cluster_nctarank();
  const long long i = blockIdx.x / cl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = static_cast<int>(rank) * 256 + threadIdx.x, step = static_cast<int>(cl) * 256;
  float s = 0.f;
  const long long count = static_cast<long long>(a.T) * a.nblk;
  const float* sq = a.sq + i * count;
#pragma unroll 8
  for (long long t = t0; t < count; t += step) s += ld_l2(sq + t);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) s_warp[warp] = s;
  __syncthreads();
  cluster_wait();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int w = 0; w < 8; ++w) t += s_warp[w];
    if (cl == 1)
      s_cta[0] = t;
    else
      st_cluster_f32(map_to_rank(&s_cta[rank], 0), t);
  }
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) {
    float t = 0.f;
    for (uint32_t r = 0; r < cl; ++r) t += s_cta[r];
    t *= a.scale * a.scale;
    n[i] = a.accumulate ? n[i] + t : t;
  }
}

__global__ void embed_norm_zero_kernel(float* n, long long B) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < B) n[i] = 0.f;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The widest access that divides a row's pitch (the bases are 16-byte aligned).
int access_bytes(int64_t d, int elem) {
  const int64_t row = d * elem;
  return row % 16 == 0 ? 16 : row % 8 == 0 ? 8 : row % 4 == 0 ? 4 : 2;
}

struct SegPlan {
  int aw = 16, nblk = 1, threads = 32, ncb = 1;
  int64_t nranges = 0, dpad = 0;
  size_t part_off = 0, long_off = 0, sq_off = 0, total = 0;
};

SegPlan seg_plan(dprc_dtype dt, int64_t N, int64_t d, bool norm) {
  SegPlan s;
  const int elem = dt == DPRC_F32 ? 4 : 2;
  s.aw = access_bytes(d, elem);
  const int64_t nvec = d * elem / s.aw;
  s.nblk = static_cast<int>((nvec + kSegThreads - 1) / kSegThreads);
  s.threads = nvec >= kSegThreads ? kSegThreads : static_cast<int>((nvec + 31) / 32 * 32);
  s.nranges = (N + kRange - 1) / kRange;
  s.dpad = (d + kLongCols - 1) / kLongCols * kLongCols;
  s.ncb = static_cast<int>(s.dpad / kLongCols);
  size_t off = 0;
  s.long_off = off;
  off = up256(off + static_cast<size_t>(s.nranges) * 4);
  s.part_off = off;
  off = up256(off + static_cast<size_t>(s.nranges) * 2 * s.dpad * 4);
  if (norm) {
    s.sq_off = off;
    off = up256(off + static_cast<size_t>(s.nblk) * N * 4);
  }
  s.total = off > 0 ? off : 256;
  return s;
}

// The plan: sorted keys and positions at the front; behind them, where the
// radix sort runs, its second buffers and counts.
struct SortPlan {
  int passes = 0, bits = 0, tiles = 0;  // passes 0: by ranks
  int64_t per = 0;
  size_t key_off[2] = {0, 0}, pos_off[2] = {0, 0}, count_off = 0, total = 0;
};

SortPlan sort_plan(int64_t N, int64_t V) {
  SortPlan s;
  size_t off = 0;
  for (int b = 0; b < (N > kRankMax ? 2 : 1); ++b) {
    s.key_off[b] = off;
    off = up256(off + static_cast<size_t>(N) * 4);
    s.pos_off[b] = off;
    off = up256(off + static_cast<size_t>(N) * 4);
  }
  if (N > kRankMax) {
    int bits = 1;
    while ((int64_t(1) << bits) <= V) ++bits;  // keys 0..V
    s.passes = (bits + kSortMaxBits - 1) / kSortMaxBits;
    s.bits = (bits + s.passes - 1) / s.passes;
    const int64_t tiles = std::min<int64_t>((N + kSortTile - 1) / kSortTile, kSortMaxTiles);
    s.per = ((N + tiles * kSortWarps - 1) / (tiles * kSortWarps) + 31) / 32 * 32;
    s.tiles = static_cast<int>((N + s.per * kSortWarps - 1) / (s.per * kSortWarps));
    s.count_off = off;
    off = up256(off + (static_cast<size_t>(s.tiles * s.passes) << s.bits) * 4);
  }
  s.total = off > 0 ? off : 256;
  return s;
}

SegArgs seg_args(const EmbedCall& c, const SegPlan& p, const SortPlan& sp, char* ws) {
  SegArgs a;
  const char* plan = static_cast<const char*>(c.plan);
  a.key = reinterpret_cast<const uint32_t*>(plan + sp.key_off[0]);
  a.pos = reinterpret_cast<const int*>(plan + sp.pos_off[0]);
  a.N = static_cast<int>(c.B * c.T);
  a.T = static_cast<int>(c.T > 0 ? c.T : 1);
  a.t_inv = a.T == 1 ? 0 : ~0ull / static_cast<unsigned>(a.T) + 1;
  a.V = static_cast<int>(c.V);
  a.d = c.d;
  a.nblk = p.nblk;
  a.nranges = static_cast<int>(p.nranges);
  a.scale = c.scale;
  a.sq = reinterpret_cast<float*>(ws + p.sq_off);
  a.c = nullptr;
  a.accumulate = c.accumulate;
  a.part = reinterpret_cast<float*>(ws + p.part_off);
  a.dpad = p.dpad;
  a.long_at = reinterpret_cast<int*>(ws + p.long_off);
  a.zero_units = 0;
  a.zero_chunks = 1;
  return a;
}

template <typename T, int AW, bool kNorm>
cudaError_t launch_segments_t(const SegArgs& a, const SegPlan& p, const void* G, void* dW,
                              cudaStream_t s) {
  const long long zero_ctas = (a.zero_units * 32 + p.threads - 1) / p.threads;
  const long long ctas = static_cast<long long>(a.nranges) * a.nblk + zero_ctas;
  if (ctas > 0) {
    const cudaError_t e =
        launch_after(embed_segment_kernel<T, AW, kNorm>, dim3(static_cast<unsigned>(ctas)),
                     p.threads, 1, s, 0, a, static_cast<const T*>(G), static_cast<T*>(dW));
    if (e != cudaSuccess) return e;
  }
  if (a.N > kRange) {
    const dim3 grid(static_cast<unsigned>((a.nranges + kLongRanges - 1) / kLongRanges),
                    static_cast<unsigned>(p.ncb));
    return launch_after(embed_long_kernel<T, kNorm>, grid, 32 * kLongWarps, 1, s, 0, a,
                        static_cast<T*>(dW));
  }
  return cudaSuccess;
}

template <bool kNorm>
cudaError_t launch_segments(dprc_dtype dt, const SegArgs& a, const SegPlan& p, const void* G,
                            void* dW, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (dt == DPRC_F32) {
    switch (p.aw) {
      case 16: return launch_segments_t<float, 16, kNorm>(a, p, G, dW, s);
      case 8: return launch_segments_t<float, 8, kNorm>(a, p, G, dW, s);
      default: return launch_segments_t<float, 4, kNorm>(a, p, G, dW, s);
    }
  }
  switch (p.aw) {
    case 16: return launch_segments_t<bf16, 16, kNorm>(a, p, G, dW, s);
    case 8: return launch_segments_t<bf16, 8, kNorm>(a, p, G, dW, s);
    case 4: return launch_segments_t<bf16, 4, kNorm>(a, p, G, dW, s);
    default: return launch_segments_t<bf16, 2, kNorm>(a, p, G, dW, s);
  }
}

template <typename T, int AW, typename TOK>
cudaError_t launch_lookup_t(const void* W, const void* tokens, int64_t N, int64_t V, int64_t d,
                            float scale, void* out, cudaStream_t s) {
  const int64_t nvec = d * static_cast<int64_t>(sizeof(T)) / AW;
  int lanes = 1;
  while (lanes < 32 && lanes < nvec) lanes *= 2;
  const int64_t upr = (nvec + lanes * kLookupUnroll - 1) / (lanes * kLookupUnroll);
  const int64_t threads = N * upr * lanes;
  int64_t ctas = (threads + 255) / 256;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 64;
  if (ctas > cap) ctas = cap;
  return launch_after(embed_lookup_kernel<T, AW, TOK>, dim3(static_cast<unsigned>(ctas)), 256, 1, s,
                      0, static_cast<const T*>(W), static_cast<const TOK*>(tokens),
                      static_cast<long long>(N), static_cast<int>(V), static_cast<long long>(d),
                      scale, static_cast<T*>(out), lanes, static_cast<int>(upr));
}

template <typename TOK>
cudaError_t launch_plan_t(const TOK* tokens, int64_t N, int64_t V, char* plan, cudaStream_t s) {
  const SortPlan sp = sort_plan(N, V);
  uint32_t* key[2];
  int* pos[2];
  for (int b = 0; b < 2; ++b) {
    key[b] = reinterpret_cast<uint32_t*>(plan + sp.key_off[b]);
    pos[b] = reinterpret_cast<int*>(plan + sp.pos_off[b]);
  }
  if (sp.passes == 0) {
    const int64_t warps = (N + kRankPer - 1) / kRankPer;
    const unsigned ctas = static_cast<unsigned>((warps + kRankWarps - 1) / kRankWarps);
    const size_t smem = static_cast<size_t>((N + 127) / 128 * 128) * 4;  // at most 32 KB
    return launch_after(token_rank_kernel<TOK>, dim3(ctas), 32 * kRankWarps, 1, s, smem, tokens,
                        static_cast<int>(N), static_cast<int>(V), key[0], pos[0]);
  }
  SortArgs a;
  a.N = static_cast<int>(N);
  a.per = static_cast<int>(sp.per);
  a.V = static_cast<int>(V);
  a.bits = sp.bits;
  a.counts = reinterpret_cast<int*>(plan + sp.count_off);
  a.passes = sp.passes;
  const size_t smem = static_cast<size_t>(kSortWarps + 2) * (size_t(1) << sp.bits) * 4;  // <= 40 KB
  for (int p = 0; p < sp.passes; ++p) {
    const int dst = (sp.passes - 1 - p) & 1;  // the last pass writes buffer 0
    a.shift = p * sp.bits;
    a.pos_in = p == 0 ? nullptr : pos[dst ^ 1];
    a.key_out = key[dst];
    a.pos_out = pos[dst];
    a.next = p + 1 < sp.passes ? a.counts + (static_cast<int64_t>(sp.tiles) << sp.bits) : nullptr;
    const dim3 grid(sp.tiles);
    const uint32_t* in = key[dst ^ 1];
    cudaError_t e = cudaSuccess;
    if (p == 0) e = launch_after(token_count_kernel<TOK>, grid, kSortThreads, 1, s, 0, tokens, a);
    if (e != cudaSuccess) return e;
    e = p == 0
            ? launch_after(token_scatter_kernel<TOK>, grid, kSortThreads, 1, s, smem, tokens, a)
            : launch_after(token_scatter_kernel<uint32_t>, grid, kSortThreads, 1, s, smem, in, a);
    if (e != cudaSuccess) return e;
    a.counts = a.next;
  }
  return cudaSuccess;
}

template <typename TOK>
cudaError_t launch_lookup_tok(const void* W, dprc_dtype dt, const void* tokens, int64_t N,
                              int64_t V, int64_t d, float scale, void* out, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  const int aw = access_bytes(d, dt == DPRC_F32 ? 4 : 2);
  if (dt == DPRC_F32) {
    switch (aw) {
      case 16: return launch_lookup_t<float, 16, TOK>(W, tokens, N, V, d, scale, out, s);
      case 8: return launch_lookup_t<float, 8, TOK>(W, tokens, N, V, d, scale, out, s);
      default: return launch_lookup_t<float, 4, TOK>(W, tokens, N, V, d, scale, out, s);
    }
  }
  switch (aw) {
    case 16: return launch_lookup_t<bf16, 16, TOK>(W, tokens, N, V, d, scale, out, s);
    case 8: return launch_lookup_t<bf16, 8, TOK>(W, tokens, N, V, d, scale, out, s);
    case 4: return launch_lookup_t<bf16, 4, TOK>(W, tokens, N, V, d, scale, out, s);
    default: return launch_lookup_t<bf16, 2, TOK>(W, tokens, N, V, d, scale, out, s);
  }
}

}  // namespace

cudaError_t read_device_error_embed(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

size_t embed_plan_bytes(int64_t N, int64_t V) { return sort_plan(N, V).total; }

size_t embed_norm_ws_bytes(dprc_dtype dt, int64_t N, int64_t d) {
  return seg_plan(dt, N, d, true).total;
}

cudaError_t launch_embed_lookup(const void* W, dprc_dtype dt, const void* tokens,
                                int token_bytes, int64_t N, int64_t V, int64_t d, float scale,
                                void* out, cudaStream_t s) {
  if (N == 0) return cudaSuccess;
  return token_bytes == 4
             ? launch_lookup_tok<int32_t>(W, dt, tokens, N, V, d, scale, out, s)
             : launch_lookup_tok<long long>(W, dt, tokens, N, V, d, scale, out, s);
}

cudaError_t launch_embed_plan(const void* tokens, int token_bytes, int64_t N, int64_t V,
                              void* plan, cudaStream_t s) {
  if (N == 0) return cudaSuccess;
  char* p = static_cast<char*>(plan);
  return token_bytes == 4 ? launch_plan_t(static_cast<const int32_t*>(tokens), N, V, p, s)
                          : launch_plan_t(static_cast<const long long*>(tokens), N, V, p, s);
}

cudaError_t launch_embed_norm(const EmbedCall& c, float* n, void* ws, cudaStream_t s) {
  if (c.B * c.T == 0) {
    if (c.accumulate) return cudaSuccess;
    embed_norm_zero_kernel<<<static_cast<unsigned>((c.B + 255) / 256), 256, 0, s>>>(n, c.B);
    return cudaGetLastError();
  }
  const SegPlan p = seg_plan(c.dtype, c.B * c.T, c.d, true);
  const SegArgs a = seg_args(c, p, sort_plan(c.B * c.T, c.V), static_cast<char*>(ws));
  cudaError_t e = launch_segments<true>(c.dtype, a, p, c.G, nullptr, s);
  if (e != cudaSuccess) return e;
  // One CTA per sample where a sample has at most two values a thread, else a
  // cluster of 8: whole norms of 4 x 4096 tokens of 2048 bf16 24.2 and 20.9 us, of
  // 3 x 1000 of 321 fp32 13.3 and 11.4; of 4 x 128 of 64 fp32 5.6 with one CTA.
  const int cl = static_cast<int64_t>(a.T) * p.nblk > 512 ? 8 : 1;
  return launch_after(embed_norm_finish_kernel, dim3(static_cast<unsigned>(c.B * cl)), 256, cl, s,
                      0, a, n);
}

cudaError_t launch_embed_grad(const EmbedCall& c, const float* clip, void* dW, void* ws,
                              cudaStream_t s) {
  const SegPlan p = seg_plan(c.dtype, c.B * c.T, c.d, false);
  SegArgs a = seg_args(c, p, sort_plan(c.B * c.T, c.V), static_cast<char*>(ws));
  a.c = clip;
  a.zero_chunks = static_cast<int>(
      (c.d * (c.dtype == DPRC_F32 ? 4 : 2) + kZeroBytes - 1) / kZeroBytes);
  a.zero_units = c.accumulate ? 0 : (c.V + 31) / 32 * a.zero_chunks;
  return launch_segments<false>(c.dtype, a, p, c.G, dW, s);
}

}  // namespace dprc
