// The embedding of a DP-SGD-RC step: lookup, the sorted token order that its
// gradient is taken in, the exact per-sample squared norm of that gradient and
// the clipped gradient itself.
//
// The weight W [V][d] of an embedding gets, from sample i, the gradient
//   dW_i[v] = s * sum over t with tok_it = v of G_it      (G the gradient of the output)
// so  ||dW_i||^2 = s^2 sum_v || sum_{t: tok_it = v} G_it ||^2   and
//     sum_i c_i dW_i[v] = s sum_i c_i sum_{t: tok_it = v} G_it.
// Both are sums over groups of equal tokens.  The tokens are sorted once,
// stably, with their positions (token_sort_kernel); a group is then a run of
// consecutive entries, a token's entries of one sample are a run inside it,
// and one pass over the rows of G in that order gives either result with no
// atomics: every sum has one fixed order, so results repeat bitwise.
//
// What bounds them: bytes.  The lookup writes N d values, the norm reads them
// once, the gradient reads them once and writes all V rows.

#include "common.cuh"
#include "internal.h"

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
// ---------------------------------------------------------------------------
constexpr int kLookupUnroll = 4;

template <typename T, int AW, typename TOK>
__global__ void __launch_bounds__(256)
    embed_lookup_kernel(const T* __restrict__ W, const TOK* __restrict__ tokens, long long N,
                        int V, long long d, float scale, T* __restrict__ out, int lanes,
                        int units_per_row) {
  using R = typename Raw<AW>::type;
  constexpr int VE = AW / static_cast<int>(sizeof(T));
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
      if (have && v < nvec) raw[j] = __ldg(src + v);
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
// Stable radix sort of (token, position), one launch of one cluster.
//
// Keys have `bits` bits (tokens and the key V of "no token"), taken in
// `passes` digits of `dbits` <= 10 bits, least significant first.  Every warp
// of the cluster owns a contiguous range of the input; per pass it counts its
// digits in shared memory, the counts become start offsets (over digits, then
// CTAs, then warps: the order of a stable sort), and it writes its range out
// 32 entries at a time, each rank being the number of equal digits in lower
// lanes.  The passes are separated by the cluster's hardware barrier, so
// nothing spins, and the data goes through L2, so any N fits.
//
// One cluster of 8 CTAs and not the whole GPU: a grid-wide barrier needs a
// cooperative launch and spinning, and the sort moves 16 bytes per token and
// pass against the 2 d or 4 d bytes per token of the pass over G.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxDigit = 1024;
constexpr int kSortBatch = 8;  // entries a lane loads ahead

struct SortArgs {
  long long N;
  int V, passes, dbits;
  uint32_t* key[2];  // [0] holds the result
  int* pos[2];
  int* ghist;        // [CTAs][digits], per-CTA digit counts of the current pass
};

template <typename TOK>
__global__ void __launch_bounds__(kSortThreads, 1)
    token_sort_kernel(const TOK* __restrict__ tokens, const SortArgs a) {
  extern __shared__ int s_hist[];  // [kSortWarps][digits]
  __shared__ int s_scan[kSortWarps];
  const int nd = 1 << a.dbits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const long long per =
      ((a.N + static_cast<long long>(ctas) * kSortWarps - 1) / (ctas * kSortWarps) + 31) / 32 * 32;
  const long long lo = (static_cast<long long>(cta) * kSortWarps + warp) * per;
  const long long hi = lo + per < a.N ? lo + per : a.N;
  int* hist = s_hist + warp * nd;
  const uint32_t lt = (1u << lane) - 1u;

  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.dbits;
    // the last pass writes buffer 0; before it they alternate
    const int dst = (a.passes - 1 - p) & 1, src = dst ^ 1;
    for (int i = threadIdx.x; i < kSortWarps * nd; i += kSortThreads) s_hist[i] = 0;
    __syncthreads();

    for (long long b0 = lo; b0 < hi; b0 += 32 * kSortBatch) {
      uint32_t key[kSortBatch];
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j) {
        const long long i = b0 + j * 32 + lane;
        if (i < hi) key[j] = p == 0 ? token_key(tokens[i], a.V) : __ldcg(a.key[src] + i);
      }
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j) {
        const bool live = b0 + j * 32 + lane < hi;
        const uint32_t dg = live ? (key[j] >> shift) & (nd - 1) : 0xFFFFFFFFu;
        const uint32_t same = __match_any_sync(0xffffffffu, dg);
        if (live && (same & lt) == 0) hist[dg] += __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();

    // per digit: this CTA's count, and each warp's offset within the CTA
    const int dg = threadIdx.x;  // digits <= threads
    if (dg < nd) {
      int run = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = s_hist[w * nd + dg];
        s_hist[w * nd + dg] = run;
        run += c;
      }
      __stcg(a.ghist + cta * nd + dg, run);
    }
    cluster_sync_all();
    // start of each digit over the cluster, then of this CTA's share of it
    int total = 0, before = 0;
    if (dg < nd) {
      for (int c = 0; c < ctas; ++c) {
        const int v = __ldcg(a.ghist + c * nd + dg);
        if (c < cta) before += v;
        total += v;
      }
    }
    int incl = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int v = s_scan[lane];
      int sum = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
      }
      s_scan[lane] = sum - v;
    }
    __syncthreads();
    if (dg < nd) {
      const int base = s_scan[warp] + incl - total + before;
      for (int w = 0; w < kSortWarps; ++w) s_hist[w * nd + dg] += base;
    }
    __syncthreads();

    for (long long b0 = lo; b0 < hi; b0 += 32 * kSortBatch) {
      uint32_t key[kSortBatch];
      int pos[kSortBatch];
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j) {
        const long long i = b0 + j * 32 + lane;
        if (i < hi) {
          key[j] = p == 0 ? token_key(tokens[i], a.V) : __ldcg(a.key[src] + i);
          pos[j] = p == 0 ? static_cast<int>(i) : __ldcg(a.pos[src] + i);
        }
      }
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j) {
        const bool live = b0 + j * 32 + lane < hi;
        const uint32_t dgt = live ? (key[j] >> shift) & (nd - 1) : 0xFFFFFFFFu;
        const uint32_t same = __match_any_sync(0xffffffffu, dgt);
        int at = 0;
        if (live) at = hist[dgt] + __popc(same & lt);
        __syncwarp();
        if (live && (same & lt) == 0) hist[dgt] += __popc(same);
        __syncwarp();
        if (live && DPRC_IN(at >= 0 && at < a.N)) {
          __stcg(a.key[dst] + at, key[j]);
          __stcg(a.pos[dst] + at, pos[j]);
        }
      }
    }
    cluster_sync_all();
  }
}

// ---------------------------------------------------------------------------
// The pass over G in sorted order.
//
// A warp takes `R` <= 32 consecutive entries [a, a + R) of the order and one
// slice of the columns, and adds up rows in fp32 registers, run by run.  A run
// of up to kShortRun entries belongs whole to the warp whose range holds its
// first entry (which then reads past its range), so most results need no
// second step.  A longer run is cut at the ranges' ends: each piece leaves its
// partial sum in the workspace and embed_long_kernel adds a run's pieces in
// order.  A range holds at most two such pieces: one that covers its first
// entry (slot 0) and one that begins later and reaches past its end (slot 1).
//
// The entries' runs come from comparing neighbours in a window of 32 entries
// before the range, the range, and up to 64 after its first entry; bit masks
// of run starts then answer every question about a run's extent.
//
// Rows are prefetched kRowsAhead at a time across run boundaries: most runs
// are one row long, and bytes in flight are what the pass lives on.
// ---------------------------------------------------------------------------
constexpr int kShortRun = 32;
constexpr int kRowsAhead = 4;
constexpr int kSegWarps = 4;  // warps per CTA of the segment pass

struct SegArgs {
  const uint32_t* key;
  const int* pos;
  long long N;        // entries
  long long T;        // tokens per sample
  int V;
  long long d;
  int R;              // entries per range
  int nslices;
  long long nranges;
  float scale;
  // norm: squared sums by original position [nslices][N]; grad: the weights
  float* sq;
  float* long_sq;     // norm: [nranges][column blocks] squares of the long runs
  const float* c;     // per-sample factors or null
  int accumulate;
  float* part;        // [nranges][2][dpad] partial sums of long runs
  long long dpad;
  int* long_at;       // [nranges]: 0, or 1 + slot of the long run that begins here
  // grad: rows no token names
  long long zero_units;
};

// kNorm: runs are equal (token, sample) pairs; otherwise equal tokens.
template <bool kNorm>
__device__ __forceinline__ bool run_starts(const SegArgs& a, long long i, uint32_t k, int p) {
  if (i == 0) return true;
  const uint32_t kp = __ldg(a.key + i - 1);
  if (kp != k) return true;
  if (kNorm) return __ldg(a.pos + i - 1) / static_cast<int>(a.T) != p / static_cast<int>(a.T);
  return false;
}

template <typename T, int AW, int NV, bool kNorm>
__device__ __forceinline__ void segment_range(const SegArgs& a, const T* __restrict__ G,
                                              T* __restrict__ dW, long long range, int slice) {
  using RawT = typename Raw<AW>::type;
  constexpr int VE = AW / static_cast<int>(sizeof(T));
  constexpr int NA = NV * VE;
  const int lane = threadIdx.x & 31;
  const long long a0 = range * a.R;
  const int R = static_cast<int>(a.N - a0 < a.R ? a.N - a0 : a.R);

  // run starts: S0 bit j = entry a0 - 32 + j, M bit j = entry a0 + j; entries
  // past the last token count as starts (they end the run before them)
  uint32_t S0 = 0;
  unsigned long long M = 0;
  uint32_t key1 = 0, key2 = 0;
  int pos1 = 0, pos2 = 0;
  unsigned long long none = 0;  // entries that hold no token
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    const long long i = a0 - 32 + w * 32 + lane;
    const bool in = i >= 0 && i < a.N;
    const uint32_t k = in ? __ldg(a.key + i) : static_cast<uint32_t>(a.V);
    const int p = in ? __ldg(a.pos + i) : 0;
    const bool tok = in && k < static_cast<uint32_t>(a.V);
    const bool st = i >= 0 && (!tok || run_starts<kNorm>(a, i, k, p));
    const uint32_t b = __ballot_sync(0xffffffffu, st);
    const uint32_t nt = __ballot_sync(0xffffffffu, !tok);
    if (w == 0) S0 = b;
    if (w == 1) { M = b; none = nt; key1 = k; pos1 = p; }
    if (w == 2) {
      M |= static_cast<unsigned long long>(b) << 32;
      none |= static_cast<unsigned long long>(nt) << 32;
      key2 = k;
      pos2 = p;
    }
  }
  // entries of the range that hold a token come first
  const int Rt = none == 0 ? R : min(R, __ffsll(static_cast<long long>(none)) - 1);

  // rows [first, last) of the window are this warp's; E bit: last row of a run
  // or piece, Lg bit: a row of a long run
  int first = 0, last = 0;
  unsigned long long E = 0, Lg = 0;
  int begins = 0;  // 1 + slot of the long run that begins here
  int o = 0;
  if (Rt > 0 && (M & 1ull) == 0) {
    // the range begins inside a run
    const int e = M == 0 ? 64 : __ffsll(static_cast<long long>(M)) - 1;
    const int before = S0 == 0 ? 64 : 32 - (31 - __clz(S0));
    if (before + e > kShortRun) {
      const int cut = min(e, R);
      Lg |= cut >= 64 ? ~0ull : (1ull << cut) - 1ull;
      E |= 1ull << (cut - 1);
      last = cut;
      o = cut;
    } else {
      first = e;
      last = e;
      o = e;
    }
  }
  while (o < Rt) {
    const unsigned long long rest = o >= 63 ? 0ull : M >> (o + 1);
    const int len = rest == 0 ? 64 : __ffsll(static_cast<long long>(rest));
    if (len > kShortRun) {  // reaches past the range (R <= kShortRun)
      Lg |= ((1ull << R) - 1ull) & ~((1ull << o) - 1ull);
      E |= 1ull << (R - 1);
      begins = o == 0 ? 1 : 2;
      last = R;
      break;
    }
    E |= 1ull << (o + len - 1);
    o += len;
    last = o;
  }
  if (slice == 0 && lane == 0 && DPRC_IN(range < a.nranges)) a.long_at[range] = begins;

  const int nvec = static_cast<int>(a.d / VE);
  const int v0 = slice * 32 * NV + lane;  // this lane's accesses: v0 + 32 j
  float acc[NA];
#pragma unroll
  for (int e = 0; e < NA; ++e) acc[e] = 0.f;
  float sq1 = 0.f, sq2 = 0.f;  // norm: squares by window entry lane, lane + 32
  int run0 = first;

  for (int r0 = first; r0 < last; r0 += kRowsAhead) {
    RawT raw[kRowsAhead][NV];
    float wgt[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int r = r0 + u;
      const int p = __shfl_sync(0xffffffffu, r < 32 ? pos1 : pos2, r & 31);
      wgt[u] = 1.f;
      if (r < last) {
        const RawT* row = reinterpret_cast<const RawT*>(G + static_cast<long long>(p) * a.d);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (v0 + 32 * j < nvec && DPRC_IN(p >= 0 && p < a.N)) raw[u][j] = __ldcs(row + v0 + 32 * j);
        if (!kNorm && a.c != nullptr) wgt[u] = __ldg(a.c + p / static_cast<int>(a.T));
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int r = r0 + u;
      if (r >= last) break;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (v0 + 32 * j < nvec) {
          float f[VE];
          unpack<T, AW>(raw[u][j], f);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            if (kNorm)
              acc[j * VE + e] += f[e];
            else
              acc[j * VE + e] = fmaf(wgt[u], f[e], acc[j * VE + e]);
          }
        }
      }
      if ((E >> r) & 1ull) {
        if ((Lg >> r) & 1ull) {
          // a piece of a long run: the one over the range's first entry is slot 0
          const int slot = run0 == 0 ? 0 : 1;
          float* out = a.part + (range * 2 + slot) * a.dpad;
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (v0 + 32 * j < nvec)
#pragma unroll
              for (int e = 0; e < VE; ++e)
                if (DPRC_IN((v0 + 32 * j) * VE + e < a.dpad))
                  out[static_cast<long long>(v0 + 32 * j) * VE + e] = acc[j * VE + e];
        } else if (kNorm) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < NA; ++e) s = fmaf(acc[e], acc[e], s);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
          if (lane == (run0 & 31)) {
            if (run0 < 32) sq1 = s; else sq2 = s;
          }
        } else {
          const uint32_t k = __shfl_sync(0xffffffffu, r < 32 ? key1 : key2, r & 31);
          RawT* out = reinterpret_cast<RawT*>(dW + static_cast<long long>(k) * a.d);
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (v0 + 32 * j < nvec && DPRC_IN(k < static_cast<uint32_t>(a.V))) {
              float f[VE];
              if (a.accumulate) {
                unpack<T, AW>(out[v0 + 32 * j], f);
#pragma unroll
                for (int e = 0; e < VE; ++e) f[e] = fmaf(a.scale, acc[j * VE + e], f[e]);
              } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) f[e] = a.scale * acc[j * VE + e];
              }
              __stcs(out + v0 + 32 * j, pack<T, AW>(f));
            }
          }
        }
#pragma unroll
        for (int e = 0; e < NA; ++e) acc[e] = 0.f;
        run0 = r + 1;
      }
    }
  }
  if (kNorm) {
    // every entry is written once: by the warp that took its row (a run's
    // square at its first entry, zero at the others), or here if it holds no token
    float* sq = a.sq + static_cast<long long>(slice) * a.N;
    const int o1 = lane, o2 = lane + 32;
    const bool w1 = (o1 >= first && o1 < last) || (o1 >= Rt && o1 < R);
    const bool w2 = o2 >= first && o2 < last;
    if (w1 && DPRC_IN(pos1 >= 0 && pos1 < a.N)) sq[pos1] = sq1;
    if (w2 && DPRC_IN(pos2 >= 0 && pos2 < a.N)) sq[pos2] = sq2;
  }
}

// First entry >= v in the sorted keys.
__device__ __forceinline__ long long lower_bound(const uint32_t* key, long long N, uint32_t v) {
  long long lo = 0, hi = N;
  while (lo < hi) {
    const long long m = (lo + hi) >> 1;
    if (__ldg(key + m) < v) lo = m + 1; else hi = m;
  }
  return lo;
}

// Rows of dW that no token names are zero: 32 rows per warp, one search per lane.
template <typename T, int AW>
__device__ __forceinline__ void zero_rows(const SegArgs& a, T* __restrict__ dW, long long unit) {
  using RawT = typename Raw<AW>::type;
  constexpr int VE = AW / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31;
  const long long v = unit * 32 + lane;
  bool absent = false;
  if (v < a.V) {
    const long long i = lower_bound(a.key, a.N, static_cast<uint32_t>(v));
    absent = i >= a.N || __ldg(a.key + i) != static_cast<uint32_t>(v);
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
    RawT* row = reinterpret_cast<RawT*>(dW + (unit * 32 + j) * a.d);
    for (long long x = lane; x < nvec; x += 32)
      if (DPRC_IN(unit * 32 + j < a.V)) __stcs(row + x, zero);
  }
}

template <typename T, int AW, int NV, bool kNorm>
__global__ void __launch_bounds__(32 * kSegWarps)
    embed_segment_kernel(const SegArgs a, const T* __restrict__ G, T* __restrict__ dW) {
  const long long w = static_cast<long long>(blockIdx.x) * kSegWarps + (threadIdx.x >> 5);
  const long long units = a.nranges * a.nslices;
  if (w < units) {
    // neighbouring warps take the slices of one range, so a row's bytes are
    // read together
    const long long range = w / a.nslices;
    segment_range<T, AW, NV, kNorm>(a, G, dW, range, static_cast<int>(w - range * a.nslices));
  } else if (!kNorm && w - units < a.zero_units) {
    zero_rows<T, AW>(a, dW, w - units);
  }
}

// ---------------------------------------------------------------------------
// Long runs: the pieces of a run added in order.  One CTA looks at 32 ranges
// (blockIdx.x) and one block of kLongCols columns (blockIdx.y); for each range
// in which a long run begins, its warps take the run's pieces in contiguous
// shares, add them, and the shares are added in warp order.
// ---------------------------------------------------------------------------
constexpr int kLongWarps = 16;
constexpr int kLongCols = 128;  // 4 per lane

template <typename T, bool kNorm>
__global__ void __launch_bounds__(32 * kLongWarps)
    embed_long_kernel(const SegArgs a, T* __restrict__ dW) {
  __shared__ float4 s_sum[kLongWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rbase = static_cast<long long>(blockIdx.x) * 32;
  const int at = rbase + lane < a.nranges ? a.long_at[rbase + lane] : 0;
  uint32_t todo = __ballot_sync(0xffffffffu, at != 0);
  const long long col = static_cast<long long>(blockIdx.y) * kLongCols + lane * 4;  // < dpad
  while (todo != 0) {
    const int j = __ffs(static_cast<int>(todo)) - 1;
    todo &= todo - 1;
    const int slot = __shfl_sync(0xffffffffu, at, j) - 1;
    const long long range = rbase + j;
    // the run's first entry, and by a search over its successors its end
    const long long b = min((range + 1) * a.R, a.N);
    const uint32_t k = __ldg(a.key + b - 1);
    const int sample = __ldg(a.pos + b - 1) / static_cast<int>(a.T);
    long long lo = b, hi = a.N;  // first entry >= b that is not of the run
    while (lo < hi) {
      const long long m = (lo + hi) >> 1;
      const bool same = __ldg(a.key + m) == k &&
                        (!kNorm || __ldg(a.pos + m) / static_cast<int>(a.T) == sample);
      if (same) lo = m + 1; else hi = m;
    }
    const long long pieces = (lo - 1) / a.R - range + 1;  // ranges range .. range + pieces - 1
    const long long share = (pieces + kLongWarps - 1) / kLongWarps;
    const long long p0 = warp * share, p1 = min(p0 + share, pieces);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (long long p = p0; p < p1; ++p) {
      const long long slot_row = (range + p) * 2 + (p == 0 ? slot : 0);
      if (DPRC_IN(range + p < a.nranges && col + 3 < a.dpad)) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part + slot_row * a.dpad + col));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    }
    s_sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      for (int w = 0; w < kLongWarps; ++w) {
        const float4 v = s_sum[w][lane];
        f[0] += v.x;
        f[1] += v.y;
        f[2] += v.z;
        f[3] += v.w;
      }
      if (kNorm) {
        // columns past d hold whatever the workspace held
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < a.d) q = fmaf(f[e], f[e], q);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
        if (lane == 0) a.long_sq[range * gridDim.y + blockIdx.y] = q;
      } else {
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
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// n_i (+)= s^2 (sum of sample i's squares): its positions' squares of every
// slice, then the long runs that are its own, in a fixed order.  A sample's
// sum is split over the CTAs of a cluster, which add their parts in rank order.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    embed_norm_finish_kernel(const SegArgs a, int ncb, float* __restrict__ n) {
  __shared__ float s_warp[8];
  __shared__ float s_cta[8];
  const uint32_t rank = cluster_ctarank(), cl = cluster_nctarank();
  const long long i = blockIdx.x / cl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = static_cast<int>(rank) * 256 + threadIdx.x, step = static_cast<int>(cl) * 256;
  float s = 0.f;
  for (int sl = 0; sl < a.nslices; ++sl) {
    const float* sq = a.sq + static_cast<long long>(sl) * a.N + i * a.T;
#pragma unroll 4
    for (long long t = t0; t < a.T; t += step) s += __ldcg(sq + t);
  }
  for (long long r = t0; r < a.nranges; r += step) {
    if (a.long_at[r] == 0) continue;
    const long long e = min((r + 1) * a.R, a.N) - 1;  // an entry of the run that begins in r
    if (__ldg(a.pos + e) / static_cast<int>(a.T) != i) continue;
    for (int b = 0; b < ncb; ++b) s += __ldcg(a.long_sq + r * ncb + b);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) s_warp[warp] = s;
  __syncthreads();
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

// Accesses per lane and row: 16 columns of bf16 or 8 of fp32 per lane, so a
// slice is 512 or 256 columns and four rows ahead fit in registers.
constexpr int accesses(int aw) { return aw == 16 ? 2 : aw == 8 ? 4 : 8; }

// Entries per range: as many as leave about 32 warps for each of 152 SMs,
// between 4 (below it the window of neighbours costs more than the rows) and
// 32 (the longest run a warp may take whole).
int range_entries(int64_t N, int64_t nslices) {
  int R = 4;
  while (R < 32 && N * nslices > int64_t(4864) * R) R *= 2;
  return R;
}

struct SegPlan {
  int aw = 16, nslices = 1, R = 4, ncb = 1;
  int64_t nranges = 0, dpad = 0;
  size_t part_off = 0, long_off = 0, lsq_off = 0, sq_off = 0, total = 0;
};

SegPlan seg_plan(dprc_dtype dt, int64_t N, int64_t d, bool norm) {
  SegPlan s;
  const int elem = dt == DPRC_F32 ? 4 : 2;
  s.aw = access_bytes(d, elem);
  const int64_t cols = int64_t(32) * accesses(s.aw) * (s.aw / elem);
  s.nslices = static_cast<int>((d + cols - 1) / cols);
  s.R = range_entries(N, s.nslices);
  s.nranges = (N + s.R - 1) / s.R;
  s.dpad = (d + kLongCols - 1) / kLongCols * kLongCols;
  s.ncb = static_cast<int>(s.dpad / kLongCols);
  size_t off = 0;
  s.long_off = off;
  off = up256(off + static_cast<size_t>(s.nranges) * 4);
  s.part_off = off;
  off = up256(off + static_cast<size_t>(s.nranges) * 2 * s.dpad * 4);
  if (norm) {
    s.lsq_off = off;
    off = up256(off + static_cast<size_t>(s.nranges) * s.ncb * 4);
    s.sq_off = off;
    off = up256(off + static_cast<size_t>(s.nslices) * N * 4);
  }
  s.total = off > 0 ? off : 256;
  return s;
}

struct SortPlan {
  int passes = 1, dbits = 1, ctas = 1;
  size_t key_off[2], pos_off[2], hist_off = 0, total = 0;
};

SortPlan sort_plan(int64_t N, int64_t V) {
  SortPlan s;
  int bits = 1;
  while ((int64_t(1) << bits) <= V) ++bits;  // keys 0..V
  s.passes = (bits + 9) / 10;
  s.dbits = (bits + s.passes - 1) / s.passes;
  s.ctas = N <= 4096 ? 1 : 8;
  size_t off = 0;
  for (int b = 0; b < 2; ++b) {
    s.key_off[b] = off;
    off = up256(off + static_cast<size_t>(N) * 4);
    s.pos_off[b] = off;
    off = up256(off + static_cast<size_t>(N) * 4);
  }
  s.hist_off = off;
  off = up256(off + static_cast<size_t>(8) * kSortMaxDigit * 4);
  s.total = off;
  return s;
}

template <typename TOK>
cudaError_t launch_sort_t(const TOK* tokens, const SortArgs& a, int ctas, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kSortWarps) * (size_t(1) << a.dbits) * 4;
  cudaError_t e = cudaFuncSetAttribute(token_sort_kernel<TOK>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSortWarps * kSortMaxDigit * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, token_sort_kernel<TOK>, tokens, a);
}

SegArgs seg_args(const EmbedCall& c, const SegPlan& p, const SortPlan& sp, char* ws) {
  SegArgs a;
  const char* plan = static_cast<const char*>(c.plan);
  a.key = reinterpret_cast<const uint32_t*>(plan + sp.key_off[0]);
  a.pos = reinterpret_cast<const int*>(plan + sp.pos_off[0]);
  a.N = c.B * c.T;
  a.T = c.T > 0 ? c.T : 1;
  a.V = static_cast<int>(c.V);
  a.d = c.d;
  a.R = p.R;
  a.nslices = p.nslices;
  a.nranges = p.nranges;
  a.scale = c.scale;
  a.sq = reinterpret_cast<float*>(ws + p.sq_off);
  a.long_sq = reinterpret_cast<float*>(ws + p.lsq_off);
  a.c = nullptr;
  a.accumulate = c.accumulate;
  a.part = reinterpret_cast<float*>(ws + p.part_off);
  a.dpad = p.dpad;
  a.long_at = reinterpret_cast<int*>(ws + p.long_off);
  a.zero_units = 0;
  return a;
}

template <typename T, int AW, bool kNorm>
cudaError_t launch_segments_t(const SegArgs& a, const SegPlan& p, const void* G, void* dW,
                              cudaStream_t s) {
  const long long warps = a.nranges * a.nslices + a.zero_units;
  if (warps > 0) {
    const long long ctas = (warps + kSegWarps - 1) / kSegWarps;
    embed_segment_kernel<T, AW, accesses(AW), kNorm>
        <<<static_cast<unsigned>(ctas), 32 * kSegWarps, 0, s>>>(a, static_cast<const T*>(G),
                                                                static_cast<T*>(dW));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.N > kShortRun) {
    const dim3 grid(static_cast<unsigned>((a.nranges + 31) / 32), static_cast<unsigned>(p.ncb));
    embed_long_kernel<T, kNorm><<<grid, 32 * kLongWarps, 0, s>>>(a, static_cast<T*>(dW));
    return cudaGetLastError();
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
  embed_lookup_kernel<T, AW, TOK><<<static_cast<unsigned>(ctas), 256, 0, s>>>(
      static_cast<const T*>(W), static_cast<const TOK*>(tokens), N, static_cast<int>(V), d, scale,
      static_cast<T*>(out), lanes, static_cast<int>(upr));
  return cudaGetLastError();
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
  const SortPlan sp = sort_plan(N, V);
  char* p = static_cast<char*>(plan);
  SortArgs a;
  a.N = N;
  a.V = static_cast<int>(V);
  a.passes = sp.passes;
  a.dbits = sp.dbits;
  for (int b = 0; b < 2; ++b) {
    a.key[b] = reinterpret_cast<uint32_t*>(p + sp.key_off[b]);
    a.pos[b] = reinterpret_cast<int*>(p + sp.pos_off[b]);
  }
  a.ghist = reinterpret_cast<int*>(p + sp.hist_off);
  return token_bytes == 4
             ? launch_sort_t<int32_t>(static_cast<const int32_t*>(tokens), a, sp.ctas, s)
             : launch_sort_t<long long>(static_cast<const long long*>(tokens), a, sp.ctas, s);
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
  // one CTA per sample where a sample has few values, else a cluster of 8
  const int cl = a.T * p.nslices + a.nranges > 8192 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c.B * cl));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cl;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, embed_norm_finish_kernel, a, p.ncb, n);
}

cudaError_t launch_embed_grad(const EmbedCall& c, const float* clip, void* dW, void* ws,
                              cudaStream_t s) {
  const SegPlan p = seg_plan(c.dtype, c.B * c.T, c.d, false);
  SegArgs a = seg_args(c, p, sort_plan(c.B * c.T, c.V), static_cast<char*>(ws));
  a.c = clip;
  a.zero_units = c.accumulate ? 0 : (c.V + 31) / 32;
  return launch_segments<false>(c.dtype, a, p, c.G, dW, s);
}

}  // namespace dprc
