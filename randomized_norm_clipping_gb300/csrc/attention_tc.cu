// Attention on the tensor cores (tcgen05, bf16 operands, fp32 accumulators in tensor
// memory), forward and backward.
//
//   forward   S = Q K^T, P = exp2(S c - m), O += P V, with the running maximum m and sum of
//             a row (one pass over the keys); O is rescaled only when m grows by 2^8
//   dQ        per tile of rows:  S, dP = dO V^T, dS = P (dP - delta), dQ += dS K
//   dK, dV    per tile of keys:  the same transposed, dV += P^T dO, dK += dS^T Q
//
// P and dS never leave the SM: a thread owns a lane of tensor memory (a row, or a key),
// reads the scores, and writes the weights back as the bf16 first operand of the next
// product.  One warp copies tiles by TMA into a ring, one thread issues the products,
// four warps a tile of rows do the softmax (forward), sixteen the gradient's weights.
//
// The rows of a tile are the queries of all G heads that share a head of keys
// (attention.cuh): 128 / G tokens, brought by one box of G heads by tokens.  So few
// tokens fill a tile, a causal border costs 128 / G tokens and not 128, and the sum over
// the heads of a group in dK and dV is the product's.
//
// Roundings: S, dP, the statistics and the sums over keys or rows are fp32.  P and dS are rounded
// to bf16, since the products take their operands in that type; each is off by a half step of its own,
// with either sign, so that over many keys the errors add up in the mean square only: results are
// off by 0.0020 to 0.0023 of their 2-norm where their own rounding is 0.0016, gradients by 0.0027
// where that and delta's, of the rounded output, are 0.0021.  The row's sum takes P unrounded.
//
// The backward pass forms S and dP in both of its kernels (seven products for five):
// with one kernel, dQ is a sum over CTAs, whose order would have to be kept or its
// roundings change from run to run.

#include <algorithm>
#include <cfloat>

#include "attention.cuh"
#include "tmem.cuh"
#include "vec.cuh"

namespace dprc {
namespace {

constexpr int kTile = 128;           // rows, and keys, of a tile
constexpr int kBlock = kTile * 128;  // bytes of a tile's 64 columns
constexpr int kMaxKeyTiles = (1 << 20) / kTile;
constexpr float kLazy = 8.f;  // a row is rescaled when its maximum grows by 2^kLazy

constexpr uint32_t kSuspendNs = 20000;

template <bool kSuspend>
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  if constexpr (!kSuspend) return mbar_try_wait(bar, parity);
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

// Bounded wait; false once it ran out (recorded) or another role has.
template <bool kSuspend>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int code,
                                         volatile int* abort) {
  if (try_wait_long<kSuspend>(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    if (try_wait_long<kSuspend>(bar, parity)) return true;
    if (*abort != 0) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(code);
      *abort = 1;
      return false;
    }
  }
}

// The warp's number, in a form that the compiler takes for the same in all its lanes.
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}

// The same for a warp, which waits with one lane (polling lanes take issue slots).
template <bool kSuspend>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int code,
                                          volatile int* abort) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_bar<kSuspend>(bar, parity, code, abort) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The same by all lanes of a warp.
template <bool kSuspend>
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int code,
                                         volatile int* abort) {
  return __all_sync(0xffffffffu, wait_bar<kSuspend>(bar, parity, code, abort)) != 0;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int kRegs>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four values from shared memory, not ahead of what is volatile before it (hoisted, the
// 64 columns' loads take more registers than a thread has).
__device__ __forceinline__ void ld_shared4(const float* p, float (&v)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(smem_u32(p)));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Descriptors of a tile [128][64 kBlocks] at a 1024-byte boundary.  As the operand
// whose width is summed over (K-major): a step of 16 is 32 bytes, a block of 64 kBlock
// bytes.  As the operand whose rows are summed over (MN-major): a step is 16 rows.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return make_sdesc(addr, 16, 1024, kSwz128);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return make_sdesc(addr, kBlock, 1024, kSwz128);
}

__device__ __forceinline__ void commit(bool lead, uint64_t* bar) {
  if (lead) umma_commit(bar);
}

// acc = A B^T over the width D (both tiles' widths are summed over), up to 64 kBlocks.
// Unrolled, so that a step's operands are those of the first plus constants.
template <int kBlocks, bool kUnroll>
__device__ __forceinline__ void mma_width(bool lead, uint32_t acc, uint64_t a, uint64_t b,
                                          uint32_t idesc, int steps) {
  if (!lead) return;
  const auto step = [&](int k) {
    const uint32_t at = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
    umma_bf16(acc, a + at, b + at, idesc, k > 0 ? 1u : 0u);
  };
  if constexpr (kUnroll) {
#pragma unroll
    for (int k = 0; k < 4 * kBlocks; ++k)
      if (k < steps) step(k);
  } else {
#pragma unroll 1
    for (int k = 0; k < steps; ++k) step(k);
  }
}

// acc (+)= A B with A [128][128] in tensor memory and B's rows summed over.
__device__ __forceinline__ void mma_rows(bool lead, uint32_t acc, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                         bool accumulate) {
  if (!lead) return;
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
    umma_bf16_ts(acc, a_tmem + k * 8, b + ((k * 2048) >> 4), idesc, accumulate || k > 0 ? 1u : 0u);
}

struct TcArgs {
  AttnArgs a;
  int nt;        // tokens of a tile of rows
  int row_tiles; // tiles of rows of a head of keys
  int groups;    // CTAs' groups of row tiles
  int steps;     // D / 16, rounded up
  float c;       // scale log2(e)
  float c_cap;   // 2 scale log2(e) / cap
  float cap2;    // cap log2(e)
};

// A stage and the parity of its round.
struct Pos {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
  }
};

// The set bits of a list of words, in order.
struct Bits {
  const uint32_t* words;
  int n, w = 0;
  uint32_t left;
  __device__ __forceinline__ Bits(const uint32_t* words, int n)
      : words(words), n(n), left(n > 0 ? words[0] : 0u) {}
  __device__ __forceinline__ int next() {  // -1: no more
    while (left == 0u) {
      if (++w >= n) return -1;
      left = words[w];
    }
    const int b = __ffs(left) - 1;
    left &= left - 1;
    return w * 32 + b;
  }
};

// Scores of one row in units of log2, from the products q k: kForm 0 leaves them (times c
// they are the scores, which the caller takes); 1: with the bias; 2: capped; 3: both.
// The cap: tanh(u) = 1 - 2 / (1 + exp(2 u)), to 2^-22 of it.
template <int kForm, int kN>
__device__ __forceinline__ void scores(const TcArgs& x, float (&z)[kN], float slope2, float dist0) {
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    if constexpr (kForm >= 2) z[j] = fmaf(-2.f * x.cap2, rcp(1.f + ex2(z[j] * x.c_cap)), x.cap2);
    else if constexpr (kForm == 1) z[j] *= x.c;
    if constexpr (kForm == 1 || kForm == 3)
      z[j] = fmaf(-slope2, fabsf(dist0 - static_cast<float>(j)), z[j]);
  }
}

// Bits of 32 consecutive columns, of which the first n are set.
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// The columns whose document is this lane's, `theirs` being that of column `lane`: a
// ballot for each document that the warp's lanes have, mostly one or two.
__device__ __forceinline__ uint32_t same_docs(int doc, int theirs) {
  uint32_t left = 0xffffffffu, mine = 0u;
  while (left != 0u) {  // (the same for the warp)
    const int d = __shfl_sync(0xffffffffu, doc, __ffs(left) - 1);
    const uint32_t cols = __ballot_sync(0xffffffffu, theirs == d);
    const bool is = doc == d;
    if (is) mine = cols;
    left &= ~__ballot_sync(0xffffffffu, is);
  }
  return mine;
}

// Bits of the columns, 32 kWords from key j0 on, that a row sees.
template <int kWords>
__device__ __forceinline__ void seen_bits(uint32_t (&bits)[kWords], const RowSees& see,
                                          const int* docs, int j0, int Tk, bool by_doc) {
#pragma unroll
  for (int q = 0; q < kWords; ++q) {
    bits[q] = first_bits(see.lim - j0 - q * 32);
    if (by_doc) {
      const int j = j0 + q * 32 + (threadIdx.x & 31);
      bits[q] &= same_docs(see.doc, j < Tk ? docs[j] : -2);
    }
  }
}

// -inf in the columns, kN from key j0 on, that a row does not see.
template <int kN>
__device__ __forceinline__ void hide(float (&z)[kN], const RowSees& see, const int* docs, int j0,
                                     int Tk, bool by_doc) {
  uint32_t bits[kN / 32];
  seen_bits(bits, see, docs, j0, Tk, by_doc);
#pragma unroll
  for (int j = 0; j < kN; ++j)
    if (!((bits[j / 32] >> (j & 31)) & 1u)) z[j] = -INFINITY;
}

// The softmax's weights p of two products z (off: -lse, in units of log2), and in z those
// weights times the cap's slope 1 - t^2.  The two capped scores share a reciprocal (beyond
// 2^60 the sum of 1 and the exponential is held: tanh is 1 there); in the forward
// pass, which waits for chains and not for the special functions, that was slower.
template <int kForm>
__device__ __forceinline__ void weights2(const TcArgs& x, float* z, float* p, const float* slope2,
                                         const float* dist, const float* off) {
  if constexpr (kForm >= 2) {
    const float a = 1.f + ex2(fminf(z[0] * x.c_cap, 60.f)), b = 1.f + ex2(fminf(z[1] * x.c_cap, 60.f));
    const float r = -2.f * rcp(a * b);
    const float t[2] = {fmaf(r, b, 1.f), fmaf(r, a, 1.f)};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float s = fmaf(t[u], x.cap2, off[u]);
      if constexpr (kForm == 3) s = fmaf(-slope2[u], dist[u], s);
      p[u] = ex2(s);
      z[u] = p[u] * fmaf(-t[u], t[u], 1.f);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float s = fmaf(z[u], x.c, off[u]);
      if constexpr (kForm == 1) s = fmaf(-slope2[u], dist[u], s);
      z[u] = p[u] = ex2(s);
    }
  }
}

// The same of a row's consecutive columns.
template <int kForm, int kN>
__device__ __forceinline__ void weights(const TcArgs& x, float (&z)[kN], float slope2, float dist0,
                                        float off) {
  const float sl[2] = {slope2, slope2}, of[2] = {off, off};
#pragma unroll
  for (int j = 0; j < kN; j += 2) {
    const float dist[2] = {fabsf(dist0 - static_cast<float>(j)),
                           fabsf(dist0 - static_cast<float>(j + 1))};
    float p[2];
    weights2<kForm>(x, &z[j], p, sl, dist, of);
  }
}

// What the rows of this warp, of this CTA see, for the choice of tiles and masks.
struct Extent {
  int min_lim, max_lim, lo, hi;
};
__device__ __forceinline__ Extent warp_extent(bool mine, const RowSees& r) {
  Extent e;
  e.min_lim = mine ? r.lim : 0x7fffffff;
  e.max_lim = mine ? r.lim : 0;
  e.lo = mine && r.doc >= 0 ? r.doc : 0x7fffffff;
  e.hi = mine && r.doc >= 0 ? r.doc : -1;
  for (int o = 16; o > 0; o >>= 1) {
    e.min_lim = min(e.min_lim, __shfl_xor_sync(0xffffffffu, e.min_lim, o));
    e.max_lim = max(e.max_lim, __shfl_xor_sync(0xffffffffu, e.max_lim, o));
    e.lo = min(e.lo, __shfl_xor_sync(0xffffffffu, e.lo, o));
    e.hi = max(e.hi, __shfl_xor_sync(0xffffffffu, e.hi, o));
  }
  return e;
}

// Documents in the 128 keys of a tile.
__device__ __forceinline__ DocSpan key_tile_docs(const AttnArgs& a, int b, int tile) {
  const int spans = (a.Tk + kDocSpan - 1) / kDocSpan;
  const DocSpan* s = a.spans + static_cast<long long>(b) * spans;
  if (!DPRC_IN(tile >= 0 && 2 * tile < spans)) return {0, -1, 1, 0};
  DocSpan r = s[2 * tile];
  if (2 * tile + 1 < spans) {
    const DocSpan q = s[2 * tile + 1];
    r.lo = min(r.lo, q.lo);
    r.hi = max(r.hi, q.hi);
    r.pad |= q.pad;
  }
  return r;
}

// What the rows of tokens [tok0, tok1) may see, without a look at each of them: a limit, and
// the documents of the spans that they stand in.  So the copies start a load's and a
// barrier's time earlier than with the rows' own.
struct Reach {
  int top, lo, hi;
};
__device__ __forceinline__ Reach reach_of(const AttnArgs& a, int b, int tok0, int tok1, int keys,
                                          int first) {
  Reach r = {tok0 < tok1 ? keys : 0, 0, 0};
  if (a.causal && tok0 < tok1) {
    int see = first + tok1;
    if (a.prefix != nullptr) see = max(see, a.prefix[b]);
    r.top = max(0, min(see, keys));
  }
  if (a.docs != nullptr) {
    r.lo = 0x7fffffff;
    r.hi = -1;
    const int spans = (a.Tk + kDocSpan - 1) / kDocSpan;
    const int p0 = max(0, first + tok0), p1 = min(a.Tk, first + tok1);  // positions
    for (int q = p0 / kDocSpan + (threadIdx.x & 31); p0 < p1 && q <= (p1 - 1) / kDocSpan; q += 32) {
      const DocSpan s = a.spans[static_cast<long long>(b) * spans + q];
      r.lo = min(r.lo, s.lo);
      r.hi = max(r.hi, s.hi);
    }
    r.lo = __reduce_min_sync(0xffffffffu, r.lo);
    r.hi = __reduce_max_sync(0xffffffffu, r.hi);
  }
  return r;
}

// Key tiles [t0, t1) that some row of the CTA may see, as bits.
__device__ __forceinline__ void key_tile_bits(const AttnArgs& a, int b, int t0, int t1, int lo,
                                              int hi, uint32_t* bits, int words) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int w = warp; w < words; w += warps) {
    const int tile = w * 32 + lane;
    bool ok = tile >= t0 && tile < t1;
    if (ok && a.docs != nullptr) {
      const DocSpan s = key_tile_docs(a, b, tile);
      ok = s.lo <= hi && lo <= s.hi;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, ok);
    if (lane == 0 && DPRC_IN(w < kMaxKeyTiles / 32)) bits[w] = m;
  }
}

// Zeroes, by the 128 threads of a group, the rows of a tile that must not be read: 128
// bytes of each of the blocks.
template <int kBlocks>
__device__ __forceinline__ void zero_row(uint8_t* tile, int r) {
#pragma unroll
  for (int q = 0; q < kBlocks; ++q) {
    uint4* p = reinterpret_cast<uint4*>(tile + q * kBlock + r * 128);
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <int kBlocks, int kTiles>
struct FwdCfg {
  static constexpr int kQ = kTiles * kBlocks * kBlock;
  static constexpr int kSlot = kBlocks * kBlock;
  // one tile: two CTAs to an SM
  static constexpr int kStages = kTiles == 1 ? (kBlocks == 1 ? 5 : 2) : (kBlocks == 1 ? 8 : 4);
  static constexpr int kSoft = 4 * kTiles;  // warps of the softmax
  static constexpr int kThreads = 32 * (kSoft + 4);
  static constexpr int kRegs = kTiles == 1 ? 128 : 168;
  static constexpr int kMore = kTiles == 1 ? 200 : 224, kLess = 56;
  static_assert(kThreads * kRegs == 32 * kSoft * kMore + 128 * kLess, "registers of the block");
  static constexpr int kSmem = kQ + kStages * kSlot + 1024 + 1024 + kMaxKeyTiles / 8;
  // Tiles of scores in tensor memory: a third one for narrow heads, so that a group's next
  // scores are formed while it still has its last ones
  static constexpr int kBufs = kTiles == 2 && kBlocks == 1 ? 3 : kTiles;
  static constexpr int kO = 128 * kBufs;  // first column of the sums
  static constexpr int kWide = kBufs == 3 ? 64 : 128;  // columns of a tile's sums
  static constexpr int kTmem = 256 * kTiles;
  static_assert((kTiles == 1 ? 2 : 1) * (kSmem + 1024) <= 228 * 1024, "shared memory of a CTA");
};

// Two tiles of rows in turn: while a group of four warps takes the exponentials of its
// tile, the tensor core forms the other's products.  kTiles 1: few rows, whose keys are
// shared out; two CTAs to an SM, one's copies and products under the other's
// exponentials, and only the warps that have rows take part.
// Bound, for heads of 64, by the exponentials (one a pair, 16 a clock, against 512 clocks
// of products for 128 x 128 pairs) and the operations around them.  Measured, bf16, causal,
// by the pairs that are seen: 4 x 4096 tokens of 32 heads of 64 over 8, 331 us, 0.82 PFLOP/s;
// 2 x 8192 of 16 heads of 128 over 4, 421 us, 1.29 PFLOP/s; 16384 tokens of 16 heads of 128
// over 4, capped, with a prefix, 1.64 ms, 0.74 PFLOP/s (three special functions a pair).
template <int kBlocks, int kTiles, int kForm>
__global__ void __launch_bounds__(FwdCfg<kBlocks, kTiles>::kThreads, kTiles == 1 ? 2 : 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const TcArgs x) {
  using Cfg = FwdCfg<kBlocks, kTiles>;
  constexpr int kStages = Cfg::kStages;
  const AttnArgs& a = x.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = align_1024(smem_raw);
  uint8_t* ring = qs + Cfg::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * Cfg::kSlot);
  uint64_t* empty = full + kStages;
  uint64_t* qfull = empty + kStages;
  uint64_t* sfull = qfull + 1;   // [kBufs], up to 3
  uint64_t* pfull = sfull + 3;   // [kBufs]
  uint64_t* pvfull = pfull + 3;  // [2]: a product of values, where scores run ahead of it
  uint64_t* ofull = pvfull + 2;  // [2]: the last one
  uint64_t* drain = ofull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* bits = reinterpret_cast<uint32_t*>(ring + kStages * Cfg::kSlot + 512);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int bhs = a.B * a.Hkv;
  const int bh = blockIdx.x % bhs, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  const int grp = x.groups - 1 - blockIdx.x / bhs;  // the longest rows first
  // warps of a tile that have rows
  const int active =
      kTiles == 2 ? 4 : (min(x.nt, a.Tq - grp * x.nt) * a.G + 31) / 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(qfull, 1);
    for (int u = 0; u < 3; ++u) {
      mbar_init(&sfull[u], 1);
      mbar_init(&pfull[u], active);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&pvfull[w], 1);
      mbar_init(&ofull[w], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == Cfg::kSoft + 1) {
    tmem_alloc(tmem_slot, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const int w = warp >> 2;  // the tile of rows of a softmax warp
  const int r = threadIdx.x & (kTile - 1);
  const int tt = r / a.G, tok = (grp * kTiles + w) * x.nt + tt;
  const bool mine = warp < Cfg::kSoft && tt < x.nt && tok < a.Tq;
  RowSees see = {0, 0, -1};
  Extent e = {};
  const Reach reach = reach_of(a, b, grp * kTiles * x.nt, min((grp + 1) * kTiles * x.nt, a.Tq), keys, first);
  const int top = reach.top;
  const int t0 = blockIdx.z * a.per_split, t1 = min(t0 + a.per_split, (top + kTile - 1) / kTile);
  const int words = max(0, (t1 + 31) / 32);
  key_tile_bits(a, b, t0, t1, reach.lo, reach.hi, bits, words);
  if (mine) see = attn_row(a, b, tok, keys, first);
  __syncthreads();
  if (warp < Cfg::kSoft) e = warp_extent(mine, see);

  if (warp >= Cfg::kSoft) {
    regs_less<Cfg::kLess>();
    if (warp == Cfg::kSoft && lane == 0) {
      Bits it(bits, words);
      Pos pos;
      int j = it.next(), issued = 0;
      bool ok = true;
      if (j >= 0) {
        mbar_arrive_expect_tx(qfull, kTiles * kBlocks * x.nt * a.G * 128);
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
#pragma unroll
          for (int q = 0; q < kBlocks; ++q)
            tma_load_4d(qs + (u * kBlocks + q) * kBlock, &map_q, qfull, q * 64, hk * a.G,
                        (grp * kTiles + u) * x.nt, b);
      }
      const bool any = j >= 0;
      for (; j >= 0 && ok; j = it.next()) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (!wait_bar<true>(&empty[pos.s], pos.parity ^ 1, DPRC_DEVERR_PIPE_EMPTY, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[pos.s], Cfg::kSlot);
#pragma unroll
          for (int q = 0; q < kBlocks; ++q)
            tma_load_4d(ring + pos.s * Cfg::kSlot + q * kBlock, kv == 0 ? &map_k : &map_v,
                        &full[pos.s], q * 64, hk, j * kTile, b);
          ++issued;
          pos.next(kStages);
        }
      }
      // copies still under way land before the CTA can exit
      if (any) mbar_wait(qfull, 0, DPRC_DEVERR_PIPE_FULL);
      for (int k = issued - 1; k >= 0 && k >= issued - kStages; --k)
        mbar_wait(&full[k % kStages], (k / kStages) & 1, DPRC_DEVERR_PIPE_FULL);
    } else if (warp == Cfg::kSoft + 1) {
      // all lanes keep step, one issues: the descriptors stay in the warp's common registers
      const bool lead = elect_one() != 0;
      const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
      const uint32_t id_o = make_idesc_bf16(kTile, x.steps * 16, false, true);
      const uint64_t dq = desc_k(smem_u32(qs));
      const uint64_t dk = desc_k(smem_u32(ring)), dv = desc_mn(smem_u32(ring));
      int tiles = 0;
      for (int i = 0; i < words; ++i) tiles += __popc(bits[i]);
      const int total = tiles * kTiles;
      // Step i is tile i / kTiles of the keys and tile i % kTiles of the rows, its scores in
      // buffer i % kBufs; unrolled over the steps after which these repeat, so that they
      // are constants (with running numbers the issue of a step took longer than its products).
      constexpr int kBufs = Cfg::kBufs, kPeriod = kBufs == 3 ? 6 : kBufs;
      Pos kpos, vpos;  // keys lie in every second stage, values behind them
      vpos.next(kStages);
      bool ok = true, issued = false;
      const auto scores_of = [&](int u) {
        const int rows = u % kTiles, buf = u % kBufs;
        if (rows == 0) {
          if (!wait_all<false>(&full[kpos.s], kpos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag)) return false;
          tc_fence_after();
        }
        mma_width<kBlocks, kBlocks == 1>(lead, tmem + buf * 128,
                                         dq + ((rows * kBlocks * kBlock) >> 4),
                                         dk + ((kpos.s * Cfg::kSlot) >> 4), id_s, x.steps);
        commit(lead, &sfull[buf]);
        issued = true;
        if (rows == kTiles - 1) {
          commit(lead, &empty[kpos.s]);
          kpos.next(kStages);
          kpos.next(kStages);
        }
        return true;
      };
      if (total > 0) ok = wait_all<false>(qfull, 0, DPRC_DEVERR_PIPE_FULL, abort_flag);
#pragma unroll
      for (int u = 0; u < kBufs; ++u)
        if (u < total) ok = ok && scores_of(u);
      for (int i = 0; i < total && ok; i += kPeriod) {
#pragma unroll
        for (int u = 0; u < kPeriod; ++u) {
          const int rows = u % kTiles, buf = u % kBufs;
          if (i + u >= total) break;
          const int t = i / kTiles + u / kTiles;
          if (rows == 0)
            ok = ok && wait_all<false>(&full[vpos.s], vpos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
          // (a barrier a buffer: with one a group, a group whose next scores are there could
          // end two tiles while their values are waited for, and the wait would miss the first)
          ok = ok && wait_all<false>(&pfull[buf], ((i + u) / kBufs) & 1, DPRC_DEVERR_ACCUM, abort_flag);
          if (!ok) break;
          tc_fence_after();
          mma_rows(lead, tmem + Cfg::kO + rows * Cfg::kWide, tmem + buf * 128,
                   dv + ((vpos.s * Cfg::kSlot) >> 4), id_o, t > 0);
          // (where a group's next scores are formed behind its product, they tell of it)
          if (kBufs > kTiles) commit(lead, &pvfull[rows]);
          if (i + u + kTiles >= total) commit(lead, &ofull[rows]);
          if (rows == kTiles - 1) {
            commit(lead, &empty[vpos.s]);
            vpos.next(kStages);
            vpos.next(kStages);
          }
          if (i + u + kBufs < total) ok = scores_of(u + kBufs);
        }
      }
      if (issued && lead) umma_drain(drain, kWaitLimitNs);
    }
  } else {
    regs_more<Cfg::kMore>();
    if (kTiles == 2 || warp < active) {
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t to = tmem + lanes + Cfg::kO + w * Cfg::kWide;
      const int h = hk * a.G + r - tt * a.G;
      const float slope2 =
          (kForm & 1) != 0 && a.slopes != nullptr && mine ? a.slopes[h] * kLog2e : 0.f;
      const int* docs = a.docs != nullptr ? a.docs + static_cast<long long>(b) * a.Tk : nullptr;
      const int cols = x.steps * 16;
      Bits it(bits, words);
      Pos vpos;  // the ring's place of this tile's values
      vpos.next(kStages);
      float m = -INFINITY, l = 0.f;
      int n = 0, buf = w;
      uint32_t round = 0;  // of buf
      bool ok = true;
      for (int j = it.next(); j >= 0; j = it.next(), ++n) {
        ok = wait_warp<kBlocks == 2>(&sfull[buf], round, DPRC_DEVERR_ACCUM, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = tmem + lanes + buf * 128;
        uint64_t* const taken = &pfull[buf];
        buf += kTiles;
        if (buf >= Cfg::kBufs) {
          buf -= Cfg::kBufs;
          round ^= 1u;
        }
        const int j0 = j * kTile;
        bool dirty = j0 + kTile > top, by_doc = false;
        if (docs != nullptr) {
          const DocSpan s = key_tile_docs(a, b, j);
          by_doc = s.pad || s.lo != s.hi || e.lo != s.lo || e.hi != s.lo;
          dirty = dirty || s.pad;
        }
        const float mul = kForm == 0 ? x.c : 1.f;
        float z[kTile];
        if constexpr (kTiles == 2) {
          tmem_ld_128cols(ts, z);
        } else {  // (128 at once take more registers than the block is launched with)
#pragma unroll
          for (int c = 0; c < kTile; c += 32)
            tmem_ld_32cols(ts + c, reinterpret_cast<float(&)[32]>(z[c]));
        }
        scores<kForm>(x, z, slope2, static_cast<float>(see.pos - j0));
        if (j0 + kTile > e.min_lim || by_doc) hide(z, see, docs, j0, a.Tk, by_doc);
        float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
        for (int c = 4; c + 8 <= kTile; c += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], z[c + u], z[c + 4 + u]);
        mx[0] = max3(mx[0], z[kTile - 4], z[kTile - 3]);
        mx[1] = max3(mx[1], z[kTile - 2], z[kTile - 1]);
        const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * mul;
        const bool grow = mt > m + kLazy || (m == -INFINITY && mt > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m - mt) : 1.f;
          if (grow) m = mt;
          l *= f;
          if (n > 0) {
            // (these scores were formed behind the product before the last, so that the
            // barrier stands at the last or behind it; at the end it need not)
            if constexpr (Cfg::kBufs > kTiles) {
              ok = wait_warp<kBlocks == 2>(&pvfull[w], (n - 1) & 1, DPRC_DEVERR_ACCUM, abort_flag);
              if (!ok) break;
              tc_fence_after();
            }
            for (int c = 0; c < cols; c += 16) {
              float o[16];
              tmem_ld_16cols(to + c, o);
              uint32_t u[16];
#pragma unroll
              for (int q = 0; q < 16; ++q) u[q] = __float_as_uint(o[q] * f);
              tmem_st_16cols(to + c, u);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const F2 mul2 = f2(mul, mul), off2 = f2(off, off);
        F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int c0 = 0; c0 < kTile; c0 += 64) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float p0, p1;
            split(fma2(f2(z[c0 + c], z[c0 + c + 1]), mul2, off2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], f2(p0, p1));
            p[c / 2] = pack_bf16(p0, p1);
          }
          tmem_st_32cols(ts + c0 / 2, p);
        }
        {
          float s0, s1;
          split(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        }
        tmem_st_wait();
        if (dirty && w == 0) {
          // values that no row of the CTA sees may be anything, and 0 times NaN is NaN
          ok = wait_warp<kBlocks == 2>(&full[vpos.s], vpos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
          if (!ok) break;
          for (int q = r; q < kTile; q += 32 * active) {
            const int key = j0 + q;
            if (key >= top || (docs != nullptr && docs[key] < 0))
              zero_row<kBlocks>(ring + vpos.s * Cfg::kSlot, q);
          }
          fence_proxy_async_smem();
        }
        vpos.next(kStages);
        vpos.next(kStages);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(taken);
      }
      if (n > 0 && ok)
        ok = wait_warp<kBlocks == 2>(&ofull[w], 0, DPRC_DEVERR_ACCUM, abort_flag);
      tc_fence_after();
      if (ok) {
        const bool parts = a.splits > 1;
        const float inv = parts ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
        const int rows = a.Tq * a.G;
        const long long prow =
            (static_cast<long long>(blockIdx.z) * bhs + bh) * rows + tok * a.G + r - tt * a.G;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                             ((static_cast<long long>(b) * a.Tq + tok) * a.H + h) * a.D;
        for (int c = 0; c < cols; c += 16) {
          float o[16];
          if (n > 0) {
            tmem_ld_16cols(to + c, o);
          } else {
#pragma unroll
            for (int q = 0; q < 16; ++q) o[q] = 0.f;
          }
          if (mine) {
#pragma unroll
            for (int q = 0; q < 16; q += 8) {
              if (c + q >= a.D) continue;
#pragma unroll
              for (int u = 0; u < 8; ++u) o[q + u] *= inv;
              if (parts) {
                store_row<4>(a.part + prow * a.D + c + q, o + q);
                store_row<4>(a.part + prow * a.D + c + q + 4, o + q + 4);
              } else {
                store_row<8>(out + c + q, o + q);
              }
            }
          }
          __syncwarp();  // (the next read is the whole warp's)
        }
        if (mine && parts) {
          a.part_stats[prow] = make_float2(m, l);
        } else if (mine && a.lse != nullptr) {
          a.lse[(static_cast<long long>(b) * a.H + h) * a.Tq + tok] = m * kLn2 + logf(l);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::kSoft + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmem);
  }
}

template <int kBlocks, int kTiles, int kForm>
cudaError_t launch_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                       const TcArgs& x, cudaStream_t s) {
  constexpr int bytes = FwdCfg<kBlocks, kTiles>::kSmem;
  const cudaError_t e = allow_smem<attention_tc_kernel<kBlocks, kTiles, kForm>>(bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(x.a.B * x.a.Hkv * x.groups, 1, x.a.splits);
  return launch_after(attention_tc_kernel<kBlocks, kTiles, kForm>, grid, FwdCfg<kBlocks, kTiles>::kThreads, 1, s,
                      bytes, q,
                      k, v, x);
}

template <int kBlocks, int kTiles>
cudaError_t launch_fwd_form(int form, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, const TcArgs& x, cudaStream_t s) {
  if (form == 0) return launch_fwd<kBlocks, kTiles, 0>(q, k, v, x, s);
  if (form == 1) return launch_fwd<kBlocks, kTiles, 1>(q, k, v, x, s);
  if (form == 2) return launch_fwd<kBlocks, kTiles, 2>(q, k, v, x, s);
  return launch_fwd<kBlocks, kTiles, 3>(q, k, v, x, s);
}

// ---------------------------------------------------------------------------
// Few rows (up to 32 of a head of keys): the rows stand four times in the tile, once for
// each warp's lanes of tensor memory, and a warp takes a quarter of a tile's keys for
// them, with a maximum, sum and accumulator of its own (the weights of the other quarters
// are zeros that stand there from the start).  So the chain from a tile's scores to its
// weights is a quarter as long.  The weights have columns of their own, so that the
// next scores are formed meanwhile.  The four are joined in shared memory at the end.
// Bound by the keys' and values' bytes.  Measured: a token of 8 samples over 32768 keys, 32 heads
// of 64 over 8, 75 us with the join (419 MB: 5.6 TB/s; with tiles of whole rows 106 us).
// ---------------------------------------------------------------------------
constexpr int kFewRows = 32;

template <int kBlocks>
struct FewCfg {
  static constexpr int kSlot = kBlocks * kBlock;
  static constexpr int kStages = 5;
  static constexpr int kResident = kBlocks == 1 ? 2 : 1;  // CTAs to an SM
  static constexpr int kThreads = 256;
  static constexpr int kSmem = (1 + kStages) * kSlot + 1024 + 1024 + 1024 + kMaxKeyTiles / 8;
  static constexpr int kS = 0, kP = 128, kO = 192, kTmem = kBlocks == 1 ? 256 : 512;
  static_assert(kResident * (kSmem + 1024) <= 228 * 1024, "shared memory of a CTA");
  static_assert(4 * kFewRows * 64 * kBlocks * 4 <= kStages * kSlot, "the joined rows");
};

template <int kBlocks, int kForm>
__global__ void __launch_bounds__(FewCfg<kBlocks>::kThreads, FewCfg<kBlocks>::kResident)
    attention_few_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, const TcArgs x) {
  using Cfg = FewCfg<kBlocks>;
  constexpr int kStages = Cfg::kStages, kPart = 32;
  const AttnArgs& a = x.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = align_1024(smem_raw);
  uint8_t* ring = qs + Cfg::kSlot;
  uint8_t* rest = ring + kStages * Cfg::kSlot;
  uint64_t* full = reinterpret_cast<uint64_t*>(rest);
  uint64_t* empty = full + kStages;
  uint64_t* qfull = empty + kStages;
  uint64_t* sfull = qfull + 1;
  uint64_t* sread = sfull + 1;
  uint64_t* pfull = sread + 1;
  uint64_t* pvfull = pfull + 1;
  uint64_t* drain = pvfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* ext = reinterpret_cast<int*>(tmem_slot + 2);
  int* done = ext + 3;  // [4]: the warps that came to their end
  float2* stats = reinterpret_cast<float2*>(rest + 512);  // [4][kFewRows]
  uint32_t* bits = reinterpret_cast<uint32_t*>(rest + 512 + 1024);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int bhs = a.B * a.Hkv;
  const int bh = blockIdx.x % bhs, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(qfull, 1);
    mbar_init(sfull, 1);
    mbar_init(sread, 4);
    mbar_init(pfull, 4);
    mbar_init(pvfull, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
    ext[0] = 0;
    ext[1] = 0x7fffffff;
    ext[2] = -1;
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const int tok = lane / a.G, h = hk * a.G + lane - tok * a.G;
  const bool mine = warp < 4 && tok < a.Tq;
  RowSees see = {0, 0, -1};
  Extent e = {};
  if (warp < 4) {
    if (mine) see = attn_row(a, b, tok, keys, first);
    e = warp_extent(mine, see);
    if (warp == 0 && lane == 0) {
      ext[0] = e.max_lim;
      ext[1] = e.lo;
      ext[2] = e.hi;
    }
  }
  __syncthreads();
  const int top = ext[0];
  const int t0 = blockIdx.z * a.per_split, t1 = min(t0 + a.per_split, (top + kTile - 1) / kTile);
  const int words = max(0, (t1 + 31) / 32);
  key_tile_bits(a, b, t0, t1, ext[1], ext[2], bits, words);
  __syncthreads();

  if (warp == 4 && lane == 0) {
    Bits it(bits, words);
    Pos pos;
    int j = it.next(), issued = 0;
    const bool any = j >= 0;
    bool ok = true;
    if (any) {
      mbar_arrive_expect_tx(qfull, 4 * kBlocks * x.nt * a.G * 128);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < kBlocks; ++q)
          tma_load_4d(qs + q * kBlock + u * kFewRows * 128, &map_q, qfull, q * 64, hk * a.G, 0, b);
    }
    for (; j >= 0 && ok; j = it.next()) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!wait_bar<true>(&empty[pos.s], pos.parity ^ 1, DPRC_DEVERR_PIPE_EMPTY, abort_flag)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[pos.s], Cfg::kSlot);
#pragma unroll
        for (int q = 0; q < kBlocks; ++q)
          tma_load_4d(ring + pos.s * Cfg::kSlot + q * kBlock, kv == 0 ? &map_k : &map_v,
                      &full[pos.s], q * 64, hk, j * kTile, b);
        ++issued;
        pos.next(kStages);
      }
    }
    if (any) mbar_wait(qfull, 0, DPRC_DEVERR_PIPE_FULL);
    for (int k = issued - 1; k >= 0 && k >= issued - kStages; --k)
      mbar_wait(&full[k % kStages], (k / kStages) & 1, DPRC_DEVERR_PIPE_FULL);
  } else if (warp == 5) {
    const bool lead = elect_one() != 0;
    Bits it(bits, words);
    const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
    const uint32_t id_o = make_idesc_bf16(kTile, x.steps * 16, false, true);
    const uint64_t dq = desc_k(smem_u32(qs));
    const uint64_t dk = desc_k(smem_u32(ring)), dv = desc_mn(smem_u32(ring));
    Pos pos;
    int j = it.next(), n = 0;
    bool ok = j >= 0, issued = false;
    const auto filled = [&](const Pos& p) {
      const bool f = wait_all<false>(&full[p.s], p.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
      tc_fence_after();
      return f;
    };
    const auto scores_of = [&](const Pos& p) {
      mma_width<kBlocks, false>(lead, tmem + Cfg::kS, dq, dk + ((p.s * Cfg::kSlot) >> 4), id_s,
                                x.steps);
      commit(lead, sfull);
      commit(lead, &empty[p.s]);
    };
    ok = ok && wait_all<false>(qfull, 0, DPRC_DEVERR_PIPE_FULL, abort_flag) && filled(pos);
    if (ok) {
      issued = true;
      scores_of(pos);
      pos.next(kStages);
    }
    while (ok && j >= 0) {
      j = it.next();
      const Pos v = pos;
      pos.next(kStages);
      if (j >= 0) {
        ok = filled(pos) && wait_all<false>(sread, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
        if (!ok) break;
        tc_fence_after();
        scores_of(pos);
        pos.next(kStages);
      }
      ok = filled(v) && wait_all<false>(pfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
      if (!ok) break;
      tc_fence_after();
      mma_rows(lead, tmem + Cfg::kO, tmem + Cfg::kP, dv + ((v.s * Cfg::kSlot) >> 4), id_o, n > 0);
      commit(lead, pvfull);
      commit(lead, &empty[v.s]);
      ++n;
    }
    if (issued && lead) umma_drain(drain, kWaitLimitNs);
  } else if (warp < 4) {
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t ts = tmem + lanes + Cfg::kS + warp * kPart;
    const uint32_t tp = tmem + lanes + Cfg::kP, to = tmem + lanes + Cfg::kO;
    const float slope2 = (kForm & 1) != 0 && a.slopes != nullptr && mine ? a.slopes[h] * kLog2e : 0.f;
    const int* docs = a.docs != nullptr ? a.docs + static_cast<long long>(b) * a.Tk : nullptr;
    const int cols = x.steps * 16;
    {
      uint32_t zero[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) zero[u] = 0u;
      tmem_st_32cols(tp, zero);
      tmem_st_32cols(tp + 32, zero);
      tmem_st_wait();
    }
    Bits it(bits, words);
    Pos vpos;
    vpos.next(kStages);
    float m = -INFINITY, l = 0.f;
    int n = 0;
    bool ok = true;
    for (int j = it.next(); j >= 0; j = it.next(), ++n) {
      ok = wait_warp<false>(sfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const int j0 = j * kTile, jq = j0 + warp * kPart;
      bool dirty = j0 + kTile > top, by_doc = false;
      if (docs != nullptr) {
        const DocSpan s = key_tile_docs(a, b, j);
        by_doc = s.pad || s.lo != s.hi || e.lo != s.lo || e.hi != s.lo;
        dirty = dirty || s.pad;
      }
      float z[kPart];
      tmem_ld_32cols(ts, z);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sread);
      scores<kForm>(x, z, slope2, static_cast<float>(see.pos - jq));
      if (jq + kPart > e.min_lim || by_doc) hide(z, see, docs, jq, a.Tk, by_doc);
      const float mul = kForm == 0 ? x.c : 1.f;
      float mt = z[0];
#pragma unroll
      for (int c = 1; c + 2 <= kPart; c += 2) mt = max3(mt, z[c], z[c + 1]);
      mt = fmaxf(mt, z[kPart - 1]) * mul;
      const bool grow = mt > m + kLazy || (m == -INFINITY && mt > m);
      const bool rescale = __any_sync(0xffffffffu, grow);
      const float f = grow ? ex2(m - mt) : 1.f;
      if (grow) m = mt;
      l *= f;
      const float off = m == -INFINITY ? 0.f : -m;
      float sum = 0.f;
      uint32_t p[kPart / 2];
#pragma unroll
      for (int c = 0; c < kPart; c += 2) {
        const float p0 = ex2(fmaf(z[c], mul, off)), p1 = ex2(fmaf(z[c + 1], mul, off));
        sum += p0 + p1;
        p[c / 2] = pack_bf16(p0, p1);
      }
      l += sum;
      // the product of the tile before has read its weights and written its sums
      if (n > 0) {
        ok = wait_warp<false>(pvfull, (n - 1) & 1, DPRC_DEVERR_ACCUM, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (rescale) {
          for (int c = 0; c < cols; c += 16) {
            float o[16];
            tmem_ld_16cols(to + c, o);
            uint32_t u[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) u[q] = __float_as_uint(o[q] * f);
            tmem_st_16cols(to + c, u);
          }
        }
      }
      tmem_st_16cols(tp + warp * (kPart / 2), p);
      tmem_st_wait();
      if (dirty) {
        // values that no row of the CTA sees may be anything, and 0 times NaN is NaN
        ok = wait_warp<false>(&full[vpos.s], vpos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
        if (!ok) break;
        const int r = threadIdx.x, key = j0 + r;
        if (key >= top || (docs != nullptr && docs[key] < 0))
          zero_row<kBlocks>(ring + vpos.s * Cfg::kSlot, r);
        fence_proxy_async_smem();
      }
      vpos.next(kStages);
      vpos.next(kStages);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull);
    }
    if (n > 0 && ok) ok = wait_warp<false>(pvfull, (n - 1) & 1, DPRC_DEVERR_ACCUM, abort_flag);
    tc_fence_after();
    // the four quarters: their maxima and sums, then their sums of values
    stats[warp * kFewRows + lane] = make_float2(m, l);
    if (lane == 0) done[warp] = ok ? 1 : 0;
    named_bar_sync(1, 128);
    ok = (done[0] & done[1] & done[2] & done[3]) != 0;  // the same for the four
    const float2 s0 = stats[lane], s1 = stats[kFewRows + lane], s2 = stats[2 * kFewRows + lane],
                 s3 = stats[3 * kFewRows + lane];
    const float all = fmaxf(fmaxf(s0.x, s1.x), fmaxf(s2.x, s3.x));
    const float at = all == -INFINITY ? 0.f : all, f = ex2(m - at);
    const float total =
        s0.y * ex2(s0.x - at) + s1.y * ex2(s1.x - at) + s2.y * ex2(s2.x - at) + s3.y * ex2(s3.x - at);
    const int rows = a.Tq * a.G;
    float* joined = reinterpret_cast<float*>(ring);  // [4][kFewRows][cols]
    if (ok && n > 0) {
      for (int c = 0; c < cols; c += 16) {
        float o[16];
        tmem_ld_16cols(to + c, o);
        if (mine) {
#pragma unroll
          for (int q = 0; q < 16; q += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) o[q + u] *= f;
            store_row<4>(joined + (warp * kFewRows + lane) * cols + c + q, o + q);
          }
        }
        __syncwarp();
      }
    }
    named_bar_sync(1, 128);
    if (ok) {
      const bool parts = a.splits > 1;
      const long long prow = (static_cast<long long>(blockIdx.z) * bhs + bh) * rows;
      if (warp == 0 && mine) {
        stats[lane].y = parts ? 1.f : total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
        if (parts) a.part_stats[prow + lane] = make_float2(all, total);
        else if (a.lse != nullptr)
          a.lse[(static_cast<long long>(b) * a.H + h) * a.Tq + tok] = all * kLn2 + logf(total);
      }
      named_bar_sync(1, 128);
      const int eights = a.D / 8;
      for (int i = threadIdx.x; i < rows * eights; i += 128) {
        const int r = i / eights, c = (i - r * eights) * 8, t = r / a.G;
        float o[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          o[u] = 0.f;
          if (n > 0)
#pragma unroll
            for (int q = 0; q < 4; ++q) o[u] += joined[(q * kFewRows + r) * cols + c + u];
          o[u] *= stats[r].y;
        }
        if (parts) {
          store_row<4>(a.part + (prow + r) * a.D + c, o);
          store_row<4>(a.part + (prow + r) * a.D + c + 4, o + 4);
        } else {
          __nv_bfloat16* out =
              static_cast<__nv_bfloat16*>(a.out) +
              ((static_cast<long long>(b) * a.Tq + t) * a.H + hk * a.G + r - t * a.G) * a.D;
          store_row<8>(out + c, o);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmem);
  }
}

template <int kBlocks, int kForm>
cudaError_t launch_few(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                       const TcArgs& x, cudaStream_t s) {
  constexpr int bytes = FewCfg<kBlocks>::kSmem;
  const cudaError_t e = allow_smem<attention_few_tc_kernel<kBlocks, kForm>>(bytes);
  if (e != cudaSuccess) return e;
  return launch_after(attention_few_tc_kernel<kBlocks, kForm>,
                      dim3(x.a.B * x.a.Hkv, 1, x.a.splits), FewCfg<kBlocks>::kThreads, 1, s, bytes,
                      q, k, v, x);
}
template <int kBlocks>
cudaError_t launch_few_form(int form, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, const TcArgs& x, cudaStream_t s) {
  if (form == 0) return launch_few<kBlocks, 0>(q, k, v, x, s);
  if (form == 1) return launch_few<kBlocks, 1>(q, k, v, x, s);
  if (form == 2) return launch_few<kBlocks, 2>(q, k, v, x, s);
  return launch_few<kBlocks, 3>(q, k, v, x, s);
}

// ---------------------------------------------------------------------------
// Backward.  Sixteen warps share a tile: a thread has a lane and 32 of the 128
// columns (with eight and 64 columns, two warps a scheduler, the chain of a thread's
// operations was what the kernels waited for: issue slots 35 % used).  Its weights go back
// into the first half of the columns that it read (a product's steps of 16 take their
// operand from there, mma_parts), so no other thread's scores are overwritten.  While the
// weights' gradient is formed, the tensor core forms the next scores; while those are
// taken to the exponential, the gradients' products and the next dP.
// Bound by the chain scores, exponential, weights, products and by the operations on each pair, at
// 31 to 39 % of the tensor pipe.  Measured, causal, both kernels with the row sums, as five
// products a pair: 4 x 4096 of 32 heads of 64 over 8, 1.21 ms, 0.57 PFLOP/s; 2 x 4096 of 16
// heads of 128 over 4, 409 us, 0.83; packed documents of 4 x 4096, 565 us.
// ---------------------------------------------------------------------------
constexpr int kGradWarps = 16, kGradThreads = 32 * (kGradWarps + 4);
constexpr int kPart = kTile * 4 / kGradWarps;  // columns of a thread
static_assert(kPart == 32, "columns of a load");

__device__ __forceinline__ void mma_parts(bool lead, uint32_t acc, uint32_t a_tmem, uint64_t b,
                                           uint32_t idesc, bool accumulate) {
  if (!lead) return;
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
    umma_bf16_ts(acc, a_tmem + (k / (kPart / 16)) * kPart + (k % (kPart / 16)) * 8, b + ((k * 2048) >> 4), idesc,
                 accumulate || k > 0 ? 1u : 0u);
}

// This thread's columns: ds = w (dp - delta), 0 where `bits` says that the key is not
// seen (dp may be anything there), as bf16 into the first 32 of them.
// delta(c, d): those of columns c to c + 3.
template <typename Delta>
__device__ __forceinline__ void put_ds(uint32_t taddr, const float (&w)[kPart], bool masked,
                                       const uint32_t (&bits)[kPart / 32], Delta delta) {
#pragma unroll
  for (int c0 = 0; c0 < kPart; c0 += 32) {
    float dp[32];
    tmem_ld_32cols(taddr + c0, dp);
#pragma unroll
    for (int u = 0; u < 32; u += 4) {
      float d[4];
      delta(c0 + u, d);
#pragma unroll
      for (int k = 0; k < 4; ++k) dp[u + k] = w[c0 + u + k] * (dp[u + k] - d[k]);
    }
    if (masked) {
#pragma unroll
      for (int u = 0; u < 32; ++u)
        if (!((bits[c0 / 32] >> u) & 1u)) dp[u] = 0.f;
    }
    uint32_t p[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) p[u] = pack_bf16(dp[2 * u], dp[2 * u + 1]);
    tmem_st_16cols(taddr + c0 / 2, p);
  }
}

// Eight values to an address of any alignment of the type.
__device__ __forceinline__ void store_any(__nv_bfloat16* p, const float* v) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if (at % 16 == 0) {
    store_row<8>(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __float2bfloat16_rn(v[e]);
  }
}

// Rows of a gradient from tensor memory: this thread's lane, and of its 16-column pieces
// those that are the part's.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) { store_any(p, v); }
__device__ __forceinline__ void store8(float* p, const float* v) {
  store_row<4>(p, v);
  store_row<4>(p + 4, v + 4);
}
template <typename T>
__device__ __forceinline__ void store_grad(T* out, bool mine, uint32_t taddr, int part, int cols,
                                           int D, float scale, bool any) {
  for (int c = part * 16; c < cols; c += kGradWarps * 4) {
    float o[16];
    if (any) {
      tmem_ld_16cols(taddr + c, o);
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q) o[q] = 0.f;
    }
    if (mine) {
#pragma unroll
      for (int q = 0; q < 16; q += 8) {
        if (c + q >= D) continue;
#pragma unroll
        for (int u = 0; u < 8; ++u) o[q + u] *= scale;
        store8(out + c + q, o + q);
      }
    }
    __syncwarp();  // (the next read is the whole warp's)
  }
}

template <int kBlocks>
struct DqCfg {
  static constexpr int kSlot = kBlocks * kBlock;
  static constexpr int kStages = kBlocks == 1 ? 8 : 4;
  static constexpr int kSmem = (2 + kStages) * kSlot + 1024 + 1024 + kMaxKeyTiles / 8;
  static constexpr int kS = 0, kDp = 128, kAcc = 256;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

template <int kBlocks, int kForm>
__global__ void __launch_bounds__(kGradThreads, 1)
    attention_dq_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_o,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v, const TcArgs x) {
  using Cfg = DqCfg<kBlocks>;
  constexpr int kStages = Cfg::kStages;
  const AttnArgs& a = x.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = align_1024(smem_raw);
  uint8_t* os = qs + Cfg::kSlot;
  uint8_t* ring = os + Cfg::kSlot;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * Cfg::kSlot);
  uint64_t* empty = full + kStages;
  uint64_t* qfull = empty + kStages;
  uint64_t* sfull = qfull + 1;
  uint64_t* sread = sfull + 1;
  uint64_t* dpfull = sread + 1;
  uint64_t* dsfull = dpfull + 1;
  uint64_t* ofull = dsfull + 1;
  uint64_t* drain = ofull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* bits = reinterpret_cast<uint32_t*>(ring + kStages * Cfg::kSlot + 512);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int bhs = a.B * a.Hkv;
  const int bh = blockIdx.x % bhs, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  const int grp = x.groups - 1 - blockIdx.x / bhs;  // the longest rows first
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(qfull, 1);
    mbar_init(sfull, 1);
    mbar_init(sread, kGradWarps);
    mbar_init(dpfull, 1);
    mbar_init(dsfull, kGradWarps);
    mbar_init(ofull, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_o);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == kGradWarps + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  const int keys = attn_keys(a, b), first = attn_first(a, b);
  const int r = threadIdx.x & (kTile - 1), part = warp >> 2;
  const int tt = r / a.G, tok = grp * x.nt + tt;
  const bool mine = warp < kGradWarps && tt < x.nt && tok < a.Tq;
  RowSees see = {0, 0, -1};
  Extent e = {};
  const Reach reach = reach_of(a, b, grp * x.nt, min((grp + 1) * x.nt, a.Tq), keys, first);
  const int top = reach.top, t1 = (top + kTile - 1) / kTile, words = (t1 + 31) / 32;
  key_tile_bits(a, b, 0, t1, reach.lo, reach.hi, bits, words);
  if (mine) see = attn_row(a, b, tok, keys, first);
  __syncthreads();
  if (warp < kGradWarps) e = warp_extent(mine, see);

  if (warp >= kGradWarps) {
    if (warp == kGradWarps && lane == 0) {
      Bits it(bits, words);
      Pos pos;
      int j = it.next(), issued = 0;
      const bool any = j >= 0;
      bool ok = true;
      if (any) {
        mbar_arrive_expect_tx(qfull, 2 * kBlocks * x.nt * a.G * 128);
#pragma unroll
        for (int q = 0; q < kBlocks; ++q) {
          tma_load_4d(qs + q * kBlock, &map_q, qfull, q * 64, hk * a.G, grp * x.nt, b);
          tma_load_4d(os + q * kBlock, &map_o, qfull, q * 64, hk * a.G, grp * x.nt, b);
        }
      }
      for (; j >= 0 && ok; j = it.next()) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (!wait_bar<false>(&empty[pos.s], pos.parity ^ 1, DPRC_DEVERR_PIPE_EMPTY, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[pos.s], Cfg::kSlot);
#pragma unroll
          for (int q = 0; q < kBlocks; ++q)
            tma_load_4d(ring + pos.s * Cfg::kSlot + q * kBlock, kv == 0 ? &map_k : &map_v,
                        &full[pos.s], q * 64, hk, j * kTile, b);
          ++issued;
          pos.next(kStages);
        }
      }
      if (any) mbar_wait(qfull, 0, DPRC_DEVERR_PIPE_FULL);
      for (int k = issued - 1; k >= 0 && k >= issued - kStages; --k)
        mbar_wait(&full[k % kStages], (k / kStages) & 1, DPRC_DEVERR_PIPE_FULL);
    } else if (warp == kGradWarps + 1) {
      // all lanes keep step, one issues: the descriptors stay in the warp's common registers
      const bool lead = elect_one() != 0;
      Bits it(bits, words);
      const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
      const uint32_t id_g = make_idesc_bf16(kTile, x.steps * 16, false, true);
      const uint64_t dq = desc_k(smem_u32(qs)), dO = desc_k(smem_u32(os));
      const uint64_t dk = desc_k(smem_u32(ring)), dkm = desc_mn(smem_u32(ring));
      Pos pos;
      int j = it.next(), n = 0;
      bool ok = j >= 0, issued = false;
      const auto filled = [&](const Pos& p) {
        const bool f = wait_all<false>(&full[p.s], p.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
        tc_fence_after();
        return f;
      };
      const auto scores_of = [&](const Pos& p) {
        mma_width<kBlocks, true>(lead, tmem + Cfg::kS, dq, dk + ((p.s * Cfg::kSlot) >> 4), id_s, x.steps);
        commit(lead, sfull);
      };
      const auto dp_of = [&](const Pos& p) {
        mma_width<kBlocks, true>(lead, tmem + Cfg::kDp, dO, dk + ((p.s * Cfg::kSlot) >> 4), id_s, x.steps);
        commit(lead, dpfull);
        commit(lead, &empty[p.s]);
      };
      Pos kp = pos;
      pos.next(kStages);
      Pos vp = pos;
      pos.next(kStages);
      ok = ok && wait_all<false>(qfull, 0, DPRC_DEVERR_PIPE_FULL, abort_flag) && filled(kp);
      if (ok) {
        issued = true;
        scores_of(kp);
        ok = filled(vp);
        if (ok) dp_of(vp);
      }
      while (ok && j >= 0) {
        j = it.next();
        Pos kn = kp, vn = vp;
        if (j >= 0) {
          kn = pos;
          pos.next(kStages);
          vn = pos;
          pos.next(kStages);
          ok = filled(kn) && wait_all<false>(sread, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
          if (!ok) break;
          tc_fence_after();
          scores_of(kn);
        }
        ok = wait_all<false>(dsfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
        if (!ok) break;
        tc_fence_after();
        mma_parts(lead, tmem + Cfg::kAcc, tmem + Cfg::kDp, dkm + ((kp.s * Cfg::kSlot) >> 4), id_g, n > 0);
        commit(lead, &empty[kp.s]);
        if (j >= 0) {
          ok = filled(vn);
          if (ok) dp_of(vn);
        } else {
          commit(lead, ofull);
        }
        kp = kn;
        vp = vn;
        ++n;
      }
      if (issued && lead) umma_drain(drain, kWaitLimitNs);
    }
  } else {
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + Cfg::kS + part * kPart;
    const uint32_t td = tmem + lanes + Cfg::kDp + part * kPart;
    const int h = hk * a.G + r - tt * a.G;
    const long long at = (static_cast<long long>(b) * a.H + h) * a.Tq + tok;
    const float slope2 = (kForm & 1) != 0 && a.slopes != nullptr && mine ? a.slopes[h] * kLog2e : 0.f;
    const float lse = mine ? a.lse_in[at] : 0.f, delta = mine ? a.delta[at] : 0.f;
    const float off = lse == -INFINITY ? 0.f : -lse * kLog2e;
    const int* docs = a.docs != nullptr ? a.docs + static_cast<long long>(b) * a.Tk : nullptr;
    Bits it(bits, words);
    Pos kpos;
    int n = 0;
    bool ok = true;
    for (int j = it.next(); j >= 0; j = it.next(), ++n) {
      ok = wait_warp<false>(sfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const int j0 = j * kTile, jh = j0 + part * kPart;
      bool dirty = j0 + kTile > top, by_doc = false;
      if (docs != nullptr) {
        const DocSpan s = key_tile_docs(a, b, j);
        by_doc = s.pad || s.lo != s.hi || e.lo != s.lo || e.hi != s.lo;
        dirty = dirty || s.pad;
      }
      float z[kPart];
      tmem_ld_32cols(ts, z);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sread);
      uint32_t seen[kPart / 32];
#pragma unroll
      for (int q = 0; q < kPart / 32; ++q) seen[q] = 0xffffffffu;
      const bool masked = jh + kPart > e.min_lim || by_doc;
      if (masked) seen_bits(seen, see, docs, jh, a.Tk, by_doc);
      weights<kForm>(x, z, slope2, static_cast<float>(see.pos - jh), off);
      if (dirty && part == 0) {
        // keys that no row of the CTA sees may be anything, and 0 times NaN is NaN
        ok = wait_warp<false>(&full[kpos.s], kpos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
        if (!ok) break;
        const int key = j0 + r;
        if (key >= top || (docs != nullptr && docs[key] < 0))
          zero_row<kBlocks>(ring + kpos.s * Cfg::kSlot, r);
        fence_proxy_async_smem();
      }
      kpos.next(kStages);
      kpos.next(kStages);
      ok = wait_warp<false>(dpfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
      if (!ok) break;
      tc_fence_after();
      put_ds(td, z, masked, seen, [&](int, float (&d)[4]) { d[0] = d[1] = d[2] = d[3] = delta; });
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dsfull);
    }
    if (n > 0 && ok) ok = wait_warp<false>(ofull, 0, DPRC_DEVERR_ACCUM, abort_flag);
    tc_fence_after();
    if (ok)
      store_grad(static_cast<__nv_bfloat16*>(a.dQ) + b * a.dqb + tok * a.dqt + h * a.dqh, mine,
                 tmem + lanes + Cfg::kAcc, part, x.steps * 16, a.D, a.scale, n > 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kGradWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// What the keys' kernel reads of a tile's rows, kRowStages tiles in turn.
struct RowStage {
  float off[kTile];    // -lse log2(e); -inf: a row that sees nothing, or is none
  float delta[kTile];
  float slope2[kTile];
  float pos[kTile];    // against the first key of the tile
  int lim[kTile];
  int doc[kTile];
  int min_lim, lo, hi, dirty;
};
constexpr int kMaxRowTiles = 1 << 16;
constexpr int kRowStages = 4;

template <int kBlocks>
struct DkvCfg {
  static constexpr int kSlot = kBlocks * kBlock;
  static constexpr int kStages = kBlocks == 1 ? 6 : 4;
  static constexpr int kBits = kMaxRowTiles / 8;
  static constexpr int kSmem =
      (2 + kStages) * kSlot + 1024 + 512 + kBits + kRowStages * static_cast<int>(sizeof(RowStage));
  static constexpr int kS = 0, kDp = 128, kDv = 256, kDk = 384;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

template <int kBlocks, int kForm>
__global__ void __launch_bounds__(kGradThreads, 1)
    attention_dkv_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_o,
                            const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, const TcArgs x) {
  using Cfg = DkvCfg<kBlocks>;
  constexpr int kStages = Cfg::kStages;
  const AttnArgs& a = x.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ks = align_1024(smem_raw);
  uint8_t* vs = ks + Cfg::kSlot;
  uint8_t* ring = vs + Cfg::kSlot;
  uint8_t* rest = ring + kStages * Cfg::kSlot;
  uint64_t* full = reinterpret_cast<uint64_t*>(rest);
  uint64_t* empty = full + kStages;
  uint64_t* kvfull = empty + kStages;
  uint64_t* sfull = kvfull + 1;
  uint64_t* pfull = sfull + 1;
  uint64_t* dpfull = pfull + 1;
  uint64_t* dsfull = dpfull + 1;
  uint64_t* rfull = dsfull + 1;            // [kRowStages]
  uint64_t* rempty = rfull + kRowStages;   // [kRowStages]
  uint64_t* ofull = rempty + kRowStages;
  uint64_t* drain = ofull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* bits = reinterpret_cast<uint32_t*>(rest + 512);
  RowStage* stages = reinterpret_cast<RowStage*>(rest + 512 + Cfg::kBits);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int bhs = a.B * a.Hkv;
  const int bh = blockIdx.x % bhs, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  const int jt = blockIdx.x / bhs, j0 = jt * kTile;  // (the first keys have the most rows)
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(kvfull, 1);
    mbar_init(sfull, 1);
    mbar_init(pfull, kGradWarps);
    mbar_init(dpfull, 1);
    mbar_init(dsfull, kGradWarps);
    for (int s = 0; s < kRowStages; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rempty[s], kGradWarps);
    }
    mbar_init(ofull, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_o);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == kGradWarps + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // rows of a slot behind the last whole token are never copied: zero, as they are
  // summed over
  const int tail = x.nt * a.G;
  for (int i = threadIdx.x; i < kStages * (kTile - tail); i += kGradThreads)
    zero_row<kBlocks>(ring + (i / (kTile - tail)) * Cfg::kSlot, tail + i % (kTile - tail));
  if (tail < kTile) fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  const int keys = attn_keys(a, b), first = attn_first(a, b);
  // tiles of rows that may see a key of this tile
  DocSpan kd = {0, 0, 0, 0};
  if (a.docs != nullptr) kd = key_tile_docs(a, b, jt);
  const int words = j0 < keys ? (x.row_tiles + 31) / 32 : 0;
  for (int w = warp; w < words; w += kGradThreads / 32) {
    const int i = w * 32 + lane, tok0 = i * x.nt;
    bool ok = tok0 < a.Tq && i % a.row_splits == static_cast<int>(blockIdx.z);
    if (ok) {
      const int tok1 = min(tok0 + x.nt, a.Tq) - 1;
      if (a.causal) {
        int see = first + tok1 + 1;
        if (a.prefix != nullptr) see = max(see, a.prefix[b]);
        ok = see > j0;
      }
      if (a.docs != nullptr) {
        const int spans = (a.Tk + kDocSpan - 1) / kDocSpan;
        const int p0 = max(0, first + tok0), p1 = min(a.Tk - 1, first + tok1);
        bool meets = false;
        for (int q = p0 / kDocSpan; p0 <= p1 && q <= p1 / kDocSpan; ++q) {
          const DocSpan s = a.spans[static_cast<long long>(b) * spans + q];
          meets = meets || (s.lo <= kd.hi && kd.lo <= s.hi);
        }
        ok = ok && meets;
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, ok);
    if (lane == 0 && DPRC_IN(w < kMaxRowTiles / 32)) bits[w] = m;
  }
  __syncthreads();

  if (warp >= kGradWarps) {
    if (warp == kGradWarps && lane == 0) {
      Bits it(bits, words);
      Pos pos;
      int i = it.next(), issued = 0;
      const bool any = i >= 0;
      bool ok = true;
      if (any) {
        mbar_arrive_expect_tx(kvfull, 2 * Cfg::kSlot);
#pragma unroll
        for (int q = 0; q < kBlocks; ++q) {
          tma_load_4d(ks + q * kBlock, &map_k, kvfull, q * 64, hk, j0, b);
          tma_load_4d(vs + q * kBlock, &map_v, kvfull, q * 64, hk, j0, b);
        }
      }
      for (; i >= 0 && ok; i = it.next()) {
#pragma unroll
        for (int qo = 0; qo < 2; ++qo) {
          if (!wait_bar<false>(&empty[pos.s], pos.parity ^ 1, DPRC_DEVERR_PIPE_EMPTY, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[pos.s], kBlocks * x.nt * a.G * 128);
#pragma unroll
          for (int q = 0; q < kBlocks; ++q)
            tma_load_4d(ring + pos.s * Cfg::kSlot + q * kBlock, qo == 0 ? &map_q : &map_o,
                        &full[pos.s], q * 64, hk * a.G, i * x.nt, b);
          ++issued;
          pos.next(kStages);
        }
      }
      if (any) mbar_wait(kvfull, 0, DPRC_DEVERR_PIPE_FULL);
      for (int k = issued - 1; k >= 0 && k >= issued - kStages; --k)
        mbar_wait(&full[k % kStages], (k / kStages) & 1, DPRC_DEVERR_PIPE_FULL);
    } else if (warp == kGradWarps + 1) {
      // all lanes keep step, one issues: the descriptors stay in the warp's common registers
      const bool lead = elect_one() != 0;
      Bits it(bits, words);
      const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
      const uint32_t id_g = make_idesc_bf16(kTile, x.steps * 16, false, true);
      const uint64_t dk = desc_k(smem_u32(ks)), dv = desc_k(smem_u32(vs));
      const uint64_t dr = desc_k(smem_u32(ring)), drm = desc_mn(smem_u32(ring));
      Pos pos;
      int i = it.next(), n = 0;
      bool ok = i >= 0, issued = false;
      const auto filled = [&](const Pos& p) {
        const bool f = wait_all<false>(&full[p.s], p.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
        tc_fence_after();
        return f;
      };
      const auto scores_of = [&](const Pos& p) {
        mma_width<kBlocks, true>(lead, tmem + Cfg::kS, dk, dr + ((p.s * Cfg::kSlot) >> 4), id_s, x.steps);
        commit(lead, sfull);
      };
      const auto dp_of = [&](const Pos& p) {
        mma_width<kBlocks, true>(lead, tmem + Cfg::kDp, dv, dr + ((p.s * Cfg::kSlot) >> 4), id_s, x.steps);
        commit(lead, dpfull);
      };
      Pos qp = pos;
      pos.next(kStages);
      Pos op = pos;
      pos.next(kStages);
      ok = ok && wait_all<false>(kvfull, 0, DPRC_DEVERR_PIPE_FULL, abort_flag) && filled(qp);
      if (ok) {
        issued = true;
        scores_of(qp);
        ok = filled(op);
        if (ok) dp_of(op);
      }
      while (ok && i >= 0) {
        i = it.next();
        Pos qn = qp, on = op;
        ok = wait_all<false>(pfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
        if (!ok) break;
        tc_fence_after();
        mma_parts(lead, tmem + Cfg::kDv, tmem + Cfg::kS, drm + ((op.s * Cfg::kSlot) >> 4), id_g, n > 0);
        commit(lead, &empty[op.s]);
        if (i >= 0) {
          qn = pos;
          pos.next(kStages);
          on = pos;
          pos.next(kStages);
          ok = filled(qn);
          if (!ok) break;
          scores_of(qn);
        }
        ok = wait_all<false>(dsfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
        if (!ok) break;
        tc_fence_after();
        mma_parts(lead, tmem + Cfg::kDk, tmem + Cfg::kDp, drm + ((qp.s * Cfg::kSlot) >> 4), id_g, n > 0);
        commit(lead, &empty[qp.s]);
        if (i >= 0) {
          ok = filled(on);
          if (ok) dp_of(on);
        } else {
          commit(lead, ofull);
        }
        qp = qn;
        op = on;
        ++n;
      }
      if (issued && lead) umma_drain(drain, kWaitLimitNs);
    } else if (warp == kGradWarps + 2) {
      // what the rows see, their statistics and where they stand
      Bits it(bits, words);
      int n = 0;
      // Rows that are none stand as zeros, and their weights are 0 whatever their bias (lse inf),
      // unless the tile has keys that nobody sees: those may be anything, and NaN stays NaN.
      int all = keys;
      if (a.causal) {
        all = min(keys, first + a.Tq);
        if (a.prefix != nullptr) all = max(all, min(keys, a.prefix[b]));
      }
      const int none = kd.pad || j0 + kTile > all ? 0 : 0x7fffffff;
      // a tile's values are on their way while the stage is waited for
      int tt[4];
      long long at[4];  // of a head's first token
      float slope[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = q * 32 + lane;
        tt[q] = r / a.G;
        const int h = hk * a.G + r - tt[q] * a.G;
        at[q] = (static_cast<long long>(b) * a.H + h) * a.Tq;
        slope[q] = (kForm & 1) != 0 && a.slopes != nullptr && tt[q] < x.nt ? a.slopes[h] * kLog2e : 0.f;
      }
      RowSees see[4];
      float lse[4], del[4];
      const auto fetch = [&](int i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int tok = i * x.nt + tt[q];
          see[q] = {0, none, -3};
          lse[q] = INFINITY;
          del[q] = 0.f;
          if (tt[q] < x.nt && tok < a.Tq) {
            lse[q] = ld_once(a.lse_in + at[q] + tok);
            del[q] = ld_once(a.delta + at[q] + tok);
            see[q] = attn_row(a, b, tok, keys, first);
          }
        }
      };
      int i = it.next();
      if (i >= 0) fetch(i);
      for (; i >= 0; ++n) {
        RowStage& st = stages[n % kRowStages];
        if (!wait_warp<false>(&rempty[n % kRowStages], ((n / kRowStages) & 1) ^ 1, DPRC_DEVERR_PIPE_EMPTY, abort_flag)) break;
        int min_lim = 0x7fffffff, lo = 0x7fffffff, hi = -1, dirty = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = q * 32 + lane;
          if (tt[q] < x.nt && i * x.nt + tt[q] < a.Tq && see[q].doc >= 0) {
            lo = min(lo, see[q].doc);
            hi = max(hi, see[q].doc);
          }
          dirty |= lse[q] == -INFINITY;
          min_lim = min(min_lim, see[q].lim);
          st.off[r] = lse[q] == -INFINITY ? -INFINITY : -lse[q] * kLog2e;
          st.delta[r] = del[q];
          st.slope2[r] = slope[q];
          st.pos[r] = static_cast<float>(see[q].pos - j0);
          st.lim[r] = see[q].lim;
          st.doc[r] = see[q].doc;
        }
        i = it.next();
        if (i >= 0) fetch(i);
        min_lim = __reduce_min_sync(0xffffffffu, min_lim);
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        dirty = __reduce_or_sync(0xffffffffu, dirty);
        if (lane == 0) {
          st.min_lim = min_lim;
          st.lo = lo;
          st.hi = hi;
          st.dirty = dirty;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rfull[n % kRowStages]);
      }
    }
  } else {
    const int r = threadIdx.x & (kTile - 1), part = warp >> 2, key = j0 + r;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + Cfg::kS + part * kPart;
    const uint32_t td = tmem + lanes + Cfg::kDp + part * kPart;
    const float keyf = static_cast<float>(r);
    const int kdoc =
        a.docs != nullptr ? (key < a.Tk ? a.docs[static_cast<long long>(b) * a.Tk + key] : -2) : 0;
    const int kdoc0 = __shfl_sync(0xffffffffu, kdoc, 0);
    const bool one_doc = __all_sync(0xffffffffu, kdoc == kdoc0);
    const int last_key = j0 + (warp & 3) * 32 + 31;
    Bits it(bits, words);
    Pos pos;
    int n = 0;
    bool ok = true;
    for (int i = it.next(); i >= 0; i = it.next(), ++n) {
      const RowStage& st = stages[n % kRowStages];
      const int c0 = part * kPart;
      ok = wait_warp<false>(&rfull[n % kRowStages], (n / kRowStages) & 1, DPRC_DEVERR_PIPE_FULL, abort_flag) &&
           wait_warp<false>(sfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
      if (!ok) break;
      tc_fence_after();
      float z[kPart];
      tmem_ld_32cols(ts, z);
      const bool by_doc =
          a.docs != nullptr && (!one_doc || st.lo != kdoc0 || st.hi != kdoc0);
      const bool masked = last_key >= st.min_lim || by_doc;
      uint32_t seen[kPart / 32];
#pragma unroll
      for (int q = 0; q < kPart / 32; ++q) seen[q] = 0xffffffffu;
      if (masked) {
#pragma unroll
        for (int q = 0; q < kPart / 32; ++q) {
          uint32_t m = 0u;
#pragma unroll 1
          for (int u = 0; u < 32; u += 4) {
            const int4 l = *reinterpret_cast<const int4*>(&st.lim[c0 + q * 32 + u]);
            m |= (key < l.x ? 1u << u : 0u) | (key < l.y ? 2u << u : 0u) |
                 (key < l.z ? 4u << u : 0u) | (key < l.w ? 8u << u : 0u);
          }
          if (by_doc) m &= same_docs(kdoc, st.doc[c0 + q * 32 + lane]);
          seen[q] = m;
        }
      }
      // P into the scores' place; z becomes P (1 - t^2)
#pragma unroll
      for (int q = 0; q < kPart / 32; ++q) {
        uint32_t p[16];
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
          const int c = q * 32 + u;
          float of[4], sl[4] = {0.f, 0.f, 0.f, 0.f}, ps[4] = {0.f, 0.f, 0.f, 0.f};
          ld_shared4(&st.off[c0 + c], of);
          if constexpr ((kForm & 1) != 0) {
            ld_shared4(&st.slope2[c0 + c], sl);
            ld_shared4(&st.pos[c0 + c], ps);
          }
          float w[4];
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float dist[2] = {fabsf(ps[k] - keyf), fabsf(ps[k + 1] - keyf)};
            weights2<kForm>(x, &z[c + k], &w[k], &sl[k], dist, &of[k]);
          }
          p[u / 2] = pack_bf16(w[0], w[1]);
          p[u / 2 + 1] = pack_bf16(w[2], w[3]);
        }
        if (masked) {
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if (!((seen[q] >> u) & 1u)) {
              z[q * 32 + u] = 0.f;
              p[u / 2] &= u & 1 ? 0x0000ffffu : 0xffff0000u;
            }
        }
        tmem_st_16cols(ts + q * 16, p);
      }
      tmem_st_wait();
      if (st.dirty) {
        // rows that see nothing (also those whose position does, but of whose document no key
        // is below the length) may be anything, and 0 times NaN is NaN: their queries
        // and gradients are summed over (dP, which reads them too, is complete)
        ok = wait_warp<false>(dpfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (part == 0) {
          Pos op = pos;
          op.next(kStages);
          ok = wait_warp<false>(&full[pos.s], pos.parity, DPRC_DEVERR_PIPE_FULL, abort_flag) &&
               wait_warp<false>(&full[op.s], op.parity, DPRC_DEVERR_PIPE_FULL, abort_flag);
          if (!ok) break;
          if (st.off[r] == -INFINITY) {
            zero_row<kBlocks>(ring + pos.s * Cfg::kSlot, r);
            zero_row<kBlocks>(ring + op.s * Cfg::kSlot, r);
          }
          fence_proxy_async_smem();
        }
      }
      pos.next(kStages);
      pos.next(kStages);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull);
      ok = wait_warp<false>(dpfull, n & 1, DPRC_DEVERR_ACCUM, abort_flag);
      if (!ok) break;
      tc_fence_after();
      put_ds(td, z, masked, seen, [&](int c, float (&d)[4]) { ld_shared4(&st.delta[c0 + c], d); });
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(dsfull);
        mbar_arrive(&rempty[n % kRowStages]);
      }
    }
    if (n > 0 && ok) ok = wait_warp<false>(ofull, 0, DPRC_DEVERR_ACCUM, abort_flag);
    tc_fence_after();
    if (ok) {
      const bool mine = key < a.Tk;
      const int cols = x.steps * 16;
      if (a.row_splits > 1) {
        float* out = a.key_part +
                     ((static_cast<long long>(blockIdx.z) * bhs + bh) * a.Tk + key) * 2 * a.D;
        store_grad(out, mine, tmem + lanes + Cfg::kDk, part, cols, a.D, a.scale, n > 0);
        store_grad(out + a.D, mine, tmem + lanes + Cfg::kDv, part, cols, a.D, 1.f, n > 0);
      }
      if (a.row_splits == 1 && a.dV != nullptr)
        store_grad(static_cast<__nv_bfloat16*>(a.dV) + b * a.dvb + key * a.dvt + hk * a.dvh, mine,
                   tmem + lanes + Cfg::kDv, part, cols, a.D, 1.f, n > 0);
      if (a.row_splits == 1 && a.dK != nullptr)
        store_grad(static_cast<__nv_bfloat16*>(a.dK) + b * a.dkb + key * a.dkt + hk * a.dkh, mine,
                   tmem + lanes + Cfg::kDk, part, cols, a.D, a.scale, n > 0);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kGradWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct GradMaps {
  CUtensorMap q, o, k, v;
};

template <int kBlocks, int kForm>
cudaError_t launch_grad(const GradMaps& m, const TcArgs& x, cudaStream_t s) {
  const int bhs = x.a.B * x.a.Hkv;
  cudaError_t e = cudaSuccess;
  if (x.a.dQ != nullptr) {
    constexpr int bytes = DqCfg<kBlocks>::kSmem;
    e = allow_smem<attention_dq_tc_kernel<kBlocks, kForm>>(bytes);
    if (e != cudaSuccess) return e;
    e = launch_after(attention_dq_tc_kernel<kBlocks, kForm>, dim3(bhs * x.groups), kGradThreads, 1, s,
                     bytes, m.q, m.o, m.k, m.v, x);
    if (e != cudaSuccess) return e;
  }
  if (x.a.dK == nullptr && x.a.dV == nullptr) return e;
  constexpr int bytes = DkvCfg<kBlocks>::kSmem;
  e = allow_smem<attention_dkv_tc_kernel<kBlocks, kForm>>(bytes);
  if (e != cudaSuccess) return e;
  return launch_after(attention_dkv_tc_kernel<kBlocks, kForm>,
                      dim3(bhs * ((x.a.Tk + kTile - 1) / kTile), 1, x.a.row_splits), kGradThreads, 1, s, bytes, m.q, m.o,
                      m.k, m.v, x);
}

template <int kBlocks>
cudaError_t launch_grad_form(int form, const GradMaps& m, const TcArgs& x, cudaStream_t s) {
  if (form == 0) return launch_grad<kBlocks, 0>(m, x, s);
  if (form == 1) return launch_grad<kBlocks, 1>(m, x, s);
  if (form == 2) return launch_grad<kBlocks, 2>(m, x, s);
  return launch_grad<kBlocks, 3>(m, x, s);
}

// A tensor [B][T][H][D] as boxes of 64 of the width, `heads` heads and `tokens` tokens.
bool map_of(CUtensorMap* m, const void* p, long long B, long long T, long long H, long long D,
            long long sb, long long st, long long sh, int heads, int tokens) {
  const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(H),
                            static_cast<uint64_t>(T), static_cast<uint64_t>(B)};
  // (an axis of one has any stride)
  const uint64_t strides[3] = {static_cast<uint64_t>(H > 1 ? sh : 8),
                               static_cast<uint64_t>(T > 1 ? st : 8),
                               static_cast<uint64_t>(B > 1 ? sb : 8)};
  const uint32_t box[4] = {64, static_cast<uint32_t>(heads), static_cast<uint32_t>(tokens), 1};
  return make_tmap_4d_bf16(m, p, dims, strides, box);
}

TcArgs tc_args(const AttnArgs& a, int tiles) {
  TcArgs x;
  x.a = a;
  x.nt = kTile / a.G;
  x.row_tiles = (a.Tq + x.nt - 1) / x.nt;
  x.groups = (x.row_tiles + tiles - 1) / tiles;
  x.steps = (a.D + 15) / 16;
  x.c = a.scale * kLog2e;
  // (finite, so that a product of 0 stays one)
  x.c_cap = a.cap > 0.f
      ? std::clamp(2.f * a.scale * kLog2e / a.cap, -FLT_MAX, FLT_MAX) : 0.f;
  x.cap2 = a.cap * kLog2e;
  return x;
}

int form_of(const AttnArgs& a) {
  if (a.cap > 0.f) return a.slopes != nullptr ? 3 : 2;
  return a.slopes != nullptr || !(a.scale > 0.f) ? 1 : 0;  // (1: any sign of the scale)
}

bool strides_fit(const int64_t* s, int64_t B, int64_t T, int64_t H) {
  const int64_t n[3] = {B, T, H};
  for (int k = 0; k < 3; ++k)
    if (n[k] > 1 && (s[k] < 8 || s[k] % 8 != 0 || s[k] >= (int64_t(1) << 38))) return false;
  return true;
}
bool address_fits(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

// The tanh by an exponential is good to 2^-22, a score to 2^-22 of the cap: up to this cap the
// weights are better than their half step in bf16, 2^-9.
constexpr float kMaxTcCap = 4096.f;

// What the tensor copies take: 16-byte boundaries, and a group's heads in a tile.
bool attention_tc_takes(const AttentionCall& c) {
  const int64_t G = c.H / c.Hkv;
  return c.dtype == DPRC_BF16 && c.cap <= kMaxTcCap && c.D % 8 == 0 && G <= kTile && c.Tk > 0 && c.Tq > 0 &&
         c.Tq <= (int64_t(1) << 16) * (kTile / G) && address_fits(c.Q) && address_fits(c.K) &&
         address_fits(c.V) && strides_fit(c.qs, c.B, c.Tq, c.H) &&
         strides_fit(c.ks, c.B, c.Tk, c.Hkv) && strides_fit(c.vs, c.B, c.Tk, c.Hkv) &&
         c.B * c.Hkv * ((c.Tq + kTile / G - 1) / (kTile / G)) < (int64_t(1) << 31);
}

bool attention_tc_takes_grad(const AttentionGradCall& c) {
  return attention_tc_takes(c.f) && address_fits(c.dO) &&
         strides_fit(c.dos, c.f.B, c.f.Tq, c.f.H);
}

int attention_tc_rows_grad(const AttentionCall& c) {
  const int G = static_cast<int>(c.H / c.Hkv);
  return kTile / G * G;
}

int attention_tc_rows(const AttentionCall& c) {
  const int G = static_cast<int>(c.H / c.Hkv), nt = kTile / G;
  return c.Tq > nt ? 2 * nt * G : nt * G;
}

int attention_tc_resident(const AttentionCall& c) {
  const int G = static_cast<int>(c.H / c.Hkv);
  if (c.Tq * G <= kFewRows) return c.D <= 64 ? 304 : 152;
  return c.Tq > kTile / G ? 152 : 304;
}

cudaError_t launch_attention_tc(const AttnArgs& a, cudaStream_t s) {
  const bool few = a.Tq * a.G <= kFewRows;
  const int nt = (few ? kFewRows : kTile) / a.G, tiles = a.Tq > nt ? 2 : 1, form = form_of(a);
  TcArgs x = tc_args(a, tiles);
  x.nt = nt;
  CUtensorMap q, k, v;
  if (!map_of(&q, a.Q, a.B, a.Tq, a.H, a.D, a.qb, a.qt, a.qh, a.G, nt) ||
      !map_of(&k, a.K, a.B, a.Tk, a.Hkv, a.D, a.kb, a.kt, a.kh, 1, kTile) ||
      !map_of(&v, a.V, a.B, a.Tk, a.Hkv, a.D, a.vb, a.vt, a.vh, 1, kTile))
    return cudaErrorInvalidValue;
  if (few)
    return a.D <= 64 ? launch_few_form<1>(form, q, k, v, x, s)
                     : launch_few_form<2>(form, q, k, v, x, s);
  if (a.D <= 64)
    return tiles == 2 ? launch_fwd_form<1, 2>(form, q, k, v, x, s)
                      : launch_fwd_form<1, 1>(form, q, k, v, x, s);
  return tiles == 2 ? launch_fwd_form<2, 2>(form, q, k, v, x, s)
                    : launch_fwd_form<2, 1>(form, q, k, v, x, s);
}

cudaError_t launch_attention_grad_tc(const AttnArgs& a, cudaStream_t s) {
  const TcArgs x = tc_args(a, 1);
  GradMaps m;
  if (!map_of(&m.q, a.Q, a.B, a.Tq, a.H, a.D, a.qb, a.qt, a.qh, a.G, x.nt) ||
      !map_of(&m.o, a.dO, a.B, a.Tq, a.H, a.D, a.dob, a.dot, a.doh, a.G, x.nt) ||
      !map_of(&m.k, a.K, a.B, a.Tk, a.Hkv, a.D, a.kb, a.kt, a.kh, 1, kTile) ||
      !map_of(&m.v, a.V, a.B, a.Tk, a.Hkv, a.D, a.vb, a.vt, a.vh, 1, kTile))
    return cudaErrorInvalidValue;
  const int form = form_of(a);
  return a.D <= 64 ? launch_grad_form<1>(form, m, x, s) : launch_grad_form<2>(form, m, x, s);
}

cudaError_t read_device_error_attention(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

}  // namespace dprc
