// What the attention kernels share: the arguments, what a row sees, and the
// partial results of rows whose keys are split.
//
// The rows of a product are the queries of all heads that share a head of keys,
// token by token: row p is token p / G and head p % G of the G = H / Hkv.  So a tile
// of keys is read once for all of them, a few tokens still fill a tile, and the
// sums over the heads of a group (gradients of keys and values) are sums over rows.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dprc {

// What a span of kDocSpan keys holds of documents: the least and greatest id
// (of those that are no padding) and whether there is padding.
constexpr int kDocSpan = 64;
struct DocSpan {
  int lo, hi, pad, unused;
};

struct AttnArgs {
  const void *Q, *K, *V;
  long long qb, qt, qh, kb, kt, kh, vb, vt, vh;  // strides in elements
  int B, Tq, Tk, H, Hkv, D, G;
  float scale, cap;
  int causal;
  int vec;               // CUDA cores: rows are whole accesses of four
  const float* slopes;
  const int *docs, *prefix, *lengths, *first;
  const DocSpan* spans;  // [B][ceil(Tk / kDocSpan)], with docs
  // forward
  void* out;             // [B][Tq][H][D]
  float* lse;            // [B][H][Tq] or null
  int splits, per_split; // shares of the keys, in tiles
  float* part;           // [splits][B][Hkv][Tq G][D] sums of a share
  float2* part_stats;    // [splits][B][Hkv][Tq G] maximum (in units of log2) and sum
  // gradient
  const void *dO, *O;    // [B][Tq][H][D]
  long long dob, dot, doh, ob, ot, oh;
  const float* lse_in;
  float* delta;          // [B][H][Tq]
  void *dQ, *dK, *dV;
  int row_splits;        // shares of the rows in the sums of a tile of keys
  float* key_part;       // [row_splits][B][Hkv][Tk][2][D]: dK and dV of a share
  long long dqb, dqt, dqh, dkb, dkt, dkh, dvb, dvt, dvh;
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kFar = 1 << 29;  // positions beyond are taken as this one

// Keys of sample b that exist.
__device__ __forceinline__ int attn_keys(const AttnArgs& a, int b) {
  return a.lengths != nullptr ? min(max(a.lengths[b], 0), a.Tk) : a.Tk;
}
__device__ __forceinline__ int attn_first(const AttnArgs& a, int b) {
  const int f = a.first != nullptr ? a.first[b] : a.Tk - a.Tq;
  return min(max(f, -kFar), kFar);
}

// What one query sees: the keys below `lim` whose document is `doc` (with
// documents; doc < 0: none).  A key before the causal border or inside the prefix is
// below their maximum.
struct RowSees {
  int pos, lim, doc;
};
__device__ __forceinline__ RowSees attn_row(const AttnArgs& a, int b, int t, int keys, int first) {
  RowSees r;
  r.pos = first + t;
  r.lim = keys;
  if (a.causal) {
    int see = r.pos + 1;
    if (a.prefix != nullptr) see = max(see, a.prefix[b]);
    r.lim = max(0, min(see, keys));
  }
  r.doc = 0;
  if (a.docs != nullptr) {
    r.doc = r.pos >= 0 && r.pos < a.Tk ? a.docs[static_cast<long long>(b) * a.Tk + r.pos] : -1;
    if (r.doc < 0) r.lim = 0;
  }
  return r;
}

// The kernels (attention_simt.cu, attention_tc.cu).
int attention_simt_rows(long long rows, long long heads);
int attention_simt_keys(long long keys, long long heads);  // of a CTA, in the gradient
cudaError_t launch_attention_simt(const AttnArgs& a, dprc_dtype dt, cudaStream_t s);
cudaError_t launch_attention_grad_simt(const AttnArgs& a, dprc_dtype dt, cudaStream_t s);
bool attention_tc_takes(const AttentionCall& c);
bool attention_tc_takes_grad(const AttentionGradCall& c);
int attention_tc_rows(const AttentionCall& c);  // of a CTA
int attention_tc_resident(const AttentionCall& c);  // CTAs of the forward pass on the GPU
int attention_tc_rows_grad(const AttentionCall& c);
cudaError_t launch_attention_tc(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attention_grad_tc(const AttnArgs& a, cudaStream_t s);

}  // namespace dprc
