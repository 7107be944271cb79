// Attention's calls: which kernels take them, and the small kernels around them
// (what spans of keys hold of documents, the gradient's row sums, joining the
// shares of rows whose keys were split).

#include <algorithm>

#include "attention.cuh"
#include "vec.cuh"

namespace dprc {
namespace {

// One warp a span: its documents' least and greatest id, so that a tile of keys
// is met only by the rows whose documents it may hold.  Bound by its launch (4 us).
__global__ void __launch_bounds__(256) attention_spans_kernel(const int* docs, int Tk, int spans,
                                                              long long total, DocSpan* out) {
  pdl_launch_dependents();
  pdl_wait();
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= total) return;
  const int lane = threadIdx.x & 31;
  const long long b = w / spans;
  const int j0 = static_cast<int>(w - b * spans) * kDocSpan;
  int lo = 0x7fffffff, hi = -1, pad = 0;
#pragma unroll
  for (int k = 0; k < kDocSpan; k += 32) {
    const int j = j0 + k + lane;
    if (j >= Tk) continue;
    const int d = docs[b * Tk + j];
    if (d >= 0) {
      lo = min(lo, d);
      hi = max(hi, d);
    } else {
      pad = 1;
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    pad |= __shfl_xor_sync(0xffffffffu, pad, o);
  }
  if (lane == 0) out[w] = {lo, hi, pad, 0};
}

// delta[b][h][t] = sum over the width of dO O: eight threads a row, 16 bytes of
// both at a time where the width allows, four rows 32 apart, whose loads are all on their
// way before the first is used.  Bound by bytes: both are read once (4 x 4096 tokens of 32 heads of
// 64, 134 MB from cold caches: 39 us; with one row a group 40).
constexpr int kDeltaRows = 4;
template <typename T, int kE>
__global__ void __launch_bounds__(256) attention_delta_kernel(const AttnArgs a, long long rows) {
  pdl_launch_dependents();
  pdl_wait();
  const long long r0 = static_cast<long long>(blockIdx.x) * 32 * kDeltaRows, b = blockIdx.y;
  const long long tok0 = r0 / a.H;
  const int h0 = static_cast<int>(r0 - tok0 * a.H), t = threadIdx.x & 7;
  const T *dO[kDeltaRows], *O[kDeltaRows];
  float s[kDeltaRows];
#pragma unroll
  for (int k = 0; k < kDeltaRows; ++k) {
    const int i = k * 32 + (threadIdx.x >> 3), over = (h0 + i) / a.H;
    const long long tok = tok0 + over, h = h0 + i - over * a.H;
    const bool in = r0 + i < rows;  // (else the CTA's first row, which is not written)
    dO[k] = static_cast<const T*>(a.dO) + b * a.dob + (in ? tok * a.dot + h * a.doh : tok0 * a.dot + h0 * a.doh);
    O[k] = static_cast<const T*>(a.O) + b * a.ob + (in ? tok * a.ot + h * a.oh : tok0 * a.ot + h0 * a.oh);
    s[k] = 0.f;
  }
  for (int c = t * kE; c < a.D; c += 8 * kE) {
    Raw<T, kE> x[kDeltaRows], y[kDeltaRows];
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
      x[k].load(dO[k] + c);
      y[k].load(O[k] + c);
    }
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
      float u[kE], v[kE];
      x[k].get(u);
      y[k].get(v);
#pragma unroll
      for (int e = 0; e < kE; ++e) s[k] = fmaf(u[e], v[e], s[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kDeltaRows; ++k) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    const int i = k * 32 + (threadIdx.x >> 3), over = (h0 + i) / a.H;
    if (r0 + i < rows && t == 0)
      a.delta[(b * a.H + h0 + i - over * a.H) * a.Tq + tok0 + over] = s[k];
  }
}

// The shares of a row's keys, in order: a warp a row.  Bound by latency (7 us from cold caches
// for 256 rows of 4 shares, 3 behind the kernel that wrote them).
template <typename T>
__global__ void __launch_bounds__(128)
    attention_join_kernel(const AttnArgs a, long long rows) {
  pdl_launch_dependents();
  pdl_wait();
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  float m = -INFINITY;
  for (int z = lane; z < a.splits; z += 32) m = fmaxf(m, ld_l2(&a.part_stats[z * rows + r].x));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float at = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int z0 = 0; z0 < a.splits; z0 += 32) {
    const int z = z0 + lane;
    float w = 0.f, mine = 0.f;
    if (z < a.splits) {
      const float2 st = ld_l2(a.part_stats + z * rows + r);
      w = exp2f(st.x - at);
      mine = w * st.y;
    }
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    l += mine;
    const int n = min(32, a.splits - z0);
    for (int k = 0; k < n; ++k) {
      const float f = __shfl_sync(0xffffffffu, w, k);
      const float* p = a.part + ((z0 + k) * rows + r) * a.D;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c * 32 + lane < a.D) acc[c] = fmaf(f, ld_l2(p + c * 32 + lane), acc[c]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const int per = a.Tq * a.G;
  const long long bh = r / per, b = bh / a.Hkv;
  const int p = static_cast<int>(r - bh * per), t = p / a.G;
  const int h = static_cast<int>(bh - b * a.Hkv) * a.G + p - t * a.G;
  T* out = static_cast<T*>(a.out) + ((b * a.Tq + t) * a.H + h) * a.D;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c * 32 + lane < a.D) out[c * 32 + lane] = T(acc[c] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[(b * a.H + h) * a.Tq + t] = m * kLn2 + logf(l);
}

// dK and dV from the shares of the rows, in order: a thread an element of both.
template <typename T>
__global__ void __launch_bounds__(256) attention_join_keys_kernel(const AttnArgs a, long long total) {
  pdl_launch_dependents();
  pdl_wait();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const long long row = i / a.D, bh = row / a.Tk, b = bh / a.Hkv;
  const int col = static_cast<int>(i - row * a.D), key = static_cast<int>(row - bh * a.Tk);
  const int hk = static_cast<int>(bh - b * a.Hkv);
  const float* p = a.key_part + row * 2 * a.D + col;
  float k = 0.f, v = 0.f;
  for (int z = 0; z < a.row_splits; ++z) {
    k += ld_l2(p + z * total * 2);
    v += ld_l2(p + z * total * 2 + a.D);
  }
  if (a.dK != nullptr) static_cast<T*>(a.dK)[b * a.dkb + key * a.dkt + hk * a.dkh + col] = T(k);
  if (a.dV != nullptr) static_cast<T*>(a.dV)[b * a.dvb + key * a.dvt + hk * a.dvh + col] = T(v);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round16(size_t v) { return (v + 15) / 16 * 16; }

size_t stats_bytes(const AttentionCall& c, int splits) {
  return round16(static_cast<size_t>(splits) * c.B * c.Tq * c.H * sizeof(float2));
}

size_t span_bytes(const AttentionCall& c) {
  return c.docs != nullptr ? round16(c.B * cdiv(c.Tk, kDocSpan) * sizeof(DocSpan)) : 0;
}

// Shares of the keys: as many as fill the GPU where the rows alone do not, each
// of at least kLeast tiles (a share costs a partial row of its own).
constexpr int kLeast = 2;
struct Split {
  int splits, per;
};
Split split_keys(const AttentionCall& c, int tile_rows, int tile_keys, int resident) {
  const int64_t ctas = std::max<int64_t>(1, cdiv(c.Tq * (c.H / c.Hkv), tile_rows) * c.B * c.Hkv);
  const int64_t tiles = std::max<int64_t>(1, cdiv(c.Tk, tile_keys));
  int64_t want = std::max<int64_t>(1, resident / ctas);
  want = std::min(want, std::max<int64_t>(1, tiles / kLeast));
  Split s;
  s.per = static_cast<int>(cdiv(tiles, want));
  s.splits = static_cast<int>(cdiv(tiles, s.per));
  return s;
}

Split plan_split(const AttentionCall& c) {
  if (attention_tc_takes(c)) {
    return split_keys(c, attention_tc_rows(c), 128, attention_tc_resident(c));
  }
  return split_keys(c, attention_simt_rows(c.Tq * (c.H / c.Hkv), c.B * c.Hkv), 64, 608);
}

// Shares of the rows for tiles of keys that are too few to fill the GPU; their partial
// results stay below kMaxKeyPart.
constexpr int64_t kMaxKeyPart = int64_t(256) << 20;
int plan_row_splits(const AttentionCall& c, bool tc) {
  const int64_t bhs = c.B * c.Hkv, rows = c.Tq * (c.H / c.Hkv);
  const int64_t tile = tc ? 128 : attention_simt_keys(c.Tk, bhs);
  const int64_t ctas = std::max<int64_t>(1, cdiv(c.Tk, tile) * bhs);
  const int64_t steps = std::max<int64_t>(1, cdiv(rows, tc ? attention_tc_rows_grad(c) : 64));
  int64_t s = std::min<int64_t>((tc ? 152 : 304) / ctas, std::min<int64_t>(steps, 16));
  const int64_t bytes = std::max<int64_t>(1, bhs * c.Tk * 2 * c.D * 4);
  s = std::min<int64_t>(s, kMaxKeyPart / bytes);
  return static_cast<int>(std::max<int64_t>(1, s));
}
size_t key_part_bytes(const AttentionCall& c, int splits) {
  return splits > 1 ? static_cast<size_t>(splits) * c.B * c.Hkv * c.Tk * 2 * c.D * 4 : 0;
}
size_t delta_bytes(const AttentionCall& c) {
  return round16(static_cast<size_t>(c.B) * c.Tq * c.H * 4);
}

AttnArgs args_of(const AttentionCall& c, char* ws) {
  AttnArgs a = {};
  a.Q = c.Q; a.K = c.K; a.V = c.V;
  a.qb = c.qs[0]; a.qt = c.qs[1]; a.qh = c.qs[2];
  a.kb = c.ks[0]; a.kt = c.ks[1]; a.kh = c.ks[2];
  a.vb = c.vs[0]; a.vt = c.vs[1]; a.vh = c.vs[2];
  a.B = static_cast<int>(c.B);
  a.Tq = static_cast<int>(c.Tq);
  a.Tk = static_cast<int>(c.Tk);
  a.H = static_cast<int>(c.H);
  a.Hkv = static_cast<int>(c.Hkv);
  a.D = static_cast<int>(c.D);
  a.G = static_cast<int>(c.H / c.Hkv);
  a.scale = c.scale;
  a.cap = c.cap;
  a.causal = c.causal;
  a.slopes = c.slopes;
  a.docs = c.docs;
  a.prefix = c.prefix;
  a.lengths = c.lengths;
  a.first = c.first;
  a.spans = c.docs != nullptr ? reinterpret_cast<const DocSpan*>(ws) : nullptr;
  return a;
}

cudaError_t prepare_spans(const AttentionCall& c, char* ws, cudaStream_t s) {
  if (c.docs == nullptr || c.Tk == 0) return cudaSuccess;
  const int spans = static_cast<int>(cdiv(c.Tk, kDocSpan));
  const long long total = c.B * spans;
  return launch_after(attention_spans_kernel, dim3(static_cast<unsigned>(cdiv(total, 8))), 256, 1,
                      s, 0, c.docs, static_cast<int>(c.Tk), spans, total,
                      reinterpret_cast<DocSpan*>(ws));
}

template <typename T>
cudaError_t delta_rows(const AttnArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.Tq) * a.H;  // of a sample
  const dim3 grid(static_cast<unsigned>(cdiv(rows, 32 * kDeltaRows)), a.B);
  const long long all = a.D | a.dob | a.dot | a.doh | a.ob | a.ot | a.oh;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.dO) | reinterpret_cast<uintptr_t>(a.O);
  if (all % kVec16<T> == 0 && at % 16 == 0)
    return launch_after(attention_delta_kernel<T, kVec16<T>>, grid, 256, 1, s, 0, a, rows);
  return launch_after(attention_delta_kernel<T, 1>, grid, 256, 1, s, 0, a, rows);
}

}  // namespace

size_t attention_ws_bytes(const AttentionCall& c) {
  const Split sp = plan_split(c);
  const size_t part = sp.splits > 1
      ? stats_bytes(c, sp.splits) + static_cast<size_t>(sp.splits) * c.B * c.Tq * c.H * c.D * 4 : 0;
  return span_bytes(c) + part + 16;
}

size_t attention_grad_ws_bytes(const AttentionCall& c) {
  // (either kind of kernel may come to run: the other tensors decide)
  const size_t part = std::max(key_part_bytes(c, plan_row_splits(c, false)),
                               attention_tc_takes(c) ? key_part_bytes(c, plan_row_splits(c, true)) : 0);
  return span_bytes(c) + delta_bytes(c) + part + 16;
}

cudaError_t launch_attention(const AttentionCall& c, void* out, float* lse, void* ws,
                             cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  cudaError_t e = prepare_spans(c, w, s);
  if (e != cudaSuccess) return e;
  const Split sp = plan_split(c);
  AttnArgs a = args_of(c, w);
  a.out = out;
  a.lse = lse;
  a.splits = sp.splits;
  a.per_split = sp.per;
  a.part_stats = reinterpret_cast<float2*>(w + span_bytes(c));
  a.part = reinterpret_cast<float*>(w + span_bytes(c) + stats_bytes(c, sp.splits));
  e = attention_tc_takes(c) ? launch_attention_tc(a, s) : launch_attention_simt(a, c.dtype, s);
  if (e != cudaSuccess || sp.splits == 1) return e;
  const long long rows = static_cast<long long>(c.B) * c.Tq * c.H;
  const dim3 grid(static_cast<unsigned>(cdiv(rows, 4)));
  if (c.dtype == DPRC_F32)
    return launch_after(attention_join_kernel<float>, grid, 128, 1, s, 0, a, rows);
  return launch_after(attention_join_kernel<__nv_bfloat16>, grid, 128, 1, s, 0, a, rows);
}

cudaError_t launch_attention_grad(const AttentionGradCall& c, void* ws, cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  cudaError_t e = prepare_spans(c.f, w, s);
  if (e != cudaSuccess) return e;
  AttnArgs a = args_of(c.f, w);
  a.dO = c.dO;
  a.O = c.O;
  a.dob = c.dos[0]; a.dot = c.dos[1]; a.doh = c.dos[2];
  a.ob = c.os[0]; a.ot = c.os[1]; a.oh = c.os[2];
  a.lse_in = c.lse;
  a.delta = reinterpret_cast<float*>(w + span_bytes(c.f));
  a.dQ = c.dQ; a.dK = c.dK; a.dV = c.dV;
  a.dqb = c.dqs[0]; a.dqt = c.dqs[1]; a.dqh = c.dqs[2];
  a.dkb = c.dks[0]; a.dkt = c.dks[1]; a.dkh = c.dks[2];
  a.dvb = c.dvs[0]; a.dvt = c.dvs[1]; a.dvh = c.dvs[2];
  if (c.f.Tq > 0) {
    e = c.f.dtype == DPRC_F32 ? delta_rows<float>(a, s) : delta_rows<__nv_bfloat16>(a, s);
    if (e != cudaSuccess) return e;
  } else {
    a.dQ = nullptr;
  }
  if (c.f.Tk == 0) a.dK = a.dV = nullptr;
  const bool tc = attention_tc_takes_grad(c);
  a.row_splits = a.dK != nullptr || a.dV != nullptr ? plan_row_splits(c.f, tc) : 1;
  a.key_part = reinterpret_cast<float*>(w + span_bytes(c.f) + delta_bytes(c.f));
  e = tc ? launch_attention_grad_tc(a, s) : launch_attention_grad_simt(a, c.f.dtype, s);
  if (e != cudaSuccess || a.row_splits == 1) return e;
  const long long total = static_cast<long long>(c.f.B) * c.f.Hkv * c.f.Tk * c.f.D;
  const dim3 grid(static_cast<unsigned>(cdiv(total, 256)));
  if (c.f.dtype == DPRC_F32)
    return launch_after(attention_join_keys_kernel<float>, grid, 256, 1, s, 0, a, total);
  return launch_after(attention_join_keys_kernel<__nv_bfloat16>, grid, 256, 1, s, 0, a, total);
}

}  // namespace dprc
