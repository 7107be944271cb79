// Rotary positions with one or several axes.  Pair p of a head, (a, b), at the
// angle phi = pos[axis(p)] freq[p] becomes
//     (a cos phi - b sin phi, a sin phi + b cos phi)
// (the inverse turns by -phi: the gradient's way back).
//
// Bound by bytes: every element is read and written once.  A CTA takes a piece of
// tokens, forms the sines of its tokens and pairs once, in shared memory, for all
// heads, and streams the heads past them.  The angle is reduced to a part of a
// turn in fp64 (a few operations per token and pair, shared by the heads), whose three
// roundings, of 1 / (2 pi), of its product with the frequency and of that with the position,
// put it off by 3 2^-53 of itself at most: below fp32's half step of a radian up to 1.7e8
// radians, 7e-7 at 2^31; the sine itself is fp32.  Measured: 4 x 4096
// tokens of 40 heads of 64, bf16, 34.7 us (168 MB: 4.8 TB/s, 0.71 of the copy rate).

#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "vec.cuh"

namespace dprc {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTable = 2048;  // (cos, sin) pairs of a CTA
constexpr int kRotTokens = 32;   // tokens of a CTA at the most

struct RotArgs {
  long long N, T;                 // tokens, and those of a sample
  long long xb, xt, xh;           // strides of x in elements
  long long ob, ot, oh;
  int H, D, P;                    // heads, width of a head, pairs
  int axes;
  int end[kMaxRotAxes];           // first pair behind each axis's
  int tokens;                     // of a CTA
  int head_split;                 // CTAs (blockIdx.y) that share the heads
  int inverse;
};

// Whether the strides allow whole 16-byte accesses is the host's question; kE
// elements are one access.  kInter: pairs of neighbours (2p, 2p + 1), else of
// halves (p, P + p).
template <typename T, typename I, int kE, bool kInter>
__global__ void __launch_bounds__(kRotThreads)
    rotary_kernel(const T* x, const I* pos, const double* freqs, T* out, const RotArgs a) {
  __shared__ float2 cs[kRotTable];
  __shared__ long long xat[kRotTokens], oat[kRotTokens];  // where the tokens' heads begin
  pdl_launch_dependents();
  pdl_wait();
  const long long n0 = static_cast<long long>(blockIdx.x) * a.tokens;
  const int nt = static_cast<int>(min(static_cast<long long>(a.tokens), a.N - n0));
  if (static_cast<int>(threadIdx.x) < nt) {
    const long long n = n0 + threadIdx.x, b = n / a.T, t = n - b * a.T;
    xat[threadIdx.x] = b * a.xb + t * a.xt;
    oat[threadIdx.x] = b * a.ob + t * a.ot;
  }
  for (int i = threadIdx.x; i < nt * a.P; i += kRotThreads) {
    const int tk = i / a.P, p = i - tk * a.P;
    int ax = 0;
    while (ax + 1 < a.axes && p >= a.end[ax]) ++ax;
    const double turns = static_cast<double>(pos[(n0 + tk) * a.axes + ax]) *
                         (freqs[p] * 0.15915494309189533577);  // 1 / (2 pi)
    float s, c;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
    if (DPRC_IN(i < kRotTable)) cs[i] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
  // an item: kE elements of each of the two sides of its pairs (kInter: of kE / 2
  // pairs, one access; kE = 1: a pair), or kE elements behind the pairs
  const int per_item = kInter ? (kE == 1 ? 1 : kE / 2) : kE;
  const int turned = a.P / per_item;
  const int rest = (a.D - 2 * a.P) / kE;
  const int items = turned + rest;
  const int h0 = static_cast<int>(static_cast<long long>(a.H) * blockIdx.y / a.head_split);
  const int h1 = static_cast<int>(static_cast<long long>(a.H) * (blockIdx.y + 1) / a.head_split);
  const int heads = h1 - h0, total = nt * heads * items;
  for (int i = threadIdx.x; i < total; i += kRotThreads) {
    const int th = i / items, it = i - th * items;
    const int tk = th / heads, h = h0 + th - tk * heads;
    const T* xr = x + xat[tk] + h * a.xh;
    T* o = out + oat[tk] + h * a.oh;
    if (it >= turned) {
      const int at = 2 * a.P + (it - turned) * kE;
      Raw<T, kE> r;
      float v[kE];
      r.load(xr + at);
      r.get(v);
      store_row<kE>(o + at, v);
      continue;
    }
    const float2* w = cs + tk * a.P + it * per_item;
    if constexpr (kInter && kE > 1) {
      Raw<T, kE> r;
      float v[kE];
      r.load(xr + it * kE);
      r.get(v);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const float2 c = w[e / 2];
        const float u = v[e], z = v[e + 1];
        v[e] = u * c.x - z * c.y;
        v[e + 1] = u * c.y + z * c.x;
      }
      store_row<kE>(o + it * kE, v);
    } else {
      const int i0 = kInter ? 2 * it : it * kE, i1 = kInter ? 2 * it + 1 : a.P + it * kE;
      Raw<T, kE> r, q;
      float u[kE], z[kE];
      r.load(xr + i0);
      q.load(xr + i1);
      r.get(u);
      q.get(z);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float2 c = w[e];
        const float n0v = u[e] * c.x - z[e] * c.y;
        z[e] = u[e] * c.y + z[e] * c.x;
        u[e] = n0v;
      }
      store_row<kE>(o + i0, u);
      store_row<kE>(o + i1, z);
    }
  }
}

template <typename T, typename I>
cudaError_t launch_t(const RotaryCall& c, cudaStream_t s) {
  RotArgs a;
  a.N = c.B * c.T;
  a.T = c.T;
  a.xb = c.xs[0]; a.xt = c.xs[1]; a.xh = c.xs[2];
  a.ob = c.os[0]; a.ot = c.os[1]; a.oh = c.os[2];
  a.H = static_cast<int>(c.H);
  a.D = static_cast<int>(c.D);
  a.P = static_cast<int>(c.pairs);
  a.axes = c.axes;
  int at = 0;
  for (int k = 0; k < c.axes; ++k) a.end[k] = at += static_cast<int>(c.sections[k]);
  a.inverse = c.inverse;
  constexpr int kV = kVec16<T>;
  const auto whole = [](int64_t v) { return v % kV == 0; };
  bool vec = reinterpret_cast<uintptr_t>(c.X) % 16 == 0 &&
             reinterpret_cast<uintptr_t>(c.out) % 16 == 0 && whole(c.D) && whole(2 * c.pairs) &&
             (c.interleaved || whole(c.pairs));
  for (int k = 0; k < 3; ++k) vec = vec && whole(c.xs[k]) && whole(c.os[k]);
  // tokens of a CTA: four accesses a thread, or eight where that leaves four CTAs to an
  // SM (4 x 4096 tokens, 40 heads of 64: 36.1 and 34.7 us; 16 39.0), within the table; few
  // tokens share a CTA's heads out instead
  const int64_t per_token = c.H * ((c.D + (vec ? kV : 1) - 1) / (vec ? kV : 1));
  const int work = a.N * per_token >= int64_t(608) * 8 * kRotThreads ? 8 : 4;
  int64_t tk = std::max<int64_t>(1, work * kRotThreads / std::max<int64_t>(1, per_token));
  tk = std::min<int64_t>(tk, std::max<int64_t>(1, kRotTable / std::max<int64_t>(1, c.pairs)));
  tk = std::min<int64_t>(std::min<int64_t>(tk, kRotTokens), a.N);
  a.tokens = static_cast<int>(tk);
  const int64_t ctas = (a.N + tk - 1) / tk;
  int64_t split = 1;
  while (split < c.H && split < 64 && ctas * split < 304 &&
         per_token * tk / split > kRotThreads)
    split *= 2;
  a.head_split = static_cast<int>(std::min<int64_t>(split, c.H));
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(a.head_split));
  const auto go = [&](auto kernel) {
    return launch_after(kernel, grid, kRotThreads, 1, s, 0, static_cast<const T*>(c.X),
                        static_cast<const I*>(c.positions), c.freqs, static_cast<T*>(c.out), a);
  };
  if (vec) return c.interleaved ? go(rotary_kernel<T, I, kV, true>) : go(rotary_kernel<T, I, kV, false>);
  return c.interleaved ? go(rotary_kernel<T, I, 1, true>) : go(rotary_kernel<T, I, 1, false>);
}

}  // namespace

cudaError_t launch_rotary(const RotaryCall& c, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (c.dtype == DPRC_F32)
    return c.position_bytes == 4 ? launch_t<float, int32_t>(c, s) : launch_t<float, long long>(c, s);
  return c.position_bytes == 4 ? launch_t<bf16, int32_t>(c, s) : launch_t<bf16, long long>(c, s);
}

cudaError_t read_device_error_rotary(int32_t* out, bool reset) {
  return read_tu_device_error(out, reset);
}

}  // namespace dprc
