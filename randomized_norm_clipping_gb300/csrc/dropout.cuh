// The dropout mask of the library's Philox stream, shared by the kernels that
// apply it (dropout.cu, linear.cu).
//
// Element e of a tensor (row-major) is dropped when half (e & 7) of Philox
// block e >> 3 is below thr = round(p 2^16): block j as in common.cuh, its
// four words taken as eight 16-bit halves, the low half of a word first.
// What is kept is multiplied by 65536 / (65536 - thr), so the mean is exact
// for the probability thr / 65536 that is in force (p to within 2^-17).
// Sixteen bits and not a word per element: one block then covers a 16-byte
// vector of bf16, and the generator stays below the memory time (a word each
// would double the ten multiply rounds per element).
#pragma once

#include "common.cuh"

namespace dprc {

struct DropArgs {
  uint64_t seed = 0, step = 0;
  uint32_t thr = 0;    // 0: nothing is dropped, 65536: everything
  float keep = 1.f;    // 65536 / (65536 - thr)
};

inline DropArgs drop_args(double p, uint64_t seed, uint64_t step) {
  DropArgs a;
  a.seed = seed;
  a.step = step;
  const double t = p * 65536.0 + 0.5;
  a.thr = t >= 65536.0 ? 65536u : static_cast<uint32_t>(t);
  a.keep = a.thr >= 65536u ? 0.f : static_cast<float>(65536.0 / (65536.0 - a.thr));
  return a;
}

// Half h (0..7) of a block against the threshold.
__device__ __forceinline__ bool drop_keep(const uint4& w, int h, uint32_t thr) {
  const uint32_t x = h < 2 ? w.x : h < 4 ? w.y : h < 6 ? w.z : w.w;
  return ((h & 1) ? x >> 16 : x & 0xFFFFu) >= thr;
}

// v[0..7] (elements 8 j .. 8 j + 7 of the tensor) dropped and scaled.  A
// dropped element is 0 whatever it held.
__device__ __forceinline__ void drop8(float* v, const uint4& w, uint32_t thr, float keep) {
#pragma unroll
  for (int h = 0; h < 8; ++h) v[h] = drop_keep(w, h, thr) ? v[h] * keep : 0.f;
}

}  // namespace dprc
