// SwiGLU and its gradient in binary32, for the epilogues that round the result to BF16.
#pragma once
#include <hip/hip_runtime.h>

namespace mxq {

// e = e^-|g| <= 1 never overflows; with r = 1 / (1 + e): sigma(g) = r (g >= 0) or e r, 1 - sigma(g) = e r
// or r, neither by cancellation. e is 2^(-|g| log2 e) by the hardware's exponential: the rounded
// argument puts it off by |g| 2^-24 relative, and below 2^-126 (|g| > 87) it is 0. So sigma and 1 - sigma are within
// 2^-17 of exact plus 2^-126, and so is h, far inside the BF16 rounding that follows (2^-8); the
// library's expf, good to an ulp, took a third more instructions in an epilogue that is bound by them.
// A gate so far out that sigma is 0 gives 0 (also at -Inf, where g sigma would be a NaN).
__device__ __forceinline__ void sigmoid_pair(float g, float& s, float& c) {
  const float e = __builtin_amdgcn_exp2f(-1.44269504088896340736f * fabsf(g));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float er = e * r;
  s = g < 0.0f ? er : r;
  c = g < 0.0f ? r : er;
}
// h = g sigma(g) u
__device__ __forceinline__ float swiglu_forward(float g, float u) {
  float s, c;
  sigmoid_pair(g, s, c);
  return (s == 0.0f ? 0.0f : g * s) * u;
}
// dg = dh u sigma (1 + g (1 - sigma)), du = dh g sigma, h = g sigma u
// du and h as above. The derivative is within 2^-17 of the size of what it adds up, sigma (1 + |g| (1 - sigma)): of its
// own value except around its zero at g = -1.27846, where the two terms cancel and only that absolute bound is left
// (with |g| this small some 2^-24; the derivative at the gate's binary32 neighbour is 2^-25 away).
__device__ __forceinline__ void swiglu_backward(float dh, float g, float u, float& dg, float& du, float& h) {
  float s, c;
  sigmoid_pair(g, s, c);
  const float si = s == 0.0f ? 0.0f : g * s;
  const float ds = s == 0.0f ? 0.0f : c == 0.0f ? s : s * (1.0f + g * c);
  dg = dh * u * ds;
  du = dh * si;
  h = si * u;
}

}  // namespace mxq
