// Shared device helpers for the gfx950 microscaling kernels.
//
// Format facts used here (definitions restated from the pages, see mxq.h):
//  * MXFP8: 32 E4M3 values share one E8M0 (power-of-two) scale.
//  * NVFP4: E2M1 values, one E4M3 scale per 16 values, one FP32 scale per scope.
//
// gfx950 conversion instructions used, and the behaviour relied upon (checked
// exhaustively on MI355X against the CPU definitions over every finite BF16
// input and scales 2^-127 .. 2^127):
//  * v_cvt_scalef32_pk_fp8_bf16 / _f32 (x, scale): OCP E4M3 of x / scale with
//    round-to-nearest-even, sign of zero kept, E4M3 subnormals produced. Out of
//    range inputs are NOT saturated (some give NaN): callers guarantee
//    |x / scale| <= 448 (the MXFP8 round-up scale does) or clamp first.
//  * v_cvt_scalef32_pk_fp4_f32 (x, scale): E2M1 of x / scale, round-to-nearest-
//    even, saturating to +-6, sign of zero kept.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

typedef short v2s __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr float kE4M3Max = 448.0f;
constexpr float kE2M1Max = 6.0f;
constexpr float kFltMax = 3.40282346638528859812e+38f;

// ---------------------------------------------------------------------------
// Lane exchanges
// ---------------------------------------------------------------------------
// DPP quad permutations: exchange with lane ^ 1 and lane ^ 2 inside groups of 4.
__device__ __forceinline__ uint32_t dpp_xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t dpp_xor2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t shfl_xor_u32(uint32_t v, int mask) {
  return (uint32_t)__shfl_xor((int)v, mask, 64);
}

// Reductions over the wave by DPP: rotations inside the rows of 16 lanes, then the row
// broadcasts, then lane 63's value for all (scalar registers). Dependent vector operations
// instead of trips through the LDS crossbar; the order of the additions is fixed.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, ROWS == 0xF);   // other rows: 0
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f32(float v) { return __uint_as_float(dpp_u32<CTRL, ROWS>(__float_as_uint(v))); }
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)dpp_u32<CTRL, ROWS>((uint32_t)(u >> 32)) << 32 |
                                          dpp_u32<CTRL, ROWS>((uint32_t)u)));
}
__device__ __forceinline__ uint32_t lane63(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0x128, 0xF>(v));
  v = max(v, dpp_u32<0x124, 0xF>(v));
  v = max(v, dpp_u32<0x122, 0xF>(v));
  v = max(v, dpp_u32<0x121, 0xF>(v));
  v = max(v, dpp_u32<0x142, 0xA>(v));
  v = max(v, dpp_u32<0x143, 0xC>(v));
  return lane63(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0x128, 0xF>(v);
  v += dpp_f32<0x124, 0xF>(v);
  v += dpp_f32<0x122, 0xF>(v);
  v += dpp_f32<0x121, 0xF>(v);
  v += dpp_f32<0x142, 0xA>(v);
  v += dpp_f32<0x143, 0xC>(v);
  return __uint_as_float(lane63(__float_as_uint(v)));
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_f64<0x128, 0xF>(v);
  v += dpp_f64<0x124, 0xF>(v);
  v += dpp_f64<0x122, 0xF>(v);
  v += dpp_f64<0x121, 0xF>(v);
  v += dpp_f64<0x142, 0xA>(v);
  v += dpp_f64<0x143, 0xC>(v);
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)lane63((uint32_t)(u >> 32)) << 32 | lane63((uint32_t)u)));
}

// Barrier that orders LDS accesses only: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Packed maximum of two pairs of unsigned 16-bit integers (sign-cleared BF16
// bit patterns order like their magnitudes).
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  us2 x, y;
  __builtin_memcpy(&x, &a, 4);
  __builtin_memcpy(&y, &b, 4);
  us2 m = __builtin_elementwise_max(x, y);
  uint32_t r;
  __builtin_memcpy(&r, &m, 4);
  return r;
}
__device__ __forceinline__ uint32_t max_halves(uint32_t v) {
  uint32_t lo = v & 0xFFFFu, hi = v >> 16;
  return lo > hi ? lo : hi;
}

// ---------------------------------------------------------------------------
// MXFP8 scale selection
// ---------------------------------------------------------------------------
// E8M0 code for a block whose largest magnitude has sign-cleared BF16 bits
// `amax_bits`: the smallest power of two 2^e with amax <= 448 * 2^e, as
// s = clamp(e + 127, 0, 254). With amax = (1 + M/128) * 2^(E-127):
// e = E - 127 - 8 when M <= 96 (mantissa <= 1.75), else E - 127 - 7. Zero and
// BF16-subnormal maxima clamp to s = 0; the largest BF16 gives s = 247.
__device__ __forceinline__ uint32_t e8m0_from_bf16_amax(uint32_t amax_bits) {
  int E = (int)((amax_bits >> 7) & 0xFF);
  int M = (int)(amax_bits & 0x7F);
  int s = E - 8 + (M > 96 ? 1 : 0);
  return (uint32_t)(s < 0 ? 0 : s);
}
// The same rule for MXFP4 blocks (E2M1 maximum 6 = 1.5 * 2^2): the smallest 2^e with
// amax <= 6 * 2^e, s = clamp(e + 127, 0, 254): e = E - 127 - 2 when M <= 64
// (mantissa <= 1.5), else E - 127 - 1.
__device__ __forceinline__ uint32_t e8m0_from_bf16_amax_e2m1(uint32_t amax_bits) {
  int E = (int)((amax_bits >> 7) & 0xFF);
  int M = (int)(amax_bits & 0x7F);
  int s = E - 2 + (M > 64 ? 1 : 0);
  return (uint32_t)(s < 0 ? 0 : s);
}
// 2^(127-s) as a float (exact); s = 254 gives the subnormal 2^-127.
__device__ __forceinline__ float e8m0_inverse(uint32_t s) {
  return __uint_as_float(s <= 253 ? (254u - s) << 23 : 0x00400000u);
}
// 2^(s-127) as a float; s = 0 gives the subnormal 2^-127.
__device__ __forceinline__ float e8m0_to_float(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : (s << 23));
}

// Two BF16 values (one dword, element 0 in the low half) -> two E4M3 bytes,
// written into the low (hi = false) or high (hi = true) 16 bits of `old`.
__device__ __forceinline__ uint32_t cvt_fp8x2_bf16(uint32_t old, uint32_t bf2, float scale, bool hi) {
  v2s o;
  __builtin_memcpy(&o, &old, 4);
  v2bf v;
  __builtin_memcpy(&v, &bf2, 4);
  o = hi ? __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, scale, true)
         : __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, scale, false);
  uint32_t r;
  __builtin_memcpy(&r, &o, 4);
  return r;
}
__device__ __forceinline__ uint32_t cvt_fp8x2_f32(uint32_t old, float a, float b, float scale, bool hi) {
  v2s o;
  __builtin_memcpy(&o, &old, 4);
  o = hi ? __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, true)
         : __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, false);
  uint32_t r;
  __builtin_memcpy(&r, &o, 4);
  return r;
}
// Two FP32 values -> one byte of two E2M1 nibbles (a in the low nibble) placed
// at byte `sel` (0..3) of `old`; scale 1.0 converts the values as given.
template <int SEL>
__device__ __forceinline__ uint32_t cvt_fp4x2_f32(uint32_t old, float a, float b) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, 1.0f, SEL);
}

// 16-byte global load with the non-temporal (streaming) hint, for inputs read once:
// measured on MI355X to lift read-heavy streams (a 268 MB BF16 input read once by the
// MXFP8 quantizer: 4.5 -> 5.6 TB/s); plain loads otherwise.
typedef unsigned int u32x4_nt __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_nt __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 load_stream16(const void* p) {
  const u32x4_nt v = __builtin_nontemporal_load(static_cast<const u32x4_nt*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ float4 load_stream16f(const float* p) {
  const uint4 v = load_stream16(p);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// An output beyond this size leaves with non-temporal stores: half of the memory-side cache,
// which the inputs stream through too; a smaller one stays there for the kernel that reads it next.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;
template <bool STREAM>                            // not a run-time flag: the compiler would merge the two stores
__device__ __forceinline__ void store16(void* p, const uint4& v) {
  u32x4_nt* const to = static_cast<u32x4_nt*>(p);
  const u32x4_nt u = {v.x, v.y, v.z, v.w};
  if (STREAM) __builtin_nontemporal_store(u, to);
  else *to = u;
}

// BF16 element j (0/1) of a dword, widened to FP32 exactly.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// FP32 -> BF16 bits, round-to-nearest-even (finite inputs; overflow -> Inf).
__device__ __forceinline__ uint32_t f32_to_bf16_rne(float f) {
  uint32_t u = __float_as_uint(f);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return u >> 16;
}

// Two FP32 -> two BF16 (RNE), element a in the low half: gfx950's packed convert. An
// exhaustive check over every non-NaN binary32 input (denormals included, in the
// library's denormal-preserving mode) matched f32_to_bf16_rne bit for bit.
typedef __bf16 v2bf_t __attribute__((ext_vector_type(2)));
typedef float v2f_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  v2f_t f;
  f.x = a;
  f.y = b;
  const v2bf_t h = __builtin_convertvector(f, v2bf_t);
  uint32_t o;
  __builtin_memcpy(&o, &h, 4);
  return o;
}
// Byte SEL of w (two E2M1 codes, low nibble first) -> two FP32 values, exact (hardware
// decode with scale 2^0; checked against e2m1_to_f32 on all 256 bytes).
template <int SEL>
__device__ __forceinline__ v2f_t e2m1x2_to_f32(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);
}

// E4M3 byte -> FP32 (exact). Codes 0x7F/0xFF (NaN) never occur in our data.
__device__ __forceinline__ float e4m3_to_f32(uint32_t c) {
  uint32_t e = (c >> 3) & 0xF, m = c & 7;
  float mag = e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : (float)m * 0.001953125f;  // m * 2^-9
  return (c & 0x80) ? -mag : mag;
}
// E2M1 nibble -> FP32 (exact).
__device__ __forceinline__ float e2m1_to_f32(uint32_t c) {
  uint32_t e = (c >> 1) & 3, m = c & 1;
  float mag = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
  return (c & 8) ? -mag : mag;
}

// ---------------------------------------------------------------------------
// NVFP4 scale steps and packing (the order of operations is in quant_nvfp4.hip)
// ---------------------------------------------------------------------------
__device__ __forceinline__ void scope_scales(float A, float& s_enc, float& t) {
  float s = 2688.0f / A;
  if (A == 0.0f) s = 1.0f;
  if (__builtin_isinf(s)) s = kFltMax;
  s_enc = s;
  t = 1.0f / s;
}

// Block scale code and element multiplier for a 16-block with amax a_b.
__device__ __forceinline__ uint32_t block_scale(float a_b, float s_enc, float& r_b) {
  float d = (a_b / 6.0f) * s_enc;
  d = fminf(d, kE4M3Max);                                   // saturate (d >= 0)
  const uint32_t code = cvt_fp8x2_f32(0u, d, 0.0f, 1.0f, false) & 0xFFu;
  const float S = e4m3_to_f32(code);
  float r = s_enc / S;
  r = fminf(r, kFltMax);
  r_b = (S == 0.0f) ? 0.0f : r;
  return code;
}

// Eight consecutive values (a 16-block is two lanes) -> 4 packed bytes.
__device__ __forceinline__ uint32_t pack8_e2m1(const float* v, float r) {
  uint32_t o = 0;
  o = cvt_fp4x2_f32<0>(o, v[0] * r, v[1] * r);
  o = cvt_fp4x2_f32<1>(o, v[2] * r, v[3] * r);
  o = cvt_fp4x2_f32<2>(o, v[4] * r, v[5] * r);
  o = cvt_fp4x2_f32<3>(o, v[6] * r, v[7] * r);
  return o;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}

__device__ __forceinline__ float wave_max_f32(float v) {
  uint32_t u = __float_as_uint(v);  // v >= 0: bits order like values
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = shfl_xor_u32(u, off);
    u = u > o ? u : o;
  }
  return __uint_as_float(u);
}

// binary64 -> BF16 bits, one rounding: the binary32 conversion is turned into
// round-to-odd (an inexact result is truncated toward zero and gets its last bit set),
// and round-to-odd to 24 bits followed by nearest-even to 8 bits equals nearest-even
// to 8 bits directly (24 >= 8 + 2). Values past the binary32 range come out as
// FLT_MAX | 1 and then round to +-Inf, values below its subnormals as +-2^-149 and
// then to a signed zero, as the direct rounding gives.
__device__ __forceinline__ uint32_t f64_to_bf16_rne(double d) {
  float f = (float)d;
  if ((double)f != d) {
    uint32_t b = __float_as_uint(f);
    if (fabs((double)f) > fabs(d)) b -= 1u;          // magnitude rounded up: step back
    f = __uint_as_float(b | 1u);
  }
  return f32_to_bf16_rne(f);
}

}  // namespace mxq
