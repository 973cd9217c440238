// RMSNorm around a block, forward and backward: before the block with the quantizer as its
// epilogue, after it with the block's gate and the residual's and the branch's scale.
//
// Mathematics (x or y the normed row of H values, w the weight):
//   r = (mean(x^2) + eps)^(-1/2),  n = x r w
//   dn -> g = dn w,  xh = x r,  dx = r (g - xh mean(g xh)),  dw = sum over rows of dn xh
//   out = res_scale x + branch_scale gate (y r w)
// The forward norm that feeds a quantizer is rounded once to BF16 from a value whose relative
// error stays below 2^-48 (binary64 from the squares on, whose sum takes at most 16 additions in a
// lane, 6 exchanges and 15 joins of waves, and the root halves its error; binary32 where its
// roundings cannot change the result): the correctly rounded one unless the exact value lies that
// close to a rounding midpoint. The quantized bytes are those of the library's quantizers on it.
#include <type_traits>

#include "common.h"

namespace mxq {
namespace {

// E consecutive elements of a BF16 or FP32 row in a lane, as loaded. E = 8 is 16 bytes of BF16, but
// for FP32 two accesses whose lanes lie 32 bytes apart; E = 4 is 16 bytes of FP32 in whole lines, 8 of
// BF16. A kernel takes 4 where it writes FP32 or its normed rows are (times at the kernels; FP32
// gradients alone gain nothing).
template <bool F32, int E = 8>
struct Raw {
  static constexpr int N = F32 ? E : E / 2;
  uint32_t v[N];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const uint8_t* p = (const uint8_t*)base + at * (F32 ? 4 : 2);
    if (N == 2) {
      const u32x2_nt u = __builtin_nontemporal_load((const u32x2_nt*)p);
      v[0] = u.x;
      v[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i + 3 < N; i += 4) {
        const uint4 u = load_stream16(p + 4 * i);
        v[i] = u.x;
        v[i + 1] = u.y;
        v[i + 2] = u.z;
        v[i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0;
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int k = 0; k < E; ++k)
      f[k] = F32 ? __uint_as_float(v[F32 ? k : 0]) : k & 1 ? bf16_hi(v[F32 ? 0 : k / 2]) : bf16_lo(v[F32 ? 0 : k / 2]);
  }
};

// STREAM: non-temporal stores.
template <bool F32, int E, bool STREAM = false>
__device__ __forceinline__ void store_row(void* base, int64_t at, const float* f) {
  if (F32) {
#pragma unroll
    for (int k = 0; k < E; k += 4)
      store16<STREAM>((float*)base + at + k, make_uint4(__float_as_uint(f[k]), __float_as_uint(f[k + 1]),
                                                        __float_as_uint(f[k + 2]), __float_as_uint(f[k + 3])));
  } else if (E == 4) {
    const u32x2_nt u = {bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3])};
    u32x2_nt* const to = (u32x2_nt*)((uint16_t*)base + at);
    if (STREAM) __builtin_nontemporal_store(u, to);
    else *to = u;
  } else {
    store16<STREAM>((uint16_t*)base + at, make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]),
                                                     bf16x2_rne(f[E - 4], f[E - 3]), bf16x2_rne(f[E - 2], f[E - 1])));
  }
}

// Values read again by every row (weights, channel gates): cached loads. A null pointer stands
// for ones.
template <int E>
__device__ __forceinline__ void load_cached(const float* p, int64_t at, float* f) {
#pragma unroll
  for (int k = 0; k < E; k += 4) {
    const float4 a = p ? *reinterpret_cast<const float4*>(p + at + k) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    f[k] = a.x;
    f[k + 1] = a.y;
    f[k + 2] = a.z;
    f[k + 3] = a.w;
  }
}

template <int E>
__device__ __forceinline__ void zero(float* f) {
#pragma unroll
  for (int k = 0; k < E; ++k) f[k] = 0.0f;
}

// One value per wave into LDS, all of them out again after a barrier that waits for LDS only.
// A kernel that loops over rows alternates between two buffers, so one barrier a row is enough:
// whoever writes a buffer again has passed the barrier in between, and all reads of it are done.
template <int W, typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
  v = wave_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  T s = red[0];
#pragma unroll
  for (int i = 1; i < W; ++i) s += red[i];
  return s;
}

template <int W>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = wave_max_u32(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  uint32_t s = red[0];
#pragma unroll
  for (int i = 1; i < W; ++i) s = max(s, red[i]);
  return s;
}

__device__ __forceinline__ uint32_t amax8(const uint4& p) {  // two maxima in one dword
  return pk_max_u16(pk_max_u16(p.x & 0x7FFF7FFFu, p.y & 0x7FFF7FFFu), pk_max_u16(p.z & 0x7FFF7FFFu, p.w & 0x7FFF7FFFu));
}

// Eight n = f r w to BF16, each rounded once from its value in binary64.
__device__ __forceinline__ uint4 norm8_f64(const float* f, const float* w, double r) {
  uint32_t h[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) h[k] = f64_to_bf16_rne((double)f[k] * r * (double)w[k]);
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// The same eight values, mostly from binary32. v = (f r32) w carries three roundings of 2^-24
// relative, so it lies within 3 of its own ulps of f r w; where its low 16 bits differ from
// 0x8000 by more than 4, both lie on the same side of every BF16 midpoint and rounding v gives
// the correctly rounded value. False where a value lies closer than that (one vector in 900), is
// nonzero and below 2^-100, or has a weight beyond 2^15: then binary64 decides. (2^-100 and 2^15
// keep f r32 a normal number; r itself is checked by the caller. A zero v is a zero f or w, or a
// product that underflowed: |f r32| <= 2^-150, and with the weight at most 2^-135, or f r32 was not
// zero and v's own rounding was, |f r w| <= 1.5 x 2^-150. Both lie below 2^-134, half of BF16's
// smallest subnormal, so zero is the correctly rounded value.)
__device__ __forceinline__ bool norm8_f32(const float* f, const float* w, float r32, uint4& out) {
  float v[8], big = 0.0f;
  uint32_t mid = 0xFFFFFFFFu, least = 0xFFFFFFFFu;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = f[k] * r32 * w[k];
    const uint32_t u = __float_as_uint(v[k]);
    mid = min(mid, (u + 0x8004u) << 16);                    // distance above 0x8000 - 4
    least = min(least, (u << 1) - 1u);                      // zeros wrap around to the top
    big = fmaxf(big, fabsf(w[k]));
  }
  out = make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
  return mid > (8u << 16) && least >= (27u << 24) && big <= 32768.0f;
}

// ---------------------------------------------------------------------------
// Norm before a block. W waves hold a row (W = 1: four rows to a workgroup, no barrier) as it
// was loaded, NV vectors of 8 per lane, so x is read once. FMT: 1 MXFP8, 2 NVFP4 per token,
// 3 BF16 only, 4 MXFP4.
// ---------------------------------------------------------------------------
template <int FMT, bool X32, bool STREAM, int W, int NV>
__global__ void __launch_bounds__(W == 1 ? 256 : W * 64)
norm_quant_kernel(const void* __restrict__ x, int64_t rows, int cols, int64_t ld_x, const float* __restrict__ weight,
                  double eps, double inv_cols, uint16_t* __restrict__ n_out, uint8_t* __restrict__ q,
                  uint8_t* __restrict__ s, float* __restrict__ t_out, float* __restrict__ rstd) {
  __shared__ double red[W];
  __shared__ uint32_t redm[W];
  const int tid = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (W == 1 && row >= rows) return;
  auto col = [&](int i) { return 8 * (i * W * 64 + tid); };
  Raw<X32> xr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    xr[i].clear();
    if (col(i) < cols) xr[i].load(x, row * ld_x + col(i));
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[8];
    xr[i].get(f);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fma((double)f[k], (double)f[k], ss);
  }
  ss = block_sum<W>(ss, red);
  const double r = rsqrt(fma(ss, inv_cols, eps));
  if (rstd && tid == 0) rstd[row] = (float)r;

  // n from binary32; bit i of `redo`: vector i of this wave holds a value that needs binary64
  uint4 p[NV];
  uint32_t redo = 0;
  const bool wide = !(r >= 0x1p-60 && r <= 0x1p60);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    p[i] = make_uint4(0, 0, 0, 0);
    bool sure = true;
    if (col(i) < cols) {
      float f[8], w[8];
      xr[i].get(f);
      load_cached<8>(weight, col(i), w);
      sure = norm8_f32(f, w, (float)r, p[i]) && !wide;
    }
    redo |= __any(!sure) ? 1u << i : 0u;
  }
  while (redo) {                                             // uniform; its x and w come from the caches
    const int j = __ffs(redo) - 1;
    redo &= redo - 1;
    if (col(j) < cols) {
      Raw<X32> again;
      float f[8], w[8];
      again.load(x, row * ld_x + col(j));
      again.get(f);
      load_cached<8>(weight, col(j), w);
      const uint4 fixed = norm8_f64(f, w, r);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == j) p[i] = fixed;
    }
  }

  float s_enc = 1.0f;
  if (FMT == 2) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) amax = pk_max_u16(amax, amax8(p[i]));
    float t;
    scope_scales(__uint_as_float(block_max<W>(max_halves(amax), redm) << 16), s_enc, t);
    if (tid == 0) t_out[row] = t;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    // cols is a multiple of the block, so the 2 (NVFP4) or 4 lanes of a block end together;
    // lanes past the row hold zeros and only take part in the exchanges
    const int e = col(i);
    if (n_out && e < cols) store16<STREAM>(n_out + row * cols + e, p[i]);
    if (FMT == 3) continue;
    uint32_t a = max_halves(amax8(p[i]));
    a = max(a, dpp_xor1(a));
    if (FMT != 2) a = max(a, dpp_xor2(a));
    if (FMT == 1) {
      const uint32_t code = e8m0_from_bf16_amax(a);
      const float sc = e8m0_to_float(code);
      const uint32_t lo = cvt_fp8x2_bf16(cvt_fp8x2_bf16(0u, p[i].x, sc, false), p[i].y, sc, true);
      const uint32_t hi = cvt_fp8x2_bf16(cvt_fp8x2_bf16(0u, p[i].z, sc, false), p[i].w, sc, true);
      if (e < cols) {
        *reinterpret_cast<uint2*>(q + row * cols + e) = make_uint2(lo, hi);
        if ((tid & 3) == 0) s[row * (cols / 32) + e / 32] = (uint8_t)code;
      }
    } else {
      float v[8], mul;
      unpack8(p[i], v);
      uint32_t code;
      if (FMT == 2) {
        code = block_scale(__uint_as_float(a << 16), s_enc, mul);
      } else {
        code = e8m0_from_bf16_amax_e2m1(a);
        mul = e8m0_inverse(code);
      }
      const uint32_t packed = pack8_e2m1(v, mul);
      if (e < cols) {
        *reinterpret_cast<uint32_t*>(q + row * (cols / 2) + e / 2) = packed;
        constexpr int LB = FMT == 2 ? 2 : 4;                 // lanes of a block
        if ((tid & (LB - 1)) == 0) s[row * (cols / (8 * LB)) + e / (8 * LB)] = (uint8_t)code;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Norm after a block: out = res_scale x + branch_scale gate (y r w), one workgroup per row. HBM
// bounds it: 16384 x 7168, channel gate, BF16 x, FP32 y 165 us, 5.7 TB/s (177 with E = 8; 172 with
// plain stores and a new output each call); all FP32 234, 6.0 TB/s (294 with E = 8); all BF16 130, 5.4
// TB/s (140 with E = 4). Every row's x, y and out lie in memory of their own.
// GATE: 0 none, 1 one per row, 2 one per column, 3 one per element.
// ---------------------------------------------------------------------------
template <bool X32, bool Y32, int GATE, bool STREAM, int W, int NV, int E>
__global__ void __launch_bounds__(W * 64)
gate_residual_kernel(const void* __restrict__ x, const void* __restrict__ y, int64_t cols,
                     const float* __restrict__ weight, const float* __restrict__ gate, double eps, float branch_scale,
                     float res_scale, void* __restrict__ out, float* __restrict__ rstd) {
  __shared__ double red[W];
  const int64_t row = blockIdx.x;
  auto col = [&](int i) { return E * (int64_t)(i * W * 64 + (int)threadIdx.x); };
  Raw<Y32, E> yr[NV];
  Raw<X32, E> xr[NV];
  float f[NV][E];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    yr[i].clear();
    if (col(i) < cols) {
      yr[i].load(y, row * cols + col(i));
      xr[i].load(x, row * cols + col(i));
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    yr[i].get(f[i]);
#pragma unroll
    for (int k = 0; k < E; ++k) ss = fma((double)f[i][k], (double)f[i][k], ss);
  }
  ss = block_sum<W>(ss, red);
  const float r = (float)(1.0 / sqrt(ss / (double)cols + eps));
  if (rstd && threadIdx.x == 0) rstd[row] = r;
  const float c = GATE == 1 ? branch_scale * gate[row] : branch_scale;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = col(i);
    if (e >= cols) continue;
    float w[E], g[E], xv[E], o[E];
    load_cached<E>(weight, e, w);
    if (GATE == 2) load_cached<E>(gate, e, g);
    if (GATE == 3) {
      Raw<true, E> gr;
      gr.load(gate, row * cols + e);
      gr.get(g);
    }
    xr[i].get(xv);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      float b = f[i][k] * r * w[k];
      if (GATE >= 2) b *= g[k];
      o[k] = fmaf(b, c, res_scale * xv[k]);
    }
    store_row<X32, E, STREAM>(out, row * cols + e, o);
  }
}

// ---------------------------------------------------------------------------
// Backward of both: dn = scale (d + d2) gate,  dy = r (g - yh mean(g yh)) + res_scale res.
// Workgroups take rows b, b + grid, ...; each keeps the column sums of its rows in registers and
// leaves them as one row of the workspace, which column_sum_kernel adds up in row order: no
// atomics, the same bits on every run. GATE: 0 none, 1 one per row, 3 one per element. A gate per
// column is constant over the rows as the weight is, so it is multiplied into the weight (GATE 0)
// and one sum, S = sum over the rows of scale d yh, gives both gradients: dw = gate S, dgate = w S.
// HBM bounds it: 16381 x 7168 with two FP32 gradients and the residual's 300 us, 5.5 TB/s (317 us
// with plain stores of dx); 8191 x 7168 after a block, FP32 y, 109 us, 5.4 TB/s (123 with E = 8, 117
// with plain stores); all FP32, 16384 x 7168, 242 us, 5.8 TB/s (292 with E = 8); all BF16 123, 5.7 TB/s
// (120 with E = 4, but at 16384 x 2048 52 against 58). With sixteen waves (rows beyond 8192) 128 registers
// a lane are all there are, and up to 62 spill (FP32 rows, token gate); 8192 x 16384 still runs at the
// copy's rate, 313 us of 315 for all FP32 and 250 of 262 with BF16 gradients.
// ---------------------------------------------------------------------------
struct NormGrad {
  const void *d, *d2, *y, *res;
  const float *rstd, *weight, *gate;  // gate: per row or element, or (GATE 0) per column or NULL
  float scale, res_scale;
  int64_t rows, cols;
  void* dy;
  float *part, *dgate;                // partial sums (NULL: not wanted); gate gradient (GATE 1 and 3)
};

template <bool D32, bool Y32, int GATE, bool STREAM, int W, int NV, int E>
__global__ void __launch_bounds__(W * 64)
norm_backward_kernel(NormGrad a) {
  __shared__ float red[2][W], redg[2][W];
  const int64_t cols = a.cols;
  auto col = [&](int i) { return E * (int64_t)(i * W * 64 + (int)threadIdx.x); };
  float w[NV][E], sum[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    zero<E>(w[i]);
    zero<E>(sum[i]);
    if (col(i) < cols) {
      load_cached<E>(a.weight, col(i), w[i]);
      if (GATE == 0) {
        float g[E];
        load_cached<E>(a.gate, col(i), g);
#pragma unroll
        for (int k = 0; k < E; ++k) w[i][k] *= g[k];
      }
    }
  }
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    Raw<D32, E> dr[NV], d2r[NV];
    Raw<Y32, E> yr[NV], rr[NV];
    const int64_t at = row * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      dr[i].clear();
      yr[i].clear();
      if (col(i) < cols) {
        dr[i].load(a.d, at + col(i));
        yr[i].load(a.y, at + col(i));
      }
    }
    if (a.d2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        d2r[i].clear();
        if (col(i) < cols) d2r[i].load(a.d2, at + col(i));
      }
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < cols) rr[i].load(a.res, at + col(i));
    }
    const float r = a.rstd[row];
    const float gr = GATE == 1 ? a.gate[row] : 1.0f;
    float d[NV][E], yh[NV][E], m = 0.0f, dgr = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = col(i);
      dr[i].get(d[i]);
      yr[i].get(yh[i]);
      if (a.d2) {
        float d2[E];
        d2r[i].get(d2);
#pragma unroll
        for (int k = 0; k < E; ++k) d[i][k] += d2[k];
      }
      float ge[E];
      if (GATE == 3) {
        zero<E>(ge);
        if (e < cols) {
          Raw<true, E> gr;
          gr.load(a.gate, at + e);
          gr.get(ge);
        }
      }
#pragma unroll
      for (int k = 0; k < E; ++k) {
        yh[i][k] *= r;
        float dn = a.scale * d[i][k];
        if (GATE == 1) {
          dgr += dn * (yh[i][k] * w[i][k]);
          dn *= gr;
        }
        if (GATE == 3) {
          const float dg = dn * (yh[i][k] * w[i][k]);
          dn *= ge[k];
          ge[k] = dg;
        }
        sum[i][k] = fmaf(dn, yh[i][k], sum[i][k]);
        d[i][k] = dn * w[i][k];
        m = fmaf(d[i][k], yh[i][k], m);
      }
      if (GATE == 3 && e < cols && a.dgate) store_row<true, E>(a.dgate, at + e, ge);
    }
    m = block_sum<W>(m, red[buf]) / (float)cols;
    if (GATE == 1 && a.dgate) {
      dgr = block_sum<W>(dgr, redg[buf]);
      if (threadIdx.x == 0) a.dgate[row] = dgr;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) >= cols) continue;
      float o[E];
#pragma unroll
      for (int k = 0; k < E; ++k) o[k] = r * fmaf(-yh[i][k], m, d[i][k]);
      if (a.res) {
        float rs[E];
        rr[i].get(rs);
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = fmaf(a.res_scale, rs[k], o[k]);
      }
      store_row<Y32, E, STREAM>(a.dy, at + col(i), o);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col(i) < cols) store_row<true, E>(a.part, (int64_t)blockIdx.x * cols + col(i), sum[i]);
}

// S[c] = sum over `parts` rows of part[., c]: 64 columns per workgroup, its sixteen waves on
// every sixteenth row, joined in wave order. dw = S times the channel gate (NULL: S), and
// dgate = S times the weight (NULL: S); either may be NULL.
constexpr int kSumWaves = 16;
__global__ void __launch_bounds__(kSumWaves * 64)
column_sum_kernel(const float* __restrict__ part, int64_t parts, int64_t cols, const float* __restrict__ weight,
                  const float* __restrict__ gate, float* __restrict__ dw, float* __restrict__ dgate) {
  __shared__ float red[kSumWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int64_t p = w; p < parts; p += kSumWaves) s += part[p * cols + c];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < kSumWaves; ++i) s += red[i][lane];
    if (dw) dw[c] = gate ? s * gate[c] : s;
    if (dgate) dgate[c] = weight ? s * weight[c] : s;
  }
}

// Waves that hold a row and vectors of 8 per lane: two vectors wherever the row has them. More
// vectors to a lane cost registers and with them rows in flight, more waves cost barriers and
// reductions (norm + MXFP8, 16384 x 7168: one wave of 16 vectors 138 us, 2 x 8 118, 4 x 4 119,
// 8 x 2 115, 16 x 1 137; NVFP4, 16384 x 4096: 1 x 8 66, 2 x 4 59, 4 x 2 59, 8 x 1 79).
template <typename F>
void with_row(int64_t cols, F&& go) {
  using std::integral_constant;
  const int64_t v = (cols / 8 + 63) / 64;                   // vectors a lane of one wave would hold
  if (v <= 1) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (v <= 2) go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  else if (v <= 4) go(integral_constant<int, 2>{}, integral_constant<int, 2>{});
  else if (v <= 8) go(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  else if (v <= 16) go(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 16>{}, integral_constant<int, 2>{});   // cols <= 16384
}

template <typename F>
void with_bool(bool b, F&& go) {
  if (b) go(std::true_type{});
  else go(std::false_type{});
}

template <typename F>
void with_gate(int gate, F&& go) {
  if (gate == 0) go(std::integral_constant<int, 0>{});
  else if (gate == 1) go(std::integral_constant<int, 1>{});
  else if (gate == 2) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, 3>{});
}

// Rows of a launch: a grid holds fewer than 2^32 threads (1024 to a row at most). More rows take
// more launches.
constexpr int64_t kLaunchRows = (int64_t)1 << 21;

// Workgroups of a backward, each with its column sums: two a CU. (us with 256, 512, 1024 and 2048; two BF16
// gradients of n, BF16 x and residual: 16381 x 7168 206, 215, 217, 220; 16384 x 4096 137, 123, 132, 135;
// 4096 x 2048 31, 24, 25, 29; 16384 x 2048 100, 66, 63, 67. Narrower rows leave SIMDs without a wave and
// would take more workgroups: 16384 x 1024 85, 52, 40, 40.)
int64_t backward_parts(int64_t rows) { return rows < 512 ? rows : 512; }

}  // namespace

size_t norm_backward_ws_bytes(int64_t rows, int64_t cols) {
  return (size_t)(backward_parts(rows) * cols * 4);        // one row of column sums per workgroup
}

hipError_t launch_norm_quant(int fmt, const void* x, int x32, int64_t rows, int64_t cols, int64_t ld_x,
                             const float* weight, double eps, void* n, void* q, void* s, float* t, float* rstd,
                             hipStream_t st) {
  const int64_t q_row = fmt == 1 ? cols : cols / 2, s_row = cols / (fmt == 2 ? 16 : 32);   // bytes
  auto go = [&](auto F) {
    with_bool(x32, [&](auto X) {
      with_bool(n && rows * cols * 2 > kStreamBytes, [&](auto L) {
        with_row(cols, [&](auto N, auto V) {
          constexpr int W = decltype(N)::value;
          for (int64_t r0 = 0; r0 < rows; r0 += kLaunchRows) {
            const int64_t some = rows - r0 < kLaunchRows ? rows - r0 : kLaunchRows;
            hipLaunchKernelGGL(
                (norm_quant_kernel<decltype(F)::value, decltype(X)::value, decltype(L)::value, W, decltype(V)::value>),
                dim3((unsigned)(W == 1 ? (some + 3) / 4 : some)), dim3(W == 1 ? 256 : W * 64), 0, st,
                (const uint8_t*)x + r0 * ld_x * (x32 ? 4 : 2), some, (int)cols, ld_x, weight, eps, 1.0 / (double)cols,
                n ? (uint16_t*)n + r0 * cols : nullptr, q ? (uint8_t*)q + r0 * q_row : nullptr,
                s ? (uint8_t*)s + r0 * s_row : nullptr, t ? t + r0 : nullptr, rstd ? rstd + r0 : nullptr);
          }
        });
      });
    });
  };
  if (fmt == 1) go(std::integral_constant<int, 1>{});
  else if (fmt == 2) go(std::integral_constant<int, 2>{});
  else if (fmt == 3) go(std::integral_constant<int, 3>{});
  else go(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t launch_gate_residual(const void* x, int x32, const void* y, int y32, int64_t rows, int64_t cols,
                                const float* weight, const float* gate, int gate_mode, double eps, float branch_scale,
                                float res_scale, void* out, float* rstd, hipStream_t st) {
  auto go = [&](auto X, auto Y, auto G, auto L) {
    with_row(cols, [&](auto N, auto V) {
      constexpr bool XF = decltype(X)::value, YF = decltype(Y)::value;
      constexpr int W = decltype(N)::value, GATE = decltype(G)::value, E = XF || YF ? 4 : 8;
      for (int64_t r0 = 0; r0 < rows; r0 += kLaunchRows) {
        const int64_t some = rows - r0 < kLaunchRows ? rows - r0 : kLaunchRows;
        hipLaunchKernelGGL(
            (gate_residual_kernel<XF, YF, GATE, decltype(L)::value, W, decltype(V)::value * 8 / E, E>),
            dim3((unsigned)some), dim3(W * 64), 0, st, (const uint8_t*)x + r0 * cols * (x32 ? 4 : 2),
            (const uint8_t*)y + r0 * cols * (y32 ? 4 : 2), cols, weight,
            GATE == 1 ? gate + r0 : GATE == 3 ? gate + r0 * cols : gate, eps, branch_scale, res_scale,
            (uint8_t*)out + r0 * cols * (x32 ? 4 : 2), rstd ? rstd + r0 : nullptr);
      }
    });
  };
  const bool large = rows * cols * (x32 ? 4 : 2) > kStreamBytes;
  with_bool(x32, [&](auto X) {
    with_bool(y32, [&](auto Y) {
      with_bool(large, [&](auto L) { with_gate(gate_mode, [&](auto G) { go(X, Y, G, L); }); });
    });
  });
  return hipGetLastError();
}

hipError_t launch_norm_backward(const void* d, const void* d2, int d32, const void* y, int y32, const float* rstd,
                                const float* weight, const float* gate, int gate_mode, float scale, const void* res,
                                float res_scale, int64_t rows, int64_t cols, void* dy, float* dw, float* dgate,
                                void* ws, hipStream_t st) {
  const int64_t parts = backward_parts(rows);
  const bool channel = gate_mode == 2, sums = dw || (channel && dgate);
  if (rows > 0) {
    const NormGrad a{d, d2, y, res, rstd, weight, gate, scale, res_scale, rows, cols, dy, sums ? (float*)ws : nullptr,
                     dgate};
    const bool large = rows * cols * (y32 ? 4 : 2) > kStreamBytes;
    auto go = [&](auto D, auto Y, auto G, auto L) {
      with_row(cols, [&](auto N, auto V) {
        constexpr bool YF = decltype(Y)::value;
        constexpr int W = decltype(N)::value, E = YF ? 4 : 8;
        hipLaunchKernelGGL((norm_backward_kernel<decltype(D)::value, YF, decltype(G)::value, decltype(L)::value, W,
                                                 decltype(V)::value * 8 / E, E>),
                           dim3((unsigned)parts), dim3(W * 64), 0, st, a);
      });
    };
    auto gate_kind = [&](auto D, auto Y, auto L) {
      if (gate_mode == 1) go(D, Y, std::integral_constant<int, 1>{}, L);
      else if (gate_mode == 3) go(D, Y, std::integral_constant<int, 3>{}, L);
      else go(D, Y, std::integral_constant<int, 0>{}, L);
    };
    with_bool(d32, [&](auto D) {
      with_bool(y32, [&](auto Y) { with_bool(large, [&](auto L) { gate_kind(D, Y, L); }); });
    });
  }
  if (sums)
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(kSumWaves * 64), 0, st,
                       (const float*)ws, parts, cols, weight, channel ? gate : nullptr, dw, channel ? dgate : nullptr);
  return hipGetLastError();
}

}  // namespace mxq
