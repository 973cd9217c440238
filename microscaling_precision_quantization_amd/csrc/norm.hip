// RMSNorm around a block, forward and backward: before the block with the quantizer as its
// epilogue, after it with the block's gate and the residual's and the branch's scale.
//
// Mathematics (x or y the normed row of H values, w the weight):
//   r = (mean(x^2) + eps)^(-1/2),  n = x r w
//   dn -> g = dn w,  xh = x r,  dx = r (g - xh mean(g xh)),  dw = sum over rows of dn xh
//   out = res_scale x + branch_scale gate (y r w)
// The forward norm that feeds a quantizer is evaluated in binary64 from the squares on and
// rounded once to BF16: its relative error stays below 2^-50, so the BF16 value is the
// correctly rounded one unless the exact value lies that close to a rounding midpoint, and
// the quantized bytes are those of the library's quantizers on it.
#include <type_traits>

#include "common.h"

namespace mxq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// Eight consecutive elements of a BF16 or FP32 row, as FP32.
template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* f) {
  if (F32) {
    const float4 a = load_stream16f((const float*)base + at), b = load_stream16f((const float*)base + at + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack8(load_stream16((const uint16_t*)base + at), f);
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* f) {
  if (F32) {
    float4* o = reinterpret_cast<float4*>((float*)base + at);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>((uint16_t*)base + at) =
        make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7]));
  }
}

// Eight values read again by every row (weights, channel gates): cached loads. A null
// pointer stands for ones.
__device__ __forceinline__ void load8_cached(const float* p, int64_t at, float* f) {
  if (!p) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 1.0f;
    return;
  }
  const float4 a = *reinterpret_cast<const float4*>(p + at), b = *reinterpret_cast<const float4*>(p + at + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void zero8(float* f) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = 0.0f;
}

// Sum over the workgroup, the same for all threads (fixed order). `red` holds one value per
// wave; a barrier separates two uses of it.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  T s = red[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) s += red[i];
  __syncthreads();
  return s;
}

__device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max_f32(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) s = fmaxf(s, red[i]);
  return s;
}

// ---------------------------------------------------------------------------
// Norm before a block: one workgroup per row, the row kept in registers (NV vectors of 8 per
// thread), so x is read once. FMT: 1 MXFP8, 2 NVFP4 per token, 3 BF16 only, 4 MXFP4.
// ---------------------------------------------------------------------------
template <int FMT, bool X32, int NV>
__global__ void __launch_bounds__(kThreads)
norm_quant_kernel(const void* __restrict__ x, int64_t cols, int64_t ld_x, const float* __restrict__ weight, double eps,
                  uint16_t* __restrict__ n_out, uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                  float* __restrict__ t_out, float* __restrict__ rstd) {
  __shared__ double red[kWaves];
  __shared__ float redm[kWaves];
  const int64_t row = blockIdx.x;
  float f[NV][8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
    zero8(f[i]);
    if (e < cols) load8<X32>(x, row * ld_x + e, f[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fma((double)f[i][k], (double)f[i][k], ss);
  ss = block_sum(ss, red);
  const double r = 1.0 / sqrt(ss / (double)cols + eps);
  if (rstd && threadIdx.x == 0) rstd[row] = (float)r;
  uint4 p[NV];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
    p[i] = make_uint4(0, 0, 0, 0);
    if (e >= cols) continue;
    float w[8];
    load8_cached(weight, e, w);
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = f64_to_bf16_rne((double)f[i][k] * r * (double)w[k]);
    p[i] = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
    if (n_out) *reinterpret_cast<uint4*>(n_out + row * cols + e) = p[i];
    if (FMT == 2)
      amax = pk_max_u16(amax, pk_max_u16(pk_max_u16(p[i].x & 0x7FFF7FFFu, p[i].y & 0x7FFF7FFFu),
                                         pk_max_u16(p[i].z & 0x7FFF7FFFu, p[i].w & 0x7FFF7FFFu)));
  }
  if (FMT == 3) return;
  float s_enc = 1.0f;
  if (FMT == 2) {
    float t;
    scope_scales(block_max(__uint_as_float(max_halves(amax) << 16), redm), s_enc, t);
    if (threadIdx.x == 0) t_out[row] = t;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
    // cols is a multiple of the block, so the 2 (NVFP4) or 4 lanes of a block leave together;
    // lanes past the row hold zeros and only take part in the exchanges
    uint32_t a = pk_max_u16(pk_max_u16(p[i].x & 0x7FFF7FFFu, p[i].y & 0x7FFF7FFFu),
                            pk_max_u16(p[i].z & 0x7FFF7FFFu, p[i].w & 0x7FFF7FFFu));
    a = max_halves(a);
    a = max(a, dpp_xor1(a));
    if (FMT != 2) a = max(a, dpp_xor2(a));
    if (FMT == 1) {
      const uint32_t code = e8m0_from_bf16_amax(a);
      const float sc = e8m0_to_float(code);
      const uint32_t lo = cvt_fp8x2_bf16(cvt_fp8x2_bf16(0u, p[i].x, sc, false), p[i].y, sc, true);
      const uint32_t hi = cvt_fp8x2_bf16(cvt_fp8x2_bf16(0u, p[i].z, sc, false), p[i].w, sc, true);
      if (e < cols) {
        *reinterpret_cast<uint2*>(q + row * cols + e) = make_uint2(lo, hi);
        if ((threadIdx.x & 3) == 0) s[row * (cols / 32) + e / 32] = (uint8_t)code;
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
        if ((threadIdx.x & (LB - 1)) == 0) s[row * (cols / (8 * LB)) + e / (8 * LB)] = (uint8_t)code;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Norm after a block: out = res_scale x + branch_scale gate (y r w), one workgroup per row.
// GATE: 0 none, 1 one per row, 2 one per column, 3 one per element.
// ---------------------------------------------------------------------------
template <bool X32, bool Y32, int GATE, int NV>
__global__ void __launch_bounds__(kThreads)
gate_residual_kernel(const void* __restrict__ x, const void* __restrict__ y, int64_t cols,
                     const float* __restrict__ weight, const float* __restrict__ gate, double eps, float branch_scale,
                     float res_scale, void* __restrict__ out, float* __restrict__ rstd) {
  __shared__ double red[kWaves];
  const int64_t row = blockIdx.x;
  float f[NV][8], xv[NV][8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
    zero8(f[i]);
    if (e < cols) {
      load8<Y32>(y, row * cols + e, f[i]);
      load8<X32>(x, row * cols + e, xv[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fma((double)f[i][k], (double)f[i][k], ss);
  ss = block_sum(ss, red);
  const float r = (float)(1.0 / sqrt(ss / (double)cols + eps));
  if (rstd && threadIdx.x == 0) rstd[row] = r;
  const float c = GATE == 1 ? branch_scale * gate[row] : branch_scale;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
    if (e >= cols) continue;
    float w[8], g[8], o[8];
    load8_cached(weight, e, w);
    if (GATE == 2) load8_cached(gate, e, g);
    if (GATE == 3) load8<true>(gate, row * cols + e, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float b = f[i][k] * r * w[k];
      if (GATE >= 2) b *= g[k];
      o[k] = fmaf(b, c, res_scale * xv[i][k]);
    }
    store8<X32>(out, row * cols + e, o);
  }
}

// ---------------------------------------------------------------------------
// Backward of both: dn = scale (d + d2) gate,  dy = r (g - yh mean(g yh)) + res_scale res.
// Workgroups take rows b, b + grid, ...; each keeps the sums over its rows of dw (and of a
// column gate's gradient) in registers and leaves them as one row of the workspace, which
// column_sum_kernel adds up in row order: no atomics, the same bits on every run.
// ---------------------------------------------------------------------------
struct NormGrad {
  const void *d, *d2, *y, *res;
  const float *rstd, *weight, *gate;
  float scale, res_scale;
  int64_t rows, cols;
  void* dy;
  float *dw_part, *dg_part, *dgate;   // partial sums (NULL: not wanted); gate gradient (GATE 1 and 3)
};

template <bool D32, bool Y32, int GATE, int NV>
__global__ void __launch_bounds__(kThreads)
norm_backward_kernel(NormGrad a) {
  __shared__ float red[kWaves];
  const int64_t cols = a.cols;
  float w[NV][8], dw[NV][8], gc[GATE == 2 ? NV : 1][8], dgc[GATE == 2 ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
    zero8(w[i]);
    zero8(dw[i]);
    if (e < cols) load8_cached(a.weight, e, w[i]);
    if (GATE == 2) {
      zero8(gc[i]);
      zero8(dgc[i]);
      if (e < cols) load8_cached(a.gate, e, gc[i]);
    }
  }
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float r = a.rstd[row];
    const float gr = GATE == 1 ? a.gate[row] : 1.0f;
    float d[NV][8], yh[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
      zero8(d[i]);
      zero8(yh[i]);
      if (e < cols) {
        load8<D32>(a.d, row * cols + e, d[i]);
        load8<Y32>(a.y, row * cols + e, yh[i]);
      }
    }
    if (a.d2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
        if (e >= cols) continue;
        float d2[8];
        load8<D32>(a.d2, row * cols + e, d2);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[i][k] += d2[k];
      }
    }
    float m = 0.0f, dgr = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
      float ge[8];
      if (GATE == 3 && e < cols) load8<true>(a.gate, row * cols + e, ge);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        yh[i][k] *= r;
        float dn = a.scale * d[i][k];
        const float dg = dn * (yh[i][k] * w[i][k]);
        if (GATE == 1) dgr += dg;
        if (GATE == 2) dgc[i][k] += dg;
        if (GATE == 1) dn *= gr;
        if (GATE == 2) dn *= gc[i][k];
        if (GATE == 3) {
          dn = e < cols ? dn * ge[k] : 0.0f;
          ge[k] = dg;
        }
        dw[i][k] += dn * yh[i][k];
        d[i][k] = dn * w[i][k];
        m = fmaf(d[i][k], yh[i][k], m);
      }
      if (GATE == 3 && e < cols && a.dgate) store8<true>(a.dgate, row * cols + e, ge);
    }
    m = block_sum(m, red) / (float)cols;
    if (GATE == 1 && a.dgate) {
      dgr = block_sum(dgr, red);
      if (threadIdx.x == 0) a.dgate[row] = dgr;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
      if (e >= cols) continue;
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = r * fmaf(-yh[i][k], m, d[i][k]);
      if (a.res) {
        float rs[8];
        load8<Y32>(a.res, row * cols + e, rs);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = fmaf(a.res_scale, rs[k], o[k]);
      }
      store8<Y32>(a.dy, row * cols + e, o);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
    if (e >= cols) continue;
    if (a.dw_part) store8<true>(a.dw_part, (int64_t)blockIdx.x * cols + e, dw[i]);
    if (GATE == 2 && a.dg_part) store8<true>(a.dg_part, (int64_t)blockIdx.x * cols + e, dgc[i]);
  }
}

// out[c] = sum over `parts` rows of part[., c]: 64 columns per workgroup, its four waves on
// every fourth row, joined in wave order. blockIdx.y picks one of two (partials, sums) pairs.
__global__ void __launch_bounds__(kThreads)
column_sum_kernel(const float* __restrict__ part0, float* __restrict__ out0, const float* __restrict__ part1,
                  float* __restrict__ out1, int64_t parts, int64_t cols) {
  __shared__ float red[kWaves][64];
  const float* part = blockIdx.y ? part1 : part0;
  float* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int64_t p = w; p < parts; p += kWaves) s += part[p * cols + c];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < kWaves; ++i) s += red[i][lane];
    out[c] = s;
  }
}

template <typename F>
void with_vectors(int64_t cols, F&& go) {                   // vectors of 8 per thread
  const int64_t nv = (cols / 8 + kThreads - 1) / kThreads;
  if (nv <= 1) go(std::integral_constant<int, 1>{});
  else if (nv <= 2) go(std::integral_constant<int, 2>{});
  else if (nv <= 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});                // cols <= 16384
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

int64_t backward_parts(int64_t rows) { return rows < 512 ? rows : 512; }

}  // namespace

size_t norm_backward_ws_bytes(int64_t rows, int64_t cols) {
  return (size_t)(2 * backward_parts(rows) * cols * 4);    // dw and a column gate's gradient
}

hipError_t launch_norm_quant(int fmt, const void* x, int x32, int64_t rows, int64_t cols, int64_t ld_x,
                             const float* weight, double eps, void* n, void* q, void* s, float* t, float* rstd,
                             hipStream_t st) {
  const dim3 grid((unsigned)rows), block(kThreads);
  auto go = [&](auto F) {
    with_bool(x32, [&](auto X) {
      with_vectors(cols, [&](auto V) {
        hipLaunchKernelGGL((norm_quant_kernel<decltype(F)::value, decltype(X)::value, decltype(V)::value>), grid, block,
                           0, st, x, cols, ld_x, weight, eps, (uint16_t*)n, (uint8_t*)q, (uint8_t*)s, t, rstd);
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
  with_bool(x32, [&](auto X) {
    with_bool(y32, [&](auto Y) {
      with_gate(gate_mode, [&](auto G) {
        with_vectors(cols, [&](auto V) {
          hipLaunchKernelGGL(
              (gate_residual_kernel<decltype(X)::value, decltype(Y)::value, decltype(G)::value, decltype(V)::value>),
              dim3((unsigned)rows), dim3(kThreads), 0, st, x, y, cols, weight, gate, eps, branch_scale, res_scale, out,
              rstd);
        });
      });
    });
  });
  return hipGetLastError();
}

hipError_t launch_norm_backward(const void* d, const void* d2, int d32, const void* y, int y32, const float* rstd,
                                const float* weight, const float* gate, int gate_mode, float scale, const void* res,
                                float res_scale, int64_t rows, int64_t cols, void* dy, float* dw, float* dgate,
                                void* ws, hipStream_t st) {
  const int64_t parts = backward_parts(rows);
  float* dg_sum = gate_mode == 2 ? dgate : nullptr;
  float *dw_part = (float*)ws, *dg_part = (float*)ws + parts * cols;
  if (rows > 0) {
    const NormGrad a{d, d2, y, res, rstd, weight, gate, scale, res_scale, rows, cols, dy, dw ? dw_part : nullptr,
                     dg_sum ? dg_part : nullptr, dgate};
    with_bool(d32, [&](auto D) {
      with_bool(y32, [&](auto Y) {
        with_gate(gate_mode, [&](auto G) {
          with_vectors(cols, [&](auto V) {
            hipLaunchKernelGGL(
                (norm_backward_kernel<decltype(D)::value, decltype(Y)::value, decltype(G)::value, decltype(V)::value>),
                dim3((unsigned)parts), dim3(kThreads), 0, st, a);
          });
        });
      });
    });
  }
  if (dw || dg_sum)
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((cols + 63) / 64), dg_sum ? 2 : 1), dim3(kThreads), 0, st,
                       dw_part, dw, dg_part, dg_sum, parts, cols);
  return hipGetLastError();
}

}  // namespace mxq
