// Router of an expert layer: top-k choice of experts, combine weights, expert-major slots, the
// balance loss, and the gradients (through the combine to the expert outputs and weights, and
// from the weights and the loss to the logits).
//
// Mathematics, z the logits of a token over G experts:
//   chosen: the k largest z, ties to the lower expert; w_j = e^(z_j) / sum over the chosen
//   p = softmax(z) over all experts, counts_e the tokens that chose e, A their sum, N the tokens
//   loss = coef G sum_e (counts_e / A) (1/N) sum_t p_te
//   dz = w (dw - sum_chosen w dw) on the chosen  +  p (c - sum_e p c),  c_e = d_loss coef G counts_e / (A N)
//   combine y_t = sum_j w_tj O[slot_tj]:  dO[slot_tj] = w_tj dy_t,  dw_tj = <dy_t, O[slot_tj]>
// Slots are expert-major, tokens ascending inside an expert. A block of 64 tokens describes an
// expert's takers as one 64-bit mask (a token takes an expert at most once), so a token's rank in
// its expert is a count of lower bits plus the count of earlier blocks: integers only, the same
// plan on every run, no sort and no atomics whose order matters.
#include <type_traits>

#include "common.h"

namespace mxq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kTok = 64;                         // tokens per workgroup (one bit each of a mask)

// Order-preserving key of a logit: 0 for NaN, kNegInf for -inf, larger for larger values; -0
// equals +0. An expert is usable when its key lies above kNegInf.
constexpr uint32_t kNegInf = 0x007FFFFFu;
__device__ __forceinline__ uint32_t logit_key(float z) {
  if (z != z) return 0;
  const uint32_t u = __float_as_uint(z + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = shfl_xor_u32(v, off);
    v = v > o ? v : o;
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// ---------------------------------------------------------------------------
// Choice: one wave per token, NE experts per lane (expert = lane * NE + i). Writes topk_idx and
// weights; per block and expert the number of takers and, for the loss, the sum of p.
// ---------------------------------------------------------------------------
template <int NE>
__global__ void __launch_bounds__(kThreads)
route_choose_kernel(const float* __restrict__ logits, const uint8_t* __restrict__ valid, int64_t tokens, int experts,
                    int64_t ld, int topk, int32_t* __restrict__ topk_idx, float* __restrict__ weights,
                    int32_t* __restrict__ hist, float* __restrict__ psum, int32_t* __restrict__ routed_part) {
  extern __shared__ uint64_t mask[];             // [experts], then kWaves * experts floats for psum
  float* lp = reinterpret_cast<float*>(mask + experts);
  __shared__ int32_t routed_w[kWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < experts; e += kThreads) mask[e] = 0;
  __syncthreads();
  float acc[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
  int32_t routed = 0;
  for (int tl = w; tl < kTok; tl += kWaves) {
    const int64_t t = (int64_t)blockIdx.x * kTok + tl;
    if (t >= tokens) break;
    uint32_t key[NE], all[NE];
    const bool on = !valid || valid[t];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane * NE + i;
      key[i] = on && e < experts ? logit_key(logits[t * ld + e]) : 0u;
      all[i] = key[i];
    }
    float top = 0.0f, my = 0.0f;                 // largest logit; lane j: the j-th chosen one's numerator
    int my_e = -1;
    for (int j = 0; j < topk; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) best = key[i] > best ? key[i] : best;
      best = wave_max_u32(best);
      if (best <= kNegInf) break;                // no usable expert left (uniform over the wave)
      int at = NE;                               // this lane's first expert with that key
#pragma unroll
      for (int i = NE - 1; i >= 0; --i)
        if (key[i] == best) at = i;
      const uint64_t has = __ballot(at < NE);
      const int owner = __ffsll((unsigned long long)has) - 1;
      const int at_o = __shfl(at, owner, 64);
      const int e = owner * NE + at_o;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lane == owner && i == at_o) key[i] = 0;
      const float z = key_logit(best);
      if (j == 0) top = z;
      if (lane == j) {
        my = expf(z - top);
        my_e = e;
      }
      if (lane == 0) atomicOr((unsigned long long*)&mask[e], 1ull << tl);
    }
    const float sum = wave_sum(my);
    if (lane < topk) {
      topk_idx[t * topk + lane] = my_e;
      weights[t * topk + lane] = my_e < 0 ? 0.0f : my / sum;
    }
    const bool any = __shfl(my_e, 0, 64) >= 0;
    routed += any;
    if (psum && any) {
      float p[NE], z = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        p[i] = all[i] > kNegInf ? expf(key_logit(all[i]) - top) : 0.0f;
        z += p[i];
      }
      const float inv = 1.0f / wave_sum(z);
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] += p[i] * inv;
    }
  }
  if (lane == 0) routed_w[w] = routed;
  if (psum) {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane * NE + i < experts) lp[w * experts + lane * NE + i] = acc[i];
  }
  __syncthreads();
  if (threadIdx.x == 0) routed_part[blockIdx.x] = routed_w[0] + routed_w[1] + routed_w[2] + routed_w[3];
  for (int e = threadIdx.x; e < experts; e += kThreads) {
    hist[(int64_t)blockIdx.x * experts + e] = __popcll((unsigned long long)mask[e]);
    if (psum) psum[(int64_t)blockIdx.x * experts + e] = (lp[e] + lp[experts + e]) + (lp[2 * experts + e] + lp[3 * experts + e]);
  }
}

// ---------------------------------------------------------------------------
// Plan: one workgroup. hist becomes its exclusive prefix over the blocks; counts, padded offsets
// (what is left of `total` is dealt out in units of pad, low experts first), loss.
// ---------------------------------------------------------------------------
constexpr int kMaxExperts = 1024;

__global__ void __launch_bounds__(kMaxExperts)
route_plan_kernel(int32_t* __restrict__ hist, const float* __restrict__ psum, const int32_t* __restrict__ routed_part,
                  int64_t blocks, int experts, int64_t pad, int64_t total, float coef, int32_t* __restrict__ counts,
                  int64_t* __restrict__ offsets, float* __restrict__ loss) {
  __shared__ int64_t units[kMaxExperts + 1];
  __shared__ double dot[kMaxExperts];
  __shared__ int64_t taken[kMaxExperts];
  const int e = threadIdx.x;
  int32_t c = 0;
  double p = 0.0;
  if (e < experts) {
    for (int64_t b = 0; b < blocks; ++b) {
      const int32_t h = hist[b * experts + e];
      hist[b * experts + e] = c;
      c += h;
      if (psum) p += psum[b * experts + e];
    }
    counts[e] = c;
  }
  units[e] = (c + pad - 1) / pad;
  dot[e] = (double)c * p;
  taken[e] = c;
  __syncthreads();
  if (e == 0) {
    int64_t used = 0, a = 0, routed = 0;
    double s = 0.0;
    for (int i = 0; i < experts; ++i) {
      used += units[i];
      a += taken[i];
      s += dot[i];
    }
    for (int64_t b = 0; b < blocks; ++b) routed += routed_part[b];
    counts[experts] = (int32_t)routed;
    const int64_t spare = total / pad - used;
    int64_t at = 0;
    for (int i = 0; i < experts; ++i) {
      offsets[i] = at;
      at += (units[i] + spare / experts + (i < spare % experts ? 1 : 0)) * pad;
    }
    offsets[experts] = at;
    if (loss) *loss = routed ? (float)((double)coef * experts * (s / ((double)a * (double)routed))) : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Slots: the choice's token blocks again; slot_of and row_index, -1 in the padding slots.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads)
route_slots_kernel(const int32_t* __restrict__ topk_idx, const int32_t* __restrict__ base,
                   const int32_t* __restrict__ counts, const int64_t* __restrict__ offsets, int64_t tokens,
                   int experts, int topk, int32_t* __restrict__ row_index, int64_t* __restrict__ slot_of) {
  extern __shared__ uint64_t mask[];
  for (int e = threadIdx.x; e < experts; e += kThreads) mask[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int n = (int)(tokens - t0 < kTok ? tokens - t0 : kTok) * topk;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int32_t e = topk_idx[t0 * topk + i];
    if (e >= 0) atomicOr((unsigned long long*)&mask[e], 1ull << (i / topk));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int32_t e = topk_idx[t0 * topk + i];
    const int tl = i / topk;
    int64_t slot = -1;
    if (e >= 0) {
      slot = offsets[e] + base[(int64_t)blockIdx.x * experts + e] +
             __popcll((unsigned long long)(mask[e] & ((1ull << tl) - 1)));
      row_index[slot] = (int32_t)(t0 + tl);
    }
    slot_of[t0 * topk + i] = slot;
  }
  for (int e = blockIdx.x; e < experts; e += gridDim.x)
    for (int64_t s = offsets[e] + counts[e] + threadIdx.x; s < offsets[e + 1]; s += kThreads) row_index[s] = -1;
}

// ---------------------------------------------------------------------------
// Backward to the logits: one wave per token.
// ---------------------------------------------------------------------------
template <int NE>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const float* __restrict__ logits, int64_t tokens, int experts, int64_t ld, int topk,
                      const int32_t* __restrict__ topk_idx, const float* __restrict__ weights,
                      const float* __restrict__ d_weights, const int32_t* __restrict__ counts,
                      const float* __restrict__ d_loss, float coef, float* __restrict__ d_logits) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= tokens) return;
  const int my_e = lane < topk ? topk_idx[t * topk + lane] : -1;
  float d[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) d[i] = 0.0f;
  const bool any = __shfl(my_e, 0, 64) >= 0;
  if (any && d_loss) {
    int a = 0;
    float z[NE], c[NE], top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane * NE + i;
      z[i] = e < experts ? logits[t * ld + e] : -__builtin_inff();
      const int n = e < experts ? counts[e] : 0;
      c[i] = (float)n;
      a += n;
      top = fmaxf(top, z[i]);
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      top = fmaxf(top, __shfl_xor(top, off, 64));
      a += __shfl_xor(a, off, 64);
    }
    float sum = 0.0f, pc = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      z[i] = z[i] > -__builtin_inff() ? expf(z[i] - top) : 0.0f;   // an unusable expert has p = 0
      sum += z[i];
      pc += z[i] * c[i];
    }
    sum = wave_sum(sum);
    pc = wave_sum(pc) / sum;
    const float scale = *d_loss * ((coef * experts) / ((float)a * (float)counts[experts])) / sum;
#pragma unroll
    for (int i = 0; i < NE; ++i) d[i] = scale * z[i] * (c[i] - pc);
  }
  if (d_weights) {
    const float w = my_e >= 0 ? weights[t * topk + lane] : 0.0f;
    const float dw = my_e >= 0 ? d_weights[t * topk + lane] : 0.0f;
    const float g = w * (dw - wave_sum(w * dw));
    for (int j = 0; j < topk; ++j) {
      const int e = __shfl(my_e, j, 64);
      const float gj = __shfl(g, j, 64);
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (e == lane * NE + i) d[i] += gj;
    }
  }
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (lane * NE + i < experts) d_logits[t * experts + lane * NE + i] = d[i];
}

// ---------------------------------------------------------------------------
// Backward of the combine: one workgroup per token, dy kept in registers; the grid's last
// workgroups clear the padding slots' rows of dO.
// ---------------------------------------------------------------------------
template <bool D32, int NV>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const void* __restrict__ dy, const float* __restrict__ o, int64_t total, int64_t tokens,
                        int topk, int64_t hidden, const int64_t* __restrict__ slot_of,
                        const float* __restrict__ weights, const int32_t* __restrict__ row_index,
                        uint16_t* __restrict__ d_o, float* __restrict__ d_weights) {
  if (blockIdx.x >= tokens) {
    for (int64_t s = blockIdx.x - tokens; s < total; s += gridDim.x - tokens) {
      if (row_index[s] >= 0) continue;
      for (int64_t e = 8 * (int64_t)threadIdx.x; e < hidden; e += 8 * kThreads)
        *reinterpret_cast<uint4*>(d_o + s * hidden + e) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  __shared__ float red[kWaves];
  const int64_t t = blockIdx.x;
  float d[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
#pragma unroll
    for (int k = 0; k < 8; ++k) d[i][k] = 0.0f;
    if (e < hidden) {
      if (D32) {
        const float4 a = load_stream16f((const float*)dy + t * hidden + e);
        const float4 b = load_stream16f((const float*)dy + t * hidden + e + 4);
        d[i][0] = a.x; d[i][1] = a.y; d[i][2] = a.z; d[i][3] = a.w;
        d[i][4] = b.x; d[i][5] = b.y; d[i][6] = b.z; d[i][7] = b.w;
      } else {
        unpack8(load_stream16((const uint16_t*)dy + t * hidden + e), d[i]);
      }
    }
  }
  for (int j = 0; j < topk; ++j) {
    const int64_t slot = slot_of[t * topk + j];
    const bool in = slot >= 0 && slot < total;               // others contribute nothing
    float dot = 0.0f;
    if (in) {
      const float w = weights[t * topk + j];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t e = 8 * ((int64_t)i * kThreads + threadIdx.x);
        if (e >= hidden) continue;
        const float4 a = load_stream16f(o + slot * hidden + e), b = load_stream16f(o + slot * hidden + e + 4);
        dot += d[i][0] * a.x + d[i][1] * a.y + d[i][2] * a.z + d[i][3] * a.w;
        dot += d[i][4] * b.x + d[i][5] * b.y + d[i][6] * b.z + d[i][7] * b.w;
        *reinterpret_cast<uint4*>(d_o + slot * hidden + e) =
            make_uint4(bf16x2_rne(w * d[i][0], w * d[i][1]), bf16x2_rne(w * d[i][2], w * d[i][3]),
                       bf16x2_rne(w * d[i][4], w * d[i][5]), bf16x2_rne(w * d[i][6], w * d[i][7]));
      }
    }
    dot = wave_sum(dot);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) d_weights[t * topk + j] = (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
  }
}

template <typename F>
void with_experts(int64_t experts, F&& go) {                 // experts per lane
  if (experts <= 64) go(std::integral_constant<int, 1>{});
  else if (experts <= 128) go(std::integral_constant<int, 2>{});
  else if (experts <= 256) go(std::integral_constant<int, 4>{});
  else if (experts <= 512) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 16>{});                // experts <= kMaxExperts
}

int64_t route_blocks(int64_t tokens) { return (tokens + kTok - 1) / kTok; }

}  // namespace

// Workspace: hist (blocks, experts) int32, routed tokens per block, psum (blocks, experts) float.
size_t route_ws_bytes(int64_t tokens, int64_t experts) {
  return (size_t)(route_blocks(tokens) * (2 * experts + 1) * 4);
}

hipError_t launch_route(const float* logits, const uint8_t* valid, int64_t tokens, int64_t experts, int64_t ld,
                        int64_t topk, int64_t pad, int64_t total, float coef, int32_t* topk_idx, float* weights,
                        int32_t* counts, int64_t* offsets, int32_t* row_index, int64_t* slot_of, float* loss, void* ws,
                        hipStream_t st) {
  const int64_t nb = route_blocks(tokens);
  int32_t* hist = (int32_t*)ws;
  int32_t* routed = hist + nb * experts;
  float* psum = loss ? (float*)(routed + nb) : nullptr;
  const size_t lds = experts * 8;
  if (nb)
    with_experts(experts, [&](auto NE) {
      hipLaunchKernelGGL((route_choose_kernel<decltype(NE)::value>), dim3((unsigned)nb), dim3(kThreads),
                         lds + kWaves * experts * 4, st, logits, valid, tokens, (int)experts, ld, (int)topk, topk_idx,
                         weights, hist, psum, routed);
    });
  hipLaunchKernelGGL(route_plan_kernel, dim3(1), dim3(kMaxExperts), 0, st, hist, psum, routed, nb, (int)experts, pad,
                     total, coef, counts, offsets, loss);
  hipLaunchKernelGGL(route_slots_kernel, dim3((unsigned)(nb ? nb : 1)), dim3(kThreads), lds, st, topk_idx, hist, counts,
                     offsets, tokens, (int)experts, (int)topk, row_index, slot_of);
  return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, int64_t tokens, int64_t experts, int64_t ld, int64_t topk,
                                 const int32_t* topk_idx, const float* weights, const float* d_weights,
                                 const int32_t* counts, const float* d_loss, float coef, float* d_logits,
                                 hipStream_t st) {
  with_experts(experts, [&](auto NE) {
    hipLaunchKernelGGL((route_backward_kernel<decltype(NE)::value>), dim3((unsigned)((tokens + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, st, logits, tokens, (int)experts, ld, (int)topk, topk_idx, weights, d_weights,
                       counts, d_loss, coef, d_logits);
  });
  return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dy, int d32, const float* o, int64_t total, int64_t tokens,
                                   int64_t topk, int64_t hidden, const int64_t* slot_of, const float* weights,
                                   const int32_t* row_index, void* d_o, float* d_weights, hipStream_t st) {
  const dim3 grid((unsigned)(tokens + (total + 63) / 64)), block(kThreads);
  auto go = [&](auto D, auto V) {
    hipLaunchKernelGGL((combine_backward_kernel<decltype(D)::value, decltype(V)::value>), grid, block, 0, st, dy, o,
                       total, tokens, (int)topk, hidden, slot_of, weights, row_index, (uint16_t*)d_o, d_weights);
  };
  auto vectors = [&](auto D) {
    const int64_t nv = (hidden / 8 + kThreads - 1) / kThreads;
    if (nv <= 1) go(D, std::integral_constant<int, 1>{});
    else if (nv <= 2) go(D, std::integral_constant<int, 2>{});
    else if (nv <= 4) go(D, std::integral_constant<int, 4>{});
    else go(D, std::integral_constant<int, 8>{});
  };
  if (d32) vectors(std::true_type{});
  else vectors(std::false_type{});
  return hipGetLastError();
}

}  // namespace mxq
