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
constexpr int kMaxTok = 64;                      // most tokens of a block (one bit each of a mask)
constexpr int kTallies = 16;
constexpr int kMaxTopk = 32;

// Order-preserving key of a logit: larger for larger values, -0 as +0, NaN as -inf. An expert is
// usable when its key lies above that of -inf, 0x007FFFFF.
__device__ __forceinline__ uint32_t logit_key(float z) {
  const uint32_t u = __float_as_uint(fmaxf(z, -__builtin_inff()) + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Key and expert in one binary64: the key as an integer, and below its units bit `rest`, larger
// for lower experts. Every expert of a token has another value, in the order of the choice, so a
// maximum names its expert and sorting by maxima and minima (two instructions an exchange) keeps
// equal logits in order. (A 32-bit integer leaves 21 bits of the significand.)
__device__ __forceinline__ double ranked(uint32_t key, uint32_t rest) {
  return __longlong_as_double(__double_as_longlong((double)key) | rest);
}
constexpr double kUsable = 8388608.0;            // 0x00800000

// e^(z - top) for z <= top; 0 for an expert that is not usable (-inf, NaN: fmaxf drops it). The
// exponent of two is formed with log2(e) in two parts, so it carries the roundings of z - top and
// of the fused multiply-add only: 2 u |z - top| relative, and an ulp of the instruction.
__device__ __forceinline__ float softmax_term(float z, float top) {
  const float x = fmaxf(z, -__builtin_inff()) - top;
  return __builtin_amdgcn_exp2f(fmaf(x, 1.44269502e+00f, x * 1.92596299e-08f));
}

// A lane's NE consecutive logits of a row, NaN past the row, in loads as wide as the row's end
// allows (whatever its alignment).
template <int NE>
__device__ __forceinline__ void load_logits(const float* row, int experts, int lane, float* z) {
  constexpr int C = NE < 4 ? NE : 4;
  const int e = lane * NE, left = experts - e;
#pragma unroll
  for (int i = 0; i < NE; ++i) z[i] = __builtin_nanf("");
  if (experts % NE == 0) {
    if (left > 0) __builtin_memcpy(z, row + e, NE * 4);
    return;
  }
#pragma unroll
  for (int i = 0; i < NE; i += C) {
    if (left >= i + C) __builtin_memcpy(z + i, row + e + i, C * 4);
    else
#pragma unroll
      for (int k = 0; k < C; ++k)
        if (left > i + k) z[i + k] = row[e + i + k];
  }
}

// Sorts a lane's values in descending order (Batcher's odd-even merge sort, 1968: 63 exchanges for
// 16 values).
template <int NE>
__device__ __forceinline__ void sort_desc(double* v) {
#pragma unroll
  for (int p = 1; p < NE; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < NE; j += 2 * k)
#pragma unroll
        for (int i = j; i < j + k && i + k < NE; ++i)
          if (i / (2 * p) == (i + k) / (2 * p)) {
            const double hi = fmax(v[i], v[i + k]), lo = fmin(v[i], v[i + k]);
            v[i] = hi;
            v[i + k] = lo;
          }
}

// The maximum of two ordinary numbers, as the one instruction: fmax() first quiets operands that
// could be signalling NaNs, which ranked values never are.
__device__ __forceinline__ double max2(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// Reductions over the L lanes of a token (a row of 16, two rows, or the wave), in all of them. The
// swap of a value with itself leaves both rows of a pair the even row's and the odd row's.
__device__ __forceinline__ double pair_max(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  return max2(__longlong_as_double((long long)((uint64_t)hi[0] << 32 | lo[0])),
              __longlong_as_double((long long)((uint64_t)hi[1] << 32 | lo[1])));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
template <int L>
__device__ __forceinline__ double lanes_max(double v) {
  v = max2(v, dpp_f64<0x128, 0xF>(v));
  v = max2(v, dpp_f64<0x124, 0xF>(v));
  v = max2(v, dpp_f64<0x122, 0xF>(v));
  v = max2(v, dpp_f64<0x121, 0xF>(v));
  if (L == 16) return v;
  if (L == 32) return pair_max(v);
  v = max2(v, dpp_f64<0x142, 0xA>(v));           // positive values: the zeros of the other rows lose
  v = max2(v, dpp_f64<0x143, 0xC>(v));
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)lane63((uint32_t)(u >> 32)) << 32 | lane63((uint32_t)u)));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if (L == 64) return wave_sum(v);
  v += dpp_f32<0x128, 0xF>(v);
  v += dpp_f32<0x124, 0xF>(v);
  v += dpp_f32<0x122, 0xF>(v);
  v += dpp_f32<0x121, 0xF>(v);
  return L == 32 ? pair_sum(v) : v;
}

struct Route {
  const float* logits;
  const uint8_t* valid;
  int64_t tokens, ld, pad, total;
  int experts, topk, units, tok;                 // units: total / pad; tok: tokens of a block
  float coef;
  int32_t* topk_idx;
  float* weights;
  int32_t* counts;
  int64_t* offsets;
  int32_t* row_index;
  int64_t* slot_of;
  float* loss;
  uint8_t* hist;                                 // (blocks, hist_cols): takers per expert, then routed tokens
  int32_t* base;                                 // (blocks, hist_cols): hist summed over earlier blocks
  int32_t* sums;                                 // (hist_cols): hist summed over all blocks
  float* psum;                                   // (blocks, experts): sums of p
  uint64_t* tally;                               // (1 + kTallies), 64 bytes apart: sums of the loss and counts
};

__host__ __device__ inline int hist_cols(int experts) { return (experts + 4) / 4 * 4; }

// Waves of a workgroup that chooses: sixteen keep four on every SIMD; eight where sixteen rows of
// sums would not fit beside the masks in 64 KB.
constexpr int choose_waves(int lanes, int ne) { return lanes * ne <= 512 ? 16 : 8; }

// Sums of N values over the wave's tokens (four rows, or two halves), lane by lane, spread over
// them: row r is left with value i + N/4 * (r % 2) + N/2 * (r / 2) in v[i], i < N/4; half h with
// value i + N/2 * h, i < N/2. Each step swaps halves of the wave between two values and adds, so it
// sums two at once.
template <int L, int N>
__device__ __forceinline__ void sum_of_tokens(float* v) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + N / 2]), false, false);
    v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if (L == 32) return;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + N / 4]), false, false);
    v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
}

// ---------------------------------------------------------------------------
// Choice of one block of a.tok tokens: L lanes to a token, NE experts per lane (expert =
// lane * NE + i). Every lane sorts its experts and keeps the first KEEP >= min(topk, NE); then the
// token's largest first value is chosen topk times and its lane moves on to the next. Writes
// topk_idx and weights, leaves the experts' masks in LDS and the waves' sums of p in lp (waves,
// experts). With L = 16 sixteen waves take 64 tokens at once, four tokens sharing every
// instruction; L = 32 and 64 serve more experts (NE <= 16) or more choices than a row of lanes holds.
// A choice moves only as many heads as there are choices to come. (Top-8, the whole call: 16384 x 256
// 16.8 us with L = 16, 17.7 without the last KEEP choices unrolled, 25.0 with L = 64; 16384 x 384 24.5
// with L = 32, 29.8 with 64. Bound by vector instructions and the chain from one choice to the next;
// lanes that hold four chunks of four experts, so that a load takes whole lines, are no faster.)
// ---------------------------------------------------------------------------
template <int L, int NE, int KEEP>
__device__ __forceinline__ int choose_tokens(const Route& a, int64_t t0, uint64_t* mask, float* lp) {
  constexpr int W = choose_waves(L, NE), GROUPS = W * 64 / L, M = L * NE - 1;
  const int lane = threadIdx.x & (L - 1), w = threadIdx.x >> 6;
  const int group = L == 64 ? __builtin_amdgcn_readfirstlane(w) : threadIdx.x / L;
  const int n = (int)(a.tokens - t0 < a.tok ? a.tokens - t0 : a.tok);
  int routed = 0;
  float next[NE], acc[NE];
  bool on_next = false;
  auto fetch = [&](int tl) {
    on_next = tl < n;
    if (!on_next) return;
    load_logits<NE>(a.logits + (t0 + tl) * a.ld, a.experts, lane, next);
    if (a.valid) on_next = a.valid[t0 + tl];
  };
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    next[i] = __builtin_nanf("");
    acc[i] = 0.0f;
  }
  fetch(group);
  for (int tl = group; tl < n; tl += GROUPS) {
    const int64_t t = t0 + tl;
    const bool on = on_next;
    float z[NE];
    double v[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      z[i] = next[i];
      v[i] = ranked(logit_key(z[i]), (uint32_t)((M - (NE - 1) - lane * NE) | (NE - 1 - i)));
    }
    if (GROUPS < kMaxTok) fetch(tl + GROUPS);
    sort_desc<NE>(v);
    double head[KEEP + 1], my_v = 0.0;           // lane j: the j-th chosen expert
#pragma unroll
    for (int i = 0; i < KEEP; ++i) head[i] = v[i];
    head[KEEP] = 0.0;
    const double top_v = lanes_max<L>(v[0]);
    auto take = [&](int j, int left) {           // `left`: the choices still to come, as many heads to keep
      const double best = lanes_max<L>(head[0]);
      my_v = lane == j ? best : my_v;
      const bool up = head[0] == best;           // its lane's next one moves up
#pragma unroll
      for (int i = 0; i < KEEP; ++i)
        if (i < left) head[i] = up ? head[i + 1] : head[i];
    };
    int j = 0;
    for (; j < a.topk - KEEP; ++j) take(j, KEEP);
#pragma unroll
    for (int left = KEEP - 1; left >= 0; --left)
      if (left < a.topk) take(j++, left);
    const bool mine = on && my_v >= kUsable, any = on && top_v >= kUsable;
    const int my_e = mine ? M - (int)((uint32_t)__double_as_longlong(my_v) & M) : -1;
    const float top = key_logit((uint32_t)top_v);                          // conversions truncate `rest`
    const float num = mine ? expf(key_logit((uint32_t)my_v) - top) : 0.0f;
    const float den = lanes_sum<L>(num);
    if (lane < a.topk) {
      a.topk_idx[t * a.topk + lane] = my_e;
      a.weights[t * a.topk + lane] = mine ? num / den : 0.0f;
    }
    if (mine) atomicOr((unsigned long long*)&mask[my_e], 1ull << tl);
    routed += __popcll(__ballot(any && lane == 0));
    if (a.loss && any) {                         // all lanes of a token or none
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        z[i] = softmax_term(z[i], top);
        sum += z[i];
      }
      const float inv = 1.0f / lanes_sum<L>(sum);
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] = fmaf(z[i], inv, acc[i]);
    }
  }
  if (a.loss) {
    if (L < 64) sum_of_tokens<L, NE>(acc);
    constexpr int MINE = NE * L / 64;            // the wave's tokens share out the experts
    const int e0 = lane * NE + MINE * ((threadIdx.x & 63) / L);
#pragma unroll
    for (int i = 0; i < MINE; ++i)
      if (e0 + i < a.experts) lp[w * a.experts + e0 + i] = acc[i];
  }
  return routed;
}

// One block's masks, routed tokens and (loss wanted) sums of p, in LDS: mask[experts], the
// waves' routed tokens, then waves x experts floats whose first row ends up as the sums.
template <int L, int NE, int KEEP>
__device__ __forceinline__ int choose_block(const Route& a, int64_t t0, uint64_t* mask) {
  constexpr int waves = choose_waves(L, NE);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int* routed_w = reinterpret_cast<int*>(mask + a.experts);
  float* lp = reinterpret_cast<float*>(routed_w + 16);
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) mask[e] = 0;
  __syncthreads();
  const int routed = choose_tokens<L, NE, KEEP>(a, t0, mask, lp);
  if (lane == 0) routed_w[w] = routed;
  __syncthreads();
  int sum = 0;
  for (int i = 0; i < waves; ++i) sum += routed_w[i];
  if (a.loss)
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
      float s = lp[e];
      for (int i = 1; i < waves; ++i) s += lp[i * a.experts + e];
      lp[e] = s;
    }
  return sum;
}

size_t choose_lds(int experts, int waves, bool loss) {
  return (size_t)experts * 8 + 64 + (loss ? (size_t)waves * experts * 4 : 0);
}

template <int L, int NE, int KEEP>
__global__ void __launch_bounds__(choose_waves(L, NE) * 64)
route_choose_kernel(Route a) {
  extern __shared__ uint64_t mask[];
  const int routed = choose_block<L, NE, KEEP>(a, (int64_t)blockIdx.x * a.tok, mask);
  const float* lp = reinterpret_cast<const float*>(mask + a.experts) + 16;
  const int cols = hist_cols(a.experts);
  for (int e = threadIdx.x; e < cols; e += blockDim.x)
    a.hist[(int64_t)blockIdx.x * cols + e] =
        (uint8_t)(e < a.experts ? __popcll((unsigned long long)mask[e]) : e == a.experts ? routed : 0);
  if (a.loss) {
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.psum[(int64_t)blockIdx.x * a.experts + e] = lp[e];
    if (blockIdx.x == 0 && threadIdx.x <= kTallies) a.tally[8 * threadIdx.x] = 0;
  }
}

constexpr int kMaxExperts = 1024;

__device__ __forceinline__ int wave_scan(int v) {            // inclusive
  v += (int)dpp_u32<0x111, 0xF>((uint32_t)v);                // inside the rows of 16 lanes, shifted by 1, 2, 4, 8
  v += (int)dpp_u32<0x112, 0xF>((uint32_t)v);
  v += (int)dpp_u32<0x114, 0xF>((uint32_t)v);
  v += (int)dpp_u32<0x118, 0xF>((uint32_t)v);
  v += (int)dpp_u32<0x142, 0xA>((uint32_t)v);                // the rows' sums onwards
  v += (int)dpp_u32<0x143, 0xC>((uint32_t)v);
  return v;
}

// Offsets from the counts, by one workgroup: every expert's units of pad, what is left of `total`
// dealt out evenly, low experts first. cnt[experts] and off[experts + 1] in LDS, cnt published.
// One wave scans (its lanes take consecutive experts): no partial sums of waves to exchange. The
// last thread, of another wave where there is one, does `beside` meanwhile.
template <typename F>
__device__ __forceinline__ void padded_offsets(const Route& a, const int* cnt, int* off, F&& beside) {
  const int lane = threadIdx.x & 63, G = a.experts, pad = (int)a.pad;
  for (int e = threadIdx.x; e < G; e += blockDim.x) off[e + 1] = cnt[e] ? (cnt[e] - 1) / pad + 1 : 0;
  lds_barrier();
  if (threadIdx.x < 64) {
    const int per = (G + 63) / 64, e0 = lane * per, e1 = min(e0 + per, G);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += off[e + 1];
    int at = wave_scan(sum);
    const int used = (int)lane63((uint32_t)at);
    at -= sum;
    const int spare = a.units - used, each = spare / G, more = spare % G;
    for (int e = e0; e < e1; ++e) {
      at += off[e + 1];
      off[e + 1] = (at + (e + 1) * each + min(e + 1, more)) * pad;
    }
    if (lane == 0) off[0] = 0;
  }
  if (threadIdx.x == blockDim.x - 1) beside();
  lds_barrier();
}

// The slot of choice i of a block of tokens, expert e (-1: none). `start[e]`: where the block's
// tokens begin in expert e's slots.
__device__ __forceinline__ void write_slot(const Route& a, int64_t t0, int i, int e, const uint64_t* mask,
                                           const int* start) {
  const int tl = i / a.topk;
  int64_t slot = -1;
  if (e >= 0) {
    slot = start[e] + __popcll((unsigned long long)(mask[e] & ((1ull << tl) - 1)));
    a.row_index[slot] = (int32_t)(t0 + tl);
  }
  a.slot_of[t0 * a.topk + i] = slot;
}

// This workgroup's share of the padding slots' -1, 16 lanes an expert.
__device__ __forceinline__ void write_padding(const Route& a, const int* cnt, const int* off) {
  const int group = (blockIdx.x * blockDim.x + threadIdx.x) / 16, groups = gridDim.x * blockDim.x / 16;
  for (int e = group; e < a.experts; e += groups)
    for (int64_t s = (int64_t)off[e] + cnt[e] + (threadIdx.x & 15); s < off[e + 1]; s += 16) a.row_index[s] = -1;
}

__device__ __forceinline__ void write_counts(const Route& a, const int* cnt, const int* off, int routed) {
  for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) {
    a.counts[e] = e < a.experts ? cnt[e] : routed;
    a.offsets[e] = off[e];
  }
}

// loss / coef of one block of tokens: experts / (A N) sum over e of counts_e psum_e. loss_terms()
// leaves the waves' sums in LDS (`p` is psum_e of expert threadIdx.x + i blockDim.x, in turn); after
// a barrier block_loss() adds them up.
template <typename P>
__device__ __forceinline__ void loss_terms(const Route& a, const int* cnt, P&& p, double (*red)[2]) {
  double dot = 0.0, all = 0.0;
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    dot += (double)cnt[e] * (double)p(e);
    all += (double)cnt[e];
  }
  dot = wave_sum(dot);
  all = wave_sum(all);
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6][0] = dot;
    red[threadIdx.x >> 6][1] = all;
  }
}
template <int W>
__device__ __forceinline__ double block_loss(const Route& a, int routed, const double (*red)[2]) {
  double dot = red[0][0], all = red[0][1];
#pragma unroll
  for (int i = 1; i < W; ++i) {
    dot += red[i][0];
    all += red[i][1];
  }
  return routed ? (double)a.experts * dot / (all * (double)routed) : 0.0;
}

// ---------------------------------------------------------------------------
// At most one block of tokens: everything in one launch.
// ---------------------------------------------------------------------------
template <int L, int NE, int KEEP>
__global__ void __launch_bounds__(choose_waves(L, NE) * 64)
route_one_block_kernel(Route a) {
  extern __shared__ uint64_t mask[];
  __shared__ int cnt[NE * L], off[NE * L + 1];
  __shared__ double red[16][2];
  const int routed = choose_block<L, NE, KEEP>(a, 0, mask);
  const float* lp = reinterpret_cast<const float*>(mask + a.experts) + 16;
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) cnt[e] = __popcll((unsigned long long)mask[e]);
  __syncthreads();
  if (a.loss) loss_terms(a, cnt, [&](int e) { return lp[e]; }, red);
  padded_offsets(a, cnt, off, [&] {
    if (a.loss) *a.loss = (float)((double)a.coef * block_loss<choose_waves(L, NE)>(a, routed, red));
  });
  write_counts(a, cnt, off, routed);
  const int n = (int)a.tokens * a.topk;
  for (int i = threadIdx.x; i < n; i += blockDim.x) write_slot(a, 0, i, a.topk_idx[i], mask, off);
  write_padding(a, cnt, off);
}

// ---------------------------------------------------------------------------
// Sums of the blocks' histograms, one wave per column: base (exclusive over the blocks), sums.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads)
route_scan_kernel(Route a, int blocks) {
  const int lane = threadIdx.x & 63, cols = hist_cols(a.experts);
  const int c = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (c > a.experts) return;
  int carry = 0;
  for (int b0 = 0; b0 < blocks; b0 += 64) {
    const int b = b0 + lane;
    const int v = b < blocks ? a.hist[(int64_t)b * cols + c] : 0;
    const int incl = wave_scan(v);
    if (b < blocks) a.base[(int64_t)b * cols + c] = carry + incl - v;
    carry += (int)lane63((uint32_t)incl);
  }
  if (lane == 0) a.sums[c] = carry;
}

// A block's share of loss / coef goes into the tallies (cleared by route_choose_kernel); whoever
// completes them writes the loss. One atomic carries the workgroups' count (above bit `frac` + 11)
// and the sum so far in fixed point: loss / coef is at most experts <= 2^10. Integers, so the order
// does not matter, and whoever makes the count complete holds the whole sum. 65536 blocks leave 34
// bits of fraction. Workgroups meet in kTallies first ones, whose last arrivals meet in one more:
// atomics on one address follow one another 10 ns apart.
struct Tally {
  int frac;
  __device__ explicit Tally(int blocks) : frac(62 - (32 - __clz(blocks)) - 11) {}
  __device__ uint64_t one() const { return 1ull << (frac + 11); }
  __device__ uint64_t fixed(double v) const {                // in range whatever the logits
    return (uint64_t)llrint(ldexp(fmin(fmax(v, 0.0), 1024.0), frac));
  }
  __device__ uint64_t add(uint64_t* tally, uint64_t sum) const {
    return atomicAdd((unsigned long long*)tally, (unsigned long long)(one() + sum)) + one() + sum;
  }
  __device__ bool complete(uint64_t total, int parties) const { return total >> (frac + 11) == (uint64_t)parties; }
  __device__ uint64_t sum(uint64_t total) const { return total & (one() - 1); }
};

// ---------------------------------------------------------------------------
// Slots of one block of tokens per workgroup. SCANNED: base and sums come from route_scan_kernel;
// otherwise every workgroup adds up the histograms itself. Each workgroup weighs its block's sums
// of p with the counts for the loss; its atomic starts beside the scan of the offsets and is
// waited for at the end. Latency bounds it: 16384 tokens, 256 experts, about 6 us of which the
// histograms' loads take 1, their sums and the offsets' scan 1 each.
// ---------------------------------------------------------------------------
constexpr int kSlotThreads = 1024;               // one workgroup a CU fills its waves
constexpr int kAhead = 18;                       // histogram loads in flight: 270 blocks of 256 experts in one trip

template <bool SCANNED>
__global__ void __launch_bounds__(kSlotThreads)
route_slots_kernel(Route a, int blocks) {
  extern __shared__ uint64_t mask[];
  __shared__ int cnt[kMaxExperts + 4], off[kMaxExperts + 1], start[kMaxExperts + 4];
  __shared__ uint32_t pairs[4][kMaxExperts / 4 + 1];         // sums of 16 bits, columns 4 i and 4 i + 2, 4 i + 1 and
                                                             // 4 i + 3: over all blocks, then over earlier ones
  __shared__ double red[16][2];
  const int cols = hist_cols(a.experts), blk = blockIdx.x;
  const int64_t t0 = (int64_t)blk * a.tok;
  // what does not depend on the histograms is on its way while they are added up
  const float psum = a.loss && threadIdx.x < a.experts ? a.psum[(int64_t)blk * a.experts + threadIdx.x] : 0.0f;
  const int n = (int)(a.tokens - t0 < a.tok ? a.tokens - t0 : a.tok) * a.topk;
  constexpr int kChoices = kMaxTok * kMaxTopk / kSlotThreads;
  int choice[kChoices];
#pragma unroll
  for (int m = 0; m < kChoices; ++m) {
    const int i = threadIdx.x + m * kSlotThreads;
    choice[m] = i < n ? a.topk_idx[t0 * a.topk + i] : -1;
  }
  for (int e = threadIdx.x; e < a.experts; e += kSlotThreads) mask[e] = 0;
  if (SCANNED) {
    for (int e = threadIdx.x; e <= a.experts; e += kSlotThreads) {
      cnt[e] = a.sums[e];
      start[e] = a.base[(int64_t)blk * cols + e];
    }
    __syncthreads();
  } else {
    // four columns a thread and dword, summed as two pairs of 16 bits (at most kMaxUnscanned
    // blocks of 64)
    for (int i = threadIdx.x; i < cols / 4; i += kSlotThreads) pairs[0][i] = pairs[1][i] = pairs[2][i] = pairs[3][i] = 0;
    lds_barrier();
    const int quads = cols / 4, groups = kSlotThreads / quads;         // quads <= 257
    const int qd = threadIdx.x % quads, first = threadIdx.x / quads;
    if (first < groups) {
      uint32_t lo = 0, hi = 0, blo = 0, bhi = 0;
      for (int b0 = first; b0 < blocks; b0 += kAhead * groups) {
        uint32_t v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)                     // past the end: the last one, not counted
          v[u] = *reinterpret_cast<const uint32_t*>(a.hist + (int64_t)min(b0 + u * groups, blocks - 1) * cols + 4 * qd);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int b = b0 + u * groups;
          const uint32_t some = b < blocks ? v[u] : 0u;
          const uint32_t l = some & 0x00FF00FFu, h = (some >> 8) & 0x00FF00FFu;
          lo += l;
          hi += h;
          blo += b < blk ? l : 0u;
          bhi += b < blk ? h : 0u;
        }
      }
      atomicAdd(&pairs[0][qd], lo);                          // integer sums: the order does not matter
      atomicAdd(&pairs[1][qd], hi);
      atomicAdd(&pairs[2][qd], blo);
      atomicAdd(&pairs[3][qd], bhi);
    }
    lds_barrier();
    for (int e = threadIdx.x; e <= a.experts; e += kSlotThreads) {
      cnt[e] = (int)((pairs[e & 1][e / 4] >> (8 * (e & 2))) & 0xFFFFu);
      start[e] = (int)((pairs[2 + (e & 1)][e / 4] >> (8 * (e & 2))) & 0xFFFFu);
    }
  }
#pragma unroll
  for (int m = 0; m < kChoices; ++m)
    if (choice[m] >= 0)
      atomicOr((unsigned long long*)&mask[choice[m]], 1ull << ((threadIdx.x + m * kSlotThreads) / a.topk));
  if (a.loss) loss_terms(a, cnt, [&](int) { return psum; }, red);      // an expert a thread, as cnt above
  const Tally tally(blocks);
  const int first_tally = blk % kTallies;
  uint64_t met = 0;                                          // not waited for before the slots are written
  padded_offsets(a, cnt, off, [&] {
    if (a.loss) met = tally.add(a.tally + 8 * (1 + first_tally), tally.fixed(block_loss<kSlotThreads / 64>(a, cnt[a.experts], red)));
  });
  for (int e = threadIdx.x; e < a.experts; e += kSlotThreads) start[e] += off[e];
  lds_barrier();
#pragma unroll
  for (int m = 0; m < kChoices; ++m) {
    const int i = threadIdx.x + m * kSlotThreads;
    if (i < n) write_slot(a, t0, i, choice[m], mask, start);
  }
  write_padding(a, cnt, off);
  if (blk == 0) write_counts(a, cnt, off, cnt[a.experts]);
  if (!a.loss || threadIdx.x != kSlotThreads - 1) return;
  if (!tally.complete(met, (blocks - first_tally + kTallies - 1) / kTallies)) return;
  met = tally.add(a.tally, tally.sum(met));
  if (tally.complete(met, min(blocks, kTallies)))
    *a.loss = (float)((double)a.coef * ldexp((double)tally.sum(met), -tally.frac));
}

// ---------------------------------------------------------------------------
// Backward to the logits: one wave per token at a time; the counts stay in registers over the
// tokens of a wave, and the next token's logits are on their way while it works on one. (16384 x
// 256, top-8, both gradients: 11.0 us, 3.2 TB/s of logits and gradients; four tokens to a wave, 16
// lanes each, leave too few waves to wait for memory: 13.6.)
// ---------------------------------------------------------------------------
template <bool OUT32, int NE>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const float* __restrict__ logits, int64_t tokens, int experts, int64_t ld, int topk,
                      const int32_t* __restrict__ topk_idx, const float* __restrict__ weights,
                      const float* __restrict__ d_weights, const int32_t* __restrict__ counts,
                      const float* __restrict__ d_loss, float coef, void* __restrict__ d_logits) {
  __shared__ __attribute__((aligned(16))) float share[kWaves][NE * 64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int i = 0; i < NE; ++i) share[w][lane * NE + i] = 0.0f;    // a row per wave: no barrier
  const int64_t step = (int64_t)gridDim.x * kWaves;
  int64_t t = (int64_t)blockIdx.x * kWaves + w;
  if (t >= tokens) return;
  float c[NE], ahead[NE], scale = 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) c[i] = ahead[i] = 0.0f;
  int e_ahead = -1;
  float w_ahead = 0.0f, dw_ahead = 0.0f;
  auto fetch = [&](int64_t at) {
    if (at >= tokens) return;
    if (d_loss) load_logits<NE>(logits + at * ld, experts, lane, ahead);
    if (lane < topk) {
      e_ahead = topk_idx[at * topk + lane];
      if (d_weights) {
        w_ahead = weights[at * topk + lane];
        dw_ahead = d_weights[at * topk + lane];
      }
    }
  };
  fetch(t);
  if (d_loss) {
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane * NE + i;
      c[i] = e < experts ? (float)counts[e] : 0.0f;
      all += c[i];
    }
    scale = *d_loss * ((coef * experts) / (wave_sum(all) * (float)counts[experts]));
  }
  for (; t < tokens; t += step) {
    const int my_e = e_ahead;
    const float wj = my_e >= 0 ? w_ahead : 0.0f, dwj = my_e >= 0 ? dw_ahead : 0.0f;
    float z[NE], d[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      z[i] = ahead[i];
      d[i] = 0.0f;
    }
    fetch(t + step);
    if (d_loss && __builtin_amdgcn_readlane(my_e, 0) >= 0) {
      float most = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < NE; ++i) most = fmaxf(most, z[i]);
      const float top = key_logit(wave_max_u32(logit_key(most)));
      float sum = 0.0f, pc = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        z[i] = softmax_term(z[i], top);
        sum += z[i];
        pc += z[i] * c[i];
      }
      const float inv = 1.0f / wave_sum(sum), mean = wave_sum(pc) * inv;
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] = (scale * inv) * z[i] * (c[i] - mean);
    }
    if (d_weights) {
      // lane j's share goes to its expert's lane through a row of LDS that is zero in between
      const float g = wj * (dwj - wave_sum(wj * dwj));
      const bool in = my_e >= 0 && my_e < experts;
      if (in) share[w][my_e] = g;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] += share[w][lane * NE + i];
      __builtin_amdgcn_wave_barrier();
      if (in) share[w][my_e] = 0.0f;
    }
    const int64_t at = t * experts + lane * NE;
    const int some = max(0, min(NE, experts - lane * NE));   // this lane's experts
    if (OUT32) {
      if (some == NE) __builtin_memcpy((float*)d_logits + at, d, NE * 4);
      else
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (i < some) ((float*)d_logits)[at + i] = d[i];
    } else {
      uint16_t h[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) h[i] = (uint16_t)bf16x2_rne(d[i], 0.0f);
      if (some == NE) __builtin_memcpy((uint16_t*)d_logits + at, h, NE * 2);
      else
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (i < some) ((uint16_t*)d_logits)[at + i] = h[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Backward of the combine: one workgroup of W waves per token, dy kept in registers (NV vectors
// of 8 per lane) over its slots; the dot products meet in LDS. HBM bounds it. A barrier that waits
// for LDS only keeps the waves on the same slot's rows, which are contiguous (8192 tokens x 8 slots
// x 7168: 638 us without it, 624 with it). A large dO leaves with non-temporal stores (1 GB: 650 ->
// 624 us; 33 MB with plain ones 21.8 us, non-temporal 22.6). The grid's last workgroups clear the
// padding slots of dO.
// ---------------------------------------------------------------------------
template <bool D32, bool STREAM, int W, int NV>
__global__ void __launch_bounds__(W * 64)
combine_backward_kernel(const void* __restrict__ dy, const float* __restrict__ o, int64_t total, int64_t tokens,
                        int topk, int64_t hidden, const int64_t* __restrict__ slot_of,
                        const float* __restrict__ weights, const int32_t* __restrict__ row_index,
                        uint16_t* __restrict__ d_o, float* __restrict__ d_weights) {
  auto col = [&](int i) { return 8 * (int64_t)(i * W * 64 + (int)threadIdx.x); };
  if (blockIdx.x >= tokens) {
    for (int64_t s = blockIdx.x - tokens; s < total; s += gridDim.x - tokens) {
      if (row_index[s] >= 0) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < hidden) *reinterpret_cast<uint4*>(d_o + s * hidden + col(i)) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  __shared__ float red[kMaxTopk][W];
  const int64_t t = blockIdx.x;
  float d[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) d[i][k] = 0.0f;
    if (col(i) < hidden) {
      if (D32) {
        const float4 a = load_stream16f((const float*)dy + t * hidden + col(i));
        const float4 b = load_stream16f((const float*)dy + t * hidden + col(i) + 4);
        d[i][0] = a.x; d[i][1] = a.y; d[i][2] = a.z; d[i][3] = a.w;
        d[i][4] = b.x; d[i][5] = b.y; d[i][6] = b.z; d[i][7] = b.w;
      } else {
        unpack8(load_stream16((const uint16_t*)dy + t * hidden + col(i)), d[i]);
      }
    }
  }
  for (int j = 0; j < topk; ++j) {
    const int64_t slot = slot_of[t * topk + j];
    float dot = 0.0f;
    if (slot >= 0 && slot < total) {                         // others contribute nothing
      const float w = weights[t * topk + j];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) >= hidden) continue;
        const float* p = o + slot * hidden + col(i);
        const float4 a = load_stream16f(p), b = load_stream16f(p + 4);
        dot = fmaf(d[i][0], a.x, fmaf(d[i][1], a.y, fmaf(d[i][2], a.z, fmaf(d[i][3], a.w, dot))));
        dot = fmaf(d[i][4], b.x, fmaf(d[i][5], b.y, fmaf(d[i][6], b.z, fmaf(d[i][7], b.w, dot))));
        store16<STREAM>(d_o + slot * hidden + col(i),
                        make_uint4(bf16x2_rne(w * d[i][0], w * d[i][1]), bf16x2_rne(w * d[i][2], w * d[i][3]),
                                   bf16x2_rne(w * d[i][4], w * d[i][5]), bf16x2_rne(w * d[i][6], w * d[i][7])));
      }
    }
    dot = wave_sum(dot);
    if ((threadIdx.x & 63) == 0) red[j][threadIdx.x >> 6] = dot;
    lds_barrier();
  }
  if (threadIdx.x < topk) {
    float s = red[threadIdx.x][0];
#pragma unroll
    for (int i = 1; i < W; ++i) s += red[threadIdx.x][i];
    d_weights[t * topk + threadIdx.x] = s;
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

// Lanes per token, experts per lane, sorted ones kept: as few lanes as hold 16 experts each and the
// choices. (A wave per token gains nothing where there are few: 8 tokens of 256 experts 5.2 us either
// way.)
template <typename F>
void with_choice(int64_t experts, int64_t topk, F&& go) {
  using std::integral_constant;
  const integral_constant<int, 16> i16;
  const integral_constant<int, 32> i32;
  const integral_constant<int, 8> i8;
  const integral_constant<int, 4> i4;
  if (experts <= 256 && topk <= 16) {
    if (experts <= 64) go(i16, i4, i4);
    else if (experts <= 128) go(i16, i8, i8);
    else if (topk <= 8) go(i16, i16, i8);
    else go(i16, i16, i16);
  } else if (experts <= 512) {
    if (experts <= 128) go(i32, i4, i4);
    else if (experts <= 256) go(i32, i8, i8);
    else if (topk <= 8) go(i32, i16, i8);
    else go(i32, i16, i16);
  } else {
    go(integral_constant<int, 64>{}, i16, i16);
  }
}

// Tokens of a block: as few as keep 256 blocks, one a CU (with the balance loss, 2048 x 256, top-12
// 15.4 -> 12.5 us, 4096 x 256, top-8 14.1 -> 12.0, 8192 x 256 15.3 -> 13.4, against 64), but few
// tokens (those that a workgroup's lanes take at once) are one block and one launch.
int64_t block_tokens(int64_t tokens, int64_t experts) {
  if (tokens <= (experts <= 256 ? 64 : experts <= 512 ? 32 : 16) || tokens > 8192) return 64;
  return tokens <= 4096 ? 16 : 32;
}
int64_t route_blocks(int64_t tokens, int64_t experts) {
  const int64_t tok = block_tokens(tokens, experts);
  return (tokens + tok - 1) / tok;
}

// Whether every slots workgroup adds up all histograms itself, which saves the scan's launch; its
// reads grow with the square of the blocks. (us without and with the scan: 256 blocks of 256 experts
// 16.6 / 18.2, 512 of 256 30.3 / 28.8, 938 of 256 63.0 / 48.3, 512 of 64 17.0 / 18.3, 938 of 64
// 27.8 / 29.5.) The sums have 16 bits, 64 a block.
constexpr int64_t kMaxUnscanned = 1023, kUnscannedBytes = 96 << 10;
bool unscanned(int64_t blocks, int64_t cols) { return blocks <= kMaxUnscanned && blocks * cols <= kUnscannedBytes; }

}  // namespace

// Workspace: tally, psum, base, sums, hist (see Route).
size_t route_ws_bytes(int64_t tokens, int64_t experts) {
  const int64_t nb = route_blocks(tokens, experts), cols = hist_cols((int)experts);
  return (size_t)(64 * (1 + kTallies) + 4 * nb * experts + 4 * nb * cols + 4 * cols + nb * cols);
}

hipError_t launch_route(const float* logits, const uint8_t* valid, int64_t tokens, int64_t experts, int64_t ld,
                        int64_t topk, int64_t pad, int64_t total, float coef, int32_t* topk_idx, float* weights,
                        int32_t* counts, int64_t* offsets, int32_t* row_index, int64_t* slot_of, float* loss, void* ws,
                        hipStream_t st) {
  const int64_t nb = route_blocks(tokens, experts), cols = hist_cols((int)experts);
  Route a{logits, valid, tokens, ld, pad, total, (int)experts, (int)topk, (int)(total / pad),
          (int)block_tokens(tokens, experts), coef, topk_idx, weights, counts, offsets, row_index, slot_of, loss, nullptr,
          nullptr, nullptr, nullptr, nullptr};
  a.tally = (uint64_t*)ws;
  a.psum = (float*)(a.tally + 8 * (1 + kTallies));
  a.base = (int32_t*)(a.psum + nb * experts);
  a.sums = a.base + nb * cols;
  a.hist = (uint8_t*)(a.sums + cols);
  with_choice(experts, topk, [&](auto J, auto N, auto K) {
    constexpr int L = decltype(J)::value, NE = decltype(N)::value, KEEP = decltype(K)::value, W = choose_waves(L, NE);
    const size_t lds = choose_lds((int)experts, W, loss != nullptr);
    if (nb <= 1)
      hipLaunchKernelGGL((route_one_block_kernel<L, NE, KEEP>), dim3(1), dim3(W * 64), lds, st, a);
    else
      hipLaunchKernelGGL((route_choose_kernel<L, NE, KEEP>), dim3((unsigned)nb), dim3(W * 64), lds, st, a);
  });
  if (nb <= 1) return hipGetLastError();
  if (!unscanned(nb, cols)) {
    hipLaunchKernelGGL(route_scan_kernel, dim3((unsigned)((experts + kWaves) / kWaves)), dim3(kThreads), 0, st, a,
                       (int)nb);
    hipLaunchKernelGGL((route_slots_kernel<true>), dim3((unsigned)nb), dim3(kSlotThreads), experts * 8, st, a, (int)nb);
  } else {
    hipLaunchKernelGGL((route_slots_kernel<false>), dim3((unsigned)nb), dim3(kSlotThreads), experts * 8, st, a, (int)nb);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, int64_t tokens, int64_t experts, int64_t ld, int64_t topk,
                                 const int32_t* topk_idx, const float* weights, const float* d_weights,
                                 const int32_t* counts, const float* d_loss, float coef, void* d_logits, int out32,
                                 hipStream_t st) {
  const int64_t want = (tokens + kWaves - 1) / kWaves;
  const dim3 grid((unsigned)(want < 2048 ? want : 2048)), block(kThreads);       // eight workgroups a CU
  auto go = [&](auto O) {
    with_experts(experts, [&](auto N) {
      hipLaunchKernelGGL((route_backward_kernel<decltype(O)::value, decltype(N)::value>), grid, block, 0, st, logits,
                         tokens, (int)experts, ld, (int)topk, topk_idx, weights, d_weights, counts, d_loss, coef,
                         d_logits);
    });
  };
  if (out32) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dy, int d32, const float* o, int64_t total, int64_t tokens,
                                   int64_t topk, int64_t hidden, const int64_t* slot_of, const float* weights,
                                   const int32_t* row_index, void* d_o, float* d_weights, hipStream_t st) {
  using std::integral_constant;
  const bool large = total * hidden * 2 > kStreamBytes;
  // a grid holds fewer than 2^32 threads (1024 to a token at most): more tokens take more launches,
  // and the last one clears the padding slots (rows of no elements: none, row_index is not read)
  const int64_t clearing = hidden > 0 ? (total + 63) / 64 : 0;
  constexpr int64_t kLaunchTokens = (int64_t)1 << 21;
  auto go = [&](auto D, auto N, auto V) {
    constexpr int W = decltype(N)::value, NV = decltype(V)::value;
    constexpr bool DF = decltype(D)::value;
    const auto kernel = large ? combine_backward_kernel<DF, true, W, NV> : combine_backward_kernel<DF, false, W, NV>;
    int64_t t0 = 0;
    do {
      const bool last = tokens - t0 <= kLaunchTokens;
      const int64_t some = last ? tokens - t0 : kLaunchTokens;
      const dim3 grid((unsigned)(some + (last ? clearing : 0)));
      hipLaunchKernelGGL(kernel, grid, dim3(W * 64), 0, st, (const uint8_t*)dy + t0 * hidden * (DF ? 4 : 2), o, total,
                         some, (int)topk, hidden, slot_of + t0 * topk, weights + t0 * topk, row_index,
                         (uint16_t*)d_o, d_weights + t0 * topk);
      t0 += some;
    } while (t0 < tokens);
  };
  auto vectors = [&](auto D) {
    const int64_t v = (hidden / 8 + 63) / 64;               // vectors a lane of one wave would hold
    if (v <= 1) go(D, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (v <= 2) go(D, integral_constant<int, 1>{}, integral_constant<int, 2>{});
    else if (v <= 4) go(D, integral_constant<int, 2>{}, integral_constant<int, 2>{});
    else if (v <= 8) go(D, integral_constant<int, 4>{}, integral_constant<int, 2>{});
    else if (v <= 16) go(D, integral_constant<int, 8>{}, integral_constant<int, 2>{});
    else go(D, integral_constant<int, 16>{}, integral_constant<int, 2>{});
  };
  if (d32) vectors(std::true_type{});
  else vectors(std::false_type{});
  return hipGetLastError();
}

}  // namespace mxq
