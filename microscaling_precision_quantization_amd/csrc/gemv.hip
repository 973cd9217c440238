// Matrix-vector products with 4-bit weights and group scales: a few BF16 rows (the tokens of a decoding
// step) against NVFP4 or MXFP4 weights as the quantizers store them, without quantizing the rows.
//   y[r, n] = t_n sum_k x[r, k] q[n, k] S[n, k / B]                        (gemv)
//   h[r, i] = silu(y[r, i]) y[r, inter + i]                                (gemv_swiglu)
// and the same over the experts a token has chosen, expert by expert: every chosen expert's weight is
// read once, whatever the number of tokens that chose it (moe_decode_gate_up), the down projection with
// the combine behind it (moe_decode_down).
//
// The weights' bytes are all that counts (4.5 or 4.25 bits a weight; one multiplication a weight and
// token). A wave takes tiles of 16 weight rows in chunks of 128 K: lane (n = l % 16, g = l / 16) loads the
// 16 bytes of row n that hold K [32 g, 32 g + 32) of the chunk, makes q S in BF16 from them -- exactly: at
// most six significant bits -- and feeds four 16x16x32 BF16 MFMAs, the rows' x the other operand in the same
// order of K (which order does not matter to a sum, as long as both agree). Sums are binary32; the
// FP32 scale t multiplies the sum. K is split over the waves of a workgroup, whose partial sums meet in
// LDS in a fixed order.
// Element-wise 4-bit weights under group scales: remio.ai ("Miles Blackwell RL"), section "La
// Compatibilidad ..."; moving expert weights through memory can bind harder than arithmetic: same page,
// section "NVFP4 por token ...".
#include <type_traits>

#include "common.h"
#include "swiglu.h"

namespace mxq {

template <int I> using ic = std::integral_constant<int, I>;

namespace gv {

constexpr int kTile = 16;        // weight rows of a tile, and x rows of a column tile
constexpr int kChunk = 128;      // K of a chunk: 32 a lane

__device__ __forceinline__ v8bf as_bf(const uint4& v) {
  v8bf r;
  __builtin_memcpy(&r, &v, 16);
  return r;
}

// Eight E2M1 codes (a dword) times their block scale -> BF16, exact. MXFP4: `s` is the E8M0 code, whose
// power of two the convert applies; NVFP4: S in binary32, multiplied there.
template <int FMT>
__device__ __forceinline__ v8bf weights8(uint32_t w, float S) {
  uint32_t p[4];
  if constexpr (FMT == 4) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, S, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, S, 1);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, S, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, S, 3);
    __builtin_memcpy(&p[0], &a, 4); __builtin_memcpy(&p[1], &b, 4);
    __builtin_memcpy(&p[2], &c, 4); __builtin_memcpy(&p[3], &d, 4);
  } else {
    const v2f_t a = e2m1x2_to_f32<0>(w), b = e2m1x2_to_f32<1>(w), c = e2m1x2_to_f32<2>(w), d = e2m1x2_to_f32<3>(w);
    p[0] = bf16x2_rne(a.x * S, a.y * S);
    p[1] = bf16x2_rne(b.x * S, b.y * S);
    p[2] = bf16x2_rne(c.x * S, c.y * S);
    p[3] = bf16x2_rne(d.x * S, d.y * S);
  }
  return as_bf(make_uint4(p[0], p[1], p[2], p[3]));
}

// The scale codes of a lane's 32 K of a chunk: two E4M3 bytes (NVFP4) or one E8M0 byte (MXFP4).
template <int FMT>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* s) {
  if constexpr (FMT == 2) return *reinterpret_cast<const uint16_t*>(s);
  else return *s;
}

// ... as what multiplies the lane's first and second 16 K.
template <int FMT>
__device__ __forceinline__ void scales_of(uint32_t codes, float (&S)[2]) {
  if constexpr (FMT == 2) {
    S[0] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 0);
    S[1] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 1);
  } else {
    S[0] = S[1] = __uint_as_float(codes << 23);
  }
}

// acc[nt][tt] += the products of NT row tiles and TT column tiles over chunks [c0, c1). wp, sp: the lane's
// row (bytes, scales) at its 32 K of chunk 0; xp: its x row there; on[tt]: the lane's column exists.
template <int FMT, int NT, int TT>
__device__ __forceinline__ void dot(const uint8_t* const (&wp)[NT], const uint8_t* const (&sp)[NT],
                                    const uint16_t* const (&xp)[TT], const bool (&on)[TT], int K, int c0, int c1,
                                    v4f (&acc)[NT][TT]) {
  constexpr int U = TT == 1 ? 4 : TT == 2 ? 2 : 1;        // chunks whose loads go out together
  constexpr int SB = FMT == 2 ? 8 : 4;                    // scale bytes of a row and chunk
  const int g = (threadIdx.x & 63) >> 4;
  for (int c = c0; c < c1; c += U) {
    uint4 w[U][NT], x[U][TT][4];
    uint32_t s[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // chunks past the wave's share and a last chunk's K past the end multiply zeros
      const bool in = c + u < c1 && (c + u) * kChunk + 32 * g < K;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        w[u][n] = make_uint4(0, 0, 0, 0);
        s[u][n] = 0;
        if (in) {
          w[u][n] = *reinterpret_cast<const uint4*>(wp[n] + (int64_t)(c + u) * (kChunk / 2));
          s[u][n] = load_codes<FMT>(sp[n] + (int64_t)(c + u) * SB);
        }
      }
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[u][t][i] = make_uint4(0, 0, 0, 0);
          if (in && on[t]) x[u][t][i] = *reinterpret_cast<const uint4*>(xp[t] + (int64_t)(c + u) * kChunk + 8 * i);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t d[4] = {w[u][n].x, w[u][n].y, w[u][n].z, w[u][n].w};
        float S[2];
        scales_of<FMT>(s[u][n], S);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v8bf a = weights8<FMT>(d[i], S[i / 2]);
#pragma unroll
          for (int t = 0; t < TT; ++t)
            acc[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf(x[u][t][i]), acc[n][t], 0, 0, 0);
        }
      }
  }
}

// The same for at most four x rows, where a column tile of 16 would be mostly empty and cost four loads of x
// for each of weights: the free columns split K further. MFMA row i = (weight row i / 4 of four, K segment i % 4),
// column j = (x row j / 4, segment j % 4), a lane's segment 32 K; only where both segments agree is a
// product of the row and the column, so of a lane's four accumulators one counts, and the four lanes of a
// quad hold the segments' sums. A chunk is 512 K of 16 weight rows: four loads of weights, 64 consecutive
// bytes of a row to four lanes, and four of x.
constexpr int kWide = 512;
template <int FMT, int NT>
__device__ __forceinline__ void dot4(const uint8_t* const (&wp)[NT], const uint8_t* const (&sp)[NT], int64_t row_bytes,
                                     int64_t row_scales, const int (&step)[4], const uint16_t* xp, bool on, int K, int c0,
                                     int c1, v4f (&acc)[NT][4]) {
  constexpr int SB = FMT == 2 ? 32 : 16;                  // scale bytes of a row and chunk
  const int lane = threadIdx.x & 63;
  const int at = 128 * (lane >> 4) + 32 * (lane & 3);     // the lane's K of a chunk
  for (int c = c0; c < c1; ++c) {
    uint4 w[NT][4], x[4];
    uint32_t s[NT][4];
    const bool in = c * kWide + at < K;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        w[n][r] = make_uint4(0, 0, 0, 0);
        if (in) w[n][r] = *reinterpret_cast<const uint4*>(wp[n] + step[r] * row_bytes + (int64_t)c * (kWide / 2));
      }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[n][r] = 0;
        if (in) s[n][r] = load_codes<FMT>(sp[n] + step[r] * row_scales + (int64_t)c * SB);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (in && on) x[i] = *reinterpret_cast<const uint4*>(xp + (int64_t)c * kWide + 8 * i);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t d[4] = {w[n][r].x, w[n][r].y, w[n][r].z, w[n][r].w};
        float S[2];
        scales_of<FMT>(s[n][r], S);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[n][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights8<FMT>(d[i], S[i / 2]), as_bf(x[i]), acc[n][r], 0, 0, 0);
      }
  }
}
// Lane l's result: weight row 4 (l % 4) + l / 16 of the tile, x row (l % 16) / 4.
__device__ __forceinline__ float gather4(const v4f (&acc)[4]) {
  const int seg = threadIdx.x & 3;
  float out = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float v = seg == 0 ? acc[r][0] : seg == 1 ? acc[r][1] : seg == 2 ? acc[r][2] : acc[r][3];
    v += __uint_as_float(dpp_xor1(__float_as_uint(v)));
    v += __uint_as_float(dpp_xor2(__float_as_uint(v)));
    if (seg == r) out = v;
  }
  return out;
}

// The wave's share of a row tile's chunks.
__device__ __forceinline__ void share(int chunks, int part, int parts, int& c0, int& c1) {
  const int per = (chunks + parts - 1) / parts;
  c0 = min(part * per, chunks);
  c1 = min(c0 + per, chunks);
}

// Choices of expert e, in order: the lane gets the (first + q)-th, q = lane % 16 / 4 its x row, or -1; the return
// value is how many there are in all. `col`: four ints of LDS of the wave's own.
__device__ __forceinline__ int choices_of(const int32_t* idx, int n, int e, int first, int* col, int& mine) {
  const int lane = threadIdx.x & 63, q = (lane >> 2) & 3;
  int seen = 0;
  for (int b = 0; b < n; b += 64) {
    const bool hit = b + lane < n && idx[b + lane] == e;
    const uint64_t m = __ballot(hit);
    const int at = seen + __popcll(m & ((1ull << lane) - 1)) - first;
    if (hit && at >= 0 && at < 4) col[at] = b + lane;
    seen += __popcll(m);
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);                     // lgkmcnt(0)
  __builtin_amdgcn_wave_barrier();
  mine = first + q < seen ? col[q] : -1;
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_wave_barrier();
  return seen;
}

// The lane's weight pointers for dot4: rows 4 r + (l % 16) / 4 of the tile at row0 + n0, step[r] rows on from
// the first; rows past the end (n rows) are the last one again, and what they give is not stored.
template <int FMT>
__device__ __forceinline__ void rows4(const uint8_t* w, const uint8_t* s, int64_t row0, int64_t n0, int64_t n, int K,
                                      const uint8_t*& wp, const uint8_t*& sp, int (&step)[4]) {
  const int lane = threadIdx.x & 63, q = (lane >> 2) & 3, seg = 4 * (lane >> 4) + (lane & 3);
  const int left = (int)min((int64_t)kTile, n - n0) - 1;
  const int at = min(q, left);
#pragma unroll
  for (int r = 0; r < 4; ++r) step[r] = min(4 * r + q, left) - at;
  const int64_t row = row0 + n0 + at;
  wp = w + row * (K / 2) + 16 * seg;
  sp = s + row * (K / (FMT == 2 ? 16 : 32)) + (FMT == 2 ? 2 : 1) * seg;
}

}  // namespace gv

struct GemvArgs {
  const uint16_t* x;       // BF16 rows, ld_x apart
  int64_t ld_x;
  int rows;                // dense: x rows. Experts: choices (tokens topk)
  int topk;                // experts: choices a token
  const int32_t* idx;      // experts: (tokens, topk)
  int experts;
  const uint8_t* w;        // (rows, K / 2), experts stacked
  const uint8_t* s;
  const float* t;          // NVFP4
  int t_mode;              // 0 a row, 1 one (of an expert)
  int64_t n;               // rows of the product, gated: inter
  int K;
  void* y;                 // (rows, n): BF16 (gated, out32 = 0) or FP32
  int64_t ld_y;
  int out32;
};

// A workgroup: one tile of 16 rows of the product (gated: the tile's gates and ups), K split over its WV
// waves; TT column tiles hold all x rows.
template <int FMT, bool GATED, int TT, int WV>
__global__ void __launch_bounds__(64 * WV)
gemv_kernel(GemvArgs a) {
  using namespace gv;
  constexpr int NT = GATED ? 2 : 1;
  __shared__ float part[WV][NT][TT][4][64];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kTile;
  const uint8_t *wp[NT], *sp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // rows past the end read the last one's bytes; what they give is not stored
    const int64_t row = n * a.n + min(n0 + lane % kTile, a.n - 1);
    wp[n] = a.w + row * (a.K / 2) + 16 * g;
    sp[n] = a.s + row * (a.K / (FMT == 2 ? 16 : 32)) + (FMT == 2 ? 2 : 1) * g;
  }
  int c0, c1;
  share((a.K + kChunk - 1) / kChunk, wave, WV, c0, c1);
  const uint16_t* xp[TT];
  bool on[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int r = t * kTile + lane % kTile;
    on[t] = r < a.rows;
    xp[t] = a.x + (on[t] ? r : 0) * a.ld_x + 32 * g;
  }
  v4f acc[NT][TT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[n][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  dot<FMT, NT, TT>(wp, sp, xp, on, a.K, c0, c1, acc);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][n][t][r][lane] = acc[n][t][r];
  __syncthreads();
  // accumulator r of lane l is (row 4 (l / 16) + r, column l % 16) of the tile
  for (int o = tid; o < TT * 256; o += 64 * WV) {
    const int t = o >> 8, n = o & 15, c = (o >> 4) & 15;
    const int l = 16 * (n >> 2) + c, r = n & 3, at = t * kTile + c;
    if (at >= a.rows || n0 + n >= a.n) continue;
    float y[NT];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      float v = part[0][k][t][r][l];
#pragma unroll
      for (int w = 1; w < WV; ++w) v += part[w][k][t][r][l];
      if constexpr (FMT == 2) v *= a.t[a.t_mode == 0 ? k * a.n + n0 + n : 0];
      y[k] = v;
    }
    const int64_t to = at * a.ld_y + n0 + n;
    if constexpr (GATED) ((uint16_t*)a.y)[to] = (uint16_t)f32_to_bf16_rne(swiglu_forward(y[0], y[1]));
    else if (a.out32) ((float*)a.y)[to] = y[0];
    else ((uint16_t*)a.y)[to] = (uint16_t)f32_to_bf16_rne(y[0]);
  }
}

// At most four x rows at a time (dot4). Dense: all of them. Experts: blockIdx.y names the expert, either as
// itself or (by_choice) as the choice that names it first; its choices come four by four.
template <int FMT, bool GATED, bool MOE, int WV>
__global__ void __launch_bounds__(64 * WV)
gemv4_kernel(GemvArgs a, int by_choice) {
  using namespace gv;
  constexpr int NT = GATED ? 2 : 1;
  __shared__ float part[2][WV][NT][64];
  __shared__ int col[WV][4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kTile;
  int64_t base = 0;                                       // the expert's first weight row
  int e = 0;
  if constexpr (MOE) {
    if (by_choice) {
      e = a.idx[blockIdx.y];
      bool earlier = false;
      for (int b = 0; b < (int)blockIdx.y; b += 64)
        earlier = earlier || __ballot(b + lane < (int)blockIdx.y && a.idx[b + lane] == e) != 0;
      if ((unsigned)e < (unsigned)a.experts && earlier) return;
    } else {
      e = blockIdx.y;
    }
    // the rows of choices without an expert: zeros
    for (int c = by_choice ? (int)blockIdx.y : 0; c < (by_choice ? (int)blockIdx.y + 1 : blockIdx.y ? 0 : a.rows); ++c) {
      if ((unsigned)a.idx[c] < (unsigned)a.experts) continue;
      if (tid < kTile && n0 + tid < a.n) ((uint16_t*)a.y)[c * a.ld_y + n0 + tid] = 0;
    }
    if ((unsigned)e >= (unsigned)a.experts) return;
    base = (int64_t)e * (GATED ? 2 : 1) * a.n;
  }
  const uint8_t *wp[NT], *sp[NT];
  int step[4];
#pragma unroll
  for (int n = 0; n < NT; ++n) rows4<FMT>(a.w, a.s, base + n * a.n, n0, a.n, a.K, wp[n], sp[n], step);
  int c0, c1;
  share((a.K + kWide - 1) / kWide, wave, WV, c0, c1);
  const int q = (lane >> 2) & 3, n = 4 * (lane & 3) + (lane >> 4);   // the lane's x row and result row
  int seen = a.rows;
  for (int first = 0, buf = 0; first < seen; first += 4, buf ^= 1) {
    int mine = first + q < seen ? first + q : -1;
    if constexpr (MOE) {
      seen = choices_of(a.idx, a.rows, e, first, col[wave], mine);
      if (seen == 0) return;                              // an expert nobody chose (all waves alike)
    }
    const bool on = mine >= 0;
    const uint16_t* xp = a.x + (on ? (MOE ? mine / a.topk : mine) : 0) * a.ld_x + 128 * (lane >> 4) + 32 * (lane & 3);
    v4f acc[NT][4];
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[k][r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    dot4<FMT, NT>(wp, sp, a.K / 2, a.K / (FMT == 2 ? 16 : 32), step, xp, on, a.K, c0, c1, acc);
#pragma unroll
    for (int k = 0; k < NT; ++k) part[buf][wave][k][lane] = gather4(acc[k]);
    __syncthreads();                                      // two buffers: the next pass writes the other one
    if (wave == 0 && on && n0 + n < a.n) {
      float y[NT];
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        float v = part[buf][0][k][lane];
#pragma unroll
        for (int w = 1; w < WV; ++w) v += part[buf][w][k][lane];
        if constexpr (FMT == 2) v *= a.t[a.t_mode == 0 ? base + k * a.n + n0 + n : MOE ? e : 0];
        y[k] = v;
      }
      const int64_t to = mine * a.ld_y + n0 + n;
      if constexpr (GATED) ((uint16_t*)a.y)[to] = (uint16_t)f32_to_bf16_rne(swiglu_forward(y[0], y[1]));
      else if (a.out32) ((float*)a.y)[to] = y[0];
      else ((uint16_t*)a.y)[to] = (uint16_t)f32_to_bf16_rne(y[0]);
    }
  }
}

struct DownArgs {
  const uint16_t* h;       // BF16 (tokens topk, K)
  int tokens, topk;
  const int32_t* idx;
  const float* weights;
  int experts;
  const uint8_t* w;        // (experts, n, K / 2)
  const uint8_t* s;
  const float* t;
  int t_mode;
  int64_t n;
  int K;
  void* y;                 // (tokens, n)
  int out32;
};

// y[t] = sum over the choices j of t of weights[t, j] (W_e h[t, j]): a workgroup has one tile of 16 rows of
// y; its waves share out the chosen experts (and, with few of them, parts of K), each adding to an own
// copy of the tile's (tokens, 16) sums in LDS; the copies meet in wave order.
constexpr int kMaxDecodeExperts = 1024;
template <int FMT, int TCAP, int WV>
__global__ void __launch_bounds__(64 * WV)
decode_down_kernel(DownArgs a, int kparts) {
  using namespace gv;
  __shared__ float sum[WV][TCAP][kTile];
  __shared__ int first_of[kMaxDecodeExperts];
  __shared__ int list[kMaxDecodeExperts];                 // the chosen experts, by first choice
  __shared__ int col[WV][4], found[WV];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kTile;
  const int S = a.tokens * a.topk;
  for (int i = tid; i < a.experts; i += 64 * WV) first_of[i] = 0x7FFFFFFF;
  for (int i = lane; i < TCAP * kTile; i += 64) (&sum[wave][0][0])[i] = 0.0f;
  __syncthreads();
  for (int c = tid; c < S; c += 64 * WV) {
    const int e = a.idx[c];
    if ((unsigned)e < (unsigned)a.experts) atomicMin(&first_of[e], c);
  }
  __syncthreads();
  int experts = 0;
  for (int b = 0; b < S; b += 64 * WV) {                  // compacted in the order of the choices
    const int c = b + tid;
    const int e = c < S ? a.idx[c] : -1;
    const bool lead = (unsigned)e < (unsigned)a.experts && first_of[e] == c;
    const uint64_t m = __ballot(lead);
    if (lane == 0) found[wave] = __popcll(m);
    __syncthreads();
    int before = experts, here = 0;
    for (int w = 0; w < WV; ++w) {
      before += w < wave ? found[w] : 0;
      here += found[w];
    }
    if (lead) list[before + __popcll(m & ((1ull << lane) - 1))] = e;
    experts += here;
    __syncthreads();
  }
  const int chunks = (a.K + kWide - 1) / kWide;
  const int n = 4 * (lane & 3) + (lane >> 4);             // the lane's result row
  for (int item = wave; item < experts * kparts; item += WV) {
    const int e = __builtin_amdgcn_readfirstlane(list[item / kparts]);
    int c0, c1, step[4];
    share(chunks, item % kparts, kparts, c0, c1);
    const uint8_t *wp[1], *sp[1];
    rows4<FMT>(a.w, a.s, (int64_t)e * a.n, n0, a.n, a.K, wp[0], sp[0], step);
    float tw = 1.0f;
    if constexpr (FMT == 2) tw = a.t[a.t_mode == 0 ? (int64_t)e * a.n + min(n0 + n, a.n - 1) : e];
    int seen = 1;
    for (int first = 0; first < seen; first += 4) {
      int mine;
      seen = choices_of(a.idx, S, e, first, col[wave], mine);
      const bool on = mine >= 0;
      const uint16_t* xp = a.h + (int64_t)(on ? mine : 0) * a.K + 128 * (lane >> 4) + 32 * (lane & 3);
      const float wt = on ? a.weights[mine] : 0.0f;
      v4f acc[1][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[0][r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      dot4<FMT, 1>(wp, sp, a.K / 2, a.K / (FMT == 2 ? 16 : 32), step, xp, on, a.K, c0, c1, acc);
      const float v = gather4(acc[0]) * tw;
      // an add in LDS: two lanes meet here where a token names an expert twice
      if (on) atomicAdd(&sum[wave][mine / a.topk][n], wt * v);
    }
  }
  __syncthreads();
  for (int o = tid; o < a.tokens * kTile; o += 64 * WV) {
    const int t = o >> 4, n = o & 15;
    if (n0 + n >= a.n) continue;
    float v = sum[0][t][n];
#pragma unroll
    for (int w = 1; w < WV; ++w) v += sum[w][t][n];
    const int64_t to = (int64_t)t * a.n + n0 + n;
    if (a.out32) ((float*)a.y)[to] = v;
    else ((uint16_t*)a.y)[to] = (uint16_t)f32_to_bf16_rne(v);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// fmt: 2 NVFP4, 4 MXFP4
template <typename F>
static void by_format(int fmt, F&& go) {
  if (fmt == 2) go(ic<2>{});
  else go(ic<4>{});
}

hipError_t launch_gemv(int fmt, int gated, int64_t rows, int64_t n, int64_t K, const void* x, int64_t ld_x, const void* w,
                       const void* s, const float* t, int t_mode, void* y, int64_t ld_y, int out32, hipStream_t st) {
  const GemvArgs a{(const uint16_t*)x, ld_x, (int)rows, 1, nullptr, 1, (const uint8_t*)w, (const uint8_t*)s, t, t_mode, n,
                   (int)K, y, ld_y, out32};
  const dim3 grid((unsigned)((n + gv::kTile - 1) / gv::kTile));
  by_format(fmt, [&](auto F) {
    constexpr int FMT = decltype(F)::value;
    auto go = [&](auto G) {
      constexpr bool GATED = decltype(G)::value != 0;
      constexpr int WV = 8;
      if (rows <= 4) {
        if (K <= 4 * gv::kWide) hipLaunchKernelGGL((gemv4_kernel<FMT, GATED, false, 4>), grid, dim3(64 * 4), 0, st, a, 0);
        else hipLaunchKernelGGL((gemv4_kernel<FMT, GATED, false, 8>), grid, dim3(64 * 8), 0, st, a, 0);
      }
      else if (rows <= 16) hipLaunchKernelGGL((gemv_kernel<FMT, GATED, 1, WV>), grid, dim3(64 * WV), 0, st, a);
      else if (rows <= 32) hipLaunchKernelGGL((gemv_kernel<FMT, GATED, 2, WV>), grid, dim3(64 * WV), 0, st, a);
      else hipLaunchKernelGGL((gemv_kernel<FMT, GATED, 4, WV>), grid, dim3(64 * WV), 0, st, a);
    };
    if (gated) go(ic<1>{});
    else go(ic<0>{});
  });
  return hipGetLastError();
}

hipError_t launch_decode_gate_up(int fmt, int64_t tokens, int64_t topk, int64_t experts, int64_t inter, int64_t K,
                                 const void* x, int64_t ld_x, const int32_t* idx, const void* w, const void* s,
                                 const float* t, int t_mode, void* h, hipStream_t st) {
  const int64_t S = tokens * topk;
  const GemvArgs a{(const uint16_t*)x, ld_x, (int)S, (int)topk, idx, (int)experts, (const uint8_t*)w, (const uint8_t*)s, t,
                   t_mode, inter, (int)K, h, inter, 0};
  // one row of workgroups per expert that can be named: the choices, or the experts where those are fewer
  const int by_choice = S < experts;
  const dim3 grid((unsigned)((inter + gv::kTile - 1) / gv::kTile), (unsigned)(by_choice ? S : experts));
  by_format(fmt, [&](auto F) {
    constexpr int FMT = decltype(F)::value;
    if (K <= 4 * gv::kWide) hipLaunchKernelGGL((gemv4_kernel<FMT, true, true, 4>), grid, dim3(64 * 4), 0, st, a, by_choice);
    else hipLaunchKernelGGL((gemv4_kernel<FMT, true, true, 8>), grid, dim3(64 * 8), 0, st, a, by_choice);
  });
  return hipGetLastError();
}

hipError_t launch_decode_down(int fmt, int64_t tokens, int64_t topk, int64_t experts, int64_t n, int64_t K, const void* h,
                              const int32_t* idx, const float* weights, const void* w, const void* s, const float* t,
                              int t_mode, void* y, int out32, hipStream_t st) {
  const DownArgs a{(const uint16_t*)h, (int)tokens, (int)topk, idx, weights, (int)experts, (const uint8_t*)w,
                   (const uint8_t*)s, t, t_mode, n, (int)K, y, out32};
  constexpr int WV = 16;
  // parts of K so that a few choices still give every wave one
  const int64_t S = tokens * topk, chunks = (K + gv::kWide - 1) / gv::kWide;
  int kparts = 1;
  while (S * kparts < WV && 2 * kparts <= chunks) kparts *= 2;
  const dim3 grid((unsigned)((n + gv::kTile - 1) / gv::kTile));
  by_format(fmt, [&](auto F) {
    if (tokens <= 16)
      hipLaunchKernelGGL((decode_down_kernel<decltype(F)::value, 16, WV>), grid, dim3(64 * WV), 0, st, a, kparts);
    else
      hipLaunchKernelGGL((decode_down_kernel<decltype(F)::value, 64, WV>), grid, dim3(64 * WV), 0, st, a, kparts);
  });
  return hipGetLastError();
}

}  // namespace mxq
