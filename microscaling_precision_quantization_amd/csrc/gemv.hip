// Matrix-vector products with 4-bit weights and group scales: a few BF16 rows (the tokens of a decoding
// step) against NVFP4 or MXFP4 weights as the quantizers store them, without quantizing the rows.
//   y[r, n] = t_n sum_k x[r, k] q[n, k] S[n, k / B]                        (gemv)
//   h[r, i] = silu(y[r, i]) y[r, inter + i]                                (gemv_swiglu)
// and the same over the experts a token has chosen, expert by expert: every chosen expert's weight is
// read once, whatever the number of tokens that chose it (moe_decode_gate_up), the down projection with
// the combine behind it (moe_decode_down).
//
// The weights' bytes are all that counts (4.5 or 4.25 bits a weight; one multiplication a weight and token), so
// they go from memory straight into the registers that the matrix core reads, and nothing is staged: a wave has
// a tile of 16 weight rows (gated: eight gates and their ups) and a share of K, its loads all issued before the
// first product. q S is made in BF16 -- exactly: at most six significant bits -- or, up to four x rows, S follows
// the products. Sums are binary32; the FP32 scale t multiplies the sum. The shares of K meet in LDS in a fixed order.
// A GEMM's tile would be mostly empty and would have to quantize x. At 16 rows and more x out of the L2 takes longer than
// the weights: 64 rows, 7168 -> 2 x 2048 gated 33.8 us, where gemm_swiglu with K in parts takes 25 on BF16 weights of
// 3.5 times the bytes.
// Element-wise 4-bit weights under group scales: remio.ai ("Miles Blackwell RL"), section "La
// Compatibilidad ..."; moving expert weights through memory can bind harder than arithmetic: same page,
// section "NVFP4 por token ...".
#include <algorithm>
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

// Eight E2M1 codes (a dword) times a power of two -> BF16, exact.
__device__ __forceinline__ v8bf codes8(uint32_t w, float p2) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p2, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p2, 1);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p2, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p2, 3);
  v8bf r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1]; r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}
// ... times their block scale: MXFP4, the E8M0 code's power of two; NVFP4: S, multiplied in binary32.
template <int FMT>
__device__ __forceinline__ v8bf weights8(uint32_t w, float S) {
  if constexpr (FMT == 4) {
    return codes8(w, S);
  } else {
    uint32_t p[4];
    const v2f_t a = e2m1x2_to_f32<0>(w), b = e2m1x2_to_f32<1>(w), c = e2m1x2_to_f32<2>(w), d = e2m1x2_to_f32<3>(w);
    p[0] = bf16x2_rne(a.x * S, a.y * S);
    p[1] = bf16x2_rne(b.x * S, b.y * S);
    p[2] = bf16x2_rne(c.x * S, c.y * S);
    p[3] = bf16x2_rne(d.x * S, d.y * S);
    return as_bf(make_uint4(p[0], p[1], p[2], p[3]));
  }
}

// ... the scale codes of a lane's 32 K of a chunk (two E4M3 bytes, or one E8M0 byte) as what multiplies its
// first and second 16 K.
// E8M0: the code becomes the exponent field of what the scaled convert takes, which reads that field alone, so that
// code 0, a +0, is the scale 2^-127 and the weights are BF16 subnormals, which the MFMA keeps.
template <int FMT>
__device__ __forceinline__ void scales_of(uint32_t codes, float (&S)[2]) {
  if constexpr (FMT == 2) {
    S[0] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 0);
    S[1] = __builtin_amdgcn_cvt_f32_fp8((int)codes, 1);
  } else {
    S[0] = S[1] = __uint_as_float(codes << 23);
  }
}

// Loads go through buffer descriptors: what lies past their end, or is switched off by kOff, reads zeros, so
// rows past the last, K past the end and absent x rows need no branch.
constexpr uint32_t kOff = 0x80000000u;
constexpr uint32_t kMaxRecords = 0x7FFFFFFFu;
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)min(bytes, (int64_t)kMaxRecords), 0x00020000);
}
__device__ __forceinline__ uint4 load16(Rsrc r, uint32_t voff, uint32_t soff) {
  typedef unsigned int v4u_t __attribute__((ext_vector_type(4)));
  const v4u_t v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <int FMT>
__device__ __forceinline__ uint32_t load_codes(Rsrc r, uint32_t voff, uint32_t soff) {
  if constexpr (FMT == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)voff, (int)soff, 0);
  else return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, (int)voff, (int)soff, 0);
}
template <int FMT> constexpr int kScaleK = FMT == 2 ? 16 : 32;      // K of a scale
template <int FMT> constexpr int kCodes = FMT == 2 ? 2 : 1;         // codes of a lane's 32 K

// ---------------------------------------------------------------------------
// More than four x rows: a column tile of 16 is 16 x rows
// ---------------------------------------------------------------------------
// acc[r][t] += the products of RT row tiles and TT column tiles over chunks [c0, c1). rw, rs: the tiles' weights
// and scales; wo, so: the lane's row at its 32 K of chunk 0; xo[t]: its x row there.
template <int FMT, int RT, int TT, bool AHEAD>
__device__ __forceinline__ void dot16(const Rsrc (&rw)[RT], const Rsrc (&rs)[RT], Rsrc rx, uint32_t wo, uint32_t so,
                                      const uint32_t (&xo)[TT], int K, int c0, int c1, v4f (&acc)[RT][TT]) {
  constexpr int U = RT * TT >= 4 ? 1 : RT * TT == 2 ? 2 : 4;   // chunks whose weights' loads go out together
  const int k0 = 32 * ((threadIdx.x & 63) >> 4);
  for (int c = c0; c < c1; c += U) {
    uint4 w[U][RT];
    uint32_t s[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = c + u < c1 && (c + u) * kChunk + k0 < K;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        w[u][r] = load16(rw[r], in ? wo : kOff, (uint32_t)(c + u) * (kChunk / 2));
        s[u][r] = load_codes<FMT>(rs[r], in ? so : kOff, (uint32_t)(c + u) * (kChunk / kScaleK<FMT>));
      }
    }
    uint4 x[AHEAD ? U : 1][TT][4];
    auto load_x = [&](int u) {
      const bool in = c + u < c1 && (c + u) * kChunk + k0 < K;
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[AHEAD ? u : 0][t][i] = load16(rx, (in ? xo[t] : kOff) + 16 * i, (uint32_t)(c + u) * (2 * kChunk));
    };
    if constexpr (AHEAD) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_x(u);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u >= c1) break;
      if constexpr (!AHEAD) load_x(u);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t d[4] = {w[u][r].x, w[u][r].y, w[u][r].z, w[u][r].w};
        float S[2];
        scales_of<FMT>(s[u][r], S);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v8bf a = weights8<FMT>(d[i], S[i / 2]);
#pragma unroll
          for (int t = 0; t < TT; ++t)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf(x[AHEAD ? u : 0][t][i]), acc[r][t], 0, 0, 0);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// At most four x rows
// ---------------------------------------------------------------------------
// A column tile of 16 x rows would be mostly empty, so the 4x4x4 MFMA takes over, which is sixteen independent
// 4 x 4 products: block b = l / 4 is a K segment of 32, its four lanes four weight rows of A and four x
// rows of B, and each instruction advances every block by four K. A chunk is 512 K of the tile's 16 weight
// rows: four loads of weights (lane l: row 4 r + l % 4, 16 bytes), and four of x (x row l % 4). As no sum crosses
// lanes before the end, NVFP4's block scale can follow the products: the codes go to BF16 as they are
// (one convert a pair), 16 K sum up in the matrix core, and one FMA a weight row, its scale read from the
// lane of the quad that holds the row, adds them: 0.75 vector instructions a weight against 2 for scaled
// BF16 operands.
constexpr int kWide = 512;
typedef short v4s __attribute__((ext_vector_type(4)));
// The lane's part of the tile: two descriptors (rows 0 .. 7 and 8 .. 15), its offsets within each.
struct Rows4 {
  Rsrc w[2], s[2];
  uint32_t wo, so, w4, s4;                                // w4, s4: four rows on
};
// first[h]: the weight row that half h of the tile begins with, rows[h] (at most 8) how many it has
template <int FMT>
__device__ __forceinline__ Rows4 rows4(const uint8_t* w, const uint8_t* s, const int64_t (&first)[2],
                                       const int64_t (&rows)[2], int K) {
  const int lane = threadIdx.x & 63, i = lane & 3, seg = lane >> 2;
  const int64_t wb = K / 2, sb = K / kScaleK<FMT>;
  Rows4 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    r.w[h] = rsrc(w + first[h] * wb, rows[h] * wb);
    r.s[h] = rsrc(s + first[h] * sb, rows[h] * sb);
  }
  r.wo = (uint32_t)(i * wb) + 16 * seg;
  r.so = (uint32_t)(i * sb) + kCodes<FMT> * seg;
  r.w4 = (uint32_t)(4 * wb);
  r.s4 = (uint32_t)(4 * sb);
  return r;
}
__device__ __forceinline__ v4s half8(const v8bf& v, int h) {
  v4s r;
  __builtin_memcpy(&r, reinterpret_cast<const char*>(&v) + 8 * h, 8);
  return r;
}
template <int R>
__device__ __forceinline__ float quad_lane(float v) {      // lane R of the quad's
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), R * 0x55, 0xF, 0xF, true));
}
// acc[r][i] += the lane's segment of weight row 4 r + i times x row l % 4, over chunks [c0, c1). x_of() is asked for
// the lane's x row at its K of chunk 0 (or kOff), with the first weights on their way.
template <int FMT, typename F>
__device__ __forceinline__ void dot4(const Rows4& rows, Rsrc rx, F&& x_of, int K, int c0, int c1, v4f (&acc)[4]) {
  const int at = 32 * ((threadIdx.x & 63) >> 2);          // the lane's K of a chunk
  uint32_t xo = kOff;
  for (int c = c0; c < c1; ++c) {
    uint4 w[4], x[4];
    uint32_t s[4];
    const bool in = c * kWide + at < K;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      w[r] = load16(rows.w[r / 2], in ? rows.wo + r % 2 * rows.w4 : kOff, (uint32_t)c * (kWide / 2));
#pragma unroll
    for (int r = 0; r < 4; ++r)
      s[r] = load_codes<FMT>(rows.s[r / 2], in ? rows.so + r % 2 * rows.s4 : kOff, (uint32_t)c * (kWide / kScaleK<FMT>));
    if (c == c0) xo = x_of();
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = load16(rx, (in ? xo : kOff) + 16 * i, (uint32_t)c * (2 * kWide));
    __builtin_amdgcn_sched_barrier(0);                    // all of them in flight: the scheduler would sink some
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t d[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
      float S[2];
      scales_of<FMT>(s[r], S);
#pragma unroll
      for (int h = 0; h < 2; ++h) {                       // the lane's first and second 16 K
        v4f sum = FMT == 4 ? acc[r] : v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 2 * h; i < 2 * h + 2; ++i) {
          const v8bf q = codes8(d[i], FMT == 4 ? S[h] : 1.0f), xi = as_bf(x[i]);
          sum = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(half8(q, 0), half8(xi, 0), sum, 0, 0, 0);
          sum = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(half8(q, 1), half8(xi, 1), sum, 0, 0, 0);
        }
        if constexpr (FMT == 4) {
          acc[r] = sum;
        } else {
          acc[r][0] = __builtin_fmaf(quad_lane<0>(S[h]), sum[0], acc[r][0]);
          acc[r][1] = __builtin_fmaf(quad_lane<1>(S[h]), sum[1], acc[r][1]);
          acc[r][2] = __builtin_fmaf(quad_lane<2>(S[h]), sum[2], acc[r][2]);
          acc[r][3] = __builtin_fmaf(quad_lane<3>(S[h]), sum[3], acc[r][3]);
        }
      }
    }
  }
}
// The sums over the four segments of each row of 16 lanes: lane l of it is left with weight rows 4 (l / 4) + (0 .. 3)
// of the tile, x row l % 4.
__device__ __forceinline__ float4 gather4(v4f (&acc)[4]) {
  const int quad = (threadIdx.x >> 2) & 3;
  float out[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = acc[r][i];
      v += dpp_f32<0x124, 0xF>(v);                        // rotations by 4 and 8 lanes
      v += dpp_f32<0x128, 0xF>(v);
      if (r == 0) out[i] = v;
      else out[i] = quad == r ? v : out[i];
    }
  return make_float4(out[0], out[1], out[2], out[3]);
}
__device__ __forceinline__ uint32_t x_off4() { return 64 * ((threadIdx.x & 63) >> 2); }

// The wave's share of a row tile's chunks.
__device__ __forceinline__ void share(int chunks, int part, int parts, int& c0, int& c1) {
  const int per = (chunks + parts - 1) / parts;
  c0 = min(part * per, chunks);
  c1 = min(c0 + per, chunks);
}

// Choices as bits, 64 a word.
template <int NB>
struct Who {
  uint64_t m[NB];
  __device__ __forceinline__ int count() const {
    int n = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) n += __popcll(m[b]);
    return n;
  }
  // the lane's: the (first + q)-th, q = lane % 4 its x row, or -1
  __device__ __forceinline__ int pick(int first) const {
    int left = first + (threadIdx.x & 3), at = -1;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = __popcll(m[b]);
      if (at < 0 && left < n) {
        uint64_t w = m[b];
        for (; left > 0; --left) w &= w - 1;
        at = 64 * b + __builtin_ctzll(w);
      }
      left -= n;
    }
    return at;
  }
};

// Choices of expert e, in order: the lane gets the (first + q)-th, q = lane % 4 its x row, or -1; the return
// value is how many there are in all. `col`: four ints of LDS of the wave's own.
__device__ __forceinline__ int choices_of(const int32_t* idx, int n, int e, int first, int* col, int& mine) {
  const int lane = threadIdx.x & 63, q = lane & 3;
  int seen = 0;
  for (int b = 0; b < n; b += 256) {                      // four loads in flight
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = b + 64 * i + lane < n ? idx[b + 64 * i + lane] : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool hit = v[i] == e;                         // e >= 0
      const uint64_t m = __ballot(hit);
      const int at = seen + __popcll(m & ((1ull << lane) - 1)) - first;
      if (hit && at >= 0 && at < 4) col[at] = b + 64 * i + lane;
      seen += __popcll(m);
    }
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);                     // lgkmcnt(0)
  __builtin_amdgcn_wave_barrier();
  mine = first + q < seen ? col[q] : -1;
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_wave_barrier();
  return seen;
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
  int64_t n;               // columns of the result: rows of the product, gated: inter
  int K;
  void* y;                 // (rows, n): BF16 (gated, out32 = 0) or FP32
  int64_t ld_y;
  int out32;
};

// A workgroup has one tile of 16 weight rows: 16 columns of the result, or (gated) 8, their gates and their ups.
template <bool GATED> constexpr int kTileOut = GATED ? 8 : 16;

__device__ __forceinline__ void store_y(void* y, int64_t at, float v, int f32) {
  if (f32) ((float*)y)[at] = v;
  else ((uint16_t*)y)[at] = (uint16_t)f32_to_bf16_rne(v);
}

// TT column tiles hold all x rows. A workgroup has WV waves: KS of them share a tile's K, the others have tiles of
// their own, RT each, and the same x at about the same time. The weights a descriptor spans (gated: all 2 n rows
// from the tile on) are below 2^31 bytes: the dense calls refuse more, launch_choices sends it to gemv4_kernel.
// A tile needs all of x, 2 rows bytes for every 8 of its weights' bytes: past 16 rows the reads of x out of the L2
// are what takes the time (2048 x 7168 gated, 16 rows 12.8 us, 32 20.4, 64 33.8; the weights alone 3.1), below it
// the latency of three loads in turn. AH: x ahead of the products along with the weights (32 rows 23.0 -> 20.4, 16 rows, 129280 x 7168 245 -> 205);
// short shares with one column tile lose by it (7168 x 2048 7.9 -> 9.0).
// MOE: blockIdx.y is an expert, its choices are listed in LDS and taken 16 TT at a time.
constexpr int kMaxChoices = 2048;
template <int FMT, bool GATED, int TT, int RT, int KS, int WV, bool MOE>
__global__ void __launch_bounds__(64 * WV)
gemv_kernel(GemvArgs a) {
  using namespace gv;
  constexpr int NO = kTileOut<GATED>, NW = WV / KS;
  constexpr bool AH = KS == 16 || TT >= 2 || RT == 2;
  constexpr int PER = NW * RT * NO;                       // columns of the result
  __shared__ float part[WV][RT][TT][4][64];
  __shared__ uint16_t list[MOE ? kMaxChoices : 1];
  __shared__ int hits[MOE ? kMaxChoices / 64 : 1];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t b0 = (int64_t)blockIdx.x * PER;
  int64_t base = 0;                                       // the expert's first weight row
  int e = 0, seen = a.rows;
  if constexpr (MOE) {
    e = blockIdx.y;
    base = (int64_t)e * (GATED ? 2 : 1) * a.n;
    if (GATED && e == 0) {                                // choices without an expert
      for (int c = tid; c < a.rows; c += 64 * WV)
        if ((unsigned)a.idx[c] >= (unsigned)a.experts)
          for (int i = 0; i < PER && b0 + i < a.n; ++i) ((uint16_t*)a.y)[c * a.ld_y + b0 + i] = 0;
    }
    constexpr int W = kMaxChoices / 64 / WV;              // words of 64 choices a wave
    uint64_t m[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int c = 64 * (i * WV + wave) + lane;
      m[i] = __ballot(c < a.rows && a.idx[c] == e);
      if (lane == 0) hits[i * WV + wave] = __popcll(m[i]);
    }
    __syncthreads();
    seen = 0;
#pragma unroll
    for (int i = 0; i < W; ++i)
      for (int w = 0; w < WV; ++w) {
        if (w == wave && (m[i] >> lane & 1)) list[seen + __popcll(m[i] & ((1ull << lane) - 1))] = 64 * (i * WV + w) + lane;
        seen += hits[i * WV + w];
      }
    if (seen == 0) return;                                // all waves alike
    __syncthreads();
  }
  const int64_t wb = a.K / 2, sb = a.K / kScaleK<FMT>;
  Rsrc rw[RT], rs[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {                          // a tile past the end has no rows
    const int64_t n0 = b0 + (wave / KS * RT + r) * NO;
    const int64_t rows = n0 >= a.n ? 0 : (GATED ? 2 * a.n : min(a.n, n0 + kTile)) - n0;   // gates past n read ups, not stored
    rw[r] = rsrc(a.w + (base + n0) * wb, rows * wb);
    rs[r] = rsrc(a.s + (base + n0) * sb, rows * sb);
  }
  const int m = lane % kTile;
  const int64_t row = GATED && m >= 8 ? a.n + m - 8 : m;
  const uint32_t wo = (uint32_t)(row * wb) + 16 * g, so = (uint32_t)(row * sb) + kCodes<FMT> * g;
  const Rsrc rx = rsrc(a.x, (((MOE ? a.rows / a.topk : a.rows) - 1) * a.ld_x + a.K) * 2);
  int c0, c1;
  share((a.K + kChunk - 1) / kChunk, wave % KS, KS, c0, c1);
  for (int first = 0; first < seen; first += 16 * TT) {
    uint32_t xo[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int r = first + t * kTile + m;
      xo[t] = r < seen ? (uint32_t)((MOE ? list[r] / a.topk : r) * a.ld_x + 32 * g) * 2 : kOff;
    }
    v4f acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    dot16<FMT, RT, TT, AH>(rw, rs, rx, wo, so, xo, a.K, c0, c1, acc);
    if (MOE && first) __syncthreads();                    // part has been read
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][r][t][i][lane] = acc[r][t][i];
    __syncthreads();
    // accumulator r of lane l is (row 4 (l / 16) + r, column l % 16) of the tile
    for (int o = tid; o < TT * 16 * PER; o += 64 * WV) {
      const int n = o % PER, at = o / PER, tile = n / NO;
      if (first + at >= seen || b0 + n >= a.n) continue;
      float y[2];
#pragma unroll
      for (int k = 0; k < (GATED ? 2 : 1); ++k) {
        const int i = n % NO + 8 * k, l = 16 * (i >> 2) + at % 16;
        const float* q = &part[tile / RT * KS][tile % RT][at / 16][i & 3][l];
        float v = q[0];
#pragma unroll
        for (int w = 1; w < KS; ++w) v += q[w * (RT * TT * 256)];
        if constexpr (FMT == 2) v *= a.t[a.t_mode == 0 ? base + k * a.n + b0 + n : e];
        y[k] = v;
      }
      const int to = MOE ? list[first + at] : at;
      store_y(a.y, to * a.ld_y + b0 + n, GATED ? swiglu_forward(y[0], y[1]) : y[0], !GATED && a.out32);
    }
    if (!MOE) return;                                     // dense: 16 TT hold all rows
  }
}

// At most four x rows at a time (dot4). Dense: all of them. Experts: the choices of one expert, four by four.
// Up to 512 choices are looked at by every wave at once and kept as bits (NB words of 64); NB = 0 finds them
// through LDS, pass by pass (one token, 8 of 256 experts: 38 us, as bits 30). blockIdx.y is a choice, which works
// for its expert if it is the first to name it, or (by_choice = 0) the expert.
// Bound by the weights' way from memory: one token, 8 of 256 experts, 2048 x 7168, gate_up 30.0 us = 4.4 TB/s (a
// large copy 5.06), down 16 + 4 us for the combine; 32 tokens, 8 of 128, 768 x 2048, gate_up 46 us = 4.1 TB/s,
// down 28 + 4 (its K of 768 leaves half of every second chunk empty). Small ones are latency: the launch, the
// first loads, the join: 2048 x 7168, one row, 4.7 us for 1.6 us of bytes.
// Waves a SIMD: as many as leave no spills (six at 64 choices, four where x rows are dense).
constexpr int kDense = -1;
// KS waves share a tile's K; a workgroup has at least four waves, so 4 / KS tiles.
template <int FMT, bool GATED, int NB, int KS>
__global__ void __launch_bounds__(64 * (KS < 4 ? 4 : KS)) __attribute__((amdgpu_waves_per_eu(NB == 1 ? 6 : NB == kDense ? 4 : 5)))
gemv4_kernel(GemvArgs a, int by_choice) {
  using namespace gv;
  constexpr int WV = KS < 4 ? 4 : KS, TILES = WV / KS;
  constexpr bool MOE = NB != kDense;
  constexpr int NO = kTileOut<GATED>;
  __shared__ __attribute__((aligned(16))) float part[2][4 * WV][64];
  __shared__ int col[NB == 0 ? WV : 1][4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = ((int64_t)blockIdx.x * TILES + wave / KS) * NO;     // a tile past the end: no rows, no stores
  const int64_t b0 = (int64_t)blockIdx.x * TILES * NO;                   // the workgroup's first column
  int64_t base = 0;                                       // the expert's first weight row
  int e = 0, seen = a.rows;
  Who<(NB > 0 ? NB : 1)> who;
  if constexpr (MOE) {
    const int y = blockIdx.y;
    auto none = [&](int i) { return (unsigned)i >= (unsigned)a.experts; };
    auto zero_row = [&](int c) {                          // by one thread: the choice c has no expert
      if constexpr (GATED)                                // (the down call's join skips it)
          for (int i = 0; i < TILES * NO && b0 + i < a.n; ++i) ((uint16_t*)a.y)[c * a.ld_y + b0 + i] = 0;
    };
    if constexpr (NB > 0) {
      int v[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) v[b] = 64 * b + lane < a.rows ? a.idx[64 * b + lane] : -1;
      e = y;
      if (by_choice) {
        e = __builtin_amdgcn_readfirstlane(a.idx[y]);
        if (none(e)) {
          if (tid == 0) zero_row(y);
          return;
        }
      } else if (y == 0) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (wave == b % WV && 64 * b + lane < a.rows && none(v[b])) zero_row(64 * b + lane);
      }
      bool earlier = false;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        who.m[b] = __ballot(v[b] == e);
        const int before = y - 64 * b;                    // choices of this word ahead of y
        if (before > 0) earlier = earlier || (who.m[b] << (before < 64 ? 64 - before : 0)) != 0;
      }
      seen = who.count();
      if (seen == 0 || (by_choice && earlier)) return;
    } else {
      if (by_choice) {
        e = __builtin_amdgcn_readfirstlane(a.idx[y]);
        if (none(e)) {
          if (tid == 0) zero_row(y);
          return;
        }
        for (int b = 0; b < y; b += 64)
          if (__ballot(b + lane < y && a.idx[b + lane] == e)) return;
      } else {
        e = y;
        if (y == 0)
          for (int c = tid; c < a.rows; c += 64 * WV)
            if (none(a.idx[c])) zero_row(c);
      }
    }
    base = (int64_t)e * (GATED ? 2 : 1) * a.n;
  }
  const int64_t second = GATED ? a.n + n0 : n0 + 8;       // the tile's second half: the ups, or eight rows on
  const Rows4 rows = rows4<FMT>(a.w, a.s, {base + n0, base + second},
                                {max(min(a.n - n0, (int64_t)8), (int64_t)0),
                                 max(min((GATED ? 2 : 1) * a.n - second, (int64_t)8), (int64_t)0)},
                                a.K);
  const Rsrc rx = rsrc(a.x, (((MOE ? a.rows / a.topk : a.rows) - 1) * a.ld_x + a.K) * 2);
  int c0, c1;
  share((a.K + kWide - 1) / kWide, wave % KS, KS, c0, c1);
  // lane l of the tile's first wave joins the sums of x row l % 4, product row l / 4
  const int i = lane >> 2, n = GATED ? i % 8 : i;
  float t = 1.0f;
  if (FMT == 2 && wave % KS == 0 && n0 + n < a.n) t = a.t[a.t_mode == 0 ? base + (GATED ? i / 8 * a.n : 0) + n0 + n : MOE ? e : 0];
  for (int first = 0, buf = 0; first < seen; first += 4, buf ^= 1) {
    int mine = -1;                                        // the lane's x row, or choice
    if constexpr (NB == 0) {
      seen = choices_of(a.idx, a.rows, e, first, col[wave], mine);
      if (seen == 0) return;                              // an expert nobody chose (all waves alike)
    }
    auto x_of = [&]() -> uint32_t {
      if constexpr (NB > 0) mine = who.pick(first);
      if constexpr (NB == kDense) mine = first + lane % 4 < seen ? first + lane % 4 : -1;
      return mine >= 0 ? (uint32_t)((MOE ? mine / a.topk : mine) * a.ld_x * 2) + x_off4() : kOff;
    };
    v4f acc[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    dot4<FMT>(rows, rx, x_of, a.K, c0, c1, acc);
    *reinterpret_cast<float4*>(&part[buf][wave * 4 + lane / 16][4 * (lane % 16)]) = gather4(acc);
    if constexpr (KS > 1) __syncthreads();                // two buffers: the next pass writes the other one
    else __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0): the wave's own
    if (wave % KS == 0) {
      const float* p = &part[buf][4 * wave][16 * (i / 4) + 4 * (lane % 4) + i % 4];
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 4 * KS; ++w) v += p[64 * w];
      if constexpr (FMT == 2) v *= t;
      const bool store = mine >= 0 && n0 + n < a.n;
      if constexpr (GATED) {                              // the up of lane l's gate is 32 lanes on
        const float up = __shfl_xor(v, 32, 64);
        if (store && i < 8) store_y(a.y, mine * a.ld_y + n0 + n, swiglu_forward(v, up), 0);
      } else {
        if (store) store_y(a.y, mine * a.ld_y + n0 + n, v, a.out32);
      }
    }
  }
}

// The combine of the down call: y[t, n] = sum over j of weights[t, j] parts[t topk + j, n], in the order of j, the
// choices that name no expert left out (their rows of parts were not written: read, so that no load waits for
// another's answer, but not used).
__global__ void __launch_bounds__(256)
decode_join_kernel(const float* __restrict__ parts, const int32_t* __restrict__ idx, const float* __restrict__ weights,
                   int topk, int experts, int64_t n, void* __restrict__ y, int out32) {
  constexpr int U = 8;                                    // loads in flight
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int c0 = blockIdx.y * topk;
  if (col >= n) return;
  float v = 0.0f;
  for (int j = 0; j < topk; j += U) {
    float p[U], w[U];
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + min(j + u, topk - 1);
      p[u] = parts[c * n + col];
      e[u] = idx[c];
      w[u] = weights[c];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + u < topk && (unsigned)e[u] < (unsigned)experts) v = __builtin_fmaf(w[u], p[u], v);
  }
  store_y(y, blockIdx.y * n + col, v, out32);
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

// `each` workgroups in y. K is split over as few waves as make 16384, four times what the CUs hold at once: a wave's
// fixed work (finding its choices, joining sums) is worth one to two chunks, but waves that end at different times
// keep loads in flight. With 4096 / 8192 / 16384: 32 tokens, 8 of 128 experts, gate_up 51 / 51 / 46.5 us; one row
// of x, 65536 x 4096 35.3 / 35.4 / 33.0, 129280 x 7168 115 / 112 / 108, 16384 x 4096 11.0 / 11.9 / 11.9.
template <int FMT, bool GATED, int NB>
static void launch_gemv4(const GemvArgs& a, int64_t tiles, int64_t each, int by_choice, hipStream_t st) {
  const int64_t chunks = (a.K + gv::kWide - 1) / gv::kWide, waves = tiles * each;
  auto go = [&](auto KSC) {
    constexpr int KS = decltype(KSC)::value, TILES = KS < 4 ? 4 / KS : 1;
    hipLaunchKernelGGL((gemv4_kernel<FMT, GATED, NB, KS>), dim3((unsigned)((tiles + TILES - 1) / TILES), (unsigned)each),
                       dim3(64 * (KS < 4 ? 4 : KS)), 0, st, a, by_choice);
  };
  int ks = 1;
  while (ks < 8 && 2 * ks <= chunks && waves * ks < 16384) ks *= 2;
  if (ks == 1) go(ic<1>{});
  else if (ks == 2) go(ic<2>{});
  else if (ks == 4) go(ic<4>{});
  else go(ic<8>{});
}

hipError_t launch_gemv(int fmt, int gated, int64_t rows, int64_t n, int64_t K, const void* x, int64_t ld_x, const void* w,
                       const void* s, const float* t, int t_mode, void* y, int64_t ld_y, int out32, hipStream_t st) {
  const GemvArgs a{(const uint16_t*)x, ld_x, (int)rows, 1, nullptr, 1, (const uint8_t*)w, (const uint8_t*)s, t, t_mode, n,
                   (int)K, y, ld_y, out32};
  const int64_t tile = gated ? kTileOut<true> : kTileOut<false>, tiles = (n + tile - 1) / tile;
  by_format(fmt, [&](auto F) {
    constexpr int FMT = decltype(F)::value;
    auto go = [&](auto G) {
      constexpr bool GATED = decltype(G)::value != 0;
      if (rows <= 4) {
        launch_gemv4<FMT, GATED, kDense>(a, tiles, 1, 0, st);
        return;
      }
      auto by_rows = [&](auto R, auto S, auto W) {
        constexpr int RT = decltype(R)::value, KS = decltype(S)::value, WV = decltype(W)::value;
        const int64_t per = WV / KS * RT;
        const dim3 grid((unsigned)((tiles + per - 1) / per)), block(64 * WV);
        if (rows <= 16) hipLaunchKernelGGL((gemv_kernel<FMT, GATED, 1, RT, KS, WV, false>), grid, block, 0, st, a);
        else if (rows <= 32) hipLaunchKernelGGL((gemv_kernel<FMT, GATED, 2, RT, KS, WV, false>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((gemv_kernel<FMT, GATED, 4, RT, KS, WV, false>), grid, block, 0, st, a);
      };
      // Many tiles fill the CUs by themselves: a wave takes two over all of K and reads x once for both. Fewer share K
      // until some 4096 to 8192 waves read at once. 7168 columns, 16 / 64 rows, us: 129280 rows of w two tiles a wave
      // 205 / 527, one 307 / 916; 32768 x 4096 16 rows K in two 49, in four 52. 16384 x 4096 in two 25, whole 45;
      // 8192 x 4096 in eight 15, in two 24, in sixteen 18. 2048 x 7168 gated in sixteen 12.8, in eight 13.6; short K
      // is not cut further (7168 x 2048 in eight 7.9, in sixteen 12.9).
      if (tiles >= 16 * 256) by_rows(ic<2>{}, ic<1>{}, ic<8>{});
      else if (tiles >= 4 * 256) by_rows(ic<1>{}, ic<2>{}, ic<8>{});
      else if (K <= 16 * gv::kChunk || tiles > 256) by_rows(ic<1>{}, ic<8>{}, ic<8>{});
      else by_rows(ic<1>{}, ic<16>{}, ic<16>{});
    };
    if (gated) go(ic<1>{});
    else go(ic<0>{});
  });
  return hipGetLastError();
}

// Over the experts that a.rows choices name. Up to six choices an expert, four by four: a row of workgroups per
// expert that can be named: the choices, or the experts where those are fewer. More: 32 by 32, two tiles a wave,
// the other way 64 tokens, 2 of 8 experts, 2048 x 4096 take 90 / 49 us (gate_up / down) against 50 / 34, 8 of 64,
// 768 x 2048 71 / 51 against 59 / 37, but with four an expert (8 of 128) 83 / 54 against 93 / 54. K in four
// where there are few tiles: 64 tokens, 2 of 8, in two 62 / 40; 4 of 32, 1024 x 4096, down in four 50, in two 45.
// Gated experts of 2^31 bytes and more go four by four whatever their choices: an up row lies too far behind its gate.
template <bool GATED>
static void launch_choices(int fmt, const GemvArgs& a, hipStream_t st) {
  const int64_t S = a.rows, by_choice = S < a.experts, each = by_choice ? S : a.experts;
  const int64_t tiles = (a.n + kTileOut<GATED> - 1) / kTileOut<GATED>;
  // gates and ups behind one descriptor (gemv_kernel) or one of eight rows each
  const bool one_descriptor = !GATED || a.n <= 0x7FFFFFFF / a.K;
  by_format(fmt, [&](auto F) {
    constexpr int FMT = decltype(F)::value;
    if (S >= 6 * a.experts && one_descriptor) {
      auto many = [&](auto KSC) {
        constexpr int KS = decltype(KSC)::value, PER = 8 / KS * 2;
        hipLaunchKernelGGL((gemv_kernel<FMT, GATED, 2, 2, KS, 8, true>),
                           dim3((unsigned)((tiles + PER - 1) / PER), (unsigned)a.experts), dim3(512), 0, st, a);
      };
      if (tiles * a.experts <= 4096) many(ic<4>{});
      else many(ic<2>{});
      return;
    }
    if (S <= 64) launch_gemv4<FMT, GATED, 1>(a, tiles, each, by_choice, st);
    else if (S <= 256) launch_gemv4<FMT, GATED, 4>(a, tiles, each, by_choice, st);
    else if (S <= 512) launch_gemv4<FMT, GATED, 8>(a, tiles, each, by_choice, st);
    else launch_gemv4<FMT, GATED, 0>(a, tiles, each, by_choice, st);
  });
}

hipError_t launch_decode_gate_up(int fmt, int64_t tokens, int64_t topk, int64_t experts, int64_t inter, int64_t K,
                                 const void* x, int64_t ld_x, const int32_t* idx, const void* w, const void* s,
                                 const float* t, int t_mode, void* h, hipStream_t st) {
  launch_choices<true>(fmt, GemvArgs{(const uint16_t*)x, ld_x, (int)(tokens * topk), (int)topk, idx, (int)experts,
                                     (const uint8_t*)w, (const uint8_t*)s, t, t_mode, inter, (int)K, h, inter, 0}, st);
  return hipGetLastError();
}

size_t decode_down_ws_bytes(int64_t choices, int64_t n) { return (size_t)((choices * n * 4 + 255) / 256 * 256); }

hipError_t launch_decode_down(int fmt, int64_t tokens, int64_t topk, int64_t experts, int64_t n, int64_t K, const void* h,
                              const int32_t* idx, const float* weights, const void* w, const void* s, const float* t,
                              int t_mode, void* y, int out32, void* ws, hipStream_t st) {
  launch_choices<false>(fmt, GemvArgs{(const uint16_t*)h, K, (int)(tokens * topk), 1, idx, (int)experts, (const uint8_t*)w,
                                      (const uint8_t*)s, t, t_mode, n, (int)K, ws, n, 1}, st);
  hipLaunchKernelGGL(decode_join_kernel, dim3((unsigned)((n + 255) / 256), (unsigned)tokens), dim3(256), 0, st,
                     (const float*)ws, idx, weights, (int)topk, (int)experts, n, y, out32);
  return hipGetLastError();
}

}  // namespace mxq
