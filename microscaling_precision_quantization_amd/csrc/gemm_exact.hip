// Block-scaled GEMMs with FP32-grade accumulation:
//   C[m, n] = tA tB * sum_k A_hat[m, k] B_hat[n, k]   ("TN", FP32 output)
//
// MXFP8, NVFP4 and BF16 run on the gfx950 16-bit MFMAs (v_mfma_f32_32x32x16_bf16/f16):
// every operand value is formed EXACTLY in a 16-bit format right before the matrix
// core consumes it, and the matrix core accumulates at FP32 precision (measured on
// MI355X: 2^20 + 2^-3 sums exactly at every operand position):
//   * MXFP8 (E4M3, E8M0 per 32 along K): q * 2^(s-127) has 4 significant bits and
//     stays in BF16 range, so the gfx950 scaled convert (which applies the
//     power-of-two scale exactly) yields it in BF16 -> BF16 MFMA.
//   * NVFP4 (E2M1, E4M3 per 16 along K, FP32 per row/tensor/expert): q * S has
//     at most 6 significant bits and lies in [2^-10, 2688], inside FP16's normal
//     range. S = 2^e * m (m = 1..1.875): the scaled convert applies 2^e, a packed
//     FP16 multiply applies m (exact) -> FP16 MFMA; tA tB in the epilogue.
//   * MXFP4 (E2M1, E8M0 per 32 along K) runs on the native FP4 form of the scaled
//     MFMA (v_mfma_scale_f32_32x32x64_f8f6f4), which applies the E8M0 scales itself.
//     Measured on MI355X: lane l supplies row l % 32 and the whole 32-K block h = l / 32
//     of the instruction's 64 K (16 bytes, low nibble first), with that block's scale;
//     products of one block sum exactly, and a result differs from the exact value by
//     at most 2^-23.6 of the sum of the magnitudes of its terms (FP32-grade, unlike the
//     FP8 form's ~2^-13 window), so this path meets the same accuracy bound.
//   * Blockwise FP8 (E4M3, FP32 scale per row and 128-K block of A, per row or per
//     128 x 128 block of B): the E4M3 values are exact in BF16 -> BF16 MFMA into a
//     per-block partial sum; at the end of each 128-K stage the FP32 scales are applied
//     in software (acc += partial * sA sB, one FMA per accumulator).
//   * BF16 operands as they are -> BF16 MFMA.
// Definitions: microscaling blocks along the reduction dimension ("Miles
// Blackwell RL", remio.ai, section "Un Cuantizador Compartido Es el Mecanismo
// Real"); two-level NVFP4 (7minutos.es NVFP4 page, section "Que es realmente
// NVFP4"); dequantized-backward BF16 GEMMs and the BF16 shared expert (remio.ai,
// sections "La Compatibilidad ..." and "NVFP4 por token ...").
// The native scaled-FP8 MFMA (format 0) is not used for gemm_block_scaled: it sums each
// group of 8 consecutive K products of a lane in a fixed-point window about 13 bits
// below the group's largest product, dropping lower bits, and accumulates the group
// sums at FP32 precision (measured on MI355X), which breaks the 2e-5 bound on
// outlier-heavy data. It runs gemm_mxfp8_matrix_core (LD 5 below): the same pipeline
// with 128-K stages, one instruction per 64 K taking both operands' E8M0 bytes.
// Its operand layout (measured): lane l supplies row l % 32; with h = l / 32, bytes
// 0..15 are elements [16h, 16h+16) of the first 32-K block and bytes 16..31 the same
// elements of the second block; the scale of block b comes from lane (l % 32) + 32 b.
//
// Data movement: raw operand tiles go global -> LDS with gfx950's direct loads
// (buffer_load_dwordx4 ... lds: lane l of a wave instruction lands at LDS base +
// 16 l), through a 16-byte XOR swizzle chosen so that each 16-lane fragment read
// (ds_read_b128) covers all 64 banks (measured conflict-free). A stage holds 64 K
// (128 B/row BF16, 64 B/row MXFP8, 32 B/row NVFP4 / MXFP4), or 128 B/row for every
// format in the dense kernels when K allows chunked scales (128 K MXFP8, 256 K NVFP4
// and MXFP4: fewer barriers, larger loads). NS stages keep NS - 1 tiles in flight; explicit
// vmcnt waits + one barrier per stage. Scales travel either per stage into
// 4-byte LDS slots, or as 16-byte chunks per row (16 blocks) double-buffered in
// LDS and read into registers once per chunk. Out-of-range rows and K chunks
// read zeros (buffer range checks).
//
// Operand layouts of the 32x32x16 16-bit MFMAs (measured): lane l supplies row
// l % 32 and 8 consecutive K; accumulator r of lane l is
// C[(r / 4) * 8 + (l / 32) * 4 + r % 4][l % 32].
#include "gemm_tile.h"

namespace mxq {

template <int LD, int BM, int BN, int SM, bool WIDE>
__global__ void __launch_bounds__(256, 1) __attribute__((amdgpu_waves_per_eu(1, 1))) exact_dense_kernel(ExactProblem p, int64_t tiles_m, int64_t tiles_n) {
  using C = gx::Cfg<LD, BM, BN, SM, 1, WIDE>;
  MXQ_EXACT_LDS(C)
  int64_t tm, tn;
  if (!exact_map_tile(blockIdx.x, tiles_m, tiles_n, tm, tn)) return;
  exact_gemm_tile<LD, BM, BN, SM, 1, WIDE>(p, tm * BM, tn * BN, lds0, lds1, lds2, lds3, ldsc);
}

// Two workgroups per CU (each half the LDS, two stages): for the blockwise FP8 tiles, whose
// second accumulator set rules out larger tiles, one workgroup's scale FMAs, prologue and
// epilogue overlap the other's main loop (20-30% faster than one workgroup per CU).
template <int LD, int BM, int BN, int SM>
__global__ void __launch_bounds__(256, 2) __attribute__((amdgpu_waves_per_eu(2, 2))) exact_dense_occ2_kernel(ExactProblem p, int64_t tiles_m, int64_t tiles_n) {
  using C = gx::Cfg<LD, BM, BN, SM, 2, false>;
  MXQ_EXACT_LDS(C)
  int64_t tm, tn;
  if (!exact_map_tile(blockIdx.x, tiles_m, tiles_n, tm, tn)) return;
  exact_gemm_tile<LD, BM, BN, SM, 2, false>(p, tm * BM, tn * BN, lds0, lds1, lds2, lds3, ldsc);
}

// Several independent dense problems in one launch (e.g. the fprop, dgrad and wgrad GEMMs
// of a layer): workgroups [block0, block0 + 8 ceil(tiles / 8)) belong to job j. The host
// orders jobs by K, longest first, so the long tiles start first and the epilogue stores of
// finished tiles overlap the main loops of others.
constexpr int kMaxBatch = 8;
struct BatchJob {
  ExactProblem p;
  int64_t tiles_m, tiles_n, block0;
};
struct BatchJobs {
  BatchJob j[kMaxBatch];
  int n;
};

template <int LD, int BM, int BN, int SM, bool WIDE>
__global__ void __launch_bounds__(256, 1) __attribute__((amdgpu_waves_per_eu(1, 1))) exact_batch_kernel(const BatchJobs jobs) {
  using C = gx::Cfg<LD, BM, BN, SM, 1, WIDE>;
  MXQ_EXACT_LDS(C)
  int jsel = 0;
#pragma unroll
  for (int i = 1; i < kMaxBatch; ++i)
    if (i < jobs.n && (int64_t)blockIdx.x >= jobs.j[i].block0) jsel = i;
  int64_t tm = 0, tn = 0;
  ExactProblem p;
  bool ok = false;
  // static indices only: the table stays in kernel arguments
#pragma unroll
  for (int i = 0; i < kMaxBatch; ++i)
    if (i == jsel) {
      p = jobs.j[i].p;
      ok = exact_map_tile((int64_t)blockIdx.x - jobs.j[i].block0, jobs.j[i].tiles_m, jobs.j[i].tiles_n, tm, tn);
    }
  if (!ok) return;
  exact_gemm_tile<LD, BM, BN, SM, 1, WIDE>(p, tm * BM, tn * BN, lds0, lds1, lds2, lds3, ldsc);
}

// The same over 128 x 256 tiles with two workgroups per CU (each workgroup half the LDS):
// one's prologue and FP32 epilogue overlap the other's main loop.
template <int LD, int SM>
__global__ void __launch_bounds__(256, 2) __attribute__((amdgpu_waves_per_eu(2, 2))) exact_batch_rect_kernel(const BatchJobs jobs) {
  using C = gx::Cfg<LD, 128, 256, SM, 2, false>;
  MXQ_EXACT_LDS(C)
  int jsel = 0;
#pragma unroll
  for (int i = 1; i < kMaxBatch; ++i)
    if (i < jobs.n && (int64_t)blockIdx.x >= jobs.j[i].block0) jsel = i;
  int64_t tm = 0, tn = 0;
  ExactProblem p;
  bool ok = false;
#pragma unroll
  for (int i = 0; i < kMaxBatch; ++i)
    if (i == jsel) {
      p = jobs.j[i].p;
      ok = exact_map_tile((int64_t)blockIdx.x - jobs.j[i].block0, jobs.j[i].tiles_m, jobs.j[i].tiles_n, tm, tn);
    }
  if (!ok) return;
  exact_gemm_tile<LD, 128, 256, SM, 2, false>(p, tm * 128, tn * 256, lds0, lds1, lds2, lds3, ldsc);
}

// The same for blockwise FP8 (two accumulator sets): 128 x 128 tiles, two workgroups per CU.
template <int LD, int SM>
__global__ void __launch_bounds__(256, 2) __attribute__((amdgpu_waves_per_eu(2, 2))) exact_batch_occ2_kernel(const BatchJobs jobs) {
  using C = gx::Cfg<LD, 128, 128, SM, 2, false>;
  MXQ_EXACT_LDS(C)
  int jsel = 0;
#pragma unroll
  for (int i = 1; i < kMaxBatch; ++i)
    if (i < jobs.n && (int64_t)blockIdx.x >= jobs.j[i].block0) jsel = i;
  int64_t tm = 0, tn = 0;
  ExactProblem p;
  bool ok = false;
#pragma unroll
  for (int i = 0; i < kMaxBatch; ++i)
    if (i == jsel) {
      p = jobs.j[i].p;
      ok = exact_map_tile((int64_t)blockIdx.x - jobs.j[i].block0, jobs.j[i].tiles_m, jobs.j[i].tiles_n, tm, tn);
    }
  if (!ok) return;
  exact_gemm_tile<LD, 128, 128, SM, 2, false>(p, tm * 128, tn * 128, lds0, lds1, lds2, lds3, ldsc);
}

// Grouped: tile_prefix[g] = first tile of group g.
//   vary_k = 0: group g covers slots [off[g], off[g+1]), B_g = expert g of a stacked B;
//   vary_k = 1: group g reduces over k in [off[g], off[g+1]) into C_g = C + g*M*N.
// OCC = 2 gives each workgroup half the LDS, so two share a CU and one's prologue and
// epilogue overlap the other's main loop (expert tiles are short in K or in rows).
//
// Row groups (vary_k = 0) are walked XCD by XCD: dispatch order b goes to XCD b % 8, and
// each XCD takes a contiguous run of the logical tile list, so an expert's tiles share
// one L2. Inside a group the tiles go in column bands of kRowGroupBand row tiles: the row
// tiles that read one weight column slab run side by side (Qwen3-shaped gate_up: L2
// misses 1110 -> 275 MB per launch and 9% faster; DeepSeek-shaped fused dgrads 3-4%
// faster). Weight gradients (vary_k = 1) keep the plain order: there the XCD runs made
// the kernels 2-14% slower (their time goes to the FP32 output stores, not to reads).
constexpr int kRowGroupBand = 4;
template <int LD, int BM, int BN, int SM, int OCC, bool WIDE, bool AKM = false>
__global__ void __launch_bounds__(256, OCC) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
exact_grouped_kernel(ExactProblem base, const int64_t* __restrict__ offsets, const int64_t* __restrict__ tile_prefix,
                     int64_t groups, int vary_k, int64_t M, int64_t N, int64_t tiles_n) {
  using C = gx::Cfg<LD, BM, BN, SM, OCC, WIDE>;
  MXQ_EXACT_LDS(C)
  const int64_t total = tile_prefix[groups];
  int64_t tile = blockIdx.x;
  if (!vary_k) {
    const int64_t T8 = (total + 7) / 8;
    if (tile >= 8 * T8) return;                     // the grid may exceed the tile count
    tile = (tile % 8) * T8 + tile / 8;
  }
  if (tile >= total) return;
  // weight gradients: every group has the same tiles_m x tiles_n tiles (the prefix is g times
  // that, or all zero when the offsets were rejected), so the group needs no search
  const int64_t per_group = (M + BM - 1) / BM * tiles_n;
  const int64_t g = vary_k ? tile / per_group : find_group(tile_prefix, groups, tile);
  const int64_t local = vary_k ? tile - g * per_group : tile - tile_prefix[g];
  int64_t tm = local / tiles_n, tn = local % tiles_n;
  if (!vary_k) {
    const int64_t tiles_m = (tile_prefix[g + 1] - tile_prefix[g]) / tiles_n;
    const int64_t band = local / (kRowGroupBand * tiles_n);
    const int64_t rows_in_band = min((int64_t)kRowGroupBand, tiles_m - band * kRowGroupBand);
    const int64_t idx = local - band * kRowGroupBand * tiles_n;
    tm = band * kRowGroupBand + idx % rows_in_band;
    tn = idx / rows_in_band;
  }
  ExactProblem p = base;
  if (!vary_k) {
    p.a_base = offsets[g];
    p.m_valid = offsets[g + 1] - offsets[g];
    const int64_t b_elems = g * N * base.ldb;
    p.B = base.B + k_bytes<LD>(b_elems);
    if constexpr (LD == 6) {                      // group g's weight: K rows of N (= ldb) NVFP4 elements
      const int64_t w_elems = g * base.k_end * base.ldb;
      p.B = base.B + w_elems / 2;
      p.sB = base.sB + w_elems / 16;
      p.tB = base.tB + g;
    }
    if (LD == 1 || LD == 3) p.sB = base.sB + b_elems / 32;
    if (LD == 2) {
      p.sB = base.sB + b_elems / 16;
      if (base.tB_mode == 2) { p.tB = base.tB + g; p.tB_mode = 1; }
      else p.tB = base.tB + g * N;
    }
    p.C = base.C + offsets[g] * base.ldc;
  } else {
    p.k_begin = offsets[g];
    p.k_end = offsets[g + 1];
    p.C = base.C + g * M * N;
  }
  // the expert-tail specialization pays on the converting forward formats (NVFP4 gate_up /
  // down 3-6% faster); the BF16 kernels at one workgroup per CU measured no gain from it
  constexpr bool PART = LD != 0 && LD != 6;
  exact_gemm_tile<LD, BM, BN, SM, OCC, WIDE, AKM, PART>(p, tm * BM, tn * BN, lds0, lds1, lds2, lds3, ldsc);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

static int pick_tile(int64_t M, int64_t N) {
  // 256 x 256 unless that leaves most of the 256 CUs idle; then 128 x 128.
  const int64_t t256 = ((M + 255) / 256) * ((N + 255) / 256);
  return t256 >= 192 ? 256 : 128;
}

template <int LD, int BT, int SM>
static void launch_dense_t(const ExactProblem& p, int64_t M, int64_t N, hipStream_t st) {
  const int64_t tm = (M + BT - 1) / BT, tn = (N + BT - 1) / BT;
  const int64_t blocks = (tm * tn + 7) / 8 * 8;
  constexpr bool WIDE = SM == 2 && LD != 0;       // measured: 3-6% faster dense tiles
  hipLaunchKernelGGL((exact_dense_kernel<LD, BT, BT, SM, WIDE>), dim3((unsigned)blocks), dim3(256), 0, st, p, tm, tn);
}

// Scale mode: 2 when K % 64 == 0 and every scale row starts 16-byte aligned
// (K % 512 == 0 for MXFP8 / MXFP4, K % 256 == 0 for NVFP4), 1 when K % 64 == 0, else 0.
static int scale_mode(int ld, int64_t K, bool vary_k) {
  if (ld == 5) return K % 512 == 0 ? 2 : K % 128 == 0 ? 1 : 0;   // 128-K stages
  if (vary_k || K % 64) return 0;
  if ((ld == 1 || ld == 3) && K % 512 == 0) return 2;
  if (ld == 2 && K % 256 == 0) return 2;
  return 1;
}

template <int LD, int BT>
static void launch_dense_bt(const ExactProblem& p, int64_t M, int64_t N, int sm, hipStream_t st) {
  if constexpr (LD != 0) {
    if (sm == 2) { launch_dense_t<LD, BT, 2>(p, M, N, st); return; }
  }
  if (sm == 2) launch_dense_t<LD, BT, 1>(p, M, N, st);
  else if (sm == 1) launch_dense_t<LD, BT, 1>(p, M, N, st);
  else launch_dense_t<LD, BT, 0>(p, M, N, st);
}

template <int LD>
static void launch_dense_ld(const ExactProblem& p, int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const int sm = scale_mode(LD, K, false);
  if (pick_tile(M, N) == 256) launch_dense_bt<LD, 256>(p, M, N, sm, st);
  else launch_dense_bt<LD, 128>(p, M, N, sm, st);
}

hipError_t launch_gemm(int fmt, int64_t M, int64_t N, int64_t K, const void* A, const void* sA, const float* tA,
                       int tA_mode, const void* B, const void* sB, const float* tB, int tB_mode, float* C,
                       int64_t ldc, hipStream_t st) {
  ExactProblem p;
  p.A = (const uint8_t*)A; p.sA = (const uint8_t*)sA; p.tA = tA; p.tA_mode = tA_mode;
  p.a_idx = nullptr; p.a_rows = M; p.a_base = 0; p.m_valid = M; p.lda = K;
  p.B = (const uint8_t*)B; p.sB = (const uint8_t*)sB; p.tB = tB; p.tB_mode = tB_mode; p.n_valid = N; p.ldb = K;
  p.k_begin = 0; p.k_end = K; p.C = C; p.ldc = ldc;
  // fmt: 1 MXFP8, 2 NVFP4, 3 BF16, 4 MXFP4, 5 blockwise FP8 (tB_mode: 0 per B row, 1 per
  // 128 x 128 block; 128 x 128 tiles, K % 128 == 0), 6 MXFP8 on the scaled FP8 MFMA
  if (fmt == 5) {
    const int64_t tm = (M + 127) / 128, tn = (N + 127) / 128;
    hipLaunchKernelGGL((exact_dense_occ2_kernel<4, 128, 128, 1>), dim3((unsigned)((tm * tn + 7) / 8 * 8)), dim3(256), 0,
                       st, p, tm, tn);
  }
  else if (fmt == 6) launch_dense_ld<5>(p, M, N, K, st);      // MXFP8 on the scaled FP8 MFMA
  else if (fmt == 1) launch_dense_ld<1>(p, M, N, K, st);
  else if (fmt == 2) launch_dense_ld<2>(p, M, N, K, st);
  else if (fmt == 4) launch_dense_ld<3>(p, M, N, K, st);
  else launch_dense_ld<0>(p, M, N, K, st);
  return hipGetLastError();
}

hipError_t launch_gemm(int fmt, int64_t M, int64_t N, int64_t K, const void* A, const void* sA, const float* tA,
                       int tA_mode, const void* B, const void* sB, const float* tB, int tB_mode, float* C,
                       int64_t ldc, hipStream_t st);

// Batched dense GEMMs of one format: one launch, jobs ordered by K (longest first), one
// tile size and scale mode for all (the largest the batch allows). With 256 x 256 tiles, a
// job that would cover fewer than 128 of them (too few to share the CUs with the others
// for long) runs as its own launch with the single-problem tile rule instead.
hipError_t launch_gemm_batch(int fmt, int n, const int64_t* M, const int64_t* N, const int64_t* K,
                             const void* const* A, const void* const* sA, const float* const* tA, const int* tA_mode,
                             const void* const* B, const void* const* sB, const float* const* tB, const int* tB_mode,
                             float* const* C, const int64_t* ldc, hipStream_t st) {
  const int ld = fmt == 1 ? 1 : fmt == 2 ? 2 : fmt == 4 ? 3 : fmt == 5 ? 4 : 0;
  int order[kMaxBatch];
  for (int i = 0; i < n; ++i) order[i] = i;
  for (int i = 1; i < n; ++i)                          // insertion sort, K descending (stable)
    for (int k = i; k > 0 && K[order[k]] > K[order[k - 1]]; --k) std::swap(order[k], order[k - 1]);
  if (ld == 4) {
    // blockwise FP8 (fmt 5, tB_mode = b_blocks): every problem on the single call's 128 x 128
    // tiles at two workgroups per CU, so a long-K problem (a layer's dgrad) shares the CUs
    // with the others instead of leaving half the slots idle
    BatchJobs jobs;
    jobs.n = 0;
    int64_t blocks = 0;
    for (int q = 0; q < n; ++q) {
      const int i = order[q];
      ExactProblem& p = jobs.j[jobs.n].p;
      p.A = (const uint8_t*)A[i]; p.sA = (const uint8_t*)sA[i]; p.tA = nullptr; p.tA_mode = 0;
      p.a_idx = nullptr; p.a_rows = M[i]; p.a_base = 0; p.m_valid = M[i]; p.lda = K[i];
      p.B = (const uint8_t*)B[i]; p.sB = (const uint8_t*)sB[i]; p.tB = nullptr; p.tB_mode = tB_mode[i];
      p.n_valid = N[i]; p.ldb = K[i];
      p.k_begin = 0; p.k_end = K[i]; p.C = C[i]; p.ldc = ldc[i];
      jobs.j[jobs.n].tiles_m = (M[i] + 127) / 128;
      jobs.j[jobs.n].tiles_n = (N[i] + 127) / 128;
      jobs.j[jobs.n].block0 = blocks;
      blocks += (jobs.j[jobs.n].tiles_m * jobs.j[jobs.n].tiles_n + 7) / 8 * 8;
      ++jobs.n;
    }
    if (blocks > 0) hipLaunchKernelGGL((exact_batch_occ2_kernel<4, 1>), dim3((unsigned)blocks), dim3(256), 0, st, jobs);
    return hipGetLastError();
  }
  int64_t t256 = 0;
  for (int i = 0; i < n; ++i) t256 += ((M[i] + 255) / 256) * ((N[i] + 255) / 256);
  const int bt = t256 >= 192 ? 256 : 128;
  // MXFP8 with 16-byte scale chunks (every K % 512 == 0) and a few 256-tiles per CU: every
  // problem on 128 x 256 tiles at two workgroups per CU, none alone (the linear layer's
  // three GEMMs: 6% faster than 256 x 256 tiles plus a separate 128 x 128 dgrad). Batches of
  // four or more 256-tiles per CU (three 8192^3 GEMMs) keep the 256 x 256 tiles.
  int sm_all = 2;
  for (int i = 0; i < n; ++i) sm_all = std::min(sm_all, scale_mode(ld, K[i], false));
  const bool rect = ld == 1 && sm_all == 2 && t256 >= 192 && t256 < 1024;
  bool alone[kMaxBatch];
  int sm = 2, nb = 0;
  for (int i = 0; i < n; ++i) {
    alone[i] = !rect && bt == 256 && ((M[i] + 255) / 256) * ((N[i] + 255) / 256) < 128;
    if (!alone[i]) { sm = std::min(sm, scale_mode(ld, K[i], false)); ++nb; }
  }
  BatchJobs jobs;
  jobs.n = 0;
  int64_t blocks = 0;
  for (int q = 0; q < n; ++q) {
    const int i = order[q];
    if (alone[i]) continue;
    const int qq = jobs.n++;
    ExactProblem& p = jobs.j[qq].p;
    p.A = (const uint8_t*)A[i]; p.sA = (const uint8_t*)sA[i]; p.tA = tA[i]; p.tA_mode = tA_mode[i];
    p.a_idx = nullptr; p.a_rows = M[i]; p.a_base = 0; p.m_valid = M[i]; p.lda = K[i];
    p.B = (const uint8_t*)B[i]; p.sB = (const uint8_t*)sB[i]; p.tB = tB[i]; p.tB_mode = tB_mode[i];
    p.n_valid = N[i]; p.ldb = K[i];
    p.k_begin = 0; p.k_end = K[i]; p.C = C[i]; p.ldc = ldc[i];
    jobs.j[qq].tiles_m = (M[i] + (rect ? 128 : bt) - 1) / (rect ? 128 : bt);
    jobs.j[qq].tiles_n = (N[i] + (rect ? 256 : bt) - 1) / (rect ? 256 : bt);
    jobs.j[qq].block0 = blocks;
    blocks += (jobs.j[qq].tiles_m * jobs.j[qq].tiles_n + 7) / 8 * 8;    // XCD-aware raster per job
  }
  for (int q = 0; q < n; ++q) {                       // the jobs that run alone, longest K first
    const int i = order[q];
    if (!alone[i]) continue;
    const hipError_t e = launch_gemm(fmt, M[i], N[i], K[i], A[i], sA[i], tA[i], tA_mode[i], B[i], sB[i], tB[i],
                                     tB_mode[i], C[i], ldc[i], st);
    if (e != hipSuccess) return e;
  }
  if (nb == 0 || blocks == 0) return hipGetLastError();
  if (rect) {
    hipLaunchKernelGGL((exact_batch_rect_kernel<1, 2>), dim3((unsigned)blocks), dim3(256), 0, st, jobs);
    return hipGetLastError();
  }
  auto go = [&](auto LDC, auto BTC, auto SMC) {
    constexpr int L = decltype(LDC)::value, T = decltype(BTC)::value, S = decltype(SMC)::value;
    constexpr bool WIDE = S == 2 && L != 0;
    hipLaunchKernelGGL((exact_batch_kernel<L, T, T, S, WIDE>), dim3((unsigned)blocks), dim3(256), 0, st, jobs);
  };
  auto by_sm = [&](auto LDC, auto BTC) {
    if constexpr (decltype(LDC)::value != 0) {
      if (sm == 2) { go(LDC, BTC, ic<2>{}); return; }
    }
    if (sm >= 1) go(LDC, BTC, ic<1>{});
    else go(LDC, BTC, ic<0>{});
  };
  auto by_bt = [&](auto LDC) {
    if (bt == 256) by_sm(LDC, ic<256>{});
    else by_sm(LDC, ic<128>{});
  };
  if (ld == 1) by_bt(ic<1>{});
  else if (ld == 2) by_bt(ic<2>{});
  else if (ld == 3) by_bt(ic<3>{});
  else by_bt(ic<0>{});
  return hipGetLastError();
}

// One wave: checks that the offsets partition [0, total) (aligned to `align` when they
// split the reduction axis) and writes the exclusive prefix of the per-group tile counts,
// 64 groups per round (lane scan with shuffles). Invalid offsets give an all-zero prefix,
// so no tile runs.
__global__ void __launch_bounds__(64) tile_prefix_kernel(const int64_t* __restrict__ offsets, int64_t groups,
                                                         int64_t total, int vary_k, int64_t align, int64_t bm,
                                                         int64_t tiles_m_fixed, int64_t tiles_n,
                                                         int64_t* __restrict__ prefix) {
  const int lane = threadIdx.x;
  bool bad = false;
  for (int64_t g0 = 0; g0 < groups; g0 += 64) {
    const int64_t g = g0 + lane;
    if (g < groups) {
      const int64_t a = offsets[g], b = offsets[g + 1];
      bad = bad || b < a || (vary_k && (a % align != 0));
    }
  }
  bad = bad || offsets[0] != 0 || offsets[groups] != total;
  const bool ok = __ballot(bad) == 0;
  int64_t carry = 0;
  for (int64_t g0 = 0; g0 < groups; g0 += 64) {
    const int64_t g = g0 + lane;
    int64_t cnt = 0;
    if (g < groups) cnt = vary_k ? tiles_m_fixed : (offsets[g + 1] - offsets[g] + bm - 1) / bm;
    cnt *= tiles_n;
    int64_t incl = cnt;                                   // inclusive scan over the 64 lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    if (g < groups) prefix[g] = ok ? carry + incl - cnt : 0;
    carry += __shfl(incl, 63, 64);
  }
  if (lane == 0) prefix[groups] = ok ? carry : 0;
}

void launch_tile_prefix(const int64_t* offsets, int64_t groups, int64_t total, int64_t bm, int64_t tiles_n, int64_t* prefix,
                        hipStream_t st) {
  hipLaunchKernelGGL(tile_prefix_kernel, dim3(1), dim3(64), 0, st, offsets, groups, total, 0, (int64_t)1, bm, (int64_t)0,
                     tiles_n, prefix);
}

size_t grouped_gemm_ws_bytes(int64_t groups) { return (size_t)(((groups + 1) * 8 + 255) / 256 * 256); }

template <int LD, int BT, int SM, bool AKM = false>
static void launch_grouped_t(const ExactProblem& p, const int64_t* offsets, const int64_t* prefix, int64_t max_tiles,
                             int64_t groups, int vary_k, int64_t M, int64_t N, hipStream_t st) {
  const int64_t tn = (N + BT - 1) / BT;
  // expert tiles keep the narrow stages: wide NVFP4 stages leave two LDS stages at half LDS.
  // 128 x 128 tiles run two workgroups per CU, 256 x 256 tiles one.
  constexpr int OCC = BT == 256 ? 1 : 2;
  hipLaunchKernelGGL((exact_grouped_kernel<LD, BT, BT, SM, OCC, false, AKM>), dim3((unsigned)max_tiles), dim3(256), 0, st,
                     p, offsets, prefix, groups, vary_k, M, N, tn);
}

// Row-grouped NVFP4 with chunked scales: 128-row tiles keep the expert padding small,
// 256 columns halve the A re-reads, two workgroups per CU.
template <int SM>
static void launch_grouped_nv_rect(const ExactProblem& p, const int64_t* offsets, const int64_t* prefix,
                                   int64_t max_tiles, int64_t groups, int64_t M, int64_t N, hipStream_t st) {
  const int64_t tn = (N + 255) / 256;
  hipLaunchKernelGGL((exact_grouped_kernel<2, 128, 256, SM, 2, false>), dim3((unsigned)max_tiles), dim3(256), 0, st, p,
                     offsets, prefix, groups, 0, M, N, tn);
}

hipError_t launch_grouped_gemm(int fmt, int64_t groups, const int64_t* offsets, int vary_k, int64_t total, int64_t M,
                               int64_t N, int64_t K, const int32_t* a_row_index, int64_t a_rows, const void* A,
                               const void* sA, const float* tA, int tA_mode, const void* B, const void* sB,
                               const float* tB, int tB_mode, float* C, void* ws, hipStream_t st) {
  int64_t* prefix = (int64_t*)ws;
  // Expert groups are small (hundreds of rows): 128 x 128 tiles. A weight gradient
  // (vary_k) has the full (M, N) output per group: 256 x 256 tiles once that gives each
  // group at least 64 of them. BF16 row groups averaging 384 rows or more also take
  // 256 x 256 tiles: their per-flop speed outweighs the extra row padding there (DeepSeek
  // expert dgrads, ~527 rows per expert: 7% faster). NVFP4 showed no gain.
  const bool big_rows = (fmt == 3 || fmt == 7) && !vary_k && groups > 0 && total / groups >= 384;
  // Row-grouped NVFP4 with chunked scales: 128 x 256 tiles (DeepSeek expert gate_up 12%
  // faster than 128 x 128, Qwen3 8%).
  const bool nv_rect = fmt == 2 && !vary_k && scale_mode(2, K, false) == 2;
  // Weight gradients (vary_k) with large outputs: 256 x 256 tiles. (With the unguarded
  // interior-tile epilogue the DeepSeek expert wgrads run 5% faster on them than on 128 x 256
  // tiles at two workgroups per CU; with per-element guarded stores it was the reverse.)
  const bool wide_out = vary_k && ((M + 255) / 256) * ((N + 255) / 256) >= 64;
  const int BT = fmt == 7 ? 256 : (wide_out || big_rows) ? 256 : 128;
  const int BTN = nv_rect ? 256 : BT;
  const int64_t tiles_n = (N + BTN - 1) / BTN;
  const int64_t tiles_m_fixed = vary_k ? (M + BT - 1) / BT : 0;
  const int64_t align = (fmt == 1 || fmt == 4) ? 32 : fmt == 2 ? 16 : 8;
  hipLaunchKernelGGL(tile_prefix_kernel, dim3(1), dim3(64), 0, st, offsets, groups, total, vary_k, align, (int64_t)BT,
                     tiles_m_fixed, tiles_n, prefix);
  // Row groups: an upper bound on the tiles (the device prefix holds the count), rounded
  // up to a multiple of 8 so that the XCD-contiguous order reaches every logical tile
  // below 8 ceil(tiles / 8) (the kernel maps dispatch index b to (b % 8) ceil(tiles / 8) + b / 8).
  const int64_t max_tiles = vary_k ? groups * tiles_m_fixed * tiles_n
                                   : ((((total + BT - 1) / BT + groups) * tiles_n + 7) / 8) * 8;
  if (max_tiles <= 0) return hipGetLastError();
  ExactProblem p;
  p.A = (const uint8_t*)A; p.sA = (const uint8_t*)sA; p.tA = tA; p.tA_mode = tA_mode;
  p.a_idx = a_row_index; p.a_rows = a_rows; p.a_base = 0;
  p.B = (const uint8_t*)B; p.sB = (const uint8_t*)sB; p.tB = tB; p.tB_mode = tB_mode; p.C = C; p.ldc = N;
  if (!vary_k) {
    p.m_valid = 0; p.lda = K; p.n_valid = N; p.ldb = K; p.k_begin = 0; p.k_end = K;
  } else {
    // vary_k 2: A is given K-major, (total, M) row-major (the slot-major gradient itself)
    p.m_valid = M; p.lda = vary_k == 2 ? M : total; p.n_valid = N; p.ldb = total; p.k_begin = 0; p.k_end = 0;
  }
  if (vary_k == 2) {
    if (BT == 256) launch_grouped_t<0, 256, 0, true>(p, offsets, prefix, max_tiles, groups, vary_k, M, N, st);
    else launch_grouped_t<0, 128, 0, true>(p, offsets, prefix, max_tiles, groups, vary_k, M, N, st);
    return hipGetLastError();
  }
  if (fmt == 7) {
    // BF16 A x the stacked NVFP4 weights (K, N) per group, read transposed: B_g[n][k] is the
    // BF16 dequantization of W_g[k][n], built in the loader (no BF16 weight copy in HBM)
    p.ldb = N;
    const int64_t tn = (N + 255) / 256;
    hipLaunchKernelGGL((exact_grouped_kernel<6, 256, 256, 0, 1, false>), dim3((unsigned)max_tiles), dim3(256), 0, st, p,
                       offsets, prefix, groups, 0, M, N, tn);
    return hipGetLastError();
  }
  const int ld = fmt == 1 ? 1 : fmt == 2 ? 2 : fmt == 4 ? 3 : 0;
  const int sm = scale_mode(ld, p.lda, vary_k != 0);
  auto go = [&](auto LDC, auto SMC) {
    constexpr int L = decltype(LDC)::value, S = decltype(SMC)::value;
    if constexpr (L == 0 || (S == 0 && L != 2)) {   // 256 tiles: BF16, or vary_k (SM 0, never NVFP4)
      if (BT == 256) {
        launch_grouped_t<L, 256, S>(p, offsets, prefix, max_tiles, groups, vary_k, M, N, st);
        return;
      }
    }
    launch_grouped_t<L, 128, S>(p, offsets, prefix, max_tiles, groups, vary_k, M, N, st);
  };
  auto by_sm = [&](auto LDC) {
    if constexpr (decltype(LDC)::value != 0) {
      if (sm == 2) { go(LDC, ic<2>{}); return; }
    }
    if (sm == 2) go(LDC, ic<1>{});
    else if (sm == 1) go(LDC, ic<1>{});
    else go(LDC, ic<0>{});
  };
  if (ld == 1) by_sm(ic<1>{});
  else if (ld == 2 && nv_rect) launch_grouped_nv_rect<2>(p, offsets, prefix, max_tiles, groups, M, N, st);
  else if (ld == 2) by_sm(ic<2>{});
  else if (ld == 3) by_sm(ic<3>{});
  else by_sm(ic<0>{});
  return hipGetLastError();
}

}  // namespace mxq
