// Gated feed-forward block: both projections, SwiGLU and the product in one kernel, and the
// gradient of that.
//   forward   (g | u) = A_hat W_gu_hat^T;  h = g sigma(g) u, and (g | u) kept for the backward
//   backward  dh = dO_hat W_d_hat;  d_gate = dh u sigma(g) (1 + g (1 - sigma(g)));  d_up = dh g sigma(g)
// Dense and per expert. The product is the tile loop of gemm_tile.h; what is new is how a tile's
// columns are chosen (a wave holds the gate and the up of the same h columns) and its epilogue:
// the FP32 product never reaches memory, each output is rounded to BF16 once, from the FP32 sums.
// Bound by the matrix core in the main loop; the epilogue (vector instructions and 16-byte stores, FP32 strips
// through LDS) runs beside another tile's main loop only where two workgroups share a CU, so large dense tiles pay
// for it in full. 16384 x 7168 -> 2 x 2048 BF16 with (g | u) kept 786-811 us (1.19-1.22 PFLOP/s; a library product
// alone 690), its backward 442-452 (floor 345); 2011 x 2048 -> 2 x 4096 MXFP8 56-59 (48), backward 44-47 (24: 512
// tiles of 128 x 128, two a CU, which start and end together, so that neither hides the other's start or
// epilogue); 4096 tokens, 8 of 128 experts, 2048 -> 2 x 768 NVFP4 244 (148: conversions, 263 rows an expert on
// 128-row tiles), backward against the NVFP4 W_d 245 (109 in bytes: FP32 (g | u) read and dGU written behind a
// main loop that converts the weights). Dense NVFP4, 16384 x 7168 -> 2 x 2048 760 (690).
// SwiGLU experts whose gate and up projections enter one fused GEMM: remio.ai ("Miles Blackwell RL"),
// section "Un Cuantizador Compartido Es el Mecanismo Real".
#include "gemm_tile.h"

namespace mxq {

void launch_tile_prefix(const int64_t* offsets, int64_t groups, int64_t total, int64_t bm, int64_t tiles_n, int64_t* prefix,
                        hipStream_t st);

size_t grouped_gemm_ws_bytes(int64_t groups);

template <int LD, int BN> constexpr bool kShort = LD == 0 && BN == 256;

// h columns of a tile
template <int BN, int EPI> constexpr int kTileCols = EPI == 1 ? BN / 2 : BN;

template <int LD, int BM, int BN, int SM, int OCC, bool WIDE, int EPI>
__global__ void __launch_bounds__(256, OCC) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
gated_dense_kernel(ExactProblem p, GatedArgs ga, int64_t tiles_m, int64_t tiles_n) {
  using C = gx::Cfg<LD, BM, BN, SM, OCC, WIDE, EPI, kShort<LD, BN>>;
  MXQ_EXACT_LDS(C)
  int64_t tm, tn;
  if (!exact_map_tile(blockIdx.x, tiles_m, tiles_n, tm, tn)) return;
  exact_gemm_tile<LD, BM, BN, SM, OCC, WIDE, false, false, EPI, kShort<LD, BN>>(p, tm * BM, tn * kTileCols<BN, EPI>, lds0, lds1,
                                                                               lds2, lds3, ldsc, ga);
}

// Up to kScanGroups groups are looked through by every wave, four a lane, so that no kernel has to run before to
// lay out the tiles: one load's latency and a scan over the lanes, against a launch and three loads in turn (BF16
// 64 experts of 8 rows, 512 -> 2 x 128: 9.1 us against 11.4; 256 of 100, 512 -> 2 x 256: 36.7 against 40.0). More
// groups would take more loads a lane; they get the prefix kernel of the plain grouped GEMMs.
constexpr int64_t kScanGroups = 256;
struct GroupTile {
  int64_t g, local, tiles_m, first_row, rows;
};
// The tile's group, its place in it and the group's rows; false: offsets that do not fit (no tile runs), or no tile.
// Tiles in XCD order: dispatch order b goes to XCD b % 8, and each XCD takes a contiguous run of the tiles.
template <int BM>
__device__ __forceinline__ bool scan_groups(const int64_t* __restrict__ offsets, int64_t groups, int64_t rows,
                                            int64_t tiles_n, GroupTile& at) {
  const int lane = threadIdx.x & 63;
  int64_t o[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) o[i] = offsets[min((int64_t)(4 * lane + i), groups)];
  bool bad = (lane == 0 && o[0] != 0) || (lane == 63 && o[4] != rows);
#pragma unroll
  for (int i = 0; i < 4; ++i) bad = bad || o[i + 1] < o[i];
  if (__ballot(bad)) return false;
  int n[4], sum = 0;                                      // row tiles: of all groups below 2^31
#pragma unroll
  for (int i = 0; i < 4; ++i) sum += n[i] = (int)((o[i + 1] - o[i] + BM - 1) / BM);
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d, 64);
    if (lane >= d) upto += v;
  }
  const int64_t total = __builtin_amdgcn_readlane(upto, 63) * tiles_n, T8 = (total + 7) / 8;
  if ((int64_t)blockIdx.x >= 8 * T8) return false;        // the grid may exceed the tile count
  const int64_t tile = (int64_t)blockIdx.x % 8 * T8 + blockIdx.x / 8;
  if (tile >= total) return false;
  const int src = __builtin_ctzll(__ballot(tile < upto * tiles_n));
  int64_t local = tile - __builtin_amdgcn_readlane(upto - sum, src) * tiles_n;
  int i = 0;
  int64_t tiles_m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {                           // among the lane's four
    const int64_t t = __builtin_amdgcn_readlane(n[j], src);
    if (i == j) {
      tiles_m = t;
      if (local >= t * tiles_n) {
        local -= t * tiles_n;
        ++i;
      }
    }
  }
  at.g = 4 * src + i;
  at.local = local;
  at.tiles_m = tiles_m;
  at.first_row = offsets[at.g];
  at.rows = offsets[at.g + 1] - at.first_row;
  return true;
}

// Per expert: group g covers the slots [offsets[g], offsets[g + 1]); tile order as in
// exact_grouped_kernel (each XCD a contiguous run, bands of row tiles down a weight slab).
// tile_prefix: NULL up to kScanGroups groups.
constexpr int kGatedBand = 4;
template <int LD, int BM, int BN, int SM, int OCC, int EPI>
__global__ void __launch_bounds__(256, OCC) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
gated_grouped_kernel(ExactProblem base, GatedArgs ga, const int64_t* __restrict__ offsets,
                     const int64_t* __restrict__ tile_prefix, int64_t groups, int64_t rows, int64_t tiles_n) {
  using C = gx::Cfg<LD, BM, BN, SM, OCC, false, EPI>;
  MXQ_EXACT_LDS(C)
  GroupTile at;
  if (!tile_prefix) {
    if (!scan_groups<BM>(offsets, groups, rows, tiles_n, at)) return;
  } else {
    const int64_t total = tile_prefix[groups];
    const int64_t T8 = (total + 7) / 8;
    if ((int64_t)blockIdx.x >= 8 * T8) return;            // the grid may exceed the tile count
    const int64_t tile = (int64_t)blockIdx.x % 8 * T8 + blockIdx.x / 8;
    if (tile >= total) return;
    at.g = find_group(tile_prefix, groups, tile);
    at.local = tile - tile_prefix[at.g];
    at.tiles_m = (tile_prefix[at.g + 1] - tile_prefix[at.g]) / tiles_n;
    at.first_row = offsets[at.g];
    at.rows = offsets[at.g + 1] - at.first_row;
  }
  const int64_t g = at.g;
  const int64_t band = at.local / (kGatedBand * tiles_n);
  const int64_t rows_in_band = min((int64_t)kGatedBand, at.tiles_m - band * kGatedBand);
  const int64_t idx = at.local - band * kGatedBand * tiles_n;
  const int64_t tm = band * kGatedBand + idx % rows_in_band, tn = idx / rows_in_band;
  ExactProblem p = base;
  p.a_base = at.first_row;
  p.m_valid = at.rows;
  const int64_t n = EPI == 1 ? 2 * ga.inter : ga.inter;   // rows of the expert's B
  if constexpr (LD == 6) {                                // K rows of inter NVFP4 elements
    const int64_t w_elems = g * base.k_end * base.ldb;
    p.B = base.B + w_elems / 2;
    p.sB = base.sB + w_elems / 16;
    p.tB = base.tB + g;
  } else {
    const int64_t b_elems = g * n * base.ldb;
    p.B = base.B + k_bytes<LD>(b_elems);
    if constexpr (LD == 2) {
      p.sB = base.sB + b_elems / 16;
      if (base.tB_mode == 2) { p.tB = base.tB + g; p.tB_mode = 1; }
      else p.tB = base.tB + g * n;
    }
  }
  // expert tails (waves with no or few valid rows skip their matrix work): NVFP4 as in exact_grouped_kernel;
  // against the transposed NVFP4 weights 2% with experts of 263 rows, nothing for BF16
  constexpr bool PART = LD == 2 || LD == 6;
  exact_gemm_tile<LD, BM, BN, SM, OCC, false, false, PART, EPI>(p, tm * BM, tn * kTileCols<BN, EPI>, lds0, lds1, lds2, lds3,
                                                                ldsc, ga);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

size_t gated_grouped_ws_bytes(int64_t groups) { return groups <= kScanGroups ? 0 : grouped_gemm_ws_bytes(groups); }

static ExactProblem gated_problem(int64_t rows, int64_t n, int64_t K, const void* A, const void* sA, const float* tA,
                                  int tA_mode, const void* B, const void* sB, const float* tB, int tB_mode) {
  ExactProblem p;
  p.A = (const uint8_t*)A; p.sA = (const uint8_t*)sA; p.tA = tA; p.tA_mode = tA_mode;
  p.a_idx = nullptr; p.a_rows = rows; p.a_base = 0; p.m_valid = rows; p.lda = K;
  p.B = (const uint8_t*)B; p.sB = (const uint8_t*)sB; p.tB = tB; p.tB_mode = tB_mode; p.n_valid = n; p.ldb = K;
  p.k_begin = 0; p.k_end = K; p.C = nullptr; p.ldc = 0;
  return p;
}

// As the plain GEMMs choose: 2 where K fills whole stages and the scale rows start 16-byte aligned, 1
// where K fills whole stages, else 0.
static int gated_scale_mode(int ld, int64_t K) {
  if (K % 64) return 0;
  return ld == 1 && K % 512 == 0 ? 2 : ld == 2 && K % 256 == 0 ? 2 : 1;
}

template <int LD, int SM, int EPI>
static void launch_gated_dense_t(const ExactProblem& p, const GatedArgs& ga, hipStream_t st) {
  auto go = [&](auto BMC, auto BNC, auto OC) {
    constexpr int BM = decltype(BMC)::value, BN = decltype(BNC)::value, OCC = decltype(OC)::value;
    const int64_t tm = (p.m_valid + BM - 1) / BM, tn = (ga.inter + kTileCols<BN, EPI> - 1) / kTileCols<BN, EPI>;
    hipLaunchKernelGGL((gated_dense_kernel<LD, BM, BN, SM, OCC, SM == 2 && OCC == 1, EPI>), dim3((unsigned)((tm * tn + 7) / 8 * 8)), dim3(256),
                       0, st, p, ga, tm, tn);
  };
  // 256 x 256 unless that leaves most of the 256 CUs idle
  const int64_t n = EPI == 1 ? 2 * ga.inter : ga.inter;
  if (((p.m_valid + 255) / 256) * ((n + 255) / 256) >= 192) go(ic<256>{}, ic<256>{}, ic<1>{});
  // small tiles, more than one a CU: two share it, one's epilogue beside the other's main loop (4096 x 2048 -> 2 x 768
  // BF16 43 -> 36 us, backward 2011 x 2048 of 4096 MXFP8 52 -> 49); one a CU keeps all of LDS for its stages (1024 x
  // 7168 -> 2 x 2048 BF16 72 against 103)
  else if (((p.m_valid + 127) / 128) * ((n + 127) / 128) > 256) go(ic<128>{}, ic<128>{}, ic<2>{});
  else go(ic<128>{}, ic<128>{}, ic<1>{});
}

template <int LD, int EPI>
static void launch_gated_dense_ld(const ExactProblem& p, const GatedArgs& ga, hipStream_t st) {
  const int sm = gated_scale_mode(LD, p.lda);
  if constexpr (LD != 0) {
    if (sm == 2) { launch_gated_dense_t<LD, 2, EPI>(p, ga, st); return; }
  }
  if (sm >= 1) launch_gated_dense_t<LD, 1, EPI>(p, ga, st);
  else launch_gated_dense_t<LD, 0, EPI>(p, ga, st);
}

// ---------------------------------------------------------------------------
// Few tiles: K split over them, the parts joined by a second kernel
// ---------------------------------------------------------------------------
// A tile walks K at some 0.45 us per 64, whatever else runs; with fewer tiles than half the CUs that walk is the
// call's time (64 x 7168 -> 2 x 2048 BF16: 58 us against 12 for its bytes). Parts of 512 K and more each leave
// their FP32 product in the workspace; the join adds them in order and ends as the epilogue does (25 us there).
// The parts double as long as the walk saved is longer than writing and reading the products that come
// with it, at 5 TB/s, and at first the second launch: 512 x 2048 -> 2 x 2048 MXFP8 stays whole (18 us against 22).
constexpr int64_t kPartK = 512;                           // a part's K is a multiple: whole stages and scale chunks
static int64_t gated_parts(int64_t M, int64_t n, int64_t K) {
  const int64_t tiles = ((M + 127) / 128) * ((n + 127) / 128);
  int64_t parts = 1;
  while (parts < 8 && tiles * parts * 2 <= 256 && K >= 2 * parts * kPartK) {
    const int64_t saved_ns = K / (2 * parts) * 7, product_ns = M * n * 8 / 5000;
    if (saved_ns <= (parts == 1 ? 2 * product_ns + 2500 : parts * product_ns)) break;
    parts *= 2;
  }
  return parts;
}
size_t gated_ws_bytes(int64_t M, int64_t n, int64_t K) {
  const int64_t parts = gated_parts(M, n, K);
  return parts == 1 ? 0 : (size_t)((parts * M * n * 4 + 255) / 256 * 256);
}

template <int LD, int SM>
__global__ void __launch_bounds__(256, 1) __attribute__((amdgpu_waves_per_eu(1, 1)))
gated_part_kernel(ExactProblem p, int64_t part_k, int64_t tiles_m, int64_t tiles_n) {
  constexpr bool WIDE = SM == 2;
  using C = gx::Cfg<LD, 128, 128, SM, 1, WIDE>;
  MXQ_EXACT_LDS(C)
  int64_t tm, tn;
  if (!exact_map_tile(blockIdx.x, tiles_m, tiles_n, tm, tn)) return;
  p.k_begin = (int64_t)blockIdx.y * part_k;
  p.k_end = min(p.k_begin + part_k, p.lda);
  p.C += (int64_t)blockIdx.y * p.m_valid * p.ldc;
  exact_gemm_tile<LD, 128, 128, SM, 1, WIDE>(p, tm * 128, tn * 128, lds0, lds1, lds2, lds3, ldsc);
}

// One thread: 8 h columns of a row.
template <int EPI, bool GU32>
__global__ void __launch_bounds__(256) gated_join_kernel(const float* __restrict__ parts, int n_parts, int64_t M, GatedArgs ga) {
  const int64_t I = ga.inter, n = EPI == 1 ? 2 * I : I, per_row = I / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= M * per_row) return;
  const int64_t row = at / per_row, col = at % per_row * 8;
  auto row8 = [&](const float* q, float* v) {
    const float4 x = reinterpret_cast<const float4*>(q)[0], y = reinterpret_cast<const float4*>(q)[1];
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  };
  auto sum8 = [&](int64_t c, float* v) {
    const float* q = parts + row * n + c;
    row8(q, v);
    for (int s = 1; s < n_parts; ++s) {
      float w[8];
      row8(q + s * M * n, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
  };
  auto put8 = [](uint16_t* to, const float* v) {
    *reinterpret_cast<uint4*>(to) = make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
                                               bf16x2_rne(v[6], v[7]));
  };
  float a[8], b[8], h[8];
  sum8(col, a);
  if constexpr (EPI == 1) {
    sum8(I + col, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = swiglu_forward(a[e], b[e]);
    put8(ga.h + row * I + col, h);
    if (ga.gu) {
      put8(ga.gu + row * 2 * I + col, a);
      put8(ga.gu + row * 2 * I + I + col, b);
    }
  } else {
    float g[8], u[8], dg[8], du[8];
    if constexpr (GU32) {
      row8((const float*)ga.gu_in + row * 2 * I + col, g);
      row8((const float*)ga.gu_in + row * 2 * I + I + col, u);
    } else {
      unpack8(*reinterpret_cast<const uint4*>((const uint16_t*)ga.gu_in + row * 2 * I + col), g);
      unpack8(*reinterpret_cast<const uint4*>((const uint16_t*)ga.gu_in + row * 2 * I + I + col), u);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) swiglu_backward(a[e], g[e], u[e], dg[e], du[e], h[e]);
    put8(ga.gu + row * 2 * I + col, dg);
    put8(ga.gu + row * 2 * I + I + col, du);
    if (ga.h) put8(ga.h + row * I + col, h);
  }
}

template <int LD, int EPI>
static void launch_gated_parts(ExactProblem p, const GatedArgs& ga, int64_t parts, void* ws, hipStream_t st) {
  const int64_t M = p.m_valid, n = EPI == 1 ? 2 * ga.inter : ga.inter, K = p.lda;
  const int64_t part_k = (K + parts * kPartK - 1) / (parts * kPartK) * kPartK, used = (K + part_k - 1) / part_k;
  p.n_valid = n;
  p.C = (float*)ws;
  p.ldc = n;
  const int64_t tm = (M + 127) / 128, tn = (n + 127) / 128;
  const dim3 grid((unsigned)((tm * tn + 7) / 8 * 8), (unsigned)used);
  auto go = [&](auto SMC) {
    hipLaunchKernelGGL((gated_part_kernel<LD, decltype(SMC)::value>), grid, dim3(256), 0, st, p, part_k, tm, tn);
  };
  const int sm = gated_scale_mode(LD, K);
  if constexpr (LD != 0) {
    if (sm == 2) go(ic<2>{});
  }
  if (LD == 0 || sm != 2) {
    if (sm >= 1) go(ic<1>{});
    else go(ic<0>{});
  }
  const dim3 join((unsigned)((M * (ga.inter / 8) + 255) / 256));
  if (EPI == 2 && ga.gu32)
    hipLaunchKernelGGL((gated_join_kernel<EPI, true>), join, dim3(256), 0, st, (const float*)ws, (int)used, M, ga);
  else hipLaunchKernelGGL((gated_join_kernel<EPI, false>), join, dim3(256), 0, st, (const float*)ws, (int)used, M, ga);
}

template <int LD, int EPI>
static void launch_gated_any(const ExactProblem& p, const GatedArgs& ga, void* ws, hipStream_t st) {
  const int64_t parts = gated_parts(p.m_valid, EPI == 1 ? 2 * ga.inter : ga.inter, p.lda);
  if (parts > 1) launch_gated_parts<LD, EPI>(p, ga, parts, ws, st);
  else launch_gated_dense_ld<LD, EPI>(p, ga, st);
}

// fmt: 1 MXFP8, 2 NVFP4, 3 BF16
hipError_t launch_gemm_swiglu(int fmt, int64_t M, int64_t inter, int64_t K, const void* A, const void* sA, const float* tA,
                              int tA_mode, const void* B, const void* sB, const float* tB, int tB_mode, void* h,
                              void* gate_up, void* ws, hipStream_t st) {
  const ExactProblem p = gated_problem(M, inter, K, A, sA, tA, tA_mode, B, sB, tB, tB_mode);
  const GatedArgs ga{inter, (uint16_t*)h, (uint16_t*)gate_up, nullptr, 0};
  if (fmt == 1) launch_gated_any<1, 1>(p, ga, ws, st);
  else if (fmt == 2) launch_gated_any<2, 1>(p, ga, ws, st);
  else launch_gated_any<0, 1>(p, ga, ws, st);
  return hipGetLastError();
}

// fmt: 1 MXFP8, 3 BF16
hipError_t launch_gemm_swiglu_backward(int fmt, int64_t M, int64_t inter, int64_t K, const void* A, const void* sA,
                                       const void* B, const void* sB, const void* gate_up, int gu32, void* d_gate_up,
                                       void* h, void* ws, hipStream_t st) {
  const ExactProblem p = gated_problem(M, inter, K, A, sA, nullptr, 0, B, sB, nullptr, 0);
  const GatedArgs ga{inter, (uint16_t*)h, (uint16_t*)d_gate_up, gate_up, gu32};
  if (fmt == 1) launch_gated_any<1, 2>(p, ga, ws, st);
  else launch_gated_any<0, 2>(p, ga, ws, st);
  return hipGetLastError();
}

template <int LD, int BM, int BN, int SM, int OCC, int EPI>
static void launch_gated_grouped_t(const ExactProblem& p, const GatedArgs& ga, const int64_t* offsets, int64_t groups,
                                   int64_t total, int64_t* prefix, hipStream_t st) {
  const int64_t tn = (ga.inter + kTileCols<BN, EPI> - 1) / kTileCols<BN, EPI>;
  if (groups <= kScanGroups) prefix = nullptr;
  else launch_tile_prefix(offsets, groups, total, BM, tn, prefix, st);
  // an upper bound on the tiles, a multiple of 8 so that the XCD order reaches every one
  const int64_t tiles = (((total + BM - 1) / BM + groups) * tn + 7) / 8 * 8;
  hipLaunchKernelGGL((gated_grouped_kernel<LD, BM, BN, SM, OCC, EPI>), dim3((unsigned)tiles), dim3(256), 0, st, p, ga,
                     offsets, prefix, groups, total, tn);
}

template <int EPI>
static void launch_gated_grouped_bf16(const ExactProblem& p, const GatedArgs& ga, const int64_t* offsets, int64_t groups,
                                      int64_t total, int64_t* prefix, hipStream_t st) {
  auto by_sm = [&](auto SMC) {
    constexpr int SM = decltype(SMC)::value;
    // experts of 384 rows and more on average fill 256-row tiles
    if (total / groups >= 384) launch_gated_grouped_t<0, 256, 256, SM, 1, EPI>(p, ga, offsets, groups, total, prefix, st);
    else launch_gated_grouped_t<0, 128, 128, SM, 2, EPI>(p, ga, offsets, groups, total, prefix, st);
  };
  if (gated_scale_mode(0, p.lda)) by_sm(ic<1>{});
  else by_sm(ic<0>{});
}

// fmt: 2 NVFP4, 3 BF16
hipError_t launch_grouped_gemm_swiglu(int fmt, int64_t groups, const int64_t* offsets, int64_t total, int64_t inter,
                                      int64_t K, const int32_t* a_row_index, int64_t a_rows, const void* A, const void* sA,
                                      const float* tA, int tA_mode, const void* B, const void* sB, const float* tB,
                                      int tB_mode, void* h, void* gate_up, void* ws, hipStream_t st) {
  ExactProblem p = gated_problem(0, inter, K, A, sA, tA, tA_mode, B, sB, tB, tB_mode);
  p.a_idx = a_row_index; p.a_rows = a_rows;
  const GatedArgs ga{inter, (uint16_t*)h, (uint16_t*)gate_up, nullptr, 0};
  int64_t* prefix = (int64_t*)ws;
  if (fmt == 2) {
    const int sm = gated_scale_mode(2, K);
    if (sm == 2) launch_gated_grouped_t<2, 128, 256, 2, 2, 1>(p, ga, offsets, groups, total, prefix, st);
    else if (sm == 1) launch_gated_grouped_t<2, 128, 128, 1, 2, 1>(p, ga, offsets, groups, total, prefix, st);
    else launch_gated_grouped_t<2, 128, 128, 0, 2, 1>(p, ga, offsets, groups, total, prefix, st);
  } else {
    launch_gated_grouped_bf16<1>(p, ga, offsets, groups, total, prefix, st);
  }
  return hipGetLastError();
}

// fmt: 3 BF16 (B the stacked (inter, K) transposes of W_d), 7 BF16 A x the stacked NVFP4 W_d (K, inter)
hipError_t launch_grouped_gemm_swiglu_backward(int fmt, int64_t groups, const int64_t* offsets, int64_t total,
                                               int64_t inter, int64_t K, const void* A, const void* B, const void* sB,
                                               const float* tB, const void* gate_up, int gu32, void* d_gate_up, void* h,
                                               void* ws, hipStream_t st) {
  ExactProblem p = gated_problem(0, inter, K, A, nullptr, nullptr, 0, B, sB, tB, 0);
  const GatedArgs ga{inter, (uint16_t*)h, (uint16_t*)d_gate_up, gate_up, gu32};
  int64_t* prefix = (int64_t*)ws;
  if (fmt == 7) {
    p.ldb = inter;
    // 256-row tiles where the experts fill them and the CUs get one each (1024 rows x 16 experts x 2048 columns
    // 680 us against 753); else 128 rows (263 rows x 128 experts x 768 columns 250 against 263-272, 512 x 8 x 1024
    // 96 against 140)
    const bool tall = total / groups >= 384 && (total + 255) / 256 * ((inter + 255) / 256) >= 192;
    if (tall) launch_gated_grouped_t<6, 256, 256, 0, 1, 2>(p, ga, offsets, groups, total, prefix, st);
    else launch_gated_grouped_t<6, 128, 256, 0, 1, 2>(p, ga, offsets, groups, total, prefix, st);
  } else {
    launch_gated_grouped_bf16<2>(p, ga, offsets, groups, total, prefix, st);
  }
  return hipGetLastError();
}

}  // namespace mxq
