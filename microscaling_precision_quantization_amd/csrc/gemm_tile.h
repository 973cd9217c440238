// The tile loop of the block-scaled GEMMs (gemm_exact.hip, gemm_swiglu.hip): one BM x BN tile of
//   C[m, n] = tA tB * sum_k A_hat[m, k] B_hat[n, k]
// from global memory through LDS and the matrix core to its epilogue. The formats, the data movement
// and the operand layouts are described in gemm_exact.hip.
#pragma once
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "swiglu.h"

namespace mxq {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float f32x4_nt __attribute__((ext_vector_type(4)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

namespace gx {
constexpr int kLdsBytes = 160 * 1024;           // gfx950 LDS per workgroup
template <int LD> struct RowBytes;
template <> struct RowBytes<0> { static constexpr int v = 128; };   // BF16
template <> struct RowBytes<1> { static constexpr int v = 64; };    // MXFP8
template <> struct RowBytes<2> { static constexpr int v = 32; };    // NVFP4
template <> struct RowBytes<3> { static constexpr int v = 32; };    // MXFP4
template <> struct RowBytes<4> { static constexpr int v = 128; };   // blockwise FP8: one 128-K block per stage
template <> struct RowBytes<5> { static constexpr int v = 128; };   // MXFP8 on the scaled FP8 MFMA: 128 K per stage
template <> struct RowBytes<6> { static constexpr int v = 128; };   // BF16 A x BF16 B built from NVFP4 weights (LDS rows BF16)

// Scale modes (SM):
//   0  general: K tiles may end early; per stage, one direct load per row and scale
//      unit (MXFP8 / MXFP4: 1 byte = one 32-block per unit, NVFP4: 2 bytes = two
//      16-blocks).
//   1  K % 64 == 0: per stage, one load per row of all the stage's blocks (2 / 4 bytes).
//   2  K % 64 == 0 and 16-byte aligned scale rows: 16 bytes per row (8 MXFP8 / 4 NVFP4
//      / 8 MXFP4 narrow stages) in one load, double-buffered in a separate LDS area;
//      cuts the scale cache-line requests by that factor.
// Each per-stage load lands in a 4-byte LDS slot per row (gfx950 places 1/2/4-byte
// direct loads at base + 4 lane); chunked scales in a 16-byte slot per row.
// Blockwise FP8 (LD 4): one FP32 scale per row and 128-K block, one dword load per row
// and stage (SU 1, SZ 4) whatever SM is.
template <int LD, int SM> struct ScaleDma {
  static constexpr int SU = LD == 4 ? 1 : (LD == 0 || LD == 6 || SM == 2) ? 0 : (SM == 1 ? 1 : 2);
  static constexpr int SZ = LD == 4 ? 4 : (LD == 1 || LD == 3) ? (SM >= 1 ? 2 : 1) : (SM >= 1 ? 4 : 2);
};

// OCC = workgroups meant to share one CU: the LDS budget of a workgroup is 1 / OCC of it.
// WIDE (chunked-scale mode only): 128 bytes per row and stage for every format (MXFP8 128 K,
// NVFP4 256 K per stage), i.e. fewer barriers and larger loads per stage.
// EPI: what the tile ends with (see exact_gemm_tile). SHORT (BF16): stages of 32 K, four in LDS, their loads
// one at a time between the matrix instructions.
template <int LD, int BM, int BN, int SM, int OCC = 1, bool WIDE = false, int EPI = 0, bool SHORT = false>
struct Cfg {
  static_assert(!SHORT || LD == 0, "short stages: BF16");
  static constexpr int RB = SHORT ? 64 : (WIDE && LD != 0) ? 128 : RowBytes<LD>::v;
  static constexpr int GS = SHORT ? 1 : 4;                // direct loads a unit (one M0 write)
  static constexpr int BK = (LD == 0 || LD == 6) ? RB / 2 : (LD == 1 || LD == 4 || LD == 5) ? RB : 2 * RB;   // K per stage
  static constexpr int SBS = LD == 5 ? RB / 64 : RB / 32;                 // sub-blocks per stage
  static_assert(!WIDE || SM == 2, "wide stages need chunked scales");
  static constexpr int A_BYTES = BM * RB, B_BYTES = BN * RB;
  static constexpr int SU = ScaleDma<LD, SM>::SU, SZ = ScaleDma<LD, SM>::SZ;
  static constexpr bool CH = SM == 2 && LD != 0 && LD != 4 && LD != 6;      // chunked scales
  // stages per 16-byte scale chunk (16 blocks)
  static constexpr int SPC = (LD == 1 || LD == 3 || LD == 5) ? 16 / (BK / 32) : LD == 2 ? 16 / (BK / 16) : 4;
  // chunk loads per wave: 64 rows of 16 bytes each; rows past BM + BN (a 128 x 256 tile
  // has 384) read zeros into the buffer's tail
  static constexpr int XS = CH ? (BM + BN + 255) / 256 : 0;
  static constexpr int CH_HALF = CH ? XS * 4096 : 0;              // one chunk buffer
  static constexpr int S_BYTES = SU * (BM + BN) * 4;              // scale slots of one stage
  static constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;
  static constexpr int FREE = kLdsBytes / OCC - 2 * CH_HALF;
  static constexpr int NS_LDS = (4 * STAGE <= FREE) ? 4 : (3 * STAGE <= FREE ? 3 : 2);
  static constexpr int NS = LD == 6 ? 2 : (CH && NS_LDS > SPC + 1) ? SPC + 1 : NS_LDS;   // (LD 6: see its B buffers)
  // 1 KiB wave instructions per wave (LD 6 builds its B tile through registers instead)
  static constexpr int IA = A_BYTES / 4096, IB = LD == 6 ? 0 : B_BYTES / 4096;
  static constexpr int IS = SU * (BM + BN) / 256;                 // 64-row scale loads per wave
  static_assert(SU == 0 || (BM + BN) % 256 == 0, "per-stage scale loads need BM + BN a multiple of 256");
  static constexpr int TI = BM / 64, TJ = BN / 64;                // 32x32 MFMA tiles per wave
  // staged epilogue (NVFP4, SwiGLU): per wave 32 rows x (BN/2 + 8) FP32 in LDS
  static constexpr bool EPI_STAGED = LD == 2 || EPI != 0;
  static constexpr int EPI_PITCH = BN / 2 + 8;
  static constexpr int EPI_BYTES = EPI_STAGED ? 4 * 32 * EPI_PITCH * 4 : 0;
  static constexpr int LDS_MAIN = NS * STAGE + (CH ? 2 * CH_HALF : 0);
  // (SwiGLU on NVFP4: tA of the tile's rows behind all of it)
  static constexpr int LDS_TOTAL = (LDS_MAIN > EPI_BYTES ? LDS_MAIN : EPI_BYTES) + (LD == 2 && EPI != 0 ? BM * 4 : 0);
  static_assert(A_BYTES % 4096 == 0 && B_BYTES % 4096 == 0, "tile must split into 1 KiB wave loads");
  // chunk c + 1 is issued at stage SPC c ahead of that stage's loads (tile SPC c + NS - 1);
  // the wait for tile SPC (c + 1) must cover it
  static_assert(!CH || NS - 1 <= SPC, "scale chunk must land with the tiles it covers");
};
}  // namespace gx

struct ExactProblem {
  const uint8_t* A;        // MXFP8: (rows, lda) bytes; NVFP4 / MXFP4: (rows, lda/2); BF16: (rows, lda) x 2 bytes
  const uint8_t* sA;       // MXFP8 / MXFP4 (rows, lda/32) E8M0; NVFP4 (rows, lda/16) E4M3
  const float* tA;         // NVFP4 decode scales (tA_mode 0 per A row, 1 tensor)
  int tA_mode;
  const int32_t* a_idx;    // optional gather of A rows
  int64_t a_rows, a_base, m_valid, lda;
  const uint8_t* B;
  const uint8_t* sB;
  const float* tB;
  int tB_mode;             // 0 per B row, 1 tensor
  int64_t n_valid, ldb;
  int64_t k_begin, k_end;  // reduction range (elements)
  float* C;
  int64_t ldc;
};

// The gated epilogues (rows of p.m_valid and p.a_base: the tile's group). EPI 1: the product is
// (gate | up), 2 inter wide; EPI 2: the product is dh, inter wide.
struct GatedArgs {
  int64_t inter;
  uint16_t* h;             // BF16 (rows, inter); EPI 2: NULL = not written
  uint16_t* gu;            // EPI 1: BF16 (rows, 2 inter), NULL = not written; EPI 2: d_gate_up, BF16 (rows, 2 inter)
  const void* gu_in;       // EPI 2: (rows, 2 inter) FP32 (gu32) or BF16
  int gu32;
};

__device__ __forceinline__ int64_t exact_src_row(const ExactProblem& p, int64_t r) {
  if (!p.a_idx) return p.a_base + r;
  const int64_t ar = p.a_idx[p.a_base + r];
  return (ar >= 0 && ar < p.a_rows) ? ar : -1;
}

template <int RB>
__device__ __forceinline__ int swz(int row) {
  return (row / (256 / RB)) % (RB / 16);
}

// s_waitcnt vmcnt(n) leaving lgkmcnt / expcnt unconstrained (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Raw buffer resource (stride 0): reads at offset o (VGPR offset + SGPR offset,
// both counted in the range check) return zeros when o + size > num_records.
__device__ __forceinline__ v4i make_rsrc(const void* base, uint32_t num_records) {
  const uint64_t a = (uint64_t)base;
  v4i r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu));
  r[2] = __builtin_amdgcn_readfirstlane((int)num_records);
  r[3] = __builtin_amdgcn_readfirstlane(0x00020000);     // 32-bit data format, no swizzle
  return r;
}
constexpr uint32_t kOutOfRange = 0x80000000u;            // beyond every num_records used here

__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}

// Buffer -> LDS direct loads. M0 holds the wave's LDS destination; lane l's data
// lands at M0 + 16 l (dwordx4) or M0 + 4 l (ubyte / ushort / dword, zero-extended).
// Issued through inline asm so that the compiler adds none of its own waits: all
// ordering is explicit (vmcnt waits before each stage barrier, a final vmcnt(0)).
// M0 is not otherwise used by these kernels.
template <int SZ>
__device__ __forceinline__ void buf_dma(v4i rs, uint32_t voff, uint32_t soff, uint32_t m0) {
  soff = __builtin_amdgcn_readfirstlane(soff);           // uniform values, kept in SGPRs
  m0 = __builtin_amdgcn_readfirstlane(m0);
  if constexpr (SZ == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(rs), "s"(soff) : "memory");
  else if constexpr (SZ == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(rs), "s"(soff) : "memory");
  else if constexpr (SZ == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ushort %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(rs), "s"(soff) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(rs), "s"(soff) : "memory");
}

// N (1..4) dwordx4 loads sharing one M0 write: load n lands at M0 + 1024 n + 16 lane.
// The instruction offset applies to the LDS destination and to the buffer offset
// alike (32-bit wrap-around), so each VGPR offset is pre-biased by -1024 n.
template <int N>
__device__ __forceinline__ void buf_dma16_group(v4i rs, const uint32_t* vo, uint32_t soff, uint32_t m0) {
  soff = __builtin_amdgcn_readfirstlane(soff);
  m0 = __builtin_amdgcn_readfirstlane(m0);
  if constexpr (N == 1)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(m0), "v"(vo[0]), "s"(rs), "s"(soff) : "memory");
  else if constexpr (N == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %3, %4 offen lds\n\t"
                 "buffer_load_dwordx4 %2, %3, %4 offen offset:1024 lds" ::"s"(m0), "v"(vo[0]), "v"(vo[1]), "s"(rs), "s"(soff) : "memory");
  else if constexpr (N == 3)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %4, %5 offen lds\n\t"
                 "buffer_load_dwordx4 %2, %4, %5 offen offset:1024 lds\n\tbuffer_load_dwordx4 %3, %4, %5 offen offset:2048 lds"
                 ::"s"(m0), "v"(vo[0]), "v"(vo[1]), "v"(vo[2]), "s"(rs), "s"(soff) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %5, %6 offen lds\n\t"
                 "buffer_load_dwordx4 %2, %5, %6 offen offset:1024 lds\n\tbuffer_load_dwordx4 %3, %5, %6 offen offset:2048 lds\n\t"
                 "buffer_load_dwordx4 %4, %5, %6 offen offset:%7 lds"
                 ::"s"(m0), "v"(vo[0]), "v"(vo[1]), "v"(vo[2]), "v"(vo[3]), "s"(rs), "s"(soff), "i"(3 * 1024) : "memory");
}

template <int LD>
__device__ __forceinline__ int64_t k_bytes(int64_t k) {
  return (LD == 0 || LD == 6) ? k * 2 : (LD == 1 || LD == 4 || LD == 5) ? k : k / 2;
}

typedef __attribute__((address_space(3))) const uint8_t* lds_cptr;
__device__ __forceinline__ lds_cptr as_lds(uint32_t a) { return (lds_cptr)(uintptr_t)a; }
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 lds_ld16(lds_cptr p) { return *(const __attribute__((address_space(3))) u32x4*)p; }

__device__ __forceinline__ void exact_drain() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// 8 E4M3 bytes (two dwords) -> 8 BF16, each exactly q * 2^(s-127).
__device__ __forceinline__ v8bf mx_to_bf16(uint32_t w0, uint32_t w1, float sc) {
  v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, sc, false);
  v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, sc, true);
  v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, sc, false);
  v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, sc, true);
  v8bf r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1]; r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}

// 2 x 16 E4M3 bytes as the A/B operand of the FP8 form of the scaled MFMA.
__device__ __forceinline__ v8i fp8_operand(const u32x4& lo, const u32x4& hi) {
  v8i v;
  v[0] = (int)lo.x; v[1] = (int)lo.y; v[2] = (int)lo.z; v[3] = (int)lo.w;
  v[4] = (int)hi.x; v[5] = (int)hi.y; v[6] = (int)hi.z; v[7] = (int)hi.w;
  return v;
}

// 32 E2M1 values (16 bytes) as the A/B operand of the FP4 form of the scaled MFMA, which
// reads the low four dwords.
__device__ __forceinline__ v8i fp4_operand(const u32x4& r) {
  v8i v;
  v[0] = (int)r.x; v[1] = (int)r.y; v[2] = (int)r.z; v[3] = (int)r.w;
  v[4] = 0; v[5] = 0; v[6] = 0; v[7] = 0;
  return v;
}

// 8 E2M1 values (one dword, low nibble first) times the E4M3 block scale S -> 8
// FP16, exactly: convert with the power-of-two part of S, multiply by its mantissa.
__device__ __forceinline__ v8h nv_to_f16(uint32_t w, float p2, v2h m2) {
  v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, p2, 0);
  v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, p2, 1);
  v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, p2, 2);
  v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, p2, 3);
  a = a * m2; b = b * m2; c = c * m2; d = d * m2;
  v8h r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1]; r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}

// The scaled converts use only the exponent field of their FP32 scale operand, an
// exponent field of 0 acting as 2^-127 (measured on MI355X). So an E8M0 code s is
// passed as the bits s << 23 (s = 0 included), and an E4M3 block scale S as S itself.

// E8M0 code -> scale operand of the MXFP8 converts.
__device__ __forceinline__ float mx_cvt_scale(uint32_t s) { return __uint_as_float(s << 23); }

// Byte SEL of `codes` (a positive E4M3 block scale S) -> the converts' scale operand
// (applies the power-of-two part 2^e of S) and the mantissa factor S / 2^e = 1.mmm as
// packed FP16 (exact). E4M3 subnormals are normal in FP32, so the split holds for
// them too; S = 0 scales by 2^-127, which flushes every E2M1 value to zero in FP16.
template <int SEL>
__device__ __forceinline__ void e4m3_split(uint32_t codes, float& p2, v2h& m2) {
  p2 = __builtin_amdgcn_cvt_f32_fp8((int)codes, SEL);
  const uint32_t mh = 0x3C00u | ((__float_as_uint(p2) >> 13) & 0x3FFu);
  const uint32_t pair = mh | (mh << 16);
  __builtin_memcpy(&m2, &pair, 4);
}

// Both bytes of a scale pair at once: p0 / p1 carry 2^e of bytes 0 / 1 as above, and mm holds
// their mantissa factors 1.mmm as packed FP16 (byte 0 low). The E4M3 codes convert to FP16
// exactly (subnormal codes become normal FP16), and forcing the FP16 exponent field to 15
// keeps just the factor S / 2^e -- the same values as the FP32 route.
__device__ __forceinline__ void e4m3_split2(uint32_t codes, float& p0, float& p1, v2h& mm) {
  p0 = __builtin_amdgcn_cvt_f32_fp8((int)codes, 0);
  p1 = __builtin_amdgcn_cvt_f32_fp8((int)codes, 1);
  const v2h s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, false);
  uint32_t b;
  __builtin_memcpy(&b, &s, 4);
  b = (b & 0x03FF03FFu) | 0x3C003C00u;
  __builtin_memcpy(&mm, &b, 4);
}

// nv_to_f16 with half H of a packed mantissa pair broadcast to both lanes of the multiply.
template <int H>
__device__ __forceinline__ v8h nv_to_f16_h(uint32_t w, float p2, v2h mm) {
  const v2h m2 = __builtin_shufflevector(mm, mm, H, H);
  return nv_to_f16(w, p2, m2);
}

template <int I> using ic = std::integral_constant<int, I>;

constexpr int gcd_int(int a, int b) { return b == 0 ? a : gcd_int(b, a % b); }
constexpr int lcm_int(int a, int b) { return a / gcd_int(a, b) * b; }

// Compile-time loop: f(ic<0>), ..., f(ic<N-1>).
template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(ic<I>{});
    static_for<I + 1, N>(f);
  }
}

// ---------------------------------------------------------------------------
// SwiGLU in the epilogue
// ---------------------------------------------------------------------------
// Rows of a wave's strip as a buffer: reads past them give zeros, writes past them are dropped, so that no
// access needs a branch (columns past the end take an offset past it).
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t strip_rsrc(const void* base, int64_t row, int64_t rows, int64_t row_bytes) {
  const int64_t bytes = rows > 0 ? rows * row_bytes : 0;
  return __builtin_amdgcn_make_buffer_rsrc((void*)((const char*)base + (rows > 0 ? row * row_bytes : 0)), (short)0, (int)bytes,
                                           0x00020000);
}
constexpr int kNonTemporal = 2;                           // the cache policy of the streaming stores
__device__ __forceinline__ void store8_bf16(__amdgpu_buffer_rsrc_t rs, const float* v, uint32_t off) {
  const v4u p = {bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
  __builtin_amdgcn_raw_buffer_store_b128(p, rs, (int)off, 0, kNonTemporal);
}

// Each 32-row strip of the wave's accumulators (NVFP4: times tB) goes to LDS as FP32; a lane then takes 8
// consecutive h columns of a row (NVFP4: times the row's tA, which the tile's prologue has put into LDS), so
// that every access to memory is 16 bytes and a row's segments are whole lines. The backward's reads of
// (g | u) of the next strip are on their way while one is worked on.
template <int LD, int BM, int BN, int TI, int TJ, int P, int EPI, bool GU32, typename Acc>
__device__ __forceinline__ void gated_epilogue(const ExactProblem& p, const GatedArgs& ga, int64_t m0, int64_t n0,
                                               const Acc& acc, uint8_t* lds, const float* lds_ta) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int h = lane >> 5, lr = lane & 31;
  constexpr int W = EPI == 1 ? BN / 4 : BN / 2;           // h columns of the wave
  constexpr int CPR = W / 8, RPI = 64 / CPR, KP = 32 / RPI;   // chunks of 8 columns a row, rows a pass, passes
  constexpr int ES = GU32 ? 4 : 2;
  float* stg = reinterpret_cast<float*>(lds) + wave * 32 * P;
  const int64_t I = ga.inter, col0 = n0 + wn * W, col = col0 + 8 * (lane % CPR);
  float tb[TJ];
  if constexpr (LD == 2) {
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int64_t c = col0 + (EPI == 1 ? j % (TJ / 2) : j) * 32 + lr;
      const int64_t row = EPI == 1 && j >= TJ / 2 ? I + c : c;
      tb[j] = c < I ? (p.tB_mode == 0 ? p.tB[row] : p.tB[0]) : 0.0f;
    }
  }
  // offsets of the lane's chunk in a row of I (h) and, for the row of pass k, in the strip
  const uint32_t rl0 = lane / CPR;
  const bool in = col < I;
  // the backward's reads run one unit ahead: a strip of BF16, half a strip of FP32 (64 registers either way)
  constexpr int NU = EPI == 2 && GU32 ? 2 : 1, UP = KP / NU, NQ = GU32 ? 4 : 2;
  v4u gu[EPI == 2 ? 2 : 1][UP][NQ];                       // per pass g (first half of NQ), u
  auto fetch = [&](int unit, auto B) {
    if constexpr (EPI == 2) {
      const int64_t r0 = m0 + wm * (BM / 2) + unit / NU * 32;
      const auto rs = strip_rsrc(ga.gu_in, p.a_base + r0, min((int64_t)32, p.m_valid - r0), 2 * I * ES);
#pragma unroll
      for (int k = 0; k < UP; ++k) {
        const uint32_t o = in ? (uint32_t)((rl0 + (unit % NU * UP + k) * RPI) * 2 * I + col) * ES : kOutOfRange;
#pragma unroll
        for (int q = 0; q < NQ / 2; ++q) {
          gu[decltype(B)::value][k][q] = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(o + 16 * q), 0, kNonTemporal);
          gu[decltype(B)::value][k][NQ / 2 + q] =
              __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(o + 16 * q), (int)(I * ES), kNonTemporal);
        }
      }
    }
  };
  fetch(0, ic<0>{});
  __syncthreads();                                        // every wave is done with the stage buffers
  static_for<0, TI>([&](auto IC) {
    constexpr int i = decltype(IC)::value;
    const int64_t r0 = m0 + wm * (BM / 2) + i * 32, rows = min((int64_t)32, p.m_valid - r0);
    const auto rsh = strip_rsrc(ga.h, p.a_base + r0, ga.h ? rows : 0, I * 2);
    const auto rsg = strip_rsrc(ga.gu, p.a_base + r0, ga.gu ? rows : 0, I * 4);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int rl = (r / 4) * 8 + h * 4 + (r % 4);
#pragma unroll
      for (int j = 0; j < TJ; ++j) stg[rl * P + j * 32 + lr] = LD == 2 ? acc[i][j][r] * tb[j] : acc[i][j][r];
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);                   // lgkmcnt(0): this wave's LDS writes landed
    static_for<0, KP>([&](auto KC) {
      constexpr int k = decltype(KC)::value, unit = i * NU + k / UP, B = EPI == 2 ? unit % 2 : 0;
      if constexpr (EPI == 2 && k % UP == 0 && unit + 1 < TI * NU) fetch(unit + 1, ic<(unit + 1) % 2>{});
      const uint32_t rl = rl0 + k * RPI;
      const float* src = stg + rl * P + 8 * (lane % CPR);
      const float ta = LD == 2 ? lds_ta[wm * (BM / 2) + i * 32 + rl] : 1.0f;
      float a[8], b[8], hv[8];
      auto row8 = [&](const float* q, float* v) {
        const float4 x = reinterpret_cast<const float4*>(q)[0], y = reinterpret_cast<const float4*>(q)[1];
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        if constexpr (LD == 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= ta;
        }
      };
      const uint32_t oh = in ? (uint32_t)(rl * I + col) * 2 : kOutOfRange;
      const uint32_t og = in ? (uint32_t)(rl * 2 * I + col) * 2 : kOutOfRange;
      row8(src, a);
      if constexpr (EPI == 1) {
        row8(src + W, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[e] = swiglu_forward(a[e], b[e]);
        store8_bf16(rsh, hv, oh);
        if (ga.gu) {
          store8_bf16(rsg, a, og);
          store8_bf16(rsg, b, in ? og + (uint32_t)(2 * I) : kOutOfRange);
        }
      } else {
        float dg[8], du[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float g, u;
          if constexpr (GU32) {
            g = __uint_as_float(gu[B][k % UP][e / 4][e % 4]);
            u = __uint_as_float(gu[B][k % UP][2 + e / 4][e % 4]);
          } else {
            const uint32_t gw = gu[B][k % UP][0][e / 2], uw = gu[B][k % UP][1][e / 2];
            g = e % 2 ? bf16_hi(gw) : bf16_lo(gw);
            u = e % 2 ? bf16_hi(uw) : bf16_lo(uw);
          }
          swiglu_backward(a[e], g, u, dg[e], du[e], hv[e]);
        }
        store8_bf16(rsg, dg, og);
        store8_bf16(rsg, du, in ? og + (uint32_t)(2 * I) : kOutOfRange);
        if (ga.h) store8_bf16(rsh, hv, oh);
      }
    });
    __builtin_amdgcn_s_waitcnt(0xC07F);                   // reads done before the next strip overwrites
  });
}

// Tile of BM x BN outputs over K in [k_begin, k_end); 4 waves in a 2 x 2 grid,
// each owning (BM/2) x (BN/2) accumulators.
//
// K advances in stages of 64 (NS stages in LDS, NS - 1 loads in flight); a stage
// splits into SBS sub-blocks of one 16-byte chunk per lane and fragment (BF16: 4
// of 16 K, MXFP8: 2 of 32 K, NVFP4: 1 of 64 K). The raw fragments of the next
// sub-block are read from LDS while the matrix core works on the current one;
// the loads of the stage NS - 1 ahead are interleaved with the first sub-block's
// MFMAs, and the barrier that publishes the next stage sits halfway through the
// last sub-block.
// AKM: A is given K-major -- (k, m) row-major, p.lda = m per row -- as the slot-major
// gradients of a weight-gradient GEMM are; BF16 with per-chunk K tails (SM 0) only.
// EPI 0: C, FP32. EPI 1 (SwiGLU): B is (2 inter, K), gate rows and then up rows, and n0 counts h columns:
// the tile covers BN / 2 of them, each wave BN / 4, its first BN / 4 product columns the gates and the
// others the ups of the same h columns, so that both meet in one wave's accumulators. EPI 2 (SwiGLU
// backward): the product is dh. Both write what swiglu_forward / swiglu_backward say.
template <int LD, int BM, int BN, int SM, int OCC = 1, bool WIDE = false, bool AKM = false, bool PART = false, int EPI = 0,
          bool SHORT = false>
__device__ __forceinline__ void exact_gemm_tile(const ExactProblem& p, int64_t m0, int64_t n0, uint8_t* lds0,
                                                uint8_t* lds1, uint8_t* lds2, uint8_t* lds3, uint8_t* ldsc,
                                                const GatedArgs& ga = GatedArgs{}) {
  using C = gx::Cfg<LD, BM, BN, SM, OCC, WIDE, EPI, SHORT>;
  constexpr int GS = C::GS;
  constexpr bool PAIR = EPI == 1;
  constexpr bool AL = SM >= 1;                            // every K tile full and 64-aligned
  constexpr bool CH = C::CH;
  constexpr int XS = C::XS, SPC = C::SPC;
  constexpr int RB = C::RB, NS = C::NS, TI = C::TI, TJ = C::TJ, IA = C::IA, IB = C::IB, IS = C::IS;
  constexpr int SBS = C::SBS;                             // sub-blocks per stage
  constexpr int NF = TI + TJ;                             // fragments per lane and sub-block
  constexpr int BS = LD == 4 ? 128 : (LD == 1 || LD == 3 || LD == 5) ? 32 : 16;   // elements per scale block
  constexpr int SEB = LD == 4 ? 4 : 1;                    // bytes per scale entry
  constexpr int EPC = (LD == 0 || LD == 6) ? 8 : (LD == 1 || LD == 4 || LD == 5) ? 16 : 32;   // elements per 16-byte chunk
  constexpr int OPS = IA + IB + IS;                       // direct loads per stage and wave (chunks aside)
  // stages per unrolled round (LD 6: four, one per B register buffer)
  constexpr int R = CH ? lcm_int(SPC, NS) : (LD == 6 ? 4 : NS);
  static_assert(R % NS == 0 && (!CH || R % SPC == 0), "round must cover whole slot and chunk cycles");
  static_assert((R * SBS) % 2 == 0, "fragment double buffer needs an even sub-block count per round");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int h = lane >> 5, lr = lane & 31;

  const int64_t ldA = k_bytes<LD>(p.lda), ldB = k_bytes<LD>(p.ldb);
  const int64_t a_rows_tile = max((int64_t)0, min((int64_t)BM, p.m_valid - m0));
  // PAIR: the rows from the tile's first gate row to the last up row; gate rows past inter read up rows,
  // up rows past the end zeros, and both only feed columns that are not stored
  const int64_t b_rows_tile = PAIR ? 2 * ga.inter - n0 : max((int64_t)0, min((int64_t)BN, p.n_valid - n0));
  const auto b_row = [&](int r) {
    if constexpr (PAIR) {
      constexpr int H = BN / 4;
      return (r / H) % 2 * ga.inter + r / (2 * H) * H + r % H;
    } else {
      return r;
    }
  };

  // --- operand descriptors and per-lane offsets (fixed over K) -------------------
  // A: rebased at the tile's first row, or (gather) at the operand start with
  // per-row offsets; rows outside the tile's valid range read zeros.
  const v4i rsA = p.a_idx ? make_rsrc(p.A, (uint32_t)min(p.a_rows * ldA, (int64_t)0x7FFFFFFF))
                          : make_rsrc(p.A + (p.a_base + m0) * ldA, (uint32_t)(a_rows_tile * ldA));
  const v4i rsB = LD == 6 ? rsA : make_rsrc(p.B + n0 * ldB, (uint32_t)(b_rows_tile * ldB));
  uint32_t voA[IA], voB[IB > 0 ? IB : 1];
  static_assert(!AKM || (LD == 0 && SM == 0 && C::BK == 64), "K-major A: BF16 weight gradients");
  // K-major A: LDS row k of a stage holds the tile's BM values of operand row k0 + k (2 BM
  // bytes), 16-byte chunk c at position c ^ 4 (k % 4) -- so that the transpose reads of one
  // 32-lane half (4 rows x 64 bytes) cover all 64 banks once.
  constexpr int AROW = 2 * BM;
  static_assert(!AKM || AROW >= 256, "K-major A swizzle spans 16 chunks of a row");
#pragma unroll
  for (int j = 0; j < IA; ++j) {
    const int pos = (wave * IA + j) * 1024 + lane * 16;   // byte in the A tile
    uint32_t o;
    if constexpr (AKM) {
      const int row = pos / AROW;
      const int lc = ((pos % AROW) / 16) ^ (4 * (row % 4));
      o = (uint32_t)(row * ldA + lc * 16);
    } else {
      const int row = pos / RB;
      const int lc = ((pos % RB) / 16) ^ swz<RB>(row);    // logical chunk stored at this position
      o = (uint32_t)(row * ldA + lc * 16);
      if (p.a_idx) {
        const int64_t src = row < a_rows_tile ? exact_src_row(p, m0 + row) : -1;
        o = src >= 0 ? (uint32_t)(src * ldA + lc * 16) : kOutOfRange;
      }
    }
    voA[j] = o - 1024u * (uint32_t)(j % GS);               // see buf_dma16_group
  }
#pragma unroll
  for (int j = 0; j < IB; ++j) {
    const int pos = (wave * IB + j) * 1024 + lane * 16;
    const int row = pos / RB;
    const int lc = ((pos % RB) / 16) ^ swz<RB>(row);
    voB[j] = (uint32_t)(b_row(row) * ldB + lc * 16) - 1024u * (uint32_t)(j % GS);
  }
  // Scales: load q of IS per wave covers 64 consecutive items of the [A rows | B rows]
  // list of unit u (SU units per stage); each lands in a 4-byte LDS slot per row.
  constexpr int BPU = ((LD == 1 || LD == 3) ? 2 : 4) / (C::SU > 0 ? C::SU : 1);   // blocks per unit
  v4i rsS[IS > 0 ? IS : 1];
  uint32_t voS[IS > 0 ? IS : 1];
#pragma unroll
  for (int q = 0; q < IS; ++q) {
    const int item0 = (wave * IS + q) * 64;
    const int u = item0 / (BM + BN);
    const int r0 = item0 % (BM + BN);
    const int row = r0 + lane;
    if (r0 < BM) {
      const int64_t lds_ = p.lda / BS * SEB;
      if (p.a_idx) {
        rsS[q] = make_rsrc(p.sA, (uint32_t)min(p.a_rows * lds_, (int64_t)0x7FFFFFFF));
        const int64_t src = row < a_rows_tile ? exact_src_row(p, m0 + row) : -1;
        voS[q] = src >= 0 ? (uint32_t)(src * lds_ + u * BPU) : kOutOfRange;
      } else {
        rsS[q] = make_rsrc(p.sA + (p.a_base + m0) * lds_, (uint32_t)(a_rows_tile * lds_));
        voS[q] = (uint32_t)(row * lds_ + u * BPU);
      }
    } else if (LD == 4 && p.tB_mode == 1) {
      // one scale per 128 x 128 block of B: every row of a 128-row block reads its block's
      // entry (n0 is a multiple of 128)
      const int64_t lds_ = p.ldb / BS * SEB;
      rsS[q] = make_rsrc(p.sB + (n0 / 128) * lds_, (uint32_t)((b_rows_tile + 127) / 128 * lds_));
      voS[q] = (uint32_t)(((row - BM) / 128) * lds_);
    } else {
      const int64_t lds_ = p.ldb / BS * SEB;
      rsS[q] = make_rsrc(p.sB + n0 * lds_, (uint32_t)(b_rows_tile * lds_));
      voS[q] = (uint32_t)(b_row(row - BM) * lds_ + u * BPU);
    }
  }

  // Chunked scales: load q of XS per wave covers rows (wave XS + q) 64 + lane of the
  // [A rows | B rows] list, 16 bytes (one chunk) per row; all loads of a wave fall in
  // one operand (BM is a multiple of 64 XS) and share one M0 write.
  v4i rsX = rsA;
  uint32_t voX[XS > 0 ? XS : 1];
  if constexpr (CH) {
    static_assert(BM % (64 * XS) == 0, "chunk loads of a wave must stay in one operand");
    const bool xa = wave * XS * 64 < BM;
    const int64_t lds_ = (xa ? p.lda : p.ldb) / BS;        // scale bytes per row
#pragma unroll
    for (int q = 0; q < XS; ++q) {
      const int row = (wave * XS + q) * 64 + lane;
      uint32_t o;
      if (xa && p.a_idx) {
        const int64_t src = row < a_rows_tile ? exact_src_row(p, m0 + row) : -1;
        o = src >= 0 ? (uint32_t)(src * lds_) : kOutOfRange;
      } else {
        o = (uint32_t)((xa ? row : b_row(row - BM)) * lds_);
      }
      voX[q] = o - 1024u * (uint32_t)q;
    }
    if (xa) rsX = p.a_idx ? make_rsrc(p.sA, (uint32_t)min(p.a_rows * lds_, (int64_t)0x7FFFFFFF))
                          : make_rsrc(p.sA + (p.a_base + m0) * lds_, (uint32_t)(a_rows_tile * lds_));
    else rsX = make_rsrc(p.sB + n0 * lds_, (uint32_t)(b_rows_tile * lds_));
  }
  const uint32_t lbase_c = lds_addr(ldsc);

  const uint32_t lbase[4] = {lds_addr(lds0), lds_addr(lds1), lds_addr(lds2), lds_addr(lds3)};

  // LD 6: the B tile is made from NVFP4 weight rows W[k][n] (E2M1 pairs along n, one E4M3
  // scale per 16 n, one FP32 decode scale t for the whole group): B[n][k] =
  // RNE_bf16(fl32(fl32(q S) t)), the dequantized weight transposed. It is kept K-major in
  // LDS -- row k of a stage holds the tile's 256 BF16 values of W row k0 + k, 16-byte chunk
  // c at position c ^ 5 (k % 4) -- and the MFMA fragments come out through transpose reads,
  // like a K-major A. Lane (w, l) of the 256 threads owns stage row kr = 16 w + 4 (l / 16) +
  // (l / 2) % 4 and, with q = 2 ((l / 8) % 2) + l % 2, the 32-n pieces q and q + 4 of it: two
  // 16-byte loads of packed E2M1 and four scale bytes per stage (six loads; narrow 8 x 8
  // blocks took sixteen and ran the DeepSeek-shaped dgrads 5-6% slower). Sub-block b
  // converts 16 values (two chunks); the last one writes the block's eight chunks (1% faster
  // than writing each sub-block's pair as it is made). The LDS takes 16-byte writes 8 lanes
  // (128 bytes) at a time: each such group holds 4 rows x 2 adjacent pieces, which the
  // rotation puts on 32 different banks (4 pieces of 2 rows per group, the first lane order,
  // cost 25% of the LDS cycles in bank conflicts); each 32-lane pass of the transpose reads
  // covers all 64 banks.
  const int kb_ = (int)p.k_begin;
  const int nk_ = ((int)p.k_end - kb_ + C::BK - 1) / C::BK;
  constexpr bool NVT = LD == 6;
  static_assert(!NVT || (BN == 256 && C::BK == 64 && C::SBS == 4 && TJ / 2 - 1 == 1 && (C::IA == 8 || C::IA == 4)),
                "the NVFP4-transposed B path is laid out for 256 x 64 stages of four sub-blocks");
  constexpr int BROW6 = 2 * BN;                           // bytes of one K-major B row in LDS
  constexpr int NB6 = 6;                                  // B loads per lane and stage
  __amdgpu_buffer_rsrc_t rsB6, rsS6;
  uint32_t voB6 = 0, voS6 = 0;
  uint32_t wo6[NVT ? 4 : 1] = {};                         // LDS offset of the lane's chunk c of piece q
  float t6 = 0.0f;
  int64_t rowB6 = 0, rowS6 = 0;
  if constexpr (NVT) {
    const int kr6 = 16 * wave + 4 * (lane >> 4) + ((lane >> 1) & 3), q6 = 2 * ((lane >> 3) & 1) + (lane & 1);
    const int a6 = kr6 & 3;
    rowB6 = p.ldb / 2;                                    // bytes per W row (p.ldb = N elements)
    rowS6 = p.ldb / 16;
    rsB6 = __builtin_amdgcn_make_buffer_rsrc((void*)p.B, (short)0, (int)min(p.k_end * rowB6, (int64_t)0x7FFFFFFF),
                                             0x00020000);
    rsS6 = __builtin_amdgcn_make_buffer_rsrc((void*)p.sB, (short)0, (int)min(p.k_end * rowS6, (int64_t)0x7FFFFFFF),
                                             0x00020000);
    // Columns at or past n_valid read whatever in-range bytes follow, or zeros past the
    // buffer; they only feed accumulator columns the epilogue never stores.
    const int64_t n = n0 + 32 * q6;
    voB6 = (uint32_t)(kr6 * rowB6 + n / 2);               // piece q; piece q + 4 is 64 bytes on
    voS6 = (uint32_t)(kr6 * rowS6 + n / 16);              // its two scale bytes; piece q + 4's at + 8
#pragma unroll
    for (int c = 0; c < 4; ++c) wo6[c] = (uint32_t)(kr6 * BROW6 + 16 * (4 * (q6 ^ a6) + (c ^ a6)));
    t6 = p.tB[0];
  }
  // Four register buffers: the B loads of tile t + 4 go out during stage t, so each block has
  // three stages to arrive before stage t + 3 converts it (16 values in each sub-block) and
  // writes it to its slot (2-4% faster dgrads than two buffers, one stage ahead; rounds of
  // four stages keep the buffer indices static).
  uint32_t bq6[4][NVT ? 8 : 1], bs6[4][NVT ? 4 : 1];
  uint32_t out6[NVT ? 32 : 1];                            // the converted block: chunk pairs of sub-blocks 0..3
  // loads of B tile t into buffer BUF, in the order the sub-blocks use them (rows at or past
  // k_end, and tiles past the end, read zeros)
  auto nvt_issue = [&](int t, auto BUF) {
    if constexpr (NVT) {
      constexpr int bf = decltype(BUF)::value;
      typedef unsigned int v4u_t __attribute__((ext_vector_type(4)));
      const int k0 = kb_ + t * C::BK;
      const bool past = t >= nk_;
      const int so = (int)(past ? kOutOfRange : (uint32_t)(k0 * rowB6));
      const int ss = (int)(past ? kOutOfRange : (uint32_t)(k0 * rowS6));
      const v4u_t d0 = __builtin_amdgcn_raw_buffer_load_b128(rsB6, (int)voB6, so, 0);
      bs6[bf][0] = __builtin_amdgcn_raw_buffer_load_b8(rsS6, (int)voS6, ss, 0);
      bs6[bf][1] = __builtin_amdgcn_raw_buffer_load_b8(rsS6, (int)(voS6 + 1), ss, 0);
      const v4u_t d1 = __builtin_amdgcn_raw_buffer_load_b128(rsB6, (int)(voB6 + 64), so, 0);
      bs6[bf][2] = __builtin_amdgcn_raw_buffer_load_b8(rsS6, (int)(voS6 + 8), ss, 0);
      bs6[bf][3] = __builtin_amdgcn_raw_buffer_load_b8(rsS6, (int)(voS6 + 9), ss, 0);
      bq6[bf][0] = d0.x; bq6[bf][1] = d0.y; bq6[bf][2] = d0.z; bq6[bf][3] = d0.w;
      bq6[bf][4] = d1.x; bq6[bf][5] = d1.y; bq6[bf][6] = d1.z; bq6[bf][7] = d1.w;
    }
  };
  // half H (8 values) of sub-block b's 16 values of the block in buffer BUF -> out6[8 b + 4 H ..],
  // BF16 pairs of adjacent n
  auto nvt_conv = [&](auto BUF, auto SB, auto H) {
    if constexpr (NVT) {
      constexpr int bf = decltype(BUF)::value, b = decltype(SB)::value, hh = decltype(H)::value;
      const uint32_t w = bq6[bf][4 * (b / 2) + 2 * (b % 2) + hh];
      const float Sb = __builtin_amdgcn_cvt_f32_fp8((int)bs6[bf][b], 0);   // exact E4M3 decode, no branch
      const v2f_t e0 = e2m1x2_to_f32<0>(w), e1 = e2m1x2_to_f32<1>(w);
      const v2f_t e2 = e2m1x2_to_f32<2>(w), e3 = e2m1x2_to_f32<3>(w);
      out6[8 * b + 4 * hh + 0] = bf16x2_rne((e0.x * Sb) * t6, (e0.y * Sb) * t6);   // q S exact, then * t
      out6[8 * b + 4 * hh + 1] = bf16x2_rne((e1.x * Sb) * t6, (e1.y * Sb) * t6);
      out6[8 * b + 4 * hh + 2] = bf16x2_rne((e2.x * Sb) * t6, (e2.y * Sb) * t6);
      out6[8 * b + 4 * hh + 3] = bf16x2_rne((e3.x * Sb) * t6, (e3.y * Sb) * t6);
    }
  };
  // sub-block b's two chunks (piece q + 4 (b / 2), chunks 2 (b % 2) and 2 (b % 2) + 1) into
  // the B area of slot S
  auto nvt_write = [&](auto SLOT, auto SB) {
    if constexpr (NVT) {
      constexpr int S = decltype(SLOT)::value, b = decltype(SB)::value;
      const uint32_t base = lbase[S] + C::A_BYTES + (uint32_t)(256 * (b / 2));
      const u32x4 v0 = {out6[8 * b + 0], out6[8 * b + 1], out6[8 * b + 2], out6[8 * b + 3]};
      const u32x4 v1 = {out6[8 * b + 4], out6[8 * b + 5], out6[8 * b + 6], out6[8 * b + 7]};
      *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(base + wo6[2 * (b % 2)]) = v0;
      *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(base + wo6[2 * (b % 2) + 1]) = v1;
    }
  };
  auto nvt_store = [&](auto BUF, auto SLOT) {
    static_for<0, 4>([&](auto SB) {
      nvt_conv(BUF, SB, ic<0>{});
      nvt_conv(BUF, SB, ic<1>{});
      nvt_write(SLOT, SB);
    });
  };

  const int kb = (int)p.k_begin, ke = (int)p.k_end;       // K <= 2^22
  const int nk = (ke - kb + C::BK - 1) / C::BK;

  // Uniform load parameters of tile t. Tiles past the end read zeros (out-of-range
  // SGPR offset); in the last tile, chunks and scale units at or beyond k_end are
  // turned out of range per lane.
  struct TileK { uint32_t sod, sos; int k0; bool tail; v4i rsa; };
  auto tile_k = [&](int t) {
    TileK r;
    r.k0 = kb + t * C::BK;
    const bool past = t >= nk;
    if constexpr (AKM) {
      // the stage's rows of the K-major A, clipped at k_end (rows past it read zeros; the
      // columns past m_valid of the last row read bytes that only feed unstored outputs)
      const int64_t rows = past ? 0 : min((int64_t)C::BK, (int64_t)(ke - r.k0));
      const int64_t bytes = rows > 0 ? rows * ldA - m0 * 2 : 0;
      r.rsa = make_rsrc(p.A + (int64_t)r.k0 * ldA + m0 * 2, (uint32_t)min(bytes, (int64_t)0x7FFFFFFF));
    }
    r.sod = past ? kOutOfRange : (uint32_t)((LD == 0 || LD == 6) ? 2 * r.k0 : (LD == 1 || LD == 4 || LD == 5) ? r.k0 : r.k0 / 2);
    r.sos = past ? kOutOfRange : (uint32_t)(r.k0 / BS * SEB);
    r.tail = !AL && !past && r.k0 + C::BK > ke;
    return r;
  };
  // DMA unit d of a tile into slot S: units 0 .. GA-1 are groups of up to 4 A loads,
  // GA .. GA+GB-1 groups of B loads, then the IS scale loads.
  constexpr int GA = (IA + GS - 1) / GS, GB = (IB + GS - 1) / GS, UNITS = GA + GB + IS;
  auto issue_unit = [&](const TileK& tk, auto SLOT, auto D) {
    constexpr int S = decltype(SLOT)::value, d = decltype(D)::value;
    const uint32_t lb = lbase[S];
    if constexpr (d < GA + GB) {
      constexpr bool isA = d < GA;
      constexpr int g = isA ? d : d - GA;
      constexpr int NI = isA ? IA : IB;
      constexpr int N = (NI - GS * g) < GS ? NI - GS * g : GS;
      uint32_t vo[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int j = GS * g + n;
        vo[n] = isA ? voA[j] : voB[j];
        if constexpr (!AL && !(AKM && isA)) {
          if (tk.tail) {
            const int pos = (wave * NI + j) * 1024 + lane * 16;
            const int lc = ((pos % RB) / 16) ^ swz<RB>(pos / RB);
            if (tk.k0 + lc * EPC >= ke) vo[n] = kOutOfRange - 1024u * (uint32_t)n;
          }
        }
      }
      const uint32_t m0v = lb + (isA ? 0 : C::A_BYTES) + (uint32_t)(wave * NI + GS * g) * 1024u;
      if constexpr (AKM && isA) buf_dma16_group<N>(tk.rsa, vo, 0u, m0v);
      else buf_dma16_group<N>(isA ? rsA : rsB, vo, tk.sod, m0v);
    } else if constexpr (IS > 0) {
      constexpr int q = d - GA - GB;
      uint32_t vo = voS[q];
      if constexpr (!AL) {
        const int u = ((wave * IS + q) * 64) / (BM + BN);
        if (tk.tail && tk.k0 + u * BPU * BS >= ke) vo = kOutOfRange;
      }
      const uint32_t m0v = lb + C::A_BYTES + C::B_BYTES + (uint32_t)(wave * IS + q) * 256u;
      buf_dma<C::SZ>(rsS[q], vo, tk.sos, m0v);
    }
  };
  // units [LO, HI) of a tile
  auto issue_range = [&](const TileK& tk, auto SLOT, auto LO, auto HI) {
    static_for<decltype(LO)::value, decltype(HI)::value>([&](auto D) { issue_unit(tk, SLOT, D); });
  };
  // scale chunk c (stages [SPC c, SPC c + SPC)) into chunk buffer c % 2 (k_begin is a multiple of a chunk's K)
  auto issue_chunk = [&](int c) {
    if constexpr (CH) {
      const uint32_t so = c * SPC < nk ? (uint32_t)(kb / BS + 16 * c) : kOutOfRange;
      const uint32_t m0v = lbase_c + (uint32_t)(c & 1) * C::CH_HALF + (uint32_t)(wave * XS) * 1024u;
      buf_dma16_group<XS>(rsX, voX, so, m0v);
    }
  };

  // --- fragments ---------------------------------------------------------------
  // raw[f]: the lane's 16-byte chunk of fragment f (A rows i = 0..TI-1, then B rows
  // j = 0..TJ-1) for one sub-block; sc[f]: its scale byte(s).
  // LD 5: raw holds K [16h, 16h+16) of the sub-block's first 32-K block, raw2 the same of
  // its second block (the scaled FP8 MFMA's operand layout).
  struct Frag { u32x4 raw[NF]; u32x4 raw2[LD == 5 ? NF : 1]; uint32_t sc[NF]; };
  Frag F[2];

  // LDS addresses of the fragment reads. Fragment rows start at multiples of 32 and
  // the swizzle period is 16 rows, so the swizzle depends on lr alone: the lane part
  // (xo) is one VGPR per sub-block, the wave part is uniform and the fragment part
  // is an instruction offset.
  uint32_t xo[SBS];
#pragma unroll
  for (int b = 0; b < SBS; ++b)
    xo[b] = (uint32_t)(lr * RB + ((((LD == 5 ? 4 : 2) * b + h) ^ swz<RB>(lr)) << 4));
  uint32_t xo2[LD == 5 ? SBS : 1];
  if constexpr (LD == 5) {
#pragma unroll
    for (int b = 0; b < SBS; ++b) xo2[b] = (uint32_t)(lr * RB + (((4 * b + 2 + h) ^ swz<RB>(lr)) << 4));
  }
  const uint32_t wA = (uint32_t)(wm * (BM / 2) * RB), wB = (uint32_t)(C::A_BYTES + wn * (BN / 2) * RB);
  const uint32_t xs = (uint32_t)(lr * 4);                 // scale slot of the lane's row
  const uint32_t wsA = (uint32_t)(C::A_BYTES + C::B_BYTES + wm * (BM / 2) * 4);
  const uint32_t wsB = (uint32_t)(C::A_BYTES + C::B_BYTES + (BM + wn * (BN / 2)) * 4);
  constexpr int SC_UNIT = (BM + BN) * 4;                  // bytes between scale units (SU == 2)

  // Chunked scales: the 16-byte chunk row of each fragment row (one per lane) is read into
  // registers once per chunk (SPC stages), at its first stage, and the stage's bytes are
  // taken from there: row r's byte (MXFP8 block b, MXFP4 block 2b + h) or byte pair (NVFP4
  // blocks 2h, 2h+1) of stage t sits at chunk + 16 r + (t % SPC) * bytes per stage. (Byte-wise LDS reads of
  // 16-byte-strided rows would each take several conflicting passes.)
  const uint32_t wcA = (uint32_t)(wm * (BM / 2) * 16), wcB = (uint32_t)((BM + wn * (BN / 2)) * 16);
  u32x4 chr[CH ? NF : 1];
  // K-major A fragments: two LDS transpose reads (ds_read_b64_tr_b16) per 32 x 16 fragment.
  // In a 16-lane group, lane i receives element i % 4 of the 8-byte rows addressed by
  // lanes i / 4 + 4 j (measured); lane (gq, l16) therefore addresses row 4 q + l16 / 4 of
  // the group's k block (q: first or second 4 k of the lane half) at the 4 m values
  // 4 (l16 % 4) onward, and receives 4 consecutive k of its own m -- the 16-bit MFMA
  // operand. akm_lane[i]: the lane's offset for fragment i, whose 4 chunks are the row's
  // chunk group q = wm TI + i, stored at group q ^ (k % 4).
  uint32_t akm_lane[AKM ? TI : 1] = {};
  if constexpr (AKM) {
    const int gq = lane >> 4, l16 = lane & 15, r = l16 >> 2;
    const int xa = 2 * (gq & 1) + ((l16 & 3) >> 1);
    const uint32_t rowoff = (uint32_t)((8 * (gq >> 1) + r) * AROW) + (uint32_t)((l16 & 1) * 8);
#pragma unroll
    for (int i = 0; i < TI; ++i) akm_lane[i] = rowoff + (uint32_t)((4 * ((wm * TI + i) ^ r) + xa) * 16);
  }
  // LD 6 B fragments, read the same way from the K-major B rows (chunk group q = wn TJ + j
  // of row k at group q ^ (k % 4), its chunk x at x ^ (k % 4)).
  uint32_t bkm_lane[NVT ? TJ : 1] = {};
  if constexpr (NVT) {
    const int gq = lane >> 4, l16 = lane & 15, r = l16 >> 2;
    const int xa = 2 * (gq & 1) + ((l16 & 3) >> 1);
    const uint32_t rowoff = (uint32_t)(C::A_BYTES + (8 * (gq >> 1) + r) * BROW6 + (l16 & 1) * 8);
#pragma unroll
    for (int j = 0; j < TJ; ++j) bkm_lane[j] = rowoff + (uint32_t)(16 * (4 * ((wn * TJ + j) ^ r) + (xa ^ r)));
  }
  // two transpose reads: rows k .. k + 3 of the lane's group at a, k + 4 .. k + 7 at a + 4 rows
  auto tr_frag = [&](uint32_t a, uint32_t row_bytes) {
    typedef short v4s16 __attribute__((ext_vector_type(4)));
    const v4s16 r0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s16*)(uintptr_t)a);
    const v4s16 r1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4s16*)(uintptr_t)(a + 4 * row_bytes));
    uint32_t w[4];
    __builtin_memcpy(&w[0], &r0, 8);
    __builtin_memcpy(&w[2], &r1, 8);
    return u32x4{w[0], w[1], w[2], w[3]};
  };
  // TP = t % SPC, known at compile time in the unrolled rounds (R is a multiple of SPC)
  auto read_sub = [&](int t, auto SLOT, auto SB, auto TP, Frag& fr, auto TIAC) {
    constexpr int S = decltype(SLOT)::value, b = decltype(SB)::value, tp = decltype(TP)::value;
    constexpr int TIA = decltype(TIAC)::value;           // A fragments this wave needs
    const lds_cptr pa = as_lds(lbase[S] + wA + xo[b]);
    const lds_cptr pb = as_lds(lbase[S] + wB + xo[b]);
    if constexpr (AKM) {
#pragma unroll
      for (int i = 0; i < TIA; ++i) fr.raw[i] = tr_frag(lbase[S] + akm_lane[i] + (uint32_t)(16 * b * AROW), AROW);
    } else {
#pragma unroll
      for (int i = 0; i < TIA; ++i) fr.raw[i] = lds_ld16(pa + i * 32 * RB);
    }
    if constexpr (NVT) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        fr.raw[TI + j] = tr_frag(lbase[S] + bkm_lane[j] + (uint32_t)(16 * b * BROW6), BROW6);
    } else {
#pragma unroll
      for (int j = 0; j < TJ; ++j) fr.raw[TI + j] = lds_ld16(pb + j * 32 * RB);
    }
    if constexpr (LD == 5) {
      const lds_cptr pa2 = as_lds(lbase[S] + wA + xo2[b]);
      const lds_cptr pb2 = as_lds(lbase[S] + wB + xo2[b]);
#pragma unroll
      for (int i = 0; i < TIA; ++i) fr.raw2[i] = lds_ld16(pa2 + i * 32 * RB);
#pragma unroll
      for (int j = 0; j < TJ; ++j) fr.raw2[TI + j] = lds_ld16(pb2 + j * 32 * RB);
    }
    if constexpr (CH) {
      if constexpr (tp == 0 && b == 0) {
        const uint32_t cb = lbase_c + (uint32_t)((t / SPC) & 1) * C::CH_HALF + (uint32_t)(lr * 16);
#pragma unroll
        for (int f = 0; f < NF; ++f)
          chr[f] = lds_ld16(as_lds(cb + (f < TI ? wcA + f * 512 : wcB + (f - TI) * 512)));
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if constexpr (LD == 1) {                      // one block per sub-block
          constexpr int idx = tp * SBS + b;
          fr.sc[f] = (chr[f][idx / 4] >> (8 * (idx % 4))) & 0xFFu;
        } else if constexpr (LD == 3 || LD == 5) {    // two blocks per sub-block, one per lane half
          constexpr int idx = tp * 2 * SBS + 2 * b;    // even: idx % 4 + h stays in its dword
          fr.sc[f] = (chr[f][idx / 4] >> (8 * (idx % 4 + h))) & 0xFFu;
        } else {                                      // four blocks per sub-block, two per lane
          fr.sc[f] = (chr[f][tp * SBS + b] >> (16 * h)) & 0xFFFFu;
        }
      }
    } else if constexpr (LD != 0 && LD != 4 && LD != 6) {
      const lds_cptr sa = as_lds(lbase[S] + wsA + xs), sb = as_lds(lbase[S] + wsB + xs);
      // MXFP8: the byte of block b; NVFP4: the two bytes of blocks 2h, 2h+1; MXFP4 (one
      // sub-block per stage): the byte of block h
      // LD 5 (four blocks per stage, two per sub-block): the byte of block 2b + h
      const int so = LD == 1 ? (C::SU == 1 ? b : b * SC_UNIT)
                   : LD == 2 ? (C::SU == 1 ? 2 * h : h * SC_UNIT)
                   : LD == 5 ? (C::SU == 1 ? 2 * b + h : b * SC_UNIT + h) : (C::SU == 1 ? h : h * SC_UNIT);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const lds_cptr q = (f < TI ? sa + f * 128 : sb + (f - TI) * 128) + so;
        fr.sc[f] = LD != 2 ? (uint32_t)*q : (uint32_t)*(const __attribute__((address_space(3))) uint16_t*)q;
      }
    }
  };

  v16f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  // Blockwise FP8: the matrix core sums one 128-K block into `part`; at the end of the
  // stage the block's FP32 scales are applied in software, acc += part * (sA[row] sB[col]),
  // and part restarts from zero.
  constexpr int TI4 = LD == 4 ? TI : 1, TJ4 = LD == 4 ? TJ : 1;
  v16f part[TI4][TJ4];
  float sa4[TI4][16], sb4[TJ4];
#pragma unroll
  for (int i = 0; i < TI4; ++i)
#pragma unroll
    for (int j = 0; j < TJ4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) part[i][j][r] = 0.0f;
  auto dst = [&](int i, int j) -> v16f& {
    if constexpr (LD == 4) return part[i][j];
    else return acc[i][j];
  };
  // the stage's scales (slot S, published by the barrier that ended the previous stage)
  auto read_scales4 = [&](auto SLOT) {
    if constexpr (LD == 4) {
      constexpr int S = decltype(SLOT)::value;
      const uint32_t base = lbase[S] + C::A_BYTES + C::B_BYTES;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {        // accumulator rows 8 g + 4 h + 0..3 of MFMA tile i
          const int row = wm * (BM / 2) + i * 32 + g * 8 + h * 4;
          const u32x4 v4 = lds_ld16(as_lds(base + (uint32_t)(row * 4)));
          sa4[i][4 * g + 0] = __uint_as_float(v4.x);
          sa4[i][4 * g + 1] = __uint_as_float(v4.y);
          sa4[i][4 * g + 2] = __uint_as_float(v4.z);
          sa4[i][4 * g + 3] = __uint_as_float(v4.w);
        }
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        sb4[j] = *(const __attribute__((address_space(3))) float*)as_lds(
            base + (uint32_t)((BM + wn * (BN / 2) + j * 32 + lr) * 4));
    }
  };
  auto promote4 = [&]() {
    if constexpr (LD == 4) {
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            acc[i][j][r] = __builtin_fmaf(part[i][j][r], sa4[i][r] * sb4[j], acc[i][j][r]);
            part[i][j][r] = 0.0f;
          }
    }
  };

  // Convert + MFMA one sub-block; hook(jj) runs after the MFMAs of B fragment jj.
  auto mma_sub = [&](const Frag& fr, auto TIAC, auto&& hook) {
    constexpr int TIA = decltype(TIAC)::value;
    if constexpr (LD == 0 || LD == 6) {
      v8bf fa[TI];
#pragma unroll
      for (int i = 0; i < TIA; ++i) __builtin_memcpy(&fa[i], &fr.raw[i], 16);
      static_for<0, TJ>([&](auto JJ) {
        constexpr int j = decltype(JJ)::value;
        v8bf fb;
        __builtin_memcpy(&fb, &fr.raw[TI + j], 16);
#pragma unroll
        for (int i = 0; i < TIA; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb, acc[i][j], 0, 0, 0);
        hook(JJ);
      });
    } else if constexpr (LD == 1 || LD == 4) {
      // MXFP8: E4M3 * 2^(s-127); blockwise FP8: the E4M3 values themselves (scale 2^0)
      v8bf fa0[TI], fa1[TI];
#pragma unroll
      for (int i = 0; i < TIA; ++i) {
        const float s = LD == 4 ? 1.0f : mx_cvt_scale(fr.sc[i]);
        fa0[i] = mx_to_bf16(fr.raw[i].x, fr.raw[i].y, s);
        fa1[i] = mx_to_bf16(fr.raw[i].z, fr.raw[i].w, s);
      }
      static_for<0, TJ>([&](auto JJ) {
        constexpr int j = decltype(JJ)::value;
        const float s = LD == 4 ? 1.0f : mx_cvt_scale(fr.sc[TI + j]);
        const v8bf fb0 = mx_to_bf16(fr.raw[TI + j].x, fr.raw[TI + j].y, s);
        const v8bf fb1 = mx_to_bf16(fr.raw[TI + j].z, fr.raw[TI + j].w, s);
#pragma unroll
        for (int i = 0; i < TIA; ++i) dst(i, j) = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa0[i], fb0, dst(i, j), 0, 0, 0);
#pragma unroll
        for (int i = 0; i < TIA; ++i) dst(i, j) = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa1[i], fb1, dst(i, j), 0, 0, 0);
        hook(JJ);
      });
    } else if constexpr (LD == 5) {
      // Native E4M3 x E4M3 scaled MFMA, 64 K per instruction: lane half h supplies K
      // [16h, 16h+16) of both 32-K blocks of the sub-block and the E8M0 byte of block h.
      v8i fa[TI];
#pragma unroll
      for (int i = 0; i < TIA; ++i) fa[i] = fp8_operand(fr.raw[i], fr.raw2[i]);
      static_for<0, TJ>([&](auto JJ) {
        constexpr int j = decltype(JJ)::value;
        const v8i fb = fp8_operand(fr.raw[TI + j], fr.raw2[TI + j]);
#pragma unroll
        for (int i = 0; i < TIA; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb, acc[i][j], 0, 0, 0, (int)fr.sc[i], 0,
                                                                     (int)fr.sc[TI + j]);
        hook(JJ);
      });
    } else if constexpr (LD == 3) {
      // Native E2M1 x E2M1 scaled MFMA, 64 K per instruction: lane half h supplies the
      // whole 32-K block of its chunk and that block's E8M0 byte (the operand layout the
      // sub-block reads already have).
      v8i fa[TI];
#pragma unroll
      for (int i = 0; i < TIA; ++i) fa[i] = fp4_operand(fr.raw[i]);
      static_for<0, TJ>([&](auto JJ) {
        constexpr int j = decltype(JJ)::value;
        const v8i fb = fp4_operand(fr.raw[TI + j]);
#pragma unroll
        for (int i = 0; i < TIA; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb, acc[i][j], 4, 4, 0, (int)fr.sc[i], 0,
                                                                     (int)fr.sc[TI + j]);
        hook(JJ);
      });
    } else {
      v8h fa[2][2][TI];        // [half][dword pair][i]
#pragma unroll
      for (int i = 0; i < TIA; ++i)
      {
        float p0, p1;
        v2h mm;
        e4m3_split2(fr.sc[i], p0, p1, mm);
        fa[0][0][i] = nv_to_f16_h<0>(fr.raw[i].x, p0, mm);
        fa[0][1][i] = nv_to_f16_h<0>(fr.raw[i].y, p0, mm);
        fa[1][0][i] = nv_to_f16_h<1>(fr.raw[i].z, p1, mm);
        fa[1][1][i] = nv_to_f16_h<1>(fr.raw[i].w, p1, mm);
      }
      static_for<0, TJ>([&](auto JJ) {
        constexpr int j = decltype(JJ)::value;
        float pb0, pb1;
        v2h mb;
        e4m3_split2(fr.sc[TI + j], pb0, pb1, mb);
        static_for<0, 2>([&](auto HF) {
          constexpr int hf = decltype(HF)::value;
          const float p2 = hf ? pb1 : pb0;
          const v8h fb0 = nv_to_f16_h<hf>(hf ? fr.raw[TI + j].z : fr.raw[TI + j].x, p2, mb);
          const v8h fb1 = nv_to_f16_h<hf>(hf ? fr.raw[TI + j].w : fr.raw[TI + j].y, p2, mb);
#pragma unroll
          for (int i = 0; i < TIA; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[hf][0][i], fb0, acc[i][j], 0, 0, 0);
#pragma unroll
          for (int i = 0; i < TIA; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[hf][1][i], fb1, acc[i][j], 0, 0, 0);
        });
        hook(JJ);
      });
    }
  };

  // The loads of tile t + NS - 1 are spread over the first PJ B-fragment steps of
  // sub-block 0; the barrier comes after B fragment BJ of the last sub-block.
  constexpr int BJ = TJ / 2 - 1;
  // SHORT: over all steps up to the barrier, so that the address path keeps up with four waves' loads
  // (all in sub-block 0 they take it twice as long as that sub-block's matrix work)
  constexpr int PJ = SHORT ? (SBS - 1) * TJ + BJ + 1 : SBS == 1 ? BJ + 1 : TJ;

  // Loads issued after tile t+1's data (issued in stage t+2-NS): the data of the
  // NS-2 later tiles, plus the chunk loads of chunk-start stages among the last NS-2
  // stages (issued ahead of their stage's data).
  auto allowed = [](auto RI) constexpr {
    constexpr int ri = decltype(RI)::value;
    int n = (NS - 2) * OPS + (NVT ? NB6 : 0);
    if constexpr (CH)
      for (int d = 0; d <= NS - 3; ++d)
        if (((ri - d) % R + R) % R % SPC == 0) n += XS;
    return n;
  };

  // One stage: tile kt (round position RI) in slot RI % NS.
  auto stage = [&](int kt, auto RI, auto TIAC) {
    constexpr int ri = decltype(RI)::value;
    constexpr int S = ri % NS;
    constexpr int SN = (ri + 1) % NS;                    // slot of the next tile
    constexpr int SL = (ri + NS - 1) % NS;               // slot refilled now
    constexpr int WAIT = allowed(RI);
    static_assert(WAIT < 64, "vmcnt range");
    const TileK tk = tile_k(kt + NS - 1);
    read_scales4(ic<S>{});
    static_for<0, SBS>([&](auto SB) {
      constexpr int b = decltype(SB)::value;
      constexpr int cur = (ri * SBS + b) & 1;
      if constexpr (b + 1 < SBS) {
        read_sub(kt, ic<S>{}, ic<b + 1>{}, ic<ri % SPC>{}, F[cur ^ 1], TIAC);
        __builtin_amdgcn_sched_barrier(0);              // keep the prefetch ahead of this sub-block's MFMAs
      }
      mma_sub(F[cur], TIAC, [&](auto JJ) {
        constexpr int jj = decltype(JJ)::value;
        if constexpr (b == 0 && jj == 0 && CH && ri % SPC == 0) {
          __builtin_amdgcn_sched_barrier(0);
          issue_chunk(kt / SPC + 1);                    // the next chunk, ahead of this stage's data loads
          __builtin_amdgcn_sched_barrier(0);
        }
        // LD 6: the B block of tile kt + 1 was loaded three stages ago, before the A loads that
        // the last barrier waited for, so it has landed (loads return in order). Sub-block b
        // converts its 16 values, interleaved with the matrix work (a scheduling barrier keeps
        // each sub-block's conversion in its sub-block: 1% faster than letting it rise into
        // the previous one). The last sub-block writes the block to tile kt + 1's slot before
        // the barrier. Tile kt + 1's A loads and the B register loads of tile kt + 4 go out
        // during sub-block 0.
        if constexpr (NVT && jj == 0) __builtin_amdgcn_sched_barrier(0);
        constexpr int step = b * TJ + jj;
        if constexpr ((SHORT || b == 0) && step < PJ) {
          __builtin_amdgcn_sched_barrier(0);
          issue_range(tk, ic<SL>{}, ic<(UNITS * step) / PJ>{}, ic<(UNITS * (step + 1)) / PJ>{});
          if constexpr (NVT && jj == PJ - 1) nvt_issue(kt + 4, ic<ri % 4>{});
          __builtin_amdgcn_sched_barrier(0);
        }
        // the first 8 values after fragment 0, the other 8 after fragment 1 (no scheduling
        // barrier: the scheduler interleaves them with the MFMAs)
        if constexpr (NVT && jj == 0) nvt_conv(ic<(ri + 1) % 4>{}, ic<b>{}, ic<0>{});
        if constexpr (NVT && jj == 1) {
          nvt_conv(ic<(ri + 1) % 4>{}, ic<b>{}, ic<1>{});
          if constexpr (b + 1 == SBS) {
            __builtin_amdgcn_sched_barrier(0);
            static_for<0, 4>([&](auto BB) { nvt_write(ic<SL>{}, BB); });
          }
        }
        if constexpr (b + 1 == SBS && jj == BJ) {
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (NVT) __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): B writes have landed
          wait_vmcnt<WAIT>();                           // tile kt + 1 has landed (this wave's loads)
          __builtin_amdgcn_s_barrier();                 // ... and every wave's; slot S fully read
          __builtin_amdgcn_sched_barrier(0);
          read_sub(kt + 1, ic<SN>{}, ic<0>{}, ic<(ri + 1) % SPC>{}, F[cur ^ 1], TIAC);
          __builtin_amdgcn_sched_barrier(0);
        }
      });
    });
    promote4();
  };

  if constexpr (LD == 2 && EPI != 0) {                    // the epilogue's row scales, out of its way
    if (threadIdx.x < BM) {
      const int64_t row = m0 + threadIdx.x;
      const int64_t src = row < p.m_valid ? exact_src_row(p, row) : -1;
      reinterpret_cast<float*>(lds0 + C::LDS_TOTAL - BM * 4)[threadIdx.x] =
          src < 0 ? 0.0f : p.tA_mode == 0 ? p.tA[src] : p.tA[0];
    }
  }
  // prologue: scale chunk 0, tiles 0 .. NS-2 in flight, then the first sub-block's fragments
  issue_chunk(0);
  static_for<0, NS - 1>([&](auto T) { issue_range(tile_k(T.value), T, ic<0>{}, ic<UNITS>{}); });
  if constexpr (NVT) {
    static_assert(NS == 2 && R == 4, "the B register buffers rotate with rounds of four stages over two slots");
    nvt_issue(0, ic<0>{});
    nvt_store(ic<0>{}, ic<0>{});                        // tile 0 into slot 0 (waits for everything)
    nvt_issue(1, ic<1>{});                              // in flight into the first stages
    nvt_issue(2, ic<2>{});
    nvt_issue(3, ic<3>{});
    __builtin_amdgcn_s_waitcnt(0xC07F);
  }
  wait_vmcnt<(NS - 2) * OPS + (NVT ? NB6 : 0)>();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);

  // Whole rounds of R stages: stages past the end multiply zeros (their loads are
  // out of range), which adds nothing to the accumulators.
  const int rounds = (nk + R - 1) / R;
  // BF16 tiles sharing a CU: the workgroup in its main loop issues ahead of one in its
  // prologue or FP32 epilogue (DeepSeek expert wgrads 5% faster; no gain measured for the
  // NVFP4 and MXFP8 kernels, which keep equal priorities)
  constexpr bool PRIO = OCC > 1 && LD == 0;
  // main loop for a wave that needs its first TIA 32-row A fragments (the others cover
  // only rows past m_valid: their MFMAs would multiply zeros into rows never stored)
  auto main_loop = [&](auto TIAC) {
    read_sub(0, ic<0>{}, ic<0>{}, ic<0>{}, F[0], TIAC);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (PRIO) __builtin_amdgcn_s_setprio(1);
    for (int r = 0; r < rounds; ++r) {
      const int kt = r * R;
      static_for<0, R>([&](auto RI) { stage(kt + RI.value, RI, TIAC); });
    }
    if constexpr (PRIO) __builtin_amdgcn_s_setprio(0);
  };
  if constexpr (PART) {
    // Row-grouped tiles end where their expert does: in an expert's last row tile a wave
    // whose rows are all or mostly padding runs the loop with fewer A fragments (every
    // wave still does its share of the loads, conversions and barriers).
    const int64_t rows_left = p.m_valid - (m0 + wm * (BM / 2));
    const int vg = rows_left <= 0 ? 0 : (int)min((rows_left + 31) / 32, (int64_t)TI);
    if (vg >= TI) main_loop(ic<TI>{});
    else if (vg == 0) main_loop(ic<0>{});
    else if (vg == 1) main_loop(ic<1>{});
    else if (vg == 2) main_loop(ic<(TI > 2 ? 2 : TI)>{});
    else main_loop(ic<TI>{});
  } else {
    main_loop(ic<TI>{});
  }
  wait_vmcnt<0>();                    // no direct load may still target this workgroup's LDS
  exact_drain();

  if constexpr (EPI != 0) {
    const float* ta = reinterpret_cast<const float*>(lds0 + C::LDS_TOTAL - (LD == 2 ? BM * 4 : 0));
    if (EPI == 2 && ga.gu32) gated_epilogue<LD, BM, BN, TI, TJ, C::EPI_PITCH, EPI, true>(p, ga, m0, n0, acc, lds0, ta);
    else gated_epilogue<LD, BM, BN, TI, TJ, C::EPI_PITCH, EPI, false>(p, ga, m0, n0, acc, lds0, ta);
  } else if constexpr (C::EPI_STAGED) {
    // NVFP4: C = tA tB acc. Each 32-row strip of the wave's block is scaled into LDS, then
    // leaves as 16-byte row segments (measured: 12-40% faster dense NVFP4 GEMMs than
    // scaling and storing element by element; no gain for the other formats).
    __syncthreads();                    // every wave is done with the stage buffers
    constexpr int P = C::EPI_PITCH;
    float* stg = reinterpret_cast<float*>(lds0) + wave * 32 * P;
    const int64_t col0 = n0 + wn * (BN / 2);
    float tbj[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int64_t col = col0 + j * 32 + lr;
      tbj[j] = col < p.n_valid ? (p.tB_mode == 0 ? p.tB[col] : p.tB[0]) : 0.0f;
    }
    const bool vec_ok = (p.ldc % 4 == 0) && ((reinterpret_cast<uintptr_t>(p.C) & 15) == 0);
    // tA of the lane's 16 rows of each strip, all loads issued before the first is used
    float ta[TI][16];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t row = m0 + wm * (BM / 2) + i * 32 + (r / 4) * 8 + h * 4 + (r % 4);
        const int64_t arow = row < p.m_valid ? exact_src_row(p, row) : -1;
        ta[i][r] = arow < 0 ? 0.0f : p.tA_mode == 0 ? p.tA[arow] : p.tA[0];
      }
    // interior tile with 16-byte aligned rows: no per-chunk checks; each store instruction
    // covers whole staged rows, lane l taking chunk l % CPR of row l / CPR
    const bool interior = vec_ok && m0 + BM <= p.m_valid && n0 + BN <= p.n_valid;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int64_t rbase = m0 + wm * (BM / 2) + i * 32;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int rl = (r / 4) * 8 + h * 4 + (r % 4);
#pragma unroll
        for (int j = 0; j < TJ; ++j) stg[rl * P + j * 32 + lr] = (acc[i][j][r] * ta[i][r]) * tbj[j];
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt(0): this wave's LDS writes landed
      constexpr int CPR = BN / 8;                    // 16-byte chunks per staged row
      constexpr int RPI = 64 / CPR;                  // staged rows per store instruction
      if (interior) {
        const int lrow = lane / CPR, lch = lane % CPR;
        float* dst = p.C + (rbase + lrow) * p.ldc + col0 + 4 * lch;
        const float* src = stg + lrow * P + 4 * lch;
#pragma unroll
        for (int k = 0; k < 32 / RPI; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(src + k * RPI * P);
          const f32x4_nt vv = {v.x, v.y, v.z, v.w};
          __builtin_nontemporal_store(vv, reinterpret_cast<f32x4_nt*>(dst + k * RPI * p.ldc));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 32 * CPR / 64; ++k) {
          const int idx = k * 64 + lane;
          const int rl = idx / CPR, ch = idx % CPR;
          const int64_t row = rbase + rl, col = col0 + ch * 4;
          if (row >= p.m_valid) continue;
          const float4 v = *reinterpret_cast<const float4*>(stg + rl * P + ch * 4);
          float* dstp = p.C + row * p.ldc + col;
          if (vec_ok && col + 4 <= p.n_valid) {
            const f32x4_nt vv = {v.x, v.y, v.z, v.w};
            __builtin_nontemporal_store(vv, reinterpret_cast<f32x4_nt*>(dstp));
          } else {
            if (col < p.n_valid) dstp[0] = v.x;
            if (col + 1 < p.n_valid) dstp[1] = v.y;
            if (col + 2 < p.n_valid) dstp[2] = v.z;
            if (col + 3 < p.n_valid) dstp[3] = v.w;
          }
        }
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);           // reads done before the next strip overwrites
    }
  } else if (m0 + BM <= p.m_valid && n0 + BN <= p.n_valid) {
    // interior tile (the common case): no per-element bounds checks, one row pointer per
    // accumulator row and the TJ column blocks at fixed offsets from it
    float* cw = p.C + (m0 + wm * (BM / 2) + h * 4) * p.ldc + n0 + wn * (BN / 2) + lr;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float* cr = cw + (int64_t)(i * 32 + (r / 4) * 8 + (r % 4)) * p.ldc;
#pragma unroll
        for (int j = 0; j < TJ; ++j) __builtin_nontemporal_store(acc[i][j][r], cr + j * 32);
      }
  } else {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t row = m0 + wm * (BM / 2) + i * 32 + (r / 4) * 8 + h * 4 + (r % 4);
        if (row >= p.m_valid) continue;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const int64_t col = n0 + wn * (BN / 2) + j * 32 + lr;
          if (col < p.n_valid) __builtin_nontemporal_store(acc[i][j][r], p.C + row * p.ldc + col);
        }
      }
  }
}

// XCD-aware raster: dispatch order b round-robins over the 8 XCDs; each XCD gets a
// contiguous run of logical tiles, walked in bands of 4 tile rows so the
// workgroups resident on one XCD share operand tiles in its L2.
__device__ __forceinline__ bool exact_map_tile(int64_t b, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn) {
  const int64_t T = tiles_m * tiles_n;
  const int64_t T8 = (T + 7) / 8;
  const int64_t L = (b % 8) * T8 + b / 8;
  if (L >= T) return false;
  const int64_t band = L / (4 * tiles_n);
  const int64_t rows_in_band = min((int64_t)4, tiles_m - band * 4);
  const int64_t idx = L - band * 4 * tiles_n;
  tm = band * 4 + idx % rows_in_band;
  tn = idx / rows_in_band;
  return true;
}

// One LDS block per workgroup, carved into the NS stage slots and the scale-chunk buffers
// (and reused by the staged epilogue once the main loop is done).
#define MXQ_EXACT_LDS(C)                                                                         \
  __shared__ __attribute__((aligned(1024))) uint8_t lds_all[C::LDS_TOTAL];                         \
  uint8_t* lds0 = lds_all;                                                                        \
  uint8_t* lds1 = lds_all + C::STAGE;                                                             \
  uint8_t* lds2 = lds_all + 2 * C::STAGE;                                                         \
  uint8_t* lds3 = lds_all + 3 * C::STAGE;                                                         \
  uint8_t* ldsc = lds_all + C::NS * C::STAGE;

// Group of a tile: the largest g with tile_prefix[g] <= tile (tile_prefix is non-decreasing
// and tile < tile_prefix[groups]). Each wave narrows the range 64-fold per round with one
// load per lane and a ballot (two rounds for up to 4096 groups).
__device__ __forceinline__ int64_t find_group(const int64_t* __restrict__ prefix, int64_t groups, int64_t tile) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, span = groups;                 // answer in [lo, lo + span)
  while (span > 1) {
    const int64_t step = (span + 63) / 64;
    const int64_t g = lo + (int64_t)lane * step;
    const bool ok = g < lo + span && prefix[g] <= tile;
    const uint64_t m = __ballot(ok);              // lanes 0 .. last are set (lane 0 always)
    const int last = 63 - __builtin_clzll(m);
    const int64_t nlo = lo + (int64_t)last * step;
    span = min(step, lo + span - nlo);
    lo = nlo;
  }
  return lo;
}

}  // namespace mxq
