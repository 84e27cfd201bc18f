// Block-scaled GEMM C = A B^T on 16 x 16 x 128 matrix instructions: FP8 x FP8 under
// fp32 scales per 1 x 128 of A and 128 x 128 of B, dense or by expert (groups.h),
// and MXFP4 x MXFP4 by expert (dense: gemm_mx.hip, gemm_mxfp4.hip).
//
// FP8: a K step of 128 is one scale block, so the step's MFMA starts from
// zero, and the vector ALU adds its partial sum times s_A(row) s_B(tile):
//   C[i][j] = sum over blocks q of s_A[i][q] s_B[j / 128][q] P_q[i][j].
// gfx950's FP8 MFMAs lose low bits inside their 128-term sum: of 8 products
// added together, each loses less than 2^-13 of the largest (measured with one
// large product and seven small ones; 1.4e-5 of the result on quantized normal
// values). A bf16 result has an error of 1.7e-3 from its own rounding, so it
// takes P from the FP8 MFMA, at twice the rate of the bf16 one (times in us with it / with
// the bf16 one: 64 x 2048 x 4096 10.1 / 11.5, 300 x 2048 x 4096 14.9 / 18.8, 1500 x 2048 x 4096
// 27.6 / 37.2, 6000 x 8192 x 8192 337 / 764). An fp32
// result takes P from four bf16 MFMAs (EXACT): every E4M3 value is a bf16
// value, and those return the rounded exact sum. (Few rows of A: gemm_few_rows.hip, exact
// for both.)
// MXFP4: the MFMA applies both E8M0 scales and accumulates.
//
// Operands and A's (MXFP4: both) scales go HBM -> LDS directly (buffer_load ...
// lds) into a ring of NS stages, a K step each, NS - 1 of them in flight: with few tiles the
// loads' latency is what a step takes. A step is 128 bytes of each row, a whole line:
// 128 K of FP8, 256 K (two MFMAs) of MXFP4. The buffer view of a tile ends with
// the group's rows, so rows past the end load as zeros. The 16-byte chunk c of LDS
// row r sits in slot c ^ swz(r), so that the 16 lanes that read one column of
// chunks hit distinct banks.
//
// B goes first into the MFMA: lane r + 16 g then holds C[row r][columns 4 g ..
// 4 g + 3] of a tile, one row (one s_A) and a run of columns to store.
#include <type_traits>

#include "bf16.h"
#include "fp8_encode.h"
#include "groups.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
using fp8::bf16x8;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
constexpr uint32_t kOOB = 0x80000000u;        // an offset past every buffer's range
constexpr int kNonTemporal = 2;               // cache policy of a load: streamed
constexpr int kChain = 48;                    // MFMAs per accumulation chain (fp32 results)
constexpr int kRow = 128, kCpr = kRow / 16;   // LDS bytes and chunks of a row's K step
constexpr int kRpb = 64 / kCpr;               // rows per 1 KB load of a wave

// Tile geometry: waves of 16 TMW x 16 TNW, WM x WN of them; NS stages. ALIGNED: a
// row's MXFP4 scales start on dwords (K % 128 = 0), so that a step's eight are
// two loads; otherwise they are eight loads of a byte, which LDS holds as a dword.
// STREAM_B: B's loads are non-temporal.
template <int FMT, int TMW_, int TNW_, int WM_, int WN_, int NS_, bool ALIGNED_ = true, bool STREAM_B_ = false>
struct Geo {
  static constexpr int TMW = TMW_, TNW = TNW_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr bool kAligned = ALIGNED_;
  static constexpr bool kStreamB = STREAM_B_;
  static constexpr int BM = 16 * TMW * WM, BN = 16 * TNW * WN;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr bool kFp8 = FMT == kFP8B128;
  static constexpr int kOffB = BM * kRow;
  // Scales, a dword a row, loaded 64 rows at a time: FP8 s_A of A's rows; MXFP4
  // four of the step's of A's and then of B's rows, and the other four, or (not
  // ALIGNED) that eight times, a byte of each.
  static constexpr int kOffS = kOffB + BN * kRow;
  static constexpr int kScaleA = (BM + 63) / 64, kScaleGroups = kFp8 ? kScaleA : kScaleA + (BN + 63) / 64;
  static constexpr int kScaleParts = kFp8 ? 1 : kAligned ? 2 : 8, kScaleLoads = kScaleGroups * kScaleParts;
  static constexpr int kCodeLoads = (BM + BN) / kRpb;
  // Loads of a wave and step: every wave the same number, so that a count of
  // outstanding loads means the same steps in all (the rest go nowhere: out of
  // range, into LDS that nobody reads).
  static constexpr int kLoads = (kCodeLoads + kScaleLoads + kWaves - 1) / kWaves;
  static constexpr int kStage = kOffS + kScaleLoads * 256;
  static constexpr int kDummy = NS * kStage, kSmem = kDummy + 1024;
  static_assert(kSmem <= 160 * 1024 && (NS - 1) * kLoads < 64 && BM / kRpb % kWaves == 0 && BN / kRpb % kWaves == 0, "tile");
};

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

struct Args {
  const uint8_t *A, *SA, *B, *SB;
  void* C;
  const int* offsets;  // null: dense (FP8)
  int64_t ldc;
  int groups, M, N, K, tiles_n;
};

template <int FMT, bool EXACT, int OUT, class G>
__global__ __launch_bounds__(G::kThreads) void gemm_block_kernel(Args p) {
  constexpr bool FP8 = G::kFp8;
  constexpr int kSeg = FP8 ? kChain : kChain / 2;  // steps of a chain
  __shared__ __attribute__((aligned(1024))) uint8_t smem[G::kSmem];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / G::WN, wn = wave % G::WN;
  const int r = lane & 15, g = lane >> 4;

  groups::Tile t;
  if (!groups::tile_of<G::BM>(p.offsets, p.groups, p.M, p.tiles_n, blockIdx.x, t)) return;
  const int n0 = t.tn * G::BN;
  const int mrows = min(t.rows, G::BM), nrows = min(p.N - n0, G::BN);
  const uint32_t rowbytes = (uint32_t)(FP8 ? p.K : p.K / 2);
  const int nk = (int)((rowbytes + kRow - 1) / kRow);
  const int kblocks = p.K / 32;                   // MXFP4: scales per row
  const int64_t brow = (int64_t)t.group * p.N + n0;  // row of B among all weights

  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.A + (int64_t)t.row * rowbytes), 0, (int)((uint32_t)mrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.B + brow * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);
  const uint32_t sstride = (uint32_t)(FP8 ? nk * 4 : kblocks);  // scale bytes per row of A
  const __amdgpu_buffer_rsrc_t rSA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.SA + (int64_t)t.row * sstride), 0, (int)((uint32_t)mrows * sstride), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rSB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.SB + (FP8 ? 0 : brow * sstride)), 0, FP8 ? 0 : (int)((uint32_t)nrows * sstride), kRsrcFlags);
  // FP8: the scales of this wave's 128 columns (its last tile past N: any).
  const int nb = min(n0 + wn * 16 * G::TNW, p.N - 1) / 128;
  const float* sb_row = (const float*)p.SB + ((int64_t)t.group * ((p.N + 127) / 128) + nb) * nk;

  // Loads of step s into its stage: A's and B's codes, 1 KB (kRpb rows) each, then
  // scales, 64 rows each. Steps past the last load nothing, but are counted.
  auto issue = [&](int s, uint8_t* stage) __attribute__((always_inline)) {
    constexpr int kA = G::BM / kRpb;
#pragma unroll
    for (int i = 0; i < G::kCodeLoads / G::kWaves; i++) {
      const bool isA = i * G::kWaves < kA;  // (of all waves)
      const int b = wave + i * G::kWaves;
      const int row = (isA ? b : b - kA) * kRpb + lane / kCpr;
      const uint32_t kb = (uint32_t)s * kRow + (uint32_t)((lane % kCpr) ^ swz(row)) * 16u;
      const uint32_t off = kb < rowbytes ? (uint32_t)row * rowbytes + kb : kOOB;
      if (isA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr_t)(stage + b * 1024), 16, off, 0, 0, 0);
      else if (G::kStreamB)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)(stage + b * 1024), 16, off, 0, 0, kNonTemporal);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)(stage + b * 1024), 16, off, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < G::kLoads - G::kCodeLoads / G::kWaves; i++) {
      const int q = wave + i * G::kWaves;
      const bool real = s < nk && q < G::kScaleLoads;
      uint8_t* dst = real ? stage + G::kOffS + q * 256 : smem + G::kDummy;
      if (FP8) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rSA, (lds_ptr_t)dst, 4, (uint32_t)(q * 64 + lane) * sstride,
                                                 real ? 4 * s : (int)kOOB, 0, 0);
      } else {
        const int grp = q % G::kScaleGroups, at = 8 * s + q / G::kScaleGroups * (G::kAligned ? 4 : 1);
        const bool isA = grp < G::kScaleA;
        const uint32_t off = (uint32_t)((isA ? grp : grp - G::kScaleA) * 64 + lane) * sstride;
        const int so = real && at < kblocks ? at : (int)kOOB;
        if (G::kAligned)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(isA ? rSA : rSB, (lds_ptr_t)dst, 4, off, so, 0, 0);
        else
          __builtin_amdgcn_raw_ptr_buffer_load_lds(isA ? rSA : rSB, (lds_ptr_t)dst, 1, off, so, 0, 0);
      }
    }
  };

  f32x4 acc[G::TMW][G::TNW], tot[OUT == kOutF32 ? G::TMW : 1][OUT == kOutF32 ? G::TNW : 1];
#pragma unroll
  for (int i = 0; i < G::TMW; i++)
#pragma unroll
    for (int j = 0; j < G::TNW; j++) {
      acc[i][j] = f32x4{0, 0, 0, 0};
      if (OUT == kOutF32) tot[i][j] = f32x4{0, 0, 0, 0};
    }

  // FP8: s_B of this wave's columns, 64 steps at a time, lane l's step s0 + l.
  float sbs = 0.0f;
#pragma unroll
  for (int d = 0; d < G::NS - 1; d++) issue(d, smem + d * G::kStage);
  int at = 0;  // step s's stage
  for (int s = 0; s < nk; s++) {
    if (FP8 && s % 64 == 0) sbs = s + lane < nk ? sb_row[s + lane] : 0.0f;
    // Step s has arrived (the later steps' loads may still be out), and every
    // wave is done with step s - 1, whose stage takes step s + NS - 1.
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"((G::NS - 2) * G::kLoads) : "memory");
    const uint8_t* cur = smem + at * G::kStage;
    issue(s + G::NS - 1, smem + (at == 0 ? G::NS - 1 : at - 1) * G::kStage);
    at = at == G::NS - 1 ? 0 : at + 1;
    const float sb = FP8 ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sbs), s & 63)) : 0.0f;
    if constexpr (FP8) {
      // A lane's 32 bytes of the step: chunks g and g + 4 of its row (any
      // order of K is right, if A's and B's are the same).
      auto frag = [&](const uint8_t* rows, int row) {
        const i32x4 lo = *(const i32x4*)(rows + row * 128 + ((g ^ swz(row)) * 16));
        const i32x4 hi = *(const i32x4*)(rows + row * 128 + (((g + 4) ^ swz(row)) * 16));
        return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      };
      i32x8 bf[G::TNW];
#pragma unroll
      for (int j = 0; j < G::TNW; j++) bf[j] = frag(cur + G::kOffB, wn * 16 * G::TNW + j * 16 + r);
      if constexpr (EXACT) {
        bf16x8 be[G::TNW][4];
#pragma unroll
        for (int j = 0; j < G::TNW; j++)
#pragma unroll
          for (int q = 0; q < 4; q++) be[j][q] = fp8::expand8(bf[j][2 * q], bf[j][2 * q + 1]);
#pragma unroll
        for (int i = 0; i < G::TMW; i++) {
          const int row = wm * 16 * G::TMW + i * 16 + r;
          const float f = *(const float*)(cur + G::kOffS + row * 4) * sb;
          const i32x8 af = frag(cur, row);
          bf16x8 ae[4];
#pragma unroll
          for (int q = 0; q < 4; q++) ae[q] = fp8::expand8(af[2 * q], af[2 * q + 1]);
#pragma unroll
          for (int j = 0; j < G::TNW; j++) {
            f32x4 P = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; q++) P = __builtin_amdgcn_mfma_f32_16x16x32_bf16(be[j][q], ae[q], P, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][j][e] = __builtin_fmaf(P[e], f, acc[i][j][e]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < G::TMW; i++) {
          const int row = wm * 16 * G::TMW + i * 16 + r;
          const float f = *(const float*)(cur + G::kOffS + row * 4) * sb;
          const i32x8 af = frag(cur, row);
          f32x4 P[G::TNW];
#pragma unroll
          for (int j = 0; j < G::TNW; j++)
            P[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af, f32x4{0, 0, 0, 0}, 0, 0, 0, 127, 0, 127);
#pragma unroll
          for (int j = 0; j < G::TNW; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][j][e] = __builtin_fmaf(P[j][e], f, acc[i][j][e]);
        }
      }
    } else {
      // Of 128 K h, lane (r, g) supplies block g of its row and that block's scale.
#pragma unroll
      for (int h = 0; h < 2; h++) {
        auto frag = [&](const uint8_t* rows, int row) {
          const i32x4 v = *(const i32x4*)(rows + row * 128 + (((4 * h + g) ^ swz(row)) * 16));
          return i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
        };
        auto scale = [&](int at) {  // at: row of A, or 64 kScaleA + row of B
          constexpr int kPart = 64 * G::kScaleGroups;
          return (int)cur[G::kOffS + (G::kAligned ? (h * kPart + at) * 4 + g : ((4 * h + g) * kPart + at) * 4)];
        };
        i32x8 bf[G::TNW];
        int sbb[G::TNW];
#pragma unroll
        for (int j = 0; j < G::TNW; j++) {
          const int row = wn * 16 * G::TNW + j * 16 + r;
          bf[j] = frag(cur + G::kOffB, row);
          sbb[j] = scale(64 * G::kScaleA + row);
        }
#pragma unroll
        for (int i = 0; i < G::TMW; i++) {
          const int row = wm * 16 * G::TMW + i * 16 + r;
          const i32x8 af = frag(cur, row);
          const int sa = scale(row);
#pragma unroll
          for (int j = 0; j < G::TNW; j++)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af, acc[i][j], 4, 4, 0, sbb[j], 0, sa);
        }
      }
    }
    if constexpr (OUT == kOutF32) {
      if ((s + 1) % kSeg == 0 && s + 1 < nk) {
#pragma unroll
        for (int i = 0; i < G::TMW; i++)
#pragma unroll
          for (int j = 0; j < G::TNW; j++) {
            tot[i][j] += acc[i][j];
            acc[i][j] = f32x4{0, 0, 0, 0};
          }
      }
    }
  }

  const bool vec_ok = p.ldc % 4 == 0;
#pragma unroll
  for (int i = 0; i < G::TMW; i++) {
    const int lrow = wm * 16 * G::TMW + i * 16 + r;
    if (lrow >= mrows) continue;
#pragma unroll
    for (int j = 0; j < G::TNW; j++) {
      const int col = n0 + wn * 16 * G::TNW + j * 16 + 4 * g;
      f32x4 v = acc[i][j];
      if (OUT == kOutF32) v = nk > kSeg ? v + tot[i][j] : v;
      const int64_t at = (int64_t)(t.row + lrow) * p.ldc + col;
      if (vec_ok && col + 4 <= p.N) {
        if (OUT == kOutF32)
          *(f32x4*)((float*)p.C + at) = v;
        else
          *(u32x2*)((uint16_t*)p.C + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (col + e < p.N) {
            if (OUT == kOutF32)
              ((float*)p.C)[at + e] = v[e];
            else
              ((uint16_t*)p.C)[at + e] = bf16_bits(v[e]);
          }
      }
    }
  }
}

// Experts that have rows, and rows each, as far as the host can know.
int64_t used(const Args& p) { return !p.offsets ? 1 : p.groups < p.M ? p.groups : p.M; }
int64_t rows_each(const Args& p) { return p.M / used(p); }

// Tiles to expect: an expert's last row tile half full.
int64_t tiles(const Args& p, int bm, int bn) {
  const int64_t tm = p.offsets ? (p.M + used(p) * (bm / 2)) / bm : (p.M + bm - 1) / bm;
  return tm * ((p.N + bn - 1) / bn);
}

template <int FMT, bool EXACT, int OUT, class G>
hipError_t launch(const Args& a, hipStream_t s) {
  Args p = a;
  p.tiles_n = (int)((p.N + G::BN - 1) / G::BN);
  const int64_t n = p.offsets ? groups::max_row_tiles(p.M, p.groups, G::BM) : (p.M + G::BM - 1) / G::BM;
  return launch_kernel(&gemm_block_kernel<FMT, EXACT, OUT, G>, dim3((unsigned)groups::grid_size(n, p.tiles_n)),
                       G::kThreads, 0, s, p);
}

// The tile. While tiles are fewer than CUs, smaller ones, spread over more CUs, are
// faster; with enough tiles larger ones are, which read less for their outputs.
// Three stages are enough, more only keep workgroups from sharing a CU (64 x 64, 4 waves, fp8
// 1500 x 2048 x 4096: 27.5 us with three, 30.8 with four, 43.8 with eight).
// Times in us of 32 / 64 / 64 x 128 / 128 tiles, M x N x K:
//   fp8, bf16 result: 32 x 14336 x 4096 12 / 15 / - / 28, 128 x 8192 x 4096 - / 13.8 / 17.8 / 25,
//   777 x 2048 x 4096 - / 19.0 / 17.7 / -, 1500 x 1000 x 2432 - / 12.8 / 11.8 / -,
//   128 x 28672 x 4096 - / 54 / 43 / 34, 800 rows over 8 x 2048 x 4096 - / 21 / 19.2 / 31;
//   1000 over 64 x 2048 x 4096 - / - / 123 / 133, 4000 163 / 165;
//   mxfp4: 1500 over 5 x 1000 x 2816 - / 12.6 / 9.7 / -, 800 over 8 x 2048 x 4096 - / 28 / 25.6 / 19.3,
//   1920 over 64 x 2048 x 4096 - / 108 / 94 / 76.
template <int FMT, bool EXACT, int OUT, bool ALIGNED>
hipError_t by_tile(const Args& p, hipStream_t s) {
  if ((p.offsets || p.M > 48) && tiles(p, 128, 128) >= (FMT == kMXFP4 ? 150 : 200)) {
    if constexpr (EXACT) {
      // Expanding codes is as much work as the MFMAs: 8 waves, so that a SIMD's
      // second wave does one beside the other (2000 x 2000 x 2432 34 us with 4
      // waves, 28 with 8), and, where rounds of CUs allow, 256 x 128 tiles, which expand less
      // (8192 cubed 1480 / 1255 / 1100; a tile of 256 x 128 takes 2.15 us a step, of
      // 128 x 128 1.25).
      auto rounds = [](int64_t n) { return (n + 255) / 256; };
      if (7 * rounds(tiles(p, 256, 128)) < 4 * rounds(tiles(p, 128, 128)))
        return launch<FMT, EXACT, OUT, Geo<FMT, 4, 4, 4, 2, 3, ALIGNED>>(p, s);
      return launch<FMT, EXACT, OUT, Geo<FMT, 4, 2, 2, 4, 3, ALIGNED>>(p, s);
    } else if constexpr (FMT == kMXFP4) {
      // Few rows an expert: weights from HBM, and two workgroups a CU are faster
      // (600 rows over 64 x 2048 x 4096: 63 us, 72 with three stages; 4000: 102 and 98).
      if (rows_each(p) <= 32) return launch<FMT, EXACT, OUT, Geo<FMT, 4, 4, 2, 2, 2, ALIGNED>>(p, s);
      return launch<FMT, EXACT, OUT, Geo<FMT, 4, 4, 2, 2, 3, ALIGNED>>(p, s);
    } else {
      if (!p.offsets) return launch<FMT, EXACT, OUT, Geo<FMT, 4, 4, 2, 2, 3, ALIGNED>>(p, s);
      // Few rows an expert: a weight is read once, so non-temporally (208 rows over
      // 16 x 4096 x 4096: 58 us, 90 without; 1000 over 64 x 2048 x 4096 109 and 118; 4000 166 and 157).
      if (rows_each(p) <= 32) return launch<FMT, EXACT, OUT, Geo<FMT, 2, 2, 2, 4, 3, ALIGNED, true>>(p, s);
      return launch<FMT, EXACT, OUT, Geo<FMT, 2, 2, 2, 4, 3, ALIGNED>>(p, s);
    }
  }
  if (tiles(p, 64, 64) >= (p.M > 32 ? 200 : 300)) {
    if constexpr (EXACT) {
      // (777 x 2000 x 2432: 17.9 us; 64 x 128 with 8 waves 18.3, 64 x 64 with 8 20.9.)
      return launch<FMT, EXACT, OUT, Geo<FMT, 2, 2, 2, 2, 3, ALIGNED>>(p, s);
    } else {
      // More than one tile of 64 x 64 a CU: 64 x 128. (Both of 8 waves: one
      // round, 777 x 1000 x 2432 fp8, 9.0 us, with 4 waves 9.7.)
      if (tiles(p, 64, 64) > 256) return launch<FMT, EXACT, OUT, Geo<FMT, 2, 2, 2, 4, 3, ALIGNED>>(p, s);
      return launch<FMT, EXACT, OUT, Geo<FMT, 2, 1, 2, 4, 3, ALIGNED>>(p, s);
    }
  }
  return launch<FMT, EXACT, OUT, Geo<FMT, 1, 1, 2, 2, 4, ALIGNED>>(p, s);
}

// Few rows of A: a stream of weights, which needs long rows of them. Times in us of that
// kernel / the tiles:
//   dense: 16 x 2048 x 2048 fp8 4.6 / 6.2, 16 x 4096 x 4096 7.4 / 10, 16 x 4096 x 1024
//   3.9 / 4.4, but 16 x 14336 x 1024 7.7 / 5.4;
//   by expert, rows over experts x N x K: fp8 704 over 64 x 2048 x 4096 107 / 116, 896 132 / 118;
//   80 over 16 x 2048 x 2048 14.2 / 14.5, 128 15.7 / 14.2; mxfp4 320 over 64 x 2048 x 4096 55 / 60,
//   512 64 / 61; fp8 32 over 64 x 2048 x 1024 13.5 / 10.9, mxfp4 14.7 / 8.3.
// The host does not know the rows' distribution, and an even one is the slowest for both. With all
// rows at one expert of 64 x 2048 x 4096 (each pass of 16 rows reads its weight): fp8 128 rows 12.8 / 17.6,
// 384 30 / 22, 768 57 / 23 (even 96 / 127); mxfp4 128 9.7 / 16.7, 320 18.2 / 16.9 (even 47 / 63).
bool few_rows(const Args& p, int fmt) {
  if (!p.offsets) return p.M <= 16 && (p.K >= 16 * 128 || p.N <= 8192);
  const int64_t steps = (fmt == kMXFP4 ? p.K / 2 : p.K) / 128;  // lines of a row
  return p.M <= (steps >= 32 ? 12 : steps >= 16 ? 6 : 0) * (int64_t)p.groups;
}

}  // namespace

// Whether the kernels' 32-bit offsets hold (256 rows of codes and of scales)
// and the grid its 2^32 threads: tiles of 128 x 128 or, by expert and for at most
// 48 rows, 64 x 128 of 512 (64 x 64 of 256 for fp32 results; smaller ones are for few).
bool gemm_block_fits(int64_t M, int64_t N, int64_t K, int64_t groups) {
  if (K > ((int64_t)1 << 22)) return false;
  const int64_t tm = groups > 0 ? groups::max_row_tiles(M, groups, 64) : (M + 127) / 128;
  return groups::grid_size(tm, (N + 127) / 128) < ((int64_t)1 << 23);
}

hipError_t gemm_block(int fmt, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                      const void* b, const void* sb, const int32_t* offsets, int64_t groups,
                      int out_dtype, void* c, int64_t ldc, hipStream_t s) {
  const Args p{(const uint8_t*)a, (const uint8_t*)sa, (const uint8_t*)b, (const uint8_t*)sb, c, offsets,
               ldc, (int)groups, (int)M, (int)N, (int)K, 0};
  const bool f32 = out_dtype == kOutF32;
  if (few_rows(p, fmt) && gemm_few_rows_fits(M, N, K, offsets ? groups : 0, out_dtype))
    return gemm_few_rows(fmt, M, N, K, a, sa, b, sb, offsets, groups, out_dtype, c, ldc, s);
  // Tiles of 256 x 256, for a third of the CUs or more, where most are more than half full.
  // (Times of 256 / the best of the smaller tiles: fp8 1500 x 8192 x 4096 (192 tiles)
  // 50 / 83, 777 x 8192 x 4096 (128) 44 / 55, 256 x 28672 x 4096 (112) 61 / 59, 1500 x 4096 x
  // 4096 (96) 44 / 55, 300 x 8192 x 4096 (64) 43 / 26, 128 x 28672 x 4096 (112, half full) 54 / 34;
  // fp8 1600 rows over 16 x 2048 x 2048 (112) 25 / 27, 2000 over 8 x 2048 x 4096 (88) 45 / 42;
  // mxfp4 2400 over 16 x 2048 x 2048 (136) 18 / 23, 2000 over 8 x 2048 x 4096 (88) 28 / 34,
  // 800 over 8 (56) 28 / 19.)
  const bool large = rows_each(p) > (offsets ? 64 : 128) && tiles(p, 256, 256) >= (fmt == kMXFP4 ? 80 : 90);
  if (fmt == kMXFP4) {
    if (large && gemm_mxfp4_fits(0, N, K))
      return gemm_mxfp4_grouped(M, N, K, a, sa, b, sb, offsets, groups, out_dtype, c, ldc, s);
    if (K % 128 != 0)
      return f32 ? by_tile<kMXFP4, false, kOutF32, false>(p, s) : by_tile<kMXFP4, false, kOutBF16, false>(p, s);
    return f32 ? by_tile<kMXFP4, false, kOutF32, true>(p, s) : by_tile<kMXFP4, false, kOutBF16, true>(p, s);
  }
  if (f32) return by_tile<kFP8B128, true, kOutF32, true>(p, s);
  if (large) return gemm_fp8_large(M, N, K, a, sa, b, sb, offsets, groups, c, ldc, s);
  return by_tile<kFP8B128, false, kOutBF16, true>(p, s);
}

}  // namespace mx
