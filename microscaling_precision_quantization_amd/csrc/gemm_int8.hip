// GEMM of 8-bit integers under a scale per row of A and of B, dense or by expert
// (groups.h):
//   C[i][j] = s_A[i] s_B[j] sum over k of A[i][k] B[j][k],
// the sum exact in int32 (|code| <= 128 and K < 2^17), the scales applied to it
// once (int8.h). This file: the choice of kernel, and tiles of 32 x 32 to 128 x 128 on
// 16 x 16 x 64 matrix instructions. (256 x 256: gemm_int8_large.hip; few rows of A:
// gemm_few_rows.hip.)
//
// A K step is 128 bytes of each row, a whole line. Operands go HBM -> LDS directly
// (buffer_load ... lds) into a ring of NS stages, a step each, NS - 1 of them in
// flight: with few tiles the loads' latency is what a step takes. The buffer view
// of a tile ends with the group's rows, so rows past the end load as zeros, and so do
// the 16-byte chunks past a row's end in its last step. The chunk c of LDS row
// r sits in slot c ^ swz(r), so that the 16 lanes that read one column of chunks
// hit distinct banks.
//
// B goes first into the MFMA: lane r + 16 g then holds C[row r][columns 4 g ..
// 4 g + 3] of a tile, one row (one s_A) and a run of columns to store.
#include "bf16.h"
#include "groups.h"
#include "int8.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
constexpr uint32_t kOOB = 0x80000000u;        // an offset past every buffer's range
constexpr int kRow = 128, kCpr = kRow / 16;   // LDS bytes and chunks of a row's K step
constexpr int kRpb = 64 / kCpr;               // rows per 1 KB load of a wave

// Tile geometry: waves of 16 TMW x 16 TNW, WM x WN of them; NS stages.
template <int TMW_, int TNW_, int WM_, int WN_, int NS_>
struct Geo {
  static constexpr int TMW = TMW_, TNW = TNW_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int BM = 16 * TMW * WM, BN = 16 * TNW * WN;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kOffB = BM * kRow, kStage = kOffB + BN * kRow;
  static constexpr int kLoads = (BM + BN) / kRpb / kWaves;  // of a wave and step
  static constexpr int kSmem = NS * kStage;
  static_assert(kSmem <= 160 * 1024 && (NS - 1) * kLoads < 64 && BM / kRpb % kWaves == 0 && BN / kRpb % kWaves == 0, "tile");
};

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

struct Args {
  const uint8_t *A, *B;
  const float *SA, *SB;
  void* C;
  const int* offsets;  // null: dense
  int64_t ldc;
  int groups, M, N, K, tiles_n;
};

template <int OUT, class G>
__global__ __launch_bounds__(G::kThreads) void gemm_int8_kernel(Args p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[G::kSmem];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / G::WN, wn = wave % G::WN;
  const int r = lane & 15, g = lane >> 4;

  groups::Tile t;
  if (!groups::tile_of<G::BM>(p.offsets, p.groups, p.M, p.tiles_n, blockIdx.x, t)) return;
  const int n0 = t.tn * G::BN;
  const int mrows = min(t.rows, G::BM), nrows = min(p.N - n0, G::BN);
  const uint32_t rowbytes = (uint32_t)p.K;
  const int nk = (p.K + kRow - 1) / kRow;
  const int64_t brow = (int64_t)t.group * p.N + n0;  // row of B among all weights
  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.A + (int64_t)t.row * rowbytes), 0, (int)((uint32_t)mrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.B + brow * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);

  // Loads of step s into its stage: A's and B's codes, 1 KB (kRpb rows) each. Steps
  // past the last load nothing, but are counted.
  auto issue = [&](int s, uint8_t* stage) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < G::kLoads; i++) {
      constexpr int kA = G::BM / kRpb;
      const bool isA = i * G::kWaves < kA;  // (of all waves)
      const int b = wave + i * G::kWaves;
      const int row = (isA ? b : b - kA) * kRpb + lane / kCpr;
      const uint32_t kb = (uint32_t)s * kRow + (uint32_t)((lane % kCpr) ^ swz(row)) * 16u;
      const uint32_t off = kb < rowbytes ? (uint32_t)row * rowbytes + kb : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(isA ? rA : rB, (lds_ptr_t)(stage + b * 1024), 16, off, 0, 0, 0);
    }
  };

  i32x4 acc[G::TMW][G::TNW];
#pragma unroll
  for (int i = 0; i < G::TMW; i++)
#pragma unroll
    for (int j = 0; j < G::TNW; j++) acc[i][j] = i32x4{0, 0, 0, 0};

#pragma unroll
  for (int d = 0; d < G::NS - 1; d++) issue(d, smem + d * G::kStage);
  int at = 0;  // step s's stage
  for (int s = 0; s < nk; s++) {
    // Step s has arrived (the later steps' loads may still be out), and every
    // wave is done with step s - 1, whose stage takes step s + NS - 1.
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"((G::NS - 2) * G::kLoads) : "memory");
    const uint8_t* cur = smem + at * G::kStage;
    issue(s + G::NS - 1, smem + (at == 0 ? G::NS - 1 : at - 1) * G::kStage);
    at = at == G::NS - 1 ? 0 : at + 1;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      auto frag = [&](const uint8_t* rows, int row) __attribute__((always_inline)) {
        return *(const i32x4*)(rows + row * kRow + (((4 * h + g) ^ swz(row)) * 16));
      };
      i32x4 bf[G::TNW];
#pragma unroll
      for (int j = 0; j < G::TNW; j++) bf[j] = frag(cur + G::kOffB, wn * 16 * G::TNW + j * 16 + r);
#pragma unroll
      for (int i = 0; i < G::TMW; i++) {
        const i32x4 af = frag(cur, wm * 16 * G::TMW + i * 16 + r);
#pragma unroll
        for (int j = 0; j < G::TNW; j++) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[j], af, acc[i][j], 0, 0, 0);
      }
    }
  }
  // (The loads of steps past the last have nowhere to go, but count as out until here.)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  const bool vec_ok = p.ldc % 4 == 0;
#pragma unroll
  for (int j = 0; j < G::TNW; j++) {
    const int col = n0 + wn * 16 * G::TNW + j * 16 + 4 * g;
    int8::Scale sb[4];
#pragma unroll
    for (int e = 0; e < 4; e++) sb[e] = int8::split(col + e < p.N ? p.SB[(int64_t)t.group * p.N + col + e] : 0.0f);
#pragma unroll
    for (int i = 0; i < G::TMW; i++) {
      const int lrow = wm * 16 * G::TMW + i * 16 + r;
      if (lrow >= mrows) continue;
      const int8::Scale sa = int8::split(p.SA[t.row + lrow]);
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = int8::apply(acc[i][j][e], sa, sb[e]);
      const int64_t at_c = (int64_t)(t.row + lrow) * p.ldc + col;
      if (vec_ok && col + 4 <= p.N) {
        if (OUT == kOutF32)
          *(f32x4*)((float*)p.C + at_c) = v;
        else
          *(u32x2*)((uint16_t*)p.C + at_c) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (col + e < p.N) {
            if (OUT == kOutF32)
              ((float*)p.C)[at_c + e] = v[e];
            else
              ((uint16_t*)p.C)[at_c + e] = bf16_bits(v[e]);
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

template <int OUT, class G>
hipError_t launch(const Args& a, hipStream_t s) {
  Args p = a;
  p.tiles_n = (int)((p.N + G::BN - 1) / G::BN);
  const int64_t n = p.offsets ? groups::max_row_tiles(p.M, p.groups, G::BM) : (p.M + G::BM - 1) / G::BM;
  return launch_kernel(&gemm_int8_kernel<OUT, G>, dim3((unsigned)groups::grid_size(n, p.tiles_n)), G::kThreads, 0, s, p);
}

// The tile. While tiles are fewer than CUs, smaller ones, spread over more CUs, are
// faster; with enough tiles larger ones are, which read less for their outputs.
template <int OUT>
hipError_t by_tile(const Args& p, hipStream_t s) {
  if ((p.offsets || p.M > 48) && tiles(p, 128, 128) >= 200) return launch<OUT, Geo<4, 4, 2, 2, 3>>(p, s);
  if (tiles(p, 64, 64) >= (p.M > 32 ? 200 : 300)) {
    if (tiles(p, 64, 64) > 256) return launch<OUT, Geo<2, 2, 2, 4, 3>>(p, s);
    return launch<OUT, Geo<2, 1, 2, 4, 3>>(p, s);
  }
  return launch<OUT, Geo<1, 1, 2, 2, 4>>(p, s);
}

// Few rows of A: a stream of weights, which needs long rows of them.
bool few_rows(const Args& p) {
  if (!p.offsets) return p.M <= 16 && (p.K >= 16 * 128 || p.N <= 8192);
  return p.M <= (p.K >= 32 * 128 ? 12 : p.K >= 16 * 128 ? 6 : 0) * (int64_t)p.groups;
}

}  // namespace

hipError_t gemm_int8(int64_t M, int64_t N, int64_t K, const void* a, const void* sa, const void* b, const void* sb,
                     const int32_t* offsets, int64_t groups, int out_dtype, void* c, int64_t ldc, hipStream_t s) {
  const Args p{(const uint8_t*)a, (const uint8_t*)b, (const float*)sa, (const float*)sb, c, offsets,
               ldc, (int)groups, (int)M, (int)N, (int)K, 0};
  if (few_rows(p) && gemm_few_rows_fits(kINT8, M, N, K, offsets ? groups : 0, out_dtype))
    return gemm_few_rows(kINT8, M, N, K, a, sa, b, sb, offsets, groups, out_dtype, c, ldc, s);
  // Tiles of 256 x 256, for a third of the CUs or more, where most are more than half full.
  if (rows_each(p) > (offsets ? 64 : 128) && tiles(p, 256, 256) >= 90)
    return gemm_int8_large(M, N, K, a, sa, b, sb, offsets, groups, out_dtype, c, ldc, s);
  return out_dtype == kOutF32 ? by_tile<kOutF32>(p, s) : by_tile<kOutBF16>(p, s);
}

}  // namespace mx
