// GEMM of 8-bit integers under a scale per row of A and of B, dense or by expert
// (groups.h):
//   C[i][j] = s_A[i] s_B[j] sum over k of A[i][k] B[j][k],
// the sum exact in int32 (|code| <= 128 and K < 2^17), the scales applied to it
// once (int8.h). This file: the choice of kernel, and tiles of 32 x 32 to 128 x 128 on
// 16 x 16 x 64 matrix instructions. (256 x 256: gemm_int8_large.hip; few rows of A:
// gemm_few_rows.hip.)
//
// A K step is kRow = 64 WK KPW bytes of each row, a whole line. Operands go HBM -> LDS directly
// (buffer_load ... lds) into a ring of NS stages, a step each, NS - 2 of them in flight beside the
// one that is read. The buffer view of a tile ends with the group's rows, so rows past the end load as
// zeros, and so do the 16-byte chunks past a row's end in its last step. The chunk c
// of LDS row r sits in slot c ^ swz(r), so that the 16 lanes that read one column of
// chunks hit distinct banks.
//
// A step's fragments are read from LDS beside the products of the step before (1500 x 2048 x 4096 24.0 -> 22.8
// us, 64 x 2048 x 4096 7.5 -> 6.7). 128 x 128 tiles have 8 waves of 64 x 64: WK = 2 groups of WM x WN waves, which
// take half of each step's K each, so that a fragment is read as often as by 4 waves; their sums,
// exact integers, meet in LDS at the end. What bounds the small tiles: the rate of loads into LDS, about
// 75 KB/us a CU where rows begin on lines and 48 where they do not (120 and 70 alone; 777 x 2000 fp32 results of
// K = 2448 14.7 us, of 2432 11.9), the first loads, and the chain of loads and stores at the end (below).
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

// Tile geometry: waves of 16 TMW x 16 TNW, WM x WN of them in each of WK groups, which
// take KPW matrix instructions' K of a step; NS stages.
template <int TMW_, int TNW_, int WM_, int WN_, int WK_, int KPW_, int NS_>
struct Geo {
  static constexpr int TMW = TMW_, TNW = TNW_, WM = WM_, WN = WN_, WK = WK_, KPW = KPW_, NS = NS_;
  static constexpr int BM = 16 * TMW * WM, BN = 16 * TNW * WN;
  static constexpr int kWaves = WM * WN * WK, kThreads = 64 * kWaves;
  static constexpr int kRow = 64 * WK * KPW, kCpr = kRow / 16;  // LDS bytes and chunks of a row's K step
  static constexpr int kRpb = 64 / kCpr;                        // rows per 1 KB load of a wave
  static constexpr int kOffB = BM * kRow, kStage = kOffB + BN * kRow;
  static constexpr int kLoads = (BM + BN) / kRpb / kWaves;  // of a wave and step
  static constexpr int kReads = KPW * (TMW + TNW);          // LDS reads of its fragments
  static_assert(kReads <= 15, "a wait's count");
  static constexpr int kSums = WK > 1 ? kWaves * TMW * TNW * 1024 : 0;
  static constexpr int kSmem = NS * kStage > kSums ? NS * kStage : kSums;
  static_assert(kRow >= 128 && kRow <= 1024 && kSmem <= 160 * 1024 && (NS - 1) * kLoads < 64 && NS >= 3, "step");
  static_assert(BM / kRpb % kWaves == 0 && BN / kRpb % kWaves == 0 && TMW * TNW % WK == 0, "tile");
  // (Rows of 128 bytes: two of them lie in one turn of the banks.)
  static __device__ __forceinline__ int swz(int row) { return kRow == 128 ? (row >> 1) & 7 : row & 7; }
};

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
  constexpr int kRow = G::kRow;
  const int wk = wave / (G::WM * G::WN), wm = wave / G::WN % G::WM, wn = wave % G::WN;
  const int r = lane & 15, g = lane >> 4;

  groups::Tile t;
  if (!groups::tile_of<G::BM>(p.offsets, p.groups, p.M, p.tiles_n, blockIdx.x, t)) return;
  const int n0 = t.tn * G::BN;
  const int mrows = min(t.rows, G::BM), nrows = min(p.N - n0, G::BN);
  const uint32_t rowbytes = (uint32_t)p.K;
  const int nk = (p.K + kRow - 1) / kRow;  // (kRow: a power of two)
  const int64_t brow = (int64_t)t.group * p.N + n0;  // row of B among all weights
  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.A + (int64_t)t.row * rowbytes), 0, (int)((uint32_t)mrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.B + brow * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);

  // Loads of step s into its stage: A's and B's codes, 1 KB each. Steps
  // past the last load nothing, but are counted.
  auto issue = [&](int s, uint8_t* stage) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < G::kLoads; i++) {
      constexpr int kA = G::BM / G::kRpb;
      const bool isA = i * G::kWaves < kA;  // (of all waves)
      const int b = wave + i * G::kWaves;
      const int row = (isA ? b : b - kA) * G::kRpb + lane / G::kCpr;
      const uint32_t kb = (uint32_t)s * kRow + (uint32_t)((lane % G::kCpr) ^ G::swz(row)) * 16u;
      const uint32_t off = kb < rowbytes ? (uint32_t)row * rowbytes + kb : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(isA ? rA : rB, (lds_ptr_t)(stage + b * 1024), 16, off, 0, 0, 0);
    }
  };

  i32x4 acc[G::TMW][G::TNW];
#pragma unroll
  for (int i = 0; i < G::TMW; i++)
#pragma unroll
    for (int j = 0; j < G::TNW; j++) acc[i][j] = i32x4{0, 0, 0, 0};

  // Fragments of a step: this group's part of its K.
  struct Frags {
    i32x4 a[G::KPW][G::TMW], b[G::KPW][G::TNW];
  };
  auto read = [&](const uint8_t* stage, Frags& f) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < G::KPW; h++) {
      auto frag = [&](const uint8_t* rows, int row) __attribute__((always_inline)) {
        return *(const i32x4*)(rows + row * kRow + (((4 * (wk * G::KPW + h) + g) ^ G::swz(row)) * 16));
      };
#pragma unroll
      for (int j = 0; j < G::TNW; j++) f.b[h][j] = frag(stage + G::kOffB, wn * 16 * G::TNW + j * 16 + r);
#pragma unroll
      for (int i = 0; i < G::TMW; i++) f.a[h][i] = frag(stage, wm * 16 * G::TMW + i * 16 + r);
    }
  };
  auto multiply = [&](const Frags& f) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < G::KPW; h++)
#pragma unroll
      for (int i = 0; i < G::TMW; i++)
#pragma unroll
        for (int j = 0; j < G::TNW; j++) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[h][j], f.a[h][i], acc[i][j], 0, 0, 0);
  };
#pragma unroll
  for (int d = 0; d < G::NS - 1; d++) issue(d, smem + d * G::kStage);
  Frags f[2];
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"i"((G::NS - 2) * G::kLoads) : "memory");
  read(smem, f[0]);
  int at = 0;  // step s's stage
  // Step s's products, beside the reads of step s + 1's fragments.
  auto step = [&](int s, const Frags& cur, Frags& nxt) __attribute__((always_inline)) {
    // Step s + 1 has arrived (the later steps' loads may still be out), and every wave
    // has the fragments of step s - 1 (those of step s may still be out), whose stage takes step s + NS - 1.
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(%1)\n\ts_barrier" ::"i"((G::NS - 3) * G::kLoads), "i"(G::kReads) : "memory");
    issue(s + G::NS - 1, smem + (at == 0 ? G::NS - 1 : at - 1) * G::kStage);
    at = at == G::NS - 1 ? 0 : at + 1;
    read(smem + at * G::kStage, nxt);
    multiply(cur);
  };
  int s = 0;
  for (; s + 1 < nk; s += 2) {
    step(s, f[0], f[1]);
    step(s + 1, f[1], f[0]);
  }
  if (s < nk) multiply(f[0]);
  // (The loads of steps past the last have nowhere to go, but count as out until here.)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if constexpr (G::WK > 1) {
    // The groups' sums: of a wave's tiles each group adds up every WK-th.
    i32x4(*sums)[G::TMW * G::TNW][64] = (i32x4(*)[G::TMW * G::TNW][64])smem;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int q = 0; q < G::TMW * G::TNW; q++) sums[wave][q][lane] = acc[q / G::TNW][q % G::TNW];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int q = 0; q < G::TMW * G::TNW; q += G::WK) {
      i32x4 v = sums[wave % (G::WM * G::WN)][q + wk][lane];
#pragma unroll
      for (int k = 1; k < G::WK; k++) v += sums[wave % (G::WM * G::WN) + k * G::WM * G::WN][q + wk][lane];
      acc[q / G::TNW][q % G::TNW] = v;
    }
  }

  const bool vec_ok = p.ldc % 4 == 0;
#pragma unroll
  for (int q = 0; q < G::TMW * G::TNW; q += G::WK) {
    // (Column by column of tiles where one wave has them all. The compiler loads each tile's five scales anew, and
    // waits for them and for the store before: a chain of such round trips ends the kernel.)
    const int at = G::WK > 1 ? q : q % G::TMW * G::TNW + q / G::TMW, tile = at + (G::WK > 1 ? wk : 0);
    const int col = n0 + (wn * G::TNW + tile % G::TNW) * 16 + 4 * g, lrow = (wm * G::TMW + tile / G::TNW) * 16 + r;
    if (lrow >= mrows) continue;
    const int8::Scale sa = int8::split(p.SA[t.row + lrow]);
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; e++)
      v[e] = int8::apply(acc[at / G::TNW][at % G::TNW][e], sa, int8::split(col + e < p.N ? p.SB[(int64_t)t.group * p.N + col + e] : 0.0f));
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

// Experts that have rows, and rows each, as far as the host can know.
int64_t used(const Args& p) { return !p.offsets ? 1 : p.groups < p.M ? p.groups : p.M; }

int64_t rows_each(const Args& p) { return p.M / used(p); }

// Tiles to expect: an expert's last row tile half full.
int64_t tiles(const Args& p, int bm, int bn) {
  const int64_t tm = p.offsets ? (p.M + used(p) * (bm / 2)) / bm : (p.M + bm - 1) / bm;
  return tm * ((p.N + bn - 1) / bn);
}

template <class G>
int64_t workgroups(const Args& p) {
  const int64_t n = p.offsets ? groups::max_row_tiles(p.M, p.groups, G::BM) : (p.M + G::BM - 1) / G::BM;
  return groups::grid_size(n, (p.N + G::BN - 1) / G::BN);
}

// Whether a grid's 2^32 threads are enough. (gemm_block_fits: those of 64 x 128 by expert and 128 x 128 are.)
template <class G>
bool fits(const Args& p) {
  return workgroups<G>(p) * G::kThreads < (int64_t)1 << 32;
}

template <int OUT, class G>
hipError_t launch(const Args& a, hipStream_t s) {
  Args p = a;
  p.tiles_n = (int)((p.N + G::BN - 1) / G::BN);
  return launch_kernel(&gemm_int8_kernel<OUT, G>, dim3((unsigned)workgroups<G>(p)), G::kThreads, 0, s, p);
}

// The tile: 32 x 32, 64 x 64, 64 x 128 or 128 x 128 (the last in 8 waves that divide K: 36 us, 39
// with 4 waves, at 128 x 28672 x 4096). While tiles are fewer than CUs, smaller ones, spread over more
// CUs, are faster; with enough tiles larger ones are, which read less for their outputs. Stages: as
// many as leave a CU the workgroups that there are. Times in us of 32 / 64 / 64 x 128 / 128 tiles:
//   M x N x K: 64 x 2048 x 4096 6.7 / 10.7 / - / -, 48 x 8192 x 8192 14.7 / 18.1 / - / -, 32 x 14336 x 4096
//   11.7 / 12.4 / - / -, 500 x 500 x 8000 10.8 / 18.4 / - / -, 300 x 2048 x 4096 12.0 / 11.9 / - / -, 128 x
//   8192 x 4096 15.7 / 12.6 / 15.3 / -, 1000 x 1000 x 16000 47 / 32 / 38 / 54, 777 x 2000 x 2448 (fp32 result)
//   - / 15.4 / 14.2 / -, 1500 x 1000 x 2432 - / 11.2 / 11.0 / -, 1500 x 2048 x 4096 - / 23.7 / 25.4 / 22.8,
//   2000 x 2000 x 2432 (fp32) - / 20.7 / 19.2 / 19.1, 1000 x 4096 x 1024 - / 14.2 / 13.0 / 13.8;
//   rows over experts x N x K: 800 over 64 x 2048 x 4096 101 / 137 / 139 / 135, 1500 122 / 135 / 142 / 145,
//   300 over 32 x 1024 x 2048 14.8 / 13.5 / 14.3 / 15.7, 400 over 16 x 2048 x 2048 16.2 / 14.5 / 15.8 / 16, 800
//   over 8 x 2048 x 4096 - / 22.5 / 24.9 / 23.4, 1600 over 16 x 2048 x 2048 - / 25.5 / 29.8 / 30.2, 1500 over
//   5 x 1000 x 2880 (fp32) - / 16.5 / 15.3 / 17.8, 3000 over 8 x 1024 x 1024 - / 14.3 / 12.8 / 14.3.
template <int OUT>
hipError_t by_tile(const Args& p, hipStream_t s) {
  const int64_t t64 = tiles(p, 64, 64);
  using Tile32 = Geo<1, 1, 2, 2, 1, 2, 6>;
  using Tile64 = Geo<2, 1, 2, 4, 1, 2, 3>;
  using Tile64x128 = Geo<2, 2, 2, 4, 1, 2, 3>;
  if ((p.M <= 32 || t64 < 150 || (p.offsets && rows_each(p) <= 24)) && fits<Tile32>(p)) return launch<OUT, Tile32>(p, s);
  if (t64 <= 256) return launch<OUT, Geo<2, 1, 2, 4, 1, 2, 4>>(p, s);
  if (tiles(p, 64, 128) <= 256) return launch<OUT, Geo<2, 2, 2, 4, 1, 2, 4>>(p, s);
  if (p.offsets && p.K > 1024 && fits<Tile64>(p)) return launch<OUT, Tile64>(p, s);
  if (p.offsets || (p.K <= 1024 && fits<Tile64x128>(p))) return launch<OUT, Tile64x128>(p, s);
  return launch<OUT, Geo<4, 4, 2, 2, 2, 1, 4>>(p, s);
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
  // Tiles of 256 x 256, for 100 of the CUs or (by expert) 140 or more, where most are more than half
  // full or experts' weights, read once so, are the bound. (Times of 256 / the best of the smaller tiles:
  // 1500 x 8192 x 4096 (192 tiles) 48 / 67, 777 x 8192 x 4096 (128) 45 / 44, 2000 x 4096 x 4096 (128)
  // 44.7 / 45.2, 256 x 28672 x 4096 (112) 57 / 59, 1500 x 4096 x 4096 (96) 44.5 / 42.2; 2000 rows over 64 x
  // 2048 x 4096 (312) 132 / 139, 1500 (296) 131 / 122, 600 over 16 x 4096 x 4096 (160) 69 / 73, 2000 over 16 x
  // 2048 x 2048 (120) 28.5 / 26.9, 2000 over 8 x 2048 x 4096 (88) 45 / 40.)
  if (rows_each(p) > (offsets ? 24 : 128) && tiles(p, 256, 256) >= (offsets ? 140 : 100))
    return gemm_int8_large(M, N, K, a, sa, b, sb, offsets, groups, out_dtype, c, ldc, s);
  return out_dtype == kOutF32 ? by_tile<kOutF32>(p, s) : by_tile<kOutBF16>(p, s);
}

}  // namespace mx
