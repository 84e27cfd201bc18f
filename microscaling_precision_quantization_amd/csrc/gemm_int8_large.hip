// GEMM of 8-bit integers under a scale per row of A and of B, the large-tile kernel
// (dense or by expert; the mathematics is gemm_int8.hip's).
//
// Bound by the matrix cores: a K step of 128 takes a 256 x 256 tile's SIMDs 2048
// cycles of MFMA each, against 1536 of LDS reads and 512 of writes. Measured, 6000 x 8192 x 8192
// (bf16 result): 300 us, 2.7 POPS, the MFMAs 64% busy at the 1.95 GHz that the clock falls to; a step 1.3 us (1.07 us at
// 2.3 GHz without its loads), first loads and epilogue, with its waits for scales, 10 us a round of tiles. 32 x 32 x 32 MFMAs: 310 us; 4 waves
// of 128 x 128, which read a third less LDS but leave a SIMD one wave: 310 to 325.
//  * 8 waves (two per SIMD) of 128 x 64. A wave's step is 8 groups of eight 16 x 16 x 64
//    MFMAs, one group per 16 rows; the tile's 16-row groups go to the two rows of
//    waves in turn, so that a partly filled tile (the last one of an expert) of at
//    most 128 or 64 rows is done in 4 or 2 groups a step. A group's A fragment is read
//    two groups ahead.
//  * The last group of a step is issued after the barrier, beside the next
//    step's first fragment reads: it is their latency's cover. Each B fragment
//    is overwritten right after that group's last MFMA on it.
//  * Operands go HBM -> LDS directly, into double buffers, a step ahead. By
//    expert, weights come from HBM, whose latency is about a step: there every
//    wave has read its B fragments early in a step, and after one more barrier
//    B's buffer takes B of two steps ahead. The chunk swizzle, the buffer views that end
//    with the group's rows and the operand order are gemm_int8.hip's.
#include <type_traits>

#include "bf16.h"
#include "groups.h"
#include "int8.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
constexpr uint32_t kOOB = 0x80000000u;        // an offset past every buffer's range
constexpr int BM = 256, BN = 256, kWN = 4, kThreads = 512;
constexpr int kOffB = BM * 128, kStage = kOffB + BN * 128, kSmem = 2 * kStage;  // a stage: A's and B's codes

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

struct Args {
  const uint8_t *A, *B;
  const float *SA, *SB;
  void* C;
  const int* offsets;  // null: dense
  int64_t ldc;
  int groups, M, N, K, tiles_n;
};

struct Frag {
  i32x4 h[2];  // chunks g and g + 4 of a row's step
};

// GROUPED: p.offsets given.
template <int OUT, bool GROUPED>
__global__ __launch_bounds__(kThreads, 1) void gemm_int8_large_kernel(Args p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kSmem];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWN, wn = wave % kWN;
  const int r = lane & 15, g = lane >> 4;

  groups::Tile t;
  if (!groups::tile_of<BM>(GROUPED ? p.offsets : nullptr, p.groups, p.M, p.tiles_n, blockIdx.x, t)) return;
  const int n0 = t.tn * BN;
  const int mrows = min(t.rows, BM), nrows = min(p.N - n0, BN);
  const uint32_t rowbytes = (uint32_t)p.K;
  const int nk = (p.K + 127) / 128;
  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.A + (int64_t)t.row * rowbytes), 0, (int)((uint32_t)mrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.B + ((int64_t)t.group * p.N + n0) * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);

  // Lane parts of the load addresses: a load covers 8 rows of 128 bytes, lane
  // l slot l % 8 of row l / 8, which holds chunk slot ^ swz(row); swz(row)
  // depends on the parity of the load's block of 8 rows. In a row's last step, chunks
  // past its end are left out.
  const uint32_t left = rowbytes - 128u * (uint32_t)(nk - 1);
  uint32_t loff[2], loff_last[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const uint32_t chunk = (uint32_t)(((lane & 7) ^ swz(8 * h + (lane >> 3))) * 16);
    loff[h] = (uint32_t)(lane >> 3) * rowbytes + chunk;
    loff_last[h] = chunk < left ? loff[h] : kOOB;
  }
  // Loads P = 0..3 of A's and of B's 8-row blocks 4 wave + P. The row and step
  // go into the scalar offset, which the range check counts too.
  const uint32_t rows8 = 8 * rowbytes;
  auto load_a = [&](int s, uint8_t* stage, int P) __attribute__((always_inline)) {
    const int b = wave * 4 + P;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr_t)(stage + b * 1024), 16, s < nk - 1 ? loff[P & 1] : loff_last[P & 1],
                                             (int)((uint32_t)b * rows8) + s * 128, 0, 0);
  };
  auto load_b = [&](int s, uint8_t* stage, int P) __attribute__((always_inline)) {
    const int b = wave * 4 + P;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)(stage + kOffB + b * 1024), 16, s < nk - 1 ? loff[P & 1] : loff_last[P & 1],
                                             (int)((uint32_t)b * rows8) + s * 128, 0, 0);
  };

  i32x4 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = i32x4{0, 0, 0, 0};

  // Fragment addresses: chunks g and g + 4 of row r of a 16-row tile; swz(r)
  // is the same in every tile. The wave's group i is rows 32 i + 16 wm + r.
  const int c0 = (g ^ swz(r)) * 16, c1 = ((g + 4) ^ swz(r)) * 16;
  const int arow = (wm * 16 + r) * 128, brow = kOffB + (wn * 64 + r) * 128;
  auto frag = [&](const uint8_t* row) __attribute__((always_inline)) {
    return Frag{{*(const i32x4*)(row + c0), *(const i32x4*)(row + c1)}};
  };

  Frag bf[4], a[3];
#pragma unroll
  for (int j = 0; j < 4; j++) bf[j] = Frag{{i32x4{0, 0, 0, 0}, i32x4{0, 0, 0, 0}}};
  auto mfma = [&](const i32x4& bv, const i32x4& av, i32x4& c) __attribute__((always_inline)) {
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv, av, c, 0, 0, 0);
  };

#pragma unroll
  for (int q = 0; q < 4; q++) {
    load_a(0, smem, q);
    load_b(0, smem, q);
  }
  if (GROUPED) {
    fence();
#pragma unroll
    for (int q = 0; q < 4; q++) load_b(min(1, nk - 1), smem + kStage, q);
    fence();
  }
  // All steps, with NI groups a step. On entry of a step `last` is the last group of
  // the step before (its MFMAs still to do, on bf; before the first step
  // zeros). The source is in issue order: a fence after each MFMA and what runs beside it.
  auto run = [&](auto ni) __attribute__((always_inline)) {
    constexpr int NI = decltype(ni)::value;
    constexpr int kLast = (NI - 1) % 3;  // where a step leaves its last fragment
    Frag last = Frag{{i32x4{0, 0, 0, 0}, i32x4{0, 0, 0, 0}}};
    auto step = [&](int s, uint8_t* cur, uint8_t* nxt) __attribute__((always_inline)) {
      // This step's operands have arrived (GROUPED: the last four loads are
      // the next step's B), and every wave is done with the last step's.
      if (GROUPED)
        asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      fence();
      // (The last steps load the last one again, for nobody.)
      const int s1 = min(s + 1, nk - 1), s2 = min(s + 2, nk - 1);
      a[0] = frag(cur + arow);
      fence();
#pragma unroll
      for (int j = 0; j < 4; j++) {
        mfma(bf[j].h[0], last.h[0], acc[NI - 1][j]);
        fence();
        load_a(s1, nxt, j);
        fence();
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        mfma(bf[j].h[1], last.h[1], acc[NI - 1][j]);
        fence();
        bf[j] = frag(cur + brow + j * 2048);
        fence();
      }
      a[1] = frag(cur + arow + 4096);
#pragma unroll
      for (int i = 0; i < NI - 1; i++) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            mfma(bf[j].h[h], a[i % 3].h[h], acc[i][j]);
            if (h == 0 && j == 1 && i + 2 < NI) a[(i + 2) % 3] = frag(cur + arow + (i + 2) * 4096);
            if (GROUPED && i == 1 && h == 0) load_b(s2, cur, j);
            if (!GROUPED && i == 0 && h == 0) load_b(s1, nxt, j);
            fence();
          }
        if (GROUPED && i == 0) {
          // Every wave has its B fragments (group 0's MFMAs took them).
          asm volatile("s_barrier" ::: "memory");
          fence();
          if (NI == 2) {
#pragma unroll
            for (int j = 0; j < 4; j++) load_b(s2, cur, j);
            fence();
          }
        }
      }
      last = a[kLast];
    };
    int s = 0;
    for (; s + 1 < nk; s += 2) {
      step(s, smem, smem + kStage);
      step(s + 1, smem + kStage, smem);
    }
    if (s < nk) step(s, smem, smem + kStage);
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int j = 0; j < 4; j++) mfma(bf[j].h[h], last.h[h], acc[NI - 1][j]);
  };
  if (mrows > 128)
    run(std::integral_constant<int, 8>{});
  else if (mrows > 64)
    run(std::integral_constant<int, 4>{});
  else
    run(std::integral_constant<int, 2>{});

  // Epilogue: each wave stages its rows x 64 columns, four groups (fp32: two) at a time,
  // in its own LDS and writes whole rows of 128 or 256 bytes.
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  constexpr int kEs = OUT == kOutF32 ? 4 : 2, kPitch = 64 * kEs + 16;
  constexpr int kPass = OUT == kOutF32 ? 2 : 4;  // groups staged at a time
  uint8_t* buf = smem + wave * (kPass * 16 * kPitch);
  static_assert(8 * kPass * 16 * kPitch <= kSmem, "epilogue");
  const bool vec_ok = p.ldc % (16 / kEs) == 0;
  int8::Scale sb[4][4];
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const int col = n0 + wn * 64 + j * 16 + 4 * g + e;
      sb[j][e] = int8::split(col < p.N ? p.SB[(int64_t)t.group * p.N + col] : 0.0f);
    }
#pragma unroll
  for (int h = 0; h < 8 / kPass; h++) {
    if (h * 32 * kPass >= mrows) break;
#pragma unroll
    for (int i = 0; i < kPass; i++) {
      const int row = (h * kPass + i) * 32 + wm * 16 + r;
      const int8::Scale sa = int8::split(row < mrows ? p.SA[t.row + row] : 0.0f);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = int8::apply(acc[kPass * h + i][j][e], sa, sb[j][e]);
        uint8_t* dst = buf + (i * 16 + r) * kPitch + (j * 16 + 4 * g) * kEs;
        if (OUT == kOutF32)
          *(f32x4*)dst = f32x4{v[0], v[1], v[2], v[3]};
        else
          *(u32x2*)dst = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
    constexpr int kLanes = 64 * kEs / 16, kRows = 64 / kLanes;  // lanes of a row, rows of a store
#pragma unroll
    for (int q = 0; q < kPass * 16 / kRows; q++) {
      const int lrow = q * kRows + lane / kLanes, lcol = (lane % kLanes) * (16 / kEs);
      const u32x4 v = *(const u32x4*)(buf + lrow * kPitch + lcol * kEs);
      const int row = (h * kPass + lrow / 16) * 32 + wm * 16 + lrow % 16, col = n0 + wn * 64 + lcol;
      if (row >= mrows) continue;
      uint8_t* dst = (uint8_t*)p.C + ((int64_t)(t.row + row) * p.ldc + col) * kEs;
      if (vec_ok && col + 16 / kEs <= p.N) {
        __builtin_nontemporal_store(v, (u32x4*)dst);
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 16 / kEs; e++)
          if (col + e < p.N) {
            if (OUT == kOutF32)
              ((uint32_t*)dst)[e] = w[e];
            else
              ((uint16_t*)dst)[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
          }
      }
    }
  }
}

}  // namespace

hipError_t gemm_int8_large(int64_t M, int64_t N, int64_t K, const void* a, const void* sa, const void* b, const void* sb,
                           const int32_t* offsets, int64_t groups, int out_dtype, void* c, int64_t ldc, hipStream_t s) {
  const Args p{(const uint8_t*)a, (const uint8_t*)b, (const float*)sa, (const float*)sb, c, offsets,
               ldc, (int)groups, (int)M, (int)N, (int)K, (int)((N + BN - 1) / BN)};
  const int64_t tm = offsets ? groups::max_row_tiles(M, groups, BM) : (M + BM - 1) / BM;
  const dim3 grid((unsigned)groups::grid_size(tm, p.tiles_n));
  const bool f32 = out_dtype == kOutF32;
  if (offsets && f32) return launch_kernel(&gemm_int8_large_kernel<kOutF32, true>, grid, kThreads, 0, s, p);
  if (offsets) return launch_kernel(&gemm_int8_large_kernel<kOutBF16, true>, grid, kThreads, 0, s, p);
  if (f32) return launch_kernel(&gemm_int8_large_kernel<kOutF32, false>, grid, kThreads, 0, s, p);
  return launch_kernel(&gemm_int8_large_kernel<kOutBF16, false>, grid, kThreads, 0, s, p);
}

}  // namespace mx
