// FP8 x FP8 GEMM under fp32 scales per 1 x 128 of A and 128 x 128 of B, bf16
// result, the large-tile kernel (dense or by expert; the mathematics and the
// choice of the FP8 MFMA are described in gemm_block.hip):
//   C[i][j] = sum over 128-K blocks q of s_A[i][q] s_B[j / 128][q] P_q[i][j].
//
// Bound by the matrix cores: a K step of 128 takes a 256 x 256 tile's SIMDs 2048
// cycles of FP8 MFMA each, against 1024 of fma on the vector ALU and 1536 of LDS reads.
//  * 8 waves (two per SIMD) of 128 x 64, because the vector ALU adds to the
//    accumulators: they and the partial sums must fit one wave's VGPRs. The
//    SIMD's second wave issues MFMAs while the first one adds.
//  * A wave's step is 8 groups of four 16 x 16 x 128 MFMAs, one group per 16
//    rows; the tile's 16-row groups go to the two rows of waves in turn, so that a
//    partly filled tile (the last one of an expert) of at most 128 or 64 rows
//    is done in 4 or 2 groups a step. A group's partial sums are added
//    beside the next group's MFMAs (four behind; three behind: 1.3% slower),
//    and its A fragment is read two groups ahead, so that neither is waited for.
//  * The last group of a step is issued after the barrier, beside the next
//    step's first fragment reads: it is their latency's cover. Each B fragment
//    is overwritten right after that group's MFMA on it.
//  * Operands go HBM -> LDS directly, into double buffers, a step ahead. By
//    expert, weights come from HBM, whose latency is about a step: there every
//    wave has read its B fragments early in a step, and after one more barrier
//    B's buffer takes B of two steps ahead (8 experts of 8192 x 4096, 16384
//    rows: 523 us, 548 a step ahead). A dense product finds B in the caches
//    and is faster without that barrier (469 us, 479 with it). The chunk
//    swizzle, the buffer views that end with the group's rows and the operand
//    order are gemm_block.hip's.
#include <type_traits>

#include "bf16.h"
#include "groups.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
constexpr uint32_t kOOB = 0x80000000u;        // an offset past every buffer's range
constexpr int BM = 256, BN = 256, kWN = 4, kThreads = 512;
// A stage: A's and B's codes. Behind the two stages, s_A of four steps at a time
// (16 bytes a row; loaded 4 bytes a row each step it costs 5% of the time),
// double-buffered, and 1 KB that nobody reads.
constexpr int kOffB = BM * 128, kStage = kOffB + BN * 128;
constexpr int kScales = BM * 16, kDummy = 2 * kStage + 2 * kScales, kSmem = kDummy + 1024;
constexpr int kPitch = 64 * 2 + 16;  // epilogue row of a wave

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

struct Args {
  const uint8_t *A, *B;
  const float *SA, *SB;
  uint16_t* C;
  const int* offsets;  // null: dense
  int64_t ldc;
  int groups, M, N, K, tiles_n;
};

// GROUPED: p.offsets given.
template <bool GROUPED>
__global__ __launch_bounds__(kThreads, 1) void gemm_fp8_large_kernel(Args p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kSmem];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWN, wn = wave % kWN;
  const int r = lane & 15, g = lane >> 4;

  groups::Tile t;
  if (!groups::tile_of<BM>(GROUPED ? p.offsets : nullptr, p.groups, p.M, p.tiles_n, blockIdx.x, t)) return;
  const int n0 = t.tn * BN;
  const int mrows = min(t.rows, BM), nrows = min(p.N - n0, BN);
  const uint32_t rowbytes = (uint32_t)p.K;
  const int nk = p.K / 128;
  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.A + (int64_t)t.row * rowbytes), 0, (int)((uint32_t)mrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.B + ((int64_t)t.group * p.N + n0) * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rS = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.SA + (int64_t)t.row * nk), 0, (int)((uint32_t)mrows * (uint32_t)nk * 4u), kRsrcFlags);
  const int nb = min(n0 + wn * 64, p.N - 1) / 128;  // (a wave wholly past N: any)
  const float* sb_row = p.SB + ((int64_t)t.group * ((p.N + 127) / 128) + nb) * nk;

  // Lane parts of the load addresses: a load covers 8 rows of 128 bytes, lane
  // l slot l % 8 of row l / 8, which holds chunk slot ^ swz(row); swz(row)
  // depends on the parity of the load's block of 8 rows.
  uint32_t loff[2];
#pragma unroll
  for (int h = 0; h < 2; h++)
    loff[h] = (uint32_t)(lane >> 3) * rowbytes + (uint32_t)(((lane & 7) ^ swz(8 * h + (lane >> 3))) * 16);
  const uint32_t soff = (uint32_t)((wave & 3) * 64 + lane) * (uint32_t)nk * 4u;
  // Loads P = 0..3 of A's and of B's 8-row blocks 4 wave + P. The row and step
  // go into the scalar offset, which the range check counts too.
  const uint32_t rows8 = 8 * rowbytes;
  auto load_a = [&](int s, uint8_t* stage, int P) __attribute__((always_inline)) {
    const int b = wave * 4 + P;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr_t)(stage + b * 1024), 16, loff[P & 1],
                                             (int)((uint32_t)b * rows8) + s * 128, 0, 0);
  };
  auto load_b = [&](int s, uint8_t* stage, int P) __attribute__((always_inline)) {
    const int b = wave * 4 + P;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)(stage + kOffB + b * 1024), 16, loff[P & 1],
                                             (int)((uint32_t)b * rows8) + s * 128, 0, 0);
  };
  // s_A of steps 4 q .. 4 q + 3 for the rows of wave w (0..3). (A row's scales
  // are only aligned to 4 bytes, which is enough; past its last one come the
  // next row's, unused, and the range check works dword by dword.) The other
  // waves run the same load, out of range, into the LDS that nobody reads.
  auto load_s = [&](int q, int w) __attribute__((always_inline)) {
    const bool mine = wave == w;
    uint8_t* dst = smem + (mine ? 2 * kStage + (q & 1) * kScales + w * 1024 : kDummy);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_ptr_t)dst, 16, soff, mine ? q * 16 : (int)kOOB, 0, 0);
  };

  f32x4 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = f32x4{0, 0, 0, 0};

  // Fragment addresses: chunks g and g + 4 of row r of a 16-row tile; swz(r)
  // is the same in every tile. The wave's group i is rows 32 i + 16 wm + r.
  const int c0 = (g ^ swz(r)) * 16, c1 = ((g + 4) ^ swz(r)) * 16;
  const int arow = (wm * 16 + r) * 128, brow = kOffB + (wn * 64 + r) * 128, srow = 2 * kStage + (wm * 16 + r) * 16;
  auto frag = [&](const uint8_t* row) __attribute__((always_inline)) {
    const i32x4 lo = *(const i32x4*)(row + c0), hi = *(const i32x4*)(row + c1);
    return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  };

  i32x8 bf[4], a[3];
  float f[3];        // s_A of a's rows
  f32x4 P[2][4];     // partial sums of an even and of an odd group
#pragma unroll
  for (int j = 0; j < 4; j++) {
    bf[j] = i32x8{0, 0, 0, 0, 0, 0, 0, 0};
    P[0][j] = f32x4{0, 0, 0, 0};
  }
  auto mfma = [&](const i32x8& bv, const i32x8& av) __attribute__((always_inline)) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, f32x4{0, 0, 0, 0}, 0, 0, 0, 127, 0, 127);
  };
  auto add = [&](const f32x4& o, float w, f32x4& c) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; e++) c[e] = __builtin_fmaf(o[e], w, c[e]);
  };

#pragma unroll
  for (int q = 0; q < 4; q++) {
    load_a(0, smem, q);
    load_b(0, smem, q);
  }
#pragma unroll
  for (int w = 0; w < 4; w++) load_s(0, w);
  if (GROUPED) {
    fence();
#pragma unroll
    for (int q = 0; q < 4; q++) load_b(min(1, nk - 1), smem + kStage, q);
    fence();
  }
  float sb = sb_row[0];
  // All steps, with NI groups a step. On entry of a step: `last` is the last
  // group of the step before (its MFMAs still to do, on bf, and to add times
  // wl), P[0] is of its last but one (still to add times wk). (Before
  // the first step all of them are zero, and add nothing.) The source is in
  // issue order: a fence after each MFMA and what runs beside it.
  auto run = [&](auto ni) __attribute__((always_inline)) {
    constexpr int NI = decltype(ni)::value;
    constexpr int kLast = (NI - 1) % 3;  // where a step leaves its last fragment
    constexpr int kS = GROUPED || NI < 8 ? 0 : 3;  // the group that loads s_A (before the next B)
    i32x8 last = i32x8{0, 0, 0, 0, 0, 0, 0, 0};
    float wk = 0.0f, wl = 0.0f;
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
      const float sbn = sb_row[s1];
      a[0] = frag(cur + arow);
      const uint8_t* sc = smem + srow + ((s >> 2) & 1) * kScales + (s & 3) * 4;
      f[0] = *(const float*)sc;
      fence();
#pragma unroll
      for (int j = 0; j < 4; j++) {
        P[1][j] = mfma(bf[j], last);
        add(P[0][j], wk, acc[NI - 2][j]);
        fence();
        bf[j] = frag(cur + brow + j * 2048);
        load_a(s1, nxt, j);
        fence();
      }
      a[1] = frag(cur + arow + 4096);
      f[1] = *(const float*)(sc + 512);
      float w = wl;
#pragma unroll
      for (int i = 0; i < NI - 1; i++) {
        const float wi = f[i % 3] * sb;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          P[i & 1][j] = mfma(bf[j], a[i % 3]);
          if (j == 1 && i + 2 < NI) {
            a[(i + 2) % 3] = frag(cur + arow + (i + 2) * 4096);
            f[(i + 2) % 3] = *(const float*)(sc + (i + 2) * 512);
          }
          if (GROUPED && i == 1) load_b(s2, cur, j);
          if (!GROUPED && i == 0) load_b(s1, nxt, j);
          if (i == kS && j == 3) load_s((s >> 2) + 1, s & 3);
          add(P[(i + 1) & 1][j], w, acc[(i + NI - 1) % NI][j]);
          fence();
        }
        w = wi;
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
      wk = w;
      wl = f[kLast] * sb;
      sb = sbn;
    };
    int s = 0;
    for (; s + 1 < nk; s += 2) {
      step(s, smem, smem + kStage);
      step(s + 1, smem + kStage, smem);
    }
    if (s < nk) step(s, smem, smem + kStage);
#pragma unroll
    for (int j = 0; j < 4; j++) add(P[0][j], wk, acc[NI - 2][j]);
#pragma unroll
    for (int j = 0; j < 4; j++) add(mfma(bf[j], last), wl, acc[NI - 1][j]);
  };
  if (mrows > 128)
    run(std::integral_constant<int, 8>{});
  else if (mrows > 64)
    run(std::integral_constant<int, 4>{});
  else
    run(std::integral_constant<int, 2>{});

  // Epilogue: each wave stages its rows x 64 columns in two halves of 64 rows
  // (4 groups) in its own LDS and writes whole 128-byte rows.
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  uint8_t* buf = smem + wave * (64 * kPitch);
  const bool vec_ok = p.ldc % 8 == 0;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    if (h * 128 >= mrows) break;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const f32x4 v = acc[4 * h + i][j];
        *(u32x2*)(buf + (i * 16 + r) * kPitch + (j * 16 + 4 * g) * 2) =
            u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
#pragma unroll
    for (int q = 0; q < 8; q++) {
      const int lrow = q * 8 + (lane >> 3), lcol = (lane & 7) * 8;
      const u32x4 v = *(const u32x4*)(buf + lrow * kPitch + lcol * 2);
      const int row = h * 128 + lrow / 16 * 32 + wm * 16 + lrow % 16, col = n0 + wn * 64 + lcol;
      if (row >= mrows) continue;
      uint16_t* dst = p.C + (int64_t)(t.row + row) * p.ldc + col;
      if (vec_ok && col + 8 <= p.N) {
        __builtin_nontemporal_store(v, (u32x4*)dst);
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (col + e < p.N) dst[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
      }
    }
  }
}

}  // namespace

hipError_t gemm_fp8_large(int64_t M, int64_t N, int64_t K, const void* a, const void* sa, const void* b,
                          const void* sb, const int32_t* offsets, int64_t groups, void* c, int64_t ldc,
                          hipStream_t s) {
  const Args p{(const uint8_t*)a, (const uint8_t*)b, (const float*)sa, (const float*)sb, (uint16_t*)c, offsets,
               ldc, (int)groups, (int)M, (int)N, (int)K, (int)((N + BN - 1) / BN)};
  const int64_t tm = offsets ? groups::max_row_tiles(M, groups, BM) : (M + BM - 1) / BM;
  const dim3 grid((unsigned)groups::grid_size(tm, p.tiles_n));
  if (offsets) return launch_kernel(&gemm_fp8_large_kernel<true>, grid, kThreads, 0, s, p);
  return launch_kernel(&gemm_fp8_large_kernel<false>, grid, kThreads, 0, s, p);
}

}  // namespace mx
