// Block-scaled GEMM C = A B^T for few rows of A (decode): FP8 x FP8 under fp32 scales
// per 1 x 128 of A and 128 x 128 of B, dense or by expert, MXFP4 x MXFP4 by
// expert, and INT8 x INT8 under a scale per row, dense or by expert. (The mathematics is
// gemm_block.hip's and gemm_int8.hip's.)
//
// Bound by HBM: every weight byte is read once and meets 16 rows of A, so
// the kernel is a stream of weights from HBM through VGPRs to the matrix core.
//  * A workgroup takes T tiles of 16 weight rows of one expert. K goes to its
//    waves in chunks of W S steps of 128 bytes (128 K of FP8, 256 K of
//    MXFP4), S consecutive steps each. A wave keeps A's fragments (and scales) of
//    its S steps in VGPRs and runs tile by tile: the waves' loads are 16 rows x 128 W S
//    contiguous bytes, which keeps DRAM pages open, and A's cost is shared
//    by T tiles. The waves' sums meet in LDS at the end, in a fixed order.
//  * Weights go HBM -> LDS directly, whole 128-byte lines, 8 rows a load, into a
//    ring of D steps of the wave's own: no barrier, D - 1 steps in flight, and no
//    VGPRs for them. The loads are non-temporal (38 us instead of 43). (Loading
//    fragments, 64 bytes of 16 rows a load, into VGPRs reached 4.5-5.2 TB/s at
//    16 x 28672 x 8192; this does 6.2.) The chunk swizzle of LDS rows is gemm_block.hip's.
//  * In a step lane (r, g) = (l % 16, l / 16) takes chunks g and g + 4 of row r of
//    the tile; the same order of K in A.
//  * Loads are range-checked buffer loads without a branch: rows past the
//    group's or N, steps past K and 32-element blocks past K read as zeros.
//  * FP8 codes meet in bf16 MFMAs, expanded exactly, for either result: the matrix core and
//    the vector ALU wait for HBM, and the FP8 MFMA, which loses bits of a sum, would
//    gain nothing (16 rows, FP8 MFMA / bf16: 28672 x 8192 37.8 / 37.8 us, 4096 x 4096
//    6.8 / 6.9, 8192 x 28672 44.0 / 44.5; 128 rows over 64 x 2048 x 4096 73.4 / 73.9).
//  * A group with more than 16 rows takes further passes over the weights, each in
//    workgroups of its own, which find their group and rows from the offsets: all
//    CUs share the passes of the one expert that a router may send everything to.
#include <type_traits>
#include <utility>

#include "bf16.h"
#include "fp8_encode.h"
#include "groups.h"
#include "int8.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
// Lane and scalar offsets past every buffer's range (256 rows of at most 2^22
// bytes); their sum is one too.
constexpr uint32_t kOOB = 0x80000000u, kScalarOOB = 0x40000000u;
typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr int kNonTemporal = 2;                // cache policy of a load: streamed

struct Args {
  const uint8_t *A, *SA, *B, *SB;
  void* C;
  const int* offsets;  // null: dense (FP8 and INT8, M at most 16)
  int64_t ldc;
  int groups, M, N, K;
};

template <typename F, int... K>
__device__ __forceinline__ void unroll_at(F&& f, std::integer_sequence<int, K...>) {
  (f(std::integral_constant<int, K>{}), ...);
}
// f(0), f(1), ..., f(N - 1), each with its number as a constant.
template <int N, typename F>
__device__ __forceinline__ void unroll(F&& f) {
  unroll_at(std::forward<F>(f), std::make_integer_sequence<int, N>{});
}

// ALIGNED: a row's MXFP4 scales start on dwords (K % 128 = 0).
// W: waves.
template <int FMT, bool ALIGNED, int OUT, int W, int S, int T, int D>
__global__ __launch_bounds__(64 * W) void gemm_few_rows_kernel(Args p) {
  constexpr bool FP4 = FMT == kMXFP4, FP8 = FMT == kFP8B128, INT8 = FMT == kINT8;
  using Sum = typename std::conditional<INT8, int, float>::type;
  using Sum4 = typename std::conditional<INT8, i32x4, f32x4>::type;
  constexpr int kWaves = W;
  constexpr int kSlot = 2048, kRing = kWaves * D * kSlot, kSums = kWaves * T * 4 * 64 * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kRing > kSums ? kRing : kSums];
  Sum(*part)[T][4][64] = (Sum(*)[T][4][64])smem;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * T);
  int group = 0, m0 = 0, mrows = p.M;
  if ((FP4 || p.offsets) && !groups::pass_of(p.offsets, p.groups, p.M, blockIdx.y, group, m0, mrows)) return;

  const int nrows = min(p.N - n0, 16 * T);
  const uint32_t rowbytes = (uint32_t)(FP4 ? p.K / 2 : p.K);
  const int nk = (int)((rowbytes + 127) / 128);
  const uint32_t sstride = FP8 ? (uint32_t)(nk * 4) : FP4 ? (uint32_t)(p.K / 32) : 0;  // scale bytes per row
  const int64_t brow = (int64_t)group * p.N + n0;
  const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.B + brow * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);
  // FP8: the scale rows of this workgroup's 128-row blocks (they may be two or more).
  const int nb0 = n0 / 128, nbs = (p.N + 127) / 128;
  const __amdgpu_buffer_rsrc_t rSB =
      FP8 ? __builtin_amdgcn_make_buffer_rsrc((void*)(p.SB + ((int64_t)group * nbs + nb0) * sstride), 0,
                                              (int)((uint32_t)(nbs - nb0) * sstride), kRsrcFlags)
          : __builtin_amdgcn_make_buffer_rsrc((void*)(p.SB + brow * sstride), 0, (int)((uint32_t)nrows * sstride), kRsrcFlags);
  // (INT8's scales are the result's, read at the end.)
  // Lane offsets within a tile, for A's fragments (row r, chunks g and g + 4)
  // and for the weights' loads (row l / 8 + 8 h, the chunk that belongs into slot
  // l % 8): the step and the tile go into the scalar offset, which the range
  // check counts too. In the last step of an MXFP4 or INT8 row that is no multiple
  // of 128 bytes long, chunks past its end are left out.
  const uint32_t left = rowbytes - 128u * (uint32_t)(nk - 1);
  uint32_t va[2], va_last[2], vb[2], vb_last[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const uint32_t ca = 16u * (uint32_t)(g + 4 * h), cb = 16u * (uint32_t)((lane & 7) ^ (4 * h + (lane >> 4)));
    va[h] = (uint32_t)r * rowbytes + ca;
    vb[h] = (uint32_t)(8 * h + (lane >> 3)) * rowbytes + cb;
    va_last[h] = FP8 || ca < left ? va[h] : kOOB;
    vb_last[h] = FP8 || cb < left ? vb[h] : kOOB;
  }
  const uint32_t soff = (uint32_t)r * sstride;
  const int chunks = (nk + kWaves * S - 1) / (kWaves * S);
  uint8_t* ring = smem + wave * (D * kSlot);
  const int frag0 = r * 128 + ((g ^ (r >> 1)) & 7) * 16, frag1 = r * 128 + (((g + 4) ^ (r >> 1)) & 7) * 16;

  auto step_at = [&](uint32_t row, int s) __attribute__((always_inline)) {
    return (int)(s < nk ? row + (uint32_t)s * 128u : kScalarOOB);
  };
  // MXFP4: the scales of step s, blocks 0..3 and 4..7 (this lane uses byte g of
  // each dword). Bytes past the row's end are left out: they are another
  // row's and might be NaN.
  auto load_scales = [&](__amdgpu_buffer_rsrc_t rs, uint32_t row, int s) __attribute__((always_inline)) {
    const uint32_t so = s < nk ? row + (uint32_t)s * 8u : kScalarOOB;
    if (ALIGNED) {
      u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, soff, (int)so, 0));
      if (s * 8 + 4 >= (int)sstride) v.y = 0;  // (K % 256 = 128)
      return v;
    }
    const uint32_t b = (uint32_t)s * 8u + (uint32_t)g;
    const uint32_t x = __builtin_amdgcn_raw_buffer_load_b8(rs, b < sstride ? soff + g : kOOB, (int)so, 0);
    const uint32_t y = __builtin_amdgcn_raw_buffer_load_b8(rs, b + 4u < sstride ? soff + 4u + g : kOOB, (int)so, 0);
    return u32x2{x << (8 * g), y << (8 * g)};
  };

  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.A + (int64_t)m0 * rowbytes), 0, (int)((uint32_t)mrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rSA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.SA + (int64_t)m0 * sstride), 0, (int)((uint32_t)mrows * sstride), kRsrcFlags);
  Sum4 acc[T];
#pragma unroll
  for (int j = 0; j < T; j++) acc[j] = Sum4{0, 0, 0, 0};

  for (int c = 0; c < chunks; c++) {
    const int s0 = (c * kWaves + wave) * S;
    // The ring's first weights, then A of all S steps, then (FP8) the
    // weights' scales: lane l's is step s0 + l's.
    u32x2 wsc[D];  // MXFP4: the ring's scales
    auto load = [&](int k) __attribute__((always_inline)) {
      const int t = k / S, s = s0 + k % S;
      const int so = step_at((uint32_t)(16 * t) * rowbytes, s);
#pragma unroll
      for (int h = 0; h < 2; h++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)(ring + (k % D) * kSlot + h * 1024), 16,
                                                 FP8 || s < nk - 1 ? vb[h] : vb_last[h], so, 0, kNonTemporal);
      if (FP4) wsc[k % D] = load_scales(rSB, (uint32_t)(16 * t) * sstride, s);
    };
#pragma unroll
    for (int k = 0; k < D - 1; k++)
      if (k < T * S) load(k);
    i32x8 a[S];
    float sa[S];
    u32x2 sc[S];
#pragma unroll
    for (int s = 0; s < S; s++) {
      const int so = step_at(0, s0 + s);
      const bool full = FP8 || s0 + s < nk - 1;
      const i32x4 x = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, full ? va[0] : va_last[0], so, 0));
      const i32x4 y = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, full ? va[1] : va_last[1], so, 0));
      a[s] = i32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      if (FP8)
        sa[s] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
            rSA, soff, (int)(s0 + s < nk ? (uint32_t)(s0 + s) * 4u : kScalarOOB), 0));
      else if (FP4)
        sc[s] = load_scales(rSA, 0, s0 + s);
    }
    float sb[T];
    if (FP8) {
#pragma unroll
      for (int t = 0; t < T; t++) {
        const uint32_t nb = (uint32_t)((n0 + 16 * t) / 128 - nb0);  // (a tile past N: out of range)
        sb[t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
            rSB, s0 + lane < nk ? (uint32_t)lane * 4u : kOOB, (int)(nb * sstride + (uint32_t)s0 * 4u), 0));
      }
    }
    // Step k + 1's fragments are read before step k's MFMAs. Loads end in
    // order: step k + 1's have arrived when only the later steps' are out
    // (the first time, A's too, which came last).
    constexpr int kLoads = !FP4 ? 2 : ALIGNED ? 3 : 4;  // of a step
    auto arrived = [&](auto n) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(%0)" ::"i"(decltype(n)::value) : "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto read = [&](int k) __attribute__((always_inline)) {
      const i32x4 x = *(const i32x4*)(ring + (k % D) * kSlot + frag0), y = *(const i32x4*)(ring + (k % D) * kSlot + frag1);
      return i32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };
    arrived(std::integral_constant<int, 0>{});
    i32x8 next = read(0);
    unroll<T * S>([&](auto kk) __attribute__((always_inline)) {
      constexpr int k = decltype(kk)::value, t = k / S, s = k % S;
      const i32x8 bv = next;
      if (k + D - 1 < T * S) load(k + D - 1);
      if constexpr (k + 1 < T * S) {
        // Steps loaded behind k + 1 (the first D - 1 have all arrived).
        constexpr int last = k + D - 1 < T * S ? k + D - 1 : T * S - 1;
        constexpr int behind = last - (k + 1);
        if constexpr (k + 1 >= D - 1) arrived(std::integral_constant<int, behind * kLoads>{});
        next = read(k + 1);
      }
      const u32x2 wscale = wsc[k % D];
      if constexpr (FP8) {
        const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sb[t]), s));
        const float f = sa[s] * w;
        f32x4 P = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 4; h++)
          P = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8::expand8(bv[2 * h], bv[2 * h + 1]),
                                                      fp8::expand8(a[s][2 * h], a[s][2 * h + 1]), P, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[t][e] = __builtin_fmaf(P[e], f, acc[t][e]);
      } else if constexpr (INT8) {
#pragma unroll
        for (int h = 0; h < 2; h++)
          acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(i32x4{bv[4 * h], bv[4 * h + 1], bv[4 * h + 2], bv[4 * h + 3]},
                                                         i32x4{a[s][4 * h], a[s][4 * h + 1], a[s][4 * h + 2], a[s][4 * h + 3]}, acc[t], 0, 0, 0);
      } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const i32x8 bh = {bv[4 * h], bv[4 * h + 1], bv[4 * h + 2], bv[4 * h + 3], 0, 0, 0, 0};
          const int wb = (int)((wscale[h] >> (8 * g)) & 0xFFu);
          const i32x8 av = {a[s][4 * h], a[s][4 * h + 1], a[s][4 * h + 2], a[s][4 * h + 3], 0, 0, 0, 0};
          const int wa = (int)((sc[s][h] >> (8 * g)) & 0xFFu);
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bh, av, acc[t], 4, 4, 0, wb, 0, wa);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  // The waves' sums, added in their order. acc[j][e] of lane (r, g) is row r,
  // column 16 j + 4 g + e.
  __syncthreads();  // (every ring has been read)
#pragma unroll
  for (int j = 0; j < T; j++)
#pragma unroll
    for (int e = 0; e < 4; e++) part[wave][j][e][lane] = acc[j][e];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < (T + kWaves - 1) / kWaves; u++) {
    const int j = u * kWaves + wave;
    if (j >= T) break;
    Sum4 sum;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      sum[e] = part[0][j][e][lane];
#pragma unroll
      for (int w = 1; w < kWaves; w++) sum[e] += part[w][j][e][lane];
    }
    const int col = n0 + 16 * j + 4 * g;
    if (r >= mrows) continue;
    f32x4 v;
    if constexpr (INT8) {
      const int8::Scale sa = int8::split(((const float*)p.SA)[m0 + r]);
      const float* sb = (const float*)p.SB + (int64_t)group * p.N + col;
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = int8::apply(sum[e], sa, int8::split(col + e < p.N ? sb[e] : 0.0f));
    } else {
      v = sum;
    }
    const int64_t at = (int64_t)(m0 + r) * p.ldc + col;
    if (p.ldc % 4 == 0 && col + 4 <= p.N) {
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

// Passes of 16 rows that any offsets can need (dense: one).
int64_t passes(int64_t M, int64_t groups) { return groups > 0 ? groups::max_row_tiles(M, groups, 16) : 1; }

template <int FMT, bool ALIGNED, int OUT, int W, int S, int T, int D>
hipError_t launch(const Args& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 16 * T - 1) / (16 * T)), (unsigned)passes(p.M, p.offsets ? p.groups : 0));
  return launch_kernel(&gemm_few_rows_kernel<FMT, ALIGNED, OUT, W, S, T, D>, grid, 64 * W, 0, s, p);
}

// Rounds of the 256 CUs that workgroups of T tiles make, one a CU at a time.
int64_t rounds(int64_t tiles, int T) { return (tiles + 256 * T - 1) / (256 * T); }

// Experts that have rows are taken as min(groups, M). Times in us at 16 rows,
// FP8, N x K (by expert: rows over experts x N x K). INT8 takes the same, as its rows are as long; of it were measured
// 2048 x 2048 2.8 (one row), 4096 x 4096 6.0, 10240 x 8192 17.3, 28672 x 8192 37.6 and, 128 rows over 64 x 2048 x 4096, 64.
template <int FMT, bool ALIGNED, int OUT>
hipError_t dispatch(const Args& p, hipStream_t s) {
  if constexpr (FMT != kMXFP4) {
    const int64_t tiles = (p.N + 15) / 16 * (!p.offsets ? 1 : p.M < p.groups ? p.M : p.groups);
    const int nk = (p.K + 127) / 128;
    if (p.offsets) {
      // Few experts with rows: 4 waves on long runs (8 rows over 32 x 2048 x 4096: 12.0,
      // below 14.7; 128 over 64: 60.2 and 59.2, 32 over 16 x 4096 x 7168: 79 and 65).
      if (nk > 16 && tiles >= 512 && tiles < 2048) return launch<FMT, ALIGNED, OUT, 4, 8, 2, 8>(p, s);
    } else {
      // Long rows, many of them: 7 tiles share A in a workgroup of 8 waves, one a CU, or 4 in one
      // of 4 waves (below), whichever's rounds of CUs take fewer tiles (K = 8192, N = 14336 / 18432 /
      // 28672 / 29568 / 32768 / 43008 / 57344 / 65536 / 86016 / 128256: 7 tiles 30 / 29 / 38 / 59 / 59 / 62 / 76 / 97 /
      // 113 / 172, 4 tiles 24 / 38 / 40 / 41 / 45 / 59 / 78 / 86 / 119 / 167; K = 4096, N = 18432 / 28672: 21 / 26
      // and 21 / 23).
      if (nk >= 48 && tiles > 768 && 7 * rounds(tiles, 7) <= 4 * rounds(tiles, 4))
        return launch<FMT, ALIGNED, OUT, 8, 8, 7, 8>(p, s);
      // The fewest tiles a workgroup that need one round of CUs (T = 1 / 2 / 3:
      // 4096 x 4096 6.6 / 7.3 / 8.7, 6144 x 4096 9.7 / 7.6 / 9.2, 10240 x 8192 - / 24.9 / 16.8;
      // 14336 x 4096: 13.6, with T = 2 13.9, T = 3 16.5).
      if (tiles <= 256) return launch<FMT, ALIGNED, OUT, 8, 2, 1, 3>(p, s);
      // (8192 x 28672: 4 waves on long runs 44.4, T = 2 46.5; one row 37.2 and 41.5.)
      if (tiles <= 512 && nk >= 128) return launch<FMT, ALIGNED, OUT, 4, 8, 2, 8>(p, s);
      if (tiles > 512 && tiles <= 768) return launch<FMT, ALIGNED, OUT, 8, 1, 3, 4>(p, s);
      if (tiles > 768 && nk > 16) return launch<FMT, ALIGNED, OUT, 4, 8, 4, 9>(p, s);
    }
  }
  // Two tiles, a step of each in a wave's chunk: eight waves on one run of a row
  // (mxfp4 128 over 64 x 2048 x 4096: 35.4, with 4 waves on runs of 4 steps 42.9, four tiles 37.7).
  return launch<FMT, ALIGNED, OUT, 8, 1, 2, 3>(p, s);
}

template <bool ALIGNED>
hipError_t mxfp4(const Args& p, bool f32, hipStream_t s) {
  if (f32) return dispatch<kMXFP4, ALIGNED, kOutF32>(p, s);
  return dispatch<kMXFP4, ALIGNED, kOutBF16>(p, s);
}

}  // namespace

// fp32 results but INT8's: accumulation chains of at most 48 matrix instructions or scale
// blocks, of 128 K, in a wave.
bool gemm_few_rows_fits(int fmt, int64_t M, int64_t N, int64_t K, int64_t groups, int out_dtype) {
  // (The grid: 16 columns a workgroup across, passes down.)
  if (N > ((int64_t)1 << 27) || passes(M, groups) > 65535) return false;
  return fmt == kINT8 || out_dtype != kOutF32 || K <= (int64_t)48 * 128 * 4;
}

hipError_t gemm_few_rows(int fmt, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                         const void* b, const void* sb, const int32_t* offsets, int64_t groups,
                         int out_dtype, void* c, int64_t ldc, hipStream_t s) {
  const Args p{(const uint8_t*)a, (const uint8_t*)sa, (const uint8_t*)b, (const uint8_t*)sb, c, offsets,
               ldc, (int)groups, (int)M, (int)N, (int)K};
  const bool f32 = out_dtype == kOutF32;
  if (fmt == kMXFP4) return K % 128 == 0 ? mxfp4<true>(p, f32, s) : mxfp4<false>(p, f32, s);
  if (fmt == kINT8) return f32 ? dispatch<kINT8, true, kOutF32>(p, s) : dispatch<kINT8, true, kOutBF16>(p, s);
  return f32 ? dispatch<kFP8B128, true, kOutF32>(p, s) : dispatch<kFP8B128, true, kOutBF16>(p, s);
}

}  // namespace mx
