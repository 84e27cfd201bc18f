// Block-scaled GEMM C = A B^T for few rows of A (decode), dense or by expert:
// MXFP4 x MXFP4, and FP8 x FP8 under fp32 scales per 1 x 128 of A and 128 x 128
// of B. (The mathematics and the choice between the FP8 and the bf16 MFMA are
// gemm_block.hip's.)
//
// Bound by HBM: every weight byte is read once and meets 16 MT rows of A, so
// the kernel is a stream of weights from HBM through VGPRs to the matrix core.
//  * A workgroup takes 16 NT weight rows of one expert; its waves split K step by
//    step, so that together they read 128 kWaves contiguous bytes of a row, and
//    their sums meet in LDS at the end, in a fixed order.
//  * A step is 128 bytes of a row (128 K of FP8, 256 K of MXFP4): lane (r, g) =
//    (l % 16, l / 16) reads bytes 16 g and 64 + 16 g of row r of each tile, 64
//    contiguous bytes a row and load; the same order of K in A. Operands and
//    scales go through a ring of kDepth steps in VGPRs.
//  * Loads are range-checked buffer loads without a branch: rows past the
//    group's or N, steps past K and 32-element blocks past K read as zeros.
//  * A group with more than 16 MT rows takes further passes over the weights.
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
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
constexpr uint32_t kOOB = 0x80000000u;        // an offset past every buffer's range
constexpr int kWaves = 4, kThreads = 64 * kWaves;

struct Args {
  const uint8_t *A, *SA, *B, *SB;
  void* C;
  const int* offsets;  // null: dense
  int64_t ldc;
  int M, N, K;
};

// 8 E4M3 codes as bf16.
__device__ __forceinline__ bf16x8 expand8(int lo, int hi) {
  u32x4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, true));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, false));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, true));
  return __builtin_bit_cast(bf16x8, o);
}

// A lane's share of one step: 32 bytes of MT rows of A and NT of B, and the
// scales. FP8: s_A of the row (sa[m][0]), s_B (sb[0][0]). MXFP4: dwords 0 and 1
// hold the scales of the step's blocks 0..3 and 4..7 of the row.
template <int MT, int NT>
struct Step {
  i32x4 a[MT][2], b[NT][2];
  u32x2 sa[MT], sb[NT];
};

// ALIGNED: a row's MXFP4 scales start on dwords (K % 128 = 0).
template <bool FP8, bool EXACT, bool ALIGNED, int OUT, int MT, int NT, int DEPTH>
__global__ __launch_bounds__(kThreads) void gemm_few_rows_kernel(Args p) {
  __shared__ float part[kWaves][MT][NT][4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT), group = blockIdx.y;
  int lo = 0, hi = p.M;
  if (p.offsets) groups::rows_of(p.offsets, p.M, group, lo, hi);
  if (lo >= hi) return;

  const int nrows = min(p.N - n0, 16 * NT);
  const uint32_t rowbytes = (uint32_t)(FP8 ? p.K : p.K / 2);
  const int nk = (int)((rowbytes + 127) / 128);
  const int steps = (nk + kWaves - 1) / kWaves;  // of each wave
  // Scale bytes per row, and the weights' first scale.
  const uint32_t sstride = FP8 ? (uint32_t)(nk * 4) : (uint32_t)(p.K / 32);
  const int64_t brow = (int64_t)group * p.N + n0;
  const __amdgpu_buffer_rsrc_t rB = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.B + brow * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rSB =
      FP8 ? __builtin_amdgcn_make_buffer_rsrc(
                (void*)(p.SB + ((int64_t)group * ((p.N + 127) / 128) + n0 / 128) * sstride), 0, (int)sstride, kRsrcFlags)
          : __builtin_amdgcn_make_buffer_rsrc((void*)(p.SB + brow * sstride), 0, (int)((uint32_t)nrows * sstride), kRsrcFlags);

  for (int m0 = lo; m0 < hi; m0 += 16 * MT) {
    const int mrows = min(hi - m0, 16 * MT);
    const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.A + (int64_t)m0 * rowbytes), 0, (int)((uint32_t)mrows * rowbytes), kRsrcFlags);
    const __amdgpu_buffer_rsrc_t rSA = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.SA + (int64_t)m0 * sstride), 0, (int)((uint32_t)mrows * sstride), kRsrcFlags);

    // Two dwords of MXFP4 scales of a row at step s; bytes past the row's end
    // (they are another row's) do not matter, their codes being zeros, unless
    // they are NaN: those are left out.
    auto scales4 = [&](__amdgpu_buffer_rsrc_t rs, uint32_t row, int s, bool in) __attribute__((always_inline)) {
      const uint32_t off = row + (uint32_t)s * 8u;
      if (ALIGNED) {
        // (a row's last step may hold one dword of it: K % 256 = 128)
        const uint32_t x = __builtin_amdgcn_raw_buffer_load_b32(rs, in ? off : kOOB, 0, 0);
        const uint32_t y = __builtin_amdgcn_raw_buffer_load_b32(rs, in && s * 8 + 4 < (int)sstride ? off + 4u : kOOB, 0, 0);
        return u32x2{x, y};
      }
      // Bytes g and 4 + g, all that this lane uses.
      const uint32_t x = __builtin_amdgcn_raw_buffer_load_b8(rs, in && s * 8 + g < (int)sstride ? off + g : kOOB, 0, 0);
      const uint32_t y = __builtin_amdgcn_raw_buffer_load_b8(rs, in && s * 8 + 4 + g < (int)sstride ? off + 4u + g : kOOB, 0, 0);
      return u32x2{x << (8 * g), y << (8 * g)};
    };
    auto load = [&](Step<MT, NT>& q, int i) __attribute__((always_inline)) {
      const int s = i * kWaves + wave;
      const bool in = s < nk;
      const uint32_t k0 = (uint32_t)s * 128u + 16u * g, k1 = k0 + 64u;
#pragma unroll
      for (int t = 0; t < NT; t++) {
        const uint32_t row = (uint32_t)(16 * t + r) * rowbytes;
        q.b[t][0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rB, k0 < rowbytes ? row + k0 : kOOB, 0, 0));
        q.b[t][1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rB, k1 < rowbytes ? row + k1 : kOOB, 0, 0));
        if (!FP8) q.sb[t] = scales4(rSB, (uint32_t)(16 * t + r) * sstride, s, in);
      }
      if (FP8) q.sb[0].x = __builtin_amdgcn_raw_buffer_load_b32(rSB, in ? (uint32_t)s * 4u : kOOB, 0, 0);
#pragma unroll
      for (int t = 0; t < MT; t++) {
        const uint32_t row = (uint32_t)(16 * t + r) * rowbytes;
        q.a[t][0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, k0 < rowbytes ? row + k0 : kOOB, 0, 0));
        q.a[t][1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, k1 < rowbytes ? row + k1 : kOOB, 0, 0));
        const uint32_t srow = (uint32_t)(16 * t + r) * sstride;
        if (FP8)
          q.sa[t].x = __builtin_amdgcn_raw_buffer_load_b32(rSA, in ? srow + (uint32_t)s * 4u : kOOB, 0, 0);
        else
          q.sa[t] = scales4(rSA, srow, s, in);
      }
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int j = 0; j < NT; j++) acc[i][j] = f32x4{0, 0, 0, 0};
    auto compute = [&](const Step<MT, NT>& q) __attribute__((always_inline)) {
      if constexpr (FP8) {
        const float sb = __builtin_bit_cast(float, q.sb[0].x);
#pragma unroll
        for (int i = 0; i < MT; i++) {
          const float f = __builtin_bit_cast(float, q.sa[i].x) * sb;
          const i32x8 av = {q.a[i][0].x, q.a[i][0].y, q.a[i][0].z, q.a[i][0].w,
                            q.a[i][1].x, q.a[i][1].y, q.a[i][1].z, q.a[i][1].w};
#pragma unroll
          for (int j = 0; j < NT; j++) {
            const i32x8 bv = {q.b[j][0].x, q.b[j][0].y, q.b[j][0].z, q.b[j][0].w,
                              q.b[j][1].x, q.b[j][1].y, q.b[j][1].z, q.b[j][1].w};
            f32x4 P = f32x4{0, 0, 0, 0};
            if (EXACT) {
#pragma unroll
              for (int h = 0; h < 4; h++)
                P = __builtin_amdgcn_mfma_f32_16x16x32_bf16(expand8(bv[2 * h], bv[2 * h + 1]),
                                                            expand8(av[2 * h], av[2 * h + 1]), P, 0, 0, 0);
            } else {
              P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, P, 0, 0, 0, 127, 0, 127);
            }
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][j][e] = __builtin_fmaf(P[e], f, acc[i][j][e]);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int i = 0; i < MT; i++) {
            const i32x8 av = {q.a[i][h].x, q.a[i][h].y, q.a[i][h].z, q.a[i][h].w, 0, 0, 0, 0};
            const int sa = (int)((q.sa[i][h] >> (8 * g)) & 0xFFu);
#pragma unroll
            for (int j = 0; j < NT; j++) {
              const i32x8 bv = {q.b[j][h].x, q.b[j][h].y, q.b[j][h].z, q.b[j][h].w, 0, 0, 0, 0};
              const int sb = (int)((q.sb[j][h] >> (8 * g)) & 0xFFu);
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc[i][j], 4, 4, 0, sb, 0, sa);
            }
          }
      }
    };

    Step<MT, NT> ring[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH - 1; d++) load(ring[d], d);
    for (int i = 0; i < steps; i += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; d++) {
        if (i + d >= steps) break;
        load(ring[(d + DEPTH - 1) % DEPTH], i + d + DEPTH - 1);
        compute(ring[d]);
      }
    }

    // The waves' sums, added in their order. acc[i][j][e] of lane (r, g) is row
    // 16 i + r, column 16 j + 4 g + e.
    if (m0 != lo) __syncthreads();  // (the last pass's sums have been read)
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) part[wave][i][j][e][lane] = acc[i][j][e];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < (MT * NT + kWaves - 1) / kWaves; u++) {
      const int ij = u * kWaves + wave, i = ij / NT, j = ij % NT;
      if (ij >= MT * NT) break;
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        v[e] = part[0][i][j][e][lane];
#pragma unroll
        for (int w = 1; w < kWaves; w++) v[e] += part[w][i][j][e][lane];
      }
      const int row = 16 * i + r, col = n0 + 16 * j + 4 * g;
      if (row >= mrows) continue;
      const int64_t at = (int64_t)(m0 + row) * p.ldc + col;
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
}

template <bool FP8, bool EXACT, bool ALIGNED, int OUT, int MT, int NT, int DEPTH>
hipError_t launch(const Args& p, int64_t groups, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 16 * NT - 1) / (16 * NT)), (unsigned)groups);
  return launch_kernel(&gemm_few_rows_kernel<FP8, EXACT, ALIGNED, OUT, MT, NT, DEPTH>, grid, kThreads, 0, s, p);
}

template <bool FP8, bool EXACT, bool ALIGNED, int OUT>
hipError_t dispatch(const Args& p, int64_t groups, int64_t per, hipStream_t s) {
  if (per <= 16) return launch<FP8, EXACT, ALIGNED, OUT, 1, 4, 3>(p, groups, s);
  if (per <= 32) return launch<FP8, EXACT, ALIGNED, OUT, 2, 4, 2>(p, groups, s);
  return launch<FP8, EXACT, ALIGNED, OUT, 4, 4, 2>(p, groups, s);
}

template <bool ALIGNED>
hipError_t mxfp4(const Args& p, int64_t groups, int64_t per, bool f32, hipStream_t s) {
  if (f32) return dispatch<false, false, ALIGNED, kOutF32>(p, groups, per, s);
  return dispatch<false, false, ALIGNED, kOutBF16>(p, groups, per, s);
}

}  // namespace

// fp32 results: accumulation chains of at most 48 matrix instructions or scale
// blocks, of 128 K, in a wave.
bool gemm_few_rows_fits(int64_t K, int out_dtype) {
  return out_dtype != kOutF32 || K <= (int64_t)48 * 128 * kWaves;
}

hipError_t gemm_few_rows(int fmt, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                         const void* b, const void* sb, const int32_t* offsets, int64_t groups,
                         int out_dtype, void* c, int64_t ldc, hipStream_t s) {
  const Args p{(const uint8_t*)a, (const uint8_t*)sa, (const uint8_t*)b, (const uint8_t*)sb, c, offsets,
               ldc, (int)M, (int)N, (int)K};
  const int64_t per = offsets ? (M + groups - 1) / groups : M;
  const int64_t g = offsets ? groups : 1;
  const bool f32 = out_dtype == kOutF32;
  if (fmt == kMXFP4) return K % 128 == 0 ? mxfp4<true>(p, g, per, f32, s) : mxfp4<false>(p, g, per, f32, s);
  return f32 ? dispatch<true, true, true, kOutF32>(p, g, per, s) : dispatch<true, false, true, kOutBF16>(p, g, per, s);
}

}  // namespace mx
