// A mixture-of-experts layer for a few tokens (decode), bf16 activations on quantized
// weights (MXFP4, FP8 under fp32 scales per 128 x 128, INT8 under a scale per row):
//   y_t = sum over j of w_tj down_e( silu(gate_e x_t) * up_e x_t ),  e = ids_tj.
//
// Bound by HBM: every weight of the experts that a token chose is read once, and meets
// at most 16 tokens at a time. Tokens of one expert are a group; up to 16 of them a
// pass; the (token, expert) pairs, sorted by expert and token, are the rows of h and of the
// partial results.
//  1. moe_up: workgroups of (pass, columns of the gate and up projections). Each finds
//     its pass from the ids by itself: a bit per token and expert in LDS, counted
//     and scanned. Those of the first columns write the passes down for what follows.
//     h = silu(gate) up in fp32, rounded to bf16, the activations' type, as the
//     matrix cores take it.
//  2. moe_down: workgroups of (pass, columns of the result): a row's partial result, fp32.
//  3. moe_combine: each token's partial results times their weights, in the ids' order.
//
// The products (1 and 2): 8 waves share a workgroup's K, in steps of 128 bytes of each
// weight row (256 K of MXFP4, 128 of the others), S consecutive steps a wave. A wave keeps
// the activations' fragments of its steps in VGPRs and runs tile by tile of 16 weight
// rows, whose codes go HBM -> LDS directly, whole lines, 8 rows a load, into a ring
// of D steps of the wave's own. Codes are expanded exactly to bf16; the sums are fp32. FP8 starts a
// step's sum from zero and adds it times the step's scale; MXFP4's scales are applied in the
// expansion, INT8's to the result. The waves' sums meet in LDS, in their order.
#include <type_traits>
#include <utility>

#include "bf16.h"
#include "fp8_encode.h"
#include "groups.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
using fp8::bf16x8;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
// Lane and scalar offsets past every buffer's range (256 rows of at most 2^22
// bytes); their sum is one too.
constexpr uint32_t kOOB = 0x80000000u, kScalarOOB = 0x40000000u;
constexpr int kNonTemporal = 2;                // cache policy of a load: streamed
constexpr int W = 8;                           // waves of a workgroup

// Where the parts of the workspace are: the number of passes, the passes, each slot's
// row (-1: no expert of this call's), h and the partial results.
struct Pass {
  int expert, row, rows, unused;  // first row, rows
};
struct Work {
  int* count;
  Pass* pass;
  int* row_of;
  uint16_t* h;
  float* part;
};

struct Args {
  const uint16_t* x;
  const int* ids;
  const float* weights;
  const uint8_t *up, *down;
  const void *up_scales, *down_scales;
  void* y;
  int64_t ldx, ldy;
  int tokens, top, experts, hidden, inter;
  Work w;
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

// 8 MXFP4 codes times 2^(E - 127) as bf16 (E = 255: NaN), E byte j of `scales`.
__device__ __forceinline__ bf16x8 expand_fp4(uint32_t q, uint32_t scales, int j) {
  uint32_t e = (j < 3 ? scales << (23 - 8 * j) : scales >> 1) & 0x7F800000u;
  e = e > 0x00400000u ? e : 0x00400000u;  // (E = 0: 2^-127, a subnormal)
  const float s = __builtin_bit_cast(float, e);
  u32x4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  return __builtin_bit_cast(bf16x8, o);
}

// 8 integers as bf16: their fp32 forms' high halves (8 bits are enough for each).
__device__ __forceinline__ bf16x8 expand_int8(uint32_t lo, uint32_t hi) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t q = i < 2 ? lo : hi;
    const int at = 16 * (i % 2);
    const uint32_t a = __builtin_bit_cast(uint32_t, (float)(int8_t)(q >> at));
    const uint32_t b = __builtin_bit_cast(uint32_t, (float)(int8_t)(q >> (at + 8)));
    o[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8, o);
}

// v or-ed over the four lanes of the same l % 16.
__device__ __forceinline__ uint32_t or_over_rows(uint32_t v) {
  auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = a[0] | a[1];
  a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return a[0] | a[1];
}

// Sums of one workgroup: rows of A (bf16; lane (r, g) supplies row r, whose bytes
// begin at lane offset `arow` of rA, or kOOB) times T tiles of 16 weight rows, K
// elements each. Tile t's codes begin at row tile_row(t) of view(t); the views end with
// the rows there are. `sum(t, column e)` of lane (r, g) of wave t % W, afterwards: row r,
// columns 4 g + e of tile t.
template <int FMT, bool ALIGNED, int S, int T, int D>
struct Stream {
  static constexpr bool FP4 = FMT == kMXFP4, FP8 = FMT == kFP8B128X128;
  static constexpr int kSlot = 2048, kRing = W * D * kSlot, kSums = W * T * 4 * 64 * 4;
  static constexpr int kSmem = kRing > kSums ? kRing : kSums;
  static constexpr int kFrags = FP4 ? 8 : 4;  // MFMAs of a step, of 32 K each

  template <class View, class ScaleView, class TileRow, class Fp8Row>
  static __device__ __forceinline__ void run(uint8_t* smem, int K, __amdgpu_buffer_rsrc_t rA, uint32_t arow, View view,
                                             ScaleView sview, TileRow tile_row, Fp8Row fp8_row) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const uint32_t rowbytes = (uint32_t)(FP4 ? K / 2 : K);
    const int nk = (int)((rowbytes + 127) / 128);
    const uint32_t sstride = (uint32_t)(K / 32);  // MXFP4: scale bytes per row
    // Lane offsets within a tile for the weights' loads (row l / 8 + 8 h, the chunk that
    // belongs into slot l % 8); in a row's last step, chunks past its end are left out.
    const uint32_t left = rowbytes - 128u * (uint32_t)(nk - 1);
    uint32_t vb[2], vb_last[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t cb = 16u * (uint32_t)((lane & 7) ^ (4 * h + (lane >> 4)));
      vb[h] = (uint32_t)(8 * h + (lane >> 3)) * rowbytes + cb;
      vb_last[h] = cb < left ? vb[h] : kOOB;
    }
    const uint32_t soff = (uint32_t)r * sstride;
    const int chunks = (nk + W * S - 1) / (W * S);
    uint8_t* ring = smem + wave * (D * kSlot);
    // MFMA j takes the step's elements 32 j .. 32 j + 31, lane (r, g) 8 of row r from
    // 32 j + 8 g on: of A 64 bytes of each row together in one load, of the codes 4 (MXFP4) or 8 bytes
    // at an address of slots that j changes in its own bits only.
    const int frag = FP4 ? r * 128 + ((r >> 1) & 7) * 16 + 4 * g : r * 128 + (((r >> 1) & 7) ^ (g >> 1)) * 16 + 8 * (g & 1);
    const uint32_t alane = arow == kOOB ? kOOB : arow + 16u * (uint32_t)g;
    const uint32_t alane_half = g < 2 ? alane : kOOB;  // INT8: K may end in the middle of 32

    // MXFP4: the scales of step s's 8 blocks, without the bytes past the row's end, which are
    // another row's.
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
      return u32x2{x << (8 * g), y << (8 * g)};  // (of the lanes of a row together)
    };

    f32x4 acc[T];
#pragma unroll
    for (int j = 0; j < T; j++) acc[j] = f32x4{0, 0, 0, 0};

    for (int c = 0; c < chunks; c++) {
      const int s0 = (c * W + wave) * S;
      // The ring's first weights, then A of all S steps, then (FP8) the weights' scales.
      u32x2 wsc[D];  // MXFP4: the ring's scales
      auto load = [&](int k) __attribute__((always_inline)) {
        const int t = k / S, s = s0 + k % S;
        const int so = s < nk ? (int)(tile_row(t) * rowbytes + (uint32_t)s * 128u) : (int)kScalarOOB;
#pragma unroll
        for (int h = 0; h < 2; h++)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(view(t), (lds_ptr_t)(ring + (k % D) * kSlot + h * 1024), 16,
                                                   s < nk - 1 ? vb[h] : vb_last[h], so, 0, kNonTemporal);
        if (FP4) wsc[k % D] = load_scales(sview(t), tile_row(t) * sstride, s);
      };
#pragma unroll
      for (int k = 0; k < D - 1; k++)
        if (k < T * S) load(k);
      // A's fragments. (The step and MFMA go into the scalar offset.)
      u32x4 a[S][kFrags];
#pragma unroll
      for (int s = 0; s < S; s++)
#pragma unroll
        for (int i = 0; i < kFrags; i++) {
          const int k = ((s0 + s) * kFrags + i) * 32;
          a[s][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rA, FMT != kINT8 || k + 32 <= K ? alane : alane_half, k < K ? k * 2 : (int)kScalarOOB, 0));
        }
      float sb[T];
      if (FP8) {
#pragma unroll
        for (int t = 0; t < T; t++) {
          const float* p = fp8_row(t);  // null: a tile past the end
          sb[t] = p && s0 + lane < nk ? p[s0 + lane] : 0.0f;
        }
      }
      // Step k + 1's fragments are read before step k's MFMAs. Loads end in
      // order: step k + 1's have arrived when only the later steps' are out
      // (the first time, A's too, which came last).
      constexpr int kLoads = FP4 ? (ALIGNED ? 3 : 4) : 2;  // of a step
      auto arrived = [&](auto n) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"i"(decltype(n)::value) : "memory");
        __builtin_amdgcn_sched_barrier(0);
      };
      struct Codes {
        uint32_t q[8];
      };
      auto read = [&](int k) __attribute__((always_inline)) {
        const uint8_t* at = ring + (k % D) * kSlot;
        Codes c;
#pragma unroll
        for (int j = 0; j < kFrags; j++) {
          if constexpr (FP4) {
            c.q[j] = *(const uint32_t*)(at + (frag ^ (16 * j)));
          } else {
            const u32x2 v = *(const u32x2*)(at + (frag ^ (32 * j)));
            c.q[2 * j] = v.x;
            c.q[2 * j + 1] = v.y;
          }
        }
        return c;
      };
      arrived(std::integral_constant<int, 0>{});
      Codes next = read(0);
      unroll<T * S>([&](auto kk) __attribute__((always_inline)) {
        constexpr int k = decltype(kk)::value, t = k / S, s = k % S;
        const Codes bv = next;
        u32x2 wscale = wsc[k % D];
        if (k + D - 1 < T * S) load(k + D - 1);
        if constexpr (k + 1 < T * S) {
          // Steps loaded behind k + 1 (the first D - 1 have all arrived).
          constexpr int last = k + D - 1 < T * S ? k + D - 1 : T * S - 1;
          constexpr int behind = last - (k + 1);
          if constexpr (k + 1 >= D - 1) arrived(std::integral_constant<int, behind * kLoads>{});
          next = read(k + 1);
        }
        f32x4 P = FP8 ? f32x4{0, 0, 0, 0} : acc[t];
        if (FP4 && !ALIGNED) wscale = u32x2{or_over_rows(wscale.x), or_over_rows(wscale.y)};
#pragma unroll
        for (int j = 0; j < kFrags; j++) {
          bf16x8 w;
          if constexpr (FP4)
            w = expand_fp4(bv.q[j], wscale[j / 4], j % 4);
          else
            w = FP8 ? fp8::expand8((int)bv.q[2 * j], (int)bv.q[2 * j + 1]) : expand_int8(bv.q[2 * j], bv.q[2 * j + 1]);
          P = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, a[s][j]), P, 0, 0, 0);
        }
        if constexpr (FP8) {
          const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sb[t]), s));
#pragma unroll
          for (int e = 0; e < 4; e++) acc[t][e] = __builtin_fmaf(P[e], f, acc[t][e]);
        } else {
          acc[t] = P;
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    __syncthreads();  // (every ring has been read)
    float(*part)[T][4][64] = (float(*)[T][4][64])smem;
#pragma unroll
    for (int j = 0; j < T; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) part[wave][j][e][lane] = acc[j][e];
    __syncthreads();
  }

  // Tile j's sums over the waves, of this lane.
  static __device__ __forceinline__ f32x4 sum(const uint8_t* smem, int j) {
    const float(*part)[T][4][64] = (const float(*)[T][4][64])smem;
    const int lane = threadIdx.x & 63;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      v[e] = part[0][j][e][lane];
#pragma unroll
      for (int w = 1; w < W; w++) v[e] += part[w][j][e][lane];
    }
    return v;
  }
};

// Pass `want` of the ids' (kMoeMaxExperts words of LDS: the tokens of each expert): its expert, rows
// before it, rows, and its tokens with all of their expert's (`skip` of these come first);
// false: there is none. `passes`: how many there are.
__device__ __forceinline__ bool route(const Args& p, unsigned long long* tokens_of, int want, Pass& pass,
                                      unsigned long long& tokens, int& skip, int& passes) {
  const int tid = threadIdx.x, lane = tid & 63, slots = p.tokens * p.top;
  for (int i = tid; i < p.experts; i += 64 * W) tokens_of[i] = 0;
  __syncthreads();
  for (int i = tid; i < slots; i += 64 * W) {
    const int id = p.ids[i];
    if (id >= 0 && id < p.experts) atomicOr(&tokens_of[id], 1ull << (i / p.top));
  }
  __syncthreads();
  bool found = false;
  int rows0 = 0;
  passes = 0;
  for (int c = 0; c < p.experts; c += 64) {
    const unsigned long long m = c + lane < p.experts ? tokens_of[c + lane] : 0;
    const int n = __builtin_popcountll(m);
    // Rows and passes up to this lane's expert, in one scan.
    const int upto = groups::wave_scan(n << 16 | (n + 15) / 16);
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (!found && want < passes + (all & 0xFFFF)) {
      const int l = __builtin_ctzll(__ballot(passes + (upto & 0xFFFF) > want));
      const int before = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0;
      const int own = __builtin_amdgcn_readlane(n, l);
      skip = (want - passes - (before & 0xFFFF)) * 16;
      pass = {c + l, rows0 + (before >> 16) + skip, min(own - skip, 16), 0};
      tokens = (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)m, l) |
               (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(m >> 32), l) << 32;
      found = true;
    }
    passes += all & 0xFFFF;
    rows0 += all >> 16;
  }
  return found;
}

// (Said to be the same in all lanes, for the compiler to keep it in scalars.)
__device__ __forceinline__ void uniform(Pass& p) {
  p.expert = __builtin_amdgcn_readfirstlane(p.expert);
  p.row = __builtin_amdgcn_readfirstlane(p.row);
  p.rows = __builtin_amdgcn_readfirstlane(p.rows);
}

// T: tiles, of the gate's and the up projection's rows in turn.
template <int FMT, bool ALIGNED, int S, int T, int D>
__global__ __launch_bounds__(64 * W) void moe_up_kernel(Args p) {
  using St = Stream<FMT, ALIGNED, S, T, D>;
  constexpr int kMask = kMoeMaxExperts * 8;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[St::kSmem > kMask ? St::kSmem : kMask];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  Pass pass;
  unsigned long long tokens;
  int skip, passes;
  const bool some = route(p, (unsigned long long*)smem, blockIdx.y, pass, tokens, skip, passes);
  if (blockIdx.x == 0 && wave == 0) {
    // The passes, for the kernels that follow.
    if (blockIdx.y == 0) {
      if (lane == 0) *p.w.count = passes;
      for (int i = lane; i < p.tokens * p.top; i += 64)
        if (p.ids[i] < 0 || p.ids[i] >= p.experts) p.w.row_of[i] = -1;
    }
    if (some) {
      if (lane == 0) p.w.pass[blockIdx.y] = pass;
      const int at = __builtin_popcountll(tokens & ((1ull << lane) - 1)) - skip;
      if ((tokens >> lane & 1) && at >= 0 && at < pass.rows)
        for (int j = 0; j < p.top; j++)
          if (p.ids[lane * p.top + j] == pass.expert) p.w.row_of[lane * p.top + j] = pass.row + at;
    }
  }
  if (!some) return;
  uniform(pass);
  __syncthreads();  // (the masks have been read)

  const int K = p.hidden, I = p.inter, i0 = blockIdx.x * (8 * T);
  // Lane (r, g)'s token: the one of rank skip + r.
  for (int i = 0; i < skip + r; i++) tokens &= tokens - 1;
  const uint32_t arow = r < pass.rows ? (uint32_t)__builtin_ctzll(tokens) * (uint32_t)p.ldx * 2u : kOOB;
  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)p.x, 0, (int)(((uint32_t)(p.tokens - 1) * (uint32_t)p.ldx + (uint32_t)K) * 2u), kRsrcFlags);
  const uint32_t rowbytes = (uint32_t)(FMT == kMXFP4 ? K / 2 : K), sstride = (uint32_t)(K / 32);
  const int nrows = min(I - i0, 8 * T);
  const int64_t row0 = (int64_t)pass.expert * 2 * I + i0;
  __amdgpu_buffer_rsrc_t rB[2], rS[2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    rB[u] = __builtin_amdgcn_make_buffer_rsrc((void*)(p.up + (row0 + (int64_t)u * I) * rowbytes), 0,
                                              (int)((uint32_t)nrows * rowbytes), kRsrcFlags);
    rS[u] = __builtin_amdgcn_make_buffer_rsrc((void*)((const uint8_t*)p.up_scales + (FMT == kMXFP4 ? (row0 + (int64_t)u * I) * sstride : 0)), 0,
                                              FMT == kMXFP4 ? (int)((uint32_t)nrows * sstride) : 0, kRsrcFlags);
  }
  St::run(
      smem, K, rA, arow, [&](int t) { return rB[t % 2]; }, [&](int t) { return rS[t % 2]; }, [&](int t) { return (uint32_t)(t / 2 * 16); },
      [&](int t) {
        // (I is a multiple of 128: a tile has one row of scales.)
        const int64_t row = i0 + t / 2 * 16 + (int64_t)(t % 2) * I;
        return t / 2 * 16 < nrows ? (const float*)p.up_scales + ((int64_t)pass.expert * (2 * I / 128) + row / 128) * (K / 128) : nullptr;
      });
#pragma unroll
  for (int u = 0; u < (T / 2 + W - 1) / W; u++) {
    const int j = u * W + wave, col = i0 + 16 * j + 4 * g;
    if (j >= T / 2 || 16 * j >= nrows || r >= pass.rows) break;
    f32x4 gate = St::sum(smem, 2 * j), up = St::sum(smem, 2 * j + 1);
    if (FMT == kINT8) {
      const float* s = (const float*)p.up_scales + (int64_t)pass.expert * 2 * I + col;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        gate[e] *= s[e];
        up[e] *= s[I + e];
      }
    }
    float h[4];
#pragma unroll
    for (int e = 0; e < 4; e++) h[e] = gate[e] / (1.0f + expf(-gate[e])) * up[e];
    *(u32x2*)(p.w.h + (int64_t)(pass.row + r) * I + col) = u32x2{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
  }
}

template <int FMT, bool ALIGNED, int S, int T, int D>
__global__ __launch_bounds__(64 * W) void moe_down_kernel(Args p) {
  using St = Stream<FMT, ALIGNED, S, T, D>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[St::kSmem];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  if ((int)blockIdx.y >= *p.w.count) return;
  Pass pass = p.w.pass[blockIdx.y];
  uniform(pass);
  const int K = p.inter, N = p.hidden, n0 = blockIdx.x * (16 * T);
  const __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.w.h + (int64_t)pass.row * K), 0, (int)((uint32_t)(pass.rows * K) * 2u), kRsrcFlags);
  const uint32_t rowbytes = (uint32_t)(FMT == kMXFP4 ? K / 2 : K), sstride = (uint32_t)(K / 32);
  const int nrows = min(N - n0, 16 * T);
  const int64_t row0 = (int64_t)pass.expert * N + n0;
  const __amdgpu_buffer_rsrc_t rB =
      __builtin_amdgcn_make_buffer_rsrc((void*)(p.down + row0 * rowbytes), 0, (int)((uint32_t)nrows * rowbytes), kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rS = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const uint8_t*)p.down_scales + (FMT == kMXFP4 ? row0 * sstride : 0)), 0, FMT == kMXFP4 ? (int)((uint32_t)nrows * sstride) : 0, kRsrcFlags);
  St::run(
      smem, K, rA, r < pass.rows ? (uint32_t)(r * K) * 2u : kOOB, [&](int) { return rB; }, [&](int) { return rS; },
      [&](int t) { return (uint32_t)(t * 16); },
      [&](int t) {
        return t * 16 < nrows ? (const float*)p.down_scales + ((int64_t)pass.expert * ((N + 127) / 128) + (n0 + t * 16) / 128) * (K / 128) : nullptr;
      });
#pragma unroll
  for (int u = 0; u < (T + W - 1) / W; u++) {
    const int j = u * W + wave, col = n0 + 16 * j + 4 * g;
    if (j >= T || 16 * j >= nrows || r >= pass.rows) break;
    f32x4 v = St::sum(smem, j);
    if (FMT == kINT8) {
      const float* s = (const float*)p.down_scales + (int64_t)pass.expert * N + col;
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] *= s[e];
    }
    *(f32x4*)(p.w.part + (int64_t)(pass.row + r) * N + col) = v;
  }
}

template <int OUT>
__global__ __launch_bounds__(256) void moe_combine_kernel(Args p) {
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
  if (n >= p.hidden) return;
  f32x4 y = {0, 0, 0, 0};
  for (int j = 0; j < p.top; j++) {
    const int row = p.w.row_of[t * p.top + j];
    if (row < 0) continue;
    const f32x4 v = *(const f32x4*)(p.w.part + (int64_t)row * p.hidden + n);
    const float w = p.weights[t * p.top + j];
#pragma unroll
    for (int e = 0; e < 4; e++) y[e] = __builtin_fmaf(w, v[e], y[e]);
  }
  if (OUT == kOutF32)
    *(f32x4*)((float*)p.y + t * p.ldy + n) = y;
  else
    *(u32x2*)((uint16_t*)p.y + t * p.ldy + n) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

int64_t align(int64_t n) { return (n + 255) / 256 * 256; }

// Passes that any ids can need.
int64_t most_passes(int64_t slots, int64_t experts) { return groups::max_row_tiles(slots, experts, 16); }

template <int FMT, bool UP, int S, int T, int D>
hipError_t launch(const Args& p, hipStream_t s) {
  const int64_t tiles = UP ? (p.inter + 8 * T - 1) / (8 * T) : (p.hidden + 16 * T - 1) / (16 * T);
  const dim3 grid((unsigned)tiles, (unsigned)most_passes((int64_t)p.tokens * p.top, p.experts));
  const int K = UP ? p.hidden : p.inter;
  if constexpr (UP) {
    if (FMT == kMXFP4 && K % 128 != 0) return launch_kernel(&moe_up_kernel<FMT, false, S, T, D>, grid, 64 * W, 0, s, p);
    return launch_kernel(&moe_up_kernel<FMT, true, S, T, D>, grid, 64 * W, 0, s, p);
  } else {
    if (FMT == kMXFP4 && K % 128 != 0) return launch_kernel(&moe_down_kernel<FMT, false, S, T, D>, grid, 64 * W, 0, s, p);
    return launch_kernel(&moe_down_kernel<FMT, true, S, T, D>, grid, 64 * W, 0, s, p);
  }
}

template <int FMT>
hipError_t run(const Args& p, int out_dtype, hipStream_t s) {
  MX_TRY((launch<FMT, true, 1, 2, 3>(p, s)));
  MX_TRY((launch<FMT, false, 1, 2, 3>(p, s)));
  const dim3 grid((unsigned)((p.hidden + 1023) / 1024), (unsigned)p.tokens);
  if (out_dtype == kOutF32) return launch_kernel(&moe_combine_kernel<kOutF32>, grid, 256, 0, s, p);
  return launch_kernel(&moe_combine_kernel<kOutBF16>, grid, 256, 0, s, p);
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t top, int64_t experts, int64_t hidden, int64_t inter) {
  const int64_t slots = tokens * top;
  return (size_t)(256 + align(most_passes(slots, experts) * (int64_t)sizeof(Pass)) + align(slots * 4) + align(slots * inter * 2) +
                  align(slots * hidden * 4));
}

hipError_t moe(int fmt, int64_t tokens, int64_t top, int64_t experts, int64_t hidden, int64_t inter, const void* x, int64_t ldx,
               const int32_t* ids, const float* weights, const void* up, const void* up_scales, const void* down,
               const void* down_scales, int out_dtype, void* y, int64_t ldy, void* workspace, hipStream_t s) {
  const int64_t slots = tokens * top;
  uint8_t* at = (uint8_t*)workspace;
  auto take = [&](int64_t bytes) {
    uint8_t* r = at;
    at += align(bytes);
    return r;
  };
  Work w;
  w.count = (int*)take(4);
  w.pass = (Pass*)take(most_passes(slots, experts) * (int64_t)sizeof(Pass));
  w.row_of = (int*)take(slots * 4);
  w.h = (uint16_t*)take(slots * inter * 2);
  w.part = (float*)take(slots * hidden * 4);
  const Args p{(const uint16_t*)x, ids, weights, (const uint8_t*)up, (const uint8_t*)down, up_scales, down_scales, y, ldx, ldy,
               (int)tokens, (int)top, (int)experts, (int)hidden, (int)inter, w};
  if (fmt == kMXFP4) return run<kMXFP4>(p, out_dtype, s);
  if (fmt == kFP8B128X128) return run<kFP8B128X128>(p, out_dtype, s);
  return run<kINT8>(p, out_dtype, s);
}

}  // namespace mx
