// A mixture-of-experts layer for a few tokens (decode), bf16 activations on quantized
// weights (MXFP4, FP8 under fp32 scales per 128 x 128, INT8 under a scale per row):
//   y_t = sum over j of w_tj down_e( silu(gate_e x_t) * up_e x_t ),  e = ids_tj.
//
// Bound by HBM: every weight of the experts that a token chose is read once for each 16 of the
// tokens that chose it. Tokens of one expert are a group; up to 16 of them a
// pass; the (token, expert) pairs, sorted by expert and token, are the rows of h and of the
// partial results.
//  1. moe_up: h = silu(gate) up, in fp32, written as two bf16 numbers for the matrix cores, the nearest
//     and what is left. (One alone, a rounding of 2^-8 of each element, put bf16 results 2.4e-3 from 64
//     bits, which their own rounding puts 1.7e-3 from it, and fp32 results as far.) Each workgroup finds
//     the passes from the ids by itself: a bit per token and expert in LDS, counted and scanned. Those
//     with a pass's first columns write it down for what follows, and each what its like of moe_down
//     begins with (which would else find that from the number of passes and its pass, one load after the
//     other: 0.7 us), once its own first loads are out.
//  2. moe_down: the rows' partial results, fp32.
//  3. moe_combine: each token's partial results times their weights, in the ids' order. (In moe_down,
//     by the last pass to be done with a column: no faster, as XCDs see each other's results only past
//     their L2s. One token, 8 of 32 experts of 4096 x 2048, both then 31 us; 4 tokens 48 so, 45 with a launch.)
//
// The products (1 and 2): 8 waves share a workgroup's K, in steps of 128 bytes of each
// weight row (256 K of MXFP4, 128 of the others), S steps a wave. A wave keeps
// the activations' fragments of its steps in VGPRs and runs tile by tile of 16 weight
// rows, whose codes go HBM -> LDS directly, whole lines, 8 rows a load, into a ring
// of D steps of the wave's own. Codes are expanded exactly to bf16; the sums are fp32. FP8 starts a
// step's sum from zero and adds it times the step's scale; MXFP4's scales are applied in the
// expansion, INT8's to the result. The waves' sums meet in LDS, in their order.
//
// Measured in us, experts of 4096 x 2048 (gate and up + down + combine, traced): MXFP4, one token, 8 experts, 17 + 9 +
// 3 (at 6.56 TB/s, a large copy's rate, its weights would take 11 + 5.5; each launch is about 3 us short of that
// rate); 64 tokens, all of 64 experts, 110 + 59 + 5 (5.2 and 4.8 TB/s of codes and scales; h in one part 107 + 55; 61
// experts so 98 + 56, without the expansion the same, without sums and results 92 + 48); INT8, 32 tokens, 46 experts, 118
// + 63 + 5 (6.7 and 6.3 TB/s). Rows of several rounds, whole layers: FP8, 4 tokens, 11 of 16 experts of 5120 x 5120 198
// (132 at that rate), 14 of 32 of 7168 x 2048 126 (91); INT8, 11 of 16 of 5120 x 5120 201 (132): a second round of S = 4 steps
// a wave has little to do, and each round waits for all loads before it begins.
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
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
using fp8::bf16x8;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kRsrcFlags = 0x00020000u;  // raw buffer, gfx9 data format
// Lane and scalar offsets past every view's range (at most 2^30 bytes). A lane's offset of
// kOOB and a scalar one of kScalarOOB past a view's last row do not meet: their sum may wrap.
constexpr uint32_t kOOB = 0x80000000u, kScalarOOB = 0x40000000u;
constexpr int kNonTemporal = 2;                // cache policy of a load: streamed
constexpr int W = 8;                           // waves of a workgroup

// Where the parts of the workspace are: what each workgroup of moe_down begins with, the passes, each slot's
// row (of ids of experts), h and the partial results.
struct Pass {
  int expert, row, rows, unused;  // first row, rows
};
struct Share {
  int at, end, pass, col;  // of columns of 16 of all passes, one after the other; pass and column of `at`
};
struct Begin {
  Share share;
  Pass pass;
};
struct Work {
  Begin* begin;
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

// 8 MXFP4 codes times 2^(E - 127) as bf16 (E = 255: NaN), E in `scale`'s bits 30:23. The scaled
// converts read nothing else of their scale (checked for every E, 0 and 255 among them, with
// any sign and significand), so what lies beside E may stay.
__device__ __forceinline__ bf16x8 expand_fp4(uint32_t q, uint32_t scale) {
  const float s = __builtin_bit_cast(float, scale);
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

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A view of memory that is the same in all lanes, said so for the compiler to keep it in scalars (with
// views in VGPRs it loops over the lanes' at each load: 102 -> 99 us of a gate and up product of 64 tokens).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t view(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  const uint64_t u = (uint64_t)(uint32_t)uniform((int)(uint32_t)b) | (uint64_t)(uint32_t)uniform((int)(b >> 32)) << 32;
  return __builtin_amdgcn_make_buffer_rsrc((void*)u, 0, uniform((int)bytes), kRsrcFlags);
}

// A number as two in bf16: the nearest (or, next to fp32's largest, the largest), as bits, and what is left. Their sum is
// within 2^-17 of it: what is left is at most half a step of the first, exactly, and is rounded by half of its own.
struct Split {
  uint32_t high;
  float low;
};
__device__ __forceinline__ Split split(float v) {
  const bool finite = __builtin_fabsf(v) < __builtin_inff();
  uint32_t high = bf16_bits(v);
  if (finite && (high & 0x7FFFu) == 0x7F80u) high = __builtin_bit_cast(uint32_t, v) >> 16;
  return {high, finite ? v - __builtin_bit_cast(float, high << 16) : 0.0f};
}

// Lane (r, g)'s value from lane ((r + 8) % 16, g).
__device__ __forceinline__ float row_plus8(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128 /* row_ror:8 */, 0xF, 0xF, false));
}

// What a workgroup does of one pass: `n` tiles of 16 weight rows, tile t of kind t % KINDS (the
// gate's and the up projection's rows) from row 16 (t / KINDS) of its kind's view on. The views end
// with the tiles there are. A's view and lane (r, g)'s row's first byte in it (kOOB: no such row).
// Scales: MXFP4 a view of the tiles' rows, FP8 of all scales of the expert's kind, the views' first
// row being row `row0` there.
template <int KINDS>
struct Segment {
  __amdgpu_buffer_rsrc_t rA, rB[KINDS], rS[KINDS];
  uint32_t arow;
  int n, row0;
  Pass pass;
};

// The products of a workgroup: its segments' rows of A (bf16) times their weight rows, K elements
// each. Wave w takes the K steps w, w + W, ..., S of them; a row of more than W S steps takes several
// rounds (MULTI). next(segment) gives one segment after the other, false behind the last. opened() is called
// when its first loads are on their way, or there is none.
// G tiles at a time, done(segment, first tile, sums) is called with the waves' sums in LDS,
// sums[wave][tile][lane]: lane (r, g)'s row r, columns 4 g .. 4 g + 3 of the tile.
// PARTS: 1, or 2 where a row of A holds K numbers' high parts and then their low ones (split), which
// take registers and matrix instructions of their own.
template <int FMT, bool ALIGNED, int KINDS, int S, bool MULTI, int PARTS>
struct Stream {
  static constexpr bool FP4 = FMT == kMXFP4, FP8 = FMT == kFP8B128X128;
  // (D = 6, with which G is 4 or 6: 2 to 6% slower. S = 4 leaves VGPRs for the sums of 4 tiles.)
  static constexpr int D = 4, G = S == 4 ? 4 : 8;
  static constexpr int kSlot = 2048, kRing = W * D * kSlot, kSums = W * G * 1024, kSmem = kRing + kSums;
  static constexpr int kFrags = FP4 ? 8 : 4;  // MFMAs of a step, of 32 K each
  static constexpr int kLoads = FP4 ? (ALIGNED ? 3 : 4) : FP8 ? 3 : 2;  // of a tile's step
  static_assert(G * S % D == 0 && G % KINDS == 0, "the ring's slots and the tiles' kinds are those of a place in the group");
  using Seg = Segment<KINDS>;

  template <class Next, class Opened, class Done>
  static __device__ __forceinline__ void run(uint8_t* smem, int K, Next next_segment, Opened opened, Done done) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const uint32_t rowbytes = (uint32_t)(FP4 ? K / 2 : K);
    const int nk = (int)((rowbytes + 127) / 128);
    const uint32_t sstride = FP8 ? (uint32_t)(K / 128 * 4) : (uint32_t)(K / 32);  // scale bytes per row
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
    uint8_t* ring = smem + wave * (D * kSlot);
    f32x4(*sums)[G][64] = (f32x4(*)[G][64])(smem + kRing);
    // A lane's 32 bytes of the step: chunks g and g + 4 of its row.
    const int frag0 = r * 128 + ((g ^ (r >> 1)) & 7) * 16, frag1 = r * 128 + (((g + 4) ^ (r >> 1)) & 7) * 16;
    const uint32_t rot = (uint32_t)(8 * g + 9) & 31u;  // MXFP4: rotating right by it takes byte g to bits 30:23

    const int rounds = MULTI ? (nk + W * S - 1) / (W * S) : 1;
    int round = 0;
    auto step = [&](int i) __attribute__((always_inline)) { return (round * S + i) * W + wave; };
    Seg seg;
    // The scales of a tile's step: MXFP4's of blocks 0..3 and 4..7 (this lane uses byte g of
    // each dword, or, not ALIGNED, has only that), without the bytes past the row's end, which are
    // another row's and might be NaN; FP8's one.
    u32x2 wsc[D];
    auto load = [&](auto kk, int first) __attribute__((always_inline)) {
      // Place k from tile `first` on. (Tiles past the segment's last are past the views' ends.)
      constexpr int k = decltype(kk)::value, kind = k / S % KINDS;
      const int s = step(k % S);
      const uint32_t row = (uint32_t)(first / KINDS * 16 + k / S / KINDS * 16);
      const int so = (int)(row * rowbytes + (s < nk ? (uint32_t)s * 128u : kScalarOOB));
#pragma unroll
      for (int h = 0; h < 2; h++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(seg.rB[kind], (lds_ptr_t)(ring + (k % D) * kSlot + h * 1024), 16,
                                                 s != nk - 1 ? vb[h] : vb_last[h], so, 0, kNonTemporal);
      if (FP4) {
        const int at = (int)(row * sstride + (s < nk ? (uint32_t)s * 8u : kScalarOOB));
        if (ALIGNED) {
          wsc[k % D] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(seg.rS[kind], soff, at, 0));
        } else {
          const uint32_t b = (uint32_t)s * 8u + (uint32_t)g;
          wsc[k % D].x = __builtin_amdgcn_raw_buffer_load_b8(seg.rS[kind], b < sstride ? soff + g : kOOB, at, 0);
          wsc[k % D].y = __builtin_amdgcn_raw_buffer_load_b8(seg.rS[kind], b + 4u < sstride ? soff + 4u + g : kOOB, at, 0);
        }
      }
      if (FP8)
        wsc[k % D].x = __builtin_amdgcn_raw_buffer_load_b32(
            seg.rS[kind], 0, (int)(((uint32_t)seg.row0 + row) / 128u * sstride + (s < nk ? (uint32_t)s * 4u : kScalarOOB)), 0);
    };
    u32x4 a[PARTS][S][kFrags];  // (of lanes without a row: anything, for rows of the result that nobody reads)
    // A's fragments, then the ring's first weights. (The other way round A's loads wait for the weights'.)
    auto start = [&](int first) __attribute__((always_inline)) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (the ring is free)
#pragma unroll
      for (int n = 0; n < PARTS * S * kFrags; n++) {
        const int part = n / (S * kFrags), i = n / kFrags % S, j = n % kFrags;
        constexpr int kPer = kFrags / 2;  // 16-byte pieces of A that meet a 16-byte chunk of codes
        const uint32_t chunk = (uint32_t)(step(i) * 8 + j / kPer * 4 + g);
        a[part][i][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            seg.rA, chunk * 16u < rowbytes ? seg.arow + (uint32_t)g * (16u * kPer) : kOOB,
            part * 2 * K + (step(i) * 8 + j / kPer * 4) * (16 * kPer) + j % kPer * 16, 0));
      }
      __builtin_amdgcn_sched_barrier(0);
      unroll<D - 1>([&](auto kk) __attribute__((always_inline)) { load(kk, first); });
    };
    auto started = [&]() __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    struct Codes {
      u32x4 h[2];
    };
    auto read = [&](int k) __attribute__((always_inline)) {
      const uint8_t* at = ring + (k % D) * kSlot;
      return Codes{{*(const u32x4*)(at + frag0), *(const u32x4*)(at + frag1)}};
    };

    bool more = next_segment(seg);
    if (!more) return opened();
    if (!MULTI) start(0);
    while (more) {
      const int n = seg.n;
      const Pass pass = seg.pass;
      const int row0 = seg.row0;
      // (What comes next is found out beside the first loads.)
      opened();
      Seg after;
      more = next_segment(after);
      if (!MULTI) started();
      for (int first = 0; first < n; first += G) {
        f32x4 acc[G];
#pragma unroll
        for (int j = 0; j < G; j++) acc[j] = f32x4{0, 0, 0, 0};
        for (round = 0; round < rounds; round++) {
          if (MULTI) {
            start(first);
            started();
          }
          Codes next = read(0);
          unroll<G * S>([&](auto kk) __attribute__((always_inline)) {
            constexpr int k = decltype(kk)::value, t = k / S, i = k % S;
            if (first + t >= n) return;  // (the last group's)
            const Codes bv = next;
            u32x2 wscale = wsc[k % D];
            // Into the slot of the step before, which has been read. (MULTI: nothing past the group, as the next
            // start loads anew. Its scales would be unused, the compiler would leave their loads out, and the waits,
            // which count a step's loads, would end before they should.)
            constexpr int last = !MULTI || k + D - 1 < G * S ? k + D - 1 : G * S - 1;  // the last step loaded
            if constexpr (last == k + D - 1) load(std::integral_constant<int, last>{}, first);
            // Step k + 1's fragments are read before step k's MFMAs. Loads end in order: step k + 1's
            // have arrived when only the later steps' are out (and stores, if any, besides).
            if constexpr (last > k) {
              __builtin_amdgcn_sched_barrier(0);
              asm volatile("s_waitcnt vmcnt(%0)" ::"i"((last - (k + 1)) * kLoads) : "memory");
              __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (k + 1 < G * S) next = read(k + 1);
            f32x4 P = FP8 ? f32x4{0, 0, 0, 0} : acc[t];
            if (FP4 && ALIGNED && step(i) * 8 + 4 >= (int)sstride) wscale.y = 0;  // (K % 256 = 128)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const uint32_t scale = ALIGNED ? __builtin_amdgcn_alignbit(wscale[h], wscale[h], rot) : wscale[h] << 23;
#pragma unroll
              for (int j = 0; j < kFrags / 2; j++) {
                bf16x8 w;
                if constexpr (FP4)
                  w = expand_fp4(bv.h[h][j], scale);
                else
                  w = FP8 ? fp8::expand8((int)bv.h[h][2 * j], (int)bv.h[h][2 * j + 1]) : expand_int8(bv.h[h][2 * j], bv.h[h][2 * j + 1]);
#pragma unroll
                for (int part = 0; part < PARTS; part++)
                  P = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, a[part][i][h * (kFrags / 2) + j]), P, 0, 0, 0);
              }
            }
            if constexpr (FP8) {
              const float f = __builtin_bit_cast(float, wscale.x);
#pragma unroll
              for (int e = 0; e < 4; e++) acc[t][e] = __builtin_fmaf(P[e], f, acc[t][e]);
            } else {
              acc[t] = P;
            }
            __builtin_amdgcn_sched_barrier(0);
          });
        }
        round = 0;
        if (first + G >= n) {
          // The next segment's first loads, beside this one's last results.
          seg = after;
          if (!MULTI && more) start(0);
        }
        // (Every wave has done with the last group's sums: it has passed the barrier behind them.)
#pragma unroll
        for (int j = 0; j < G; j++) sums[wave][j][lane] = acc[j];
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        done(pass, row0, n, first, sums);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // The sums over the waves of tile j, of this lane; of its columns e, e + 1 of 4 only.
  static __device__ __forceinline__ f32x4 sum(const f32x4 (*sums)[G][64], int j) {
    const int lane = threadIdx.x & 63;
    f32x4 v = sums[0][j][lane];
#pragma unroll
    for (int w = 1; w < W; w++) v += sums[w][j][lane];
    return v;
  }
  static __device__ __forceinline__ f32x2 sum2(const f32x4 (*sums)[G][64], int j, int e) {
    const int lane = threadIdx.x & 63;
    f32x2 v = *((const f32x2*)&sums[0][j][lane] + e / 2);
#pragma unroll
    for (int w = 1; w < W; w++) v += *((const f32x2*)&sums[w][j][lane] + e / 2);
    return v;
  }
};

__device__ __forceinline__ void uniform(Pass& p) {
  p.expert = uniform(p.expert);
  p.row = uniform(p.row);
  p.rows = uniform(p.rows);
}

// The tokens of each expert as bits, from the ids, in LDS.
__device__ __forceinline__ void route(const Args& p, unsigned long long* tokens_of) {
  const int tid = threadIdx.x, slots = p.tokens * p.top;
  for (int i = tid; i < p.experts; i += 64 * W) tokens_of[i] = 0;
  __syncthreads();
  for (int i = tid; i < slots; i += 64 * W) {
    const int id = p.ids[i];
    if (id >= 0 && id < p.experts) atomicOr(&tokens_of[id], 1ull << (i / p.top));
  }
  __syncthreads();
}

// Rows and passes of experts c .. c + 63 up to this lane's, in one scan: rows << 16 | passes.
__device__ __forceinline__ int scan_passes(unsigned long long tokens) {
  const int n = __builtin_popcountll(tokens);
  return groups::wave_scan(n << 16 | (n + 15) / 16);
}

__device__ __forceinline__ int count_passes(const Args& p, const unsigned long long* tokens_of) {
  const int lane = threadIdx.x & 63;
  int passes = 0;
  for (int c = 0; c < p.experts; c += 64)
    passes += __builtin_amdgcn_readlane(scan_passes(c + lane < p.experts ? tokens_of[c + lane] : 0), 63) & 0xFFFF;
  return passes;
}

// Pass `want`, which there is, and its expert's tokens (`skip` of these come in passes before it).
__device__ __forceinline__ void find_pass(const Args& p, const unsigned long long* tokens_of, int want, Pass& pass,
                                          unsigned long long& tokens, int& skip) {
  const int lane = threadIdx.x & 63;
  int rows = 0;
  for (int c = 0; c < p.experts; c += 64) {
    const unsigned long long m = c + lane < p.experts ? tokens_of[c + lane] : 0;
    const int upto = scan_passes(m), all = __builtin_amdgcn_readlane(upto, 63);
    if (want >= (all & 0xFFFF)) {
      want -= all & 0xFFFF;
      rows += all >> 16;
      continue;
    }
    const int l = __builtin_ctzll(__ballot((upto & 0xFFFF) > want));
    const int before = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0;
    tokens = (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)m, l) |
             (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(m >> 32), l) << 32;
    skip = (want - (before & 0xFFFF)) * 16;
    pass = {c + l, rows + (before >> 16) + skip, min((int)__builtin_popcountll(tokens) - skip, 16), 0};
    break;
  }
  uniform(pass);
  skip = uniform(skip);
}

// What workgroup b does of `passes` passes over `cols` columns (of 16): all of them one after the
// other from `at` to `end`. An even share, which begins or ends within a pass, or, where that takes
// less time, a part of one pass: beginning with another pass costs about as much as kSwitch columns.
// (Always even: 17 tokens, 2 of 5 experts of 2880 x 1440, MXFP4 14.5 + 8.2 us, 12.4 + 7.0 so; always within a
// pass: 64 tokens, 61 experts of 4096 x 2048 108 + 63, 98 + 56 so.)
constexpr int kGrid = 256;  // workgroups: one a CU
constexpr int kSwitch = 2;
__device__ __forceinline__ Share share(int passes, int cols, int b) {
  Share s;
  const int all = passes * cols, each = kGrid / max(passes, 1), more = kGrid - passes * each;  // (all: at most 2^27)
  const int part = (cols + max(each, 1) - 1) / max(each, 1);
  if (each > 0 && part <= all / kGrid + 1 + kSwitch) {
    // `more` passes have a workgroup more than the others.
    const bool first = b < more * (each + 1);
    const int w = first ? each + 1 : each, i = first ? b : b - more * (each + 1), pass = i / w;
    const int n = first ? (cols + each) / (each + 1) : part;
    s.pass = (first ? 0 : more) + pass;
    s.col = min((i - pass * w) * n, cols);
    s.at = s.pass * cols + s.col;
    s.end = min(s.at + n, (s.pass + 1) * cols);
    if (s.pass >= passes) s.end = s.at;  // (no passes)
  } else {
    s.at = (int)((int64_t)all * b / kGrid);
    s.end = (int)((int64_t)all * (b + 1) / kGrid);
    s.pass = s.at / cols;
    s.col = s.at - s.pass * cols;
  }
  return {uniform(s.at), uniform(s.end), uniform(s.pass), uniform(s.col)};
}

// A view of a MXFP4 weight's scales, rows of K / 32 bytes from `row` on; of FP8 scales, `rows` / 128 blocks
// of rows of K / 128 from block row `row` on; else none.
template <int FMT>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_view(const void* scales, int64_t row, int rows, int K) {
  const int64_t stride = FMT == kMXFP4 ? K / 32 : FMT == kFP8B128X128 ? K / 128 * 4 : 0;
  return view((const uint8_t*)scales + row * stride, (uint32_t)rows * (uint32_t)stride);
}

template <int FMT, bool ALIGNED, int S, bool MULTI>
__global__ __launch_bounds__(64 * W, 2) void moe_up_kernel(Args p) {
  using St = Stream<FMT, ALIGNED, 2, S, MULTI, 1>;
  // One array for all. (With several the compiler waits for all loads under way before it reads any, as it can not
  // tell which array they go to.)
  __shared__ __attribute__((aligned(1024))) uint8_t smem[St::kSmem + kMoeMaxExperts * 8 + W * 64];
  unsigned long long* tokens_of = (unsigned long long*)(smem + St::kSmem);
  uint8_t(*token_at)[64] = (uint8_t(*)[64])(smem + St::kSmem + kMoeMaxExperts * 8);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  route(p, tokens_of);
  const int K = p.hidden, I = p.inter, cols = I / 16;
  const int passes = uniform(count_passes(p, tokens_of));
  const uint32_t rowbytes = (uint32_t)(FMT == kMXFP4 ? K / 2 : K);
  Share mine = share(passes, cols, blockIdx.x);
  // What is to be written down for the kernels that follow: the pass `opens` that this segment is the first of, with
  // its tokens; before the first one, what this workgroup of moe_down begins with.
  int opens = -1, opens_skip = 0;
  Pass opens_pass{};
  unsigned long long opens_tokens = 0;
  bool first_segment = true;
  auto next = [&](Segment<2>& seg) __attribute__((always_inline)) {
    if (mine.at >= mine.end) return false;
    const int u = mine.pass, c0 = mine.col, n = min(cols - c0, mine.end - mine.at);
    mine = {mine.at + n, mine.end, u + 1, 0};
    unsigned long long tokens = 0;
    int skip = 0;
    find_pass(p, tokens_of, u, seg.pass, tokens, skip);
    opens = c0 == 0 ? u : -1;
    opens_pass = seg.pass;
    opens_tokens = tokens;
    opens_skip = skip;
    const int rank = __builtin_popcountll(tokens & ((1ull << lane) - 1));
    const bool has = tokens >> lane & 1;
    // Row r's token is the one of rank skip + r.
    if (has) token_at[wave][rank] = (uint8_t)lane;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    seg.arow = r < seg.pass.rows ? (uint32_t)token_at[wave][skip + r] * (uint32_t)p.ldx * 2u : kOOB;
    seg.rA = view(p.x, ((uint32_t)(p.tokens - 1) * (uint32_t)p.ldx + (uint32_t)K) * 2u);
    seg.n = 2 * n;
    seg.row0 = c0 * 16;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int64_t row = ((int64_t)seg.pass.expert * 2 + k) * I + c0 * 16;
      seg.rB[k] = view(p.up + row * rowbytes, (uint32_t)(16 * n) * rowbytes);
      // (FP8: I is a multiple of 128, and so is each kind's first row.)
      if (FMT == kFP8B128X128)
        seg.rS[k] = scale_view<FMT>(p.up_scales, ((int64_t)seg.pass.expert * 2 + k) * (I / 128), I / 128, K);
      else
        seg.rS[k] = scale_view<FMT>(p.up_scales, row, 16 * n, K);
    }
    return true;
  };
  auto opened = [&]() __attribute__((always_inline)) {
    if (wave == 0 && opens >= 0) {
      const int rank = __builtin_popcountll(opens_tokens & ((1ull << lane) - 1)) - opens_skip;
      if (lane == 0) p.w.pass[opens] = opens_pass;
      if ((opens_tokens >> lane & 1) && rank >= 0 && rank < opens_pass.rows)
        for (int j0 = 0; j0 < p.top; j0 += 8) {
          int id[8];
#pragma unroll
          for (int j = 0; j < 8; j++) id[j] = p.ids[lane * p.top + min(j0 + j, p.top - 1)];
#pragma unroll
          for (int j = 0; j < 8; j++)
            if (j0 + j < p.top && id[j] == opens_pass.expert) p.w.row_of[lane * p.top + j0 + j] = opens_pass.row + rank;
        }
    }
    opens = -1;
    if (first_segment && wave == 1) {
      Begin b{share(passes, p.hidden / 16, blockIdx.x), Pass{}};
      unsigned long long tokens = 0;
      int skip = 0;
      if (b.share.at < b.share.end) find_pass(p, tokens_of, b.share.pass, b.pass, tokens, skip);
      if (lane == 0) p.w.begin[blockIdx.x] = b;
    }
    first_segment = false;
  };
  St::run(smem, K, next, opened, [&](const Pass& pass, int i0, int n, int first, const f32x4(*sums)[St::G][64]) __attribute__((always_inline)) {
    // Two columns of four of a pair of tiles a wave.
    const int j = wave / 2, e0 = wave % 2 * 2, col = i0 + 8 * first + 16 * j + 4 * g + e0;
    if (j >= St::G / 2 || first + 2 * j >= n || r >= pass.rows) return;
    f32x2 gate = St::sum2(sums, 2 * j, e0), up = St::sum2(sums, 2 * j + 1, e0);
    if (FMT == kINT8) {
      const float* s = (const float*)p.up_scales + (int64_t)pass.expert * 2 * I + col;
#pragma unroll
      for (int e = 0; e < 2; e++) {
        gate[e] *= s[e];
        up[e] *= s[I + e];
      }
    }
    Split h[2];
#pragma unroll
    for (int e = 0; e < 2; e++) h[e] = split(gate[e] / (1.0f + expf(-gate[e])) * up[e]);
    uint16_t* at = p.w.h + (int64_t)(pass.row + r) * 2 * I + col;
    *(uint32_t*)at = h[0].high | h[1].high << 16;
    *(uint32_t*)(at + I) = pack_bf16x2(h[0].low, h[1].low);
  });
}

// FEW: no pass has more than 8 rows. Their low parts are then A's rows 8 to 15, and the results of rows r and r + 8 are
// added: no more loads and products than h in one part takes (one token, 8 experts of 4096 x 2048, MXFP4, the layer 30.8
// -> 31.0 us). Else a lane's row has both, twice the loads of A and the products (64 tokens, all of 64 experts, 171.5 -> 179;
// 17 tokens, 2 of 5 of 2880 x 1440 23.0 -> 24.2; 32 tokens, INT8, 4 of 64 of 4096 x 2048 237 -> 239).
template <int FMT, bool ALIGNED, int S, bool MULTI, bool FEW>
__global__ __launch_bounds__(64 * W, 2) void moe_down_kernel(Args p) {
  using St = Stream<FMT, ALIGNED, 1, S, MULTI, FEW ? 1 : 2>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[St::kSmem];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int K = p.inter, N = p.hidden, cols = N / 16;
  const uint32_t rowbytes = (uint32_t)(FMT == kMXFP4 ? K / 2 : K);
  const Begin begin = p.w.begin[blockIdx.x];
  Share mine = {uniform(begin.share.at), uniform(begin.share.end), uniform(begin.share.pass), uniform(begin.share.col)};
  bool first_segment = true;
  auto next = [&](Segment<1>& seg) __attribute__((always_inline)) {
    if (mine.at >= mine.end) return false;
    const int u = mine.pass, c0 = mine.col, n = min(cols - c0, mine.end - mine.at);
    mine = {mine.at + n, mine.end, u + 1, 0};
    seg.pass = first_segment ? begin.pass : p.w.pass[u];
    first_segment = false;
    uniform(seg.pass);
    const int row = FEW ? r % 8 : r;
    seg.arow = row < seg.pass.rows ? (uint32_t)(row * K) * 4u + (row != r ? (uint32_t)K * 2u : 0u) : kOOB;
    seg.rA = view(p.w.h + (int64_t)seg.pass.row * 2 * K, (uint32_t)(seg.pass.rows * K) * 4u);
    seg.n = n;
    seg.row0 = c0 * 16;
    const int64_t row0 = (int64_t)seg.pass.expert * N + c0 * 16;
    seg.rB[0] = view(p.down + row0 * rowbytes, (uint32_t)(16 * n) * rowbytes);
    if (FMT == kFP8B128X128)
      seg.rS[0] = scale_view<FMT>(p.down_scales, (int64_t)seg.pass.expert * ((N + 127) / 128), (N + 127) / 128, K);
    else
      seg.rS[0] = scale_view<FMT>(p.down_scales, row0, 16 * n, K);
    return true;
  };
  St::run(smem, K, next, [] {}, [&](const Pass& pass, int n0, int n, int first, const f32x4(*sums)[St::G][64]) __attribute__((always_inline)) {
    const int col = n0 + 16 * (first + wave) + 4 * g;
    if (wave >= St::G || first + wave >= n) return;
    f32x4 v = St::sum(sums, wave);
    if (FEW) {
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] += row_plus8(v[e]);
    }
    if (r >= pass.rows) return;
    if (FMT == kINT8) {
      const float* s = (const float*)p.down_scales + (int64_t)pass.expert * N + col;
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] *= s[e];
    }
    *(f32x4*)(p.w.part + (int64_t)(pass.row + r) * N + col) = v;
  });
}

// Columns n .. n + 3 of token t's result: its partial results times their weights, in the ids' order.
template <int OUT>
__global__ __launch_bounds__(256) void moe_combine_kernel(Args p) {
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
  if (n >= p.hidden) return;
  f32x4 y = {0, 0, 0, 0};
  constexpr int kBatch = 8;  // partial results that are on their way together
  for (int j0 = 0; j0 < p.top; j0 += kBatch) {
    int row[kBatch];
    float w[kBatch];
    f32x4 v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; j++) {
      const int at = t * p.top + min(j0 + j, p.top - 1), id = p.ids[at], slot = p.w.row_of[at];
      row[j] = j0 + j < p.top && id >= 0 && id < p.experts ? slot : -1;
      w[j] = p.weights[at];
    }
#pragma unroll
    for (int j = 0; j < kBatch; j++) {
      v[j] = f32x4{0, 0, 0, 0};
      if (row[j] >= 0) v[j] = *(const f32x4*)(p.w.part + (int64_t)row[j] * p.hidden + n);
    }
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      if (row[j] >= 0)
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = __builtin_fmaf(w[j], v[j][e], y[e]);
  }
  if (OUT == kOutF32)
    *(f32x4*)((float*)p.y + t * p.ldy + n) = y;
  else
    *(u32x2*)((uint16_t*)p.y + t * p.ldy + n) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

int64_t align(int64_t n) { return (n + 255) / 256 * 256; }

// Passes that any ids can need.
int64_t most_passes(int64_t slots, int64_t experts) { return groups::max_row_tiles(slots, experts, 16); }

// FEW: of moe_down.
template <int FMT, bool UP, int S, bool MULTI, bool FEW>
hipError_t launch(const Args& p, hipStream_t s) {
  auto product = [&](auto aligned) {
    constexpr bool ALIGNED = decltype(aligned)::value;
    if constexpr (UP)
      return launch_kernel(&moe_up_kernel<FMT, ALIGNED, S, MULTI>, dim3(kGrid), 64 * W, 0, s, p);
    else
      return launch_kernel(&moe_down_kernel<FMT, ALIGNED, S, MULTI, FEW>, dim3(kGrid), 64 * W, 0, s, p);
  };
  if constexpr (FMT == kMXFP4) {
    if ((UP ? p.hidden : p.inter) % 128 != 0) return product(std::false_type{});
  }
  return product(std::true_type{});
}

// Steps a wave: as few as take a row's in one round, within the registers that A's fragments of them take (both
// parts of 4 steps of MXFP4: too many. In rounds of 2: 16 tokens, 2 of 8 experts of 4096 x 14336, 157 us; 154 with one
// part in rounds of 4).
template <int FMT, bool UP, bool FEW>
hipError_t by_length(const Args& p, hipStream_t s) {
  const int K = UP ? p.hidden : p.inter, nk = (K + (FMT == kMXFP4 ? 255 : 127)) / (FMT == kMXFP4 ? 256 : 128);
  if (nk <= W) return launch<FMT, UP, 1, false, FEW>(p, s);
  if (nk <= 2 * W) return launch<FMT, UP, 2, false, FEW>(p, s);
  if constexpr (FMT == kMXFP4 && !UP && !FEW) {
    return launch<FMT, UP, 2, true, FEW>(p, s);
  } else {
    if (nk <= 4 * W) return launch<FMT, UP, 4, false, FEW>(p, s);
    return launch<FMT, UP, 4, true, FEW>(p, s);
  }
}

template <int FMT>
hipError_t run(const Args& p, int out_dtype, hipStream_t s) {
  MX_TRY((by_length<FMT, true, false>(p, s)));
  if (p.tokens <= 8)
    MX_TRY((by_length<FMT, false, true>(p, s)));
  else
    MX_TRY((by_length<FMT, false, false>(p, s)));
  const dim3 grid((unsigned)((p.hidden + 1023) / 1024), (unsigned)p.tokens);
  if (out_dtype == kOutF32) return launch_kernel(&moe_combine_kernel<kOutF32>, grid, 256, 0, s, p);
  return launch_kernel(&moe_combine_kernel<kOutBF16>, grid, 256, 0, s, p);
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t top, int64_t experts, int64_t hidden, int64_t inter) {
  const int64_t slots = tokens * top;
  return (size_t)(align(kGrid * (int64_t)sizeof(Begin)) + align(most_passes(slots, experts) * (int64_t)sizeof(Pass)) + align(slots * 4) + align(slots * inter * 4) +
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
  w.begin = (Begin*)take(kGrid * (int64_t)sizeof(Begin));
  w.pass = (Pass*)take(most_passes(slots, experts) * (int64_t)sizeof(Pass));
  w.row_of = (int*)take(slots * 4);
  w.h = (uint16_t*)take(slots * inter * 4);
  w.part = (float*)take(slots * hidden * 4);
  const Args p{(const uint16_t*)x, ids, weights, (const uint8_t*)up, (const uint8_t*)down, up_scales, down_scales, y, ldx, ldy,
               (int)tokens, (int)top, (int)experts, (int)hidden, (int)inter, w};
  if (fmt == kMXFP4) return run<kMXFP4>(p, out_dtype, s);
  if (fmt == kFP8B128X128) return run<kFP8B128X128>(p, out_dtype, s);
  return run<kINT8>(p, out_dtype, s);
}

}  // namespace mx
