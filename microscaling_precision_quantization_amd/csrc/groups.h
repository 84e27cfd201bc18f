// Row groups of a GEMM by expert: rows offsets[g] .. offsets[g+1]-1 of A and C
// meet weight g. The offsets live on the device (a router writes them there),
// so the grid is made for the most tiles that any offsets of M rows can need,
// and each workgroup finds its tile by itself: every wave scans the groups'
// tile counts, 64 groups at a time. Offsets are clamped to [0, M], so that no
// value of theirs leads outside A or C; where they then fall, groups overlap and
// their tiles may be more than the grid and the counts hold: no tile is done.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace mx {
namespace groups {

// Row tiles of bm rows that `groups` groups over M rows need at most: each
// group that has rows ends in one partly filled tile.
inline int64_t max_row_tiles(int64_t M, int64_t n, int64_t bm) {
  const int64_t used = n < M ? n : M;
  return (M + used * (bm - 1)) / bm;
}

// Workgroups of a 1-D grid for that many row tiles and tiles_n column tiles:
// two multiples of 8 (both kinds of tiles), for tile_of below.
inline int64_t grid_size(int64_t row_tiles, int64_t tiles_n) { return (row_tiles * tiles_n + 14) / 8 * 8; }

struct Tile {
  int group;         // weight
  int row, rows;     // first row of the tile, rows of the group from there on
  int tn;            // column tile
};

// v of another lane by DPP, 0 where there is none (or ROWS leaves the row out).
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int dpp0(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}

// Inclusive sum of v over the lanes up to this one: within rows of 16 lanes
// (row_shr 1, 2, 4, 8), then the last lane of row 0 and 2 into the next row
// (row_bcast 15) and that of the first two rows into the last two (row_bcast 31).
__device__ __forceinline__ int wave_scan(int v) {
  v += dpp0<0x111>(v);
  v += dpp0<0x112>(v);
  v += dpp0<0x114>(v);
  v += dpp0<0x118>(v);
  v += dpp0<0x142, 0xA>(v);
  v += dpp0<0x143, 0xC>(v);
  return v;
}

// Pass `i` of up to 16 rows, counting each group's passes in turn: its group and first
// row, and its rows; false: there is none.
__device__ __forceinline__ bool pass_of(const int* offsets, int n, int M, int i, int& group, int& row, int& rows) {
  const int lane = threadIdx.x & 63;
  for (int c = 0; c < n; c += 64) {
    int lo = 0, hi = 0;
    if (c + lane < n) {
      lo = min(max(offsets[c + lane], 0), M);
      hi = max(min(offsets[c + lane + 1], M), lo);
    }
    const int upto = wave_scan((hi - lo + 15) / 16);
    const int sum = __builtin_amdgcn_readlane(upto, 63);
    if (i < sum) {
      const int l = __builtin_ctzll(__ballot(upto > i));
      const int before = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0;
      group = __builtin_amdgcn_readfirstlane(c + l);
      row = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_readlane(lo, l) + (i - before) * 16);
      rows = __builtin_amdgcn_readfirstlane(min(__builtin_amdgcn_readlane(hi, l) - row, 16));
      return true;
    }
    i -= sum;
  }
  return false;
}

// Tile of workgroup `bid`; false: there is none. offsets null: one group of
// all M rows. Workgroup ids go round-robin over the 8 XCDs. Tiles of more than
// BM / 2 rows ("whole") come first, an expert's last tile of fewer, which takes
// less time, at the end, so that these even out the end of the launch (FP8, 8192
// rows over 16 experts of 4096 x 4096: 164 us, 172 where only tiles of BM rows come first).
//   XCD x gets an eighth of each kind in a row, rastered in groups of 4 row
// tiles, so that its L2 holds the rows and columns its tiles share.
//   ROUNDS: the XCDs get 32 tiles (one a CU) each of one row of 256, and the next
// 256, in groups of 8 row tiles: what the XCDs read at a time is then shared between
// them too, and comes from HBM once. MXFP4, 16384 rows over 8 x 8192 x 4096: 345 us, 367
// without; but FP8, whose steps take longer for the same bytes, is 2% slower so.
template <int BM, bool ROUNDS = false>
__device__ __forceinline__ bool tile_of(const int* offsets, int n, int M, int tiles_n, int bid, Tile& t) {
  const int lane = threadIdx.x & 63;
  // Each lane's group (of 64 at a time), and the scan of the whole tiles times
  // 128 plus the others, at most 64 in a wave.
  int lo = 0, hi = 0, scan = 0, whole = 0, part = 0;
  bool falls = false;
  auto look = [&](int c) {
    lo = hi = 0;
    if (c + lane < n) {
      lo = min(max(offsets[c + lane], 0), M);
      hi = min(max(offsets[c + lane + 1], 0), M);
    }
    falls |= __ballot(hi < lo) != 0;
    scan = wave_scan((hi - lo + BM / 2 - 1) / BM * 128 + ((hi - lo) % BM != 0 && (hi - lo) % BM <= BM / 2));
    return __builtin_amdgcn_readlane(scan, 63);
  };
  if (!offsets) {
    whole = (M + BM / 2 - 1) / BM;
    part = M % BM != 0 && M % BM <= BM / 2;
  } else {
    for (int c = 0; c < n; c += 64) {
      const int all = look(c);
      whole += all / 128;
      part += all % 128;
    }
    if (falls) return false;
  }
  const int i = bid / 8, x = bid % 8;
  const int share = (whole * tiles_n + 7) / 8, share2 = (part * tiles_n + 7) / 8;
  const bool first = i < share;
  const int rows = first ? whole : part, j = first ? i : i - share;
  if (i >= share + share2) return false;
  int id;
  if constexpr (ROUNDS) {
    const int rounds = rows * tiles_n / 256, rest = rows * tiles_n - rounds * 256;
    id = j < rounds * 32 ? (j / 32 * 8 + x) * 32 + j % 32 : rounds * 256 + x * ((rest + 7) / 8) + j - rounds * 32;
  } else {
    id = x * (first ? share : share2) + j;
  }
  if (id >= rows * tiles_n) return false;
  constexpr int GM = ROUNDS ? 8 : 4;
  const int top = id / (GM * tiles_n) * GM, width = min(rows - top, GM);
  const int within = id % (GM * tiles_n);
  int tm = top + within % width;
  t.tn = within / width;
  if (!offsets) {
    t.group = 0;
    t.row = first ? tm * BM : whole * BM;
    t.rows = M - t.row;
    return true;
  }
  for (int c = 0; c < n; c += 64) {
    if (n > 64) look(c);  // (otherwise the values are those of the loop above)
    const int upto = first ? scan / 128 : scan % 128;
    const int sum = __builtin_amdgcn_readlane(upto, 63);
    if (tm < sum) {
      const int l = __builtin_ctzll(__ballot(upto > tm));
      const int before = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0;
      const int glo = __builtin_amdgcn_readlane(lo, l), ghi = __builtin_amdgcn_readlane(hi, l);
      // (Uniform as they are; said so, for the compiler to keep them in scalars.)
      t.group = __builtin_amdgcn_readfirstlane(c + l);
      t.row = __builtin_amdgcn_readfirstlane(first ? glo + (tm - before) * BM : glo + (ghi - glo) / BM * BM);
      t.rows = __builtin_amdgcn_readfirstlane(ghi - t.row);
      t.tn = __builtin_amdgcn_readfirstlane(t.tn);
      return true;
    }
    tm -= sum;
  }
  return false;
}

}  // namespace groups
}  // namespace mx
