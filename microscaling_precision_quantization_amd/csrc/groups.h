// Row groups of a GEMM by expert: rows offsets[g] .. offsets[g+1]-1 of A and C
// meet weight g. The offsets live on the device (a router writes them there),
// so the grid is made for the most tiles that any offsets of M rows can need,
// and each workgroup finds its tile by itself: every wave scans the groups'
// tile counts, 64 groups at a time. Offsets are clamped to [0, M], so that no
// value of theirs leads outside A or C.
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
// a multiple of 8, for tile_of below.
inline int64_t grid_size(int64_t row_tiles, int64_t tiles_n) { return (row_tiles * tiles_n + 7) / 8 * 8; }

struct Tile {
  int group;         // weight
  int row, rows;     // first row of the tile, rows of the group from there on
  int tn;            // column tile
};

// Rows of group g: [lo, hi).
__device__ __forceinline__ void rows_of(const int* offsets, int M, int g, int& lo, int& hi) {
  lo = min(max(offsets[g], 0), M);
  hi = max(min(offsets[g + 1], M), lo);
}

// Inclusive sum of v over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Tile of workgroup `bid`; false: there is none. offsets null: one group of
// all M rows. Workgroup ids go round-robin over the 8 XCDs; XCD x gets tiles
// [x c, (x + 1) c) of the tiles that there are, rastered in groups of 4 row
// tiles, so that its L2 holds the rows and columns its tiles share.
template <int BM>
__device__ __forceinline__ bool tile_of(const int* offsets, int n, int M, int tiles_n, int bid, Tile& t) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  int lo = 0, hi = 0, scan = 0;
  if (!offsets) {
    total = (M + BM - 1) / BM;
  } else {
    for (int c = 0; c < n; c += 64) {
      lo = hi = 0;
      if (c + lane < n) rows_of(offsets, M, c + lane, lo, hi);
      scan = wave_scan((hi - lo + BM - 1) / BM, lane);
      total += __builtin_amdgcn_readlane(scan, 63);
    }
  }
  const int tiles = total * tiles_n, share = (tiles + 7) / 8;
  const int i = bid / 8, id = (bid % 8) * share + i;
  if (i >= share || id >= tiles) return false;
  constexpr int GM = 4;
  const int first = id / (GM * tiles_n) * GM, width = min(total - first, GM);
  const int within = id % (GM * tiles_n);
  int tm = first + within % width;
  t.tn = within / width;
  if (!offsets) {
    t.group = 0;
    t.row = tm * BM;
    t.rows = M - t.row;
    return true;
  }
  for (int c = 0; c < n; c += 64) {
    if (n > 64) {  // (otherwise the values are those of the loop above)
      lo = hi = 0;
      if (c + lane < n) rows_of(offsets, M, c + lane, lo, hi);
      scan = wave_scan((hi - lo + BM - 1) / BM, lane);
    }
    const int sum = __builtin_amdgcn_readlane(scan, 63);
    if (tm < sum) {
      const int l = __builtin_ctzll(__ballot(scan > tm));
      const int before = l ? __builtin_amdgcn_readlane(scan, l - 1) : 0;
      t.group = c + l;
      t.row = __builtin_amdgcn_readlane(lo, l) + (tm - before) * BM;
      t.rows = __builtin_amdgcn_readlane(hi, l) - t.row;
      return true;
    }
    tm -= sum;
  }
  return false;
}

}  // namespace groups
}  // namespace mx
