// fp4_plan.hpp -- the 4-bit layout's index functions and sizes, and how the 4-bit dense layer cuts a call:
// plain integer functions, the same on the host and in the kernels of dense_fp4.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstddef>

namespace el {
namespace fp4 {

constexpr int kPad = 128;  // columns of a padded row: whole products of 128

// ---------------------------------------------------------------------------------------
// The layout: tiles of 32 rows by 128 columns in the order in which the matrix instructions take
// them.  Fragment i (of two) of a tile is 64 lanes of 16 bytes: lane l holds the block l / 16 of 32
// columns of row 8 (l % 16 / 4) + 4 i + l % 4.  With w as the first operand the accumulators of
// both fragments are then eight consecutive output columns of a lane, and every load of a fragment
// is one contiguous KiB (straight from row-major codes a load touched 64 separate pieces, and the
// cache's address rate, not its bytes, bounded the product: 184 us for 65536 x 1024 x 1024).
// ---------------------------------------------------------------------------------------
constexpr int kTileRows = 32, kFrag = 1024;  // bytes of a fragment's codes; 64 words hold its scales of four steps
__host__ __device__ inline int lane_of_row(int r) { return (r >> 3 & 3) * 4 + (r & 3); }  // row of a tile -> l % 16
__host__ __device__ inline int frag_of_row(int r) { return r >> 2 & 1; }
__host__ __device__ inline int row_of_lane(int frag, int l16) { return (frag >> 1) * kTileRows + (l16 >> 2) * 8 + (frag & 1) * 4 + (l16 & 3); }

// Byte of the codes of row r's eight columns 8 q .. 8 q + 7 of step k, and of its scale of their block.
__host__ __device__ inline long code_at(long r, int k, int q, int steps) {
  const int t = static_cast<int>(r & 31);
  return (((r >> 5) * steps + k) * 2 + frag_of_row(t)) * kFrag + ((q >> 2) * 16 + lane_of_row(t)) * 16 + (q & 3) * 4;
}
__host__ __device__ inline long scale_at(long r, int k, int g, int groups) {
  const int t = static_cast<int>(r & 31);
  return (((r >> 5) * groups + (k >> 2)) * 2 + frag_of_row(t)) * 256 + (g * 16 + lane_of_row(t)) * 4 + (k & 3);
}
// The same of a whole fragment f (two to a tile): step k's codes, and the scales of the four steps of k.
__host__ __device__ inline long frag_code_at(long f, int k, int steps) { return (((f >> 1) * steps + k) * 2 + (f & 1)) * kFrag; }
__host__ __device__ inline long frag_scale_at(long f, int k, int groups) { return (((f >> 1) * groups + (k >> 2)) * 2 + (f & 1)) * 256; }
// Fragments of M packed rows; the one that workgroup rb's j-th (of J) reads: the last workgroup's may end
// behind the last tile, whose fragments are read in their place.
__host__ __device__ inline int frags_of(int M) { return static_cast<int>((M + kTileRows - 1l) / kTileRows * 2); }
__host__ __device__ inline int frag_read(int rb, int J, int j, int frags) { return rb * J + j < frags ? rb * J + j : frags - 1; }

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
inline long ceil_div(long a, long b) { return (a + b - 1) / b; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
inline long steps_of(long K) { return ceil_div(K, kPad); }
inline long groups_of(long K) { return ceil_div(steps_of(K), 4); }
inline long tile_rows(long M) { return ceil_div(M, kTileRows) * kTileRows; }
inline size_t code_bytes(long M, long K) { return round256(static_cast<size_t>(tile_rows(M)) * steps_of(K) * kPad / 2); }
inline size_t scale_bytes(long M, long K) { return round256(static_cast<size_t>(tile_rows(M)) * groups_of(K) * 16); }
inline size_t x_lds(int rows, long K) { return rows * (steps_of(K) * 64 + groups_of(K) * 16); }

// How a call is cut.  A workgroup packs its rows once for all columns it walks over, so columns are
// split over workgroups only to have 512 of them; more rows a workgroup (16 J) read the weights less
// often, fewer fill the CUs sooner.  Measured in us, N = K = 1024, without a residual up to 4096 rows,
// J = 1, 2, 4: 1024 rows 6.4, 7.2, 9.6; 2048 8.0, 7.9; 4096 11.3, 10.2; 8192 21.9, 18.9, 19.4; 16384
// 47.9, 37.2, 34.0; 65536 177, 132, 116.  Columns split for 1024 workgroups rather than 512: 4099 rows
// 15.0 against 13.6, 16384 rows 28.6 against 27.4.
// Two workgroups' rows must fit a CU's LDS: J = 4 holds 136 KiB at K = 4096, 16384 rows 124, J = 2 91.
// Rows are packed in the workspace first where they are long: packing in the call, the column
// splits of few rows pack each row again.  In the call against before it, N = 1024: K = 2048, 1024
// rows 10.1 and 10.7; K = 4096, 1 row 13.8 and 13.6, 1024 rows 23.4 and 15.8, 2048 rows 25.9 and 20.1,
// 4096 rows 33.7 and 34.8, 16384 rows 91 and 116; K = 8192, 256 rows 36.4 and 26.6, 4096 rows 69.3 and
// 64.0, 16384 rows (N = 512) 170 and 155.
struct Plan {
  int J;        // 16 J rows a workgroup
  bool packed;  // x is packed in the workspace, not in LDS
  int row_blocks, passes;
  long blocks;
};
inline Plan plan_dense(long M, long K, long N) {
  Plan p{};
  p.J = M >= 8192 ? 4 : M >= 2048 ? 2 : 1;
  p.packed = K > 4096 || (K > 2048 && M < 4096);
  while (!p.packed && p.J > 1 && x_lds(16 * p.J, K) > 80 * 1024) p.J /= 2;
  p.row_blocks = static_cast<int>(ceil_div(p.packed ? tile_rows(M) : M, 16 * p.J));  // packed rows come in whole tiles
  const long all = ceil_div(N, 128);  // column passes there are
  const long split = std::min(all, std::max<long>(1, ceil_div(512, p.row_blocks)));
  p.passes = static_cast<int>(ceil_div(all, split));
  p.blocks = p.row_blocks * ceil_div(all, p.passes);
  return p;
}

}  // namespace fp4
}  // namespace el
