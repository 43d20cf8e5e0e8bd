// The 4-bit layout and the 4-bit dense layer's cut of a call (fp4_plan.hpp): every row and column is
// taken, and no fragment is read behind the packed rows.  Host code; no GPU is touched.
#include <cstdio>
#include <vector>

#include "fp4_plan.hpp"

using namespace el::fp4;

static int failures = 0;
static void expect(bool ok, const char* what, long M, long K, long N, long at) {
  if (ok) return;
  if (++failures < 20) std::printf("%s: M %ld, K %ld, N %ld, at %ld\n", what, M, K, N, at);
}

// Every eight columns of every row of two tiles have a word of their own, in the fragment and the lane
// that row_of_lane names; so have the blocks' scales.
static void check_layout(int steps) {
  const int rows = 64, groups = static_cast<int>(groups_of(long{steps} * kPad));
  std::vector<int> words(rows * steps * kPad / 8, 0), scales(rows * groups * 16, 0);
  for (int r = 0; r < rows; ++r)
    for (int k = 0; k < steps; ++k)
      for (int q = 0; q < 16; ++q) {
        const long at = code_at(r, k, q, steps);
        const int f = r / kTileRows * 2 + frag_of_row(r % kTileRows), lane = (q >> 2) * 16 + lane_of_row(r % kTileRows);
        expect(at % 4 == 0 && at / 4 < static_cast<long>(words.size()) && ++words[at / 4] == 1, "word", rows, steps, q, at);
        expect(at == frag_code_at(f, k, steps) + lane * 16 + (q & 3) * 4, "fragment", rows, steps, q, at);
        expect(row_of_lane(f, lane % 16) == r, "row of lane", rows, steps, q, r);
        if (q & 3) continue;
        const long sc = scale_at(r, k, q >> 2, groups);
        expect(sc < static_cast<long>(scales.size()) && ++scales[sc] == 1, "scale", rows, steps, q, sc);
        expect(sc == frag_scale_at(f, k, groups) + lane * 4 + (k & 3), "scale's fragment", rows, steps, q, sc);
      }
}

static void check_plan(long M, long K, long N) {
  const Plan p = plan_dense(M, K, N);
  expect(p.J == 1 || p.J == 2 || p.J == 4, "J", M, K, N, p.J);
  expect(static_cast<long>(p.row_blocks) * 16 * p.J >= M && (p.row_blocks - 1l) * 16 * p.J < tile_rows(M), "rows", M, K, N, p.row_blocks);
  const long splits = p.blocks / p.row_blocks;
  expect(p.blocks % p.row_blocks == 0 && splits * p.passes * 128 >= N && (splits - 1) * p.passes * 128 < N, "columns", M, K, N, splits);
  if (!p.packed) {
    expect(x_lds(16 * p.J, K) <= 80 * 1024, "LDS", M, K, N, static_cast<long>(x_lds(16 * p.J, K)));
    return;
  }
  const int steps = static_cast<int>(steps_of(K)), groups = static_cast<int>(groups_of(K)), frags = frags_of(static_cast<int>(M));
  for (int rb : {0, 1, p.row_blocks / 2, p.row_blocks - 2, p.row_blocks - 1}) {
    if (rb < 0 || rb >= p.row_blocks) continue;
    for (int j = 0; j < p.J; ++j) {
      const int f = frag_read(rb, p.J, j, frags);
      expect(f >= 0 && frag_code_at(f, steps - 1, steps) + kFrag <= static_cast<long>(code_bytes(M, K)), "codes", M, K, N, f);
      expect(f >= 0 && frag_scale_at(f, steps - 1, groups) + 256 <= static_cast<long>(scale_bytes(M, K)), "scales", M, K, N, f);
      // a fragment that holds a row is read itself
      if (row_of_lane(rb * p.J + j, 0) < M) expect(f == rb * p.J + j, "own", M, K, N, f);
    }
  }
}

int main() {
  for (int steps = 1; steps <= 9; ++steps) check_layout(steps);
  int packed = 0, halves = 0;
  const long ms[] = {1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 1000, 2047, 2048, 2079, 2080, 4095, 4096, 4128, 8191, 8192, 8193, 8200, 8223, 8224, 8225, 8256, 9001, 33001, 65536, 65600, 1 << 20, 4100001};
  for (long M : ms)
    for (long K : {1l, 7l, 100l, 128l, 512l, 513l, 2048l, 2049l, 4096l, 4097l, 4200l, 8201l, 70000l, 1l << 20})
      for (long N : {1l, 24l, 127l, 128l, 129l, 1000l, 4096l}) {
        if (tile_rows(M) * steps_of(K) * kPad > 1l << 34) continue;
        check_plan(M, K, N);
        const Plan p = plan_dense(M, K, N);
        packed += p.packed;
        halves += p.packed && p.row_blocks * p.J > frags_of(static_cast<int>(M));
      }
  if (!packed || !halves) std::printf("no packed rows end inside a workgroup\n"), ++failures;
  std::printf(failures ? "failed\n" : "ok\n");
  return failures != 0;
}
