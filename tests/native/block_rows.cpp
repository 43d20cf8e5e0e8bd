// The block norm's dealing of rows and gate rows (block_rows.hpp) against the definitions in 64 bits, up
// to the largest batch.  Host code; no GPU is touched.
#include <algorithm>
#include <cstdio>

#include "block_rows.hpp"

static int failures = 0;
static void expect(bool ok, const char* what, long M, long slots, long gate_rows, long at) {
  if (ok) return;
  if (++failures < 20) std::printf("%s: M %ld, slots %ld, gate_rows %ld, at %ld\n", what, M, slots, gate_rows, at);
}

// A workgroup's slots in order, PER to each of `grid`: their rows, and the gate rows in those.
static void check(long M, int grid, int per, long gate_rows) {
  const int slots = grid * per;
  long next = 0;
  for (int wg = 0; wg < grid; ++wg) {
    const el::RowRange first = el::rows_of_slot(wg * per, slots, static_cast<int>(M));
    const long begin = next;
    for (int s = wg * per; s < wg * per + per; ++s) {
      const el::RowRange r = el::rows_of_slot(s, slots, static_cast<int>(M));
      expect(r.first == next && r.n >= 0 && r.n <= first.n, "rows", M, slots, gate_rows, s);
      for (long row : {next, next + r.n - 1})
        if (r.n > 0) expect(el::slot_of_row(static_cast<int>(row), slots, static_cast<int>(M)) == s, "slot", M, slots, gate_rows, row);
      next += r.n;
    }
    if (first.n == 0) continue;
    const long n = static_cast<long>(per) * first.n;
    const el::RowRange g = el::gates_of_rows(first.first, n, static_cast<int>(gate_rows), static_cast<int>(M));
    const long last = std::min(begin + n, M) - 1;
    expect(g.first == begin / gate_rows && g.n == last / gate_rows - begin / gate_rows + 1, "gates", M, slots, gate_rows, wg);
    // every gate row that the workgroup's own rows lie in is among them, and none that does not exist
    expect(g.n >= 1 && (next - 1) / gate_rows < g.first + long{g.n}, "covered", M, slots, gate_rows, wg);
    expect(g.first + long{g.n} <= (M + gate_rows - 1) / gate_rows, "exist", M, slots, gate_rows, wg);
  }
  expect(next == M, "all rows", M, slots, gate_rows, next);
}

int main() {
  const long big = 0x7fffffff;
  for (long M : {1l, 2l, 5l, 127l, 128l, 129l, 1000l, 4099l, 65536l, 100003l, 1l << 20, (1l << 30) - 1, 1l << 30, (1l << 30) + 3, 1200000000l, big - 1, big})
    for (int per : {1, 2, 4, 8, 32, 128})
      for (int most : {256, 512, 768}) {
        const int grid = static_cast<int>(std::min<long>(most, (M + per - 1) / per));
        for (long gr : {1l, 2l, 3l, 7l, 26l, 1l << 20, 1l << 30, (1l << 30) + 1, M - 1, M})
          if (gr >= 1 && gr <= M) check(M, grid, per, gr);
      }
  std::printf(failures ? "failed\n" : "ok\n");
  return failures != 0;
}
