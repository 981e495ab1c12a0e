// Lays products out on the host over a sweep of sizes, with the library's own
// planning code in this translation unit, for an UndefinedBehaviorSanitizer
// build (tests/test_rows_sanitizers.py). Exits 0 if every layout is one that
// the kernels can run.
#include <stdio.h>
#include <stdlib.h>

#include "rows.hip"

static long checked = 0;

static void need(bool ok, const char *what, int kind, trellis_geom g, int m, int matrices) {
  if (ok) return;
  printf("%s: kind %d n %d k %d bits %d m %d matrices %d\n", what, kind, (int)g.n, (int)g.k, (int)g.bits, m, matrices);
  exit(1);
}

static void check(int kind, trellis_geom g, int m, int matrices) {
  const int cus = 256;
  const Plan p = plan_of(kind, g, m, matrices, cus);
#define NEED(e) need(e, #e, kind, g, m, matrices)
  const int64_t width = kind == kTransposed ? g.k : g.n, depth = kind == kTransposed ? g.n : g.k;
  if (p.dense) {
    const DenseShape &s = p.many;
    NEED(s.nt >= 4 && s.nt <= 8 && (kind != kGated || s.nt % 2 == 0));
    NEED(s.splits >= 1 && s.splits <= 8 && s.steps / 2 >= s.splits);
    NEED(s.steps1 % 2 == 0 && (int64_t)s.steps1 * kDenseStep >= depth);
    NEED(s.slab >= 1 && s.slab <= s.tiles && s.slab % (kind == kTransposed ? 16 : kind == kGated ? 2 : 1) == 0);
    NEED(s.tiles * 16 >= width * (kind == kGated ? 2 : 1));
    NEED((int64_t)s.ptiles * 16 >= m);
    NEED(dense_buffers(s.nt) * dense_step_bytes(s.nt) <= 160 * 1024 && dense_buffers(s.nt) >= 2);
    NEED(s.splits == 1 || s.partial_bytes >= (size_t)s.splits * m * s.slab * 64);
    NEED(p.bytes >= s.operand_bytes + s.row_bytes + s.partial_bytes);
  } else {
    const Shape &s = p.fused;
    NEED(s.mt < kMts && (kind != kTransposed || kRowTiles[s.mt] <= 6));
    const int64_t rows = ((int64_t)m + 16 * kRowTiles[s.mt] - 1) / (16 * kRowTiles[s.mt]);
    NEED(s.tiles == rows * s.groups && s.units == s.tiles * s.steps && s.units < ((int64_t)1 << 30));
    NEED(s.grid >= 1 && s.grid <= s.units);
    NEED(s.parts == 0 || (s.parts <= s.steps && s.grid == s.tiles * s.parts));
    NEED(s.lds + kTableBytes + 64 <= 160 * 1024);
    NEED(p.bytes >= s.partial_bytes && p.counters >= s.tiles);
  }
  for (int cols : {(int)g.k, (int)g.n})
    for (int rank : {1, 32, 33, TRELLIS_MAX_RANK})
      for (int count : {1, 3, 8, TRELLIS_MAX_ADAPTERS}) {
        const ShrinkShape h = shrink_shape(m, cols, count, rank, cus);
        NEED(h.spans >= 1 && h.span % 32 == 0 && (int64_t)h.spans * h.span >= cols && (int64_t)(h.spans - 1) * h.span < cols);
        NEED(h.spans <= kSpanBatch * (h.ms == 1 ? 4 : 1) && h.groups * 16 * h.ms >= m);
      }
  ++checked;
}

int main() {
  for (int path = -1; path <= 1; ++path) {
    for (int tiles : {0, 1, 16}) {
      if (tiles && path != 1) continue;
      trellis_test_force_path(path, tiles);
      for (int bits : {2, 3, 4})
        for (int k : {256, 512, 768, 1024, 5120, 17408, TRELLIS_MAX_K})
          for (int n : {4, 36, 60, 64, 260, 480, 516, 5120, 17408, TRELLIS_MAX_N})
            for (int m : {1, 15, 16, 17, 33, 65, 96, 97, 128, 129, 257, 509, 512, 1000, 4096, 5001, 70000, TRELLIS_MAX_ROWS}) {
              const trellis_geom g{n, k, 256, 12, bits};
              check(kForward, g, m, 1);
              check(kGated, g, m, 1);
              check(kTransposed, g, m, 1);
              check(kTransposed, g, m, 2);
            }
    }
  }
  printf("rows plan ok: %ld layouts\n", checked);
  return 0;
}
