// Rules of the fine-tuned layers' planning code, checked on the host with the
// library's own code in this translation unit (tests/test_rows_rules.py). Exits
// 0 if they hold.
#include <stdio.h>
#include <stdlib.h>

#include "rows.hip"

static void need(bool ok, const char *what, int kind, int n, int k, int m, int matrices) {
  if (ok) return;
  printf("%s: kind %d n %d k %d m %d matrices %d\n", what, kind, n, k, m, matrices);
  exit(1);
}

// Every launch but the last decodes whole workgroup tiles, and what it decodes
// stays within the stated bound.
static void slabs() {
  long checked = 0, several = 0;
  for (int k : {256, 1024, 4096, 8192, 17408, TRELLIS_MAX_K})
    for (int n : {4096, 17408, 131072, 151936, 262144, 300000, 524288, 1000000, 1 << 21, 3000000, TRELLIS_MAX_N})
      for (int m : {1, 96, 512, 1000, 2048, 4096, 20000})
        for (int kind : {kForward, kGated, kTransposed})
          for (int matrices = 1; matrices <= (kind == kTransposed ? 2 : 1); ++matrices) {
            const DenseShape s = dense_shape(kind, trellis_geom{n, k, 256, 12, 4}, m, matrices, 256);
#define NEED(e) need(e, #e, kind, n, k, m, matrices)
            NEED(s.slab == s.tiles || s.slab % (2 * s.nt) == 0);
            NEED(s.slab == s.tiles || kind != kTransposed || s.slab % 16 == 0);
            const size_t least = kind == kTransposed ? (size_t)512 * ((n + 63) / 64 * 64) * matrices : 0;
            NEED(s.operand_bytes <= ((size_t)1 << 30) || s.operand_bytes <= least);
            ++checked;
            several += s.slab < s.tiles;
          }
  printf("slabs ok: %ld layouts, %ld of several launches\n", checked, several);
}

int main() {
  slabs();
  return 0;
}
