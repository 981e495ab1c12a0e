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

// Layouts of the dense product within 10% of the fastest, of all that were
// measured at a size (every column tile with one to eight splits): the rule
// takes one of them.
struct Measured {
  int kind, n, k, bits, m, matrices;
  struct {
    int nt, splits;
  } good[12];
};
static const Measured kMeasured[] = {
    {kTransposed, 17408, 5120, 4, 384, 1, {{4, 3}, {4, 6}, {5, 4}, {6, 4}, {7, 4}, {7, 5}, {8, 5}, {8, 6}}},
    {kGated, 17408, 5120, 4, 512, 1, {{4, 1}, {6, 1}, {6, 2}, {8, 2}}},
    {kTransposed, 17408, 5120, 4, 700, 2, {{4, 2}, {5, 5}, {6, 3}, {6, 6}, {7, 3}, {7, 7}, {8, 3}, {8, 4}, {8, 8}}},
    {kForward, 17408, 5120, 4, 2048, 1, {{6, 1}, {7, 1}}},
    {kTransposed, 5120, 17408, 4, 512, 1, {{5, 1}, {6, 1}, {7, 1}}},
    {kForward, 5120, 17408, 4, 700, 1, {{4, 2}, {4, 4}, {5, 5}, {6, 3}, {7, 3}, {8, 4}}},
    {kTransposed, 4096, 1024, 4, 512, 1, {{4, 5}, {4, 6}, {4, 7}, {4, 8}, {5, 5}, {5, 6}, {5, 7}, {5, 8}, {6, 7}, {6, 8}}},
    {kGated, 4096, 1024, 4, 512, 1, {{4, 1}, {4, 2}, {6, 2}}},
    {kGated, 1024, 4096, 4, 384, 1, {{4, 5}, {4, 6}, {4, 7}, {4, 8}, {6, 8}}},
    {kForward, 1024, 4096, 4, 512, 1, {{4, 5}, {4, 6}, {4, 7}, {4, 8}, {5, 7}, {5, 8}}},
    {kTransposed, 2048, 2048, 3, 384, 2, {{4, 5}, {4, 6}, {4, 7}, {4, 8}, {5, 6}, {5, 7}, {5, 8}, {6, 7}, {6, 8}}},
    {kForward, 4096, 4096, 2, 200, 1, {{4, 5}, {4, 6}, {4, 7}, {4, 8}, {5, 6}, {5, 7}, {5, 8}}},
    {kTransposed, 4096, 4096, 2, 512, 2, {{4, 3}, {4, 4}, {5, 4}, {6, 4}, {6, 5}, {7, 5}, {7, 6}, {8, 6}, {8, 7}, {8, 8}}},
    {kForward, 5120, 5120, 4, 384, 1, {{4, 3}, {5, 3}, {5, 4}, {6, 4}, {7, 5}}},
    {kTransposed, 5120, 5120, 4, 1500, 2, {{4, 1}, {5, 1}, {8, 2}}},
    {kGated, 2048, 8192, 4, 512, 1, {{4, 3}, {4, 4}, {6, 5}, {8, 6}, {8, 7}, {8, 8}}},
    {kTransposed, 17408, 256, 4, 1024, 1, {{4, 6}, {4, 7}, {4, 8}, {5, 7}, {5, 8}}},
    {kTransposed, 260, 17408, 3, 512, 2, {{5, 1}, {6, 1}, {7, 1}}},
};
static void splits() {
  for (const Measured &p : kMeasured) {
    const DenseShape s = dense_shape(p.kind, trellis_geom{p.n, p.k, 256, 12, p.bits}, p.m, p.matrices, 256);
    bool good = false;
    for (const auto &c : p.good) good = good || (c.nt == s.nt && c.splits == s.splits);
    if (!good) printf("nt %d splits %d\n", s.nt, s.splits);
    need(good, "a slow layout", p.kind, p.n, p.k, p.m, p.matrices);
  }
  printf("splits ok: %d sizes\n", (int)(sizeof(kMeasured) / sizeof(kMeasured[0])));
}

int main() {
  slabs();
  splits();
  return 0;
}
