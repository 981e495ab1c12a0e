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

// Both sides' measured times (us): weights decoded in the product, and decoded
// once. The rule takes the faster one, or one that is at most a fifth slower
// (calls of some 50 us, where a few launches decide), and 1% slower on average.
struct Sides {
  int kind, n, k, bits, m, matrices;
  double fused, once;
};
static const Sides kSides[] = {
    {kForward, 17408, 5120, 4, 97, 1, 60.6, 120.4},
    {kForward, 17408, 5120, 4, 257, 1, 116.2, 146.7},
    {kForward, 17408, 5120, 4, 385, 1, 167.2, 148.7},
    {kForward, 17408, 5120, 4, 512, 1, 169, 150.1},
    {kForward, 17408, 5120, 4, 640, 1, 201.8, 195.1},
    {kForward, 17408, 5120, 4, 768, 1, 241.6, 190.4},
    {kForward, 17408, 5120, 4, 1024, 1, 291.2, 251.6},
    {kForward, 17408, 5120, 4, 2048, 1, 554, 389.9},
    {kTransposed, 17408, 5120, 4, 97, 1, 101.4, 124.7},
    {kTransposed, 17408, 5120, 4, 257, 1, 155.5, 172.1},
    {kTransposed, 17408, 5120, 4, 385, 1, 226.2, 182.8},
    {kTransposed, 17408, 5120, 4, 512, 1, 239.1, 183.4},
    {kTransposed, 17408, 5120, 4, 640, 1, 289.9, 225.5},
    {kTransposed, 17408, 5120, 4, 768, 1, 313.6, 225.1},
    {kTransposed, 17408, 5120, 4, 1024, 1, 405.9, 274.5},
    {kTransposed, 17408, 5120, 4, 2048, 1, 762.5, 436.5},
    {kGated, 17408, 5120, 4, 97, 1, 81.7, 187.8},
    {kGated, 17408, 5120, 4, 257, 1, 177, 275.7},
    {kGated, 17408, 5120, 4, 385, 1, 259.5, 288},
    {kGated, 17408, 5120, 4, 512, 1, 264.2, 293.2},
    {kGated, 17408, 5120, 4, 640, 1, 343.8, 336.2},
    {kGated, 17408, 5120, 4, 768, 1, 420.1, 339.4},
    {kGated, 17408, 5120, 4, 1024, 1, 507.3, 413.2},
    {kGated, 17408, 5120, 4, 2048, 1, 1005.8, 731.2},
    {kTransposed, 17408, 5120, 4, 97, 2, 126.3, 186.8},
    {kTransposed, 17408, 5120, 4, 257, 2, 215.5, 266.3},
    {kTransposed, 17408, 5120, 4, 385, 2, 338.9, 292.1},
    {kTransposed, 17408, 5120, 4, 512, 2, 401.8, 308.7},
    {kTransposed, 17408, 5120, 4, 640, 2, 462.7, 361.5},
    {kTransposed, 17408, 5120, 4, 768, 2, 517.4, 372.1},
    {kTransposed, 17408, 5120, 4, 1024, 2, 708.3, 454.6},
    {kTransposed, 17408, 5120, 4, 2048, 2, 1403.4, 819.9},
    {kForward, 5120, 17408, 4, 97, 1, 60.1, 106.3},
    {kForward, 5120, 17408, 4, 257, 1, 107.2, 156.7},
    {kForward, 5120, 17408, 4, 385, 1, 159.7, 163.6},
    {kForward, 5120, 17408, 4, 512, 1, 161.2, 162.4},
    {kForward, 5120, 17408, 4, 640, 1, 196.1, 216},
    {kForward, 5120, 17408, 4, 768, 1, 209.1, 213.8},
    {kForward, 5120, 17408, 4, 1024, 1, 270.2, 242.2},
    {kForward, 5120, 17408, 4, 2048, 1, 513.4, 398.4},
    {kTransposed, 5120, 17408, 4, 97, 1, 101, 126.2},
    {kTransposed, 5120, 17408, 4, 257, 1, 155.6, 171.9},
    {kTransposed, 5120, 17408, 4, 385, 1, 236.1, 177.5},
    {kTransposed, 5120, 17408, 4, 512, 1, 262.4, 175},
    {kTransposed, 5120, 17408, 4, 640, 1, 305.7, 214.4},
    {kTransposed, 5120, 17408, 4, 768, 1, 345.8, 209.9},
    {kTransposed, 5120, 17408, 4, 1024, 1, 440.5, 282.3},
    {kTransposed, 5120, 17408, 4, 2048, 1, 833.1, 443.6},
    {kGated, 5120, 17408, 4, 97, 1, 76.2, 174.8},
    {kGated, 5120, 17408, 4, 257, 1, 161.3, 245.1},
    {kGated, 5120, 17408, 4, 385, 1, 243, 255.7},
    {kGated, 5120, 17408, 4, 512, 1, 246.6, 262.9},
    {kGated, 5120, 17408, 4, 640, 1, 333.8, 322.1},
    {kGated, 5120, 17408, 4, 768, 1, 403.8, 334.3},
    {kGated, 5120, 17408, 4, 1024, 1, 474, 422.9},
    {kGated, 5120, 17408, 4, 2048, 1, 950.2, 767},
    {kTransposed, 5120, 17408, 4, 97, 2, 124, 182.9},
    {kTransposed, 5120, 17408, 4, 257, 2, 209.6, 269.7},
    {kTransposed, 5120, 17408, 4, 385, 2, 336.3, 276.6},
    {kTransposed, 5120, 17408, 4, 512, 2, 395.4, 283.1},
    {kTransposed, 5120, 17408, 4, 640, 2, 452.1, 339.8},
    {kTransposed, 5120, 17408, 4, 768, 2, 507.8, 343.3},
    {kTransposed, 5120, 17408, 4, 1024, 2, 699.9, 461.6},
    {kTransposed, 5120, 17408, 4, 2048, 2, 1376.3, 740.8},
    {kForward, 4096, 1024, 4, 97, 1, 25.4, 35.8},
    {kForward, 4096, 1024, 4, 257, 1, 27.6, 40.5},
    {kForward, 4096, 1024, 4, 385, 1, 30, 42.1},
    {kForward, 4096, 1024, 4, 512, 1, 31.2, 41.5},
    {kForward, 4096, 1024, 4, 640, 1, 40.3, 44.6},
    {kForward, 4096, 1024, 4, 768, 1, 43.5, 43.1},
    {kForward, 4096, 1024, 4, 1024, 1, 32, 44.7},
    {kForward, 4096, 1024, 4, 2048, 1, 52.9, 47.5},
    {kTransposed, 4096, 1024, 4, 97, 1, 46.8, 48.3},
    {kTransposed, 4096, 1024, 4, 257, 1, 62.1, 57.8},
    {kTransposed, 4096, 1024, 4, 385, 1, 63.7, 57.7},
    {kTransposed, 4096, 1024, 4, 512, 1, 62.1, 54},
    {kTransposed, 4096, 1024, 4, 640, 1, 66.6, 60.3},
    {kTransposed, 4096, 1024, 4, 768, 1, 71.3, 59.7},
    {kTransposed, 4096, 1024, 4, 1024, 1, 84, 62.5},
    {kTransposed, 4096, 1024, 4, 2048, 1, 99.9, 78.3},
    {kGated, 4096, 1024, 4, 97, 1, 21.9, 28.7},
    {kGated, 4096, 1024, 4, 257, 1, 28.4, 33.3},
    {kGated, 4096, 1024, 4, 385, 1, 20, 35.8},
    {kGated, 4096, 1024, 4, 512, 1, 20.2, 35.8},
    {kGated, 4096, 1024, 4, 640, 1, 37.6, 36.4},
    {kGated, 4096, 1024, 4, 768, 1, 37.5, 36.4},
    {kGated, 4096, 1024, 4, 1024, 1, 36.5, 37.4},
    {kGated, 4096, 1024, 4, 2048, 1, 68.5, 51.9},
    {kTransposed, 4096, 1024, 4, 97, 2, 43.7, 41.3},
    {kTransposed, 4096, 1024, 4, 257, 2, 56.1, 45.5},
    {kTransposed, 4096, 1024, 4, 385, 2, 50.1, 44.9},
    {kTransposed, 4096, 1024, 4, 512, 2, 54.5, 45.5},
    {kTransposed, 4096, 1024, 4, 640, 2, 55.3, 47.9},
    {kTransposed, 4096, 1024, 4, 768, 2, 54.3, 49.4},
    {kTransposed, 4096, 1024, 4, 1024, 2, 77.3, 54.7},
    {kTransposed, 4096, 1024, 4, 2048, 2, 104.2, 82.5},
    {kForward, 1024, 4096, 4, 97, 1, 33.5, 38.1},
    {kForward, 1024, 4096, 4, 257, 1, 33.2, 44.9},
    {kForward, 1024, 4096, 4, 385, 1, 39.7, 45.3},
    {kForward, 1024, 4096, 4, 512, 1, 40.7, 41.9},
    {kForward, 1024, 4096, 4, 640, 1, 36.4, 44.5},
    {kForward, 1024, 4096, 4, 768, 1, 40.5, 43.7},
    {kForward, 1024, 4096, 4, 1024, 1, 41.4, 46.8},
    {kForward, 1024, 4096, 4, 2048, 1, 51.4, 56.9},
    {kTransposed, 1024, 4096, 4, 97, 1, 37.2, 44.9},
    {kTransposed, 1024, 4096, 4, 257, 1, 50.8, 54.4},
    {kTransposed, 1024, 4096, 4, 385, 1, 54.7, 55.3},
    {kTransposed, 1024, 4096, 4, 512, 1, 54.1, 53.3},
    {kTransposed, 1024, 4096, 4, 640, 1, 56.7, 60.9},
    {kTransposed, 1024, 4096, 4, 768, 1, 59, 59.8},
    {kTransposed, 1024, 4096, 4, 1024, 1, 76.6, 59.4},
    {kTransposed, 1024, 4096, 4, 2048, 1, 103.3, 68.1},
    {kGated, 1024, 4096, 4, 97, 1, 26.6, 34.5},
    {kGated, 1024, 4096, 4, 257, 1, 23.7, 35.3},
    {kGated, 1024, 4096, 4, 385, 1, 30, 35.5},
    {kGated, 1024, 4096, 4, 512, 1, 29.5, 36.5},
    {kGated, 1024, 4096, 4, 640, 1, 29.9, 39.3},
    {kGated, 1024, 4096, 4, 768, 1, 42.3, 40.2},
    {kGated, 1024, 4096, 4, 1024, 1, 37.1, 43.8},
    {kGated, 1024, 4096, 4, 2048, 1, 52.4, 62.1},
    {kTransposed, 1024, 4096, 4, 97, 2, 28, 35.3},
    {kTransposed, 1024, 4096, 4, 257, 2, 35, 40.6},
    {kTransposed, 1024, 4096, 4, 385, 2, 37, 38.5},
    {kTransposed, 1024, 4096, 4, 512, 2, 54.2, 40.3},
    {kTransposed, 1024, 4096, 4, 640, 2, 51.3, 44},
    {kTransposed, 1024, 4096, 4, 768, 2, 45.1, 44.9},
    {kTransposed, 1024, 4096, 4, 1024, 2, 65.5, 47.4},
    {kTransposed, 1024, 4096, 4, 2048, 2, 101.8, 56.2},
    {kForward, 5120, 5120, 4, 97, 1, 35.8, 55.1},
    {kForward, 5120, 5120, 4, 257, 1, 48.6, 68.8},
    {kForward, 5120, 5120, 4, 385, 1, 68.9, 70.6},
    {kForward, 5120, 5120, 4, 512, 1, 69, 69.8},
    {kForward, 5120, 5120, 4, 640, 1, 78.9, 83.4},
    {kForward, 5120, 5120, 4, 768, 1, 77.2, 82.9},
    {kForward, 5120, 5120, 4, 1024, 1, 104.6, 96.1},
    {kForward, 5120, 5120, 4, 2048, 1, 181.8, 132.1},
    {kTransposed, 5120, 5120, 4, 97, 1, 57, 65.6},
    {kTransposed, 5120, 5120, 4, 257, 1, 79.5, 82.6},
    {kTransposed, 5120, 5120, 4, 385, 1, 106.1, 85.9},
    {kTransposed, 5120, 5120, 4, 512, 1, 99.7, 82},
    {kTransposed, 5120, 5120, 4, 640, 1, 123.3, 99.1},
    {kTransposed, 5120, 5120, 4, 768, 1, 133.7, 98.5},
    {kTransposed, 5120, 5120, 4, 1024, 1, 164.9, 113},
    {kTransposed, 5120, 5120, 4, 2048, 1, 284.7, 157.4},
    {kGated, 5120, 5120, 4, 97, 1, 32.1, 60.7},
    {kGated, 5120, 5120, 4, 257, 1, 54.1, 84},
    {kGated, 5120, 5120, 4, 385, 1, 87.9, 87.7},
    {kGated, 5120, 5120, 4, 512, 1, 91.7, 91.6},
    {kGated, 5120, 5120, 4, 640, 1, 115.3, 106},
    {kGated, 5120, 5120, 4, 768, 1, 134.8, 108.1},
    {kGated, 5120, 5120, 4, 1024, 1, 158, 129.8},
    {kGated, 5120, 5120, 4, 2048, 1, 301.1, 232.4},
    {kTransposed, 5120, 5120, 4, 97, 2, 50.9, 65.6},
    {kTransposed, 5120, 5120, 4, 257, 2, 79.3, 89.5},
    {kTransposed, 5120, 5120, 4, 385, 2, 120.3, 92.9},
    {kTransposed, 5120, 5120, 4, 512, 2, 133, 101},
    {kTransposed, 5120, 5120, 4, 640, 2, 157.8, 120.9},
    {kTransposed, 5120, 5120, 4, 768, 2, 174.8, 125.6},
    {kTransposed, 5120, 5120, 4, 1024, 2, 230.9, 150.8},
    {kTransposed, 5120, 5120, 4, 2048, 2, 434.5, 251.8},
    {kForward, 9000, 3328, 3, 97, 1, 44.5, 56.1},
    {kForward, 9000, 3328, 3, 257, 1, 59.6, 77.9},
    {kForward, 9000, 3328, 3, 385, 1, 87, 75.3},
    {kForward, 9000, 3328, 3, 512, 1, 87.1, 74.8},
    {kForward, 9000, 3328, 3, 640, 1, 98.9, 83.8},
    {kForward, 9000, 3328, 3, 768, 1, 108.3, 82.4},
    {kForward, 9000, 3328, 3, 1024, 1, 139.4, 94.9},
    {kForward, 9000, 3328, 3, 2048, 1, 243.1, 157.4},
    {kTransposed, 9000, 3328, 3, 97, 1, 65.3, 72.1},
    {kTransposed, 9000, 3328, 3, 257, 1, 89.2, 90},
    {kTransposed, 9000, 3328, 3, 385, 1, 126.8, 95.8},
    {kTransposed, 9000, 3328, 3, 512, 1, 116.7, 91.1},
    {kTransposed, 9000, 3328, 3, 640, 1, 143.9, 113.3},
    {kTransposed, 9000, 3328, 3, 768, 1, 152.1, 110.5},
    {kTransposed, 9000, 3328, 3, 1024, 1, 188.6, 129},
    {kTransposed, 9000, 3328, 3, 2048, 1, 329.6, 196.5},
    {kGated, 9000, 3328, 3, 97, 1, 43.4, 67.3},
    {kGated, 9000, 3328, 3, 257, 1, 81.8, 94.6},
    {kGated, 9000, 3328, 3, 385, 1, 114.9, 95.7},
    {kGated, 9000, 3328, 3, 512, 1, 116.1, 96.5},
    {kGated, 9000, 3328, 3, 640, 1, 137.2, 113.8},
    {kGated, 9000, 3328, 3, 768, 1, 161.3, 114.7},
    {kGated, 9000, 3328, 3, 1024, 1, 209, 164.9},
    {kGated, 9000, 3328, 3, 2048, 1, 400.4, 243.6},
    {kTransposed, 9000, 3328, 3, 97, 2, 60.8, 75.5},
    {kTransposed, 9000, 3328, 3, 257, 2, 94.6, 102.3},
    {kTransposed, 9000, 3328, 3, 385, 2, 148.3, 108.7},
    {kTransposed, 9000, 3328, 3, 512, 2, 158.3, 115.3},
    {kTransposed, 9000, 3328, 3, 640, 2, 185.4, 146.9},
    {kTransposed, 9000, 3328, 3, 768, 2, 208.7, 152.5},
    {kTransposed, 9000, 3328, 3, 1024, 2, 272.4, 188.9},
    {kTransposed, 9000, 3328, 3, 2048, 2, 506.7, 317},
};
static void sides() {
  double sum = 0, most = 0;
  int count = 0;
  for (const Sides &p : kSides) {
    const Plan plan = plan_of(p.kind, trellis_geom{p.n, p.k, 256, 12, p.bits}, p.m, p.matrices, 256);
    const double slower = (plan.dense ? p.once : p.fused) / (p.fused < p.once ? p.fused : p.once) - 1;
    if (slower > 0.05)
      printf("%.1f%% slower (%s): kind %d n %d k %d m %d matrices %d, %.1f / %.1f us\n", 100 * slower,
             plan.dense ? "once" : "in the product", p.kind, p.n, p.k, p.m, p.matrices, p.fused, p.once);
    if (slower > most) most = slower;
    sum += slower;
    ++count;
  }
  printf("sides: %d sizes, %.2f%% slower on average, %.1f%% at most\n", count, 100 * sum / count, 100 * most);
  if (most > 0.2 || sum > 0.01 * count) exit(1);
  printf("sides ok\n");
}

int main() {
  slabs();
  splits();
  sides();
  return 0;
}
