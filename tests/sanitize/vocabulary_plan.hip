// Lays the losses out on the host over a sweep of sizes, with the library's own
// planning code in this translation unit, for an UndefinedBehaviorSanitizer
// build (tests/test_vocabulary_plan.py). Exits 0 if every layout is one that the
// kernels can run. No kernel is launched.
#include <stdio.h>
#include <stdlib.h>

#include "rows.hip"

static long checked = 0;

static void need(bool ok, const char *what, trellis_geom g, int m, bool keep) {
  if (ok) return;
  printf("%s: n %d k %d bits %d m %d keep %d\n", what, (int)g.n, (int)g.k, (int)g.bits, m, (int)keep);
  exit(1);
}

static void check(trellis_geom g, int m, bool keep) {
  const int cus = 256;
#define NEED(e) need(e, #e, g, m, keep)
  const int64_t gib = (int64_t)1 << 30;
  if (!loss_by_operands(g, m, keep, cus)) {
    const Shape f = shape_of(kForward, g, m, 1, cus);
    NEED(f.units < gib);
    if (keep) {
      const Plan b = loss_back_plan(g, m, cus);
      NEED(b.dense || (b.fused.units < gib && b.bytes >= b.fused.partial_bytes && b.counters >= b.fused.tiles));
    }
    ++checked;
    return;
  }
  const LossShape s = loss_shape(g, m, keep, cus);
  const int64_t n_pad = ((int64_t)g.n + 63) / 64 * 64;
  NEED(s.rows >= 1 && s.rows <= m && (s.rows == m || s.rows % 256 == 0));
  NEED(s.rows <= 256 || ((int64_t)s.rows * g.k * 2 <= gib && (!keep || (int64_t)s.rows * n_pad * 2 <= gib)));
  NEED(s.steps % 8 == 0 && (int64_t)s.steps * 32 == g.k);
  NEED((int64_t)s.ptiles * 16 >= s.rows && s.row_bytes >= (size_t)s.ptiles * s.steps * 1024);
  NEED(s.tiles * 16 >= g.n && (int64_t)s.blocks * s.fwd.nt >= s.tiles);
  NEED(s.stat_bytes >= (size_t)s.rows * s.blocks * 8);
  const int64_t mtiles = (s.rows + 64 * s.fwd.rt - 1) / (64 * s.fwd.rt);
  NEED(mtiles * ((s.tiles + 2 * s.fwd.nt - 1) / (2 * s.fwd.nt)) < ((int64_t)1 << 31) / 512);
  if (s.fwd.decode) {
    NEED(s.fwd.nt == 4 && (s.fwd.rt == 4 || s.fwd.rt == 6) && s.slab == s.tiles);
    NEED(decode_lds(g.bits, s.fwd.rt) <= 160 * 1024 && decode_buffers(g.bits, s.fwd.rt) >= 3);
  } else {
    NEED((s.fwd.nt == 4 || s.fwd.nt == 6 || s.fwd.nt == 8) && (s.fwd.rt == 3 || s.fwd.rt == 4));
    NEED(dense_buffers(s.fwd.nt, s.fwd.rt) * dense_step_bytes(s.fwd.nt, s.fwd.rt) <= 160 * 1024);
    // whole workgroup tiles a launch: the next launch's columns start where this one's end
    NEED(s.slab == s.tiles || (s.slab > 0 && s.slab % (2 * s.fwd.nt) == 0));
    NEED(s.operand_bytes >= (size_t)(s.slab * s.steps * 1024));
  }
  if (keep) {
    NEED(s.back.nt >= 4 && s.back.nt <= 8 && (s.back.rt == 3 || s.back.rt == 4));
    NEED(s.back.splits >= 1 && s.back.splits <= 8 && s.back_steps / 2 >= s.back.splits);
    NEED((int64_t)s.back_steps * 32 == n_pad && s.e_bytes >= (size_t)s.ptiles * s.back_steps * 1024);
    // every operand tile of the contraction is written by the first product
    const int64_t unit = 2 * s.fwd.nt, written = (s.tiles + unit - 1) / unit * unit;
    NEED(written >= 2 * (int64_t)s.back_steps);
    NEED(s.back_slab >= 16 && s.back_slab % 16 == 0 && s.back_slab <= s.back_tiles);
    NEED(s.operand_bytes >= (size_t)(s.back_slab * s.back_steps * 1024));
    NEED(s.partial_bytes >= (size_t)s.back.splits * s.rows * s.back_slab * 64);
  }
  ++checked;
}

// Both ways' times on one MI355X (us): n, k, bits, rows; losses alone, few rows'
// way and many rows'; with gradient, the same. (With gradient few rows' way is
// taken with the transposed product decoding on its way; the library may take
// operands there where that is faster.)
static const struct {
  int n, k, bits, m, loss[2], keep[2];
} kMeasured[] = {
    {50004, 5120, 3, 96, {124, 223}, {249, 455}},
    {50004, 5120, 3, 128, {133, 212}, {301, 445}},
    {50004, 5120, 3, 192, {196, 206}, {403, 449}},
    {50004, 5120, 3, 256, {222, 206}, {516, 466}},
    {50004, 5120, 3, 333, {320, 256}, {704, 553}},
    {50004, 5120, 3, 384, {322, 254}, {710, 553}},
    {50004, 5120, 3, 509, {420, 381}, {1017, 730}},
    {50004, 5120, 3, 512, {428, 382}, {999, 733}},
    {50004, 5120, 3, 640, {537, 500}, {1192, 931}},
    {50004, 5120, 3, 768, {645, 504}, {1392, 938}},
    {50004, 5120, 3, 1024, {848, 625}, {1862, 1154}},
    {50004, 5120, 3, 1536, {1295, 763}, {2768, 1544}},
    {131072, 5120, 4, 96, {246, 413}, {498, 1005}},
    {131072, 5120, 4, 128, {262, 398}, {686, 1008}},
    {131072, 5120, 4, 192, {432, 399}, {949, 1040}},
    {131072, 5120, 4, 256, {522, 413}, {1267, 1073}},
    {131072, 5120, 4, 333, {761, 516}, {1757, 1335}},
    {131072, 5120, 4, 384, {808, 542}, {1783, 1325}},
    {131072, 5120, 4, 509, {1038, 792}, {2515, 1771}},
    {131072, 5120, 4, 512, {1035, 799}, {2509, 1741}},
    {131072, 5120, 4, 640, {1323, 1016}, {3089, 2225}},
    {131072, 5120, 4, 768, {1554, 1014}, {3476, 2299}},
    {131072, 5120, 4, 1024, {2027, 1413}, {4894, 2960}},
    {131072, 5120, 4, 1536, {3084, 1982}, {7038, 4076}},
    {32772, 1024, 2, 96, {40, 55}, {137, 125}},
    {32772, 1024, 2, 128, {42, 54}, {98, 124}},
    {32772, 1024, 2, 192, {55, 55}, {131, 126}},
    {32772, 1024, 2, 256, {63, 57}, {142, 130}},
    {32772, 1024, 2, 333, {78, 72}, {171, 144}},
    {32772, 1024, 2, 384, {81, 72}, {172, 145}},
    {32772, 1024, 2, 509, {100, 79}, {218, 156}},
    {32772, 1024, 2, 512, {100, 79}, {217, 155}},
    {32772, 1024, 2, 640, {119, 90}, {241, 169}},
    {32772, 1024, 2, 768, {135, 89}, {282, 171}},
    {32772, 1024, 2, 1024, {171, 101}, {367, 198}},
    {32772, 1024, 2, 1536, {248, 146}, {508, 270}},
    {8192, 2048, 4, 96, {27, 50}, {81, 85}},
    {8192, 2048, 4, 128, {28, 50}, {63, 85}},
    {8192, 2048, 4, 192, {30, 50}, {74, 87}},
    {8192, 2048, 4, 256, {34, 51}, {81, 92}},
    {8192, 2048, 4, 333, {47, 52}, {93, 90}},
    {8192, 2048, 4, 384, {47, 51}, {94, 90}},
    {8192, 2048, 4, 509, {40, 53}, {101, 96}},
    {8192, 2048, 4, 512, {41, 52}, {100, 96}},
    {8192, 2048, 4, 640, {61, 54}, {138, 103}},
    {8192, 2048, 4, 768, {62, 54}, {127, 104}},
    {8192, 2048, 4, 1024, {69, 56}, {163, 114}},
    {8192, 2048, 4, 1536, {103, 70}, {218, 143}},
    {16384, 4096, 4, 96, {41, 87}, {94, 159}},
    {16384, 4096, 4, 128, {46, 86}, {105, 155}},
    {16384, 4096, 4, 192, {55, 87}, {126, 161}},
    {16384, 4096, 4, 256, {63, 88}, {155, 171}},
    {16384, 4096, 4, 333, {98, 93}, {207, 182}},
    {16384, 4096, 4, 384, {100, 93}, {208, 183}},
    {16384, 4096, 4, 509, {118, 95}, {285, 199}},
    {16384, 4096, 4, 512, {117, 94}, {285, 200}},
    {16384, 4096, 4, 640, {151, 115}, {331, 240}},
    {16384, 4096, 4, 768, {167, 115}, {360, 244}},
    {16384, 4096, 4, 1024, {220, 143}, {497, 308}},
    {16384, 4096, 4, 1536, {324, 217}, {692, 444}}};

static void sides() {
  trellis_test_force_path(-1, 0);
  double sum = 0;
  int count = 0;
  for (const auto &p : kMeasured)
    for (int keep = 0; keep < 2; ++keep) {
      const int *us = keep ? p.keep : p.loss;
      const trellis_geom g{p.n, p.k, 256, 12, p.bits};
      const double taken = us[loss_by_operands(g, p.m, keep, 256)], best = us[0] < us[1] ? us[0] : us[1];
      need(taken <= 1.10 * best, "slower side taken", g, p.m, keep);
      sum += taken / best;
      ++count;
    }
  if (sum / count > 1.005) {
    printf("sides taken are %.4f of the faster ones on average\n", sum / count);
    exit(1);
  }
  printf("vocabulary sides ok: %.4f\n", sum / count);
}

int main() {
  sides();
  for (int path = -1; path <= 1; ++path)
    for (int tiles : {0, 1, 16, 4096}) {
      if (tiles && path != 1) continue;
      trellis_test_force_path(path, tiles);
      for (int bits : {2, 3, 4})
        for (int k : {256, 512, 768, 1024, 5120, 17408, TRELLIS_MAX_K})
          for (int n : {4, 36, 60, 64, 68, 260, 516, 5120, 17408, 50004, 131072, TRELLIS_MAX_N})
            for (int m : {1, 15, 16, 17, 33, 64, 65, 97, 129, 256, 257, 333, 385, 509, 1000, 2048, 5001, 70000, TRELLIS_MAX_ROWS})
              for (bool keep : {false, true}) {
                // (the few rows' way takes chunks of at most 1 GiB of logits)
                const int64_t most = ((int64_t)1 << 30) / (4 * (int64_t)n) / 16 * 16;
                if (path == 0 && m > most) continue;
                check({n, k, 256, 12, bits}, m, keep);
              }
    }
  printf("vocabulary plan ok: %ld layouts\n", checked);
  return 0;
}
