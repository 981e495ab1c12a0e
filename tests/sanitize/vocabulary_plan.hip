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

int main() {
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
