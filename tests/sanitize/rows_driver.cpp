// Calls the fine-tuned layers' entry points with arguments that their host-side
// validation must reject, plus in-domain calls on both product paths (which,
// with no GPU present, must fail cleanly with TRELLIS_E_HIP), for an
// AddressSanitizer / UndefinedBehaviorSanitizer build of the library's host code
// (tests/test_rows_sanitizers.py). Exits 0 if every status is the expected one.
#include <stdint.h>
#include <stdio.h>

#include "trellis.h"
#include "trellis_testing.h"

static int failures = 0;

static void expect(const char *what, int got, int want) {
  printf("%-44s %d\n", what, got);
  if (got != want) {
    printf("  expected %d\n", want);
    ++failures;
  }
}

int main() {
  alignas(16) static uint16_t buf[4096];
  uint16_t *p = buf;
  const uint32_t *c = reinterpret_cast<const uint32_t *>(buf);
  const float *gain = reinterpret_cast<const float *>(buf);
  const int32_t *index = reinterpret_cast<const int32_t *>(buf);
  const trellis_geom good{260, 512, 256, 12, 4}, bad{260, 500, 256, 12, 4}, big{1 << 22, 1 << 18, 256, 12, 2};
  expect("path hook -2", trellis_test_force_path(-2, 0), -2);
  expect("path hook 2", trellis_test_force_path(2, 0), -2);
  expect("path hook tiles", trellis_test_force_path(0, -1), -2);
  for (int path = -1; path <= 1; ++path) {
    expect("path hook", trellis_test_force_path(path, path == 1 ? 16 : 0), 0);
    for (const trellis_geom &g : {good, big})
      for (int32_t m : {1, 16, 129, 5000, TRELLIS_MAX_ROWS}) {
        expect("adapters in domain", trellis_adapters(p, m, c, p, g, p, p, gain, index, 3, 17, p, nullptr), TRELLIS_E_HIP);
        expect("adapters_backward in domain",
               trellis_adapters_backward(p, p, m, c, p, g, p, p, gain, index, TRELLIS_MAX_ADAPTERS, TRELLIS_MAX_RANK, p, p, p, nullptr),
               TRELLIS_E_HIP);
        expect("gated in domain", trellis_gated(p, m, c, p, c, p, g, p, nullptr, p, nullptr), TRELLIS_E_HIP);
        expect("gated_backward in domain", trellis_gated_backward(p, p, p, m, c, p, c, p, g, p, p, p, nullptr), TRELLIS_E_HIP);
      }
  }
  expect("adapters geometry", trellis_adapters(p, 1, c, p, bad, p, p, gain, index, 1, 1, p, nullptr), TRELLIS_E_GEOMETRY);
  expect("adapters m", trellis_adapters(p, 0, c, p, good, p, p, gain, index, 1, 1, p, nullptr), TRELLIS_E_M);
  expect("adapters count", trellis_adapters(p, 1, c, p, good, p, p, gain, index, 0, 1, p, nullptr), TRELLIS_E_ADAPTERS);
  expect("adapters rank", trellis_adapters(p, 1, c, p, good, p, p, gain, index, 1, 129, p, nullptr), TRELLIS_E_ADAPTERS);
  expect("adapters null", trellis_adapters(p, 1, c, p, good, p, p, gain, nullptr, 1, 1, p, nullptr), TRELLIS_E_NULL);
  expect("adapters align", trellis_adapters(p + 1, 1, c, p, good, p, p, gain, index, 1, 1, p, nullptr), TRELLIS_E_ALIGN);
  expect("gated null", trellis_gated(p, 1, c, p, nullptr, p, good, p, p, p, nullptr), TRELLIS_E_NULL);
  expect("gated align", trellis_gated(p, 1, c, p, c, p, good, p, p + 1, p, nullptr), TRELLIS_E_ALIGN);
  expect("gated_backward m", trellis_gated_backward(p, p, p, TRELLIS_MAX_ROWS + 1, c, p, c, p, good, p, p, p, nullptr), TRELLIS_E_M);
  if (failures) return 1;
  printf("rows driver ok\n");
  return 0;
}
