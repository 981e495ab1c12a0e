// Drives the losses' and the embedding's host code over a stand-in for the HIP
// runtime (tests/test_vocabulary_launches.py): every launch of every accepted
// size must be one that the runtime accepts (fewer than 2^32 threads along x, at
// most 65535 workgroups along y, 1024 threads and 160 KB of LDS a workgroup). No
// kernel is launched. Exits 0 if everything is as expected.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include <vector>

namespace fake {
long launches = 0, bad = 0;
std::vector<void *> live;
const char *what = "";
long long m, n, k;

hipError_t malloc(void **p, size_t) {
  *p = ::malloc(16);
  live.push_back(*p);
  return hipSuccess;
}
hipError_t capturing(hipStream_t, hipStreamCaptureStatus *s) {
  *s = hipStreamCaptureStatusNone;
  return hipSuccess;
}
hipError_t device(int *d) {
  *d = 0;
  return hipSuccess;
}
hipError_t device_attribute(int *v, hipDeviceAttribute_t, int) {
  *v = 256;
  return hipSuccess;
}
template <typename F, typename... A>
void launch(F, dim3 grid, dim3 block, size_t lds, hipStream_t, A &&...) {
  ++launches;
  const unsigned long long x = (unsigned long long)grid.x * block.x;
  if (grid.x >= 1 && x < (1ull << 32) && grid.y >= 1 && grid.y <= 65535 && grid.z == 1 && block.x <= 1024 && lds <= 160 * 1024)
    return;
  if (bad++ < 10)
    printf("%s m %lld n %lld k %lld: %u x %u workgroups of %u, %zu bytes of LDS\n", what, m, n, k, grid.x, grid.y, block.x, lds);
}
}  // namespace fake

#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL fake::launch
#define hipMalloc fake::malloc
#define hipGetLastError() hipSuccess
#define hipStreamIsCapturing fake::capturing
#define hipGetDevice fake::device
#define hipDeviceGetAttribute fake::device_attribute
#define hipFuncSetAttribute(...) hipSuccess

#include "rows.hip"

static void expect(int status) {
  if (status == TRELLIS_OK) return;
  printf("%s m %lld n %lld k %lld: status %d\n", fake::what, fake::m, fake::n, fake::k, status);
  ++fake::bad;
}

int main() {
  alignas(16) static uint16_t buf[64];
  const uint32_t *c = reinterpret_cast<const uint32_t *>(buf);
  const int32_t *i = reinterpret_cast<const int32_t *>(buf);
  const float *z = reinterpret_cast<const float *>(buf);
  float *f = reinterpret_cast<float *>(buf);
  for (int k : {256, 512, 1280, 5120, 32768, 65536, 129024, 131072, TRELLIS_MAX_K})
    for (int m : {1, 333, 4097, 70000, 262144, TRELLIS_MAX_ROWS - 1, TRELLIS_MAX_ROWS}) {
      fake::m = m;
      fake::k = k;
      fake::n = 0;
      fake::what = "loss_backward";
      expect(trellis_loss_backward(z, buf, m, k, buf, nullptr));
      fake::what = "embed_backward";
      for (int count : {1, 300, 70000, TRELLIS_MAX_TRAINED}) expect(trellis_embed_backward(buf, i, m, k, 0, count, 1.f, buf, nullptr));
      for (int n : {4, 260, 50004, TRELLIS_MAX_N}) {
        fake::n = n;
        const trellis_geom g{n, k, 256, 12, 3};
        fake::what = "embed";
        expect(trellis_embed(i, m, c, buf, g, 1.f, nullptr, 0, buf, nullptr));
        if ((double)m * n * k > 1e16) continue;  // (many chunks of rows: minutes)
        for (uint16_t *dx : {(uint16_t *)nullptr, buf}) {
          fake::what = "cross_entropy";
          expect(trellis_cross_entropy(buf, m, c, buf, g, i, f, f, dx, nullptr));
          fake::what = "distill";
          expect(trellis_distill(buf, m, c, buf, g, i, z, TRELLIS_MAX_TOP, 1.f, f, f, dx, nullptr));
        }
      }
    }
  for (void *p : fake::live) ::free(p);
  if (fake::bad) {
    printf("%ld launches or calls not as they must be\n", fake::bad);
    return 1;
  }
  printf("vocabulary launches ok: %ld\n", fake::launches);
  return 0;
}
