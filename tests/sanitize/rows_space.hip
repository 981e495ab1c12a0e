// Drives the fine-tuned layers' host code over a stand-in for the HIP runtime
// whose calls fail when told to and whose last error stays until it is read, as
// the runtime's does (tests/test_rows_runtime_errors.py): what a call returns
// when an allocation, the clearing of counters or the query of the stream
// fails, what it leaves allocated, and that no error is left behind for the
// caller's next check. No kernel is launched. Exits 0 if everything is as
// expected.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include <set>

namespace fake {
hipError_t last = hipSuccess;
int fail_mallocs = 0;           // how many of the next allocations fail
bool fail_launch = false, fail_query = false, fail_attribute = false;
hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
int launches = 0;
std::set<void *> live;

hipError_t set(hipError_t e) {
  if (e != hipSuccess) last = e;
  return e;
}
hipError_t last_error() {
  const hipError_t e = last;
  last = hipSuccess;
  return e;
}
hipError_t malloc(void **p, size_t) {
  if (fail_mallocs > 0) {
    --fail_mallocs;
    return set(hipErrorOutOfMemory);
  }
  *p = ::malloc(16);
  live.insert(*p);
  return hipSuccess;
}
hipError_t free(void *p) {
  live.erase(p);
  ::free(p);
  return hipSuccess;
}
hipError_t capturing(hipStream_t, hipStreamCaptureStatus *s) {
  *s = capture;
  return fail_query ? set(hipErrorStreamCaptureImplicit) : hipSuccess;
}
hipError_t device(int *d) {
  *d = 0;
  return hipSuccess;
}
hipError_t device_attribute(int *v, hipDeviceAttribute_t, int) {
  *v = 256;
  return hipSuccess;
}
hipError_t func_attribute(const void *, hipFuncAttribute, int) {
  return fail_attribute ? set(hipErrorInvalidValue) : hipSuccess;
}
template <typename F, typename... A>
void launch(F, dim3, dim3, size_t, hipStream_t, A &&...) {
  ++launches;
  if (fail_launch) last = hipErrorLaunchFailure;
}
}  // namespace fake

#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL fake::launch
#define hipMalloc fake::malloc
#define hipFree fake::free
#define hipGetLastError fake::last_error
#define hipStreamIsCapturing fake::capturing
#define hipGetDevice fake::device
#define hipDeviceGetAttribute fake::device_attribute
#define hipFuncSetAttribute fake::func_attribute

#include "rows.hip"

static int failures = 0;
static void expect(const char *what, long got, long want) {
  printf("%-64s %ld\n", what, got);
  if (got != want) {
    printf("  expected %ld\n", want);
    ++failures;
  }
}

static int call(int stream, int m) {
  alignas(16) static uint16_t buf[64];
  const uint32_t *c = reinterpret_cast<const uint32_t *>(buf);
  return trellis_gated(buf, m, c, buf, c, buf, trellis_geom{4096, 4096, 256, 12, 4}, buf, nullptr, nullptr,
                       reinterpret_cast<void *>((intptr_t)stream));
}

int main() {
  trellis_test_force_path(0, 0);
  expect("first call", call(1, 16), TRELLIS_OK);
  expect("its workspace and counters", (long)fake::live.size(), 2);

  fake::last = hipErrorInvalidValue;  // the caller's own, unread
  expect("first call on a stream after an error of the caller's", call(2, 16), TRELLIS_OK);

  // A third more is needed: half more does not fit, the size itself does; the
  // counters grow too.
  expect("another first call", call(5, 96), TRELLIS_OK);
  long live = (long)fake::live.size();
  fake::fail_mallocs = 1;
  expect("a grown call whose first allocation fails", call(5, 300), TRELLIS_OK);
  expect("  a workspace and counters more", (long)fake::live.size() - live, 2);
  expect("  no error left", fake::last_error(), hipSuccess);

  live = (long)fake::live.size();
  fake::fail_mallocs = 2;
  expect("a grown call without memory", call(1, 300), TRELLIS_E_HIP);
  expect("  nothing more allocated", (long)fake::live.size() - live, 0);
  expect("  no error left", fake::last_error(), hipSuccess);
  fake::fail_mallocs = 0;

  fake::fail_launch = true;
  expect("a first call that cannot clear its counters", call(3, 16), TRELLIS_E_HIP);
  expect("  its workspace alone is kept", (long)fake::live.size() - live, 1);
  expect("  no error left", fake::last_error(), hipSuccess);
  fake::fail_launch = false;
  expect("the call again", call(3, 16), TRELLIS_OK);

  live = (long)fake::live.size();
  int launches = fake::launches;
  fake::fail_query = true;
  expect("a stream whose capture cannot be told", call(4, 16), TRELLIS_E_HIP);
  fake::fail_query = false;
  fake::capture = hipStreamCaptureStatusActive;
  expect("a first call in a capture", call(4, 16), TRELLIS_E_HIP);
  fake::capture = hipStreamCaptureStatusNone;
  expect("  nothing allocated", (long)fake::live.size() - live, 0);
  expect("  nothing launched", fake::launches - launches, 0);
  expect("  no error left", fake::last_error(), hipSuccess);

  trellis_test_force_path(1, 0);
  fake::fail_attribute = true;
  expect("a kernel without its shared memory", call(1, 16), TRELLIS_E_HIP);
  expect("  no error left", fake::last_error(), hipSuccess);
  fake::fail_attribute = false;
  expect("the call again", call(1, 16), TRELLIS_OK);

  for (void *p : fake::live) ::free(p);
  if (failures) return 1;
  printf("rows space ok\n");
  return 0;
}
