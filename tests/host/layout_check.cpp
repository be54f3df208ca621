// Drives the layout check of the contiguous forms on host memory: the few HIP calls that it makes are replaced here, and an
// allocation of more than 1 MB throws, as it does where memory has run out.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <vector>

#include "dg.h"
#include "host.hpp"

static bool g_limit = false;

void* operator new(size_t n) {
  void* p = g_limit && n > ((size_t)1 << 20) ? nullptr : std::malloc(n);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

extern "C" {
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = hipStreamCaptureStatusNone;
  return hipSuccess;
}
hipError_t hipMemcpyAsync(void* d, const void* s, size_t n, hipMemcpyKind, hipStream_t) {
  std::memcpy(d, s, n);
  return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

static int g_bad = 0;
static void expect(const std::vector<int32_t>& idx, int64_t M, int want, const char* text) {
  g_limit = true;
  const int rc = dg::check_contiguous_layout(idx.data(), M, 5, nullptr);
  g_limit = false;
  if (rc == DG_OK) dg::ok();
  if (rc != want || !std::strstr(dg_get_last_error(), text)) {
    std::printf("M %lld: %d, \"%s\"\n", (long long)M, rc, dg_get_last_error());
    ++g_bad;
  }
}

int main() {
  std::vector<int32_t> idx((size_t)1 << 22, -1);
  const int64_t M = (int64_t)idx.size();
  for (int64_t b = 0; b < M / 128; b += 3)
    for (int64_t r = 0; r < 100; ++r) idx[b * 128 + r] = (int32_t)(b % 5);
  setenv("DG_CHECK_LAYOUT", "1", 1);
  expect(idx, M, DG_OK, "");
  expect(idx, M - 77, DG_OK, "");
  expect(idx, 1, DG_OK, "");
  for (int64_t at : {(int64_t)3 * 128, (int64_t)16383, (int64_t)16384, (int64_t)16385, M / 2 + 5, M - 1}) {
    auto two = idx;
    const int64_t b = at / 128 * 128;
    char text[64];
    std::snprintf(text, sizeof(text), "rows %lld..%lld ", (long long)b, (long long)b + 127);
    for (int64_t r = b; r < b + 128; ++r) two[r] = r < b + 64 ? 1 : 1 + (r == at || at < b + 64);
    if (at < b + 64) two[at] = 1;
    two[b + 127] = 2;
    expect(two, M, DG_ERR_INVALID_ARG, text);
    two[b + 127] = 99;  // padding
    for (int64_t r = b; r < b + 127; ++r) two[r] = 1;
    expect(two, M, DG_OK, "");
  }
  std::printf("%d failures\n", g_bad);
  return g_bad != 0;
}
