// Host-only harness for the int8 and expert entry points, built with
// AddressSanitizer and UndefinedBehaviorSanitizer (host code only) by
// tests/test_ops_sanitizers.py: many calls with sizes, pitches and counts from
// the ends of their ranges.  One pointer of every call is misaligned or null, so
// each is refused (or has no work) before any launch, and no GPU is needed;
// dgemm_kernel_config runs the kernel choice over many shapes.  Exit status
// 0 when every status is a documented one and none is a launch.
#include <cstdint>
#include <cstdio>
#include <random>

#include "dgemm.h"

namespace {

std::mt19937_64 rng(1);

int64_t size() {
  static const int64_t v[] = {INT64_MIN, -1, 0, 1, 2, 3, 15, 16, 17, 32, 100, 127, 128, 131071, 131072, 1 << 20,
                              (int64_t(1) << 31) - 1, int64_t(1) << 31, (int64_t(1) << 31) + 1, int64_t(1) << 40,
                              int64_t(1) << 62, INT64_MAX};
  return v[rng() % (sizeof v / sizeof *v)];
}

int type() { return (int)(rng() % 5) - 1; }

// A null pointer once in n, else a 16-byte aligned address that nothing reads.
template <class T>
T* ptr(int n) {
  return rng() % n ? (T*)(uintptr_t)(1 << 20) : nullptr;
}

// An address no call accepts: null or misaligned.
template <class T>
T* bad() {
  return (T*)(uintptr_t)(rng() % 9 ? (1 << 20) + 1 : 0);
}

}  // namespace

int main() {
  long count[16] = {0};
  char text[256];
  for (int i = 0; i < 300000; ++i) {
    int st = 0;
    switch (rng() % 8) {
      case 0:
        st = gemm_i8_scaled(size(), size(), size(), ptr<int8_t>(9), size(), ptr<int8_t>(9), size(), ptr<void>(9), size(),
                            type(), ptr<float>(9), rng() % 2 ? 1 : size(), bad<float>(), rng() % 2 ? 1 : size(),
                            (int)(rng() % 4) - 1, nullptr);
        break;
      case 1:
        st = gemm_i8_grouped(size(), size(), size(), size(), ptr<int8_t>(9), size(), size(), ptr<int32_t>(2),
                             ptr<int8_t>(9), size(), size(), ptr<void>(9), size(), type(), ptr<float>(9),
                             rng() % 2 ? 1 : size(), bad<float>(), rng() % 2 ? 1 : size(), ptr<int32_t>(9), nullptr);
        break;
      case 2:
        st = quantize_i8(size(), size(), ptr<void>(9), size(), type(), ptr<int8_t>(9), size(), bad<float>(), nullptr);
        break;
      case 3:
        (void)expert_sort_workspace(size(), size(), size());
        st = expert_sort(size(), size(), size(), ptr<void>(9), 4 << (rng() % 3), bad<int32_t>(), ptr<int32_t>(9),
                         ptr<int32_t>(9), ptr<int32_t>(2), ptr<void>(2), size(), nullptr);
        break;
      case 4:
        st = expert_dispatch(size(), size(), size(), type(), ptr<void>(9), size(), bad<int32_t>(), ptr<void>(9), size(),
                             size(), nullptr);
        break;
      case 5:
        // (k == 0 needs no slots: zeros would be written)
        st = expert_combine(size(), 1 + (size() & 7), size(), type(), ptr<void>(9), size(), size(), bad<int32_t>(),
                            ptr<float>(2), ptr<void>(9), size(), nullptr);
        break;
      case 6:
        st = expert_combine_grad(size(), size(), size(), type(), ptr<void>(9), size(), ptr<void>(9), size(), size(),
                                 bad<int32_t>(), ptr<float>(2), ptr<void>(2), size(), ptr<float>(2), nullptr);
        break;
      default:
        st = dgemm_kernel_config(6 + (int)(rng() % 3), (int)(rng() % 2), 1 + (int64_t)(rng() % 40000),
                                 1 + (int64_t)(rng() % 40000), (int64_t)(rng() % 20000), text, sizeof text);
    }
    if (st < 0 || st > DGEMM_ERR_INVALID_TYPE || st == DGEMM_ERR_HIP) {
      std::fprintf(stderr, "FAIL: status %d at call %d\n", st, i);
      return 1;
    }
    ++count[st];
  }
  for (int s = 0; s <= DGEMM_ERR_INVALID_TYPE; ++s) std::printf("%d:%ld ", s, count[s]);
  std::printf("0 failures\n");
  return 0;
}
