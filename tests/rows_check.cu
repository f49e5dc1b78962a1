// Which results nk_verify_drafts takes beside inputs whose rows lie apart, on the host with a fake CUDA runtime: prints "good" or
// what is wrong. Nothing is launched, and no pointer is followed.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

static int launches = 0;
template <class... A>
static cudaError_t fake_launch(const cudaLaunchConfig_t*, A&&...) {
  ++launches;
  return cudaSuccess;
}
#define cudaLaunchKernelEx fake_launch
#include "nk_verify.cu"

int main() {
  constexpr int B = 3, T = 3, V = 100;
  constexpr int64_t stride = 1 << 20;
  const auto at = [](int64_t x) { return reinterpret_cast<void*>((uintptr_t)x); };
  const auto f = [&](int64_t x) { return reinterpret_cast<const float*>(at(x)); };
  const auto i = [&](int64_t x) { return reinterpret_cast<int32_t*>(at(x)); };
  constexpr int64_t one = int64_t(1) << 40, two = int64_t(1) << 44, rest = int64_t(1) << 48, far = 1 << 24;
  const auto call = [&](int64_t tokens) {
    launches = 0;
    const int rc = nk_verify_drafts(f(one), stride, f(two), stride, i(rest), nullptr, f(rest + far), B, T, V, nullptr, i(tokens),
                                    i(rest + 2 * far), nullptr, nullptr, nullptr);
    return rc == NK_OK && launches == 1 ? 1 : (rc == NK_ERR_SHAPE && launches == 0 ? 0 : -1);
  };
  constexpr int64_t bytes = B * T * 4;
  int bad = 0;
  for (const int64_t base : {one, two}) {
    const int rows = base == one ? B * T : B * (T - 1);
    for (int row = -1; row < rows; ++row) {
      // the room behind a row (row -1: in front of the first)
      const int64_t begin = row < 0 ? base - 4096 : base + (row * stride + V) * 4, end = base + (row + 1) * stride * 4;
      bad += call(begin) != 1;
      bad += call((begin + end) / 2 / 4 * 4) != 1;
      if (row >= 0) bad += call(begin - 4) != 0;
      bad += call(end - bytes) != 1;
      bad += call(end - bytes + 4) != (row + 1 < rows ? 0 : 1);
    }
  }
  printf(bad ? "%d wrong\n" : "good\n", bad);
  return bad != 0;
}
