// The shared-memory limits of kernels (set_smem_limit), on the host with a fake CUDA runtime: prints "good" or what is wrong.
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <map>
#include <mutex>
#include <thread>
#include <utility>

static std::atomic<int> calls{0}, device{0};
static std::mutex mu;
static std::map<std::pair<const void*, int>, int> limits;  // what the runtime holds

static cudaError_t fake_device(int* dev) {
  *dev = device;
  return cudaSuccess;
}
static cudaError_t fake_set(const void* kernel, cudaFuncAttribute, int bytes) {
  ++calls;
  // of two sizes that are set at once the smaller arrives last
  std::this_thread::sleep_for(std::chrono::milliseconds(bytes == 300 ? 300 : bytes == 400 ? 100 : 0));
  std::lock_guard<std::mutex> lock(mu);
  limits[{kernel, device}] = bytes;
  return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#include "nk_common.cuh"

static int limit(const void* kernel) { return limits[{kernel, device}]; }

int main() {
  static char kernel[8][400];
  int bad = 0;
  const auto wrong = [&](const char* what) { bad += printf("%s\n", what) > 0; };
  // two threads, first calls of one kernel
  std::thread a([] { nk::set_smem_limit(kernel[0], 400); }), b([] { nk::set_smem_limit(kernel[0], 300); });
  a.join();
  b.join();
  if (limit(kernel[0]) < 400) wrong("a larger limit was taken back");
  // sizes that grow call after call (a conversation) leave room for other kernels
  for (int i = 1; i <= 1000; ++i) {
    nk::set_smem_limit(kernel[1], 1000 + i);
    if (limit(kernel[1]) < 1000 + i) wrong("a limit was not raised");
  }
  nk::set_smem_limit(kernel[2], 50);
  int before = calls;
  nk::set_smem_limit(kernel[2], 50);
  nk::set_smem_limit(kernel[1], 1000);
  if (calls != before || limit(kernel[1]) < 2000) wrong("a limit that was there was set again");
  // as many kernels as a library has, on another device too
  for (int d = 0; d < 2; ++d) {
    device = d;
    for (int i = 0; i < 400; ++i) nk::set_smem_limit(&kernel[3][i], 100 + i);
    before = calls;
    bool same = true;
    for (int i = 0; i < 400; ++i) {
      nk::set_smem_limit(&kernel[3][i], 100 + i);
      same = same && limit(&kernel[3][i]) == 100 + i;
    }
    if (!same) wrong("a kernel has another's limit");
    if (calls != before) wrong("the table is too small");
  }
  if (!bad) printf("good\n");
  return bad != 0;
}
