// How nk_page_select is launched on devices that hold no cluster of sixteen blocks, on the host with a fake CUDA runtime.
//   cluster_check <clusters of sixteen that the device holds>: prints the cluster, the shared memory and the workspace of a
//   few calls, and "bad" where a launch would not fit.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <cstdio>
#include <cstdlib>

static int sixteens = 0;
static int launches = 0, cluster = 0;
static size_t shared = 0;

static cudaError_t fake_device(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
template <class K>
static cudaError_t fake_set(K, cudaFuncAttribute, int) {
  return cudaSuccess;
}
static int cluster_of(const cudaLaunchConfig_t* cfg) {
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) return (int)cfg->attrs[i].val.clusterDim.x;
  return 1;
}
template <class... A>
static cudaError_t fake_launch(const cudaLaunchConfig_t* cfg, A&&...) {
  ++launches;
  cluster = cluster_of(cfg);
  shared = cfg->dynamicSmemBytes;
  return cluster > 8 && sixteens == 0 ? cudaErrorInvalidConfiguration : cudaSuccess;
}
template <class K>
static cudaError_t fake_occupancy(int* n, K, const cudaLaunchConfig_t* cfg) {
  *n = cluster_of(cfg) > 8 ? sixteens : 8;
  return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#define cudaLaunchKernelEx fake_launch
#define cudaOccupancyMaxActiveClusters fake_occupancy
#include "nk_select.cu"

namespace nk {
int check_pool(const nk_kv_pool*) { return NK_OK; }
int device_sms() { return 152; }
WaitLimits wait_limits() { return {0, -1}; }
}  // namespace nk

int main(int argc, char** argv) {
  sixteens = argc > 1 ? atoi(argv[1]) : 0;
  void* fake = reinterpret_cast<void*>(uintptr_t(1) << 20);
  int32_t* fi = reinterpret_cast<int32_t*>(fake);
  const int shapes[][4] = {{1, 1, 24, 4096}, {1, 4, 24, 4096}, {2, 1, 24, 4096}, {1, 16, 16, 4096}, {8, 4, 24, 1024}, {1, 1, 4, 16000}};
  for (const auto& s : shapes) {
    const int B = s[0], T = s[1], Hq = s[2], ctx = s[3] * 64;
    const size_t ws = nk_page_select_workspace_bytes(B, T, Hq, 4, 256, 64, ctx);
    launches = 0;
    const int rc = nk_page_select(fake, 1 << 20, 64, 4, 256, fake, fi, s[3], fi, B, T, Hq, ctx, 64, 1, 2, ws ? fake : nullptr, ws, fi,
                                  nullptr, nullptr);
    printf("%d %d %zu %zu%s\n", launches, launches == 1 ? cluster : 0, launches == 1 ? shared : 0, ws, rc == NK_OK ? "" : " bad");
  }
  return 0;
}
