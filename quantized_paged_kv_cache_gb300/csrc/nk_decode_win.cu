// nk_decode_win.cu -- decode / verify attention over a sliding window with
// sinks: the WIN instances of the mma.sync decode kernel (INT8 group-64 pools
// with fp32 scales). What differs from whole-context decode is in
// nk_common.cuh (WindowShape: which pages a unit owns) and in the kernel's
// page mapping and masks.
#include "nk_decode_mma.cuh"

namespace nk {
namespace mma {

template <int D, int NT, int CS>
static cudaError_t launch_w(const CUtensorMap& map, const DecodeParams& p, cudaStream_t st) {
  const Geometry geo = geometry(kFmtI8F32, D, NT, CS, p.P, p.B, true);
  if (geo.stages < 2 || geo.total > kSmemLimit) return cudaErrorInvalidConfiguration;
  cudaError_t e =
      set_smem_limit(reinterpret_cast<const void*>(decode_mma_kernel<D, NT, CS, kFmtI8F32, true>), geo.total);
  if (e != cudaSuccess) return e;
  return launch_chained(decode_mma_kernel<D, NT, CS, kFmtI8F32, true>, dim3(p.n_ctas), dim3(kThreads), geo.total, st,
                        map, map, p);
}

// warps per team as channel_split (nk_decode_mma.cu)
cudaError_t launch_window(const CUtensorMap& map, const DecodeParams& p, int NT, cudaStream_t st) {
  if (p.fmt != kFmtI8F32) return cudaErrorInvalidConfiguration;
  if (p.D == 256) switch (NT) {
      case 1: return launch_w<256, 1, 1>(map, p, st);
      case 2: return launch_w<256, 2, 2>(map, p, st);
      case 3: return launch_w<256, 3, 2>(map, p, st);
      case 4: return launch_w<256, 4, 4>(map, p, st);
      case 5: return launch_w<256, 5, 4>(map, p, st);
      case 6: return launch_w<256, 6, 4>(map, p, st);
      default: return cudaErrorInvalidConfiguration;
    }
  if (p.D == 128) switch (NT) {
      case 1: return launch_w<128, 1, 1>(map, p, st);
      case 2: return launch_w<128, 2, 1>(map, p, st);
      case 3: return launch_w<128, 3, 1>(map, p, st);
      case 4: return launch_w<128, 4, 2>(map, p, st);
      case 5: return launch_w<128, 5, 2>(map, p, st);
      case 6: return launch_w<128, 6, 2>(map, p, st);
      default: return cudaErrorInvalidConfiguration;
    }
  switch (NT) {
    case 1: return launch_w<64, 1, 1>(map, p, st);
    case 2: return launch_w<64, 2, 1>(map, p, st);
    case 3: return launch_w<64, 3, 1>(map, p, st);
    case 4: return launch_w<64, 4, 1>(map, p, st);
    case 5: return launch_w<64, 5, 1>(map, p, st);
    case 6: return launch_w<64, 6, 1>(map, p, st);
    default: return cudaErrorInvalidConfiguration;
  }
}

}  // namespace mma
}  // namespace nk
