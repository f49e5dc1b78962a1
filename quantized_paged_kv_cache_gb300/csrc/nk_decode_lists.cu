// nk_decode_lists.cu -- decode / verify attention over lists of pages: the
// LISTS instances of the mma.sync decode kernel (INT8 group-64 pools with fp32
// scales). Each query token of each kv-head has a list of its own, so a unit is
// one token's G rows (G <= 48) and not the T * G of a verify round. What differs
// from whole-context decode is in nk_common.cuh (SparseShape: which pages a unit
// owns) and in the kernel's page mapping and masks.
//
// Bounded by the pages' bytes, P * (2 D + D / 8) for each listed page and
// kv-head; few pages by latency (lengths, list, table, page, merge, combine:
// each a round trip behind the last).
#include "nk_decode_mma.cuh"

namespace nk {
namespace mma {

template <int D, int NT, int CS>
static cudaError_t launch_l(const CUtensorMap& map, const DecodeParams& p, cudaStream_t st) {
  const Geometry geo = geometry(kFmtI8F32, D, NT, CS, p.P, p.B, kKeysLists);
  if (geo.stages < 2 || geo.total > kSmemLimit) return cudaErrorInvalidConfiguration;
  cudaError_t e =
      set_smem_limit(reinterpret_cast<const void*>(decode_mma_kernel<D, NT, CS, kFmtI8F32, kKeysLists>), geo.total);
  if (e != cudaSuccess) return e;
  return launch_chained(decode_mma_kernel<D, NT, CS, kFmtI8F32, kKeysLists>, dim3(p.n_ctas), dim3(kThreads), geo.total,
                        st, map, map, p);
}

// warps per team as channel_split (nk_decode_mma.cu)
cudaError_t launch_lists(const CUtensorMap& map, const DecodeParams& p, int NT, cudaStream_t st) {
  if (p.fmt != kFmtI8F32) return cudaErrorInvalidConfiguration;
  if (p.D == 256) switch (NT) {
      case 1: return launch_l<256, 1, 1>(map, p, st);
      case 2: return launch_l<256, 2, 2>(map, p, st);
      case 3: return launch_l<256, 3, 2>(map, p, st);
      case 4: return launch_l<256, 4, 4>(map, p, st);
      case 5: return launch_l<256, 5, 4>(map, p, st);
      case 6: return launch_l<256, 6, 4>(map, p, st);
      default: return cudaErrorInvalidConfiguration;
    }
  if (p.D == 128) switch (NT) {
      case 1: return launch_l<128, 1, 1>(map, p, st);
      case 2: return launch_l<128, 2, 1>(map, p, st);
      case 3: return launch_l<128, 3, 1>(map, p, st);
      case 4: return launch_l<128, 4, 2>(map, p, st);
      case 5: return launch_l<128, 5, 2>(map, p, st);
      case 6: return launch_l<128, 6, 2>(map, p, st);
      default: return cudaErrorInvalidConfiguration;
    }
  switch (NT) {
    case 1: return launch_l<64, 1, 1>(map, p, st);
    case 2: return launch_l<64, 2, 1>(map, p, st);
    case 3: return launch_l<64, 3, 1>(map, p, st);
    case 4: return launch_l<64, 4, 1>(map, p, st);
    case 5: return launch_l<64, 5, 1>(map, p, st);
    case 6: return launch_l<64, 6, 1>(map, p, st);
    default: return cudaErrorInvalidConfiguration;
  }
}

}  // namespace mma

bool decode_lists_supported(int D, int G, int P) {
  if (G < 1 || G > 48 || P % 16 != 0 || P > 256 || !(D == 64 || D == 128 || D == 256)) return false;
  const int NT = (G + 7) / 8;
  return mma::geometry(kFmtI8F32, D, NT, mma::channel_split(D, NT), P, kMaxBatch, kKeysLists).stages >= 2;
}

}  // namespace nk
