// nk_chunk.cuh -- parameters and launcher of the ragged chunk attention
// (nk_chunk.cu).
#pragma once

#include "nk_common.cuh"

namespace nk {
namespace chunk {

constexpr int kRows = 128;  // query rows of a tile

struct Params {
  const uint8_t* pool;
  int num_pages, P, Hkv;
  ChunkLayout lay;
  const uint16_t* q;  // bf16 [total_q][Hq][D]
  const int32_t* cu;  // [B + 1]
  const int32_t* bt;
  int max_pages;
  const int32_t* ctx;
  int B, total_q, Hq, G;
  float scale2;  // sm_scale * log2(e)
  int max_ctx;
  int window, sinks;  // window 0: the whole context
  int n_ctas;
  // Workspace. CTA c leaves a partial of the tile it begins but does not
  // finish in slot 2 c + 1, of the tile it did not begin in slot 2 c.
  float* part_o;    // [2 n_ctas][D / 4][128] float4: normalized by the partial's own sum
  float* part_lse;  // [2 n_ctas][128]
  int4* desc;       // [n_ctas]: the tile CTA c began and did not finish, to be joined:
                    // first query row of its sequence, kv-head (-1: no such tile), first row
                    // of the tile in its unit, rows | CTAs << 8
  uint16_t* out;
  int32_t* status;
  unsigned long long wait_cycles;
  int withhold;  // failure-detection tests: K and V blocks from this number on are never handed over (-1: all are)
};

cudaError_t launch(const Params& p, int D, cudaStream_t st);

}  // namespace chunk
}  // namespace nk
