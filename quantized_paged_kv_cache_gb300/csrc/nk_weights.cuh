// nk_weights.cuh -- parameters and helpers shared by the kernels of
// nk_page_weights.
#pragma once

#include <cuda_fp16.h>

#include "nk_common.cuh"

namespace nk {

struct WeightParams {
  const uint8_t* pool;
  ChunkLayout lay;
  int num_pages, D;
  const uint16_t* q;  // bf16 [B][T][Hq][D]
  const int32_t* bt;
  const int32_t* ctx;
  SplitShape sh;
  int G, rows, chunk; // rows: T * G in whole chunks of `chunk` rows (whole tiles of eight)
  float scale2;       // sm_scale * log2(e)
  int n_ctas;
  int parts, takes;   // log-sums of a page; of a segment (the tcgen05 kernel: of 32 keys each, four)
  float* page_lse;    // [item][parts][rows], base 2, -inf: no key seen
  float* seg_lse;     // [n_ctas + B * Hkv][takes][rows]
  const float* prior; // may be NULL
  const int32_t* seen;  // may be NULL
  float* out;         // [num_pages][Hkv]
  int32_t* status;
  unsigned long long wait_cycles;  // of every bounded wait
  int withhold;                    // steps from this number on are never copied (-1: all are): tests
};

__device__ __forceinline__ float wgt_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t wgt_prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t wgt_f16(uint32_t biased, uint32_t sel) {
  const uint32_t h = wgt_prmt(biased, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h),
                            __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void wgt_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// log-sums (m: largest, l: sum of 2^(s - m); l is 0 while m is -inf)
__device__ __forceinline__ void lse_join(float& m, float& l, float m2, float l2) {
  const float mx = fmaxf(m, m2);
  if (mx == -INFINITY) {
    l += l2;  // nothing, or NaN, which stays
    return;
  }
  l = l * wgt_ex2(m - mx) + l2 * wgt_ex2(m2 - mx);
  m = mx;
}
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }

// fp16 scaling of a query row: exponent e that brings its largest |q| into
// [2^14, 2^15).
__device__ __forceinline__ int wgt_row_exp(float m) {
  if (!(m > 0.f)) return 0;
  const int e = 14 - ((int)((__float_as_uint(m) >> 23) & 0xffu) - 127);
  return e > 110 ? 110 : (e < -113 ? -113 : e);
}
__device__ __forceinline__ float wgt_pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// What a row with largest |q| m is multiplied by. An infinite one becomes NaN
// throughout: its scores could all be minus infinity, as those of a row that sees
// no key.
__device__ __forceinline__ float wgt_row_factor(float m, int e) {
  return m < INFINITY ? wgt_pow2(e) : __uint_as_float(0x7fffffffu);
}

// The first kernel on tcgen05 (nk_weights_tc.cu).
cudaError_t launch_lse_tc(const WeightParams& p, int chunks, cudaStream_t st);

}  // namespace nk
