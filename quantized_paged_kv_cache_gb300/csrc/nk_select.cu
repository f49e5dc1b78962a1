// nk_select.cu -- which pages of a long cache a query attends to: the pages'
// bounds (nk_page_bounds) and the choice by them (nk_page_select).
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "nk_common.cuh"
#include "nk_host.cuh"
#include "nk_ptx.cuh"
#include "nk_topk.cuh"

namespace nk {

// ---------------------------------------------------------------------------
// Bounds. Of each page and kv-head: hi[d] and lo[d], the largest and smallest
// value fp32(code * scale) that key channel d takes in the page's filled slots,
// as INT8 codes of one scale s = fp32(max(|hi|, |lo|) / 127), by the rounding of
// the cache's own rows. No query's score over the page is above
//   sum_d max(q_d hi_d, q_d lo_d) = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// but for the codes' rounding.
//   codes [num_pages][Hkv][hi | lo][D] int8, then scales [num_pages][Hkv] fp32.
// ---------------------------------------------------------------------------
struct BoundsView {
  uint8_t* codes;
  float* scales;
};
__host__ __device__ inline BoundsView bounds_view(void* base, int64_t num_pages, int Hkv, int D) {
  uint8_t* b = reinterpret_cast<uint8_t*>(base);
  return BoundsView{b, reinterpret_cast<float*>(b + num_pages * Hkv * 2 * D)};
}

// ---------------------------------------------------------------------------
// nk_page_bounds: the touched pages of a step (those that a new row falls in),
// from the codes that its append wrote. Every block forms the prefix of the
// sequences' touched pages itself and takes (page, kv-head) items in turns.
//
// A thread takes 16 bytes of a row at a time and keeps the extremes of its 16
// channels; D / 16 threads hold a row. With more items than blocks a warp takes an
// item, from a ring of its own in shared memory that bulk asynchronous copies fill,
// 16 keys a stage (no barrier between warps; rows merged by shuffles). With fewer
// (a step of single tokens) a block does, straight from global memory, its warps'
// extremes merged through shared memory, so that all of the item's bytes are on
// their way at once.
//
// Bounded by the K codes' and scales' bytes for prompts, by latency for a step of
// single tokens (lengths, table, codes). Codes become fp32 by a byte permute (2^23
// + 128 + code) and a packed subtraction: the conversion instruction takes an
// eighth of their rate. Eight prompts of 8K to 16K tokens (101 MB): 65 us with
// conversions and a block an item, 42 with packed ones and a warp an item that
// loads into registers, 33 with the rings, eight warps of 32 keys or sixteen of 16,
// 28.7 with neighbouring items on different SMs (each warp has two or three).
// ---------------------------------------------------------------------------
struct BoundsParams {
  const uint8_t* pool;
  ChunkLayout lay;
  int num_pages, P, Hkv;
  const int32_t* bt;
  int max_pages;
  const int32_t* start;
  const int32_t* cu;
  int B;
  BoundsView out;
  int32_t* status;
  unsigned long long wait_cycles;  // of a bounded wait
  int withhold;                    // a warp's copies from this number on are never made (-1: all are): tests
};

constexpr int kBndThreads = 512, kBndWarps = kBndThreads / 32;
constexpr int kBndWide = 256;  // threads that share an item
constexpr int kBndKeys = 16, kBndStages = 3;  // of a stage, of a warp's ring
template <int D>
constexpr int bounds_stage() {  // codes, then scales
  return kBndKeys * (D + D / kGroup * 4);
}

__device__ __forceinline__ uint32_t sel_prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// fp32(code * scale) of the four codes of w
__device__ __forceinline__ void values4(uint32_t w, uint64_t scale2, float (&v)[4]) {
  const uint64_t off = pack2(0xcb000080u, 0xcb000080u);  // -(2^23 + 128)
  const uint32_t b = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t x = pack2(sel_prmt(b, 0x4b000000u, i == 0 ? 0x7440 : 0x7442),
                             sel_prmt(b, 0x4b000000u, i == 0 ? 0x7441 : 0x7443));
    const uint64_t y = mul2(add2(x, off), scale2);
    v[2 * i] = __uint_as_float((uint32_t)y);
    v[2 * i + 1] = __uint_as_float((uint32_t)(y >> 32));
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Extremes of rows r0, r0 + step, .. below `filled` at the thread's 16 channels,
// from global or shared memory; true if a scale was not finite.
template <int D, int LOADS>
__device__ __forceinline__ bool row_extremes(const uint8_t* codes, const float* scales, int r0, int step, int filled,
                                             float (&hi)[16], float (&lo)[16]) {
  bool odd = false;
  for (; r0 < filled; r0 += step * LOADS) {
    uint4 w[LOADS];
    float sc[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int r = min(r0 + j * step, filled - 1);  // (a row twice changes nothing)
      w[j] = *reinterpret_cast<const uint4*>(codes + (int64_t)r * D);
      sc[j] = scales[r * (D / kGroup)];
    }
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      if (!(fabsf(sc[j]) < INFINITY)) {  // counts as zeros
        odd = true;
        sc[j] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < LOADS; j += 2) {
      const uint64_t s0 = pack2(__float_as_uint(sc[j]), __float_as_uint(sc[j]));
      const uint64_t s1 = pack2(__float_as_uint(sc[j + 1]), __float_as_uint(sc[j + 1]));
      const uint32_t u0[4] = {w[j].x, w[j].y, w[j].z, w[j].w}, u1[4] = {w[j + 1].x, w[j + 1].y, w[j + 1].z, w[j + 1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v0[4], v1[4];
        values4(u0[i], s0, v0);
        values4(u1[i], s1, v1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hi[4 * i + k] = max3(hi[4 * i + k], v0[k], v1[k]);
          lo[4 * i + k] = min3(lo[4 * i + k], v0[k], v1[k]);
        }
      }
    }
  }
  return odd;
}

// The code of x at scale s, with r = fp32(1 / s): the quotient by the reciprocal is
// off by less than 2^-15 (three roundings of 2^-24 of at most 127), so only one that
// near the border between two codes needs the division itself.
__device__ __forceinline__ uint32_t bound_code(float x, float s, float r) {
  float q = x * r;
  const float n = rintf(q);
  if (!(fabsf(q - n) < 0.4999f)) q = __fdiv_rn(x, s);
  return (uint32_t)(int)fminf(fmaxf(rintf(q), -127.f), 127.f) & 0xffu;
}

template <int D>
__global__ void __launch_bounds__(kBndThreads) page_bounds_kernel(const BoundsParams p) {
  constexpr int LPR = D / 16;  // threads of a row
  constexpr int GR = D / kGroup;
  extern __shared__ __align__(16) uint8_t smem[];  // the warps' rings
  __shared__ int pre[kMaxBatch + 1];               // touched pages before sequence b
  __shared__ int2 span[kMaxBatch];                 // its first new position, one past its last
  __shared__ int warp_tot[kBndWarps];
  __shared__ uint64_t bars[kBndWarps][kBndStages];
  __shared__ int4 meta[kBndWarps][kBndStages];     // record (two words), keys, the item's last
  chain_wait();
  chain_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.P;
  {
    constexpr int PER = kMaxBatch / kBndThreads;
    int v[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = tid * PER + i;
      v[i] = 0;
      if (b < p.B) {
        const int64_t s = p.start[b], n = (int64_t)p.cu[b + 1] - p.cu[b];
        span[b] = make_int2((int)s, (int)(s + n));
        if (s < 0 || n < 0 || s + n > (int64_t)p.max_pages * P || s + n > 0x7fffffff) {
          if (blockIdx.x == 0) flag(p.status, NK_DEVFLAG_BAD_POS);
        } else if (n > 0) {
          v[i] = (int)((s + n + P - 1) / P - s / P);
        }
      }
      sum += v[i];
    }
    int total;
    int run = block_exclusive<kBndThreads>(sum, warp_tot, total);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = tid * PER + i;
      if (b < p.B) pre[b] = run;
      run += v[i];
    }
    if (tid == 0) pre[p.B] = total;
    __syncthreads();
  }
  const int64_t items = (int64_t)pre[p.B] * p.Hkv;
  const int c0 = (lane % LPR) * 16;
  // Item x: what the table says of its page, and its filled slots
  const auto look = [&](int64_t x, int& filled) {
    const int k = (int)quot(x, p.Hkv);
    int b = 0, top = p.B;
    while (top - b > 1) {
      const int mid = (b + top) >> 1;
      if (pre[mid] <= k) b = mid; else top = mid;
    }
    const int2 s = span[b];
    const int logical = s.x / P + (k - pre[b]);
    filled = min(s.y - logical * P, P);
    return p.bt[(int64_t)b * p.max_pages + logical];
  };
  const auto none = [&](int page) {
    if (page >= 0 && page < p.num_pages) return false;
    if (lane == 0) flag(p.status, NK_DEVFLAG_BAD_PAGE);
    return true;
  };
  float hi[16], lo[16];
  const auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      hi[i] = -INFINITY;
      lo[i] = INFINITY;
    }
  };
  const auto merge_lanes = [&]() {  // the rows of a warp share channels: lanes LPR apart
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      }
  };
  const auto store = [&](int64_t rec) {  // by a warp
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fmaxf(fabsf(hi[i]), fabsf(lo[i])));
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = __fdiv_rn(m, 127.f);
    if (s == 0.f) s = 1.f;
    const float r = __frcp_rn(s);  // (infinite for the smallest: every quotient is then divided)
    // lanes below LPR write hi, the next LPR lo
    const bool low = lane >= LPR;
    if (lane < 2 * LPR) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i] |= bound_code(low ? lo[4 * i + j] : hi[4 * i + j], s, r) << (8 * j);
      }
      *reinterpret_cast<uint4*>(p.out.codes + rec * 2 * D + (low ? D : 0) + c0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (lane == 0) p.out.scales[rec] = s;
  };

  if (items <= gridDim.x) {  // a block for each item
    const int64_t x = blockIdx.x;
    if (x >= items || tid >= kBndWide) return;
    int filled;
    const int page = look(x, filled);
    if (none(page)) return;
    const int64_t rec = (int64_t)page * p.Hkv + x % p.Hkv;
    const uint8_t* chunk = p.pool + rec * p.lay.chunk;
    clear();
    if (row_extremes<D, 4>(chunk + c0, reinterpret_cast<const float*>(chunk + p.lay.ks) + c0 / kGroup, tid / LPR,
                           kBndWide / LPR, filled, hi, lo))
      flag(p.status, NK_DEVFLAG_RANGE);
    merge_lanes();
    float* hi_s = reinterpret_cast<float*>(smem) + warp * 2 * D;
    if (lane < LPR) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        *reinterpret_cast<float4*>(hi_s + c0 + i) = make_float4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
        *reinterpret_cast<float4*>(hi_s + D + c0 + i) = make_float4(lo[i], lo[i + 1], lo[i + 2], lo[i + 3]);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kBndWide) : "memory");
    if (warp > 0) return;
#pragma unroll
    for (int w = 0; w < kBndWide / 32; ++w)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        hi[i] = fmaxf(hi[i], reinterpret_cast<const float*>(smem)[w * 2 * D + c0 + i]);
        lo[i] = fminf(lo[i], reinterpret_cast<const float*>(smem)[w * 2 * D + D + c0 + i]);
      }
    store(rec);
    return;
  }

  // ---- a warp for each item
  constexpr int kStage = bounds_stage<D>();
  uint8_t* ring = smem + warp * kBndStages * kStage;
  const uint32_t bar0 = smem_u32(bars[warp]);
  if (lane < kBndStages) {
    mbar_init(bar0 + 8 * lane, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  const int64_t stride = (int64_t)gridDim.x * kBndWarps;
  // the next item to copy, and the one behind it, whose page's number is on its way
  // (neighbouring items on different SMs, so that the last ones are spread over all)
  int64_t x = (int64_t)warp * gridDim.x + blockIdx.x;
  int page = 0, filled = 0, page_b = 0, filled_b = 0, key = 0, issued = 0;
  if (x < items) page = look(x, filled);
  if (x + stride < items) page_b = look(x + stride, filled_b);
  const auto advance = [&]() {
    x += stride;
    page = page_b;
    filled = filled_b;
    key = 0;
    if (x + stride < items) page_b = look(x + stride, filled_b);
  };
  const auto issue = [&]() {
    while (x < items && none(page)) advance();
    if (x >= items) return;
    const int st = issued % kBndStages, rows = min(kBndKeys, filled - key), all = (rows + 15) / 16 * 16;
    const int64_t rec = (int64_t)page * p.Hkv + x % p.Hkv;
    if (lane == 0) {
      const bool held = p.withhold >= 0 && issued >= p.withhold;
      meta[warp][st] = make_int4((int)(rec >> 31), (int)(rec & 0x7fffffff), rows, key + rows >= filled);
      const uint8_t* chunk = p.pool + rec * p.lay.chunk;
      const uint32_t dst = smem_u32(ring + st * kStage), bar = bar0 + 8 * st;
      if (!held) {
        mbar_arrive_expect_tx(bar, all * (D + GR * 4));
        bulk_load(dst, chunk + (int64_t)key * D, all * D, bar);
        bulk_load(dst + kBndKeys * D, chunk + p.lay.ks + key * (GR * 4), all * (GR * 4), bar);
      }
    }
    ++issued;
    key += rows;
    if (key >= filled) advance();
  };
  for (int i = 0; i < kBndStages - 1; ++i) issue();
  clear();
  for (int n = 0; n < issued; ++n) {
    issue();
    const int st = n % kBndStages;
    // (after a wait that ran out nothing more is copied: the loop ends with the copies under way)
    const bool late = !mbar_wait(bar0 + 8 * st, (uint32_t)(n / kBndStages) & 1u, p.wait_cycles);
    if (__any_sync(0xffffffffu, late)) {
      flag(p.status, NK_DEVFLAG_TIMEOUT);
      x = items;
      continue;
    }
    const int4 m = meta[warp][st];
    const uint8_t* codes = ring + st * kStage;
    if (row_extremes<D, 4>(codes + c0, reinterpret_cast<const float*>(codes + kBndKeys * D) + c0 / kGroup, lane / LPR,
                           32 / LPR, m.z, hi, lo))
      flag(p.status, NK_DEVFLAG_RANGE);
    if (m.w) {
      merge_lanes();
      store((int64_t)m.x << 31 | m.y);
      clear();
    }
    __syncwarp();  // the stage's readers are done
  }
}

// nk_page_bounds_values: 16 codes a thread, four stores of 16 bytes.
__global__ void __launch_bounds__(256) bounds_values_kernel(BoundsView v, int64_t pieces, int per_rec, float* out) {
  chain_wait();
  chain_release();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    const uint4 w = reinterpret_cast<const uint4*>(v.codes)[i];
    const float s = v.scales[quot(i, per_rec)];
    const uint64_t s2 = pack2(__float_as_uint(s), __float_as_uint(s));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[4];
      values4(u[j], s2, x);
      reinterpret_cast<float4*>(out)[i * 4 + j] = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// nk_page_select, first kernel: the pages' scores. With one scale s_q for a
// token's rows of a kv-head, q8 = clamp(rint(q / s_q)), page scale s:
//   score = s * max over the G rows of sum_d max(q8_d, 0) hi_d + min(q8_d, 0) lo_d
// (s_q > 0 orders nothing). The sum is a whole number below 127 * 127 * 256 <
// 2^22, so fp16 operands with fp32 sums give it exactly on the tensor cores, and
// its product with s is one 64-bit product: two scores never change places by
// rounding.
//
// A warp takes 16 pages (the M of mma.m16n8k16; the token's rows are N) straight
// from global memory: a page's record is 2 D consecutive bytes, and a thread
// holds 16 consecutive channels of a group of 64, which in the product's K order
// are four steps of four. The rows stay in shared memory as fp16 whole numbers;
// their positive and negative parts are taken at the fragment. Bounded by the
// records' bytes, for one sequence by latency.
// ---------------------------------------------------------------------------
struct SelectParams {
  BoundsView bounds;
  int64_t num_pages;
  int Hkv, G;
  const uint16_t* q;  // bf16 [B][T][Hq][D]
  const int32_t* bt;
  int max_pages;
  const int32_t* ctx;
  int B, T, P, max_ctx, k, sinks, recent;
  int cols;           // tokens of a chunk of rows
  uint64_t* scores;   // [B][T][Hkv][stride]
  int64_t stride;     // pages of the longest context
  int32_t* out;       // [B][T][Hkv][k]
  int32_t* status;
};

__device__ __forceinline__ int select_len(const SelectParams& p, int b) {  // 0: refused
  const int L = p.ctx[b];
  return L < p.T || L > p.max_ctx || (int64_t)L > (int64_t)p.max_pages * p.P ? 0 : L;
}

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelRows = 64;  // query rows of a chunk, at most

// two int8 codes (biased by ^ 0x80808080) as an exact fp16 pair
__device__ __forceinline__ uint32_t sel_f16(uint32_t biased, uint32_t sel) {
  const uint32_t h = sel_prmt(biased, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h),
                            __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void sel_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_max0(uint32_t x) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&x), __halves2half2(__ushort_as_half(0), __ushort_as_half(0)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t half2_min0(uint32_t x) {
  const __half2 r = __hmin2(*reinterpret_cast<const __half2*>(&x), __halves2half2(__ushort_as_half(0), __ushort_as_half(0)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Shared memory: rows [NT * 8][D / 2 + 2 words] fp16, then a warp's products [16][NT * 8 + 1] fp32.
__host__ __device__ inline int select_smem(int D, int NT, int warps) {
  return NT * 8 * (D * 2 + 8) + warps * 16 * (NT * 8 + 1) * 4;
}

// The scores of pages 0 .. seen - 1 of a (sequence, kv-head) for tokens t0 .. t0 +
// cols - 1, 16 pages a warp from block `blk` on: store(t - t0, page, key).
template <int D, int NT, int WARPS, class Store>
__device__ __forceinline__ void score_pages(const SelectParams& p, uint8_t* smem, uint32_t* top_s, int b, int h, int t0,
                                            int cols, int seen, int blk, int stride, const Store& store) {
  constexpr int ROWS = NT * 8;
  constexpr int RS = D * 2 + 8;     // bytes of a row: 2 words past a multiple of 32, distinct banks for the fragments
  constexpr int NC = D / 64;        // 64-channel parts of a record's half
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int blocks = (seen + 15) / 16;
  // the first pages' records are on their way while the rows are made
  uint4 rec[2][2][NC];  // [page g, g + 8][hi, lo][part]
  float scale = 0.f;    // of page `lane`, lanes 0 to 15
  bool there = true;
  const auto load = [&](int bk) {
    const int mine = bk * 16 + (lane & 15);
    int page = -1;
    there = true;
    if (mine < seen) {
      page = p.bt[(int64_t)b * p.max_pages + mine];
      if (page < 0 || page >= p.num_pages) {
        if (lane < 16) flag(p.status, NK_DEVFLAG_BAD_PAGE);
        page = -1;
        there = false;
      }
    }
    if (page >= 0) scale = p.bounds.scales[(int64_t)page * p.Hkv + h];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, g + 8 * i);
      const uint4* src = reinterpret_cast<const uint4*>(p.bounds.codes + ((int64_t)(pg < 0 ? 0 : pg) * p.Hkv + h) * 2 * D);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c) rec[i][s][c] = pg < 0 ? make_uint4(0, 0, 0, 0) : src[(s * D + 64 * c) / 16 + t4];
    }
  };
  if (blk < blocks) load(blk);
  // ---- the rows as whole numbers: a scale for each token. The pieces of all rows
  // stay in registers between the search for the largest and the division.
  const int G = p.G, rows = cols * G;
  constexpr int PER = D / 8;                                          // 16-byte pieces of a row
  constexpr int PCS = (ROWS * PER + WARPS * 32 - 1) / (WARPS * 32);  // of a thread
  uint4 piece[PCS];
  if (tid < NK_MAX_T) top_s[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PCS; ++k) {
    const int i = tid + k * WARPS * 32, row = i / PER, t = row / G;
    piece[k] = make_uint4(0, 0, 0, 0);
    uint32_t m = 0;  // |q| as bits: their order is that of the numbers, infinity and NaN past all
    if (row < rows) {
      const uint16_t* src = p.q + (((int64_t)(b * p.T + t0 + t) * p.Hkv + h) * G + (row - t * G)) * D;
      piece[k] = reinterpret_cast<const uint4*>(src)[i % PER];
      const uint32_t u[4] = {piece[k].x, piece[k].y, piece[k].z, piece[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, max((u[j] << 16) & 0x7fffffffu, u[j] & 0x7fff0000u));
    }
    // (a row is a whole number of eight lanes)
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
    if ((lane & 7) == 0 && row < rows) atomicMax(&top_s[t], m);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PCS; ++k) {
    const int i = tid + k * WARPS * 32, row = i / PER, t = row / G;
    if (row >= ROWS) continue;
    uint32_t w[4] = {0, 0, 0, 0};
    const uint32_t top = row < rows ? top_s[t] : 0x7f800000u;
    if (top < 0x7f800000u) {  // (rows that are not finite choose as zeros)
      float s = __fdiv_rn(__uint_as_float(top), 127.f);
      if (s == 0.f) s = 1.f;
      const uint32_t u[4] = {piece[k].x, piece[k].y, piece[k].z, piece[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = fminf(fmaxf(rintf(__fdiv_rn(bf16_lo(u[j]), s)), -127.f), 127.f);
        const float y = fminf(fmaxf(rintf(__fdiv_rn(bf16_hi(u[j]), s)), -127.f), 127.f);
        const __half2 hh = __floats2half2_rn(x, y);
        w[j] = *reinterpret_cast<const uint32_t*>(&hh);
      }
    }
    uint2* dst = reinterpret_cast<uint2*>(smem + row * RS + (i % PER) * 16);
    dst[0] = make_uint2(w[0], w[1]);
    dst[1] = make_uint2(w[2], w[3]);
  }
  __syncthreads();
  float* prod = reinterpret_cast<float*>(smem + ROWS * RS) + warp * 16 * (ROWS + 1);
  for (; blk < blocks; blk += stride) {  // (warp-uniform)
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[nt][k] = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a[2][4];  // [hi, lo]: rows g and g + 8 (pages), channels 4 j and 4 j + 2 of the thread's 16
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint4 r0 = rec[0][s][c], r1 = rec[1][s][c];
          const uint32_t w0 = (j == 0 ? r0.x : j == 1 ? r0.y : j == 2 ? r0.z : r0.w) ^ 0x80808080u;
          const uint32_t w1 = (j == 0 ? r1.x : j == 1 ? r1.y : j == 2 ? r1.z : r1.w) ^ 0x80808080u;
          a[s][0] = sel_f16(w0, 0x4140);
          a[s][1] = sel_f16(w1, 0x4140);
          a[s][2] = sel_f16(w0, 0x4342);
          a[s][3] = sel_f16(w1, 0x4342);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = *reinterpret_cast<const uint2*>(smem + (nt * 8 + g) * RS + (64 * c + 16 * t4 + 4 * j) * 2);
          sel_mma(acc[nt], a[0][0], a[0][1], a[0][2], a[0][3], half2_max0(q.x), half2_max0(q.y));
          sel_mma(acc[nt], a[1][0], a[1][1], a[1][2], a[1][3], half2_min0(q.x), half2_min0(q.y));
        }
      }
    const float my_scale = scale;
    const bool my_there = there;
    const int base = blk * 16;
    if (blk + stride < blocks) load(blk + stride);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) prod[(g + 8 * (k >> 1)) * (ROWS + 1) + nt * 8 + 2 * t4 + (k & 1)] = acc[nt][k];
    __syncwarp();
    // a lane keeps its page: 16 pages, two tokens at once
    const int pg = lane & 15;
    const double s = (double)my_scale;
    if (base + pg < seen) {
      for (int t = lane >> 4; t < cols; t += 2) {
        const float* row = prod + pg * (ROWS + 1) + t * G;
        float m = row[0];
        for (int i = 1; i < G; ++i) m = fmaxf(m, row[i]);
        double v = (double)m * s;
        if (!my_there || !(fabs(v) < 1e300)) v = -1e300;  // no page, or bounds never made: last
        store(t, base + pg, ordered(v + 0.0));
      }
    }
    __syncwarp();
  }
}

// Two launches, for many query rows or pages: the scores through the workspace.
template <int D, int NT>
__global__ void __launch_bounds__(kSelThreads) page_score_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t top_s[NK_MAX_T];
  chain_wait();
  chain_release();
  const int b = blockIdx.y / p.Hkv, h = blockIdx.y % p.Hkv;
  const int t0 = blockIdx.z * p.cols, cols = min(p.cols, p.T - t0);
  const int L = select_len(p, b);
  if (L == 0) {
    if (threadIdx.x == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
    return;
  }
  const int seen = (L - p.T + t0 + cols - 1) / p.P + 1;  // pages that the chunk's last token sees
  if (seen <= p.k) return;                               // nothing to choose
  score_pages<D, NT, kSelWarps>(p, smem, top_s, b, h, t0, cols, seen, (int)(blockIdx.x * kSelWarps + (threadIdx.x >> 5)),
                     (int)gridDim.x * kSelWarps, [&](int t, int page, uint64_t key) {
                       p.scores[((int64_t)(b * p.T + t0 + t) * p.Hkv + h) * p.stride + page] = key;
                     });
}

// ---------------------------------------------------------------------------
// The choice: of each (token, kv-head) the k pages, by one block. The first
// `sinks` and the last `recent` pages that the token sees are always in; the
// others by score (nk_topk.cuh). get(i): key of page i; up to `room` of them are
// kept in shared memory, more are fetched anew in every pass. [klo, khi] holds all
// of them where klo <= khi.
// ---------------------------------------------------------------------------
constexpr int kPickKeep = 16384;  // keys kept in shared memory, at most

template <int NTH, class Get>
__device__ __forceinline__ void pick_pages(const SelectParams& p, int32_t* out, int seen, uint64_t* keep, int room,
                                           TopSmem<NTH>& sm, const Get& get, uint64_t klo = 1, uint64_t khi = 0) {
  const int tid = threadIdx.x;
  if (seen <= p.k) {
    for (int i = tid; i < p.k; i += NTH) out[i] = i < seen ? i : -1;
    return;
  }
  const int first = p.sinks, n = seen - p.sinks - p.recent, need = p.k - p.sinks - p.recent;  // need < n
  for (int i = tid; i < p.sinks + p.recent; i += NTH)
    out[i < p.sinks ? i : i + need] = i < p.sinks ? i : seen - p.recent + (i - p.sinks);
  if (need == 0) return;
  const bool kept = n <= room, ranged = kept && klo <= khi;
  if (ranged) {  // the first round's counts beside the fetching
    for (int i = tid; i < kTopBins; i += NTH) sm.hist[i] = 0;
    if (tid == 0) sm.count = 0;
    __syncthreads();
    const int shift = top_shift(klo, khi);
#pragma unroll 8
    for (int i = tid; i < n; i += NTH) {
      const uint64_t k = get(first + i);
      keep[i] = k;
      atomicAdd(&sm.hist[(int)((k - klo) >> shift)], 1u);
    }
    __syncthreads();
  } else if (kept) {
#pragma unroll 8
    for (int i = tid; i < n; i += NTH) keep[i] = get(first + i);
    __syncthreads();
  }
  const auto key = [&](int i) { return kept ? keep[i] : get(first + i); };
  uint64_t kt;
  int it;
  if (!ranged) block_range<NTH>(key, n, sm, klo, khi);
  block_threshold<NTH>(key, n, need, klo, khi, sm, kt, it, ranged);
  const int per = top_run<NTH>(n), a = tid * per, e = a + per < n ? a + per : n;
  const auto taken = [&](int i) {
    const uint64_t k = key(i);
    return k > kt || (k == kt && i <= it);
  };
  int mine = 0, total;
  for (int i = a; i < e; ++i) mine += taken(i);
  int at = first + block_exclusive<NTH>(mine, sm.warp, total);
  for (int i = a; i < e; ++i)
    if (taken(i)) out[at++] = first + i;
}

constexpr int kPickThreads = 512;

__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p, int room) {
  extern __shared__ uint64_t keep[];
  __shared__ TopSmem<kPickThreads> sm;
  chain_wait();
  chain_release();
  const int bt = blockIdx.x / p.Hkv, b = bt / p.T, t = bt - b * p.T;
  const int L = select_len(p, b);
  if (L == 0) return;  // (flagged by the first kernel; the list is left as it was)
  const uint64_t* src = p.scores + (int64_t)blockIdx.x * p.stride;
  pick_pages<kPickThreads>(p, p.out + (int64_t)blockIdx.x * p.k, (L - p.T + t) / p.P + 1, keep, room, sm,
                           [&](int i) { return __ldcg(src + i); });
}

// ---------------------------------------------------------------------------
// One launch: a cluster takes a (sequence, kv-head). Its CTAs share the blocks of
// 16 pages out in turn and keep their keys; then each takes a token, fetches its
// keys from all of them through distributed shared memory, and chooses. No
// workspace, no second launch: 14.2 us on the device for a choice among 4,096 pages
// of each of four kv-heads, where two launches took 12.3 and 20.5 a call against 15.8.
// ---------------------------------------------------------------------------
constexpr int kCluThreads = 512, kCluWarps = kCluThreads / 32;

// Key slots of a token in a CTA of a cluster of `cl`, for so many pages.
__host__ __device__ inline int cluster_slots(int64_t pages, int cl) {
  const int64_t blocks = (pages + 15) / 16, per = (int64_t)cl * kCluWarps;
  return (int)((blocks + per - 1) / per * kCluWarps * 16);
}

template <int D, int NT>
__global__ void __launch_bounds__(kCluThreads) page_select_kernel(const SelectParams p, int slots, int room) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t top_s[NK_MAX_T];
  __shared__ TopSmem<kCluThreads> sm;
  __shared__ uint32_t range[NK_MAX_T][2];  // least and largest upper half of this CTA's keys of a token
  cg::cluster_group cluster = cg::this_cluster();
  chain_wait();
  chain_release();
  const int rank = (int)cluster.block_rank(), cl = (int)cluster.num_blocks();
  const int b = blockIdx.y / p.Hkv, h = blockIdx.y % p.Hkv;
  const int L = select_len(p, b);
  if (L == 0) {  // (the same in all of the cluster)
    if (threadIdx.x == 0 && rank == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
    return;
  }
  uint64_t* own = reinterpret_cast<uint64_t*>(smem + select_smem(D, NT, kCluWarps));  // [T][slots]
  uint64_t* keep = own + (int64_t)p.T * slots;                             // [room]
  const int seen = (L - 1) / p.P + 1, turn = cl * kCluWarps;
  const bool choose = seen > p.k;
  if (choose) {
    if (threadIdx.x < p.T) {
      range[threadIdx.x][0] = 0xffffffffu;
      range[threadIdx.x][1] = 0;
    }
    // (score_pages has a barrier before its first store)
    score_pages<D, NT, kCluWarps>(p, smem, top_s, b, h, 0, p.T, seen, rank * kCluWarps + (int)(threadIdx.x >> 5), turn,
                                  [&](int t, int page, uint64_t key) {
                                    const int blk = page >> 4;
                                    own[t * slots + ((blk / turn) * kCluWarps + blk % kCluWarps) * 16 + (page & 15)] = key;
                                    atomicMin(&range[t][0], (uint32_t)(key >> 32));
                                    atomicMax(&range[t][1], (uint32_t)(key >> 32));
                                  });
    cluster.sync();
  }
  for (int t = rank; t < p.T; t += cl) {  // (block-uniform)
    uint32_t lo = 0xffffffffu, hi = 0;
    if (choose) {
      const uint32_t* of = cluster.map_shared_rank(&range[t][0], (threadIdx.x & 31) % cl);
      lo = __reduce_min_sync(0xffffffffu, of[0]);
      hi = __reduce_max_sync(0xffffffffu, of[1]);
    }
    pick_pages<kCluThreads>(p, p.out + ((int64_t)(b * p.T + t) * p.Hkv + h) * p.k, (L - p.T + t) / p.P + 1, keep, room, sm,
                            [&](int page) {
                              const int blk = page >> 4, w = blk % turn;
                              return *cluster.map_shared_rank(
                                  own + t * slots + ((blk / turn) * kCluWarps + w % kCluWarps) * 16 + (page & 15),
                                  w / kCluWarps);
                            },
                            (uint64_t)lo << 32, (uint64_t)hi << 32 | 0xffffffffu);
    __syncthreads();  // (keep and sm: the next token's)
  }
  if (choose) cluster.sync();  // nobody reads this CTA's keys any more
}

}  // namespace nk

using namespace nk;

namespace {

template <int D>
cudaError_t launch_bounds(const BoundsParams& p, int grid, cudaStream_t st) {
  constexpr int smem = kBndWarps * kBndStages * bounds_stage<D>();
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(page_bounds_kernel<D>), smem);
  if (e != cudaSuccess) return e;
  return launch_chained(page_bounds_kernel<D>, dim3((unsigned)grid), dim3(kBndThreads), (size_t)smem, st, p);
}

// How a call runs: in one launch where a cluster's CTA holds all rows, its keys
// and a token's keys; else in two (8 sequences of 16 tokens at 4K to 64K, 96 rows: 34.3
// us; one of 20,480 pages 58.2, where 16,384 in one launch take 30.0).
constexpr int kSelSmem = 200 * 1024;
int rows_tiles(int rows) {  // of the kernels' instances: 1, 2, 3, 4, 6, 8
  const int nt = (rows + 7) / 8;
  return nt == 5 ? 6 : (nt == 7 ? 8 : nt);
}
struct SelectPlan {
  int cl;         // CTAs of a cluster; 0: two launches
  int slots, room, smem;
  int NT;
};
// Sixteen, which is past the portable size, where the largest instance with all of
// its shared memory fits one of the device's groups of SMs sixteen times; else eight.
// Without a device sixteen (nothing can be launched then).
int largest_cluster() {
  static std::atomic<int> known[64];  // per device; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 16;
  }
  if (dev >= 0 && dev < 64) {
    const int n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  const auto kernel = page_select_kernel<256, 8>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  int clusters = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kCluThreads);
  cfg.dynamicSmemBytes = kSelSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool fits = set_smem_limit(fn, kSelSmem) == cudaSuccess &&
                    cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0;
  if (!fits) (void)cudaGetLastError();
  const int n = fits ? 16 : 8;
  if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}
SelectPlan plan_select(int64_t units, int T, int G, int D, int64_t pages) {
  SelectPlan s = {};
  if (T * G > kSelRows || pages > kPickKeep) return s;
  s.NT = rows_tiles(T * G);
  // as many CTAs for each unit, up to sixteen (eight where the device holds no cluster of
  // sixteen), as leave them all resident at once
  // (one an SM: 8 verified sequences with eight each took 15.2 us, 256 CTAs in two
  // rounds), no more than there are blocks of pages for
  const int sms = device_sms();
  s.cl = largest_cluster();
  while (s.cl > 1 && units * s.cl > (sms > 0 ? sms : 148)) s.cl /= 2;
  while (s.cl > 1 && (pages + 15) / 16 <= (int64_t)s.cl / 2 * kCluWarps) s.cl /= 2;
  s.slots = cluster_slots(pages, s.cl);
  s.room = (int)pages;
  const int64_t smem = select_smem(D, s.NT, kCluWarps) + ((int64_t)T * s.slots + s.room) * 8;
  if (smem > kSelSmem) return SelectPlan{};
  s.smem = (int)smem;
  return s;
}

template <int D, int NT>
cudaError_t launch_scores(const SelectParams& p, dim3 grid, const SelectPlan& plan, cudaStream_t st) {
  if (plan.cl > 0) {
    const void* fn = reinterpret_cast<const void*>(page_select_kernel<D, NT>);
    cudaError_t e = set_smem_limit(fn, kSelSmem);  // (once, however the contexts grow)
    if (e != cudaSuccess) return e;
    if (plan.cl > 8) {
      static std::atomic<bool> allowed[64];  // per device
      int dev = 0;
      e = cudaGetDevice(&dev);
      if (e != cudaSuccess) return e;
      if (dev < 0 || dev >= 64 || !allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) allowed[dev].store(true, std::memory_order_relaxed);
      }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.cl, (unsigned)(p.B * p.Hkv));
    cfg.blockDim = dim3(kCluThreads);
    cfg.dynamicSmemBytes = (size_t)plan.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)plan.cl;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, page_select_kernel<D, NT>, p, plan.slots, plan.room);
  }
  const int smem = select_smem(D, NT, kSelWarps);
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(page_score_kernel<D, NT>), smem);
  if (e != cudaSuccess) return e;
  return launch_chained(page_score_kernel<D, NT>, grid, dim3(kSelThreads), (size_t)smem, st, p);
}

template <int D>
cudaError_t launch_scores_d(const SelectParams& p, int NT, dim3 grid, const SelectPlan& plan, cudaStream_t st) {
  switch (NT) {
    case 1: return launch_scores<D, 1>(p, grid, plan, st);
    case 2: return launch_scores<D, 2>(p, grid, plan, st);
    case 3: return launch_scores<D, 3>(p, grid, plan, st);
    case 4: return launch_scores<D, 4>(p, grid, plan, st);
    case 6: return launch_scores<D, 6>(p, grid, plan, st);
    default: return launch_scores<D, 8>(p, grid, plan, st);
  }
}

}  // namespace

extern "C" {

size_t nk_page_bounds_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t head_dim) {
  if (num_pages < 1 || num_kv_heads < 1 || !(head_dim == 64 || head_dim == 128 || head_dim == 256)) return 0;
  return (size_t)num_pages * num_kv_heads * (2 * (size_t)head_dim + 4);
}

int nk_page_bounds(const nk_kv_pool* pool, void* bounds_dev, const int32_t* block_table_dev, int32_t max_pages_per_seq,
                   const int32_t* start_pos_dev, const int32_t* cu_new_dev, int32_t B, int32_t* status_dev,
                   void* stream) {
  const int err = check_pool(pool);
  if (err != NK_OK) return err;
  if (B < 0 || max_pages_per_seq < 1) return NK_ERR_SHAPE;
  if (B > kMaxBatch) return NK_ERR_UNSUPPORTED;
  if (B == 0) return NK_OK;
  if (!bounds_dev || !block_table_dev || !start_pos_dev || !cu_new_dev) return NK_ERR_NULL;
  if (!aligned_to(bounds_dev, 16)) return NK_ERR_SHAPE;
  const int P = pool->page_size, D = pool->head_dim;
  const WaitLimits limits = wait_limits();
  const BoundsParams p{reinterpret_cast<const uint8_t*>(pool->base_dev), ChunkLayout::make(P, D), pool->num_pages, P,
                       pool->num_kv_heads, block_table_dev, max_pages_per_seq, start_pos_dev, cu_new_dev, B,
                       bounds_view(bounds_dev, pool->num_pages, pool->num_kv_heads, D), status_dev, limits.cycles,
                       limits.withhold};
  const int sms = device_sms();
  int64_t grid = (int64_t)B * max_pages_per_seq * pool->num_kv_heads;
  const int64_t most = sms > 0 ? sms : 148;
  if (grid > most) grid = most;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 256   ? launch_bounds<256>(p, (int)grid, st)
                        : D == 128 ? launch_bounds<128>(p, (int)grid, st)
                                   : launch_bounds<64>(p, (int)grid, st);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

int nk_page_bounds_values(const void* bounds_dev, int32_t num_pages, int32_t num_kv_heads, int32_t head_dim,
                          float* values_dev, void* stream) {
  if (num_pages < 1 || num_kv_heads < 1 || !(head_dim == 64 || head_dim == 128 || head_dim == 256)) return NK_ERR_SHAPE;
  if (!bounds_dev || !values_dev) return NK_ERR_NULL;
  if (!aligned_to(bounds_dev, 16) || !aligned_to(values_dev, 16)) return NK_ERR_SHAPE;
  const int per_rec = 2 * head_dim / 16;
  const int64_t pieces = (int64_t)num_pages * num_kv_heads * per_rec, blocks = (pieces + 255) / 256;
  const int sms = device_sms();
  const int64_t most = (int64_t)(sms > 0 ? sms : 148) * 8;
  const cudaError_t e = launch_chained(bounds_values_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0,
                                       reinterpret_cast<cudaStream_t>(stream),
                                       bounds_view(const_cast<void*>(bounds_dev), num_pages, num_kv_heads, head_dim), pieces,
                                       per_rec, values_dev);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

size_t nk_page_select_workspace_bytes(int32_t B, int32_t T, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t head_dim, int32_t page_size, int32_t max_ctx) {
  if (B < 1 || T < 1 || T > NK_MAX_T || num_kv_heads < 1 || num_q_heads < num_kv_heads || page_size < 1 || max_ctx < 1)
    return 0;
  const int64_t pages = ((int64_t)max_ctx + page_size - 1) / page_size;
  if (plan_select((int64_t)B * num_kv_heads, T, num_q_heads / num_kv_heads, head_dim, pages).cl > 0) return 0;
  return (size_t)B * T * num_kv_heads * pages * 8;
}

int nk_page_select(const void* bounds_dev, int32_t num_pages, int32_t page_size, int32_t num_kv_heads, int32_t head_dim,
                   const void* q_dev, const int32_t* block_table_dev, int32_t max_pages_per_seq,
                   const int32_t* ctx_lens_dev, int32_t B, int32_t T, int32_t num_q_heads, int32_t max_ctx, int32_t k,
                   int32_t sink_pages, int32_t recent_pages, void* workspace_dev, size_t workspace_bytes,
                   int32_t* pages_dev, int32_t* status_dev, void* stream) {
  if (num_pages < 1 || page_size < 1 || num_kv_heads < 1 || B < 0 || T < 1 || T > NK_MAX_T || num_q_heads < 1 ||
      num_q_heads % num_kv_heads != 0 || !(head_dim == 64 || head_dim == 128 || head_dim == 256))
    return NK_ERR_SHAPE;
  if (k < 1 || sink_pages < 0 || recent_pages < 1 || (int64_t)sink_pages + recent_pages > k) return NK_ERR_SHAPE;
  if (B == 0) return NK_OK;
  if (!bounds_dev || !q_dev || !block_table_dev || !ctx_lens_dev || !pages_dev) return NK_ERR_NULL;
  const int G = num_q_heads / num_kv_heads;
  if (G > 48 || (int64_t)B * num_kv_heads > 65535) return NK_ERR_UNSUPPORTED;
  if (max_pages_per_seq < 1 || max_ctx < T || (int64_t)max_ctx > (int64_t)max_pages_per_seq * page_size)
    return NK_ERR_SHAPE;
  if (!aligned_to(bounds_dev, 16) || !aligned_to(q_dev, 16)) return NK_ERR_SHAPE;
  const int64_t units = (int64_t)B * num_kv_heads, pages = ((int64_t)max_ctx + page_size - 1) / page_size;
  const SelectPlan plan = plan_select(units, T, G, head_dim, pages);
  const size_t need = plan.cl > 0 ? 0 : (size_t)units * T * pages * 8;
  if (need > 0 && (!workspace_dev || workspace_bytes < need || !aligned_to(workspace_dev, 16))) return NK_ERR_WORKSPACE;
  SelectParams p = {};
  p.bounds = bounds_view(const_cast<void*>(bounds_dev), num_pages, num_kv_heads, head_dim);
  p.num_pages = num_pages;
  p.Hkv = num_kv_heads;
  p.G = G;
  p.q = reinterpret_cast<const uint16_t*>(q_dev);
  p.bt = block_table_dev;
  p.max_pages = max_pages_per_seq;
  p.ctx = ctx_lens_dev;
  p.B = B;
  p.T = T;
  p.P = page_size;
  p.max_ctx = max_ctx;
  p.k = k;
  p.sinks = sink_pages;
  p.recent = recent_pages;
  p.scores = reinterpret_cast<uint64_t*>(workspace_dev);
  p.stride = pages;
  p.out = pages_dev;
  p.status = status_dev;
  p.cols = kSelRows / G < 1 ? 1 : kSelRows / G;
  if (p.cols > T) p.cols = T;
  const int sms = device_sms();
  // eight warps of 16 pages a block; past four blocks an SM they take turns
  int64_t gx = (pages + 16 * kSelWarps - 1) / (16 * kSelWarps), most = (int64_t)(sms > 0 ? sms : 148) * 4 / units;
  if (most < 1) most = 1;
  if (gx > most) gx = most;
  const dim3 grid((unsigned)gx, (unsigned)units, (unsigned)((T + p.cols - 1) / p.cols));
  const int NT = rows_tiles(p.cols * G);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = head_dim == 256   ? launch_scores_d<256>(p, NT, grid, plan, st)
                  : head_dim == 128 ? launch_scores_d<128>(p, NT, grid, plan, st)
                                    : launch_scores_d<64>(p, NT, grid, plan, st);
  if (e == cudaSuccess && plan.cl > 0) return NK_OK;
  if (e != cudaSuccess) return NK_ERR_CUDA;
  const int room = (int)(pages < kPickKeep ? pages : kPickKeep);
  e = set_smem_limit(reinterpret_cast<const void*>(page_pick_kernel), kPickKeep * 8);
  if (e != cudaSuccess) return NK_ERR_CUDA;
  e = launch_chained(page_pick_kernel, dim3((unsigned)(units * T)), dim3(kPickThreads), (size_t)room * 8, st, p, room);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

}  // extern "C"
