// nk_step.cu -- what a serving step computes before its append and attention:
// the block tables and slot maps of the batch (nk_step_tables), and the rotary
// positions of its query and key rows (nk_mrope).
#include <math.h>

#include "nk_common.cuh"

namespace nk {

// ---------------------------------------------------------------------------
// nk_step_tables. Sequence b holds start[b] tokens in ceil(start / P) pages and
// brings new[b]. Its pages [ceil(start / P), ceil((start + new) / P)) are taken
// from the free list in order, sequence after sequence: with `off` the
// exclusive prefix of the counts, page i of them is free[off[b] + i].
//
// One launch, no workspace, no communication between blocks: every block
// reads the B lengths and forms both prefixes itself (two numbers a sequence;
// B <= 1,024), then takes its share of the fresh pages and of the rows. A row
// in a fresh page finds its page in the free list, not in the table another
// block may be writing, so nothing a block reads is written in the launch.
// Bounded by latency: one launch, the lengths' load, the block scan, one
// dependent load per row and its stores. Measured in a replayed graph: 4.0 us
// for 8 sequences of one token, 7.4 us for 1,024 ragged ones (147K rows).
// ---------------------------------------------------------------------------
struct TablesParams {
  const int32_t* start;
  const int32_t* fresh;  // new tokens of each sequence
  int B, P, num_pages;
  const int32_t* free_pages;
  int num_free;
  int32_t* table;
  int max_pages;
  int32_t* cu;
  int32_t* ctx;
  int64_t* slots;
  int32_t* pos;  // may be NULL
  int max_rows;
  int32_t* used;  // may be NULL
  int32_t* status;
};

constexpr int kTabThreads = 256;
constexpr int kTabPer = kMaxBatch / kTabThreads;  // sequences per thread
constexpr int kTabRows = 4;                       // rows (and pages) per thread and round

struct TabSeq {
  int start, pages_held;  // start: -1 for a sequence whose lengths are refused
};

__global__ void __launch_bounds__(kTabThreads) step_tables_kernel(const TablesParams p) {
  __shared__ int cu_s[kMaxBatch + 1];   // rows before sequence b
  __shared__ int off_s[kMaxBatch + 1];  // fresh pages before sequence b
  __shared__ TabSeq seq[kMaxBatch];
  __shared__ int64_t wrow[kTabThreads / 32], wpage[kTabThreads / 32];
  chain_wait();
  chain_release();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const bool lead = blockIdx.x == 0;
  int64_t rows[kTabPer], rsum = 0;
  int64_t need[kTabPer], psum = 0;
#pragma unroll
  for (int i = 0; i < kTabPer; ++i) {
    const int b = tid * kTabPer + i;
    rows[i] = 0;
    need[i] = 0;
    if (b < p.B) {
      const int s = p.start[b], n = p.fresh[b];
      const int64_t end = (int64_t)s + n;
      const bool ok = s >= 0 && n >= 0 && end <= (int64_t)p.max_pages * p.P && end <= 0x7fffffff;
      rows[i] = n > 0 ? n : 0;
      const int held = ok ? (int)(((int64_t)s + p.P - 1) / p.P) : 0;
      need[i] = ok ? (end + p.P - 1) / p.P - held : 0;
      seq[b] = TabSeq{ok ? s : -1, held};
      if (lead) {
        p.ctx[b] = ok ? (int)end : 0;
        if (!ok) flag(p.status, NK_DEVFLAG_BAD_POS);
      }
      rsum += rows[i];
      psum += need[i];
    }
  }
  // exclusive prefixes of both counts over the block
  int64_t rinc = rsum, pinc = psum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r = __shfl_up_sync(0xffffffffu, rinc, o);
    const int64_t q = __shfl_up_sync(0xffffffffu, pinc, o);
    if (lane >= o) {
      rinc += r;
      pinc += q;
    }
  }
  if (lane == 31) {
    wrow[wid] = rinc;
    wpage[wid] = pinc;
  }
  __syncthreads();
  int64_t rrun = rinc - rsum, prun = pinc - psum;
  for (int w = 0; w < wid; ++w) {
    rrun += wrow[w];
    prun += wpage[w];
  }
  auto sat = [](int64_t v) { return v > 0x7fffffff ? 0x7fffffff : (int)v; };
#pragma unroll
  for (int i = 0; i < kTabPer; ++i) {
    const int b = tid * kTabPer + i;
    if (b < p.B) {
      cu_s[b] = sat(rrun);
      off_s[b] = sat(prun);
      if (lead) p.cu[b] = sat(rrun);
    }
    rrun += rows[i];
    prun += need[i];
  }
  if (tid == kTabThreads - 1) {
    cu_s[p.B] = sat(rrun);
    off_s[p.B] = sat(prun);
    if (lead) {
      p.cu[p.B] = sat(rrun);
      if (p.used) *p.used = sat(prun);
      if (rrun > p.max_rows || rrun >= 0x7fffffff) flag(p.status, NK_DEVFLAG_BAD_POS);
      if (prun > p.num_free) flag(p.status, NK_DEVFLAG_NO_PAGES);
    }
  }
  __syncthreads();
  // 2^31 - 1 rows or more (flagged above) have no numbering: nothing is assigned
  if (cu_s[p.B] == 0x7fffffff) return;
  const int total = cu_s[p.B] < p.max_rows ? cu_s[p.B] : p.max_rows, pages = off_s[p.B];
  // the sequence b that holds item x of a prefix: pre[b] <= x < pre[b + 1]
  auto find = [&](const int* pre, int x) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  auto fresh_page = [&](int k) {  // free list entry k: -1 past its end or outside the pool
    if (k >= p.num_free) return -1;
    const int page = __ldg(p.free_pages + k);
    return page < 0 || page >= p.num_pages ? -2 : page;
  };
  const int64_t stride = (int64_t)gridDim.x * kTabThreads, first = (int64_t)blockIdx.x * kTabThreads + tid;
  for (int64_t x = first; x < pages; x += stride) {
    const int k = (int)x, b = find(off_s, k);
    const int page = fresh_page(k);
    if (page == -2) flag(p.status, NK_DEVFLAG_BAD_PAGE);
    p.table[(int64_t)b * p.max_pages + seq[b].pages_held + (k - off_s[b])] = page < 0 ? -1 : page;
  }
  for (int64_t x = first; x < total; x += stride) {
    const int j = (int)x, b = find(cu_s, j);
    const TabSeq q = seq[b];
    int64_t slot = -1;
    int pos = -1;
    if (q.start >= 0) {
      pos = q.start + (j - cu_s[b]);
      const int pi = pos / p.P;
      int page;
      if (pi >= q.pages_held) {
        page = fresh_page(off_s[b] + (pi - q.pages_held));
      } else {
        page = __ldg(p.table + (int64_t)b * p.max_pages + pi);
        if (page < 0 || page >= p.num_pages) {
          flag(p.status, NK_DEVFLAG_BAD_PAGE);
          page = -1;
        }
      }
      if (page >= 0) slot = (int64_t)page * p.P + (pos - pi * p.P);
    }
    p.slots[j] = slot;
    if (p.pos) p.pos[j] = pos;
  }
}

// ---------------------------------------------------------------------------
// nk_mrope. Head channels i and i + half (half = rot / 2) of a row turn by
// angle = position[axis(i)] * inv_freq[i]:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// computed in fp32 and rounded once to bf16; the channels past rot are copied.
//
// The angle of a far position does not survive an fp32 product (2^18 radians
// leave 2^-6 of them). The frequency therefore comes as turns per position in
// 64-bit fixed point (a fraction of 2^64, made on the host from the caller's
// doubles); position times fraction, modulo 2^64, is the exact fraction of a
// turn, whose top 32 bits, signed, go to sincospi. The product loses nothing
// at any int32 position; the fraction itself is off by the rounding of its
// double, at most 2^-54 turns, so 2^-23 turns at position 2^31.
//
// Bandwidth-bound: each row is read and written once, in 16-byte pieces. A
// block takes `per` rows and forms their half cos/sin pairs once in shared
// memory (all heads share them). A thread keeps one piece of the head (eight
// channel pairs, or eight copied channels) and goes over (row, head) from its
// first head on: no division in the loop (with one per item, 8,192 rows of 24
// + 4 heads of 256 took 43.1 us against 39.1: 6.0 TB/s, 0.89 of a copy's rate;
// 4,099 rows of 16 + 2 heads of 128, half of each turned, 11.4 against 7.3).
// Many blocks in flight cover the loads' latency; two or four items of a
// thread in flight, held in registers, were slower (60 and 87 us).
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxHalf = NK_MAX_HEAD_DIM / 2;
constexpr int kRopeMaxRows = 8;  // rows of a block, at most
constexpr int kRopeItems = 2;    // items of a thread, about (4: the same, 8: 42, 16: 50 us on the 8,192 rows)

struct RopeParams {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* qo;
  uint16_t* ko;
  int64_t q_stride, k_stride, qo_stride, ko_stride;  // elements between rows
  const int32_t* pos;  // [axes][pos_stride]
  int64_t pos_stride;
  const int32_t* num_rows;  // may be NULL
  int rows, Hq, Hkv, D, half;
  int per;  // rows of a block
  uint32_t axis[kRopeMaxHalf / 16];  // two bits a frequency
  uint64_t turns[kRopeMaxHalf];
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kRopeThreads) mrope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float cs[kRopeMaxRows][kRopeMaxHalf], sn[kRopeMaxRows][kRopeMaxHalf];
  chain_wait();
  chain_release();
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * p.per;
  int limit = p.rows;
  if (p.num_rows) limit = min(limit, __ldg(p.num_rows));
  const int n = min(p.per, limit - row0);  // rows behind the last one stay as they are
  if (n <= 0) return;
  for (int i = tid; i < n * p.half; i += kRopeThreads) {
    const int r = i / p.half, f = i - r * p.half;
    const int ax = (int)(p.axis[f >> 4] >> ((f & 15) * 2)) & 3;
    const int64_t pos = __ldg(p.pos + ax * p.pos_stride + row0 + r);
    const uint64_t turn = (uint64_t)pos * p.turns[f];
    const float t = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2 * fraction of a turn, in [-1, 1)
    sincospif(t, &sn[r][f], &cs[r][f]);
  }
  __syncthreads();
  const int heads = p.Hq + p.Hkv;
  const int pieces = p.half / 8;               // pairs of pieces that turn
  const int tail = (p.D - 2 * p.half) / 8;     // pieces that are copied
  const int per_head = pieces + tail;          // threads of a head
  const int lanes = kRopeThreads / per_head;   // heads at once
  const int c = tid % per_head, h0 = tid / per_head;
  if (h0 >= lanes) return;
  const bool turns = c < pieces;
  const int off_a = turns ? c * 8 : 2 * p.half + (c - pieces) * 8, off_b = turns ? p.half + c * 8 : off_a;
  if (h0 >= heads) return;
  int r = 0, h = h0;
  while (r < n) {
    const int row = r;
    const int64_t j = row0 + row;
    const bool isq = h < p.Hq;
    const int head = (isq ? h : h - p.Hq) * p.D;
    const uint16_t* src = (isq ? p.q + j * p.q_stride : p.k + j * p.k_stride) + head;
    uint16_t* dst = (isq ? p.qo + j * p.qo_stride : p.ko + j * p.ko_stride) + head;
    const uint4 a4 = *reinterpret_cast<const uint4*>(src + off_a);
    const uint4 b4 = *reinterpret_cast<const uint4*>(src + off_b);
    h += lanes;  // one loop over (row, head): as two loops it took 44.7 us on the 8,192 rows
    if (h >= heads) {
      h = h0;
      ++r;
    }
    if (turns) {
      const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
      uint32_t x[4], y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 co = *reinterpret_cast<const float2*>(&cs[row][c * 8 + 2 * k]);
        const float2 si = *reinterpret_cast<const float2*>(&sn[row][c * 8 + 2 * k]);
        const float a0 = bf16_lo(a[k]), a1 = bf16_hi(a[k]), b0 = bf16_lo(b[k]), b1 = bf16_hi(b[k]);
        x[k] = pack_bf16(a0 * co.x - b0 * si.x, a1 * co.y - b1 * si.y);
        y[k] = pack_bf16(b0 * co.x + a0 * si.x, b1 * co.y + a1 * si.y);
      }
      *reinterpret_cast<uint4*>(dst + off_a) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(dst + off_b) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {
      *reinterpret_cast<uint4*>(dst + off_a) = a4;
    }
  }
}

}  // namespace nk

using namespace nk;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

extern "C" {

int nk_step_tables(int32_t page_size, int32_t num_pages, const int32_t* start_pos_dev, const int32_t* new_lens_dev,
                   int32_t B, const int32_t* free_pages_dev, int32_t num_free, int32_t* block_table_dev,
                   int32_t max_pages_per_seq, int32_t* cu_new_dev, int32_t* ctx_lens_dev, int64_t* slot_map_dev,
                   int32_t* positions_dev, int32_t max_rows, int32_t* used_pages_dev, int32_t* status_dev,
                   void* stream) {
  if (page_size < 1 || num_pages < 1 || B < 0 || num_free < 0 || max_pages_per_seq < 1 || max_rows < 0)
    return NK_ERR_SHAPE;
  if (B > kMaxBatch) return NK_ERR_UNSUPPORTED;
  // (a step of no sequences still tells that it has no rows and takes no page)
  if (!cu_new_dev || (B > 0 && (!start_pos_dev || !new_lens_dev || !block_table_dev || !ctx_lens_dev ||
                                (num_free > 0 && !free_pages_dev) || (max_rows > 0 && !slot_map_dev))))
    return NK_ERR_NULL;
  // every block reads the lengths while others write the results
  if (B > 0 && (ctx_lens_dev == start_pos_dev || ctx_lens_dev == new_lens_dev)) return NK_ERR_SHAPE;
  TablesParams p{start_pos_dev, new_lens_dev, B, page_size, num_pages, free_pages_dev, num_free, block_table_dev,
                 max_pages_per_seq, cu_new_dev, ctx_lens_dev, slot_map_dev, positions_dev, max_rows, used_pages_dev,
                 status_dev};
  // every fresh page holds a new row, so the rows bound the pages too (a
  // batch past max_rows still gets its pages, by the strided loops)
  const int64_t per_block = kTabThreads * kTabRows;
  int64_t grid = ((int64_t)max_rows + per_block - 1) / per_block;
  if (grid < 1) grid = 1;
  if (grid > 304) grid = 304;
  const cudaError_t e = launch_chained(step_tables_kernel, dim3((unsigned)grid), dim3(kTabThreads), 0,
                                       reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

int nk_mrope(const void* q_dev, const void* k_dev, void* q_out_dev, void* k_out_dev, int64_t q_row_stride,
             int64_t k_row_stride, int64_t q_out_row_stride, int64_t k_out_row_stride, int32_t rows,
             int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, const int32_t* positions_dev,
             int64_t positions_stride, const double* inv_freq_host, const int32_t* sections_host, int32_t num_axes,
             int32_t interleaved, const int32_t* num_rows_dev, void* stream) {
  if (rows < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + (int64_t)num_kv_heads < 1 ||
      num_q_heads + (int64_t)num_kv_heads > 65535 || head_dim < 16 || head_dim > NK_MAX_HEAD_DIM || head_dim % 8 != 0 ||
      num_axes < 1 || num_axes > 4)
    return NK_ERR_SHAPE;
  if (!inv_freq_host || !sections_host) return NK_ERR_NULL;
  int64_t half64 = 0;
  for (int a = 0; a < num_axes; ++a) {
    if (sections_host[a] < 0) return NK_ERR_SHAPE;
    half64 += sections_host[a];
  }
  if (half64 < 8 || half64 % 8 != 0 || 2 * half64 > head_dim) return NK_ERR_SHAPE;
  const int half = (int)half64;
  RopeParams p = {};
  for (int i = 0; i < half; ++i) {
    if (!isfinite(inv_freq_host[i])) return NK_ERR_SHAPE;
    // turns per position, modulo 1, as a fraction of 2^64
    double t = inv_freq_host[i] * 0.15915494309189535;  // 1 / (2 pi)
    t -= floor(t);
    const double hi = floor(t * 4294967296.0), lo = (t * 4294967296.0 - hi) * 4294967296.0;
    p.turns[i] = ((uint64_t)hi << 32) + (uint64_t)lo;
    int ax = 0;
    if (interleaved) {
      // the axes in turn, each until its section is used up; then axis 0
      ax = i % num_axes;
      if (i >= (int64_t)num_axes * sections_host[ax]) ax = 0;
    } else {
      for (int left = i; left >= sections_host[ax]; ++ax) left -= sections_host[ax];
    }
    p.axis[i >> 4] |= (uint32_t)ax << ((i & 15) * 2);
  }
  if (rows == 0) return NK_OK;
  if (!positions_dev || (num_q_heads > 0 && (!q_dev || !q_out_dev)) || (num_kv_heads > 0 && (!k_dev || !k_out_dev)))
    return NK_ERR_NULL;
  const int64_t strides[4] = {q_row_stride, q_out_row_stride, k_row_stride, k_out_row_stride};
  for (int i = 0; i < 4; ++i) {
    const int heads = i < 2 ? num_q_heads : num_kv_heads;
    if (heads > 0 && (strides[i] % 8 != 0 || strides[i] < (int64_t)heads * head_dim)) return NK_ERR_SHAPE;
  }
  if (positions_stride < rows && num_axes > 1) return NK_ERR_SHAPE;
  if (!aligned16(q_dev) || !aligned16(k_dev) || !aligned16(q_out_dev) || !aligned16(k_out_dev)) return NK_ERR_SHAPE;
  if ((q_dev == q_out_dev && q_row_stride != q_out_row_stride && num_q_heads > 0) ||
      (k_dev == k_out_dev && k_row_stride != k_out_row_stride && num_kv_heads > 0))
    return NK_ERR_SHAPE;
  p.q = reinterpret_cast<const uint16_t*>(q_dev);
  p.k = reinterpret_cast<const uint16_t*>(k_dev);
  p.qo = reinterpret_cast<uint16_t*>(q_out_dev);
  p.ko = reinterpret_cast<uint16_t*>(k_out_dev);
  p.q_stride = q_row_stride;
  p.k_stride = k_row_stride;
  p.qo_stride = q_out_row_stride;
  p.ko_stride = k_out_row_stride;
  p.pos = positions_dev;
  p.pos_stride = positions_stride;
  p.num_rows = num_rows_dev;
  p.rows = rows;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  p.half = half;
  // rows of a block, while every SM still gets two blocks
  const int64_t per_row = (int64_t)(num_q_heads + num_kv_heads) * (head_dim / 8 - half / 8);
  int64_t per = (kRopeItems * kRopeThreads + per_row - 1) / per_row;
  if (per > kRopeMaxRows) per = kRopeMaxRows;
  while (per > 1 && (rows + per - 1) / per < 304) --per;
  p.per = (int)per;
  const cudaError_t e = launch_chained(mrope_kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(kRopeThreads), 0,
                                       reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

}  // extern "C"
