// nk_chunk.cu -- attention of ragged chunks of new tokens over the paged INT8
// group-64 cache (nk_paged_chunk_attn): sequence b brings cu_q[b+1] - cu_q[b]
// query tokens (one for a decoding sequence, thousands for a prompt), each
// seeing the keys up to its own position, or a sliding window of them and the
// first tokens (sinks).
//
//   S = Q K^T,  P = exp2(S - m),  l = sum P,  O = P V / l
// with both products on the 5th-generation tensor cores (tcgen05.mma, fp16
// operands, fp32 accumulators in tensor memory). A CTA works on tiles of 128
// query rows of one (sequence, kv-head), rows numbered token-major (row r =
// token r / G, q-head r % G), against blocks of 64 keys. Each row is one
// tensor-memory lane and one softmax thread, so the softmax needs no exchange.
//
// Operands: Q (bf16, scaled per row by a power of two into the fp16 range) and
// P are A operands in tensor memory; K and V are B operands in shared memory,
// dequantized to fp16: code * fp16(scale * 2^-e), two roundings of at most
// 2^-11 relative each where the output's bf16 rounding is 2^-8 (a row whose
// scale is below 2^-8 of its block's largest keeps fewer bits, never fewer
// than 2^-25 of that largest). The exponent e keeps the products inside the
// fp16 range for any pool: one per block for K (undone on the scores), one per
// 64-channel group for V, moved only when a block's scales leave its window
// (the accumulator is then rescaled).
//
// 16 warps in four warpgroups, one CTA per SM:
//   warps 0-3   softmax: S from tensor memory, masks, running maximum with a
//               lazy reference (moved only when a score passes it by more than
//               8, so the accumulator is rarely rescaled), P back to tensor
//               memory over S, row sums, and the tile's output;
//   warps 4-7   K blocks, warps 8-11 V blocks: codes and scales from the ring,
//               widened to fp16, scaled, stored to one of two
//               128-byte-swizzled operand buffers;
//   warp 12     issues the MMAs: QK of block j + 1 goes out before PV of block
//               j, so the tensor cores work while the softmax does;
//   warp 13     looks up the pages and fills a two-stage ring of raw blocks
//               with bulk asynchronous copies (14 and 15 are idle).
//
// Loading the codes straight into the convert warps' registers, one block
// ahead, spared the ring's shared-memory traffic but left the page lookup and
// the loads' latency in their path: 7,345 us against 4,720 on eight chunks of
// 1,024 tokens at 8K to 32K (24 q-heads over 4 kv-heads, head dim 256).
//
// Work split (stream-K): the blocks of all tiles form one list, cut into equal
// contiguous ranges, one per CTA, whatever the sequences' lengths. A tile cut
// by a range's end leaves fp32 partials with their log-sum-exp in the
// workspace; a second kernel joins them. Every mbarrier wait is bounded.
#include <math.h>

#include "nk_chunk.cuh"
#include "nk_decode_mma.cuh"

namespace nk {
namespace chunk {

using mma::ex2;
using mma::exp_of;
using mma::kEvUnset;
using mma::kSmemLimit;
using mma::named_bar;
using mma::pack_f16;
using mma::pow2i;
using mma::q_norm_exp;

constexpr int kKeys = 64;   // keys of a block
constexpr int kSoftWarps = 4, kConvWarps = 4;  // convert warps per operand
constexpr int kMmaWarp = kSoftWarps + 2 * kConvWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;  // whole warpgroups, for setmaxnreg
// Registers per thread: launched with 128 (512 threads, the whole file); the
// shares below add up to 4 * 128, so no increase waits for registers that are
// not there (checked on the host against the compiled count).
constexpr int kLaunchRegs = 128, kRegsSoft = 184, kRegsConv = 128, kRegsMma = 72;
// setmaxnreg.inc must not lower a count, .dec must not raise one (an illegal instruction otherwise).
template <int N>
__device__ __forceinline__ void set_regs() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "setmaxnreg takes multiples of 8");
  if constexpr (N > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N) : "memory");
  if constexpr (N < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N) : "memory");
}
static_assert(kRegsSoft + 2 * kRegsConv + kRegsMma == 4 * kLaunchRegs, "shares = the launch's registers");
constexpr int kTmemCols = 512;
constexpr int kStages = 2;  // raw blocks in flight (a third does not fit at head dim 256)
constexpr int kMinBlocks = 4;  // blocks a CTA takes at least (fewer CTAs work on a small batch)

template <int D>
struct Smem {
  static constexpr int kTile = kKeys * D * 2;  // one fp16 K or V block
  static constexpr int off_k = 0;              // [2]
  static constexpr int off_v = 2 * kTile;      // [2]
  static constexpr int kStage = kKeys * (2 * D + 2 * (D / 64) * 4);  // raw block: K codes | K scales | V codes | V scales
  static constexpr int off_ring = 4 * kTile;                         // [kStages]
  static constexpr int off_tab = off_ring + kStages * kStage;        // [8 convert warps][16 keys][D / 64] scales
  static constexpr int off_pre = off_tab + 8 * 16 * (D / 64) * 8;    // int64 [kMaxBatch + 1]: blocks before sequence b
  static constexpr int off_lens = off_pre + (kMaxBatch + 2) * 8;  // int [kMaxBatch]
  static constexpr int off_cu = off_lens + kMaxBatch * 4;         // int [kMaxBatch + 1]
  static constexpr int off_misc = off_cu + (kMaxBatch + 4) * 4;
  static constexpr int total = off_misc + 1024 + 1024;  // slack to align the base
};

// The blocks of a tile: `lead` sink blocks, then the blocks from `first` on.
struct TileSpan {
  int r1;            // one past its last row
  int p0, p1;        // positions of its first and last token
  int lead, first;
  int blocks;
};

__device__ __forceinline__ TileSpan span_of(const Params& p, int L, int T, int tile) {
  TileSpan s;
  const int r0 = tile * kRows, mr = T * p.G;
  s.r1 = r0 + kRows < mr ? r0 + kRows : mr;
  s.p0 = L - T + r0 / p.G;
  s.p1 = L - T + (s.r1 - 1) / p.G;
  s.first = 0;
  s.lead = 0;
  if (p.window > 0) {
    const int lo = s.p0 - p.window + 1;
    s.first = lo > 0 ? lo / kKeys : 0;
    const int sb = (int)(((int64_t)p.sinks + kKeys - 1) / kKeys);
    s.lead = sb < s.first ? sb : s.first;
  }
  s.blocks = s.p1 / kKeys + 1 - s.first + s.lead;
  return s;
}

// Position in the list of blocks.
struct Walk {
  int64_t x, end;    // next block of the CTA, one past its last
  int b, h, tile, v; // unit, tile and block number within the tile of x
  int L, T;
  TileSpan s;
};

__device__ __forceinline__ int tiles_of(const Params& p, int T) { return (int)(((int64_t)T * p.G + kRows - 1) / kRows); }

struct Tables {
  const int64_t* pre;
  const int* lens;
  const int* cu;
};

__device__ __forceinline__ void enter_tile(const Params& p, Walk& w) { w.s = span_of(p, w.L, w.T, w.tile); }

// The tile after w's (the caller knows there is one).
__device__ __forceinline__ void next_tile(const Params& p, const Tables& t, Walk& w) {
  w.v = 0;
  if (++w.tile == tiles_of(p, w.T)) {
    w.tile = 0;
    if (++w.h == p.Hkv) {
      w.h = 0;
      do ++w.b; while (t.pre[w.b + 1] == t.pre[w.b]);
      w.L = t.lens[w.b];
      w.T = t.cu[w.b + 1] - t.cu[w.b];
    }
  }
  enter_tile(p, w);
}

// Steps to the next block; false at the end of the CTA's range.
__device__ __forceinline__ bool step(const Params& p, const Tables& t, Walk& w) {
  if (++w.x >= w.end) return false;
  if (++w.v == w.s.blocks) next_tile(p, t, w);
  return true;
}

// The CTA's blocks of w's tile from w on.
__device__ __forceinline__ int blocks_left(const Walk& w) {
  const int64_t left = w.end - w.x;
  return w.s.blocks - w.v < left ? w.s.blocks - w.v : (int)left;
}

// Key block number v of a tile.
__device__ __forceinline__ int block_at(const TileSpan& s, int v) { return v < s.lead ? v : v - s.lead + s.first; }
__device__ __forceinline__ int block_of(const Walk& w) { return block_at(w.s, w.v); }

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 128-byte-swizzled operand in shared memory, atoms of 8 rows (keys) of 128
// bytes (64 channels), 1,024 bytes apart. K-major (K): `wide` is not used.
// MN-major (V, channels are the N dimension): wide bytes between groups of 64
// channels.
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t addr, uint32_t wide) { return (addr >> 4) | ((wide >> 4) << 16); }
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);  // 1,024 bytes between groups of 8 keys; swizzle

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n mov.b64 b, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Two codes as fp16: u = code + 128 in the low byte of each half is, read as
// fp16, the subnormal u 2^-24; one fma forms (u - 128) 2^-24 S from S and
// -S 2^-17 with a single rounding.
__device__ __forceinline__ uint32_t scale_codes(uint32_t u2, __half2 s, __half2 bias) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&u2), s, bias);
  return *reinterpret_cast<const uint32_t*>(&r);
}
constexpr float kOperand = 32768.f;  // 2^15: an operand holds its value times 2^-(ev + 15)

// New exponent of a group whose largest scale has exponent E: S = s 2^(9 - ev)
// then lies in [2^11, 2^12), two octaves below where the group moves up and
// five above where it moves down. beta = 2^(ev_old - ev_new).
__device__ __forceinline__ void move_exponent(int& ev, int E, float& beta) {
  const int ne = E - 2 < -110 ? -110 : E - 2;
  const int d = ev == kEvUnset ? 0 : ev - ne;
  beta = d < -126 ? 0.f : pow2i(d > 127 ? 127 : d);
  ev = ne;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Params p) {
  using SM = Smem<D>;
  constexpr int G64 = D / 64;
  constexpr int kColO = 0, kColS = D < 128 ? 128 : D, kColQ = kColS + 128;  // tensor-memory columns
  static_assert(kColQ + D / 2 <= kTmemCols, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int64_t* pre = reinterpret_cast<int64_t*>(smem + SM::off_pre);
  int* lens = reinterpret_cast<int*>(smem + SM::off_lens);
  int* cus = reinterpret_cast<int*>(smem + SM::off_cu);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::off_misc);
  uint64_t* kfull = bars;        // [2] K block in shared memory (4 warps)
  uint64_t* vfull = bars + 2;    // [2] V block (4 warps)
  uint64_t* qkdone = bars + 4;   // [2] QK MMAs: scores there, K buffer free
  uint64_t* pvdone = bars + 6;   // [2] PV MMAs: accumulator up to date, V buffer free
  uint64_t* pfull = bars + 8;    // [2] P written (4 warps)
  uint64_t* qfull = bars + 10;   // Q of a tile written (4 warps)
  uint64_t* ofree = bars + 11;   // accumulator of a tile read (4 warps)
  uint64_t* rfull = bars + 12;   // [kStages] raw block in the ring (bytes)
  uint64_t* rfree = bars + 12 + kStages;  // [kStages] read by the 8 convert warps
  int* misc = reinterpret_cast<int*>(bars + 12 + 2 * kStages);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = misc + 1;
  int* last_mma = misc + 2;                             // block number of the last MMAs committed to pvdone / qkdone
  int* start = misc + 4;                                // [4] b, h, tile, v of the CTA's first block
  int* votes = misc + 8;                                // [2 operands][2][4 warps]
  float* maxima = reinterpret_cast<float*>(misc + 24);  // [2 operands][4 warps][4 groups]
  float* kfac = reinterpret_cast<float*>(misc + 56);    // [4] 2^e of a K block
  volatile int* seg_blocks = misc + 92;                 // [2] blocks of a segment, for the MMA warp
  volatile int* info = misc + 96;                       // [kStages] of a raw block: keys there | first of its segment << 8 | bad 16-key groups << 16
  int* last_raw = misc + 100;                           // raw blocks issued
  float* vhdr = reinterpret_cast<float*>(misc + 60);    // [2][16]: moved | 4 beta | 4 of 2^e

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  chain_wait();
  chain_release();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&kfull[i]), kConvWarps);
      mbar_init(smem_u32(&vfull[i]), kConvWarps);
      mbar_init(smem_u32(&qkdone[i]), 1);
      mbar_init(smem_u32(&pvdone[i]), 1);
      mbar_init(smem_u32(&pfull[i]), kSoftWarps);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&rfull[i]), 1);
      mbar_init(smem_u32(&rfree[i]), 2 * kConvWarps);
    }
    mbar_init(smem_u32(qfull), kSoftWarps);
    mbar_init(smem_u32(ofree), kSoftWarps);
    *abort_flag = 0;
    last_mma[0] = last_mma[1] = -1;
    *last_raw = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  // ---- the list of blocks: lengths, then the blocks of every sequence
  for (int b = tid; b <= p.B; b += kThreads) cus[b] = p.cu[b];
  for (int b = tid; b < p.B; b += kThreads) lens[b] = p.ctx[b];
  __syncthreads();
  for (int b = warp; b < p.B; b += kThreads / 32) {
    const int c0 = cus[b], c1 = cus[b + 1], L = lens[b];
    const int64_t T = (int64_t)c1 - c0;
    const bool ok = c0 >= 0 && T >= 0 && c1 <= p.total_q && T <= L && L <= p.max_ctx &&
                    (int64_t)L <= (int64_t)p.max_pages * p.P;
    int64_t n = 0;
    if (ok && T > 0) {
      const int tiles = tiles_of(p, (int)T);
      for (int t = lane; t < tiles; t += 32) n += span_of(p, L, (int)T, t).blocks;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) {
      pre[b] = n * p.Hkv;
      if (!ok && blockIdx.x == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
    }
  }
  __syncthreads();
  if (warp == 0) {  // exclusive prefix
    int64_t run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      const int64_t n = b < p.B ? pre[b] : 0;
      int64_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncwarp();
      if (b < p.B) pre[b] = run + inc - n;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) pre[p.B] = run;
  }
  __syncthreads();
  const int64_t W = pre[p.B];
  const int64_t most = (W + kMinBlocks - 1) / kMinBlocks;
  const int n = most < p.n_ctas ? (int)most : p.n_ctas;  // CTAs that take part
  const int cta = blockIdx.x;
  const bool idle = cta >= n;
  Walk w0 = {};
  if (!idle) {
    w0.x = cta_begin(W, n, cta);
    w0.end = cta_begin(W, n, cta + 1);
    if (warp == 0) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= w0.x) lo = mid; else hi = mid;
      }
      const int64_t per_head = (pre[lo + 1] - pre[lo]) / p.Hkv, off = w0.x - pre[lo];
      int64_t rem = off % per_head;
      const int T = cus[lo + 1] - cus[lo], tiles = tiles_of(p, T);
      int tile = 0;
      for (int t0 = 0; t0 < tiles; t0 += 32) {
        const int t = t0 + lane;
        const int nb = t < tiles ? span_of(p, lens[lo], T, t).blocks : 0;
        int64_t inc = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, inc > rem);
        if (past) {
          const int src = __ffs(past) - 1;
          const int64_t before = __shfl_sync(0xffffffffu, inc - nb, src);
          tile = t0 + src;
          rem -= before;
          break;
        }
        rem -= __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        start[0] = lo;
        start[1] = (int)(off / per_head);
        start[2] = tile;
        start[3] = (int)rem;
      }
    }
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;  // 0: all of the SM's columns
  const Tables tab{pre, lens, cus};
  if (!idle) {
    w0.b = start[0];
    w0.h = start[1];
    w0.tile = start[2];
    w0.v = start[3];
    w0.L = lens[w0.b];
    w0.T = cus[w0.b + 1] - cus[w0.b];
    enter_tile(p, w0);
  }
  const bool work = !idle && w0.x < w0.end;

  // A bounded wait; once one has run out no wait blocks any more, no MMA is
  // issued, and the end of the kernel waits for those that were. (The flag is
  // read only while a wait blocks: a read of shared memory in front of every
  // wait was a tenth of a block's time.)
  auto wait_bar = [&](uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar);
    if (mbar_try_wait(at, parity)) return;
    const unsigned long long t0 = clock64();
    while (!mbar_try_wait(at, parity)) {
      if (*abort_flag) return;
      if (clock64() - t0 > p.wait_cycles) {
        if (lane == 0) flag(p.status, NK_DEVFLAG_TIMEOUT);
        *abort_flag = 1;
        return;
      }
    }
  };
  const uint32_t kbuf = smem_u32(smem + SM::off_k), vbuf = smem_u32(smem + SM::off_v);

  if (!work) {
    if (tid == 0 && cta < p.n_ctas) p.desc[cta] = make_int4(0, -1, 0, 0);
  } else if (warp < kSoftWarps) {
    // ======================================================= softmax warps
    set_regs<kRegsSoft>();
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const int row = warp * 32 + lane;
    Walk w = w0;
    int j = 0, q_seg = 0;
    bool have_desc = false;
    bool more = true;
    // Q of w's tile into tensor memory; returns sm_scale log2(e) 2^-e of the thread's row
    auto load_q = [&]() -> float {
      const int r = w.tile * kRows + row;
      const bool live = r < w.s.r1;
      const int rr = live ? r : 0;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + ((int64_t)(cus[w.b] + rr / p.G) * p.Hq + w.h * p.G + rr % p.G) * D);
      float m = 0.f;
      if (live) {
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = __ldg(src + c);
          const uint32_t x4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(x4[i])), fabsf(bf16_hi(x4[i]))));
        }
      }
      // the sign of sm_scale goes into Q, so that scores scale by a positive factor
      const int e = q_norm_exp(m);
      const float qs = p.scale2 < 0.f ? -pow2i(e) : (p.scale2 > 0.f ? pow2i(e) : 0.f);
#pragma unroll 1
      for (int g = 0; g < G64; ++g) {
        uint32_t r32[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (live) x = __ldg(src + g * 8 + c);
          const uint32_t x4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) r32[c * 4 + i] = pack_f16(bf16_lo(x4[i]) * qs, bf16_hi(x4[i]) * qs);
        }
        tm_st32(lane_base + kColQ + g * 32, r32);
      }
      wait_st();
      fence_before();
      if (row == 0) seg_blocks[q_seg & 1] = blocks_left(w);
      ++q_seg;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(qfull));
      return p.scale2 == 0.f ? 1.f : fabsf(p.scale2) * pow2i(-e);
    };
    float kq = load_q();
    while (more) {
      // one segment: the CTA's blocks of w's tile
      const int nblk = blocks_left(w);
      const bool head = w.v == 0, whole = head && nblk == w.s.blocks;
      const int r = w.tile * kRows + row;
      const bool live = r < w.s.r1;
      const int pos = w.L - w.T + (live ? r : w.s.r1 - 1) / p.G;
      const int base_row = cus[w.b];
      float m_ref = -INFINITY, l = 0.f;
      float unscale[G64];
      const Walk at = w;  // the tile, for the output
      for (int i = 0; i < nblk; ++i, ++j) {
        const int key0 = block_at(w.s, w.v + i) * kKeys;
        wait_bar(&qkdone[j & 1], (j >> 1) & 1);
        fence_after();
        const uint32_t scol = lane_base + kColS + (j & 1) * 64;
        uint32_t lo[32], hi[32];
        tm_ld32(scol, lo);
        tm_ld32(scol + 32, hi);
        // the factor of the raw scores, kept a normal number (a masked -inf times 0 would be NaN)
        const float f = fminf(fmaxf(kq * kfac[j & 3] * kOperand, 1.2e-38f), 3.4e38f);
        wait_ld();
        float s[64];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          s[c] = __uint_as_float(lo[c]);
          s[32 + c] = __uint_as_float(hi[c]);
        }
        if (key0 + kKeys - 1 > w.s.p0) {
          const int lim = pos - key0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > lim) s[c] = -INFINITY;
        }
        if (p.window > 0 && key0 <= w.s.p1 - p.window && key0 + kKeys - 1 >= p.sinks) {
          const int lim = pos - p.window - key0, sk = p.sinks - key0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c <= lim && c >= sk) s[c] = -INFINITY;
        }
        float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(fmaxf(m4[i], s[c + i]), s[c + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], s[60 + i]);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f;
        // the reference moves at a row's first key and when a score passes it by more than 8
        const bool raise = mx > m_ref + 8.f;
        wait_bar(&vfull[j & 1], (j >> 1) & 1);  // the block's V exponents
        const float* vh = vhdr + (j & 1) * 16;
        const bool moved = reinterpret_cast<const int*>(vh)[0] != 0;
        const bool any = __any_sync(0xffffffffu, raise);
        float alpha = 1.f;
        if (raise) {
          alpha = ex2(m_ref - mx);  // 0 while the row was empty
          l *= alpha;
          m_ref = mx;
        }
        if (i > 0 && (any || moved)) {
          wait_bar(&pvdone[(j - 1) & 1], ((j - 1) >> 1) & 1);
          fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            const float a = moved ? alpha * vh[1 + c / 2] : alpha;
            uint32_t o[32];
            tm_ld32(lane_base + kColO + c * 32, o);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            tm_st32(lane_base + kColO + c * 32, o);
          }
          wait_st();
        }
        if (moved) {
#pragma unroll
          for (int g = 0; g < G64; ++g) unscale[g] = vh[5 + g];
        }
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
        // p = 2^(score f - m), two at a time; four partial sums
        const float2 f2 = make_float2(f, f), mu2 = make_float2(-mu, -mu);
        uint32_t pk[32];
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 t2 = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), f2, mu2);
          const float2 e2 = make_float2(ex2(t2.x), ex2(t2.y));
          sum[c & 1] = __fadd2_rn(sum[c & 1], e2);
          pk[c] = pack_f16(e2.x, e2.y);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tm_st32(scol, pk);
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&pfull[j & 1]));
      }
      w.x += nblk;
      w.v += nblk;
      more = w.x < w.end;
      if (more) next_tile(p, tab, w);
      // the next tile's Q while the last products run (its QKs wait for it;
      // this tile's have all completed)
      if (more) kq = load_q();
      wait_bar(&pvdone[(j - 1) & 1], ((j - 1) >> 1) & 1);
      fence_after();
      const float inv = l > 0.f ? kOperand / l : 0.f;
      bool finite = true;
      const int64_t slot = 2 * (int64_t)cta + (head ? 1 : 0);
      uint16_t* orow = p.out + ((int64_t)(base_row + (live ? r : 0) / p.G) * p.Hq + at.h * p.G + (live ? r : 0) % p.G) * D;
      float4* po = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * kRows + row;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tm_ld32(lane_base + kColO + c * 32, o);
        wait_ld();
        float un = unscale[0];
#pragma unroll
        for (int g = 1; g < G64; ++g) un = c / 2 == g ? unscale[g] : un;
        const float sc = inv * un;
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          v[k] = __uint_as_float(o[k]) * sc;
          finite &= isfinite(v[k]) != 0;
        }
        if (whole) {
          if (live) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t b4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                b4[i] = (uint32_t)f32_to_bf16(v[k * 8 + 2 * i]) | ((uint32_t)f32_to_bf16(v[k * 8 + 2 * i + 1]) << 16);
              *reinterpret_cast<uint4*>(orow + c * 32 + k * 8) = make_uint4(b4[0], b4[1], b4[2], b4[3]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            po[(c * 8 + k) * kRows] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      }
      if (live && !finite) flag(p.status, NK_DEVFLAG_RANGE);
      if (!whole) {
        p.part_lse[slot * kRows + row] = l > 0.f ? (m_ref + log2f(l)) * kLn2 : -INFINITY;
        if (head) {
          // the tile's first blocks: this CTA leaves what the join needs
          have_desc = true;
          if (row == 0) {
            const int last = cta_of_item(W, n, at.x - at.v + at.s.blocks - 1);
            p.desc[cta] = make_int4(base_row, at.h, at.tile * kRows, (at.s.r1 - at.tile * kRows) | ((last - cta + 1) << 8));
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(ofree));
    }
    if (!have_desc && row == 0) p.desc[cta] = make_int4(0, -1, 0, 0);
  } else if (warp < kMmaWarp) {
    // ======================================================= convert warps
    set_regs<kRegsConv>();
    const bool isv = warp >= kSoftWarps + kConvWarps;
    const int cw = (warp - kSoftWarps) & 3;  // keys 16 cw .. 16 cw + 15 of a block
    // Lane -> (key, 16-channel piece) of a load: a quarter warp takes four
    // pieces of two neighbouring keys, the odd key's in the other half of the
    // 128 bytes, so that neither its 16-byte reads of the raw rows nor its
    // swizzled stores meet in a bank.
    constexpr int KPI = 512 / D, NI = 16 / KPI;  // keys of a load, loads of a block
    const int qt = lane >> 3, kp = (lane >> 2) & 1;
    const int kk = D == 256 ? kp : (D == 128 ? (qt >> 1) * 2 + kp : qt * 2 + kp);
    const int ck = D == 64 ? lane & 3 : ((lane & 3) | (((qt ^ kp) & 1) << 2) | (D == 256 ? (qt >> 1) << 3 : 0));
    const int grp = ck >> 2;
    // raw rows and scales of this warp's keys in a stage
    const uint32_t raw0 = smem_u32(smem + SM::off_ring) + (isv ? kKeys * (D + G64 * 4) : 0);
    const uint32_t codes0 = raw0 + (cw * 16 + kk) * D + ck * 16, scales0 = raw0 + kKeys * D + (cw * 16 * G64 + lane) * 4;
    // this warp's table of scales: (S, -S 2^-17) as fp16 pairs, [16 keys][G64]
    const uint32_t tab0 = smem_u32(smem + SM::off_tab) + (warp - kSoftWarps) * (16 * G64 * 8);
    constexpr int NS = (16 * G64 + 31) / 32;  // scales of a lane (group lane % G64; one of two lanes at head dim 64)
    const bool has_scale = D > 64 || lane < 16;
    const int sgrp = isv ? lane % G64 : 0;    // group whose exponent they follow
    // store addresses: row (i KPI + kk) of the buffer, chunks 2 (ck & 3) and + 1 swizzled by the row mod 8; rows
    // repeat their swizzle every 8 / KPI loads
    constexpr int NA = 8 / KPI > 1 ? 8 / KPI : 1;
    uint32_t sa[NA][2];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        sa[i][c] = (isv ? vbuf : kbuf) + grp * (kKeys * 128) + (cw * 16 + i * KPI + kk) * 128 +
                   ((((ck & 3) * 2 + c) ^ ((i * KPI + kk) & 7)) << 4);
    uint64_t* full = isv ? vfull : kfull;
    uint64_t* done = isv ? pvdone : qkdone;
    int* votes_w = votes + (isv ? 8 : 0);
    const int bar_id = isv ? 2 : 1;
    const int total = (int)(w0.end - w0.x);
    bool bad_scale = false;
    int ev[4] = {kEvUnset, kEvUnset, kEvUnset, kEvUnset};
    float inv_e = 0.f;  // 2^-ev of the lane's group (0: not set)
    int st = 0;
    uint32_t ph = 0;
    for (int j = 0; j < total; ++j) {
      wait_bar(&rfull[st], ph);
      const int inf = info[st];
      const bool first = (inf >> 8) & 1;
      const int there = ((inf >> (16 + cw)) & 1) ? 0 : (inf & 0xff) - cw * 16;  // keys of this warp's 16 that exist
      uint4 w[NI];
      float s[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i)
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s[i]) : "r"(scales0 + st * SM::kStage + i * 128));
#pragma unroll
      for (int i = 0; i < NI; ++i)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                     : "r"(codes0 + st * SM::kStage + i * (KPI * D)));
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (!has_scale || (lane + 32 * i) / G64 >= there) s[i] = 0.f;  // no such key: stale codes count as zeros
        if (!(s[i] <= 3.0e38f)) {  // the append of a non-finite row: zeros too, flagged
          s[i] = 0.f;
          bad_scale = true;
        }
        mx = fmaxf(mx, s[i]);
      }
      // ---- exponents: a group moves when a scale passes 2^6 of it, or none of the block's reaches 2^-2
      if (isv && first) inv_e = 0.f;
      const float t = mx * inv_e;
      const uint32_t bits =
          __reduce_or_sync(0xffffffffu, ((t > 64.f ? 1u : 0u) | (t >= 0.25f ? 16u : 0u)) << sgrp);
      int* vote = votes_w + (j & 1) * 4;
      if (lane == 0) vote[cw] = (int)bits;
      named_bar(bar_id, kConvWarps * 32);
      const int4 v4 = *reinterpret_cast<const int4*>(vote);
      const uint32_t seen = (uint32_t)(v4.x | v4.y | v4.z | v4.w);
      const uint32_t moving = ((seen & 15u) | (~(seen >> 4) & 15u)) & (isv ? (1u << G64) - 1u : 1u);
      float beta[4] = {1.f, 1.f, 1.f, 1.f};
      if (moving) {
        float* mxs = maxima + (isv ? 16 : 0);
        if (isv && first) {
#pragma unroll
          for (int g = 0; g < 4; ++g) ev[g] = kEvUnset;
        }
#pragma unroll
        for (int g = 0; g < G64; ++g) {
          const uint32_t v = __reduce_max_sync(0xffffffffu, (!isv || sgrp == g) ? __float_as_uint(mx) : 0u);
          if (lane == 0) mxs[cw * 4 + g] = __uint_as_float(v);
        }
        named_bar(bar_id, kConvWarps * 32);
#pragma unroll
        for (int g = 0; g < G64; ++g) {
          if (!((moving >> g) & 1u)) continue;
          const float m4 = fmaxf(fmaxf(mxs[g], mxs[4 + g]), fmaxf(mxs[8 + g], mxs[12 + g]));
          if (m4 > 0.f) move_exponent(ev[g], exp_of(m4), beta[g]);
        }
        named_bar(bar_id, kConvWarps * 32);  // maxima read before a later block writes them
        int e = ev[0];
#pragma unroll
        for (int g = 1; g < G64; ++g) e = sgrp == g ? ev[g] : e;
        inv_e = e == kEvUnset ? 0.f : pow2i(-e);
      }
      // ---- the scales as fp16: S = s 2^(9 - ev) (zero where there is none)
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const __half2 sc = __float2half2_rn(s[i] * inv_e * 512.f);
        const __half2 bias = __hmul2(sc, __float2half2_rn(-7.62939453125e-6f));  // -S 2^-17
        if (has_scale)
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tab0 + (lane + 32 * i) * 8),
                       "r"(*reinterpret_cast<const uint32_t*>(&sc)), "r"(*reinterpret_cast<const uint32_t*>(&bias))
                       : "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&rfree[st]));  // every lane holds its part of the raw block
      // ---- the buffer's previous block has been multiplied
      wait_bar(&done[j & 1], ((j >> 1) & 1) ^ 1);
      if (cw == 0 && lane == 0) {
        if (isv) {
          float* vh = vhdr + (j & 1) * 16;
          const bool tell = moving != 0 || first;
          reinterpret_cast<int*>(vh)[0] = tell ? 1 : 0;
          if (tell) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              vh[1 + g] = beta[g];
              vh[5 + g] = ev[g] == kEvUnset ? 1.f : pow2i(ev[g]);
            }
          }
        } else {
          kfac[j & 3] = ev[0] == kEvUnset ? 1.f : pow2i(ev[0]);
        }
      }
      const uint32_t half_off = (j & 1) * SM::kTile;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t scu, biu;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(scu), "=r"(biu)
                     : "r"(tab0 + ((i * KPI + kk) * G64 + grp) * 8)
                     : "memory");
        const __half2 sc = *reinterpret_cast<const __half2*>(&scu), bi = *reinterpret_cast<const __half2*>(&biu);
        const uint32_t w4[4] = {w[i].x ^ 0x80808080u, w[i].y ^ 0x80808080u, w[i].z ^ 0x80808080u, w[i].w ^ 0x80808080u};
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[2 * k] = scale_codes(mma::prmt(w4[k], 0u, 0x4140), sc, bi);
          h[2 * k + 1] = scale_codes(mma::prmt(w4[k], 0u, 0x4342), sc, bi);
        }
        const uint32_t o = half_off + (i / NA) * (NA * KPI * 128);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sa[i % NA][0] + o), "r"(h[0]), "r"(h[1]),
                     "r"(h[2]), "r"(h[3]));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sa[i % NA][1] + o), "r"(h[4]), "r"(h[5]),
                     "r"(h[6]), "r"(h[7]));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0 && (p.withhold < 0 || j < p.withhold)) mbar_arrive(smem_u32(&full[j & 1]));
      if (++st == kStages) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (__any_sync(0xffffffffu, bad_scale) && lane == 0) flag(p.status, NK_DEVFLAG_RANGE);
  } else {
    // ======================================================= MMA warp
    set_regs<kRegsMma>();
    if (warp == kMmaWarp) {
      // The whole warp runs the loop and one elected lane issues. All 512
      // columns are this CTA's, so tensor memory starts at address 0: with
      // that and the warp's uniform loop every operand of an MMA is a uniform
      // register (a lane on its own paid some 75 cycles an MMA to move them).
      constexpr uint32_t id_qk = idesc_f16_f32(kRows, kKeys, false), id_pv = idesc_f16_f32(kRows, D, true);
      const bool leader = elect_one();
      const int total = (int)(w0.end - w0.x);
      const uint32_t k_lo = sdesc_lo(kbuf, 16), v_lo = sdesc_lo(vbuf, kKeys * 128);
      int j = 0, seg = 0, left = 0;  // blocks, segments, blocks left of the segment
      bool fresh = true;             // the segment's first PV is still to come
      auto pv = [&](int q) {
        wait_bar(&vfull[q & 1], (q >> 1) & 1);
        wait_bar(&pfull[q & 1], (q >> 1) & 1);
        if (*abort_flag) return;
        if (leader) {
          fence_after();
          const uint32_t a = kColS + (q & 1) * 64, v0 = v_lo + (q & 1) * (SM::kTile >> 4);
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            mma_ts(kColO, a + ks * 8, v0 + ks * (2048 >> 4), id_pv, ks > 0 || !fresh);
          mma_commit(smem_u32(&pvdone[q & 1]));
          last_mma[1] = q;
        }
        fresh = false;
      };
      while (j < total) {
        wait_bar(qfull, seg & 1);
        left = *abort_flag ? total - j : seg_blocks[seg & 1];
        for (int i = 0; i < left; ++i, ++j) {
          wait_bar(&kfull[j & 1], (j >> 1) & 1);
          if (!*abort_flag && leader) {
            fence_after();
            const uint32_t k0 = k_lo + (j & 1) * (SM::kTile >> 4), d = kColS + (j & 1) * 64;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              mma_ts(d, kColQ + ks * 8, k0 + (((ks / 4) * (kKeys * 128) + (ks % 4) * 32) >> 4), id_qk, ks > 0);
            mma_commit(smem_u32(&qkdone[j & 1]));
            last_mma[0] = j;
          }
          __syncwarp();
          if (i == 0) {
            fresh = true;
            continue;  // the first product of a segment goes out after its second QK
          }
          if (i == 1 && seg > 0) wait_bar(ofree, (seg - 1) & 1);
          pv(j - 1);
          __syncwarp();
        }
        if (left == 1 && seg > 0) wait_bar(ofree, (seg - 1) & 1);
        pv(j - 1);
        __syncwarp();
        ++seg;
      }
    }
    if (warp == kMmaWarp + 1) {
      // ===================================================== producer warp
      // lanes 0-3 take 16 keys of a block each (P is a multiple of 16: one
      // page holds them); with pages of whole blocks lane 0 takes all 64
      const int per = p.P % kKeys == 0 ? kKeys : 16;
      constexpr int kKeyBytes = 2 * D + 2 * G64 * 4;
      Walk w = w0;
      int st = 0, page = -2;
      uint32_t ph = 1u;  // a fresh ring is free
      bool first = true;
      auto look = [&]() {  // page id of the lane's keys (-2: no such keys)
        const int pos = block_of(w) * kKeys + lane * per;
        page = -2;
        if (lane * per < kKeys && pos < w.L) page = __ldg(p.bt + (int64_t)w.b * p.max_pages + pos / p.P);
      };
      look();
      for (int q = 0;; ++q) {
        const int key0 = block_of(w) * kKeys, pos = key0 + lane * per, h = w.h;
        const int keys = w.L - key0 < kKeys ? w.L - key0 : kKeys;
        const int cur = page;
        const bool was_first = first;
        const int b = w.b, tile = w.tile;
        const bool more = step(p, tab, w);
        if (more) {
          first = w.b != b || w.h != h || w.tile != tile;
          look();
        }
        const bool ok = cur >= 0 && cur < p.num_pages;
        const unsigned copies = __ballot_sync(0xffffffffu, ok), bad = __ballot_sync(0xffffffffu, !ok && cur != -2);
        wait_bar(&rfree[st], ph);
        const bool stop = *abort_flag;
        if (__any_sync(0xffffffffu, stop)) break;
        const uint32_t bar = smem_u32(&rfull[st]);
        if (lane == 0) {
          info[st] = keys | (was_first ? 256 : 0) | ((per == kKeys ? (bad ? 15u : 0u) : (bad & 15u)) << 16);
          if (bad) flag(p.status, NK_DEVFLAG_BAD_PAGE);
          mbar_arrive_expect_tx(bar, __popc(copies) * per * kKeyBytes);
          *last_raw = q + 1;
        }
        __syncwarp();
        if (ok) {
          const int slot = pos % p.P;
          const uint8_t* c = p.pool + ((int64_t)cur * p.Hkv + h) * p.lay.chunk;
          const uint32_t dst = smem_u32(smem + SM::off_ring + st * SM::kStage);
          const int k0 = lane * per;
          bulk_load(dst + k0 * D, c + (int64_t)slot * D, per * D, bar);
          bulk_load(dst + kKeys * D + k0 * G64 * 4, c + p.lay.ks + slot * G64 * 4, per * G64 * 4, bar);
          bulk_load(dst + kKeys * (D + G64 * 4) + k0 * D, c + p.lay.vc + (int64_t)slot * D, per * D, bar);
          bulk_load(dst + kKeys * (2 * D + G64 * 4) + k0 * G64 * 4, c + p.lay.vs + slot * G64 * 4, per * G64 * 4, bar);
        }
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
        if (!more) break;
      }
    }
    __syncwarp();
  }
  // ---- every MMA and copy that was issued completes before the tensor memory is released
  fence_before();
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      const int q = last_mma[i];
      uint64_t* bar = i ? pvdone : qkdone;
      if (q >= 0) (void)mbar_wait(smem_u32(&bar[q & 1]), (q >> 1) & 1, p.wait_cycles);
    }
    for (int q = *last_raw - kStages > 0 ? *last_raw - kStages : 0; q < *last_raw; ++q)
      (void)mbar_wait(smem_u32(&rfull[q % kStages]), (q / kStages) & 1, p.wait_cycles);
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the partials of a tile that several CTAs worked on: block (c, y) takes
// 16 rows of the tile whose first blocks were CTA c's last. Partial k of it
// is CTA c + k's (its own second slot, the others' first); weights as in
// nk_combine.cu. Thread = (row, every 16th group of four channels).
constexpr int kJoinRows = 16, kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ Params p) {
  chain_wait();
  chain_release();
  const int c = blockIdx.x;
  const int4 d = p.desc[c];
  if (d.y < 0) return;
  const int rows = d.w & 0xff, S = d.w >> 8;
  const int row = blockIdx.y * kJoinRows + (threadIdx.x % kJoinRows), cg0 = threadIdx.x / kJoinRows;
  if (row >= rows) return;
  auto slot = [&](int k) { return k == 0 ? 2 * (int64_t)c + 1 : 2 * (int64_t)(c + k); };
  float mx = -INFINITY;
  for (int k = 0; k < S; ++k) mx = fmaxf(mx, p.part_lse[slot(k) * kRows + row]);
  constexpr int NC = D / 4 / (kJoinThreads / kJoinRows);  // channel groups of a thread
  float4 acc[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int k = 0; k < S; ++k) {
    const float lse = p.part_lse[slot(k) * kRows + row];
    if (lse == -INFINITY) continue;
    const float wgt = expf(lse - mx);
    sum += wgt;
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + slot(k) * (D / 4) * kRows + row;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const float4 v = src[(cg0 + i * (kJoinThreads / kJoinRows)) * kRows];
      acc[i].x = fmaf(wgt, v.x, acc[i].x);
      acc[i].y = fmaf(wgt, v.y, acc[i].y);
      acc[i].z = fmaf(wgt, v.z, acc[i].z);
      acc[i].w = fmaf(wgt, v.w, acc[i].w);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int r = d.z + row;
  uint16_t* o = p.out + ((int64_t)(d.x + r / p.G) * p.Hq + d.y * p.G + r % p.G) * D;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t w0 = f32_to_bf16(acc[i].x * inv) | ((uint32_t)f32_to_bf16(acc[i].y * inv) << 16);
    const uint32_t w1 = f32_to_bf16(acc[i].z * inv) | ((uint32_t)f32_to_bf16(acc[i].w * inv) << 16);
    *reinterpret_cast<uint2*>(o + (cg0 + i * (kJoinThreads / kJoinRows)) * 4) = make_uint2(w0, w1);
  }
}

template <int D>
static cudaError_t launch_d(const Params& p, cudaStream_t st) {
  static_assert(Smem<D>::total <= kSmemLimit, "shared memory");
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(chunk_kernel<D>), Smem<D>::total);
  if (e != cudaSuccess) return e;
  static const int regs = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, chunk_kernel<D>) == cudaSuccess ? fa.numRegs : -1;
  }();
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = launch_chained(chunk_kernel<D>, dim3(p.n_ctas), dim3(kThreads), Smem<D>::total, st, p);
  if (e != cudaSuccess) return e;
  return launch_chained(chunk_join_kernel<D>, dim3(p.n_ctas, kRows / kJoinRows), dim3(kJoinThreads), 0, st, p);
}

cudaError_t launch(const Params& p, int D, cudaStream_t st) {
  if (D == 256) return launch_d<256>(p, st);
  if (D == 128) return launch_d<128>(p, st);
  return launch_d<64>(p, st);
}

}  // namespace chunk
}  // namespace nk
