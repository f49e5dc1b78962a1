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
// 2^-11 relative each where the output's bf16 rounding is 2^-8. The exponent e
// keeps the products inside the fp16 range for any pool. It is one of 16 keys
// and all their channels (of their largest scale, groups of zeros left out),
// undone on the scores for K and put into the weights for V (P carries
// 2^(e - e_ref) beside exp2(S - m)). A value far below the largest of those 16
// keys is off by the fp16 steps at the bottom of the range instead, at most
// 2^-20 of that largest: scales are brought up to 2^15, where the operand's
// largest is above 2^-4 and two half steps of 2^-25 are what the fma and its
// rounded second operand can lose.
//
// 20 warps in five warpgroups, one CTA per SM:
//   warps 0-7   softmax, two warpgroups that take the blocks of a tile in turn,
//               one thread a row: S from tensor memory, masks, running maximum
//               with a lazy reference (moved only when a score passes it by
//               more than 8, so the accumulator is rarely rescaled; the two
//               hand it to each other), P back to tensor memory over S, row
//               sums, and the tile's output;
//   warps 8-15  K, then V, of 16 keys a warp, four warps for the blocks of even
//               number and four for the odd: codes and scales from the ring,
//               widened to fp16, scaled, stored to the operand buffer of that
//               parity; a warp's chain of waits, loads and stores is longer
//               than a block's time, so two blocks are under way;
//   warp 16     issues the MMAs: QK of block j + 1 goes out before PV of block
//               j, so the tensor cores work while the softmax does;
//   warp 17     walks the list, looks up the pages and fills a two-stage ring of
//               raw blocks with bulk asynchronous copies (18 and 19 have no
//               part: setmaxnreg takes whole warpgroups).
//
// What bounds it: per 64-key block at head dim 256 the MMAs take 1,026 cycles
// of the tensor cores, the copies, codes, fp16 tiles and MMA operands about
// 1,700 of shared memory, and about 4,800 warp instructions 1,200 issue slots
// of each scheduler; a block takes about 2,050 cycles, so the hand-offs between
// the roles count beside each of them. Eight chunks of 1,024 tokens at 8K to
// 32K (24 q-heads over 4 kv-heads): 3,525 us in a loop, under the power cap
// (1,059 TFLOP/s), 3,320 for a few calls; four in a window of 4,096: 481.
//
// Taken against, on those eight chunks (a few calls each): codes loaded straight into the convert
// warps' registers instead of the ring, 7,345 us (4,720 with the ring, other
// things equal); MMAs issued by one lane of a diverged warp 4,332 (3,518 from
// a uniform one); two threads a row, 32 keys each, that exchange their maxima
// for every block 3,880; 16 convert warps with K and V apart 3,757; the scores
// of block j + 1 read while the weights of block j are formed 4,243 (3,418
// otherwise).
//
// Work split. The tiles are one list. With more than two tiles a CTA they are
// first dealt out whole, in rounds of one tile each: neighbouring tiles, which
// share their keys, then run side by side and read them from L2 (with every
// CTA on its own stretch of the list instead, eight chunks of 1,024 tokens at
// 8K to 32K read 11.3 GB from device memory and took 3,418 us). The blocks of the remaining
// tiles, one to two a CTA, or of all tiles where there are fewer, are cut into
// contiguous ranges that even out the CTAs' totals, whatever the sequences'
// lengths (stream-K). A tile cut by a range's end leaves fp32 partials with
// their log-sum-exp in the workspace; a second kernel joins them. Every
// mbarrier wait is bounded.
#include <math.h>

#include "nk_chunk.cuh"
#include "nk_decode_mma.cuh"

namespace nk {
namespace chunk {

using mma::ex2;
using mma::exp_of;
using mma::kSmemLimit;
using mma::named_bar;
using mma::pack_f16;
using mma::pow2i;
using mma::q_norm_exp;

constexpr int kKeys = 64;   // keys of a block
constexpr int kSoftWarps = 8, kConvWarps = 8;  // half of each for blocks of even number, half for odd
constexpr int kMmaWarp = kSoftWarps + kConvWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;  // whole warpgroups, for setmaxnreg
// Registers per thread: launched with 96 (640 threads); the shares below add
// up to 5 * 96, so no increase waits for registers that are not there (checked
// on the host against the compiled count).
constexpr int kLaunchRegs = 96, kRegsSoft = 128, kRegsConv = 80, kRegsMma = 64;
// setmaxnreg.inc must not lower a count, .dec must not raise one (an illegal instruction otherwise).
template <int N>
__device__ __forceinline__ void set_regs() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "setmaxnreg takes multiples of 8");
  if constexpr (N > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N) : "memory");
  if constexpr (N < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N) : "memory");
}
static_assert(2 * kRegsSoft + 2 * kRegsConv + kRegsMma == 5 * kLaunchRegs, "shares = the launch's registers");
constexpr int kTmemCols = 512;
constexpr int kStages = 2;  // raw blocks in flight (a third does not fit at head dim 256), one of each parity
constexpr int kMaxSched = 160;  // CTAs of a call whose tiles are dealt out whole first (one per SM has fewer)

// A segment: the blocks of one tile that fall into the CTA's range. The
// producer warp, which walks the list, leaves them for the softmax and MMA
// warps; it is at most 8 blocks, so 9 segments, ahead of the softmax.
struct Seg {
  int blocks, v, lead, first;  // blocks; number of the first in its tile; the tile's TileSpan
  int p0, p1;                  // positions of the tile's first and last token
  int r0, rows;                // its first row in the unit, its rows
  int pos0;                    // position of the unit's first token
  int base, h;                 // query row of that token, kv-head
  int flags;                   // 1: begins the tile, 2: is all of it, 4: the CTA's last
  int join;                    // CTAs that work on the tile
  int pad[3];
};
static_assert(sizeof(Seg) == 64, "a slot of the ring");
constexpr int kSegs = 16;

template <int D>
struct Smem {
  static constexpr int kTile = kKeys * D * 2;  // one fp16 K or V block
  static constexpr int off_k = 0;              // [2]
  static constexpr int off_v = 2 * kTile;      // [2]
  static constexpr int kStage = kKeys * (2 * D + 2 * (D / 64) * 4);  // raw block: K codes | K scales | V codes | V scales
  static constexpr int off_ring = 4 * kTile;                         // [kStages]
  static constexpr int off_tab = off_ring + kStages * kStage;        // [8 convert warps][K | V][16 keys][D / 64] scales
  static constexpr int off_pre = off_tab + 16 * 16 * (D / 64) * 8;   // int64 [kMaxBatch + 1]: blocks before sequence b
  static constexpr int off_tiles = off_pre + (kMaxBatch + 2) * 8;  // int [kMaxBatch + 1]: tiles before sequence b
  static constexpr int off_cu = off_tiles + (kMaxBatch + 4) * 4;  // int [kMaxBatch + 1]
  static constexpr int off_pair = off_cu + (kMaxBatch + 4) * 4;   // float [6][128], int16 [2][128]: what the two softmax threads of a row hand each other
  static constexpr int off_segs = off_pair + 6 * kRows * 4 + 2 * kRows * 2;       // [kSegs] segments
  static constexpr int off_misc = off_segs + kSegs * 64;
  static constexpr int total = off_misc + 1408 + 1024;  // slack to align the base
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
  const int64_t* pre;     // blocks before a sequence
  const int* tiles;       // tiles before it (of all kv-heads)
  const int* cu;
  const int32_t* ctx;     // in device memory
  int B;
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
      w.L = __ldg(t.ctx + w.b);
      w.T = t.cu[w.b + 1] - t.cu[w.b];
    }
  }
  enter_tile(p, w);
}

// Tile number i of the list, whole.
__device__ __forceinline__ void tile_at(const Params& p, const Tables& t, int i, Walk& w) {
  int lo = 0, hi = t.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.tiles[mid] <= i) lo = mid; else hi = mid;
  }
  w.b = lo;
  w.L = __ldg(t.ctx + lo);
  w.T = t.cu[lo + 1] - t.cu[lo];
  const int per = tiles_of(p, w.T), k = i - t.tiles[lo];
  w.h = (unsigned)k / (unsigned)per;
  w.tile = k - w.h * per;
  w.v = 0;
  enter_tile(p, w);
  w.x = 0;
  w.end = w.s.blocks;
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
constexpr int kNoExp = -1000;  // 16 keys that are all zero, or not there
constexpr int kOperand = 12;  // an operand holds its value times 2^-(e + kOperand)
// Weights are held 2^kUp up. A score may pass its reference by kScoreSlack
// before that moves (by 4 only, and the accumulator is rescaled so often that
// four chunks in a window take 556 us instead of about 480), so the largest fp16 weight is
// 2^15, and one of 2^-32 of the reference weight still counts: without the 2^7,
// 131,072 keys 2^-25.5 below a dominant one were lost from the product, but not
// from the row sum (0.3 % of the result).
constexpr int kUp = 7, kScoreSlack = 8;
static_assert(kUp + kScoreSlack <= 15, "fp16 weights");

// 2^x for any whole x (0 or infinity past the range).
__device__ __forceinline__ float pow2_any(int x) { return x < -126 ? 0.f : (x > 127 ? INFINITY : pow2i(x)); }

__device__ __forceinline__ void tm_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
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
  int* tiles = reinterpret_cast<int*>(smem + SM::off_tiles);
  int* cus = reinterpret_cast<int*>(smem + SM::off_cu);
  float* pair_x = reinterpret_cast<float*>(smem + SM::off_pair);
  int16_t* pair_e = reinterpret_cast<int16_t*>(pair_x + 6 * kRows);
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
  uint64_t* segfull = bars + 12 + 2 * kStages;  // [kSegs]
  uint64_t* handed = bars + 12 + 2 * kStages + kSegs;  // [2][4] references after a block, per 32 rows
  int* misc = reinterpret_cast<int*>(bars + 20 + 2 * kStages + kSegs);
  Seg* segs = reinterpret_cast<Seg*>(smem + SM::off_segs);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort_flag = misc + 1;
  int* last_mma = misc + 2;                             // block number of the last MMAs committed to pvdone / qkdone
  int* start = misc + 4;                                // [4] b, h, tile, v of the CTA's first block
  int* exps = misc + 32;                                // [4][K | V][4]: e of 16 keys of a block
  volatile uint16_t* live = reinterpret_cast<volatile uint16_t*>(misc + 96);  // [kStages][4] of a raw block: the keys that count, a bit each
  int* last_raw = misc + 100;                           // raw blocks issued
  int* longest = misc + 101;                            // blocks of the longest tile
  int* sched = misc + 104;                              // [kMaxSched + 1] where the CTAs' shares of the last tiles begin

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  chain_wait();
  chain_release();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&kfull[i]), kConvWarps / 2);
      mbar_init(smem_u32(&vfull[i]), kConvWarps / 2);
      mbar_init(smem_u32(&qkdone[i]), 1);
      mbar_init(smem_u32(&pvdone[i]), 1);
      mbar_init(smem_u32(&pfull[i]), kSoftWarps / 2);
      for (int k = 0; k < 4; ++k) mbar_init(smem_u32(&handed[i * 4 + k]), 1);
    }
    for (int i = 0; i < kSegs; ++i) mbar_init(smem_u32(&segfull[i]), 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&rfull[i]), 1);
      mbar_init(smem_u32(&rfree[i]), kConvWarps / 2);
    }
    mbar_init(smem_u32(qfull), kSoftWarps);
    mbar_init(smem_u32(ofree), kSoftWarps);
    *abort_flag = 0;
    last_mma[0] = last_mma[1] = -1;
    *last_raw = 0;
    *longest = 1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  // ---- the list of tiles and blocks
  for (int b = tid; b <= p.B; b += kThreads) cus[b] = p.cu[b];
  __syncthreads();
  for (int b = warp; b < p.B; b += kThreads / 32) {
    const int c0 = cus[b], c1 = cus[b + 1], L = __ldg(p.ctx + b);
    const int64_t T = (int64_t)c1 - c0;
    const bool ok = c0 >= 0 && T >= 0 && c1 <= p.total_q && T <= L && L <= p.max_ctx &&
                    (int64_t)L <= (int64_t)p.max_pages * p.P;
    const int nt = ok ? tiles_of(p, (int)T) : 0;
    int64_t n = 0;
    int most = 0;
    for (int t = lane; t < nt; t += 32) {
      const int k = span_of(p, L, (int)T, t).blocks;
      n += k;
      most = max(most, k);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      pre[b] = n * p.Hkv;
      tiles[b] = nt;
      atomicMax(longest, most);
      if (!ok && blockIdx.x == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
    }
  }
  __syncthreads();
  if (warp == 0) {  // exclusive prefixes
    int64_t run = 0, trun = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      const int64_t n = b < p.B ? pre[b] : 0, nt = b < p.B ? (int64_t)tiles[b] * p.Hkv : 0;
      int64_t inc = n, tinc = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o), z = __shfl_up_sync(0xffffffffu, tinc, o);
        if (lane >= o) {
          inc += y;
          tinc += z;
        }
      }
      __syncwarp();
      if (b < p.B) {
        pre[b] = run + inc - n;
        tiles[b] = (int)min(trun + tinc - nt, (int64_t)0x7fffffff);
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
      trun += __shfl_sync(0xffffffffu, tinc, 31);
    }
    if (lane == 0) {
      pre[p.B] = run;
      tiles[p.B] = (int)min(trun, (int64_t)0x7fffffff);
    }
  }
  __syncthreads();
  const Tables tab{pre, tiles, cus, p.ctx, p.B};
  const int64_t W = pre[p.B];
  const int nctas = W < p.n_ctas ? (int)W : p.n_ctas;  // CTAs that take part, a block each at least
  const int cta = blockIdx.x;
  const bool idle = cta >= nctas;
  // ---- whole tiles first: `waves` rounds of one tile a CTA
  int waves = 0;
  if (!idle && nctas <= kMaxSched && tiles[p.B] < 0x7fffffff && W < 0x7fffffff) {
    waves = tiles[p.B] / nctas - 1;
    waves = min(waves, (int)min(quot(quot(W, nctas), *longest), (int64_t)0x7fffffff));
    waves = max(waves, 0);
  }
  const int first_split = waves * nctas;  // first tile of those that are split
  int64_t split0 = 0;                     // its first block
  if (waves > 0) {
    // what the rounds give each CTA; the rest of its share comes from the
    // split tiles (a block at least, so that no CTA between two is left out)
    if (tid < nctas) {
      int64_t got = 0;
      Walk w;
      for (int k = 0; k < waves; ++k) {
        tile_at(p, tab, tid + k * nctas, w);
        got += w.s.blocks;
      }
      sched[tid] = (int)max(quot(W, nctas) + 1 - got, (int64_t)1);
    }
    Walk w;
    tile_at(p, tab, first_split, w);  // (there are at least nctas tiles after the rounds)
    for (int k = lane; k < w.tile; k += 32) split0 += span_of(p, w.L, w.T, k).blocks;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) split0 += __shfl_xor_sync(0xffffffffu, split0, o);
    split0 += pre[w.b] + w.h * quot(pre[w.b + 1] - pre[w.b], p.Hkv);
    __syncthreads();
    if (warp == 0) {
      int run = 0;
      for (int c0 = 0; c0 <= nctas; c0 += 32) {
        const int c = c0 + lane, v = c < nctas ? sched[c] : 0;
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        __syncwarp();
        if (c <= nctas) sched[c] = run + inc - v;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    __syncthreads();
  }
  // ---- the CTA's blocks of the split tiles
  Walk w0 = {};
  int total = 0;
  if (!idle) {
    if (waves > 0) {
      w0.x = min(split0 + sched[cta], W);
      w0.end = min(split0 + sched[cta + 1], W);
    } else {
      w0.x = cta_begin(W, nctas, cta);
      w0.end = cta_begin(W, nctas, cta + 1);
    }
    if (warp == 0 && w0.x < w0.end) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= w0.x) lo = mid; else hi = mid;
      }
      const int64_t per_head = quot(pre[lo + 1] - pre[lo], p.Hkv), off = w0.x - pre[lo], head = quot(off, per_head);
      int64_t rem = off - head * per_head;
      const int T = cus[lo + 1] - cus[lo], nt = tiles_of(p, T), L = __ldg(p.ctx + lo);
      int tile = 0;
      for (int t0 = 0; t0 < nt; t0 += 32) {
        const int t = t0 + lane;
        const int nb = t < nt ? span_of(p, L, T, t).blocks : 0;
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
        start[1] = (int)head;
        start[2] = tile;
        start[3] = (int)rem;
      }
    }
    total = (int)(w0.end - w0.x);
    Walk w;
    for (int k = 0; k < waves; ++k) {
      tile_at(p, tab, cta + k * nctas, w);
      total += w.s.blocks;
    }
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;  // 0: all of the SM's columns
  const bool work = total > 0;

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
  // The segments come from the producer warp. The softmax warps meet in
  // barriers, so all of them have to go through the same segments, also after a
  // wait has run out: the producer then leaves one more, marked as the CTA's
  // last, and stops. While nothing has run out the ring of raw blocks keeps it
  // 8 blocks, so 9 segments, ahead at most; with that one they are 10 of the 16
  // slots, and no slot is written that a softmax warp may still have to read.
  auto wait_seg = [&](int sg) {
    const unsigned long long t0 = clock64();
    while (!mbar_try_wait(smem_u32(&segfull[sg % kSegs]), (sg / kSegs) & 1))
      if (clock64() - t0 > 16 * p.wait_cycles) break;
  };
  const uint32_t kbuf = smem_u32(smem + SM::off_k), vbuf = smem_u32(smem + SM::off_v);

  if (!work) {
    if (tid == 0 && cta < p.n_ctas) p.desc[cta] = make_int4(0, -1, 0, 0);
  } else if (warp < kSoftWarps) {
    // ======================================================= softmax warps
    set_regs<kRegsSoft>();
    const int quad = warp & 3, half = warp >> 2;  // rows (tensor-memory lanes); blocks of even or odd number
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const int row = quad * 32 + lane;
    int j0 = 0;  // number of the segment's first block
    bool have_desc = false;
    // Q of segment sg's tile into tensor memory (this warp: every other 64
    // channels); returns |sm_scale| log2(e) 2^-e of the thread's row
    auto load_q = [&](int sg) -> float {
      wait_seg(sg);
      const Seg& sd = segs[sg % kSegs];
      const bool live = row < sd.rows;
      const int rr = live ? sd.r0 + row : 0;
      const uint4* src =
          reinterpret_cast<const uint4*>(p.q + ((int64_t)(sd.base + rr / p.G) * p.Hq + sd.h * p.G + rr % p.G) * D);
      // the thread's channels (every other 64) in one go, their largest |q|, then the row's
      constexpr int NQ = (G64 + 1) / 2;
      uint32_t q32[NQ][32];
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < NQ; ++k)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int g = half + 2 * k;
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (live && g < G64) x = __ldg(src + g * 8 + c);
          q32[k][4 * c] = x.x;
          q32[k][4 * c + 1] = x.y;
          q32[k][4 * c + 2] = x.z;
          q32[k][4 * c + 3] = x.w;
        }
#pragma unroll
      for (int k = 0; k < NQ; ++k)
#pragma unroll
        for (int c = 0; c < 32; ++c) m = fmaxf(m, fmaxf(fabsf(bf16_lo(q32[k][c])), fabsf(bf16_hi(q32[k][c]))));
      pair_x[(4 + half) * kRows + row] = m;
      named_bar(1 + quad, 64);
      m = fmaxf(m, pair_x[(5 - half) * kRows + row]);
      // the sign of sm_scale goes into Q, so that scores scale by a positive factor
      const int e = q_norm_exp(m);
      const float qs = p.scale2 < 0.f ? -pow2i(e) : (p.scale2 > 0.f ? pow2i(e) : 0.f);
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        const int g = half + 2 * k;
        if (g < G64) {
#pragma unroll
          for (int c = 0; c < 32; ++c) q32[k][c] = pack_f16(bf16_lo(q32[k][c]) * qs, bf16_hi(q32[k][c]) * qs);
          tm_st32(lane_base + kColQ + g * 32, q32[k]);
        }
      }
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(qfull));
      return p.scale2 == 0.f ? 1.f : fabsf(p.scale2) * pow2i(-e);
    };
    float kq = load_q(0);
    bool more = true;
    for (int sg = 0; more; ++sg) {
      const Seg& sd = segs[sg % kSegs];
      const int nblk = sd.blocks;
      const int v0 = sd.v, lead = sd.lead, shift = sd.first - lead;
      const int pos = sd.pos0 + (sd.r0 + (row < sd.rows ? row : sd.rows - 1)) / p.G;
      const int causal = sd.p0 - (kKeys - 1);                               // blocks past it hold hidden keys
      const int behind = p.window > 0 ? sd.p1 - p.window : -0x7fffffff - 1;  // blocks up to it may
      // The two warpgroups take the blocks in turn, so that two are under way.
      // The references of a row's weights and of its values' exponents go
      // from block to block through shared memory; a thread's row sum follows
      // its own copy of the reference.
      float m_ref = -INFINITY, l = 0.f;
      int e_ref = kNoExp;  // the accumulator holds l O 2^(kUp - e_ref - kOperand)
      for (int i = (half ^ j0) & 1; i < nblk; i += 2) {
        const int j = j0 + i;
        const int key0 = (v0 + i < lead ? v0 + i : v0 + i + shift) * kKeys;
        wait_bar(&qkdone[half], (j >> 1) & 1);
        fence_after();
        const uint32_t scol = lane_base + kColS + half * 64;
        uint32_t lo[32], hi[32];
        tm_ld32(scol, lo);
        tm_ld32(scol + 32, hi);
        // the factors of the raw scores (16 keys each), kept normal numbers (a masked -inf times 0 would be NaN)
        const int4 ke = *reinterpret_cast<const int4*>(exps + (j & 3) * 8), ve = *reinterpret_cast<const int4*>(exps + (j & 3) * 8 + 4);
        auto factor = [&](int e) { return fminf(fmaxf(kq * pow2_any(e + kOperand), 1.2e-38f), 3.4e38f); };
        const float f[4] = {factor(ke.x), factor(ke.y), factor(ke.z), factor(ke.w)};
        int vd[4] = {ve.x, ve.y, ve.z, ve.w};
        wait_ld();
        float s[64];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          s[c] = __uint_as_float(lo[c]);
          s[32 + c] = __uint_as_float(hi[c]);
        }
        // hidden scores; 16 keys that are all hidden from the row must not set its exponents either
        if (key0 > causal) {
          const int lim = pos - key0;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (16 * g > lim) vd[g] = kNoExp;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > lim) s[c] = -INFINITY;
        }
        if (key0 <= behind && key0 + kKeys - 1 >= p.sinks) {
          const int lim = pos - p.window - key0, sk = p.sinks - key0;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (16 * g + 15 <= lim && 16 * g >= sk) vd[g] = kNoExp;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c <= lim && c >= sk) s[c] = -INFINITY;
        }
        float m4[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float a = fmaxf(s[16 * g], s[16 * g + 1]), b = fmaxf(s[16 * g + 2], s[16 * g + 3]);
#pragma unroll
          for (int c = 4; c < 16; c += 4) {
            a = fmaxf(fmaxf(a, s[16 * g + c]), s[16 * g + c + 1]);
            b = fmaxf(fmaxf(b, s[16 * g + c + 2]), s[16 * g + c + 3]);
          }
          m4[g] = fmaxf(a, b) * f[g];
        }
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const int vmax = max(max(vd[0], vd[1]), max(vd[2], vd[3]));
        // ---- the references after the block before
        const float m_own = m_ref;
        if (j > 0) wait_bar(&handed[(1 - half) * 4 + quad], ((j - 1) >> 1) & 1);
        if (i > 0) {
          m_ref = pair_x[(1 - half) * kRows + row];
          e_ref = pair_e[(1 - half) * kRows + row];
        }
        // The reference moves at a row's first key and when a score passes it
        // by more than kScoreSlack. The weights of 16 keys carry their values' exponent,
        // p 2^(ve - e_ref). e_ref follows the largest ve that the row has seen
        // (hidden keys must not cost it bits) and never falls, so that what is
        // in the accumulator only ever shrinks.
        const bool moved = vmax > e_ref;
        const bool change = __any_sync(0xffffffffu, moved || mx > m_ref + (float)kScoreSlack);  // rare
        float a = 1.f;
        if (change) {
          if (mx > m_ref + (float)kScoreSlack) {
            a = ex2(m_ref - mx);  // 0 while the row was empty
            m_ref = mx;
          }
          if (moved) {
            a *= pow2_any(e_ref - vmax);
            e_ref = vmax;
          }
        }
        pair_x[half * kRows + row] = m_ref;
        pair_e[half * kRows + row] = (int16_t)e_ref;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&handed[half * 4 + quad]));
        if (__any_sync(0xffffffffu, m_ref != m_own)) l *= m_own == -INFINITY ? 0.f : ex2(m_own - m_ref);
        if (change && i > 0) {  // the accumulator follows
          wait_bar(&pvdone[1 - half], ((j - 1) >> 1) & 1);
          fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tm_ld16(lane_base + kColO + c * 16, o);
            wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            tm_st16(lane_base + kColO + c * 16, o);
          }
          wait_st();
        }
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
        // ---- p 2^d = 2^(score f - m + d), two at a time, d = kUp + ve - e_ref of 16 keys each; the row sum is of p
        uint32_t pk[32];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int d = max(vd[g] - e_ref, -60) + kUp;  // 2^-60 of the weights is nothing in fp16
          const float2 mu2 = make_float2((float)d - mu, (float)d - mu), f2 = make_float2(f[g], f[g]);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 8 * g; c < 8 * g + 8; ++c) {
            const float2 t2 = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), f2, mu2);
            const float2 e2 = make_float2(ex2(t2.x), ex2(t2.y));
            sum = __fadd2_rn(sum, e2);
            pk[c] = pack_f16(e2.x, e2.y);
          }
          l = fmaf(sum.x + sum.y, pow2i(-d), l);
        }
        tm_st32(scol, pk);
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&pfull[half]));
      }
      j0 += nblk;
      more = !(sd.flags & 4);
      // the next tile's Q while the last products run (its QKs wait for it;
      // this tile's have all completed)
      wait_bar(&qkdone[(j0 - 1) & 1], ((j0 - 1) >> 1) & 1);  // (the other threads' block, maybe)
      if (more) kq = load_q(sg + 1);
      // ---- both threads of a row: the last block's references, the whole row sum
      wait_bar(&handed[((j0 - 1) & 1) * 4 + quad], ((j0 - 1) >> 1) & 1);
      const float m_end = pair_x[((j0 - 1) & 1) * kRows + row];
      e_ref = pair_e[((j0 - 1) & 1) * kRows + row];
      if (l > 0.f) l *= ex2(m_ref - m_end);
      m_ref = m_end;
      pair_x[(2 + half) * kRows + row] = l;
      named_bar(1 + quad, 64);
      l += pair_x[(3 - half) * kRows + row];
      wait_bar(&pvdone[(j0 - 1) & 1], ((j0 - 1) >> 1) & 1);
      fence_after();
      // back to O: 2^(e_ref + kOperand - kUp) / l (the power in two steps, each a normal number)
      const float up = e_ref == kNoExp ? 1.f : pow2i(e_ref), inv = l > 0.f ? pow2i(kOperand - kUp) / l : 0.f;
      bool finite = true;
      const bool head = sd.flags & 1, whole = sd.flags & 2, live = row < sd.rows;
      const int64_t slot = 2 * (int64_t)cta + (head ? 1 : 0);
      const int rr = live ? sd.r0 + row : 0;
      uint16_t* orow = p.out + ((int64_t)(sd.base + rr / p.G) * p.Hq + sd.h * p.G + rr % p.G) * D;
      float4* po = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * kRows + row;
#pragma unroll 1
      for (int c = half; c < D / 32; c += 2) {
        uint32_t o[32];
        tm_ld32(lane_base + kColO + c * 32, o);
        wait_ld();
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          v[k] = __uint_as_float(o[k]) * inv * up;
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
        // (a row sum that is NaN, of a query that is not finite, stays NaN through the join)
        if (half == 0) p.part_lse[slot * kRows + row] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
        if (head) {
          // the tile's first blocks: this CTA leaves what the join needs
          have_desc = true;
          if (tid == 0) p.desc[cta] = make_int4(sd.base, sd.h, sd.r0, sd.rows | (sd.join << 8));
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(ofree));
      named_bar(1 + quad, 64);  // the row sums and references are read before the next segment's are written
    }
    if (!have_desc && tid == 0) p.desc[cta] = make_int4(0, -1, 0, 0);
  } else if (warp < kMmaWarp) {
    // ======================================================= convert warps
    set_regs<kRegsConv>();
    const int odd = (warp - kSoftWarps) >> 2;  // the blocks, ring stage and operand buffers of this warp
    const int cw = (warp - kSoftWarps) & 3;    // keys 16 cw .. 16 cw + 15 of a block
    // Lane -> (key, 16-channel piece) of a load: a quarter warp takes four
    // pieces of two neighbouring keys, the odd key's in the other half of the
    // 128 bytes, so that neither its 16-byte reads of the raw rows nor its
    // swizzled stores meet in a bank.
    constexpr int KPI = 512 / D, NI = 16 / KPI;  // keys of a load, loads of a block
    const int qt = lane >> 3, kp = (lane >> 2) & 1;
    const int kk = D == 256 ? kp : (D == 128 ? (qt >> 1) * 2 + kp : qt * 2 + kp);
    const int ck = D == 64 ? lane & 3 : ((lane & 3) | (((qt ^ kp) & 1) << 2) | (D == 256 ? (qt >> 1) << 3 : 0));
    const int grp = ck >> 2;
    // raw rows and scales of this warp's keys in its stage (K; V lies kRawV bytes on)
    constexpr int kRawV = kKeys * (D + G64 * 4);
    const uint32_t raw0 = smem_u32(smem + SM::off_ring) + odd * SM::kStage;
    const uint32_t codes0 = raw0 + (cw * 16 + kk) * D + ck * 16, scales0 = raw0 + kKeys * D + (cw * 16 * G64 + lane) * 4;
    // this warp's tables of scales: (S, -S 2^-17) as fp16 pairs, [K | V][16 keys][G64]
    constexpr int kTab = 16 * G64 * 8;
    const uint32_t tab0 = smem_u32(smem + SM::off_tab) + (warp - kSoftWarps) * (2 * kTab);
    const uint32_t tabp = tab0 + (kk * G64 + grp) * 8;
    constexpr int NS = (16 * G64 + 31) / 32;  // scales of a lane (one of two lanes at head dim 64)
    const bool has_scale = D > 64 || lane < 16;
    // the first row's store address; rows i KPI further on add i KPI 128 and xor (i KPI mod 8) into the 16-byte chunk
    const uint32_t sa = kbuf + odd * SM::kTile + grp * (kKeys * 128) + (cw * 16 + kk) * 128 + ((((ck & 3) * 2) ^ (kk & 7)) << 4);
    bool bad_scale = false;
    uint32_t ph = 0;  // phase of the stage and (inverted) of the operand buffers
    static_assert(kStages == 2, "a stage per parity");
    for (int j = odd; j < total; j += 2, ph ^= 1u) {
      wait_bar(&rfull[odd], ph);
      const uint32_t keys = live[odd * 4 + cw];  // of this warp's 16: those that count
      // ---- scales of K and V, and the exponents, which have to be there with the scores
      int es[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        float s[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s[i]) : "r"(scales0 + v * kRawV + i * 128));
        float mx = 0.f, mn = INFINITY;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          if (!has_scale || !((keys >> ((lane + 32 * i) / G64)) & 1u)) s[i] = 0.f;  // (whatever the codes are)
          float a = fabsf(s[i]);
          if (!(a <= 3.4028234e38f)) {  // infinite of either sign or NaN, the append of a non-finite row: zeros too, flagged
            s[i] = a = 0.f;
            bad_scale = true;
          }
          mx = fmaxf(mx, a);
          if (a > 0.f) mn = fminf(mn, a);
        }
        float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
        const float lo = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(mn)));
        // The scale of a group whose codes are all zero says nothing of a size (the append writes 1): it must not set the
        // exponent of the 16 keys. Looked for where the largest scale could be such a one: at exactly 1, or far above the
        // smallest; elsewhere it costs no bits.
        if (m == 1.f || m > 256.f * lo) {
          mx = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            if (s[i] != 0.f) {
              uint32_t any = 0;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint4 x;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                             : "r"(raw0 + v * kRawV + cw * 16 * D + (lane + 32 * i) * 64 + c * 16));
                any |= x.x | x.y | x.z | x.w;
              }
              if (any == 0) s[i] = 0.f;
            }
            mx = fmaxf(mx, fabsf(s[i]));
          }
          m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
        }
        // the 16 keys take the exponent of their own largest scale: S = s 2^(24 - kOperand - e) lies below 2^15
        es[v] = m > 0.f ? max(exp_of(m) - 2, -110) : kNoExp;
        const float down = m > 0.f ? pow2i(24 - kOperand - es[v]) : 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const __half2 sc = __float2half2_rn(s[i] * down);
          const __half2 bias = __hmul2(sc, __float2half2_rn(-7.62939453125e-6f));  // -S 2^-17
          if (has_scale)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tab0 + v * kTab + (lane + 32 * i) * 8),
                         "r"(*reinterpret_cast<const uint32_t*>(&sc)), "r"(*reinterpret_cast<const uint32_t*>(&bias))
                         : "memory");
        }
      }
      // (the slot's last reader, the softmax of block j - 4, is done: its PV was waited for at block j - 2)
      if (lane == 0) {
        exps[(j & 3) * 8 + cw] = es[0];
        exps[(j & 3) * 8 + 4 + cw] = es[1];
      }
#pragma unroll
      for (int v = 0; v < 2; ++v) {  // K, V
        uint4 w[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                       : "r"(codes0 + v * kRawV + i * (KPI * D)));
        __syncwarp();
        if (v == 1 && lane == 0) mbar_arrive(smem_u32(&rfree[odd]));  // every lane holds its part of the raw block
        // ---- the buffer's previous block has been multiplied
        wait_bar((v ? pvdone : qkdone) + odd, ph ^ 1u);
        constexpr int NH = NI < 4 ? NI : 4;  // loads whose scales are in registers at once
#pragma unroll
        for (int i0 = 0; i0 < NI; i0 += NH) {
          uint32_t scu[NH], biu[NH];
#pragma unroll
          for (int i = 0; i < NH; ++i)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(scu[i]), "=r"(biu[i])
                         : "r"(tabp + v * kTab + (i0 + i) * (KPI * G64 * 8))
                         : "memory");
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const uint4 x = w[i0 + i];
            const __half2 sc = *reinterpret_cast<const __half2*>(&scu[i]), bi = *reinterpret_cast<const __half2*>(&biu[i]);
            const uint32_t w4[4] = {x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[2 * k] = scale_codes(mma::prmt(w4[k], 0u, 0x4140), sc, bi);
              h[2 * k + 1] = scale_codes(mma::prmt(w4[k], 0u, 0x4342), sc, bi);
            }
            const uint32_t a0 = (sa ^ ((((i0 + i) * KPI) & 7) << 4)), at = v * (2 * SM::kTile) + (i0 + i) * (KPI * 128);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a0 + at), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                         "r"(h[3]));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"((a0 ^ 16u) + at), "r"(h[4]), "r"(h[5]),
                         "r"(h[6]), "r"(h[7]));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && (p.withhold < 0 || j < p.withhold)) mbar_arrive(smem_u32((v ? vfull : kfull) + odd));
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
        left = *abort_flag ? total - j : segs[seg % kSegs].blocks;
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
      // Lane -> (array, group of keys): K codes, K scales, V codes, V scales of
      // a whole block where pages hold whole blocks, else of 16 keys each (P
      // is a multiple of 16: one page holds them). The page ids come 32 (8)
      // blocks at a time, a lane each, one batch ahead.
      const bool whole = p.P % kKeys == 0;
      const int per = whole ? kKeys : 16, batch = whole ? 32 : 8;
      constexpr int kKeyBytes = 2 * D + 2 * G64 * 4;
      const int arr = lane & 3, kg = lane >> 2;
      const bool copier = kg * per < kKeys;
      const int width = (arr & 1) ? G64 * 4 : D;  // bytes of a key in the array
      const int64_t src_off = arr == 0 ? 0 : (arr == 1 ? p.lay.ks : (arr == 2 ? p.lay.vc : p.lay.vs));
      const uint32_t dst0 = smem_u32(smem + SM::off_ring) + (arr == 0 ? 0 : (arr == 1 ? kKeys * D : (arr == 2 ? kKeys * (D + G64 * 4) : kKeys * (2 * D + G64 * 4)))) +
                            kg * per * width;
      // Page and slot of the lane's keys in the batch of w's tile from block v on. Page -1: outside the pool; -2: no such
      // keys; -3: before the window of the tile's first token and behind the sinks, so nobody sees them and their page
      // may have been given back: neither the entry nor the page is read (in a whole-block page some key is seen).
      auto look = [&](const Walk& w, int v, int n, int& page, int& slot) {
        const int i = whole ? lane : lane >> 2;
        const int pos = block_at(w.s, v + i) * kKeys + (whole ? 0 : (lane & 3) * 16);
        page = -2;
        slot = 0;
        if (i < n && pos < w.L) {
          if (!whole && p.window > 0 && pos + 15 <= w.s.p0 - p.window && pos >= p.sinks) {
            page = -3;
          } else {
            const int pi = pos / p.P;
            slot = pos - pi * p.P;
            page = __ldg(p.bt + (int64_t)w.b * p.max_pages + pi);
            if (page < 0 || page >= p.num_pages) page = -1;
          }
        }
      };
      // the tiles of the rounds, then the CTA's blocks of the split tiles
      Walk w;
      int wave = 0;
      auto begin_split = [&](Walk& a) {
        a = w0;
        a.b = start[0];
        a.h = start[1];
        a.tile = start[2];
        a.v = start[3];
        a.L = __ldg(p.ctx + a.b);
        a.T = cus[a.b + 1] - cus[a.b];
        enter_tile(p, a);
      };
      if (waves > 0) tile_at(p, tab, cta, w);
      else begin_split(w);
      int page, slot, q = 0, sg = 0;
      look(w, w.v, blocks_left(w), page, slot);
      bool more = true;
      while (more) {
        // one segment
        const int n = blocks_left(w), v0 = w.v, L = w.L, h = w.h;
        const TileSpan span = w.s;
        const bool split = wave >= waves;
        Walk ahead = w;
        const bool ends = __any_sync(0xffffffffu, *abort_flag != 0);  // a wait has run out: this segment is the last
        if (++wave < waves) {
          tile_at(p, tab, cta + wave * nctas, ahead);
        } else if (!split) {
          more = w0.x < w0.end;
          if (more) begin_split(ahead);
        } else {
          ahead.x += n;
          ahead.v += n;
          more = ahead.x < ahead.end;
          if (more) next_tile(p, tab, ahead);
        }
        if (ends) more = false;
        if (lane == 0) {
          Seg& s = segs[sg % kSegs];
          const int r0 = w.tile * kRows;
          const bool head = v0 == 0, all = head && n == span.blocks;
          s.blocks = n;
          s.v = v0;
          s.lead = span.lead;
          s.first = span.first;
          s.p0 = span.p0;
          s.p1 = span.p1;
          s.r0 = r0;
          s.rows = span.r1 - r0;
          s.pos0 = L - w.T;
          s.base = cus[w.b];
          s.h = h;
          s.flags = (head ? 1 : 0) | (all ? 2 : 0) | (more ? 0 : 4);
          s.join = 0;
          if (head && !all) {  // the CTA of the tile's last block
            const int64_t last = w.x + span.blocks - 1;
            int c = waves > 0 ? cta : cta_of_item(W, nctas, last);
            while (waves > 0 && c + 1 < nctas && split0 + sched[c + 1] <= last) ++c;
            s.join = c - cta + 1;
          }
          mbar_arrive(smem_u32(&segfull[sg % kSegs]));
        }
        ++sg;
        for (int i = 0; i < n; ++i, ++q) {
          const int at = i % batch;
          int next_page = -2, next_slot = 0;
          const bool turn = at == batch - 1 || i == n - 1;  // the batch's last block: the next batch's ids go out
          if (turn) {
            if (i < n - 1) look(w, v0 + i + 1, n - i - 1, next_page, next_slot);
            else if (more) look(ahead, ahead.v, blocks_left(ahead), next_page, next_slot);
          }
          const int from = whole ? at : at * 4 + (kg & 3);
          const int pg = __shfl_sync(0xffffffffu, page, from), sl = __shfl_sync(0xffffffffu, slot, from);
          const bool ok = copier && pg >= 0;
          const unsigned okb = __ballot_sync(0xffffffffu, ok && arr == 0);
          const unsigned outb = __ballot_sync(0xffffffffu, copier && arr == 0 && (pg == -1 || pg == -3));  // not copied: zeros
          const bool bad = __any_sync(0xffffffffu, copier && arr == 0 && pg == -1);
          const int st = q % kStages;
          wait_bar(&rfree[st], ((q / kStages) & 1) ^ 1u);
          if (__any_sync(0xffffffffu, *abort_flag != 0)) break;  // no more copies
          const uint32_t bar = smem_u32(&rfull[st]);
          if (lane == 0) {
            // The keys that count: in the sequence, in pages that were copied, and seen by some token of the tile (from
            // the window of its first token on, or a sink; not behind its last token). What nobody sees must neither set
            // an exponent nor a flag.
            const int k0 = block_at(span, v0 + i) * kKeys, end = min(span.p1 + 1 - k0, kKeys);  // (p1 < L)
            uint64_t on = ~0ull >> (kKeys - end);
            if (p.window > 0) {
              const int from = max(p.sinks - k0, 0);  // hidden: from .. to
              const int to = (int)min((int64_t)span.p0 - p.window - k0, (int64_t)(kKeys - 1));
              if (from <= to) on &= ~((~0ull >> (kKeys - 1 - to)) & (~0ull << from));
            }
            // bits 0, 4, 8, 12 of outb are the 16-key groups, bit 0 alone a whole block
#pragma unroll
            for (int c = 0; c < 4; ++c)
              live[st * 4 + c] = ((whole ? outb : outb >> (4 * c)) & 1u) ? 0 : (uint16_t)(on >> (16 * c));
            if (bad) flag(p.status, NK_DEVFLAG_BAD_PAGE);
            mbar_arrive_expect_tx(bar, __popc(okb) * per * kKeyBytes);
            *last_raw = q + 1;
          }
          __syncwarp();
          if (ok)
            bulk_load(dst0 + st * SM::kStage,
                      p.pool + ((int64_t)pg * p.Hkv + h) * p.lay.chunk + src_off + (int64_t)sl * width, per * width, bar);
          if (turn) {
            page = next_page;
            slot = next_slot;
          }
        }
        w = ahead;
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
