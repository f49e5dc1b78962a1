// nk_weights_tc.cu -- the first kernel of nk_page_weights (nk_weights.cu) for
// many query rows: the scores on the 5th-generation tensor cores (tcgen05.mma,
// fp16 operands that hold the codes exactly, fp32 accumulators in tensor memory).
//
// A CTA takes up to 128 query rows of one (sequence, kv-head) after another
// against tiles of 64 keys: the rows are M, the keys N, and each 64-channel group
// has accumulators of its own (64 columns), because its scale is the key's. A row
// is one tensor-memory lane and one thread for each half of the tile's keys, which
// multiplies the groups' columns by the key's scales (read as one float4 that all
// lanes share), adds them, and forms the log-sum over its keys of the page:
// nothing is exchanged between threads. A page of more than 32 keys leaves several
// log-sums, pages of 16 or 32 keys share a tile.
//
// 28 warps, one CTA per SM:
//   warps 0-15  four warpgroups: two halves of the keys for the tiles of even
//               number, two for the odd (each parity has a set of accumulators);
//   warps 16-23 codes from the ring to fp16 in the swizzled operand buffers, all
//               eight at a tile (with four at the even and four at the odd ones a
//               buffer's conversion and product follow each other, slower); at a
//               segment's start the unit's rows, scaled into the fp16 range;
//   warp 24     issues the MMAs;
//   warps 25-26 walk the list, look up the pages, leave a description of every
//               tile for the others, and fill the rings of the even and the odd
//               tiles with bulk asynchronous copies (codes for the converters,
//               scales for the rows' threads); 27 has no part.
// Only the copying warps know segments and tables: with the walk in every role the
// registers spilled, and beside 217 KB of shared memory no L1 is left to hold a
// spill (8 windows of 16 tokens at 8K to 64K: 204 us for this kernel then).
// Bounded by the hand-offs between the roles: 8 windows of 16 tokens at 8K to 64K (96
// rows, 274K tokens, 4 kv-heads) take 198 us with the second kernel, 1.75 us a tile, where the
// products are 0.45 and the codes' bytes 0.38.
//
// Every mbarrier wait is bounded; after one has run out every role ends at its next
// wait, and the copies and products under way are waited for.
#include <math.h>

#include "nk_ptx.cuh"
#include "nk_weights.cuh"

namespace nk {
namespace lse_tc {

constexpr int kKeys = 64;
constexpr int kRowsMost = 128;
constexpr int kSoft = 16, kConv = 8;
constexpr int kMmaWarp = kSoft + kConv, kCopyWarp = kMmaWarp + 1;  // and the one behind it
constexpr int kThreads = (kMmaWarp + 4) * 32;  // whole warpgroups, for setmaxnreg
// Registers per thread: launched with 72 (896 threads); the shares below add up to
// no more than 7 * 72, so no increase waits for registers that are not there
// (checked on the host against the compiled count).
constexpr int kLaunchRegs = 72, kRegsSoft = 88, kRegsConv = 48, kRegsRest = 56;
static_assert(4 * kRegsSoft + 2 * kRegsConv + kRegsRest <= 7 * kLaunchRegs, "shares of the launch's registers");
template <int N>
__device__ __forceinline__ void set_regs() {
  if constexpr (N > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N) : "memory");
  if constexpr (N < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N) : "memory");
}
// Tiles whose codes, and whose scales, are in flight or in use: the scales stay
// until the rows' threads are done with the tile, three steps after the codes.
constexpr int kRaw = 4, kScales = 8, kRowSets = 4;
constexpr int kCols = 512;

template <int D>
struct Smem {
  static constexpr int NG = D / kGroup;
  static constexpr int off_q = 0;                                   // [NG][128 rows][128 bytes], swizzled
  static constexpr int off_b = off_q + NG * kRowsMost * 128;        // [2][NG][64 keys][128 bytes], swizzled
  static constexpr int off_raw = off_b + 2 * NG * kKeys * 128;      // [kRaw][64][D]
  static constexpr int off_sc = off_raw + kRaw * kKeys * D;         // [kScales][64][NG]
  static constexpr int off_undo = off_sc + kScales * kKeys * NG * 4;  // [kRowSets][128]
  static constexpr int off_pre = off_undo + kRowSets * kRowsMost * 4;
  static constexpr int off_lens = off_pre + (kMaxBatch + 4) * 4;
  static constexpr int off_misc = off_lens + kMaxBatch * 4;         // barriers and the rest
  static constexpr int total = off_misc + 448 + kScales * 32 + 1024;  // (slack to align the base)
  static_assert(total <= 227 * 1024, "shared memory");
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// K-major operand, 128-byte swizzle, atoms of 8 rows of 128 bytes, 1,024 bytes apart
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr >> 4) | (1u << 16); }
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
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
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tm_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}

// What the other warps know of a tile.
struct Tile {
  int pos0, keys;   // position of its first key; keys (of 64) that its pages have
  int len;          // the sequence's length; 0: the list is at its end
  int gone;         // blocks of 16 keys whose page is none, a bit each
  int entry;        // number of its first log-sum
  int unit, seg;    // sequence * kv-heads + kv-head; the CTA's segment
  int first;        // its first tile
};
static_assert(sizeof(Tile) == 32, "two 16-byte words");

template <int D>
__global__ void __launch_bounds__(kThreads, 1) lse_tc_kernel(const __grid_constant__ WeightParams p) {
  using SM = Smem<D>;
  constexpr int NG = SM::NG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* pre = reinterpret_cast<int*>(smem + SM::off_pre);
  int* lens = reinterpret_cast<int*>(smem + SM::off_lens);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::off_misc);
  int* tail = reinterpret_cast<int*>(smem + SM::off_misc + 320);
  int* warp_tot = tail;  // [28]
  volatile int* abort_flag = tail + 28;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tail + 29);
  Tile* desc = reinterpret_cast<Tile*>(smem + SM::off_misc + 448);  // [kScales]
  const uint32_t bar0 = smem_u32(bars);
  // barriers
  const auto raw_full = [&](int i) { return bar0 + 8 * i; };
  const auto raw_empty = [&](int i) { return bar0 + 8 * (kRaw + i); };
  const auto sc_full = [&](int i) { return bar0 + 8 * (2 * kRaw + i); };
  const auto sc_empty = [&](int i) { return bar0 + 8 * (2 * kRaw + kScales + i); };
  constexpr int kB = 2 * kRaw + 2 * kScales;
  const auto b_full = [&](int i) { return bar0 + 8 * (kB + i); };
  const auto b_empty = [&](int i) { return bar0 + 8 * (kB + 2 + i); };
  const auto acc_full = [&](int i) { return bar0 + 8 * (kB + 4 + i); };
  const auto acc_empty = [&](int i) { return bar0 + 8 * (kB + 6 + i); };
  const auto rows_full = [&](int i) { return bar0 + 8 * (kB + 8 + i); };
  static_assert((kB + 8 + kRowSets) * 8 <= 320, "barriers");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), kConv);
    }
    for (int i = 0; i < kScales; ++i) {
      mbar_init(sc_full(i), 1);
      mbar_init(sc_empty(i), kSoft / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_full(i), kConv);
      mbar_init(b_empty(i), 1);
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), kSoft / 2);
    }
    for (int i = 0; i < kRowSets; ++i) mbar_init(rows_full(i), kConv);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  chain_wait();
  chain_release();
  const int row0 = blockIdx.x * p.chunk, cta = blockIdx.y;
  if (blockIdx.x == 0 && cta == 0)
    for (int b = tid; b < p.sh.B; b += kThreads)
      if (pages_of_len(p.sh, p.ctx[b]) == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
  fence_before();
  block_page_prefix_short(p.sh, p.ctx, 0, pre, warp_tot, lens);  // (ends with a barrier)
  fence_after();
  const uint32_t tmem = *tslot;
  const int64_t W = (int64_t)pre[p.sh.B] * p.sh.Hkv;
  int64_t x = W > 0 ? cta_begin(W, p.n_ctas, cta) : 0;
  const int64_t x_end = W > 0 ? cta_begin(W, p.n_ctas, cta + 1) : 0;
  {  // a warpgroup may have no tile in a segment: its log-sums of it are empty unless it says otherwise
    int64_t y = x;
    Segment seg;
    while (next_segment(p.sh, pre, y, x_end, seg))
      for (int i = tid; i < 4 * p.chunk; i += kThreads)
        p.seg_lse[(((int64_t)cta + seg.u) * 4 + i / p.chunk) * p.rows + row0 + i % p.chunk] = -INFINITY;
    __syncthreads();
  }
  const auto wait = [&](uint32_t bar, uint32_t parity) {  // by whole warps
    if (!*abort_flag && !mbar_wait(bar, parity, p.wait_cycles)) {
      flag(p.status, NK_DEVFLAG_TIMEOUT);
      *abort_flag = 1;
    }
    __syncwarp();
  };
  // After a wait, by whole warps: one of the CTA's has run out, so this role ends where
  // it is (what a wait has not confirmed is not read, least of all a tile's description).
  const auto stopped = [&]() { return __any_sync(0xffffffffu, *abort_flag != 0); };

  if (warp < kSoft) {
    set_regs<kRegsSoft>();
    // ------------------------------------------------------------ rows
    const int wg = warp >> 2, set = wg & 1, half = wg >> 1, row = (warp & 3) * 32 + lane;
    const int M = p.sh.T * p.G, P = p.sh.P;
    const bool act = (warp & 3) * 32 < p.chunk;  // (warp-uniform: some of its rows are there)
    const bool mine = row < p.chunk;
    const int behind = p.sh.T - min(row0 + row, M - 1) / p.G;  // the last key that the row sees: length - behind
    const uint32_t acc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + set * NG * kKeys + half * (kKeys / 2);
    float ms = -INFINITY, ls = 0.f, un = 0.f;
    int seg = -1, unit = 0;
    for (int n = set;; n += 2) {
      const int sl = n % kScales;
      wait(sc_full(sl), (uint32_t)(n / kScales) & 1u);
      if (stopped()) break;
      const int4 d0 = *reinterpret_cast<const int4*>(desc + sl), d1 = *(reinterpret_cast<const int4*>(desc + sl) + 1);
      const int len = d0.z;
      if (len == 0 || d1.z != seg) {
        if (seg >= 0 && mine) p.seg_lse[(((int64_t)cta + unit) * 4 + wg) * p.rows + row0 + row] = lse_of(ms, ls);
        if (len == 0) break;
        unit = d1.y;
        ms = -INFINITY;
        ls = 0.f;
      }
      wait(acc_full(set), (uint32_t)(n >> 1) & 1u);
      if (d1.z != seg) {
        // (after the product, so in its phase: the barriers of segments without a tile of
        // this warpgroup were not waited for)
        seg = d1.z;
        wait(rows_full(seg % kRowSets), (uint32_t)(seg / kRowSets) & 1u);
        un = reinterpret_cast<const float*>(smem + SM::off_undo)[(seg % kRowSets) * kRowsMost + row];
      }
      if (stopped()) break;
      fence_after();
      if (act) {
        const float* scales = reinterpret_cast<const float*>(smem + SM::off_sc) + (sl * kKeys + half * (kKeys / 2)) * NG;
        float m = -INFINITY, l = 0.f;  // m: of the scores before their factor un
        // four keys a round, the next round's accumulators on their way meanwhile (wait_ld
        // waits for all of a thread's loads)
        uint32_t v[2][NG][4];
#pragma unroll
        for (int c = 0; c < NG; ++c) tm_ld4(acc + c * kKeys, v[0][c]);
        float s[16];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          wait_ld();
          if (r < 7) {
#pragma unroll
            for (int c = 0; c < NG; ++c) tm_ld4(acc + c * kKeys + 4 * (r + 1), v[(r + 1) & 1][c]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* f = scales + (4 * r + j) * NG;
            const auto at = [&](int c) { return __uint_as_float(v[r & 1][c][j]); };
            float& y = s[(r & 3) * 4 + j];
            if constexpr (NG == 4) {
              const float4 q = *reinterpret_cast<const float4*>(f);
              y = fmaf(q.w, at(3), fmaf(q.z, at(2), fmaf(q.y, at(1), q.x * at(0))));
            } else if constexpr (NG == 2) {
              const float2 q = *reinterpret_cast<const float2*>(f);
              y = fmaf(q.y, at(1), q.x * at(0));
            } else {
              y = f[0] * at(0);
            }
          }
          if ((r & 3) != 3) continue;
          // ---- a block of 16 keys
          const int blk = r >> 2, ko = half * (kKeys / 2) + blk * 16, base = d0.x + ko;  // its first key in the tile; its position
          if (ko >= d0.y) continue;
          if (base < len && !((d0.w >> (ko / 16)) & 1)) {
            const int last = len - behind - base;  // keys past it are not seen
            if (base + 15 > len - p.sh.T) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (j > last) s[j] = -INFINITY;
            }
            float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]);
#pragma unroll
            for (int j = 4; j < 16; j += 4) {
              x0 = fmaxf(x0, fmaxf(s[j], s[j + 1]));
              x1 = fmaxf(x1, fmaxf(s[j + 2], s[j + 3]));
            }
            const float mx = fmaxf(m, fmaxf(x0, x1));
            const float off = mx == -INFINITY ? 0.f : -mx * un;
            float s0 = l * wgt_ex2(fmaf(m, un, off)), s1 = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              s0 += wgt_ex2(fmaf(s[j], un, off));
              s1 += wgt_ex2(fmaf(s[j + 1], un, off));
            }
            l = s0 + s1;
            m = mx;
          }
          if (blk == 1 || P == 16 || ko + 16 >= d0.y) {  // the last of these keys
            const float mu = m == -INFINITY ? m : m * un;
            if (mine) p.page_lse[(int64_t)(d1.x + (P == 16 ? ko / 16 : half)) * p.rows + row0 + row] = lse_of(mu, l);
            lse_join(ms, ls, mu, l);
            m = -INFINITY;
            l = 0.f;
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(acc_empty(set));
        mbar_arrive(sc_empty(sl));
      }
    }
  } else if (warp < kMmaWarp) {
    set_regs<kRegsConv>();
    // ------------------------------------------------------------ codes to fp16
    const int cw = warp - kSoft;
    for (int n = 0;; ++n) {
      const int rs = n % kRaw, buf = n & 1;
      wait(raw_full(rs), (uint32_t)(n / kRaw) & 1u);
      if (stopped()) break;
      const int4 d0 = *reinterpret_cast<const int4*>(desc + n % kScales), d1 = *(reinterpret_cast<const int4*>(desc + n % kScales) + 1);
      if (d0.z == 0) {
        // (as for any tile, after the products over the buffer's last one: two phases ahead
        // of the wait for it, the barrier would hold that up for good)
        if (n >= 2) wait(b_empty(buf), (uint32_t)((n >> 1) - 1) & 1u);
        if (!stopped() && lane == 0) mbar_arrive(b_full(buf));
        break;
      }
      if (d1.w) {
        // the unit's rows, once every product over the last unit's is done (a wait goes by
        // parity and must not begin before the phase ahead of its own has ended: this
        // one's was waited for at the tile before)
        if (n >= 1) wait(b_empty(buf ^ 1), (uint32_t)((n - 1) >> 1) & 1u);
        if (stopped()) break;
        const int T = p.sh.T, G = p.G, Hkv = p.sh.Hkv, b = d1.y / Hkv, h = d1.y - b * Hkv;
        float* undo = reinterpret_cast<float*>(smem + SM::off_undo) + (d1.z % kRowSets) * kRowsMost;
        const float sign = p.scale2 < 0.f ? -1.f : 1.f;
        for (int r = cw; r < kRowsMost; r += kConv) {
          const int row = row0 + r, t = row / G, hg = row - t * G;
          const bool there = r < p.chunk && row < T * G;
          const uint16_t* src = p.q + (((int64_t)b * T + t) * (G * Hkv) + h * G + hg) * D;
          constexpr int PER = D / 64;
          uint32_t w[PER];
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            w[i] = there ? reinterpret_cast<const uint32_t*>(src)[lane + 32 * i] : 0u;
            m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int e = wgt_row_exp(m);
          const float up = sign * wgt_row_factor(m, e);
#pragma unroll
          for (int i = 0; i < PER; ++i) {  // word lane + 32 i: channels 2 lane + 64 i, + 1, so group i
            const __half2 hh = __floats2half2_rn(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
            *reinterpret_cast<uint32_t*>(smem + SM::off_q + i * (kRowsMost * 128) + r * 128 +
                                         (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) =
                *reinterpret_cast<const uint32_t*>(&hh);
          }
          // (never 0: masked scores times 0 would be NaN)
          if (lane == 0) undo[r] = fmaxf(fabsf(p.scale2) * wgt_pow2(-e), 1e-37f);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(rows_full(d1.z % kRowSets));
      }
      if (n >= 2) wait(b_empty(buf), (uint32_t)((n >> 1) - 1) & 1u);
      if (stopped()) break;
      const uint8_t* raw = smem + SM::off_raw + rs * (kKeys * D);
      uint8_t* dst = smem + SM::off_b + buf * (NG * kKeys * 128);
      constexpr int PCS = D / 16;  // 16-code pieces of a key
#pragma unroll 4
      for (int i = cw * 32 + lane; i < kKeys * PCS; i += kConv * 32) {
        const int key = i / PCS, j = i % PCS;
        const uint4 w = *reinterpret_cast<const uint4*>(raw + i * 16);
        const uint32_t u[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
        uint4 c0, c1;  // channels 16 j .. 16 j + 7, + 8 .. 15
        c0.x = wgt_f16(u[0], 0x4140), c0.y = wgt_f16(u[0], 0x4342), c0.z = wgt_f16(u[1], 0x4140), c0.w = wgt_f16(u[1], 0x4342);
        c1.x = wgt_f16(u[2], 0x4140), c1.y = wgt_f16(u[2], 0x4342), c1.z = wgt_f16(u[3], 0x4140), c1.w = wgt_f16(u[3], 0x4342);
        uint8_t* row = dst + (j >> 2) * (kKeys * 128) + key * 128;
        const int ch = 2 * (j & 3), sw = key & 7;
        // eight lanes store at once: those of odd groups their second half first, so
        // that the eight fall on distinct banks
        const bool flip = (j >> 2) & 1;
        *reinterpret_cast<uint4*>(row + (((ch + (flip ? 1 : 0)) ^ sw) << 4)) = flip ? c1 : c0;
        *reinterpret_cast<uint4*>(row + (((ch + (flip ? 0 : 1)) ^ sw) << 4)) = flip ? c0 : c1;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(b_full(buf));
        mbar_arrive(raw_empty(rs));
      }
    }
  } else {
    set_regs<kRegsRest>();
    if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      // The whole warp runs the loop and one elected lane issues. All 512 columns are
      // this CTA's, so tensor memory starts at address 0: with that every operand of a
      // product is a uniform register (a lane on its own, with the address from shared
      // memory, took some 100 cycles for each).
      const bool leader = elect_one();
      constexpr uint32_t id = idesc_f16(kRowsMost, kKeys);
      int done[2] = {0, 0};  // commits of each set
      const uint32_t qa = desc_lo(smem_u32(smem + SM::off_q)), kb = desc_lo(smem_u32(smem + SM::off_b));
      for (int n = 0;; ++n) {
        const int buf = n & 1;
        wait(b_full(buf), (uint32_t)(n >> 1) & 1u);
        if (stopped()) break;
        const Tile* t = desc + n % kScales;
        if (t->len == 0) break;
        if (t->first) wait(rows_full(t->seg % kRowSets), (uint32_t)(t->seg / kRowSets) & 1u);
        if (n >= 2) wait(acc_empty(buf), (uint32_t)((n >> 1) - 1) & 1u);
        if (stopped()) break;
        ++done[buf];
        if (leader) {
          fence_after();
          const uint32_t d = buf * NG * kKeys, k0 = kb + buf * ((NG * kKeys * 128) >> 4);
#pragma unroll
          for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(d + c * kKeys, qa + ((c * kRowsMost * 128 + k * 32) >> 4), k0 + ((c * kKeys * 128 + k * 32) >> 4), id, k > 0);
          mma_commit(b_empty(buf));
          mma_commit(acc_full(buf));
        }
        __syncwarp();
      }
      // after a wait that ran out products may still be under way: they end before tensor memory is given back
      if (*abort_flag)
        for (int i = 0; i < 2; ++i)
          if (done[i] > 0) (void)mbar_wait(b_empty(i), (uint32_t)(done[i] - 1) & 1u, p.wait_cycles);
    } else if (warp < kCopyWarp + 2) {
      // ------------------------------------------------------------ copies
      const int P = p.sh.P, Hkv = p.sh.Hkv, odd = warp - kCopyWarp;
      const int share = P < kKeys ? kKeys / P : 1;
      int n = 0, segs = 0, item = (int)x, sent = -1;  // sent: the last tile that was copied
      Segment seg;
      bool stop = false;
      while (!stop && next_segment(p.sh, pre, x, x_end, seg)) {
        const int L = lens[seg.b], pages = seg.page_end - seg.page_begin;
        const int32_t* bt = p.bt + (int64_t)seg.b * p.sh.max_pages + seg.page_begin;
        // page ids of 32 pages of the segment, and the next 32
        int have = 0, ids = lane < pages ? bt[lane] : -1, ids2 = 32 + lane < pages ? bt[32 + lane] : -1;
        bool first = true;
        for (int pg0 = 0; pg0 < pages && !stop; pg0 += share) {
          for (int k0 = 0; k0 < P && !stop; k0 += kKeys, ++n, first = false) {
            if ((n & 1) != odd) continue;
            const int rs = n % kRaw, sl = n % kScales;
            if (pg0 - have >= 32) {  // (32 is a whole number of a tile's pages: 4, 2 or 1)
              have += 32;
              ids = ids2;
              ids2 = have + 32 + lane < pages ? bt[have + 32 + lane] : -1;
            }
            // lane i < share: page pg0 + i
            const int id = __shfl_sync(0xffffffffu, ids, (pg0 - have + lane) & 31);
            const bool mine = lane < share && pg0 + lane < pages;
            const bool bad = mine && (id < 0 || id >= p.num_pages);
            if (bad) flag(p.status, NK_DEVFLAG_BAD_PAGE);
            const int live = mine && !bad ? min(min(P - k0, kKeys), L - (seg.page_begin + pg0 + lane) * P - k0) : 0;
            const int keys = live > 0 ? (live + 15) / 16 * 16 : 0;
            int all = keys + __shfl_xor_sync(0xffffffffu, keys, 1);
            all += __shfl_xor_sync(0xffffffffu, all, 2);  // (of lanes 0 to 3)
            // blocks of 16 keys of the pages that are none
            int gone = bad ? ((1 << (min(P - k0, kKeys) / 16)) - 1) << (lane * (P / 16)) : 0;
            gone = __reduce_or_sync(0xffffffffu, gone);
            if (n >= kRaw) wait(raw_empty(rs), (uint32_t)(n / kRaw - 1) & 1u);
            if (n >= kScales) wait(sc_empty(sl), (uint32_t)(n / kScales - 1) & 1u);
            stop = stopped();
            if (stop) continue;
            const bool held = p.withhold >= 0 && n >= p.withhold;
            if (!held) sent = n;
            if (lane == 0) {
              int4* d = reinterpret_cast<int4*>(desc + sl);
              const int there = min(min(P - k0, kKeys) * min(share, pages - pg0), kKeys);
              d[0] = make_int4((seg.page_begin + pg0) * P + k0, there, L, gone);
              d[1] = make_int4((item + pg0) * p.parts + k0 / (kKeys / 2), seg.u, segs, first);
              if (held) {
                // (nobody arrives: a test of the waits)
              } else if (all > 0) {
                mbar_arrive_expect_tx(raw_full(rs), all * D);
                mbar_arrive_expect_tx(sc_full(sl), all * NG * 4);
              } else {
                mbar_arrive(raw_full(rs));
                mbar_arrive(sc_full(sl));
              }
            }
            __syncwarp();
            if (!held && keys > 0) {
              const uint8_t* chunk = p.pool + ((int64_t)id * Hkv + seg.h) * p.lay.chunk;
              const int at = lane * P;  // (lane 0 alone where pages have several tiles)
              bulk_load(smem_u32(smem + SM::off_raw + rs * (kKeys * D) + at * D), chunk + (int64_t)k0 * D, keys * D, raw_full(rs));
              bulk_load(smem_u32(smem + SM::off_sc + (sl * kKeys + at) * NG * 4), chunk + p.lay.ks + k0 * NG * 4,
                        keys * NG * 4, sc_full(sl));
            }
            __syncwarp();
          }
        }
        ++segs;
        item += pages;
      }
      // the list's end, for the roles of this warp's tiles
      if ((n & 1) != odd) ++n;
      const int rs = n % kRaw, sl = n % kScales;
      if (n >= kRaw) wait(raw_empty(rs), (uint32_t)(n / kRaw - 1) & 1u);
      if (n >= kScales) wait(sc_empty(sl), (uint32_t)(n / kScales - 1) & 1u);
      if (!stopped() && lane == 0) {
        desc[sl].len = 0;
        mbar_arrive(raw_full(rs));
        mbar_arrive(sc_full(sl));
      }
      // after a wait that ran out some copies may still be in flight: they land before the CTA ends
      if (*abort_flag) {
        for (int i = sent; i >= 0 && i > sent - kRaw; i -= 2)
          (void)mbar_wait(raw_full(i % kRaw), (uint32_t)(i / kRaw) & 1u, p.wait_cycles);
        for (int i = sent; i >= 0 && i > sent - kScales; i -= 2)
          (void)mbar_wait(sc_full(i % kScales), (uint32_t)(i / kScales) & 1u, p.wait_cycles);
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

template <int D>
static cudaError_t launch(const WeightParams& p, int chunks, cudaStream_t st) {
  static const bool regs_ok = [] {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, lse_tc_kernel<D>) != cudaSuccess) {
      (void)cudaGetLastError();
      return false;
    }
    return fa.numRegs == kLaunchRegs;
  }();
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(lse_tc_kernel<D>), Smem<D>::total);
  if (e != cudaSuccess) return e;
  return launch_chained(lse_tc_kernel<D>, dim3((unsigned)chunks, (unsigned)p.n_ctas), dim3(kThreads),
                        (size_t)Smem<D>::total, st, p);
}

}  // namespace lse_tc

cudaError_t launch_lse_tc(const WeightParams& p, int chunks, cudaStream_t st) {
  if (p.D == 256) return lse_tc::launch<256>(p, chunks, st);
  if (p.D == 128) return lse_tc::launch<128>(p, chunks, st);
  return lse_tc::launch<64>(p, chunks, st);
}

}  // namespace nk
