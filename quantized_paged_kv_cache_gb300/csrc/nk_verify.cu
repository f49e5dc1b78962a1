// nk_verify.cu -- the end of a verify round: drafted tokens accepted against
// the target's probabilities, and the next token drawn (nk_verify_drafts).
//
// Draft t of a sequence, token x, is accepted when u_t q_t(x) < p_t(x), as far
// as every one before it was, compared exactly. With a the number
// accepted, the next token is drawn from r = max(p_a - q_a, 0) (each difference
// rounded once to 32 bits) where draft a was refused, from p_a where none was
// left: the lowest i with r_0 + .. + r_i > u R, R the sum of r. Such a sum over
// a vocabulary does not survive 32 bits (a thousand tokens lie within its last
// ones), and 64-bit floating point is slow on this chip. The r are summed as
// whole multiples of 2^-62: exact to 2^-62 a token, in any order the same.
//
// One cluster a sequence, each CTA a slice of the vocabulary, each warp a part
// of that: sums up, the slices' sums exchanged through distributed shared
// memory, and the one part that the drawn number falls in is read again (from
// L2) and summed ever finer: by 256 tokens a warp, then by 32, then by one.
// Bounded by the two rows' bytes for many sequences, for few by latency: the
// drafts, their probabilities, the rows, the exchange, the part again (64 sequences
// of 131,072 tokens: 16.2 us, 4.1 TB/s; one of 50,001: 6.2 us).
#include <cooperative_groups.h>

#include "nk_common.cuh"
#include "nk_host.cuh"

namespace nk {

struct VerifyParams {
  const float* p;
  const float* q;  // may be NULL: the drafts are certain (q is 1 at the draft)
  int64_t p_stride, q_stride;
  const int32_t* drafts;  // [B][T-1]
  const int32_t* num;     // [B] or NULL
  const float* u;         // [B][T]
  const int32_t* ctx;     // [B] or NULL
  int T, V;
  int32_t* tokens;    // [B][T]
  int32_t* accepted;  // [B]
  int32_t* next;      // [B] or NULL
  int32_t* status;
};

constexpr int kVerThreads = 256, kVerWarps = kVerThreads / 32;
constexpr int kVerUnroll = 16;
constexpr uint64_t kVerCap = 0x7fffffffffffffffull;  // a sum of 2 or more ends here

__device__ __forceinline__ uint64_t ver_add(uint64_t a, uint64_t b) {  // (both at most the cap)
  const uint64_t s = a + b;
  return s > kVerCap ? kVerCap : s;
}
__device__ __forceinline__ uint64_t ver_warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = ver_add(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// r of one token as a multiple of 2^-62, cut off below; NaN and negative ones
// count as zero, more than one as one. With r = 2^(e - 127) 1.m that is 1.m at bit
// 62, moved right by 127 - e: shifts, since the conversion to 64 bits was what the
// first form waited for.
__device__ __forceinline__ uint32_t shr_all(uint32_t x, uint32_t s) {  // (0 past 31)
  uint32_t y;
  asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(s));
  return y;
}
__device__ __forceinline__ uint64_t ver_weight(float p, float q) {
  const uint32_t b = __float_as_uint(__saturatef(p - q));
  const uint32_t top = ((b << 7) & 0x3fffffffu) | 0x40000000u, s = 127u - (b >> 23);
  // (the funnel shift moves by 32 at most, the rest follows)
  const uint32_t hi = shr_all(top, s), lo = shr_all(__funnelshift_rc(0u, top, s), max(s, 32u) - 32u);
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ float ver_uniform(float u) {  // the nearest one in [0, 1); NaN: 0
  return fminf(fmaxf(u, 0.f), 0.99999994f);
}

// u q < p, exactly: with h the rounded product and e its error, u q lies on h's side
// of p, and where h is p the error's sign tells. Both sides by 2^64, so that no error
// underflows where h can be p.
__device__ __forceinline__ bool ver_accept(float u, float q, float p) {
  constexpr float up = 18446744073709551616.f;
  const float a = u * up, b = p * up, h = a * q, e = fmaf(a, q, -h);
  return h < b || (h == b && e < 0.f);
}

// A lane's share of 32 * kVerUnroll tokens as pieces of four, 128 tokens apart.
__device__ __forceinline__ void take_wide(float (&v)[kVerUnroll], const float* src) {
#pragma unroll
  for (int k = 0; k < kVerUnroll; k += 4) {
    const float4 x = *reinterpret_cast<const float4*>(src + 32 * k);
    v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
  }
}

// (Four blocks an SM: 64 sequences are 512 blocks, which then all run at once; 71
// registers instead of 63 left room for three, 20.7 us.)
template <int CL>
__global__ void __launch_bounds__(kVerThreads, 4) verify_kernel(const VerifyParams a) {
  namespace cg = cooperative_groups;
  __shared__ uint64_t part[kVerWarps];
  __shared__ uint64_t slice[2][CL];  // [round]: the slices' sums
  cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();  // (awaited before the first write to another CTA's memory)
  chain_wait();
  chain_release();
  const int rank = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = a.T, V = a.V;
  // ---- the drafts, by every warp (beside their count, which says how many of them there are)
  const float u_mine = lane < T ? ver_uniform(a.u[(int64_t)b * T + lane]) : 0.f;
  const int x = lane < T - 1 ? a.drafts[(int64_t)b * (T - 1) + lane] : -1;
  int n = T - 1;
  if (a.num) {
    n = a.num[b];
    if (n < 0 || n > T - 1) {
      if (tid == 0 && rank == 0) flag(a.status, NK_DEVFLAG_BAD_POS);
      n = n < 0 ? 0 : T - 1;
    }
  }
  bool good = false;
  if (lane < n) {
    if (x >= 0 && x < V) {
      const float px = a.p[((int64_t)b * T + lane) * a.p_stride + x];
      const float qx = a.q ? a.q[((int64_t)b * (T - 1) + lane) * a.q_stride + x] : 1.f;
      good = ver_accept(u_mine, qx, px);
    } else if (rank == 0 && warp == 0) {
      flag(a.status, NK_DEVFLAG_BAD_TOKEN);
    }
  }
  const int acc = __ffs(~__ballot_sync(0xffffffffu, good)) - 1;  // (n <= 15: a lane is left)
  const bool cut = acc < n;
  const int refused = __shfl_sync(0xffffffffu, x, acc);
  if (rank == 0 && warp == 0) {
    if (lane < acc) a.tokens[(int64_t)b * T + lane] = x;
    else if (lane > acc && lane < T) a.tokens[(int64_t)b * T + lane] = -1;
    if (lane == 0) {
      a.accepted[b] = acc;
      if (a.next) a.next[b] = a.ctx[b] - n + acc;
    }
  }
  // ---- the row
  const float* prow = a.p + ((int64_t)b * T + acc) * a.p_stride;
  const float* qrow = cut && a.q ? a.q + ((int64_t)b * (T - 1) + acc) * a.q_stride : nullptr;
  int hole = cut && !a.q ? refused : -1;  // a certain draft that was refused
  const float uf = __shfl_sync(0xffffffffu, u_mine, T - 1);
  const uint64_t u64 = __float2ull_rz(uf * 18446744073709551616.f);
  // parts of whole rounds: 32 lanes and kVerUnroll tokens each
  const int per = (V + CL * kVerWarps - 1) / (CL * kVerWarps), step = (per + 31) / 32 * 32;
  const auto begin_of = [&](int i) { return (int64_t)i * step < V ? i * step : V; };
  const int lo = begin_of(rank * kVerWarps + warp), hi = begin_of(rank * kVerWarps + warp + 1);
  const auto weight = [&](int i) {  // (i < V)
    const float pv = i == hole ? 0.f : prow[i];
    return ver_weight(pv, qrow ? qrow[i] : 0.f);
  };
  uint64_t total = 0, before = 0;  // of the row; of the slices before this one
  for (int round = 0; round < 2; ++round) {
    const bool holed = hole >= lo && hole < hi;
    // (parts begin at whole 32s: aligned rows have all their pieces of four aligned)
    const bool wide = ((reinterpret_cast<uintptr_t>(prow) | reinterpret_cast<uintptr_t>(qrow)) & 15) == 0;
    uint64_t sum = 0, over = 0;
    int j = lo;  // (warp-uniform)
    for (; j + 32 * kVerUnroll <= hi; j += 32 * kVerUnroll) {
      float pv[kVerUnroll], qv[kVerUnroll];
      if (wide) {
        take_wide(pv, prow + j + 4 * lane);
        if (qrow) take_wide(qv, qrow + j + 4 * lane);
      } else {
#pragma unroll
        for (int k = 0; k < kVerUnroll; ++k) pv[k] = prow[j + 32 * k + lane];
        if (qrow) {
#pragma unroll
          for (int k = 0; k < kVerUnroll; ++k) qv[k] = qrow[j + 32 * k + lane];
        }
      }
      if (!qrow) {
#pragma unroll
        for (int k = 0; k < kVerUnroll; ++k) qv[k] = 0.f;
      }
      if (holed) {
#pragma unroll
        for (int k = 0; k < kVerUnroll; ++k)
          if (j + (wide ? k / 4 * 128 + 4 * lane + k % 4 : 32 * k + lane) == hole) pv[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < kVerUnroll; ++k) {
        // a token adds 2^62 at most, so a sum cannot pass 2^64 without bit 63 set once
        sum += ver_weight(pv[k], qv[k]);
        over |= sum;
      }
    }
    for (int i = j + lane; i < hi; i += 32) {
      sum += weight(i);
      over |= sum;
    }
    if (over >> 63) sum = kVerCap;
    sum = ver_warp_sum(sum);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (round == 0) cluster.barrier_wait(std::move(started));
    if (warp == 0) {
      uint64_t v = lane < kVerWarps ? part[lane] : 0;
      v = ver_warp_sum(v);
      if (lane < CL) *cluster.map_shared_rank(&slice[round][rank], lane) = v;
    }
    cluster.sync();
    total = before = 0;
#pragma unroll
    for (int c = 0; c < CL; ++c) {
      if (c == rank) before = total;
      total = ver_add(total, slice[round][c]);
    }
    // nothing left of p after q: the row itself (the same in every CTA)
    if (total != 0 || !cut || round == 1) break;
    qrow = nullptr;
    hole = -1;
  }
  if (total == 0 || total == kVerCap) {  // no distribution
    if (rank == 0 && tid == 0) {
      a.tokens[(int64_t)b * T + acc] = -1;
      flag(a.status, NK_DEVFLAG_RANGE);
    }
    return;
  }
  // ---- the token: the first whose sum passes u R, so the first above its whole part
  const uint64_t want = __umul64hi(u64, total);
  int w = -1;
  uint64_t run = before;
#pragma unroll
  for (int k = 0; k < kVerWarps; ++k) {
    if (w < 0) {
      if (run + part[k] > want && run <= want) w = k;
      else run += part[k];
    }
  }
  if (w < 0) return;  // another slice's
  // (block-uniform from here) the part's tokens, in runs of whole 32s, one a warp
  const int plo = begin_of(rank * kVerWarps + w), phi = begin_of(rank * kVerWarps + w + 1);
  const int len = (((phi - plo) + kVerWarps - 1) / kVerWarps + 31) / 32 * 32;
  const int a0 = plo + warp * len < phi ? plo + warp * len : phi, a1 = a0 + len < phi ? a0 + len : phi;
  uint64_t sum = 0;
#pragma unroll 8
  for (int i = a0 + lane; i < a1; i += 32) sum += weight(i);
  sum = ver_warp_sum(sum);
  __syncthreads();  // part[] has been read
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  for (int k = 0; k < warp; ++k) run += part[k];
  if (!(run <= want && run + sum > want)) return;
  for (int i0 = a0; i0 < a1; i0 += 32) {  // (warp-uniform)
    const uint64_t v = i0 + lane < a1 ? weight(i0 + lane) : 0;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, run + incl > want);
    if (past) {
      if (lane == 0) a.tokens[(int64_t)b * T + acc] = i0 + __ffs(past) - 1;
      return;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
}

}  // namespace nk

using namespace nk;

extern "C" {

int nk_verify_drafts(const float* target_dev, int64_t target_row_stride, const float* draft_dev,
                     int64_t draft_row_stride, const int32_t* drafts_dev, const int32_t* num_drafts_dev,
                     const float* uniforms_dev, int32_t B, int32_t T, int32_t vocab, const int32_t* ctx_lens_dev,
                     int32_t* tokens_dev, int32_t* accepted_dev, int32_t* next_start_dev, int32_t* status_dev,
                     void* stream) {
  if (B < 0 || T < 1 || T > NK_MAX_T || vocab < 1) return NK_ERR_SHAPE;
  if (target_row_stride < vocab || (draft_dev && T > 1 && draft_row_stride < vocab)) return NK_ERR_SHAPE;
  if (B > 65535 || vocab > (1 << 30)) return NK_ERR_UNSUPPORTED;
  if (B == 0) return NK_OK;
  if (!target_dev || !uniforms_dev || !tokens_dev || !accepted_dev || (T > 1 && !drafts_dev) ||
      (next_start_dev && !ctx_lens_dev))
    return NK_ERR_NULL;
  // all CTAs of a sequence read the inputs while one writes the results
  const uint64_t rows = (uint64_t)B * T, drafted = (uint64_t)B * (T - 1), each = (uint64_t)B * 4;
  const Range results[] = {{tokens_dev, rows * 4}, {accepted_dev, each}, {next_start_dev, next_start_dev ? each : 0}};
  const Range inputs[] = {{target_dev, (uint64_t)vocab * 4, rows, (uint64_t)target_row_stride * 4},
                          {draft_dev, draft_dev && T > 1 ? (uint64_t)vocab * 4 : 0, drafted, (uint64_t)draft_row_stride * 4},
                          {drafts_dev, drafted * 4},
                          {num_drafts_dev, num_drafts_dev ? each : 0},
                          {uniforms_dev, rows * 4},
                          {ctx_lens_dev, next_start_dev ? each : 0}};
  for (const Range& r : results)
    for (const Range& in : inputs)
      if (overlap(r, in) && !(&r == &results[2] && &in == &inputs[5] && r.at == in.at)) return NK_ERR_SHAPE;
  if (overlap(results[0], results[1]) || overlap(results[0], results[2]) || overlap(results[1], results[2])) return NK_ERR_SHAPE;
  const VerifyParams p{target_dev, draft_dev, target_row_stride, draft_row_stride, drafts_dev, num_drafts_dev,
                       uniforms_dev, ctx_lens_dev, T, vocab, tokens_dev, accepted_dev, next_start_dev, status_dev};
  constexpr int CL = 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL, (unsigned)B);
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<CL>, p);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

}  // extern "C"
