// Eviction from the 4-bit cache: the tokens to keep, chosen by their recorded
// attention weight, and their move into another cache.
//
// Selection: a cluster of CTAs per sequence.  Each CTA owns a contiguous run
// of the tokens between the protected ends.  Weights map to order-preserving
// 32-bit keys; three digit passes (11, 11 and 10 bits, most significant first)
// find the key of the last token kept.  A pass histograms the CTA's run in
// shared memory; after a cluster barrier every CTA sums the cluster's
// histograms over distributed shared memory for itself (each reads the same
// counts, so all choose the same digit and no result has to travel back).  The
// keys stay in shared memory after the first pass.
// Then each warp counts its run's tokens above and at that key, the counts are
// prefix-summed over the warps and the cluster, and a last pass writes the
// kept indices in order; tokens at the key are taken from the smallest index.
// Integer counts only: the outcome does not depend on timing.
//
// Latency bounds it: barriers and the three dependent passes (23 us for 13
// sequences of 15K to 70K tokens in clusters of 8, 37 % of the issue slots used).
//
// The move is a copy of 16-byte chunks over all SMs, bound by memory: 106,496 kept
// tokens of 8 heads, 136 MB to read and to write, take 52 us.  225 MB are read,
// since a kept token's 64- and 16-byte pieces are fetched with their neighbours;
// the writes stay in L2 in part.
#include <cooperative_groups.h>

#include "attn_internal.h"
#include "dosa_device.cuh"

namespace cg = cooperative_groups;

namespace dosa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
// Keys a CTA keeps in shared memory after the first pass (64 KB); longer runs
// are read again from L2.
constexpr int kKept = 16384;

// Highest bin whose suffix count reaches `need`: *digit, and the count above
// it in *above.  hist: the summed counts, 2 bins per thread.
__device__ __forceinline__ void find_digit(const unsigned* hist, unsigned need, unsigned* scratch,
                                           unsigned* digit, unsigned* above) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int top = kBins - 1 - 2 * threadIdx.x;     // bins top, top - 1
  const unsigned c0 = hist[top], c1 = hist[top - 1];
  unsigned incl = c0 + c1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    unsigned v = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned n = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += n;
    }
    scratch[lane] = v;
  }
  __syncthreads();
  const unsigned excl = incl - c0 - c1 + (warp ? scratch[warp - 1] : 0);
  if (excl < need && need <= excl + c0) {
    *digit = top;
    *above = excl;
  } else if (excl + c0 < need && need <= excl + c0 + c1) {
    *digit = top - 1;
    *above = excl + c0;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictTable t, const float* __restrict__ weight,
                        int first, int last, int32_t* __restrict__ kept, int64_t kept_ld) {
  __shared__ unsigned s_hist[2][kBins];            // the CTA's counts, one buffer per pass parity
  __shared__ unsigned s_sum[kBins];
  __shared__ unsigned s_scratch[kSelWarps];
  __shared__ unsigned s_digit, s_above;
  __shared__ unsigned s_gt[kSelWarps], s_eq[kSelWarps];   // per warp, then exclusive prefixes
  __shared__ unsigned s_tot[2];                    // the CTA's counts above and at the key

  extern __shared__ unsigned s_key[];              // [kKept] the CTA's keys, or unused

  cg::cluster_group cl = cg::this_cluster();
  const int nc = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const EvictSeq e = t.s[blockIdx.x / nc];
  int32_t* out = kept + (int64_t)e.out * kept_ld;
  const int tid = rank * kSelThreads + threadIdx.x, step = nc * kSelThreads;
  for (int64_t i = e.keep + tid; i < kept_ld; i += step) out[i] = -1;
  if (e.keep >= e.n) {                             // the whole cluster takes this branch
    for (int i = tid; i < e.n; i += step) out[i] = i;
    return;
  }
  for (int i = tid; i < first; i += step) out[i] = i;
  for (int i = tid; i < last; i += step) out[e.keep - last + i] = e.n - last + i;
  const int mid = e.n - first - last;              // tokens to choose from
  const int take = e.keep - first - last;          // 0 <= take < mid
  if (take == 0) return;
  const float* w = weight + e.src0 + first;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // runs: a multiple of 32 tokens per warp
  const int run = (mid + nc * kSelWarps * 32 - 1) / (nc * kSelWarps * 32) * 32;
  const int r0 = min(mid, (rank * kSelWarps + warp) * run), r1 = min(mid, r0 + run);
  const bool cached = run * kSelWarps <= kKept;
  unsigned* const mine = s_key + warp * run;       // the warp's run, in order
  auto key_at = [&](int i) { return cached ? mine[i - r0] : ordered_key(__ldg(w + i)); };

  unsigned prefix = 0, need = (unsigned)take;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    unsigned* hist = s_hist[pass & 1];
    for (int b = threadIdx.x; b < kBins; b += kSelThreads) hist[b] = 0;
    __syncthreads();
    if (pass == 0) {
      for (int i0 = r0; i0 < r1; i0 += 128) {      // four loads in flight per lane
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e * 32 + lane;
          x[e] = i < r1 ? __ldg(w + i) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e * 32 + lane;
          if (i >= r1) continue;
          const unsigned u = ordered_key(x[e]);
          if (cached) mine[i - r0] = u;
          atomicAdd(&hist[u >> shift], 1u);
        }
      }
    } else {
      for (int i = r0 + lane; i < r1; i += 32) {
        const unsigned u = key_at(i);
        if ((u >> (shift + bits)) == prefix) atomicAdd(&hist[(u >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    cl.sync();
    for (int b = threadIdx.x; b < kBins; b += kSelThreads) {
      unsigned sum = 0;
      for (int r = 0; r < nc; ++r) sum += cl.map_shared_rank(hist, r)[b];
      s_sum[b] = sum;
    }
    __syncthreads();
    find_digit(s_sum, need, s_scratch, &s_digit, &s_above);
    prefix = (prefix << bits) | s_digit;
    need -= s_above;
    // the buffer of this pass is cleared again two passes later, which the
    // next pass's cluster barrier separates from these remote reads
  }
  // prefix: the key of the last kept token; `need` of the tokens at it stay
  unsigned gt = 0, eq = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    const unsigned u = key_at(i);
    gt += u > prefix;
    eq += u == prefix;
  }
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    unsigned a = s_gt[lane], b = s_eq[lane];
    const unsigned a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xFFFFFFFFu, a, o);
      const unsigned y = __shfl_up_sync(0xFFFFFFFFu, b, o);
      if (lane >= o) {
        a += x;
        b += y;
      }
    }
    s_gt[lane] = a - a0;
    s_eq[lane] = b - b0;
    if (lane == 31) {
      s_tot[0] = a;
      s_tot[1] = b;
    }
  }
  cl.sync();
  unsigned gt0 = s_gt[warp], eq0 = s_eq[warp];
  for (int r = 0; r < rank; ++r) {
    const unsigned* tot = cl.map_shared_rank(s_tot, r);
    gt0 += tot[0];
    eq0 += tot[1];
  }
  // kept before an index = above-key tokens before it + min(at-key before it, need)
  for (int i = r0 + lane; i - lane < r1; i += 32) {
    const unsigned u = i < r1 ? key_at(i) : 0;
    const bool g = i < r1 && u > prefix, q = i < r1 && u == prefix;
    const unsigned bg = __ballot_sync(0xFFFFFFFFu, g), bq = __ballot_sync(0xFFFFFFFFu, q);
    const unsigned below = (1u << lane) - 1u;
    const unsigned ng = gt0 + __popc(bg & below), nq = eq0 + __popc(bq & below);
    if (g || (q && nq < need)) out[first + ng + min(nq, need)] = first + i;
    gt0 += __popc(bg);
    eq0 += __popc(bq);
  }
  cl.sync();                                       // s_tot is read by the others until here
}

constexpr int kMoveThreads = 256;

// Copy: one 16-byte chunk per thread and array.  Chunk order: token fastest
// within a head for the parameters, token x 4 chunks for the codes, so stores
// are contiguous and loads nearly so (kept tokens ascend).
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictTable t, Cache4View src, Cache4View dst,
                      const int32_t* kept, int64_t kept_ld) {
  const int head = blockIdx.y;
  const int g = blockIdx.x * kMoveThreads + threadIdx.x;
  const int tok = g >> 2, part = g & 3;
  if (tok >= t.total) return;
  const int i = find_seq(t.n, tok, [&](int m) { return t.s[m].j0; });
  const EvictSeq& e = t.s[i];
  const int j = tok - e.j0;
  grid_wait();
  const int64_t from = e.src0 + kept[(int64_t)e.out * kept_ld + j], to = e.dst0 + j;
  const int64_t hs = (int64_t)head * src.cap + from, hd = (int64_t)head * dst.cap + to;
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(src.kc + hs * kVecCodes) + part);
  const uint4 b = __ldg(reinterpret_cast<const uint4*>(src.vc + hs * kVecCodes) + part);
  uint4 p;
  if (part < 2) p = __ldg(reinterpret_cast<const uint4*>((part ? src.vp : src.kp) + hs * kVecParams));
  reinterpret_cast<uint4*>(dst.kc + hd * kVecCodes)[part] = a;
  reinterpret_cast<uint4*>(dst.vc + hd * kVecCodes)[part] = b;
  if (part < 2) *reinterpret_cast<uint4*>((part ? dst.vp : dst.kp) + hd * kVecParams) = p;
  if (head == 0 && part == 2 && dst.weight) dst.weight[to] = __ldg(src.weight + from);
}

}  // namespace

cudaError_t launch_evict(const AttnHandle& h, const Cache4View& src, const Cache4View& dst,
                         const EvictTable& t, int first, int last, int max_n, int32_t* kept,
                         int64_t kept_ld, cudaStream_t stream) {
  if (t.n <= 0) return cudaSuccess;
  // A CTA that holds all of a sequence's keys in shared memory needs nobody to
  // agree with: selection and move of half of 1,056 / 4,096 / 16,384 tokens (8
  // heads) take 11 / 13 / 21 us with one CTA per sequence and 17 / 17 / 19 with
  // eight, and 16 / 46 / 151 against 49 / 80 / 178 for 32 such sequences; 70,001
  // tokens take 99 and 36.
  const int nc = max_n <= kKept ? 1 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(t.n * nc));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kKept * 4;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = nc;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(evict_select_kernel), kKept * 4, &done);
  if (e != cudaSuccess) return e;
  profile_before(DOSA_KERNEL_EVICT, stream);
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, t, (const float*)src.weight, first, last, kept,
                         kept_ld);
  profile_after(DOSA_KERNEL_EVICT, stream);
  if (e != cudaSuccess || t.total == 0) return e;
  const dim3 grid((unsigned)(((int64_t)t.total * 4 + kMoveThreads - 1) / kMoveThreads),
                  (unsigned)h.cfg.Hkv);
  profile_before(DOSA_KERNEL_EVICT, stream);
  e = launch_after(evict_move_kernel, grid, kMoveThreads, 0, stream, t, src, dst,
                   (const int32_t*)kept, kept_ld);
  profile_after(DOSA_KERNEL_EVICT, stream);
  return e;
}

}  // namespace dosa
