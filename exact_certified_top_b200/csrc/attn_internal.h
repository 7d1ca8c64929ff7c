// Internal interfaces of the attention calls: the batch tables the kernels
// take as parameters, and the launches (attn_api.cu validates and plans).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "dosa.h"
#include "dosa_internal.h"

namespace dosa {

struct AttnHandle {
  dosa_attn_config cfg;
  int G;              // query heads per key head
  float scale_log2;   // softmax scale * log2(e)
  bool fp16;
};

constexpr int kVecCodes = kHeadDim / 2;   // bytes of a head vector's 4-bit codes
constexpr int kVecParams = 16;            // bytes of its four (scale, min) pairs

// Sequences travel to the kernels as launch parameters, so a call needs no
// upload and a captured graph keeps its batch; larger batches take several
// launches.  128 entries of 40 bytes stay below the 32,764-byte limit with room.
constexpr int kSeqsPerLaunch = 128;

struct AttnSeq {
  int64_t k0;      // first key slot
  int64_t part0;   // split sequences: first partial vector; else -1
  int q0;          // first query row
  int rows;
  int pos0;        // position of the first row
  int unit0;       // first work unit of the sequence in this launch
  int nsplit;      // parts of the key axis
  int chunk;       // keys per part (attend: a multiple of 16)
};

struct AttnTable {
  int n;           // sequences
  int units;       // work units of the launch
  AttnSeq s[kSeqsPerLaunch];
};

// Sequence that owns unit (or row) `u` among ascending starts.
template <class F>
__host__ __device__ __forceinline__ int find_seq(int n, int u, F start) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start(mid) <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Programmatic dependent launch: a kernel launched with launch_after may start
// while the kernel before it in the stream ends, and waits with grid_wait before
// it touches anything that kernel wrote or reads what it writes.  Saves 1 to 2
// us per kernel.  A call's first kernel (append, read, attend) waits before its
// first access, since the kernel before it may be anyone's; and it lets its
// successor in only after that wait, so kernels further down may read the
// call's inputs (not what the call writes) before their own.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
#ifdef __CUDACC__
// Every thread, before the first access to the previous kernel's results.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's CTAs may be scheduled from here on.
__device__ __forceinline__ void grid_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The fp16 pair w of a and b, with fp16's largest number where a finite one became
// infinite.
__device__ __forceinline__ uint32_t hold_finite(uint32_t w, float a, float b) {
  if ((w & 0x7FFFu) == 0x7C00u && fabsf(a) < INFINITY) w -= 1u;
  if ((w & 0x7FFF0000u) == 0x7C000000u && fabsf(b) < INFINITY) w -= 0x10000u;
  return w;
}
#endif

struct Rows16 {
  uint16_t* ptr;
  int64_t rs, hs;   // row and head stride, elements
};

struct Cache4View {
  uint8_t *kc, *kp, *vc, *vp;
  float* weight;
  int64_t cap;
};

struct EvictSeq {
  int64_t src0, dst0;
  int n, keep;     // tokens, tokens kept (<= n)
  int j0;          // kept tokens of the launch's earlier sequences
  int out;         // row of kept_idx
};
struct EvictTable {
  int n;
  int total;       // kept tokens of the launch
  EvictSeq s[kSeqsPerLaunch];
};

int attn_sm_count();

// Once per kernel and device: allow `bytes` of dynamic shared memory.  done is
// the kernel's own record, one bit per device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* done);

cudaError_t launch_prompt(const AttnHandle& h, const Rows16& q, const Rows16& k, const Rows16& v,
                          int64_t q_rows, int64_t k_rows, const AttnTable& t, const Rows16& out,
                          float* lse, float* part_o, float* part_lse, int* err,
                          cudaStream_t stream);
// Join split sequences: `rows` of the table's split sequences x Hq vectors.  kind:
// the dosa_kernel its time counts for.
cudaError_t launch_join(const AttnHandle& h, int kind, const AttnTable& t, const Rows16& out,
                        float* lse, float* lse2, const float* part_o, const float* part_lse,
                        cudaStream_t stream);
cudaError_t launch_cache_append(const AttnHandle& h, const Cache4View& c, const Rows16& k,
                                const Rows16& v, const AttnTable& t, cudaStream_t stream);
cudaError_t launch_cache_read(const AttnHandle& h, const Cache4View& c, const Rows16& k,
                              const Rows16& v, const AttnTable& t, cudaStream_t stream);
cudaError_t launch_attend(const AttnHandle& h, const Cache4View& c, const Rows16& q,
                          const AttnTable& t, const int32_t* sel, int K, const Rows16& out,
                          float* lse, float* lse2, float* part_o, float* part_lse, float* scores,
                          cudaStream_t stream);
cudaError_t launch_attend_weights(const AttnHandle& h, const Cache4View& c, const Rows16& q,
                                  const AttnTable& t, const float* lse2, cudaStream_t stream);
// The same for a selection, from the scores launch_attend stored.
cudaError_t launch_list_weights(const AttnHandle& h, const AttnTable& t, const int32_t* sel, int K,
                                const float* scores, const float* lse2, float* row_weight,
                                float* weight, cudaStream_t stream);
cudaError_t launch_evict(const AttnHandle& h, const Cache4View& src, const Cache4View& dst,
                         const EvictTable& t, int first, int last, int max_n, int32_t* kept,
                         int64_t kept_ld, cudaStream_t stream);

// Query columns (row, head) one attend unit takes, and its unit counts: over
// all visible keys a sequence's rows x G columns share the units, over a
// selection each row has its own.
int attend_columns(const AttnHandle& h, int rows, bool selected);

}  // namespace dosa
