// Attention of a few query rows per sequence over the 4-bit cache.
//
// A unit is (sequence, up to 8 NT query columns, key head, part of the key
// axis); a column is a (row, head) pair of the key head's group.  Each of the
// CTA's 8 warps walks its own 16-token slices with a private ring of cp.async
// stages and its own running softmax, and the warps join at the end.
//
// Products run on m16n8k16 matrix instructions with the 4-bit codes as fp16
// operands straight out of the packed words: a nibble in an fp16's low bits
// is the subnormal number code * 2^-24 (and code * 2^-20 one nibble higher),
// exact, for one AND per two codes.  The scales stay out of the operands:
//   x(t,h) = sum_g s(t,g) (sum_{i in g} c(t,i) q(h,i)) + sum_g m(t,g) (sum_{i in g} q(h,i))
// with the group sums from the matrix unit (fp32), s applied in fp32 and the m
// term a product of the parameters with the query's group sums (split into
// two fp16 parts).  q is scaled by a power of two per column so that fp16
// holds bf16's bits.  For the values the scale goes to the other operand:
//   out(h,i) = sum_t (p(t,h) s(t,g)) c(t,i) + sum_t p(t,h) m(t,g)
// p is rounded to fp16 for the second sum and p s, formed in fp32, for the first:
// 2^-11 each.  p is kept 2^kLift times larger and the scales of each group by a
// power of two per warp that brings the largest below 1, so that weights keep their
// bits down to 2^-26 of the row's largest (thousands of such keys may carry a row
// whose largest weight meets a small value) and groups of any size theirs; what
// is lost below is half a step of 2^-24, at most 2^-37 of the largest weight per
// key times |min|, and 2^-36 times 15 of the group's largest scale.  Running maxima
// move only when a score exceeds them by 2^kSlack, so most slices need no
// rescaling.
//
// Bound: issue and memory together up to 8 columns (390 warp instructions per
// slice of 16 tokens; one row of 64 heads over 1M keys takes 284 us with 72 % of
// the issue slots used, 207 for the bytes), the latency of dependent products
// beyond (850 instructions per slice at 32 columns, where registers leave 2
// warps per scheduler: 4 rows 773 us).  Weight times scale in fp32 costs 32 of the
// 390 instructions: a product in fp16 took 267 us, but lost the bits of groups
// and keys beside larger ones.  Columns per unit: 8 with two CTAs per SM, else 16
// or 32 with one.  With that product, for 2 rows over 1M keys 16 columns took 375
// us with 8 warps and 255 registers (388 now), 395 with 12 warps and 168, 530 with
// two CTAs and 128; for 4 rows two units of 16 columns took 1,045 against 757.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "attn_internal.h"
#include "dosa_device.cuh"

namespace dosa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSlice = 16;                        // tokens per warp step
constexpr int kStageBytes = kSlice * 2 * (kVecCodes + kVecParams);   // 2560
constexpr int kStages = 4;
constexpr int kOffV = kSlice * kVecCodes;         // key codes, value codes, key params, value params
constexpr int kOffKp = 2 * kSlice * kVecCodes;
constexpr int kOffVp = kOffKp + kSlice * kVecParams;
constexpr float kSlack = 3.f;                     // log2 units a score may exceed the running maximum
constexpr float kLift = 12.f;                     // weights are kept 2^kLift times larger, up to
                                                  // 2^(kLift + kSlack) = 2^15: `top` is the maximum
                                                  // minus kLift
constexpr float kNegInf = -INFINITY;
// Running maximum of a column that has seen nothing: finite, so that a score of
// -infinity minus it is -infinity and not NaN.
constexpr float kNone = -3.402823466e38f;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma16816_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t movm(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void ldsm2t(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) {
  return *reinterpret_cast<const __half2*>(&w);
}
__device__ __forceinline__ uint32_t as_word(__half2 h) {
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float half_lo(uint32_t w) {
  return __low2float(*reinterpret_cast<const __half2*>(&w));
}

// Two fp32 products per instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

// 1 / x of a power of two.
__device__ __forceinline__ float pow2_inverse(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}
// The scales of two (scale, min) words.
__device__ __forceinline__ __half2 scales(uint32_t a, uint32_t b) {
  return as_half2(__byte_perm(a, b, 0x5410));
}

// Both halves that are not finite replaced by zero.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  const __half2 h = *reinterpret_cast<const __half2*>(&w);
  const __half2 z = __hsub2(h, h);                 // 0, or NaN
  return w & __heq2_mask(z, z);
}

// Shared-memory row of a stage's token, and the 16-byte chunk swizzle of a
// row: the value loads take rows 0, 2, 4, 6 (and 1, 3, 5, 7) at once, so every
// second pair of rows is swapped and rows 4-7 of each 8 exchange chunk halves;
// all 32 banks are then used once per wavefront.
__device__ __forceinline__ int stage_row(int tok) { return tok ^ ((tok >> 1) & 1); }
__device__ __forceinline__ int stage_chunk(int row, int chunk) {
  return chunk ^ (((row >> 2) & 1) << 1);
}

struct AttendParams {
  Cache4View c;
  Rows16 q, out;
  const int32_t* sel;
  int K;
  int Hq, Hkv, G;
  float scale_log2;
  float* lse;       // [Tq, Hq] natural log, or null
  float* lse2;      // [Tq, Hq] log2, or null (kept for the weights)
  float* part_o;    // split sequences: [part vector][128]
  float* part_lse;  // [part vector], log2
  float* scores;    // selection with weights: [row of the launch][K][Hq] log2 scores, or null
};

// The unit's geometry.
struct Unit {
  int head;             // key head
  int row0, nrow;       // rows of the sequence the columns come from
  int col0, ncol;       // columns col0.. of those rows x G
  int part;
  int lo, hi;           // key positions (or list entries) of this part
  int limit0;           // keys visible to the sequence's row 0 (minus row offset)
  const int32_t* list;  // selection of the row, or null
};

template <int NT>
__device__ __forceinline__ Unit unit_of(const AttendParams& p, const AttnSeq& s, int u) {
  Unit x;
  constexpr int NC = 8 * NT;
  const bool selected = p.sel != nullptr;
  x.head = u % p.Hkv;
  u /= p.Hkv;
  const int cols = selected ? p.G : s.rows * p.G;
  const int groups = (cols + NC - 1) / NC;
  const int grp = u % groups;
  u /= groups;
  x.part = u % s.nsplit;
  u /= s.nsplit;
  x.row0 = selected ? u : 0;
  x.nrow = selected ? 1 : s.rows;
  x.col0 = grp * NC;
  x.ncol = min(NC, cols - x.col0);
  int len;
  if (selected) {
    x.list = p.sel + (int64_t)(s.q0 + x.row0) * p.K;
    len = p.K;
  } else {
    x.list = nullptr;
    // the last row among this unit's columns sees the most keys
    len = s.pos0 + (x.col0 + x.ncol - 1) / p.G + 1;
  }
  x.limit0 = s.pos0 + x.row0 + 1;
  x.lo = min(len, x.part * s.chunk);
  x.hi = min(len, x.lo + s.chunk);
  return x;
}

// Query operands of the unit's columns (one column per lane group n = lane /
// 4): fp16 words in the order of the unpacked key words, the group sums, and
// the power of two they were scaled by.
// More than 8 columns: the words b lie in shared memory ([tile][group][lane]),
// where registers would leave room for half the warps.
template <int NT>
struct QueryFrags {
  uint4 b[1][4];          // group; words for nibbles (0,4), (1,5)/16, (2,6), (3,7)/16
  uint32_t at;            // the shared memory copy, NT > 1
  uint32_t sum[NT][2];    // (0, sum of group c) high and low fp16 parts
  float back[NT][2];      // columns 2c, 2c + 1: scale * log2(e) * 2^-e
};

template <int NT, bool kFp16>
__device__ __forceinline__ void load_query(const AttendParams& p, const AttnSeq& s, const Unit& x,
                                           QueryFrags<NT>& f) {
  const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int col = x.col0 + t * 8 + n;
    float q[4][8];
    float top = 0.f;
    const bool on = t * 8 + n < x.ncol;
    const int row = s.q0 + x.row0 + (on ? col / p.G : 0), head = x.head * p.G + (on ? col % p.G : 0);
    const uint16_t* src = p.q.ptr + (int64_t)row * p.q.rs + (int64_t)head * p.q.hs;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (on) u = __ldg(reinterpret_cast<const uint4*>(src + 32 * g + 8 * c));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 v;
        if constexpr (kFp16) {
          v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        } else {
          v.x = __uint_as_float(w[i] << 16);
          v.y = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        q[g][2 * i] = v.x;
        q[g][2 * i + 1] = v.y;
        top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // 2^e brings the column's largest element into [2^9, 2^10); zero or
    // infinite columns stay as they are.  e is held to +-120 so that both
    // factors are normal numbers.
    int e = 0;
    if (top > 0.f && top < INFINITY) {
      e = 136 - (int)(__float_as_uint(top) >> 23);
      e = max(-120, min(120, e));
    }
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    // scores: codes carry 2^-24
    const float back = p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
    f.back[t][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * c);
    f.back[t][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * c + 4);
    float gs[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q[g][j] *= up;
        sum += q[g][j];
      }
      const uint4 words = make_uint4(pack_half(q[g][0], q[g][4]),
                                     pack_half(q[g][1] * 0.0625f, q[g][5] * 0.0625f),
                                     pack_half(q[g][2], q[g][6]),
                                     pack_half(q[g][3] * 0.0625f, q[g][7] * 0.0625f));
      if constexpr (NT == 1) f.b[0][g] = words;
      else sts128(f.at + ((t * 4 + g) * 32 + lane) * 16, words);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      gs[g] = sum;
    }
    // operand rows are (scale, min) words: group c of the lane; the scale's
    // factor is zero
    const float mine = c == 0 ? gs[0] : c == 1 ? gs[1] : c == 2 ? gs[2] : gs[3];
    const float hi = __half2float(__float2half_rn(mine));
    f.sum[t][0] = pack_half(0.f, mine);
    f.sum[t][1] = pack_half(0.f, mine - hi);
  }
}

// Issue the copies of one slice (tokens first..first + 15 of the part).
__device__ __forceinline__ void issue_slice(const AttendParams& p, const Unit& x, int64_t k0,
                                            int first, uint32_t stage) {
  const int lane = threadIdx.x & 31;
  // the slot of token (lane & 15)
  int tok = first + (lane & 15);
  int64_t slot = -1;
  if (tok < x.hi) {
    if (x.list) {
      const int i = __ldg(x.list + tok);
      if (i >= 0 && i < x.limit0) slot = k0 + i;
    } else {
      slot = k0 + tok;
    }
  }
  const int64_t hbase = (int64_t)x.head * p.c.cap;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = k * 8 + (lane >> 2), ch = lane & 3;
    const int64_t sl = __shfl_sync(0xFFFFFFFFu, slot, t);
    const bool ok = sl >= 0;
    const int64_t off = (hbase + (ok ? sl : 0)) * kVecCodes + ch * 16;
    const int r = stage_row(t);
    const uint32_t d = stage + r * kVecCodes + stage_chunk(r, ch) * 16;
    cp16(d, p.c.kc + off, ok);
    cp16(d + kOffV, p.c.vc + off, ok);
  }
  {
    const int t = lane & 15;
    const bool ok = slot >= 0;
    const int64_t off = (hbase + (ok ? slot : 0)) * kVecParams;
    if (lane < 16)
      cp16(stage + kOffKp + t * 16, p.c.kp + off, ok);
    else
      cp16(stage + kOffVp + t * 16, p.c.vp + off, ok);
  }
  cp_commit();
}

// The copies of consecutive slices of a contiguous part: the lane's addresses
// advance by a constant, and only the part's last slice is checked.
template <bool kValues, int kKp = kOffKp>
struct SliceWalk {
  const uint8_t *k, *v, *par;
  int left;                       // tokens of the part from the next slice on
  uint32_t d0, d1, dp;            // places in a stage
  __device__ __forceinline__ SliceWalk(const AttendParams& p, const Unit& x, int64_t k0, int first) {
    const int lane = threadIdx.x & 31, t = lane >> 2, ch = lane & 3;
    const int64_t slot = (int64_t)x.head * p.c.cap + k0 + first;
    k = p.c.kc + (slot + t) * kVecCodes + ch * 16;
    v = p.c.vc + (slot + t) * kVecCodes + ch * 16;
    par = (lane < 16 ? p.c.kp : p.c.vp) + (slot + (lane & 15)) * kVecParams;
    left = x.hi - first;
    const int r0 = stage_row(t), r1 = stage_row(t + 8);
    d0 = r0 * kVecCodes + stage_chunk(r0, ch) * 16;
    d1 = r1 * kVecCodes + stage_chunk(r1, ch) * 16;
    dp = (lane < 16 ? kKp : kOffVp) + (lane & 15) * 16;
  }
  // the next slice into `stage`; `step` slices ahead is the one after it
  __device__ __forceinline__ void issue(uint32_t stage, int step) {
    const int lane = threadIdx.x & 31;
    if (left >= kSlice) {
      cp16(stage + d0, k);
      cp16(stage + d1, k + 8 * kVecCodes);
      if constexpr (kValues) {
        cp16(stage + d0 + kOffV, v);
        cp16(stage + d1 + kOffV, v + 8 * kVecCodes);
      }
      if (kValues || lane < 16) cp16(stage + dp, par);
    } else if (left > 0) {
      const int t = lane >> 2;
      // tokens behind the part: zeros, from an address that is not read
      cp16(stage + d0, t < left ? k : p0(k), t < left);
      cp16(stage + d1, t + 8 < left ? k + 8 * kVecCodes : p0(k), t + 8 < left);
      if constexpr (kValues) {
        cp16(stage + d0 + kOffV, t < left ? v : p0(v), t < left);
        cp16(stage + d1 + kOffV, t + 8 < left ? v + 8 * kVecCodes : p0(v), t + 8 < left);
      }
      const bool ok = (lane & 15) < left;
      if (kValues || lane < 16) cp16(stage + dp, ok ? par : p0(par), ok);
    }
    cp_commit();
    k += (int64_t)step * kSlice * kVecCodes;
    v += (int64_t)step * kSlice * kVecCodes;
    par += (int64_t)step * kSlice * kVecParams;
    left -= step * kSlice;
  }
  // a pointer of the same array that is always in range: the lane's, pulled back
  // to the slice's first token
  __device__ __forceinline__ const uint8_t* p0(const uint8_t* at) const {
    const int lane = threadIdx.x & 31;
    return at == par ? par - (lane & 15) * kVecParams
                     : at - (lane >> 2) * kVecCodes;
  }
};

// Scores of one slice in log2 units, without the mask: x[t][0..1] token r,
// columns 2c, 2c + 1; x[t][2..3] token r + 8 (r = lane / 4, c = lane % 4).
// kKp: where the key parameters lie in the stage.  kScaled: false leaves the
// factor `back` to the caller.
template <int NT, int kKp = kOffKp, bool kScaled = true>
__device__ __forceinline__ void slice_scores(const QueryFrags<NT>& f, uint32_t stage,
                                             float (&x)[NT][4]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int ra = stage_row(r), rb = stage_row(r + 8);
  const uint4 wa = lds128(stage + ra * kVecCodes + stage_chunk(ra, c) * 16);
  const uint4 wb = lds128(stage + rb * kVecCodes + stage_chunk(rb, c) * 16);
  const uint4 pa = lds128(stage + kKp + r * 16), pb = lds128(stage + kKp + (r + 8) * 16);
  const uint32_t ma = lds32(stage + kKp + r * 16 + c * 4);
  const uint32_t mb = lds32(stage + kKp + (r + 8) * 16 + c * 4);
  const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
  const uint32_t sa[4] = {pa.x, pa.y, pa.z, pa.w}, sb[4] = {pb.x, pb.y, pb.z, pb.w};
  float tot[NT][4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t a8 = a[g] >> 8, b8 = b[g] >> 8;
    const float fa = half_lo(sa[g]), fb = half_lo(sb[g]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint4 q;
      if constexpr (NT == 1) q = f.b[0][g];
      else q = lds128(f.at + ((t * 4 + g) * 32 + lane) * 16);
      float d[4];
      mma16816_0(d, a[g] & 0x000F000Fu, b[g] & 0x000F000Fu, a[g] & 0x00F000F0u,
                 b[g] & 0x00F000F0u, q.x, q.y);
      mma16816(d, a8 & 0x000F000Fu, b8 & 0x000F000Fu, a8 & 0x00F000F0u, b8 & 0x00F000F0u, q.z, q.w);
      tot[t][0] = g ? fmaf(d[0], fa, tot[t][0]) : d[0] * fa;
      tot[t][1] = g ? fmaf(d[1], fa, tot[t][1]) : d[1] * fa;
      tot[t][2] = g ? fmaf(d[2], fb, tot[t][2]) : d[2] * fb;
      tot[t][3] = g ? fmaf(d[3], fb, tot[t][3]) : d[3] * fb;
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float d[4];
    mma16816_0(d, ma, mb, ma, mb, f.sum[t][0], f.sum[t][1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = fmaf(tot[t][i], 16777216.f, d[i]);
      x[t][i] = kScaled ? y * f.back[t][i & 1] : y;
    }
  }
}

// Visible? Token `tok` of the part for column `col` of the unit.
__device__ __forceinline__ bool column_sees(const AttendParams& p, const Unit& x, int tok, int idx,
                                            int col) {
  if (tok >= x.hi) return false;
  if (x.list) return idx >= 0 && idx < x.limit0;
  return tok < x.limit0 + (x.col0 + col) / p.G;
}

template <int NT>
__host__ __device__ constexpr int query_smem() { return NT > 1 ? NT * 4 * 32 * 16 : 0; }
template <int NT>
constexpr int attend_smem() {
  const int ring = kWarps * kStages * kStageBytes + query_smem<NT>();
  const int join = kWarps * 8 * NT * (kHeadDim + 2) * 4;
  return ring > join ? ring : join;
}

template <int NT, bool kFp16, bool kSel>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1)
    attend_kernel(const __grid_constant__ AttnTable t, const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int NC = 8 * NT;
  const int si = find_seq(t.n, blockIdx.x, [&](int m) { return t.s[m].unit0; });
  const AttnSeq& s = t.s[si];
  const Unit x = unit_of<NT>(p, s, blockIdx.x - s.unit0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
  const int n_slices = (x.hi - x.lo + kSlice - 1) / kSlice;
  grid_wait();

  // the warp takes slices warp, warp + 8, ...; stages fill ahead
  SliceWalk<true> walk(p, x, s.k0, x.lo + warp * kSlice);
  auto fill = [&](int sl, uint32_t stage) {
    if constexpr (!kSel) walk.issue(stage, kWarps);
    else if (sl < n_slices) issue_slice(p, x, s.k0, x.lo + sl * kSlice, stage);
    else cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - (NT <= 2 ? 2 : 1); ++i) fill(warp + i * kWarps, ring + i * kStageBytes);
  QueryFrags<NT> f;
  // every warp writes the same words of the same columns
  f.at = smem_u32(smem) + kWarps * kStages * kStageBytes;
  load_query<NT, kFp16>(p, s, x, f);
  if constexpr (NT > 1) __syncthreads();

  float o[NT][8][4];                 // [value operand tile][frag]: dims x columns
  float om[NT][4];                   // rows 2g + 1: sum p m of group g
  float top[NT][2], sum[NT][2];      // running maximum (log2 units) and sum per column
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) om[n][j] = 0.f;
    top[n][0] = top[n][1] = kNone;
    sum[n][0] = sum[n][1] = 0.f;
  }
  // Value scales enter as s fs, fs a power of two per group of dimensions that
  // brings the largest seen so far below 1; fs_lim (two groups per word) is the
  // scale above which it has to move.
  float fs[4] = {1.f, 1.f, 1.f, 1.f};
  __half2 fs_lim[2] = {__float2half2_rn(0.f), __float2half2_rn(0.f)};

  // Two slices per step (one for 32 columns, where registers are short): their
  // loads, products and checks interleave.
  constexpr int kPair = NT <= 2 ? 2 : 1;
  int st = 0;
  for (int sl = warp; sl < n_slices; sl += kPair * kWarps) {
    cp_wait<kStages - 2 * kPair>();
    __syncwarp();
    uint32_t stage[kPair];
#pragma unroll
    for (int e = 0; e < kPair; ++e) stage[e] = ring + (st + e) * kStageBytes;
#pragma unroll
    for (int e = 0; e < kPair; ++e)
      fill(sl + (kStages - kPair + e) * kWarps,
           ring + ((st + kStages - kPair) % kStages + e) * kStageBytes);
    st = st + kPair == kStages ? 0 : st + kPair;

    // slices every column sees whole need no mask
    const int last = x.lo + (sl + (kPair - 1) * kWarps + 1) * kSlice;
    const bool whole = !kSel && last <= x.hi && last <= x.limit0 + x.col0 / p.G;
    float sc[kPair][NT][4];
    uint32_t seen[kPair][NT][2];      // halves of ones where a column sees token r, r + 8
    uint4 pa[kPair], pb[kPair];       // value parameters of tokens r, r + 8
    __half2 vs[2] = {__float2half2_rn(0.f), __float2half2_rn(0.f)};   // largest value scales
    bool grow = false;
#pragma unroll
    for (int e = 0; e < kPair; ++e) {
      slice_scores<NT>(f, stage[e], sc[e]);
      if (!whole) {
        const int tok = x.lo + (sl + e * kWarps) * kSlice + r;
        int ia = 0, ib = 0;
        if (kSel) {
          ia = tok < x.hi ? __ldg(x.list + tok) : -1;
          ib = tok + 8 < x.hi ? __ldg(x.list + tok + 8) : -1;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool v0 = column_sees(p, x, tok + 8 * h, h ? ib : ia, n * 8 + 2 * c);
            const bool v1 = column_sees(p, x, tok + 8 * h, h ? ib : ia, n * 8 + 2 * c + 1);
            seen[e][n][h] = (v0 ? 0xFFFFu : 0u) | (v1 ? 0xFFFF0000u : 0u);
            if (!v0) sc[e][n][2 * h] = kNegInf;
            if (!v1) sc[e][n][2 * h + 1] = kNegInf;
          }
        if constexpr (kSel) {
          if (p.scores) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (tok + 8 * h >= x.hi) continue;
              float* d = p.scores + ((int64_t)(s.q0 - t.s[0].q0 + x.row0) * p.K + tok + 8 * h) * p.Hq +
                         x.head * p.G + x.col0 + 2 * c;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (n * 8 + 2 * c + i < x.ncol) d[n * 8 + i] = sc[e][n][2 * h + i];
            }
          }
        }
      }
      pa[e] = lds128(stage[e] + kOffVp + r * 16);
      pb[e] = lds128(stage[e] + kOffVp + (r + 8) * 16);
      // a slice behind the last: its stage holds anything
      if (e > 0 && sl + e * kWarps >= n_slices) pa[e] = pb[e] = make_uint4(0, 0, 0, 0);
      vs[0] = __hmax2(vs[0], __hmax2(scales(pa[e].x, pa[e].y), scales(pb[e].x, pb[e].y)));
      vs[1] = __hmax2(vs[1], __hmax2(scales(pa[e].z, pa[e].w), scales(pb[e].z, pb[e].w)));
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          grow |= fmaxf(sc[e][n][i], sc[e][n][i + 2]) > top[n][i] + (kLift + kSlack);
    }
    grow |= (__hgt2_mask(vs[0], fs_lim[0]) | __hgt2_mask(vs[1], fs_lim[1])) != 0;
    if (__any_sync(0xFFFFFFFFu, grow)) {
      // new maxima, shared by the 8 lanes of a column; and the value scales'
      float adj[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (an infinite scale must not hide the finite ones beside it)
        __half2 m = __float2half2_rn(0.f);
#pragma unroll
        for (int e = 0; e < kPair; ++e) {
          m = __hmax2(m, as_half2(finite_only(as_word(
                             i ? scales(pa[e].z, pa[e].w) : scales(pa[e].x, pa[e].y)))));
          m = __hmax2(m, as_half2(finite_only(as_word(
                             i ? scales(pb[e].z, pb[e].w) : scales(pb[e].x, pb[e].y)))));
        }
#pragma unroll
        for (int o2 = 1; o2 < 32; o2 <<= 1)
          m = __hmax2(m, as_half2(__shfl_xor_sync(0xFFFFFFFFu, as_word(m), o2)));
        const float2 top2 = __half22float2(m), lim2 = __half22float2(fs_lim[i]);
        float lim[2] = {lim2.x, lim2.y};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float v = h ? top2.y : top2.x;
          if (v > lim[h]) {
            // v fs in [1/2, 1); v is an fp16 number, so fs is 2^-16 .. 2^23
            const uint32_t e = __float_as_uint(v) >> 23;
            const float nf = __uint_as_float((253u - e) << 23);
            adj[2 * i + h] = nf * pow2_inverse(fs[2 * i + h]);
            fs[2 * i + h] = nf;
            lim[h] = __uint_as_float((e + 1u) << 23);   // (2^16 becomes infinity)
          }
        }
        fs_lim[i] = __floats2half2_rn(lim[0], lim[1]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float k[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = fmaxf(sc[0][n][i], sc[0][n][i + 2]);
          if constexpr (kPair > 1) m = fmaxf(m, fmaxf(sc[kPair - 1][n][i], sc[kPair - 1][n][i + 2]));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
          m = fmaxf(top[n][i], m - kLift);
          k[i] = ex2(top[n][i] - m);
          top[n][i] = m;
          sum[n][i] *= k[i];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) om[n][j] *= k[j & 1];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][i][j] *= k[j & 1] * adj[i >> 1];
      }
    }
    // value words: tokens 2c, 2c + 1 and 2c + 8, 2c + 9, nibbles 16 r ..
    const int t0 = 2 * c, t1 = 2 * c + 1;
    const int r0 = stage_row(t0), r1 = stage_row(t1), r2 = stage_row(t0 + 8),
              r3 = stage_row(t1 + 8);
#pragma unroll
    for (int e = 0; e < kPair; ++e) {
      const uint32_t vb = stage[e] + kOffV + (r & 1) * 8;
      const uint2 v0 = lds64(vb + r0 * kVecCodes + stage_chunk(r0, r >> 1) * 16);
      const uint2 v1 = lds64(vb + r1 * kVecCodes + stage_chunk(r1, r >> 1) * 16);
      const uint2 v2 = lds64(vb + r2 * kVecCodes + stage_chunk(r2, r >> 1) * 16);
      const uint2 v3 = lds64(vb + r3 * kVecCodes + stage_chunk(r3, r >> 1) * 16);
      uint32_t m0, m1;
      ldsm2t(stage[e] + kOffVp + (lane & 15) * 16, m0, m1);
      __half2 pr[NT][2];              // p of token r, r + 8; columns 2c, 2c + 1
      float2 pf[NT][2];               // the same in fp32
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float p0 = ex2(sc[e][n][0] - top[n][0]), p1 = ex2(sc[e][n][1] - top[n][1]);
        const float p2 = ex2(sc[e][n][2] - top[n][0]), p3 = ex2(sc[e][n][3] - top[n][1]);
        sum[n][0] += p0 + p2;
        sum[n][1] += p1 + p3;
        pr[n][0] = __floats2half2_rn(p0, p1);
        pr[n][1] = __floats2half2_rn(p2, p3);
        pf[n][0] = make_float2(p0, p1);
        pf[n][1] = make_float2(p2, p3);
      }
      const uint32_t ha[4] = {pa[e].x, pa[e].y, pa[e].z, pa[e].w};
      const uint32_t hb[4] = {pb[e].x, pb[e].y, pb[e].z, pb[e].w};
      if (!whole) {
        // A column that does not see a token has weight 0 for it, and 0 times a
        // parameter that is not a number would not be 0: such minima leave the
        // matrix product and reach the columns that do see the token through
        // its scale (whose products are selected, not multiplied, by visibility).
        m0 = finite_only(m0);
        m1 = finite_only(m1);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
        mma16816(om[n], m0, 0u, m1, 0u, movm(as_word(pr[n][0])), movm(as_word(pr[n][1])));
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t ca = __byte_perm(g < 2 ? v0.x : v0.y, g < 2 ? v1.x : v1.y,
                                        (g & 1) ? 0x7632 : 0x5410);
        const uint32_t cb = __byte_perm(g < 2 ? v2.x : v2.y, g < 2 ? v3.x : v3.y,
                                        (g & 1) ? 0x7632 : 0x5410);
        const uint32_t ca8 = ca >> 8, cb8 = cb >> 8;
        float sa = half_lo(ha[g]) * fs[g], sb = half_lo(hb[g]) * fs[g];
        if (!whole) {
          sa = fmaf(__high2float(as_half2(ha[g])), 0.f, sa);
          sb = fmaf(__high2float(as_half2(hb[g])), 0.f, sb);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 fa = mul2(pf[n][0], make_float2(sa, sa));
          const float2 fb = mul2(pf[n][1], make_float2(sb, sb));
          uint32_t wa = pack_half(fa.x, fa.y), wb = pack_half(fb.x, fb.y);
          if (!whole) {
            wa &= seen[e][n][0];
            wb &= seen[e][n][1];
          }
          const uint32_t b0 = movm(wa), b1 = movm(wb);
          mma16816(o[n][2 * g], ca & 0x000F000Fu, ca8 & 0x000F000Fu, cb & 0x000F000Fu,
                   cb8 & 0x000F000Fu, b0, b1);
          mma16816(o[n][2 * g + 1], ca & 0x00F000F0u, ca8 & 0x00F000F0u, cb & 0x00F000F0u,
                   cb8 & 0x00F000F0u, b0, b1);
        }
      }
    }
  }
  cp_wait<0>();
  grid_release();

  // the warp's result: out = o 2^24 / fs (tile 1 of a group / 16) + om
  __syncthreads();                                 // the rings are free
  float* jo = reinterpret_cast<float*>(smem);      // [warp][column][128]
  float* jt = jo + kWarps * NC * kHeadDim;         // [warp][column] maximum
  float* js = jt + kWarps * NC;                    // [warp][column] sum
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[n][i] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][i], 4);
      sum[n][i] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][i], 8);
      sum[n][i] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][i], 16);
    }
    if (r == 0) {
      const int col = warp * NC + n * 8 + 2 * c;
      jt[col] = top[n][0];
      jt[col + 1] = top[n][1];
      js[col] = sum[n][0];
      js[col + 1] = sum[n][1];
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      // sum p m of group g sits in row 2g + 1, i.e. in lanes 4 (2g + 1) + c
      const float a0 = __shfl_sync(0xFFFFFFFFu, om[n][0], 4 * (2 * g + 1) + c);
      const float a1 = __shfl_sync(0xFFFFFFFFu, om[n][1], 4 * (2 * g + 1) + c);
      const float b = 16777216.f * pow2_inverse(fs[g]);
      float* d0 = jo + (warp * NC + n * 8 + 2 * c) * kHeadDim + 32 * g + 4 * r;
      float* d1 = d0 + kHeadDim;
      const float* e0 = o[n][2 * g];
      const float* e1 = o[n][2 * g + 1];
      *reinterpret_cast<float4*>(d0) =
          make_float4(fmaf(e0[0], b, a0), fmaf(e1[0], b * 0.0625f, a0), fmaf(e0[2], b, a0),
                      fmaf(e1[2], b * 0.0625f, a0));
      *reinterpret_cast<float4*>(d1) =
          make_float4(fmaf(e0[1], b, a1), fmaf(e1[1], b * 0.0625f, a1), fmaf(e0[3], b, a1),
                      fmaf(e1[3], b * 0.0625f, a1));
    }
  }
  __syncthreads();
  // join the warps: each warp takes columns warp, warp + 8, ..; 4 dims per lane
  for (int col = warp; col < x.ncol; col += kWarps) {
    float m = kNone;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, jt[w * NC + col]);
    float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mt = jt[w * NC + col];
      if (js[w * NC + col] == 0.f) continue;       // saw nothing
      const float k = ex2(mt - m);
      l = fmaf(js[w * NC + col], k, l);
      const float4 v = *reinterpret_cast<const float4*>(jo + (w * NC + col) * kHeadDim + 4 * lane);
      acc[0] = fmaf(v.x, k, acc[0]);
      acc[1] = fmaf(v.y, k, acc[1]);
      acc[2] = fmaf(v.z, k, acc[2]);
      acc[3] = fmaf(v.w, k, acc[3]);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);    // NaN stays NaN
    const float l2 = l == 0.f ? kNegInf : m + log2f(l);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= inv;
    const int cc = x.col0 + col;
    const int row = x.row0 + cc / p.G, head = x.head * p.G + cc % p.G;
    if (s.nsplit > 1) {
      const int64_t pv = s.part0 + ((int64_t)x.part * s.rows + row) * p.Hq + head;
      *reinterpret_cast<float4*>(p.part_o + pv * kHeadDim + 4 * lane) =
          make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (lane == 0) p.part_lse[pv] = l2;
    } else {
      const int64_t gr = s.q0 + row;
      uint2 u;
      if constexpr (kFp16) {
        u.x = pack_half(acc[0], acc[1]);
        u.y = pack_half(acc[2], acc[3]);
      } else {
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc[0], acc[1]);
        const __nv_bfloat162 h1 = __floats2bfloat162_rn(acc[2], acc[3]);
        u.x = *reinterpret_cast<const uint32_t*>(&h0);
        u.y = *reinterpret_cast<const uint32_t*>(&h1);
      }
      *reinterpret_cast<uint2*>(p.out.ptr + gr * p.out.rs + (int64_t)head * p.out.hs + 4 * lane) =
          u;
      if (lane == 0) {
        if (p.lse) p.lse[gr * p.Hq + head] = l2 * 0.6931471805599453f;
        if (p.lse2) p.lse2[gr * p.Hq + head] = l2;
      }
    }
  }
}

// ---- joining split sequences ------------------------------------------------

struct JoinParams {
  Rows16 out;
  float *lse, *lse2;
  const float *part_o, *part_lse;
  int Hq;
  bool hold;         // fp16: finite means stay finite (prompt: no value is beyond fp16's end)
};

// One warp per (row, head) vector of a split sequence, 4 dimensions per lane.
// unit0 of the table counts (row, head) vectors here.
template <bool kFp16>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnTable t,
                                                   JoinParams p) {
  const int u = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  grid_release();
  if (u >= t.units) return;
  const int si = find_seq(t.n, u, [&](int m) { return t.s[m].unit0; });
  const AttnSeq& s = t.s[si];
  const int vec = u - s.unit0;                      // row * Hq + head
  grid_wait();
  const int64_t stride = (int64_t)s.rows * p.Hq;
  const float* pl = p.part_lse + s.part0 + vec;
  float m = kNegInf;
  bool nan = false;
  for (int i = lane; i < s.nsplit; i += 32) {
    const float v = pl[i * stride];
    m = fmaxf(m, v);
    nan |= v != v;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (__any_sync(0xFFFFFFFFu, nan)) m = NAN;
  const float m0 = m == kNegInf ? 0.f : m;
  float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < s.nsplit; ++i) {
    const float v = pl[i * stride];
    if (v == kNegInf) continue;                     // this part saw nothing
    const float k = ex2(v - m0);
    const float4 a = *reinterpret_cast<const float4*>(
        p.part_o + (s.part0 + i * stride + vec) * kHeadDim + 4 * lane);
    l += k;
    acc[0] = fmaf(a.x, k, acc[0]);
    acc[1] = fmaf(a.y, k, acc[1]);
    acc[2] = fmaf(a.z, k, acc[2]);
    acc[3] = fmaf(a.w, k, acc[3]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float l2 = l == 0.f ? kNegInf : m0 + log2f(l);
  const int64_t row = s.q0 + vec / p.Hq;
  const int head = vec % p.Hq;
  uint2 o;
  if constexpr (kFp16) {
    o.x = pack_half(acc[0] * inv, acc[1] * inv);
    o.y = pack_half(acc[2] * inv, acc[3] * inv);
    if (p.hold) {
      o.x = hold_finite(o.x, acc[0] * inv, acc[1] * inv);
      o.y = hold_finite(o.y, acc[2] * inv, acc[3] * inv);
    }
  } else {
    const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
    const __nv_bfloat162 h1 = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
    o.x = *reinterpret_cast<const uint32_t*>(&h0);
    o.y = *reinterpret_cast<const uint32_t*>(&h1);
  }
  *reinterpret_cast<uint2*>(p.out.ptr + row * p.out.rs + (int64_t)head * p.out.hs + 4 * lane) = o;
  if (lane == 0) {
    if (p.lse) p.lse[row * p.Hq + head] = l2 * 0.6931471805599453f;
    if (p.lse2) p.lse2[row * p.Hq + head] = l2;
  }
}

// ---- recorded weights ---------------------------------------------------------

constexpr int kWSlices = 2;                        // slices per warp and block: 32 tokens
constexpr int kWBlock = kWSlices * kSlice;
constexpr int kWMeet = 4;                          // blocks between two meetings of the warps
constexpr int kWStage = kSlice * (kVecCodes + kVecParams);   // keys alone: 1280 bytes
constexpr int kWKp = kSlice * kVecCodes;

struct WeightParams {
  AttendParams a;
  int heads;            // key heads at a time: min(8, Hkv); 8 / heads token blocks at a time
};

// Every visible key: scores are computed again from the keys (80 bytes per token
// and key head, less than storing and reading 4 bytes per column once there are
// more than 10 columns, and no workspace of the cache's length) now that every
// column's lse is known, and summed over the columns.
// A warp keeps one key head's query operands and walks the CTA's tokens in
// blocks of 32 with the next block's keys in flight; the warps' sums of 4
// blocks meet in shared memory and are added in a fixed order, one thread per
// token.  A unit is (sequence, range of tokens).
template <int NT, bool kFp16>
__global__ void __launch_bounds__(kThreads, 2)
    weights_kernel(const __grid_constant__ AttnTable t, const __grid_constant__ WeightParams w) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_sum[2][kWarps][kWMeet * kWBlock];
  const AttendParams& p = w.a;
  constexpr int NC = 8 * NT;
  const int si = find_seq(t.n, blockIdx.x, [&](int m) { return t.s[m].unit0; });
  const AttnSeq& s = t.s[si];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int cols = s.rows * p.G;
  Unit x;
  x.row0 = 0;
  x.limit0 = s.pos0 + 1;
  x.list = nullptr;
  const int len = s.pos0 + s.rows;
  x.lo = (blockIdx.x - s.unit0) * s.chunk;
  x.hi = min(len, x.lo + s.chunk);
  const int subs = kWarps / w.heads, sub = warp / w.heads;
  const int block = kWSlices * kSlice * subs;      // tokens the CTA takes at a time
  const int n_blocks = (x.hi - x.lo + block - 1) / block;
  const uint32_t ring = smem_u32(smem) + warp * 2 * kWSlices * kWStage;
  const uint32_t q_at = smem_u32(smem) + kWarps * 2 * kWSlices * kWStage + warp * query_smem<NT>();

  for (int head0 = 0; head0 < p.Hkv; head0 += w.heads)
    for (int col0 = 0; col0 < cols; col0 += NC) {
      const bool on = sub < subs && head0 + warp % w.heads < p.Hkv;
      x.head = on ? head0 + warp % w.heads : 0;
      x.col0 = col0;
      x.ncol = min(NC, cols - col0);
      const int first = x.lo + sub * kWSlices * kSlice;
      SliceWalk<false, kWKp> walk(p, x, s.k0, first);
      auto fill = [&](int b) {                     // block b of the warp's tokens
        const uint32_t at = ring + (b & 1) * kWSlices * kWStage;
#pragma unroll
        for (int i = 0; i < kWSlices; ++i) {
          if (on)
            walk.issue(at + i * kWStage, i + 1 < kWSlices ? 1 : block / kSlice - kWSlices + 1);
        }
      };
      __syncwarp();
      fill(0);
      QueryFrags<NT> f;
      f.at = q_at;
      load_query<NT, kFp16>(p, s, x, f);
      __syncwarp();
      if (head0 == 0 && col0 == 0) {
        grid_wait();                               // lse2; the cache and q are older
        grid_release();
      }
      float l2[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = n * 8 + 2 * c + i;
          float v = INFINITY;                      // columns that do not exist add nothing
          if (col < x.ncol) {
            const int cc = col0 + col;
            v = p.lse2[(int64_t)(s.q0 + cc / p.G) * p.Hq + x.head * p.G + cc % p.G];
            if (v == kNegInf) v = INFINITY;
          }
          l2[n][i] = v;
        }
      for (int b = 0; b < n_blocks; ++b) {
        if (b + 1 < n_blocks) {
          fill(b + 1);
          cp_wait<kWSlices>();
        } else {
          cp_wait<0>();
        }
        __syncwarp();
        const uint32_t at = ring + (b & 1) * kWSlices * kWStage;
        float* sums = s_sum[b / kWMeet & 1][warp] + b % kWMeet * kWBlock;
#pragma unroll
        for (int i = 0; i < kWSlices; ++i) {
          const int tok0 = first + b * block + i * kSlice;
          float acc[2] = {0.f, 0.f};
          if (on && tok0 < x.hi) {
            float sc[NT][4];
            slice_scores<NT, kWKp, false>(f, at + i * kWStage, sc);
            // slices every column sees whole need no mask
            if (tok0 + kSlice <= x.hi && tok0 + kSlice <= x.limit0 + col0 / p.G) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  // a column without weight has l2 = infinity: 2^-infinity = 0
                  acc[j >> 1] += ex2(fmaf(sc[n][j], f.back[n][j & 1], -l2[n][j & 1]));
            } else {
              const int tok = tok0 + r;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int col = n * 8 + 2 * c + (j & 1);
                  if (l2[n][j & 1] != INFINITY &&
                      column_sees(p, x, j < 2 ? tok : tok + 8, 0, col))
                    acc[j >> 1] += ex2(fmaf(sc[n][j], f.back[n][j & 1], -l2[n][j & 1]));
                }
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v = acc[j];
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
            if (c == 0) sums[i * kSlice + j * 8 + r] = v;
          }
        }
        if (b % kWMeet != kWMeet - 1 && b + 1 < n_blocks) continue;
        // the buffer is written again two meetings later, behind the next barrier
        __syncthreads();
        const int b0 = b / kWMeet * kWMeet;
        for (int i = threadIdx.x; i < (b + 1 - b0) * block; i += kThreads) {
          const int tok = x.lo + b0 * block + i;
          if (tok >= x.hi) continue;
          const int in = i % block, first_warp = in / kWBlock * w.heads;
          const int at_sum = i / block * kWBlock + in % kWBlock;
          float v = 0.f;
          for (int k = 0; k < w.heads; ++k) v += s_sum[b / kWMeet & 1][first_warp + k][at_sum];
          atomicAdd(p.c.weight + s.k0 + tok, v);   // nothing waits for it; one thread per token
        }
      }
      __syncthreads();                             // before the next pass fills s_sum again
    }
}

// Selection: the scores the attend kernel stored, 4 bytes per entry and head (a
// second gather of the keys would move 80 bytes per entry and key head, and more
// from memory: it fetches whole lines), as weights summed over the heads.  8
// lanes per entry; a unit is (row, 32 entries of its list).  A sequence of one
// row adds to the tokens here (one that is listed twice gets two equal
// additions); several rows keep their sums for the next kernel.
constexpr int kListThreads = 256, kListChunk = kListThreads / 8;
__global__ void __launch_bounds__(kListThreads)
    weights_list_kernel(const __grid_constant__ AttnTable t, const float* scores, const float* lse2,
                        const int32_t* sel, int K, int Hq, float* row_weight, float* weight) {
  const int si = find_seq(t.n, blockIdx.x, [&](int m) { return t.s[m].unit0; });
  const AttnSeq& s = t.s[si];
  const int u = blockIdx.x - s.unit0, row = u / s.nsplit, lane = threadIdx.x & 7;
  const int64_t q = s.q0 + row, local = q - t.s[0].q0;
  const int j = u % s.nsplit * kListChunk + (threadIdx.x >> 3);
  const int idx = j < K ? __ldg(sel + q * K + j) : -1;
  grid_wait();
  grid_release();
  float v = 0.f;
  if (j < K) {
    const float* x = scores + (local * K + j) * Hq;
#pragma unroll 8
    for (int h = lane; h < Hq; h += 8) {
      const float l2 = lse2[q * Hq + h], sc = x[h];
      v += l2 == kNegInf ? 0.f : ex2(sc - l2);
    }
  }
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
  if (lane != 0 || j >= K) return;
  if (s.rows > 1) row_weight[local * K + j] = v;
  else if (idx >= 0 && idx <= s.pos0 + row) atomicAdd(weight + s.k0 + idx, v);
}

// Selection, sequences of several rows: the rows' sums go to the tokens they
// list, 4,096 entries of every list at a time and the rows in order within them (a
// CTA barrier between two rows).  Within a row a token listed twice gets two equal
// additions, so their order does not matter.  The next row's entries are loaded
// before the barrier.
constexpr int kScatterThreads = 1024, kScatterEach = 4;
__global__ void __launch_bounds__(kScatterThreads)
    weights_scatter_kernel(const __grid_constant__ AttnTable t, const int32_t* sel, int K,
                           const float* row_weight, float* weight) {
  const AttnSeq& s = t.s[blockIdx.x];
  if (s.rows <= 1) return;
  grid_wait();
  for (int k0 = 0; k0 < K; k0 += kScatterThreads * kScatterEach) {
    int idx[kScatterEach];
    float v[kScatterEach];
    auto load = [&](int row) {
#pragma unroll
      for (int i = 0; i < kScatterEach; ++i) {
        const int j = k0 + i * kScatterThreads + threadIdx.x;
        const int64_t q = s.q0 + row;
        idx[i] = j < K ? __ldg(sel + q * K + j) : -1;
        v[i] = j < K ? row_weight[(q - t.s[0].q0) * K + j] : 0.f;
      }
    };
    load(0);
    for (int row = 0; row < s.rows; ++row) {
#pragma unroll
      for (int i = 0; i < kScatterEach; ++i)
        if (idx[i] >= 0 && idx[i] <= s.pos0 + row) atomicAdd(weight + s.k0 + idx[i], v[i]);
      if (row + 1 < s.rows) load(row + 1);
      __syncthreads();
    }
  }
}

template <int NT, bool kFp16, bool kSel>
cudaError_t run_attend(const AttnTable& t, const AttendParams& p, cudaStream_t stream) {
  constexpr int smem = attend_smem<NT>();
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(attend_kernel<NT, kFp16, kSel>), smem, &done);
  if (e != cudaSuccess) return e;
  return launch_after(attend_kernel<NT, kFp16, kSel>, dim3(t.units), kThreads, smem, stream, t, p);
}

template <int NT, bool kFp16>
cudaError_t run_weights(const AttnTable& t, const WeightParams& w, cudaStream_t stream) {
  constexpr int smem = kWarps * (2 * kWSlices * kWStage + query_smem<NT>());
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(weights_kernel<NT, kFp16>), smem, &done);
  if (e != cudaSuccess) return e;
  return launch_after(weights_kernel<NT, kFp16>, dim3(t.units), kThreads, smem, stream, t, w);
}

}  // namespace

int attend_columns(const AttnHandle& h, int rows, bool selected) {
  const int64_t cols = selected ? h.G : (int64_t)rows * h.G;
  return cols <= 8 ? 8 : cols <= 16 ? 16 : 32;
}

cudaError_t launch_attend(const AttnHandle& h, const Cache4View& c, const Rows16& q,
                          const AttnTable& t, const int32_t* sel, int K, const Rows16& out,
                          float* lse, float* lse2, float* part_o, float* part_lse, float* scores,
                          cudaStream_t stream) {
  if (t.units <= 0) return cudaSuccess;
  AttendParams p;
  p.c = c;
  p.q = q;
  p.out = out;
  p.sel = sel;
  p.K = K;
  p.Hq = h.cfg.Hq;
  p.Hkv = h.cfg.Hkv;
  p.G = h.G;
  p.scale_log2 = h.scale_log2;
  p.lse = lse;
  p.lse2 = lse2;
  p.part_o = part_o;
  p.part_lse = part_lse;
  p.scores = scores;
  // every sequence of a launch takes the same column width
  const int nc = attend_columns(h, t.s[0].rows, sel != nullptr);
  profile_before(DOSA_KERNEL_ATTEND, stream);
  auto run = [&](auto nt, auto fp16) {
    return sel ? run_attend<decltype(nt)::value, decltype(fp16)::value, true>(t, p, stream)
               : run_attend<decltype(nt)::value, decltype(fp16)::value, false>(t, p, stream);
  };
  using N1 = std::integral_constant<int, 1>;
  using N2 = std::integral_constant<int, 2>;
  using N4 = std::integral_constant<int, 4>;
  auto pick = [&](auto fp16) {
    return nc == 8 ? run(N1{}, fp16) : nc == 16 ? run(N2{}, fp16) : run(N4{}, fp16);
  };
  const cudaError_t e = h.fp16 ? pick(std::true_type{}) : pick(std::false_type{});
  profile_after(DOSA_KERNEL_ATTEND, stream);
  return e;
}

cudaError_t launch_join(const AttnHandle& h, int kind, const AttnTable& t, const Rows16& out,
                        float* lse, float* lse2, const float* part_o, const float* part_lse,
                        cudaStream_t stream) {
  if (t.units <= 0) return cudaSuccess;
  JoinParams p;
  p.out = out;
  p.lse = lse;
  p.lse2 = lse2;
  p.part_o = part_o;
  p.part_lse = part_lse;
  p.Hq = h.cfg.Hq;
  p.hold = kind == DOSA_KERNEL_PROMPT;
  const unsigned grid = (unsigned)((t.units + 7) / 8);
  profile_before(kind, stream);
  const cudaError_t e = launch_after(h.fp16 ? join_kernel<true> : join_kernel<false>, dim3(grid), 256,
                                     0, stream, t, p);
  profile_after(kind, stream);
  return e;
}

cudaError_t launch_attend_weights(const AttnHandle& h, const Cache4View& c, const Rows16& q,
                                  const AttnTable& t, const float* lse2, cudaStream_t stream) {
  if (t.n <= 0) return cudaSuccess;
  WeightParams w = {};
  w.a.c = c;
  w.a.q = q;
  w.a.Hq = h.cfg.Hq;
  w.a.Hkv = h.cfg.Hkv;
  w.a.G = h.G;
  w.a.scale_log2 = h.scale_log2;
  w.a.lse2 = const_cast<float*>(lse2);
  w.heads = h.cfg.Hkv < kWarps ? h.cfg.Hkv : kWarps;
  // Here a sequence's units are ranges of tokens.  Two per SM: every CTA loads
  // its query operands once, and the shortest range is one block of 32 tokens
  // per group of warps.
  const int step = kWBlock * (kWarps / w.heads);
  AttnTable b = t;
  auto count = [&](int64_t blocks) {
    int64_t n = 0;
    for (int i = 0; i < b.n; ++i)
      n += ((int64_t)b.s[i].pos0 + b.s[i].rows + step * blocks - 1) / (step * blocks);
    return n;
  };
  int64_t longest = 1;
  int cols = 0;
  for (int i = 0; i < b.n; ++i) {
    const int64_t blocks = ((int64_t)b.s[i].pos0 + b.s[i].rows + step - 1) / step;
    if (blocks > longest) longest = blocks;
    if (b.s[i].rows * h.G > cols) cols = b.s[i].rows * h.G;
  }
  const int64_t slots = 2 * (int64_t)attn_sm_count();
  int64_t lo = 1, hi = longest;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (count(mid) <= slots) hi = mid;
    else lo = mid + 1;
  }
  int units = 0;
  for (int i = 0; i < b.n; ++i) {
    AttnSeq& s = b.s[i];
    s.chunk = (int)(lo * step);
    s.nsplit = (int)(((int64_t)s.pos0 + s.rows + s.chunk - 1) / s.chunk);
    s.unit0 = units;
    units += s.nsplit;
  }
  b.units = units;
  profile_before(DOSA_KERNEL_ATTEND, stream);
  auto pick = [&](auto fp16) {
    constexpr bool f = decltype(fp16)::value;
    return cols <= 8    ? run_weights<1, f>(b, w, stream)
           : cols <= 16 ? run_weights<2, f>(b, w, stream)
                        : run_weights<4, f>(b, w, stream);
  };
  const cudaError_t e = h.fp16 ? pick(std::true_type{}) : pick(std::false_type{});
  profile_after(DOSA_KERNEL_ATTEND, stream);
  return e;
}

cudaError_t launch_list_weights(const AttnHandle& h, const AttnTable& t, const int32_t* sel, int K,
                                const float* scores, const float* lse2, float* row_weight,
                                float* weight, cudaStream_t stream) {
  if (t.n <= 0) return cudaSuccess;
  AttnTable b = t;
  bool several = false;
  int units = 0;
  for (int i = 0; i < b.n; ++i) {
    AttnSeq& s = b.s[i];
    s.nsplit = (K + kListChunk - 1) / kListChunk;
    s.unit0 = units;
    units += s.nsplit * s.rows;
    several |= s.rows > 1;
  }
  b.units = units;
  profile_before(DOSA_KERNEL_ATTEND, stream);
  cudaError_t e = launch_after(weights_list_kernel, dim3(units), kListThreads, 0, stream, b, scores,
                               lse2, sel, K, h.cfg.Hq, row_weight, weight);
  profile_after(DOSA_KERNEL_ATTEND, stream);
  if (e != cudaSuccess || !several) return e;
  profile_before(DOSA_KERNEL_ATTEND, stream);
  e = launch_after(weights_scatter_kernel, dim3(b.n), kScatterThreads, 0, stream, b, sel, K,
                   (const float*)row_weight, weight);
  profile_after(DOSA_KERNEL_ATTEND, stream);
  return e;
}

}  // namespace dosa
