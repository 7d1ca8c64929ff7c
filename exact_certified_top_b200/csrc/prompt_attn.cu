// Causal attention of packed query rows over 16-bit keys and values
// (tcgen05 + TMEM + TMA).
//
// A unit is (sequence, 256 packed query rows, key head, part of the key axis).
// CTAs are persistent: a running CTA takes over the launch of one that has not
// started (cluster launch control), so the next unit's loads and first products
// overlap the end of this one, and set-up is paid once per SM.  Packed rows are
// (token, head of the group) pairs, tokens major: all heads that share a key
// head ride on the same key tiles, and a single token of a group of 8 already
// fills 8 rows of the tile.  The 256 rows are two MMA tiles A and B of 128;
// while one tile's scores go through the softmax the tensor core works for the
// other.
//   warps 0-3, 4-7  softmax of tile A, B: one row per thread
//   warps 8, 11     MMA issuers of tile A, B (warp 8 owns the TMEM)
//   warp 9          TMA producer; fetches the CTA's next unit
//   warp 10         checks of the values some row does not see
// One issuer per tile, because a wait costs an issuer 250 cycles when its
// products are queued ahead of it: the other tile's products fill that gap.
// Keys go in steps of 64:  S = Q K^T (both operands in shared memory, fp32 in
// TMEM), softmax in registers, P in the 16-bit type written over S in TMEM,
// O += P V (P from TMEM, V from shared memory, keys as the contraction).  Each
// tile has two S buffers, so its next scores are computed while the softmax
// works on the present ones and neither waits for the other: with one buffer of
// 128 keys a tile's softmax and products took turns, and 2,000 of 4,200 cycles
// per pair of tiles went by in waits.  The price is N = 64 in S = Q K^T, which
// takes 411 cycles per step instead of 256 (the operands' shared memory reads
// bound it): 2,510 cycles of tensor work per pair of tiles and 128 keys, against
// 2,048 with N = 128.
// TMEM columns: S_A0, S_A1, S_B0, S_B1 (64 each), O_A, O_B (128 each).  K and V
// tiles of 128 keys share one ring of four 32 KB stages.  The running maximum a
// row is scaled by moves only when it would grow by more than 2^kSlack, so O is
// rarely rescaled: P stays below 2^kSlack (2^(kSlack + kLift) in fp16), and sums are
// fp32.  A CTA's roles wait on mbarriers only; every wait is bounded.
//
// The softmax with a running maximum and sum is the online one of M. Milakov and
// N. Gimelshein (2018).  The arrangement is that of published attention for this
// tensor core: two row tiles that take turns, P over S in TMEM, a maximum that
// moves only by more than 2^8, a share of the exponentials as polynomials.
//
// Measured: 16,384 tokens, 64 heads over 8: 3.65 ms, 1.2 PFLOP/s for the 4.4
// TFLOP below the diagonal (4.2 ms when the power cap holds the clock).  Per 64
// keys of both tiles the softmax takes 1,210 of about 1,690 cycles and waits for
// the rest, the tensor core works 1,256: neither is full, and the exponentials (a
// third of them on the FMA pipe) bound what a better overlap could reach.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_internal.h"
#include "dosa_device.cuh"

namespace dosa {
namespace {

constexpr int kTile = 128;                           // rows of an MMA tile, keys of a K or V tile
constexpr int kStep = 64;                            // keys per softmax step
constexpr int kStages = 4;
constexpr uint32_t kSubBytes = kTile * 128;          // 128 rows x 64 elements
constexpr uint32_t kTileBytes = 2 * kSubBytes;       // 32 KB
constexpr int kSoftWarps = 8;
constexpr int kThreads = 384;
constexpr int kBadWords = 12;                        // 256 keys touch at most 3 tiles
constexpr uint32_t kBarBytes = 384;
constexpr int kBadUnits = 4;                         // units the checks may be ahead, plus one
constexpr uint32_t kBadBytes = 2 * kBadUnits * (kBadWords + 1) * 4;
constexpr uint32_t kOutBytes = kSoftWarps * 32 * 128;   // 128 bytes of each row on their way out
constexpr uint32_t kSmemBytes =
    1024 + (2 + kStages) * kTileBytes + kOutBytes + kBarBytes + kBadBytes;
constexpr float kSlack = 8.f;                        // log2 units
// fp16 weights are kept 2^kLift times larger, up to 2^15: an fp16 below 2^-14 has
// fewer bits, and a weight far below the row's maximum would lose them (below
// 2^-25 of it all of them, and thousands of such keys add up).  bf16 has the range.
template <bool kFp16>
constexpr float kLift = kFp16 ? 7.f : 0.f;

struct PromptParams {
  int Hq, Hkv, G, tok;       // tok: tokens per MMA tile (128 / G)
  float scale_log2;
  Rows16 v, out;
  float* lse;
  float *part_o, *part_lse;
  int* err;
};

struct PromptUnit {
  int head, part;
  int tok0;                  // first token of tile A (row of the sequence)
  int j0;                    // first key tile of the part
  int n[2];                  // key tiles of A and B in this part
  int ntok[2];               // tokens of A and B
};

__device__ __forceinline__ PromptUnit unit_of(const PromptParams& p, const AttnSeq& s, int u) {
  PromptUnit x;
  x.head = u % p.Hkv;
  u /= p.Hkv;
  x.part = u % s.nsplit;
  u /= s.nsplit;
  const int pairs = (s.rows + 2 * p.tok - 1) / (2 * p.tok);
  x.tok0 = (pairs - 1 - u) * 2 * p.tok;              // longest rows first
  x.j0 = x.part * s.chunk;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int first = x.tok0 + i * p.tok;
    const int n = min(p.tok, s.rows - first);
    x.ntok[i] = n > 0 ? n : 0;
    const int tiles = n > 0 ? (s.pos0 + first + n - 1) / kTile + 1 : 0;
    x.n[i] = max(0, min(tiles, s.nsplit > 1 ? x.j0 + s.chunk : tiles) - x.j0);
  }
  return x;
}

// ---- tcgen05 pieces this kernel adds -----------------------------------------

// D[tmem] (+)= A[tmem] * B[smem desc]
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 32 bit stores to 16 consecutive columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10,"
      " %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// V as the B operand: its tile is [keys][64 dims] per half, so the contraction
// (keys) runs along rows and the dims are contiguous (MN-major, 128-byte
// swizzle).  Leading offset: the second half of the dims, kSubBytes on; stride
// offset: 8 keys, 1024 bytes on.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)(kSubBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <bool kFp16, bool kBMn, int kN>
__host__ __device__ constexpr uint32_t idesc() {
  return (1u << 4) | ((kFp16 ? 0u : 1u) << 7) | ((kFp16 ? 0u : 1u) << 10) |
         ((kBMn ? 1u : 0u) << 16) | ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kFp16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool kFp16>
__device__ __forceinline__ float widen(uint32_t bits) {
  if constexpr (kFp16) return __half2float(__ushort_as_half((unsigned short)bits));
  return __uint_as_float(bits << 16);
}

// ---- softmax pieces ------------------------------------------------------------

// Maxima that keep NaN: a row that sees one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max32(const float (&v)[32]) {
  float a = max_nan(v[0], v[1]), b = max_nan(v[2], v[3]), c = max_nan(v[4], v[5]),
        d = max_nan(v[6], v[7]);
#pragma unroll
  for (int e = 8; e < 32; e += 8) {
    a = max3(a, v[e], v[e + 1]);
    b = max3(b, v[e + 2], v[e + 3]);
    c = max3(c, v[e + 4], v[e + 5]);
    d = max3(d, v[e + 6], v[e + 7]);
  }
  return max_nan(max3(a, b, c), d);
}

template <int kBase>
__device__ __forceinline__ void mask_from(float (&v)[32], int lim) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (kBase + e > lim) v[e] = -INFINITY;
}

// Two fp32 operations per instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// 2^x on the FMA pipe, x <= kSlack: x = n + f with n the nearest integer (taken
// out of the low bits of x + 1.5 2^23), 2^f on [-1/2, 1/2] by the degree-4
// polynomial of least relative error (2.6e-6, fitted by Remez exchange; P itself
// rounds to 2^-11 or 2^-8), times 2^n.  x is held at -127, whose factor is a zero
// of the bits: masked scores (-infinity) and what is below 2^-126.5 weigh nothing,
// however large the value.  NaN stays: a score of +infinity is one here (infinity
// minus the maximum it has become), and a zero in its place would drop the key
// and leave a row without weights.
__device__ __forceinline__ float2 ex2_poly(float2 x) {
  x = make_float2(max_nan(x.x, -127.f), max_nan(x.y, -127.f));
  const float2 r = add2(x, both(12582912.f));
  const float2 f = add2(x, fma2(r, both(-1.f), both(12582912.f)));
  float2 q = fma2(f, both(9.570102207362652e-3f), both(5.591785907745361e-2f));
  q = fma2(q, f, both(2.40247443318367e-1f));
  q = fma2(q, f, both(6.931217908859253e-1f));
  q = fma2(q, f, both(9.999992847442627e-1f));
  return mul2(q, make_float2(__uint_as_float((__float_as_uint(r.x) << 23) + 0x3F800000u),
                             __uint_as_float((__float_as_uint(r.y) << 23) + 0x3F800000u)));
}

// 32 scores to weights 2^(c v + off), added to the two sums and stored as 16
// packed columns of P.  One pair in three takes the polynomial: the exponential
// unit gives 16 results a clock and SM, and the two tiles' warps together took
// 1,150 cycles per 64 keys with it alone against 970 with the mix (one pair in
// two or in four: 1,190 and 1,140).
constexpr int kPolyEvery = 3;
template <bool kFp16>
__device__ __forceinline__ void exp_store(const float (&v)[32], float c, float off, float2& sum,
                                          uint32_t taddr) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 x = fma2(make_float2(v[2 * e], v[2 * e + 1]), both(c), both(off));
    const float2 q = e % kPolyEvery == kPolyEvery - 1 ? ex2_poly(x)
                                                       : make_float2(ex2(x.x), ex2(x.y));
    sum = add2(sum, q);
    w[e] = pack2<kFp16>(q.x, q.y);
  }
  tmem_st16(taddr, w);
}

// Multiply a row's 128 columns of O.  Out of line: it is rare, and inside the
// softmax loop it pushes the rest out of the instruction cache.
__device__ __noinline__ void rescale_row(uint32_t taddr, float k) {
#pragma unroll 1
  for (int b = 0; b < 8; ++b) {
    float o[16];
    tmem_ld16_async(taddr + b * 16, o);
    tmem_wait_ld16(o);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] *= k;
    tmem_st16(taddr + b * 16, reinterpret_cast<const uint32_t*>(o));
  }
}

// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// mbar_wait whose clock is first read after 1024 polls: reading %globaltimer
// takes as long as a matrix product, and the waits of this kernel are on its
// critical path (with the clock read up front a tile pair took 2,400 cycles in
// barriers alone).
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             int* err) {
  const uint32_t a = smem_u32(bar);
  for (int i = 0; i < 1024; ++i)
    if (mbar_try_wait(a, parity)) return true;
  return mbar_wait(bar, parity, abort, err);
}
// All lanes wait; the answer is the warp's.  The vote inside the loop keeps the
// branch uniform: a wait that is already over costs 40 cycles instead of 90.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int* err) {
  const uint32_t a = smem_u32(bar);
  for (int i = 0; i < 1024; ++i)
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(a, parity))) return true;
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort, err)) != 0;
}

// Both halves of w that are infinite or NaN as ones.
template <bool kFp16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  constexpr uint32_t e = kFp16 ? 0x7C007C00u : 0x7F807F80u;
  return __vcmpeq2(w & e, e);
}

// A row that does not see a key has weight 0 for it, and 0 times an infinity or
// NaN is NaN: the values of a tile's keys from all_see on (which some row of
// the unit does not see) must be finite in the product.  Keys nobody sees are
// cleared; of the others, elements that are not finite are cleared and the key
// noted for both tiles, and the rows that see it add the element at the end.
// One warp; the tile holds keys key0 .. key0 + 127.
template <bool kFp16>
__device__ __forceinline__ void clean_values(uint8_t* v, int key0, int all_see, int vis_end,
                                             uint32_t* bad0, uint32_t* bad1) {
  const int lane = threadIdx.x & 31;
  const int r0 = max(0, all_see - key0), r1 = min(kTile, max(vis_end - key0, 0));
  auto at = [&](int e) {                               // 16-byte chunk e % 16 of row e / 16
    return reinterpret_cast<uint4*>(v + ((e & 15) >> 3) * kSubBytes + (e >> 4) * 128 + (e & 7) * 16);
  };
#pragma unroll 8
  for (int e = max(r0, r1) * 16 + lane; e < kTile * 16; e += 32) *at(e) = make_uint4(0, 0, 0, 0);
  for (int e0 = r0 * 16 + lane; e0 < r1 * 16; e0 += 4 * 32) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = e0 + i * 32 < r1 * 16 ? *at(e0 + i * 32) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = not_finite2<kFp16>(w[i].x), b = not_finite2<kFp16>(w[i].y),
                     c = not_finite2<kFp16>(w[i].z), d = not_finite2<kFp16>(w[i].w);
      if (a | b | c | d) {
        const int e = e0 + i * 32;
        *at(e) = make_uint4(w[i].x & ~a, w[i].y & ~b, w[i].z & ~c, w[i].w & ~d);
        const int k = key0 + (e >> 4) - all_see / kTile * kTile;
        atomicOr(bad0 + (k >> 5), 1u << (k & 31));
        atomicOr(bad1 + (k >> 5), 1u << (k & 31));
        bad0[kBadWords] = bad1[kBadWords] = 1;
      }
    }
  }
}

// The noted elements of the keys a row sees, added to 128 bytes of the row in
// shared memory (swizzled chunks): `b`-th 64 dimensions of 16 bits, or 32 of fp32.
// Out of line: rare.
template <bool kFp16>
__device__ __noinline__ void add_not_finite(uint8_t* row, int swz, bool split, int b,
                                            const uint32_t* bad, int bad0, int pos,
                                            const uint16_t* v, int64_t rs) {
  const int n = split ? 32 : 64;
  for (int w = 0; w < kBadWords; ++w)
    for (uint32_t bits = bad[w]; bits; bits &= bits - 1) {
      const int key = bad0 + 32 * w + __ffs(bits) - 1;
      if (key > pos) continue;
      for (int e = 0; e < n; ++e) {
        const uint32_t x = v[key * rs + b * n + e];
        if (!(not_finite2<kFp16>(x) & 0xFFFFu)) continue;
        const int at = e * (split ? 4 : 2);
        uint8_t* to = row + ((((at >> 4) ^ swz) << 4) | (at & 15));
        if (split) {
          *reinterpret_cast<float*>(to) += widen<kFp16>(x);
        } else {
          uint16_t* t = reinterpret_cast<uint16_t*>(to);
          *t = (uint16_t)pack2<kFp16>(widen<kFp16>(*t) + widen<kFp16>(x), 0.f);
        }
      }
    }
}

// ---- units -----------------------------------------------------------------------

// Ask for the launch of a CTA that has not started; 16 bytes of answer arrive on
// the barrier.
__device__ __forceinline__ void fetch_unit(uint4* slot, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::
          "r"(smem_u32(slot)),
      "r"(smem_u32(bar))
      : "memory");
}
// The answer: that CTA's index, or -1 when none is left.
__device__ __forceinline__ int fetched_unit(const uint4* slot) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(slot))
      : "memory");
  return got ? (int)x : -1;
}

struct UnitView {
  AttnSeq s;
  PromptUnit x;
  int n_max;
  // keys below all_see are seen by every row of the unit, keys from vis_end on
  // by none
  int all_see, vis_end;
};
__device__ __forceinline__ UnitView view_unit(const PromptParams& p, const AttnTable& t, int unit) {
  UnitView v;
  v.s = t.s[find_seq(t.n, unit, [&](int m) { return t.s[m].unit0; })];
  v.x = unit_of(p, v.s, unit - v.s.unit0);
  v.n_max = max(v.x.n[0], v.x.n[1]);
  v.all_see = v.s.pos0 + v.x.tok0 + 1;
  v.vis_end = v.all_see + v.x.ntok[0] + v.x.ntok[1] - 1;
  return v;
}

template <bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ AttnTable t,
                  const __grid_constant__ PromptParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                                // tiles A, B
  uint8_t* sKV = smem + 2 * kTileBytes;
  uint8_t* sO = sKV + kStages * kTileBytes;
  uint8_t* ctl = sO + kOutBytes;
  uint4* u_slot = reinterpret_cast<uint4*>(ctl);     // [2] answers of fetch_unit
  uint64_t* u_full = reinterpret_cast<uint64_t*>(ctl + 32);
  uint64_t* u_empty = u_full + 2;
  uint64_t* q_full = u_empty + 2;                    // [2] tiles A, B
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;                    // [tile][buffer]: scores are there, and the
                                                     // product with the buffer's last P is done
  uint64_t* p_ready = s_full + 4;                    // [tile][buffer]
  uint64_t* o_full = p_ready + 4;                    // [tile]: the unit's s_bad is final
  uint64_t* v_clean = o_full + 2;                    // [stage]: the V tile has been checked
  uint64_t* kv_full = v_clean + kStages;
  uint64_t* kv_empty = kv_full + kStages;
  uint64_t* s_seen = kv_empty + kStages;             // [tile]: the unit's last s_full were seen
  uint64_t* done_bar = s_seen + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done_bar + 2);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  // per tile and last kBadUnits of its units: [kBadWords] keys with a value that is not
  // finite, and whether there are any
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(ctl + kBarBytes);
  // the same in every lane, and known to be: roles branch on it without divergence
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 3);                    // both issuers, the checks
      mbar_init(&v_clean[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], kSoftWarps + 4);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&s_seen[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&done_bar[i], 1);
    *s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == kSoftWarps) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // All 512 columns are this CTA's, so they start at 0; a constant keeps the
  // addresses of the matrix instructions out of registers.
  constexpr uint32_t tmem = 0;
  if (*s_tmem != tmem) {
    if (threadIdx.x == 0) record_error(p.err, kDevBounds);
    *s_abort = 1;
  }

  // The unit after the it-th: every warp of a role reads the answer.
  auto next_unit = [&](int it) {
    if (!warp_wait(&u_full[it & 1], (it >> 1) & 1, s_abort, p.err)) return -1;
    // the broadcast tells the compiler that the index is the warp's: what follows
    // from it stays in uniform registers, from which matrix instructions issue
    const int u = __shfl_sync(0xFFFFFFFFu, fetched_unit(&u_slot[it & 1]), 0);
    fence_proxy_async_smem();                        // read before the next answer is written
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[it & 1]);
    __syncwarp();
    return u;
  };

  if (warp >= kSoftWarps) {
    if (warp == kSoftWarps + 1) {
      // ---------------- TMA producer ----------------
      const uint32_t q_bytes = 2u * 128u * p.tok * p.G;
      uint32_t c = 0, nq[2] = {0, 0};
      int it = 0;
      for (int unit = blockIdx.x; unit >= 0; unit = next_unit(it++)) {
        const UnitView v = view_unit(p, t, unit);
        bool ok = true;
        if (lane == 0) {
          // The next unit is asked for two tiles before this one's end: early enough
          // to load on without a gap, late enough that the CTA with the least left
          // to do gets it.
          auto ask = [&] {
            ok = bounded_wait(&u_empty[it & 1], ((it >> 1) & 1) ^ 1, s_abort, p.err);
            if (ok) fetch_unit(&u_slot[it & 1], &u_full[it & 1]);
          };
          const int ask_at = v.n_max > 2 ? v.n_max - 2 : 0;
          if (v.n_max == 0) ask();
          for (int j = 0; j < v.n_max && ok; ++j) {
            if (j == ask_at) ask();
            if (!ok) break;
            for (int i = 0; i < 2 && j == 0 && ok; ++i) {
              if (v.x.n[i] == 0) continue;
              ok = bounded_wait(&q_empty[i], (nq[i] & 1) ^ 1, s_abort, p.err);
              if (!ok) break;
              mbar_arrive_expect_tx(&q_full[i], q_bytes);
              for (int sub = 0; sub < 2; ++sub)
                tma_load_3d(sQ + i * kTileBytes + sub * kSubBytes, &qmap, &q_full[i], sub * 64,
                            v.x.head * p.G, v.s.q0 + v.x.tok0 + i * p.tok);
              ++nq[i];
            }
            const int row = (int)v.s.k0 + (v.x.j0 + j) * kTile;
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const uint32_t st = c % kStages;
              ok = bounded_wait(&kv_empty[st], ((c / kStages) & 1) ^ 1, s_abort, p.err);
              if (!ok) break;
              mbar_arrive_expect_tx(&kv_full[st], kTileBytes);
              for (int sub = 0; sub < 2; ++sub)
                tma_load_3d(sKV + st * kTileBytes + sub * kSubBytes, kv ? &vmap : &kmap,
                            &kv_full[st], sub * 64, v.x.head, row);
              ++c;
            }
          }
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
      }
      if (lane == 0 && *s_abort) {
        // let what is in flight land before the CTA can exit
        mbar_wait_drain(&u_full[it & 1], (it >> 1) & 1);
        for (int i = 0; i < 2; ++i)
          if (nq[i]) mbar_wait_drain(&q_full[i], (nq[i] - 1) & 1);
        for (uint32_t i = c > (uint32_t)kStages ? c - kStages : 0; i < c; ++i)
          mbar_wait_drain(&kv_full[i % kStages], (i / kStages) & 1);
      }
      __syncwarp();
    } else if (warp == kSoftWarps || warp == kSoftWarps + 3) {
      // ---------------- MMA issuers ----------------
      // The whole warp walks the units and waits; one lane issues.  With all of it
      // in one lane's code every operand went from a vector to a uniform register
      // for each instruction.
      const int i = warp == kSoftWarps ? 0 : 1;        // tile
      const bool issuer = elect_one();
      // operand descriptors advance by constants from these bases (16-byte units)
      const uint64_t dq = smem_desc_sw128(smem_u32(sQ + i * kTileBytes)),
                     dk = smem_desc_sw128(smem_u32(sKV)), dv = smem_desc_mn(smem_u32(sKV));
      const uint32_t ts = tmem + i * kTile, to = tmem + (2 + i) * kTile;
      auto qk = [&](int hf, uint32_t st) {             // S = Q K^T of 64 keys
        const uint64_t b = dk + st * (kTileBytes >> 4) + hf * (kStep * 128 >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = ((k >> 2) * kSubBytes + (k & 3) * 32) >> 4;
          tc_mma<false>(ts + hf * kStep, dq + off, b + off, idesc<kFp16, false, kStep>(), k > 0);
        }
      };
      auto pv = [&](int hf, uint32_t st, bool first) { // O += P V of 64 keys
        const uint64_t b = dv + st * (kTileBytes >> 4) + hf * (kStep * 128 >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_ts(to, ts + hf * kStep + k * 8, b + k * (2048 >> 4),
                    idesc<kFp16, true, kTile>(), k > 0 ? 1u : (first ? 0u : 1u));
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return warp_wait(bar, parity & 1, s_abort, p.err);
      };
      uint32_t c = 0, nq = 0, np = 0;                  // ring position; units, key tiles so far
      uint32_t clean = 0;                              // phase of each stage's v_clean
      int it = 0;
      for (int unit = blockIdx.x; unit >= 0; unit = next_unit(it++)) {
        const UnitView v = view_unit(p, t, unit);
        const int n_max = v.n_max, n = i ? v.x.n[1] : v.x.n[0];
        bool ok = true;
        if (n_max > 0) {
          const uint32_t sk = c % kStages;
          // a tile that is not used is waited for all the same: an arrival before
          // it would count for the stage's previous tile
          ok = wait(&kv_full[sk], c / kStages);
          if (n > 0) {
            if (ok) ok = wait(&q_full[i], nq);
            // The softmax warps have seen the last unit's products end: a phase that
            // completed before they looked would be lost to them, and a barrier's
            // parity tells only neighbours apart.
            if (ok) ok = wait(&s_seen[i], nq + 1);
            tc_fence_after();
            if (issuer && ok) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                qk(hf, sk);
                tc_commit(&s_full[2 * i + hf]);
              }
              if (n == 1) tc_commit(&q_empty[i]);
              tc_commit(&kv_empty[sk]);
            }
            ++nq;
          } else if (issuer && ok) {
            mbar_arrive(&kv_empty[sk]);
          }
          __syncwarp();
        }
        for (int j = 0; j < n_max && ok; ++j) {
          const uint32_t cv = c + 2 * j + 1, ck = cv + 1;
          const uint32_t sv = cv % kStages, sk = ck % kStages;
          const bool masked = (v.x.j0 + j + 1) * kTile > v.all_see;
          ok = wait(&kv_full[sv], cv / kStages);
          if (ok && j + 1 < n_max) ok = wait(&kv_full[sk], ck / kStages);
          if (j < n) {
            if (ok && masked) ok = wait(&v_clean[sv], clean >> sv);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              if (ok) ok = wait(&p_ready[2 * i + hf], np);
              tc_fence_after();
              if (issuer && ok) {
                pv(hf, sv, j == 0 && hf == 0);
                if (j + 1 < n) qk(hf, sk);
                tc_commit(&s_full[2 * i + hf]);
              }
              __syncwarp();
            }
            ++np;
          }
          if (masked) clean ^= 1u << sv;
          if (issuer && ok) {
            // the last K tile this tile uses goes with its products, the others at once
            if (j < n) tc_commit(&kv_empty[sv]);
            else mbar_arrive(&kv_empty[sv]);
            if (j + 1 < n) tc_commit(&kv_empty[sk]);
            else if (j + 1 < n_max) mbar_arrive(&kv_empty[sk]);
            if (j + 2 == n) tc_commit(&q_empty[i]);
            if (j + 1 == n) mbar_arrive(&o_full[i]);
          }
          __syncwarp();
        }
        if (!ok) break;
        c += 2 * n_max;
      }
      // every MMA issued has completed once done_bar flips
      if (issuer) {
        tc_commit(&done_bar[i]);
        mbar_wait_drain(&done_bar[i], 0);
      }
      __syncwarp();
    } else {
      // ---------------- value checks ----------------
      // This warp goes over every stage and frees it too, so it is never lapped.
      uint32_t c = 0, nq[2] = {0, 0};
      int it = 0;
      for (int unit = blockIdx.x; unit >= 0; unit = next_unit(it++)) {
        const UnitView v = view_unit(p, t, unit);
        uint32_t* bad0 = s_bad + (nq[0] % kBadUnits) * (kBadWords + 1);
        uint32_t* bad1 = s_bad + (kBadUnits + nq[1] % kBadUnits) * (kBadWords + 1);
        nq[0] += v.x.n[0] > 0;
        nq[1] += v.x.n[1] > 0;
        bool ok = true;
        for (int j = 0; j < 2 * v.n_max; ++j, ++c) {   // K and V tiles
          const uint32_t st = c % kStages;
          ok = warp_wait(&kv_full[st], (c / kStages) & 1, s_abort, p.err);
          if (!ok) break;
          const int key0 = (v.x.j0 + (j >> 1)) * kTile;
          if ((j & 1) && key0 + kTile > v.all_see) {
            if (key0 <= v.all_see || j == 1) {         // the first one of the unit
              if (lane <= kBadWords) bad0[lane] = bad1[lane] = 0;
              __syncwarp();
            }
            clean_values<kFp16>(sKV + st * kTileBytes, key0, v.all_see, v.vis_end, bad0, bad1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_clean[st]);
          }
          if (lane == 0) mbar_arrive(&kv_empty[st]);
          __syncwarp();
        }
        if (!ok) break;
      }
    }
  } else {
    // ---------------- softmax ----------------
    const int i = warp >> 2;                           // tile A or B
    const int row = (warp & 3) * 32 + lane;            // packed row of the tile
    const int tok = row / p.G;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tb = tmem + lane_off + i * kTile;   // the two score buffers
    const uint32_t to = tb + 2 * kTile;
    const float c = p.scale_log2;
    uint32_t nq = 0, ph = 0;                           // units of this tile, phases of its buffers
    int it = 0;
    for (int unit = blockIdx.x; unit >= 0; unit = next_unit(it++)) {
      int n_tiles, lim, lim_warp;      // lim: the last of this thread's columns its row sees
      bool valid;
      {
        const UnitView u = view_unit(p, t, unit);
        n_tiles = i ? u.x.n[1] : u.x.n[0];
        valid = tok < (i ? u.x.ntok[1] : u.x.ntok[0]);
        const int first = u.s.pos0 + u.x.tok0 + i * p.tok - u.x.j0 * kTile;
        lim = first + tok;
        lim_warp = first + ((warp & 3) * 32) / p.G;    // the warp's first row
      }
      // A warp without a row of the unit only passes its turns on: what it leaves in
      // P reaches its own rows of O alone, which nobody reads.  Single rows of 8 heads
      // need one warp in four, and the power goes where it is used (16 rows over 5K
      // to 16K keys under the power cap: 171 -> 163 us).
      const bool live = __any_sync(0xFFFFFFFFu, valid);
      float m = -INFINITY;
      float2 sum = make_float2(0.f, 0.f);                // even and odd columns
      bool ok = true;
      if (!live) {
#pragma unroll 1
        for (int j = 0; j < 2 * n_tiles; ++j) {
          ok = warp_wait(&s_full[2 * i + (j & 1)], (ph >> (j & 1)) & 1, s_abort, p.err);
          if (!ok) break;
          ph ^= 1u << (j & 1);
          tc_fence_before();                           // the last unit's loads of O
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[2 * i + (j & 1)]);
          __syncwarp();
        }
      }
      const int steps = live ? 2 * n_tiles : 0;
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        {
          const int hf = j & 1;
          ok = warp_wait(&s_full[2 * i + hf], (ph >> hf) & 1, s_abort, p.err);
          if (!ok) break;
          ph ^= 1u << hf;
          tc_fence_after();
          const uint32_t ts = tb + hf * kStep;           // scores, then P
          float v[2][32];
          tmem_ld32_async(ts, v[0]);
          tmem_ld32_async(ts + 32, v[1]);
          tmem_wait_ld(v[0]);
          tmem_wait_ld(v[1]);
          if (lim_warp < kStep - 1) {
            mask_from<0>(v[0], lim);
            mask_from<32>(v[1], lim);
          }
          lim -= kStep;
          lim_warp -= kStep;
          const float mx = max_nan(max32(v[0]), max32(v[1]));
          // The maximum moves when a row's scores pass it by more than kSlack
          // (or are NaN).
          if (j == 0) {
            m = mx;
          } else if (__any_sync(0xFFFFFFFFu, valid && !((mx - m) * c <= kSlack))) {
            // the other buffer's next phase: O += P V of the last step is done
            ok = warp_wait(&s_full[2 * i + 1 - hf], (ph >> (1 - hf)) & 1, s_abort, p.err);
            if (!ok) break;
            tc_fence_after();
            const float was = m;
            m = max_nan(m, mx);
            const float k = m > was ? ex2((was - m) * c) : 1.f;
            sum.x *= k;
            sum.y *= k;
            rescale_row(to, k);
          }
          const float off = m == -INFINITY ? 0.f : fmaf(-m, c, kLift<kFp16>);
          exp_store<kFp16>(v[0], c, off, sum, ts);
          exp_store<kFp16>(v[1], c, off, sum, ts + 16);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[2 * i + hf]);
          __syncwarp();
        }
      }
      if (n_tiles > 0) {
        // the last products
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (ok) ok = warp_wait(&s_full[2 * i + hf], (ph >> hf) & 1, s_abort, p.err);
          ph ^= 1u << hf;
        }
        if (lane == 0) mbar_arrive(&s_seen[i]);        // the next unit's scores may come
        __syncwarp();
        if (ok) ok = warp_wait(&o_full[i], nq & 1, s_abort, p.err);
      }
      if (ok) {
        tc_fence_after();
        // the unit's place again: holding it through the loop would spill
        int again = unit;
        asm volatile("" : "+r"(again));
        const UnitView u = view_unit(p, t, again);
        const int tok0 = u.x.tok0 + i * p.tok, pos = u.s.pos0 + tok0 + tok;
        const float l = sum.x + sum.y;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse2 = l == 0.f ? -INFINITY : m * c + (log2f(l) - kLift<kFp16>);
        const int r = tok0 + tok, head = u.x.head * p.G + row % p.G;
        const bool split = u.s.nsplit > 1;
        const int64_t pv = u.s.part0 + ((int64_t)u.x.part * u.s.rows + r) * p.Hq + head;
        if (valid) {
          if (split) p.part_lse[pv] = lse2;
          else if (p.lse) p.lse[(int64_t)(u.s.q0 + r) * p.Hq + head] = lse2 * 0.6931471805599453f;
        }
        if (n_tiles > 0 && live) {
          const uint32_t* bad = s_bad + (i * kBadUnits + nq % kBadUnits) * (kBadWords + 1);
          // without a checked tile in this part the notes are an older unit's
          const bool any_bad = (u.x.j0 + u.n_max) * kTile > u.all_see && bad[kBadWords] != 0;
          // Rows leave through shared memory, 128 bytes of each at a time, so that
          // 8 lanes store one row's 128 bytes: stored by its own thread, a row
          // costs a transaction per 16 bytes (12,000 cycles per unit).
          uint8_t* dst = split ? reinterpret_cast<uint8_t*>(p.part_o + pv * kHeadDim)
                               : reinterpret_cast<uint8_t*>(p.out.ptr + (int64_t)(u.s.q0 + r) * p.out.rs +
                                                            (int64_t)head * p.out.hs);
          if (!valid) dst = nullptr;
          uint8_t* const box = sO + warp * 32 * 128;
          const uint32_t my = smem_u32(box) + lane * 128;
          const float mul = l == 0.f ? 0.f : inv;
          // `b`-th 128 bytes of the rows: from the box to their places
          auto flush = [&](int b) {
            if (any_bad && valid)
              add_not_finite<kFp16>(box + lane * 128, lane & 7, split, b, bad,
                                    u.all_see / kTile * kTile, pos,
                                    p.v.ptr + u.s.k0 * p.v.rs + (int64_t)u.x.head * p.v.hs, p.v.rs);
            __syncwarp();
            uint4 w[8];
            unsigned long long at[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) {
              const int rr = f * 4 + (lane >> 3);
              at[f] = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(dst), rr);
              w[f] = *reinterpret_cast<const uint4*>(box + rr * 128 + (((lane ^ rr) & 7) * 16));
            }
#pragma unroll
            for (int f = 0; f < 8; ++f)
              asm volatile(
                  "{\n\t.reg .pred p;\n\tsetp.ne.u64 p, %5, 0;\n\t"
                  "@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(at[f] + b * 128 + (lane & 7) * 16),
                  "r"(w[f].x), "r"(w[f].y), "r"(w[f].z), "r"(w[f].w), "l"(at[f])
                  : "memory");
            __syncwarp();
          };
          auto put = [&](int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             my + ((chunk ^ (lane & 7)) * 16)),
                         "r"(x), "r"(y), "r"(z), "r"(w)
                         : "memory");
          };
          __syncwarp();                                // TMEM loads are the whole warp's
          if (split) {
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              float o[32];
              tmem_ld32_async(to + b * 32, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int f = 0; f < 8; ++f)
                put(f, __float_as_uint(o[4 * f] * mul), __float_as_uint(o[4 * f + 1] * mul),
                    __float_as_uint(o[4 * f + 2] * mul), __float_as_uint(o[4 * f + 3] * mul));
              flush(b);
            }
          } else {
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
              float o[2][32];
              tmem_ld32_async(to + b * 64, o[0]);
              tmem_ld32_async(to + b * 64 + 32, o[1]);
              tmem_wait_ld(o[0]);
              tmem_wait_ld(o[1]);
              __half2 most = __float2half2_rn(0.f);
#pragma unroll
              for (int f = 0; f < 8; ++f) {
                const float* e = o[f >> 2] + (f & 3) * 8;
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  w[i] = pack2<kFp16>(e[2 * i] * mul, e[2 * i + 1] * mul);
                  if constexpr (kFp16)
                    most = __hmax2(most, __habs2(*reinterpret_cast<const __half2*>(&w[i])));
                }
                put(f, w[0], w[1], w[2], w[3]);
              }
              // A mean is no larger than its largest value, but weights that round up
              // can carry one near fp16's end past it: what is finite stays so.  (In
              // bf16 the last step before infinity is wider than that.)
              if (kFp16 && __hgt2_mask(most, __float2half2_rn(65504.f))) {
#pragma unroll
                for (int f = 0; f < 8; ++f) {
                  const float* e = o[f >> 2] + (f & 3) * 8;
                  uint32_t w[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float x = e[2 * i] * mul, y = e[2 * i + 1] * mul;
                    w[i] = hold_finite(pack2<kFp16>(x, y), x, y);
                  }
                  put(f, w[0], w[1], w[2], w[3]);
                }
              }
              flush(b);
            }
          }
        }
      }
      if (!ok) break;
      if (n_tiles > 0) ++nq;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Rows as a 3-D tensor [rows][heads][128] read in boxes of 64 elements x
// box_heads x box_rows (64 elements = one 128-byte swizzled row).
bool encode_map(CUtensorMap* map, const Rows16& r, bool fp16, int64_t rows, int heads,
                int box_heads, int box_rows) {
  auto enc = get_tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)rows};
  // a stride that no step uses must still be a valid one
  const cuuint64_t strides[2] = {(cuuint64_t)(r.hs ? r.hs : kHeadDim) * 2,
                                 (cuuint64_t)(r.rs ? r.rs : kHeadDim) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             r.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_prompt(const AttnHandle& h, const Rows16& q, const Rows16& k, const Rows16& v,
                          int64_t q_rows, int64_t k_rows, const AttnTable& t, const Rows16& out,
                          float* lse, float* part_o, float* part_lse, int* err,
                          cudaStream_t stream) {
  if (t.units <= 0) return cudaSuccess;
  PromptParams p;
  p.Hq = h.cfg.Hq;
  p.Hkv = h.cfg.Hkv;
  p.G = h.G;
  p.tok = kTile / h.G;
  p.scale_log2 = h.scale_log2;
  p.v = v;
  p.out = out;
  p.lse = lse;
  p.part_o = part_o;
  p.part_lse = part_lse;
  p.err = err;
  CUtensorMap qm, km, vm;
  if (!encode_map(&qm, q, h.fp16, q_rows, h.cfg.Hq, h.G, p.tok) ||
      !encode_map(&km, k, h.fp16, k_rows, h.cfg.Hkv, 1, kTile) ||
      !encode_map(&vm, v, h.fp16, k_rows, h.cfg.Hkv, 1, kTile))
    return cudaErrorInvalidValue;
  auto* fn = h.fp16 ? prompt_kernel<true> : prompt_kernel<false>;
  static std::atomic<uint64_t> done[2];
  cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(fn), (int)kSmemBytes, &done[h.fp16 ? 1 : 0]);
  if (e != cudaSuccess) return e;
  profile_before(DOSA_KERNEL_PROMPT, stream);
  fn<<<t.units, kThreads, kSmemBytes, stream>>>(qm, km, vm, t, p);
  e = cudaGetLastError();
  profile_after(DOSA_KERNEL_PROMPT, stream);
  return e;
}

}  // namespace dosa
