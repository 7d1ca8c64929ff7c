// The 4-bit cache's append and read kernels: rows of 16-bit keys and values
// quantised into their slots, and slots read back as rows.
//
// Both are memory work (256 bytes of rows and 80 of cache per vector) with
// nearly as much to issue: 8,289 tokens of 8 heads are appended and read back in
// 20 us, 12 for the bytes, with 64 and 58 % of the issue slots used and warps that
// mostly wait for loads: neither is full.  Four
// lanes take one head vector and a warp 8 consecutive tokens of one head, so
// the head-major cache is accessed in 512-byte runs of codes and 128-byte runs
// of parameters.  Append: a lane quantises one group of 32 dimensions alone (no
// reduction over lanes), then the four lanes transpose their code words so that
// each stores 16 contiguous bytes.  Read: a lane takes 16 bytes of codes, which
// hold 8 dimensions of every group, and stores four 16-byte pieces; the four
// lanes' pieces make 64-byte runs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_internal.h"

namespace dosa {
namespace {

constexpr int kTok = 8;            // tokens per warp
constexpr int kMaxThreads = 256;

template <bool kFp16>
__device__ __forceinline__ float widen_lo(uint32_t w) {
  if constexpr (kFp16) return __low2float(*reinterpret_cast<const __half2*>(&w));
  return __uint_as_float(w << 16);
}
template <bool kFp16>
__device__ __forceinline__ float widen_hi(uint32_t w) {
  if constexpr (kFp16) return __high2float(*reinterpret_cast<const __half2*>(&w));
  return __uint_as_float(w & 0xFFFF0000u);
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

// The vector of four lanes.  A CTA takes 8 tokens, its warps the key heads' keys
// and values (2 per head; further heads along grid.y), so concurrent warps
// share the rows' DRAM pages.
struct Vec {
  int row;          // row of the call
  int64_t slot;
  int head, val;
};
__device__ __forceinline__ bool vec_of(const AttnTable& t, int Hkv, Vec& v) {
  const int hv = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  v.val = hv & 1;
  v.head = hv >> 1;
  const int r = blockIdx.x * kTok + ((threadIdx.x & 31) >> 2);
  if (r >= t.units || v.head >= Hkv) return false;
  // unit0 counts the launch's rows
  const int i = find_seq(t.n, r, [&](int m) { return t.s[m].unit0; });
  const AttnSeq& s = t.s[i];
  const int k = r - s.unit0;
  v.row = s.q0 + k;
  v.slot = s.k0 + s.pos0 + k;
  return true;
}

// Minimum and maximum of packed pairs; NaN stays.
template <bool kFp16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (kFp16) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool kFp16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (kFp16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <bool kFp16>
__global__ void __launch_bounds__(kMaxThreads, 4) append_kernel(const __grid_constant__ AttnTable t,
                                                          Cache4View c, Rows16 k, Rows16 v,
                                                          int Hkv) {
  const int g = threadIdx.x & 3;                   // group of 32 dimensions
  Vec o;
  const bool on = vec_of(t, Hkv, o);
  grid_wait();
  grid_release();
  if (!__any_sync(0xFFFFFFFFu, on)) return;
  uint32_t v2[16];                                 // the group's 32 elements, packed
  {
    const Rows16 src = on && o.val ? v : k;
    const uint16_t* at = src.ptr + (on ? (int64_t)o.row * src.rs + (int64_t)o.head * src.hs : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = on ? __ldg(reinterpret_cast<const uint4*>(at + 32 * g + 8 * i))
                         : make_uint4(0, 0, 0, 0);
      v2[4 * i] = u.x;
      v2[4 * i + 1] = u.y;
      v2[4 * i + 2] = u.z;
      v2[4 * i + 3] = u.w;
    }
  }
  uint32_t lo2 = v2[0], hi2 = v2[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    lo2 = min2<kFp16>(lo2, v2[i]);
    hi2 = max2<kFp16>(hi2, v2[i]);
  }
  lo2 = min2<kFp16>(lo2, lo2 >> 16);
  hi2 = max2<kFp16>(hi2, hi2 >> 16);
  const float lo = widen_lo<kFp16>(lo2), hi = widen_lo<kFp16>(hi2);
  // scale and min round to fp16; the codes are relative to the rounded ones
  const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
  const __half hm = __float2half_rn(lo);
  // a NaN or infinite element makes the range or the minimum so
  const bool nan = __hisnan(hs) || __hisinf(hs) || __hisinf(hm);
  const float s = __half2float(hs), m = __half2float(hm);
  uint32_t w[4] = {0, 0, 0, 0};                    // dimensions 32 g + 8 i .. + 7
  if (!nan && s > 0.f) {
    // The quotient (x - min) / scale, rounded to fp32 on its way to the integer: a
    // product with the rounded reciprocal and one correction by the exact remainder
    // (P. Markstein, "Computation of elementary functions on the IBM RISC
    // System/6000 processor", 1990: correctly rounded from a correctly rounded
    // reciprocal).  Adding 1.5 2^23 rounds it to an integer (ties to even) in the sum's low bits.
    constexpr float kMagic = 12582912.f;
    const float r = __frcp_rn(s);
    // codes leave 0..15 only where the rounding of min or scale is not small
    // against the scale: then every quotient is clamped first
    const bool clamp = __fsub_rn(lo, m) * r < -0.49f || __fsub_rn(hi, m) * r > 15.49f;
    // x - min is not exact in fp32 where one of them is below 2^-13 of the other, and
    // its rounding may meet a half-integer multiple of the scale that x - min itself
    // misses.  Rounded to odd it never does (such a multiple has fewer bits), and the
    // quotient of a difference that misses misses the half by more than its own
    // rounding.  Only two kinds of group can need it: minima next to a half-integer
    // multiple of the scale with an element that is small against them (below 2^-16
    // of the minimum in bf16, where only the multiple itself is near enough, 2^-13 in
    // fp16), and minima that are small against the maximum.  One group in 250 of
    // bf16 activations is next to a multiple (fp16: in 120), next to none has the
    // small element too; taking all of the former the careful way cost 9 %.
    constexpr float kNear = kFp16 ? 0x1p-11f : 0x1p-15f;
    const float near = fmaf(-2.f * m, r, kMagic) - kMagic;   // halves of a scale in -min
    bool odd = fabsf(m) * 4096.f < hi && m != 0.f;
    if (fabsf(fmaf(near, s, 2.f * m)) <= kNear * fabsf(m)) {
      // the smallest element that is not zero, less one in its bits (zero wraps)
      const float far = fabsf(m) * 0x1p-12f;
      const uint32_t bits = kFp16 ? (uint32_t)__half_as_ushort(__float2half_ru(far))
                                  : (__float_as_uint(far) >> 16) + 1u;
      uint32_t least = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        least = __vminu2(least, __vsub2(v2[i] & 0x7FFF7FFFu, 0x00010001u));
      odd |= min(least & 0xFFFFu, least >> 16) < bits;
    }
    auto code = [&](float x, bool hold) {
      float d = __fsub_rn(x, m);
      if (hold) {
        const float lower = __fsub_rd(x, m), upper = __fsub_ru(x, m);
        if (lower != upper) d = __float_as_uint(lower) & 1u ? lower : upper;
      }
      float q = d * r;
      q = fmaf(fmaf(-q, s, d), r, q);
      if (hold) q = fminf(fmaxf(q, 0.f), 15.f);
      return __float_as_uint(q + kMagic);
    };
    auto encode = [&](bool hold) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum += code(widen_lo<kFp16>(v2[4 * i + j]), hold) << (8 * j);
          sum += code(widen_hi<kFp16>(v2[4 * i + j]), hold) << (8 * j + 4);
        }
        // the magic number's own bits, summed over the eight places
        w[i] = sum - 0x4B400000u * 0x11111111u;
      }
    };
    if (clamp || odd) encode(true);
    else encode(false);
  }
  // transpose: lane c gets word c of every group
  uint32_t y[4];
#pragma unroll
  for (int k2 = 0; k2 < 4; ++k2) {
    // lane g sends word g ^ k2 to lane g ^ k2
    const int to = g ^ k2;
    const uint32_t send = to == 0 ? w[0] : to == 1 ? w[1] : to == 2 ? w[2] : w[3];
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, send, k2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((g ^ k2) == i) y[i] = got;
  }
  if (!on) return;
  uint4 out;
  if (o.val) {
    // 16-bit pieces: row 2c is the low halves of the groups' words, 2c + 1 the high
    out = make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410),
                     __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632));
  } else {
    out = make_uint4(y[0], y[1], y[2], y[3]);
  }
  const int64_t at = (int64_t)o.head * c.cap + o.slot;
  reinterpret_cast<uint4*>((o.val ? c.vc : c.kc) + at * kVecCodes)[g] = out;
  reinterpret_cast<uint32_t*>((o.val ? c.vp : c.kp) + at * kVecParams)[g] =
      nan ? 0x7FFF7FFFu
          : (uint32_t)__half_as_ushort(hs) | ((uint32_t)__half_as_ushort(hm) << 16);
  if (c.weight && o.val == 0 && o.head == 0 && g == 0) c.weight[o.slot] = 0.f;
}

template <bool kFp16>
__global__ void __launch_bounds__(kMaxThreads) read_kernel(const __grid_constant__ AttnTable t,
                                                        Cache4View c, Rows16 k, Rows16 v,
                                                        int Hkv) {
  const int q = threadIdx.x & 3;                   // chunk: dimensions 32 g + 8 q .. + 7
  Vec o;
  const bool on = vec_of(t, Hkv, o);
  grid_wait();
  grid_release();
  if (!on) return;
  const int64_t at = (int64_t)o.head * c.cap + o.slot;
  uint4 w = __ldg(reinterpret_cast<const uint4*>((o.val ? c.vc : c.kc) + at * kVecCodes) + q);
  const uint4 pr = __ldg(reinterpret_cast<const uint4*>((o.val ? c.vp : c.kp) + at * kVecParams));
  if (o.val)
    w = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),
                   __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
  const uint32_t cw[4] = {w.x, w.y, w.z, w.w}, pw[4] = {pr.x, pr.y, pr.z, pr.w};
  const Rows16 dst = o.val ? v : k;
  uint16_t* out = dst.ptr + (int64_t)o.row * dst.rs + (int64_t)o.head * dst.hs + 8 * q;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&pw[g]));
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)                    // the product is exact: one rounding to fp32
      x[j] = fmaf(sm.x, (float)((cw[g] >> (4 * j)) & 15u), sm.y);
    *reinterpret_cast<uint4*>(out + 32 * g) =
        make_uint4(pack2<kFp16>(x[0], x[1]), pack2<kFp16>(x[2], x[3]), pack2<kFp16>(x[4], x[5]),
                   pack2<kFp16>(x[6], x[7]));
  }
}

struct Shape {
  dim3 grid;
  unsigned threads;
};
Shape shape_for(const AttnTable& t, int Hkv) {
  Shape s;
  const int warps = 2 * Hkv < kMaxThreads / 32 ? 2 * Hkv : kMaxThreads / 32;
  s.threads = 32u * warps;
  s.grid = dim3((unsigned)((t.units + kTok - 1) / kTok), (unsigned)((2 * Hkv + warps - 1) / warps));
  return s;
}

}  // namespace

cudaError_t launch_cache_append(const AttnHandle& h, const Cache4View& c, const Rows16& k,
                                const Rows16& v, const AttnTable& t, cudaStream_t stream) {
  if (t.units <= 0) return cudaSuccess;
  profile_before(DOSA_KERNEL_CACHE, stream);
  const Shape g = shape_for(t, h.cfg.Hkv);
  const cudaError_t e = launch_after(h.fp16 ? append_kernel<true> : append_kernel<false>, g.grid,
                                     g.threads, 0, stream, t, c, k, v, h.cfg.Hkv);
  profile_after(DOSA_KERNEL_CACHE, stream);
  return e;
}

cudaError_t launch_cache_read(const AttnHandle& h, const Cache4View& c, const Rows16& k,
                              const Rows16& v, const AttnTable& t, cudaStream_t stream) {
  if (t.units <= 0) return cudaSuccess;
  profile_before(DOSA_KERNEL_CACHE, stream);
  const Shape g = shape_for(t, h.cfg.Hkv);
  const cudaError_t e = launch_after(h.fp16 ? read_kernel<true> : read_kernel<false>, g.grid,
                                     g.threads, 0, stream, t, c, k, v, h.cfg.Hkv);
  profile_after(DOSA_KERNEL_CACHE, stream);
  return e;
}

}  // namespace dosa
