// What the kernels that write and read cache rows and 8-bit codes share: exact and correctly
// rounded arithmetic on bf16 values, the scales of codes, rotations, and where a token's row is.
#pragma once

#include "mla_common.cuh"

namespace mla {
namespace rows {

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// (a + b) as an exact pair (Knuth's TwoSum).
__device__ __forceinline__ void two_sum(float a, float b, float& hi, float& lo) {
  hi = __fadd_rn(a, b);
  const float z = __fsub_rn(hi, a);
  lo = __fadd_rn(__fsub_rn(a, __fsub_rn(hi, z)), __fsub_rn(b, z));
}

// a * b + c rounded to odd.
__device__ __forceinline__ float fma_odd(float a, float b, float c) {
  const float down = __fmaf_rd(a, b, c), up = __fmaf_ru(a, b, c);
  return __float_as_uint(down) & 1u ? down : up;
}

// a * b + c in fp32 of bf16 values a and b (the low 16 bits of each), rounded once to nearest, down or up: the
// instruction takes the halves of a word as they are, which saves their unpacking.  A product alone adds -0, so that a
// zero keeps its sign.
__device__ __forceinline__ float bf_fma(uint32_t a, uint32_t b, float c) {
  float d;
  asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"((uint16_t)a), "h"((uint16_t)b), "f"(c));
  return d;
}
__device__ __forceinline__ float bf_fma_rd(uint32_t a, uint32_t b, float c) {
  float d;
  asm("fma.rm.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"((uint16_t)a), "h"((uint16_t)b), "f"(c));
  return d;
}
__device__ __forceinline__ float bf_fma_ru(uint32_t a, uint32_t b, float c) {
  float d;
  asm("fma.rp.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"((uint16_t)a), "h"((uint16_t)b), "f"(c));
  return d;
}
__device__ __forceinline__ float bf_mul(uint32_t a, uint32_t b) { return bf_fma(a, b, -0.f); }
__device__ __forceinline__ float bf_fma_odd(uint32_t a, uint32_t b, float c) {   // rounded to odd
  const float down = bf_fma_rd(a, b, c), up = bf_fma_ru(a, b, c);
  return __float_as_uint(down) & 1u ? down : up;
}

// Two floats as a bf16 pair, the first in the low half; nearest, ties to even.
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A double as a float rounded to odd (truncated, the last bit set if anything was dropped).
__device__ __forceinline__ float double_odd(double x) {
  const float f = __double2float_rz(x);
  return isfinite(f) && (double)f != x ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

// 1 / sqrt(v) as ih + il, il >= 0, to some 2^-44 of its value (infinity and 0 for v = 0): v = vh + vl, vh the
// sum rounded, 2^-100 <= vh <= 2^100 or 0.  One Newton step of third order on the fp32 root, its residual
// 1 - v r^2 formed from exact products.  (In fp64 it takes some 30 operations, at a 64th of fp32's rate
// the longest part of a short row's work.)
__device__ __forceinline__ void rsqrt_pair(float vh, float vl, float& ih, float& il) {
  const float r = rsqrtf(vh);
  const float ph = __fmul_rn(r, r), pl = __fmaf_rn(r, r, -ph);
  const float qh = __fmul_rn(vh, ph), ql = __fmaf_rn(vh, ph, -qh);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(1.f, qh), ql), __fmaf_rn(vh, pl, __fmul_rn(vl, ph)));
  const float c = __fmul_rn(r, __fmul_rn(e, __fmaf_rn(e, 0.375f, 0.5f)));
  two_sum(r, c, ih, il);
  if (il < 0.f) {
    const float below = __uint_as_float(__float_as_uint(ih) - 1u);
    il = __fadd_rn(__fsub_rn(ih, below), il);
    ih = below;
  }
  if (vh == 0.f) {
    ih = __uint_as_float(0x7F800000u);
    il = 0.f;
  }
}
// hi + lo (an unevaluated sum) times 1 / n = nh + nl, plus eps, as vh + vl.
__device__ __forceinline__ void mean_plus(float hi, float lo, float nh, float nl, float eps, float& vh, float& vl) {
  const float p = __fmul_rn(hi, nh), pe = __fadd_rn(__fmaf_rn(hi, nh, -p), __fmaf_rn(hi, nl, __fmul_rn(lo, nh)));
  float s, se;
  two_sum(p, eps, s, se);
  two_sum(s, __fadd_rn(se, pe), vh, vl);
}

// Two floats worked on at once (one instruction for both).
typedef unsigned long long float2x;
__device__ __forceinline__ float2x both(float lo, float hi) {
  float2x r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void apart(float2x v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ float2x add2(float2x a, float2x b) {
  float2x r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2x sub2(float2x a, float2x b) {
  float2x r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2x mul2(float2x a, float2x b) {
  float2x r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2x fma2(float2x a, float2x b, float2x c) {
  float2x r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float2x fma2_rz(float2x a, float2x b, float2x c) {
  float2x r;
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float2x mul2_rz(float2x a, float2x b) {
  float2x r;
  asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Products of bf16 pairs, and with a sum.
__device__ __forceinline__ float2x bf_mul2(uint32_t a, uint32_t b) { return both(bf_mul(a, b), bf_mul(a >> 16, b >> 16)); }
__device__ __forceinline__ float2x bf_fma2(uint32_t a, uint32_t b, float2x c) {
  float lo, hi;
  apart(c, lo, hi);
  return both(bf_fma(a, b, lo), bf_fma(a >> 16, b >> 16, hi));
}
// A bf16 pair as two floats, and back (nearest, ties to even).
__device__ __forceinline__ float2x widen2(uint32_t v) { return both(lo_f(v), hi_f(v)); }
__device__ __forceinline__ uint32_t pack2(float2x v) {
  float lo, hi;
  apart(v, lo, hi);
  return pack(lo, hi);
}

// The least e with amax <= 7 * 2^(e - 3 + over), from bits of a bf16 magnitude: its exponent
// field counts from 2^-127, a subnormal's leading bit is found by counting.  0 for zero.
__device__ __forceinline__ int scale_exponent(uint32_t mag, int over, int low, int high) {
  if (mag == 0) return 0;
  int k = (int)(mag >> 7) - 127;
  uint32_t frac = mag & 0x7Fu;
  if ((mag >> 7) == 0) {
    const int s = __clz(frac) - 25;   // the leading one of 7 fraction bits of 2^-126
    k = -127 - s;
    frac = (frac << (s + 1)) & 0x7Fu;
  }
  const int e = k - over + (frac > 0x60u ? 1 : 0);   // 1.75 = 1 + 0x60 / 128
  return min(max(e, low), high);
}
// 2^e as a float, e >= -149; -e of a clamped exponent is never below -127
__device__ __forceinline__ float pow2(int e) {
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

// Eight values (packed bf16 pairs) as eight e4m3 codes of y * rs, rs the bits of a power of two as a bf16 value.
__device__ __forceinline__ uint2 e4m3_codes(const uint32_t (&y)[4], uint32_t rs) {
  uint32_t two[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = make_float2(bf_mul(y[i], rs), bf_mul(y[i] >> 16, rs));
    two[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(two[0] | (two[1] << 16), two[2] | (two[3] << 16));
}

// `turn` for products that fp32 does not hold.
__device__ __forceinline__ uint32_t turn_wide(uint32_t x, uint32_t f) {
  const double x0 = lo_f(x), x1 = hi_f(x), c = lo_f(f), s = hi_f(f);
  return pack(double_odd(add_odd(x0 * c, -(x1 * s))), double_odd(add_odd(x0 * s, x1 * c)));
}
// The pair (x0, x1) of `x` turned by (cos, sin) of `f`, as a bf16 pair.  Products of bf16 values
// are exact in fp32's normal range; `lost` becomes other than 0 where one is not (what it lost, rounded up, is
// +0 only if that is nothing).
__device__ __forceinline__ uint32_t turn(uint32_t x, uint32_t f, uint32_t& lost) {
  const uint32_t x1 = x >> 16, s = f >> 16;
  const float p = bf_mul(x1, s), r = bf_mul(x1, f);
  lost |= __float_as_uint(bf_fma_ru(x1, s, -p)) | __float_as_uint(bf_fma_ru(x1, f, -r));
  return pack(bf_fma_odd(x, f, -p), bf_fma_odd(x, s, r));
}
// 16 bytes of pairs.
static __device__ __noinline__ uint4 turn_wide(uint4 x, uint4 f) {
  return make_uint4(turn_wide(x.x, f.x), turn_wide(x.y, f.y), turn_wide(x.z, f.z), turn_wide(x.w, f.w));
}
__device__ __forceinline__ uint4 turn(uint4 x, uint4 f, uint32_t& lost) {
  return make_uint4(turn(x.x, f.x, lost), turn(x.y, f.y, lost), turn(x.z, f.z, lost), turn(x.w, f.w, lost));
}

struct Place {
  long long pos;   // -1: the token is left alone
  long long row;   // physical cache row
};

// Whole warp: where the tokens t of a call go, a token a group of `lanes` neighbours (a power of two up to
// 32; t is the group's, `sub` the lane's place in it).  `A` holds the call's offsets, cache_lens,
// block_table, bt_stride, ps, num_pages, B, max_seq_len and hdr.  The request is the last b with
// offsets[b] <= t, found by `lanes` probes a round (at 32, two rounds up to 1024 requests).  Tokens at or
// past offsets[B] belong to nobody and are skipped; a position or page out of range is reported.
template <class A>
__device__ __forceinline__ Place locate_groups(const A& a, int t, int lanes, int sub) {
  Place p{-1, 0};
  int lo = 0, n = a.B;   // candidates [lo, lo + n)
  const uint32_t end = a.offsets[a.B];
  const int first = (int)(threadIdx.x & 31) - sub, shift = 31 - __clz(lanes);
  const uint32_t mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1) << first;
  while (__any_sync(0xffffffffu, n > 1)) {
    const int step = (n + lanes - 1) >> shift;
    const int probe = sub * step;
    const bool below = probe < n && a.offsets[lo + probe] <= (uint32_t)t;
    const int cnt = __popc(__ballot_sync(0xffffffffu, below) & mask);
    const int skip = cnt > 0 ? (cnt - 1) * step : 0;
    lo += skip;
    n = min(step, n - skip);
  }
  const uint32_t qb = a.offsets[lo], qe = a.offsets[lo + 1], len = a.cache_lens[lo];
  if ((uint32_t)t >= end) return p;
  const long long pos = (long long)len - qe + t;
  bool ok = qb <= (uint32_t)t && (uint32_t)t < qe && pos >= 0 && pos < a.max_seq_len &&
            pos < (long long)a.bt_stride * a.ps;
  if (ok) {
    const int page = a.block_table[(size_t)lo * a.bt_stride + pos / a.ps];
    ok = page >= 0 && page < a.num_pages;
    p.row = (long long)page * a.ps + pos % a.ps;
  }
  if (ok) p.pos = pos;
  else if (sub == 0) atomicOr(&a.hdr->status, kDeviceCheckFailed);
  return p;
}
// One token for the whole warp.
template <class A>
__device__ __forceinline__ Place locate(const A& a, int t, int lane) {
  return locate_groups(a, t, 32, lane);
}

}  // namespace rows
}  // namespace mla
