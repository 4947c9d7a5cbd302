// mla_cache_append: the query tokens' new latent rows enter the paged cache.  For
// token t of request b at pos = cache_len - qlen + i, with new row [c (L) ; r (R)]:
//
//   y    = bf16( c / sqrt(mean(c^2) + eps) * gamma )            (rounded once)
//   rope = bf16( r turned by freqs_cis[pos] )                    (rounded once)
//   row  = [y ; rope] in the cache's format; the query's rope part is turned alike.
//
// bf16 stores y.  e4m3 stores y / s with one power of two s per row, e2m1 stores
// y / s with one power of two s per 32 values: the division is exact, so a stored
// code is the rounding of an exact value and depends on no order of operations.
//   e4m3: s = the least 2^e with amax <= 448 s (the format's largest value).
//   e2m1: s = the least 2^e with amax <= 7 s.  Values in (6 s, 7 s] become 6 s, off
//         by at most s, half the grid's step there; doubling s for them would double
//         the step under 2 s for all 32 values.
//
// Arithmetic.  The codes follow the last bit of y, so y is the correctly rounded
// value: squares of bf16 are exact in fp32 and are summed as an unevaluated pair
// hi + lo (Knuth's TwoSum); 1 / sqrt is taken once per row in fp64 and split into two
// floats; c * gamma is exact in fp32.  What is left is one fma, of an exact product and a
// small or exact term, and it is rounded to odd: of its value rounded down and rounded up
// the one whose last bit is set (the two are equal if it is exact).  Rounding that to
// bf16 rounds the exact value, since no odd fp32 number lies on a bf16 boundary.  The
// same goes for the rotations, where the one product that is rounded on its own is exact.  (With TwoSum and a rounding of the pair in integers, four
// times the operations, 8,483 prompt tokens took 262 us, twice the time of their bytes.)
// Rows and products outside the range in which these steps neither overflow nor
// underflow take fp64 (a rotation's sum there is rounded to odd from an exact pair).  Results equal mla_branch_prologue's bit for bit (bf16
// rows, queries; a NaN is a NaN).
//
// Layout.  A warp takes a row (16 consecutive values a lane: two lanes hold one group
// of 32); a block of 256 threads takes 16 KB of a token's queries, 16 bytes a thread
// four times, all loads out before the token's request is looked up.  Bound by HBM
// where queries are turned, by the chain of dependent reads (request, length, page,
// table) for a few tokens.
#include <cuda_fp4.h>

#include <cstdio>

#include "mla_kernels.cuh"

namespace mla {
namespace app {

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = kThreads / 32;
constexpr int kBatch = 4;                       // 16-byte pieces of the queries per thread
constexpr int kPieces = kThreads * kBatch;      // ... per block
constexpr int kMaxRope = 128;

struct Args {
  int fmt, H, N, R, L, ps, num_pages, B, T, max_seq_len, bt_stride;
  int row_blocks, q_blocks;        // blocks of rows; blocks per token of queries
  int step_h, step_c;              // heads and pieces that kThreads pieces of the queries come to
  long long row_bytes, new_stride; // cache row; elements between new rows
  double eps;
  const __nv_bfloat16* kv_new;     // [T, >= L+R]
  const __nv_bfloat16* q;          // [T, H, N+R]
  __nv_bfloat16* q_out;
  uint8_t* pool;
  float* scales;                   // e4m3: [rows]
  __nv_bfloat16* rows_out;         // [T, L+R] or NULL
  const uint32_t* offsets;
  const uint32_t* cache_lens;
  const int32_t* block_table;
  const __nv_bfloat16* freqs;
  const __nv_bfloat16* gamma;
  PlanHeader* hdr;
};

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

// `turn` for products that fp32 does not hold.
__device__ __forceinline__ uint32_t turn_wide(uint32_t x, uint32_t f) {
  const double x0 = lo_f(x), x1 = hi_f(x), c = lo_f(f), s = hi_f(f);
  return pack(double_odd(add_odd(x0 * c, -(x1 * s))), double_odd(add_odd(x0 * s, x1 * c)));
}
// The pair (x0, x1) of `x` turned by (cos, sin) of `f`, as a bf16 pair.  Products of bf16 values
// are exact in fp32's normal range; `lost` becomes other than 0 where one is not.
__device__ __forceinline__ uint32_t turn(uint32_t x, uint32_t f, uint32_t& lost) {
  const float x0 = lo_f(x), x1 = hi_f(x), c = lo_f(f), s = hi_f(f);
  const float p = __fmul_rn(x1, s), r = __fmul_rn(x1, c);
  lost |= product_lost(p, x1, s) | product_lost(r, x1, c);
  return pack(fma_odd(x0, c, -p), fma_odd(x0, s, r));
}
// 16 bytes of pairs.
__device__ __noinline__ uint4 turn_wide(uint4 x, uint4 f) {
  return make_uint4(turn_wide(x.x, f.x), turn_wide(x.y, f.y), turn_wide(x.z, f.z), turn_wide(x.w, f.w));
}
__device__ __forceinline__ uint4 turn(uint4 x, uint4 f, uint32_t& lost) {
  return make_uint4(turn(x.x, f.x, lost), turn(x.y, f.y, lost), turn(x.z, f.z, lost), turn(x.w, f.w, lost));
}

struct Place {
  long long pos;   // -1: the token is left alone
  long long row;   // physical cache row
};

// Whole warp: where token t goes.  The request is the last b with offsets[b] <= t,
// found by 32 probes a round (two rounds up to 1024 requests).  Tokens at or past
// offsets[B] belong to nobody and are skipped; a position or page out of range is
// reported.
__device__ __forceinline__ Place locate(const Args& a, int t, int lane) {
  Place p{-1, 0};
  int lo = 0, n = a.B;   // candidates [lo, lo + n)
  const uint32_t end = a.offsets[a.B];
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int probe = lane * step;
    const bool below = probe < n && a.offsets[lo + probe] <= (uint32_t)t;
    const int cnt = __popc(__ballot_sync(0xffffffffu, below));
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
  else if (lane == 0) atomicOr(&a.hdr->status, kDeviceCheckFailed);
  return p;
}

__device__ __forceinline__ void new_row(const Args& a, int t, int lane) {
  const __nv_bfloat16* src = a.kv_new + (size_t)t * a.new_stride;
  const int l0 = lane * 16;
  const bool have = l0 < a.L;   // L is a multiple of 32: a lane has 16 values or none
  uint32_t x[8] = {}, g[8] = {};
  if (have) {
    const uint4* sp = reinterpret_cast<const uint4*>(src + l0);
    const uint4 a0 = sp[0], a1 = sp[1];
    x[0] = a0.x; x[1] = a0.y; x[2] = a0.z; x[3] = a0.w;
    x[4] = a1.x; x[5] = a1.y; x[6] = a1.z; x[7] = a1.w;
    const uint4* gp = reinterpret_cast<const uint4*>(a.gamma + l0);
    const uint4 b0 = gp[0], b1 = gp[1];
    g[0] = b0.x; g[1] = b0.y; g[2] = b0.z; g[3] = b0.w;
    g[4] = b1.x; g[5] = b1.y; g[6] = b1.z; g[7] = b1.w;
  }
  uint32_t r[kMaxRope / 64];   // rope pairs lane, lane + 32
#pragma unroll
  for (int i = 0; i < kMaxRope / 64; ++i) {
    const int pr = lane + 32 * i;
    r[i] = pr < a.R / 2 ? reinterpret_cast<const uint32_t*>(src + a.L)[pr] : 0u;
  }
  const Place p = locate(a, t, lane);
  if (p.pos < 0) return;

  // mean square
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
  top = __reduce_max_sync(0xffffffffu, top);
  double sum;
  const float top_f = __uint_as_float(top << 16);
  if (top_f >= 0x1p-40f && top_f <= 0x1p55f) {
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e;
      two_sum(hi, __fmul_rn(lo_f(x[i]), lo_f(x[i])), hi, e);
      lo = __fadd_rn(lo, e);
      two_sum(hi, __fmul_rn(hi_f(x[i]), hi_f(x[i])), hi, e);
      lo = __fadd_rn(lo, e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
      float e;
      two_sum(hi, h2, hi, e);
      lo = __fadd_rn(__fadd_rn(lo, l2), e);
    }
    sum = (double)hi + (double)lo;
  } else {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum += (double)lo_f(x[i]) * (double)lo_f(x[i]);
      sum += (double)hi_f(x[i]) * (double)hi_f(x[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const double inv = rsqrt(sum / (double)a.L + a.eps);
  const float ih = (float)inv, il = (float)(inv - (double)ih);

  auto scaled = [&](float v, float gm) {   // v * inv * gm rounded to odd
    const float m = __fmul_rn(v, gm), am = fabsf(m);
    if (am >= 0x1p-40f && am <= 0x1p60f && ih >= 0x1p-60f && ih <= 0x1p60f) return fma_odd(m, ih, __fmul_rn(m, il));
    return double_odd((double)v * inv * (double)gm);
  };
  uint32_t y[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = have ? pack(scaled(lo_f(x[i]), lo_f(g[i])), scaled(hi_f(x[i]), hi_f(g[i]))) : 0u;
    amax = max(amax, max(y[i] & 0x7FFFu, (y[i] >> 16) & 0x7FFFu));
  }

  uint8_t* dst = a.pool + (size_t)p.row * a.row_bytes;
  uint8_t* dst_rope = dst + (a.row_bytes - 2 * a.R);
  uint32_t o[8];   // the values the stored row stands for
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = y[i];
  // the least e with amax <= 7 * 2^(e - 3 + over), from bits of a bf16 magnitude: its
  // exponent field counts from 2^-127, a subnormal's leading bit is found by counting
  auto exponent = [](uint32_t mag, int over, int low, int high) {
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
  };
  // 2^e as a float, e >= -149; -e of a clamped exponent is never below -127
  auto pow2 = [](int e) {
    return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << (e + 149));
  };
  if (a.fmt == MLA_CACHE_BF16) {
    if (have) {
      uint4* d = reinterpret_cast<uint4*>(dst + 2 * l0);
      d[0] = make_uint4(y[0], y[1], y[2], y[3]);
      d[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  } else if (a.fmt == MLA_CACHE_E4M3) {
    amax = __reduce_max_sync(0xffffffffu, amax);
    const bool bad = amax >= 0x7F80u;   // a NaN or an infinity: every code a NaN
    const int e = bad ? 0 : exponent(amax, 8, -126, 127);
    const float s = pow2(e), rs = pow2(-e);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t two[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t yy = y[2 * i + h];
        const float2 v = make_float2(lo_f(yy) * rs, hi_f(yy) * rs);
        two[h] = bad ? 0x7F7Fu : (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two[h], __NV_E4M3);
        const float2 back = __half22float2(__half2(hr));
        const __nv_bfloat162 b = __floats2bfloat162_rn(back.x * s, back.y * s);
        o[2 * i + h] = *reinterpret_cast<const uint32_t*>(&b);
      }
      w[i] = two[0] | (two[1] << 16);
    }
    if (have) *reinterpret_cast<uint4*>(dst + l0) = make_uint4(w[0], w[1], w[2], w[3]);
    if (lane == 0) a.scales[p.row] = s;
  } else {
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));   // two lanes hold 32 values
    const bool bad = amax >= 0x7F80u;
    const int e = bad ? 0 : exponent(amax, 2, -127, 127);
    const float s = pow2(e), rs = pow2(-e);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = make_float2(lo_f(y[i]) * rs, hi_f(y[i]) * rs);
      const uint32_t two = bad ? 0u : (uint32_t)__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest);
      const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1);
      const float2 back = __half22float2(__half2(hr));
      const __nv_bfloat162 b = __floats2bfloat162_rn(back.x * s, back.y * s);
      o[i] = bad ? 0x7FC07FC0u : *reinterpret_cast<const uint32_t*>(&b);
      w[i >> 2] |= two << (8 * (i & 3));
    }
    if (have) *reinterpret_cast<uint2*>(dst + l0 / 2) = make_uint2(w[0], w[1]);
    if (have && (lane & 1) == 0) dst[a.L / 2 + lane / 2] = bad ? 0xFF : (uint8_t)(e + 127);
    // the bytes between the scales and the rope part are zero
    for (int i = a.L / 2 + a.L / 32 + lane; i < (int)(a.row_bytes - 2 * a.R); i += 32) dst[i] = 0;
  }
  const uint32_t* f = reinterpret_cast<const uint32_t*>(a.freqs + (size_t)p.pos * a.R);
#pragma unroll
  for (int i = 0; i < kMaxRope / 64; ++i) {
    const int pr = lane + 32 * i;
    if (pr < a.R / 2) {
      uint32_t lost = 0, v = turn(r[i], f[pr], lost);
      if (lost) v = turn_wide(r[i], f[pr]);
      reinterpret_cast<uint32_t*>(dst_rope)[pr] = v;
      if (a.rows_out) reinterpret_cast<uint32_t*>(a.rows_out + (size_t)t * (a.L + a.R) + a.L)[pr] = v;
    }
  }
  if (a.rows_out && have) {
    uint4* d = reinterpret_cast<uint4*>(a.rows_out + (size_t)t * (a.L + a.R) + l0);
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// 16-byte pieces [part * kPieces, ...) of token t's queries.  In place only the rope
// pieces are walked; otherwise the others are copied.
__device__ __forceinline__ void turn_queries(const Args& a, int t, int part, int lane) {
  const bool in_place = a.q == a.q_out;
  const int per = in_place ? a.R / 8 : (a.N + a.R) / 8;   // pieces of a head walked
  const int first = in_place ? a.N / 8 : 0;
  const int total = a.H * per;
  const size_t base = (size_t)t * a.H * ((a.N + a.R) / 8);
  const uint4* src = reinterpret_cast<const uint4*>(a.q) + base;
  uint4* dst = reinterpret_cast<uint4*>(a.q_out) + base;
  uint4 v[kBatch];
  int at[kBatch], col[kBatch];
  int i = part * kPieces + (int)threadIdx.x, h = i / per, c = i - h * per;
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {   // one division a thread
    col[j] = i < total ? c + first : -1;
    at[j] = h * ((a.N + a.R) / 8) + col[j];
    if (i < total) v[j] = src[at[j]];
    i += kThreads;
    h += a.step_h;
    c += a.step_c;
    if (c >= per) {
      c -= per;
      ++h;
    }
  }
  const Place p = locate(a, t, lane);
  if (p.pos < 0) return;
  const uint4* f = reinterpret_cast<const uint4*>(a.freqs + (size_t)p.pos * a.R) - a.N / 8;
  uint32_t lost = 0;
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    if (col[j] < 0) continue;
    uint4 x = v[j];
    if (col[j] >= a.N / 8) x = turn(x, f[col[j]], lost);
    dst[at[j]] = x;
  }
  if (lost) {   // once for all pieces: a branch in the loop took longer
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (col[j] >= a.N / 8) dst[at[j]] = turn_wide(v[j], f[col[j]]);
  }
}

// Six blocks an SM, 40 registers: 8,483 prompt tokens 156 us (four with 64 registers 175, five with
// 48 162, seven with 32 158.5).
__global__ void __launch_bounds__(kThreads, 6) append_kernel(const Args a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = (int)blockIdx.x;
  if (blk < a.row_blocks) {
    const int t = blk * kRowsPerBlock + warp;
    if (t < a.T) new_row(a, t, lane);
  } else {
    const int i = blk - a.row_blocks;
    turn_queries(a, i / a.q_blocks, i % a.q_blocks, lane);
  }
}

}  // namespace app

long long cache_row_bytes(int fmt, int L, int R) {
  if (fmt == MLA_CACHE_BF16) return 2ll * (L + R);
  if (fmt == MLA_CACHE_E4M3) return (long long)L + 2 * R;
  return (long long)((L / 2 + L / 32 + 15) / 16 * 16) + 2 * R;
}

long long append_blocks(const mla_dims_t& d, int T, bool queries, bool in_place) {
  const long long pieces = (long long)d.num_heads * (in_place ? d.qk_rope : d.qk_nope + d.qk_rope) / 8;
  return ((long long)T + app::kRowsPerBlock - 1) / app::kRowsPerBlock +
         (queries ? T * ((pieces + app::kPieces - 1) / app::kPieces) : 0);
}

cudaError_t launch_append(const mla_dims_t& d, int fmt, const void* kv_new, long long new_stride,
                          const uint32_t* offsets, int B, int T, const void* q, void* q_out, void* pool,
                          float* scales, void* rows_out, const int32_t* block_table, int bt_stride,
                          const uint32_t* cache_lens, const void* freqs, int max_seq_len, const void* gamma,
                          float eps, PlanHeader* hdr, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  app::Args a{};
  a.fmt = fmt;
  a.H = d.num_heads;
  a.N = d.qk_nope;
  a.R = d.qk_rope;
  a.L = d.kv_lora_rank;
  a.ps = d.page_size;
  a.num_pages = d.num_pages;
  a.B = B;
  a.T = T;
  a.max_seq_len = max_seq_len;
  a.bt_stride = bt_stride;
  a.row_bytes = cache_row_bytes(fmt, a.L, a.R);
  a.new_stride = new_stride;
  a.eps = (double)eps;
  a.kv_new = static_cast<const __nv_bfloat16*>(kv_new);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.pool = static_cast<uint8_t*>(pool);
  a.scales = scales;
  a.rows_out = static_cast<__nv_bfloat16*>(rows_out);
  a.offsets = offsets;
  a.cache_lens = cache_lens;
  a.block_table = block_table;
  a.freqs = static_cast<const __nv_bfloat16*>(freqs);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.hdr = hdr;
  const long long blocks = append_blocks(d, T, q != nullptr, q == q_out);
  a.row_blocks = (int)append_blocks(d, T, false, false);
  a.q_blocks = (int)((blocks - a.row_blocks) / T);
  const int per = (q == q_out ? a.R : a.N + a.R) / 8;
  a.step_h = q ? app::kThreads / per : 0;
  a.step_c = q ? app::kThreads % per : 0;
  app::append_kernel<<<(unsigned)blocks, app::kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
