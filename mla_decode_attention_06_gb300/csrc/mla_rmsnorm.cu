// mla_rmsnorm_quant: what stands between a layer's residual stream (or a latent, or the
// attention's output) and a projection over 8-bit codes, in one pass over the row:
//
//   h = bf16( x + residual )                       (h = x without a residual)
//   y = bf16( h / sqrt(mean(h^2) + eps) * gamma )  (y = h without gamma)
//   e4m3: s = the least 2^e with amax|y| <= 448 s, codes y / s     (an exact quotient, rounded once)
//   int8: s = fl32(amax|y| * fl32(1 / 127)), at least 2^-126, codes y / s    (nearest, ties to even)
//
// Arithmetic.  A code follows the last bit of y, so y is the correctly rounded value.
//   Sum of squares: s' = fma(h, h, s) loses fma(h, h, s - s') exactly as long as s is not below h^2, so each
//   thread starts at a power of two B above its largest square and adds up the losses; the threads' pairs
//   (s - B, losses) are joined by Knuth's TwoSum.  Four operations a value, none of which
//   unpacks it (bf_fma).
//   1 / sqrt, once a row, as a pair of floats ih + il, il >= 0 (a zero keeps its sign).
//   y: m = h * gamma is exact in fp32, and so is the sum of fma(m, ih, m * il) but for its one rounding.
//   Truncated and its last bit set it rounds to bf16 as the exact value does (no number with that bit
//   lies on a bf16 boundary); where il = 0 the sum may be exact and the row is done one value at a time
//   (fma_odd), as are values at the ends of fp32's range.
//   x + residual needs no such care: a sum of two 8-bit significands rounded to 24 bits and then to 8
//   is rounded as if once (24 >= 2 * 8 + 2).  An int8 quotient is formed with reciprocals of s a
//   little too large and too small; where that leaves its rounding open (values that are the largest over a power of
//   two among them, three in a thousand) the sign of y less s times the half-integer decides, one exact fma.
//
// Layout.  A row is read once and stays in registers: 8 values (16 bytes) a thread V times.  Rows of
// up to 2,048 values take a warp, longer ones a block with three barriers a row (sum, 1 / sqrt,
// largest code).  Bound by HBM for many long rows (8,192 x 8,192 with residual: e4m3 71.4 us, 6.58 TB/s, 97 % of
// the copy rate; int8 82.4; bf16 81, 97 %; codes alone 4,096 x 16,384 34 us, 86 %), by the steps' latency for short
// rows (8,192 x 1,536 11.4 us) and for few (3 to 5 us).
#include "mla_kernels.cuh"
#include "mla_rows.cuh"

namespace mla {
namespace rq {

using namespace rows;

constexpr int kWarpRows = 8;          // rows of a block where a warp takes a row

struct Args {
  int fmt, T, D;
  long long x_stride;
  double eps;
  bool eps_wide;                   // past what rsqrt_pair takes, alone under the root of a row of zeros
  float inv_h, inv_l;              // 1 / D as a pair
  const __nv_bfloat16* x;          // [T, >= D]
  const __nv_bfloat16* residual;   // [T, D] or NULL
  __nv_bfloat16* residual_out;     // [T, D], may be residual
  const __nv_bfloat16* gamma;      // [D] or NULL
  __nv_bfloat16* y_out;            // [T, D] or NULL
  uint8_t* codes;                  // [T, D] or NULL
  float* scales;                   // [T]
};

constexpr uint32_t kLow = 0x2B800000u, kSpan = 0x5D800000u - kLow;   // fp32 magnitudes 2^-40 .. 2^60

// h * inv * gamma of eight values of any magnitude, each rounded to odd and then to bf16; inv = ih + il, or what
// `wide` points to.
static __device__ __noinline__ uint4 normed_any(uint4 h, uint4 g, float ih, float il, const double* wide) {
  const double inv = wide ? *wide : (double)ih + (double)il;
  uint32_t x[4] = {h.x, h.y, h.z, h.w}, y[4] = {g.x, g.y, g.z, g.w};
  const bool inner = ih >= 0x1p-60f && ih <= 0x1p60f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float v = j ? hi_f(x[i]) : lo_f(x[i]), gm = j ? hi_f(y[i]) : lo_f(y[i]), m = __fmul_rn(v, gm);
      r[j] = inner && ((__float_as_uint(m) & 0x7FFFFFFFu) - kLow <= kSpan || v == 0.f || gm == 0.f)
                 ? fma_odd(m, ih, __fmul_rn(m, il))
                 : double_odd((double)v * inv * (double)gm);
    }
    x[i] = pack(r[0], r[1]);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: an integer added to it sits in the low bits

// Eight values as int8 codes, exactly, from reciprocals of s that are too large and too small: where the two
// disagree the quotient lies next to the half-integer between, and the sign of y less that times s, which one fma
// gives, decides (32 bits of product; a scale so small that the difference could underflow is brought up with y).
static __device__ __noinline__ uint2 int8_exact(uint4 yv, float s, float above, float below) {
  const uint32_t y[4] = {yv.x, yv.y, yv.z, yv.w};
  uint32_t b[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = i & 1 ? hi_f(y[i / 2]) : lo_f(y[i / 2]);
    const float p = __fmaf_rn(v, above, kMagic), q = __fmaf_rn(v, below, kMagic);
    uint32_t code = __float_as_uint(p);
    if (p != q) {
      const float up = s < 0x1p-60f ? 0x1p60f : 1.f, half = 0.5f * ((p - kMagic) + (q - kMagic));
      const float d = __fmaf_rn(-half, __fmul_rn(s, up), __fmul_rn(v, up));
      const uint32_t more = __float_as_uint(fmaxf(p, q)), less = __float_as_uint(fminf(p, q));
      code = d > 0.f ? more : d < 0.f ? less : more & 1u ? less : more;
    }
    b[i / 4] |= (code & 0xFFu) << (8 * (i & 3));
  }
  return make_uint2(b[0], b[1]);
}

// Eight values (packed bf16 pairs) as eight int8 codes.
__device__ __forceinline__ uint2 int8_codes(const uint32_t (&y)[4], float s, float rs) {
  const float above = __fmul_rn(rs, 1.f + 0x1p-22f), below = __fmul_rn(rs, 1.f - 0x1p-22f);
  const float2x magic = both(kMagic, kMagic), above2 = both(above, above), below2 = both(below, below);
  uint32_t b[8], differ = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2x v = widen2(y[i]);
    float r0, r1, q0, q1;
    apart(fma2(v, above2, magic), r0, r1);
    apart(fma2(v, below2, magic), q0, q1);
    b[2 * i] = __float_as_uint(r0);
    b[2 * i + 1] = __float_as_uint(r1);
    differ |= (b[2 * i] ^ __float_as_uint(q0)) | (b[2 * i + 1] ^ __float_as_uint(q1));
  }
  if (differ) return int8_exact(make_uint4(y[0], y[1], y[2], y[3]), s, above, below);
  uint2 w;
  w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return w;
}

// Largest 16-bit half (0 .. 0xFFFF) of a word of two.
__device__ __forceinline__ uint32_t halves_max(uint32_t v) { return max(v & 0xFFFFu, v >> 16); }

// V pieces of 8 values a thread; kWarp: a warp takes a row, else the block does.
// Blocks of 256 threads: five an SM at 51 registers where a block takes a row (8,192 x 8,192 e4m3 71.4 us; four
// 73.7, six 72.5), four at 64 where its warps do (8,192 x 1,536 11.4 us; three 12.3, five 12.3).
template <int V, bool kWarp, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? (kWarp ? 4 : 5) : 1) rmsnorm_kernel(const Args a) {
  __shared__ float part_hi[32], part_lo[32];
  __shared__ double part_wide[32];
  __shared__ uint32_t part_max[32];
  __shared__ double inv_wide[kWarp ? kWarpRows : 1];
  __shared__ float2 inv_pair;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = kWarp ? 1 : (int)blockDim.x >> 5;
  const int first = kWarp ? lane : (int)threadIdx.x, step = kWarp ? 32 : (int)blockDim.x;
  const long long t = kWarp ? (long long)blockIdx.x * kWarpRows + warp : (long long)blockIdx.x;
  if (kWarp && t >= a.T) return;
  const int n8 = a.D >> 3;

  uint32_t h[V][4];
  {
    uint4 xv[V], rv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = first + v * step;
      xv[v] = rv[v] = make_uint4(0, 0, 0, 0);
      if (p < n8) {
        xv[v] = reinterpret_cast<const uint4*>(a.x + t * a.x_stride)[p];
        if (a.residual) rv[v] = reinterpret_cast<const uint4*>(a.residual + t * a.D)[p];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v][0] = xv[v].x; h[v][1] = xv[v].y; h[v][2] = xv[v].z; h[v][3] = xv[v].w;
      if (a.residual) {
        const uint32_t r[4] = {rv[v].x, rv[v].y, rv[v].z, rv[v].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = pack2(bf_fma2(h[v][i], 0x3F803F80u, widen2(r[i])));
        const int p = first + v * step;
        if (p < n8)
          reinterpret_cast<uint4*>(a.residual_out + t * a.D)[p] = make_uint4(h[v][0], h[v][1], h[v][2], h[v][3]);
      }
    }
  }

  uint32_t amax = 0;   // of the results, halves side by side
  if (a.gamma) {
    uint32_t top2 = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) top2 = __vmaxu2(top2, h[v][i] & 0x7FFF7FFFu);
    const uint32_t top = halves_max(top2);
    // fp64 where the squares of this thread's largest values, or epsilon, would leave fp32's inner range
    bool wide = a.eps_wide || (top != 0 && !(top >= (0x2B800000u >> 16) && top <= (0x53800000u >> 16)));   // 2^-40 .. 2^40
    const float bias = __uint_as_float(top == 0 ? 0u : (2 * (top >> 7) - 125) << 23);   // the square of twice its power of two
    float hi, lo;
    {
      float2x s = both(bias, bias), e = both(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2x n = bf_fma2(h[v][i], h[v][i], s);
          e = add2(e, bf_fma2(h[v][i], h[v][i], sub2(s, n)));
          s = n;
        }
      float s0, s1, e0, e1, f0, f1, f2;
      apart(s, s0, s1);
      apart(e, e0, e1);
      two_sum(s0, -bias, s0, f0);
      two_sum(s1, -bias, s1, f1);
      two_sum(s0, s1, hi, f2);
      lo = __fadd_rn(__fadd_rn(e0, e1), __fadd_rn(__fadd_rn(f0, f1), f2));
    }
    auto reduce_pair = [&]() {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
        float e;
        two_sum(hi, h2, hi, e);
        lo = __fadd_rn(__fadd_rn(lo, l2), e);
      }
    };
    auto reduce_wide = [&]() {
      double s = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s += (double)lo_f(h[v][i]) * (double)lo_f(h[v][i]);
          s += (double)hi_f(h[v][i]) * (double)hi_f(h[v][i]);
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return s;
    };
    reduce_pair();
    float ih, il;
    auto root = [&]() {   // of the reduced pair
      float vh, vl;
      mean_plus(hi, lo, a.inv_h, a.inv_l, (float)a.eps, vh, vl);
      rsqrt_pair(vh, vl, ih, il);
    };
    if (kWarp) {
      wide = __any_sync(0xffffffffu, wide);
      if (wide) {
        const double inv = rsqrt(reduce_wide() / (double)a.D + a.eps);
        if (lane == 0) inv_wide[warp] = inv;
        __syncwarp();
      } else {
        root();
      }
    } else {
      if (lane == 0) {
        part_hi[warp] = hi;
        part_lo[warp] = lo;
      }
      wide = __syncthreads_or(wide);
      if (wide) {   // the same for the whole block
        const double s = reduce_wide();
        if (lane == 0) part_wide[warp] = s;
        __syncthreads();
      }
      if (warp == 0) {
        if (wide) {
          double sum = 0.0;
          for (int w = 0; w < warps; ++w) sum += part_wide[w];
          if (lane == 0) inv_wide[0] = rsqrt(sum / (double)a.D + a.eps);
        } else {
          hi = lane < warps ? part_hi[lane] : 0.f;
          lo = lane < warps ? part_lo[lane] : 0.f;
          reduce_pair();
          root();
          if (lane == 0) inv_pair = make_float2(ih, il);
        }
      }
      __syncthreads();
      ih = inv_pair.x;
      il = inv_pair.y;
    }
    if (wide) {
      const double inv = inv_wide[kWarp ? warp : 0];
      ih = __double2float_rd(inv);
      il = (float)(inv - (double)ih);
    }
    // The quick way gives every y right whose magnitude, before it is rounded to bf16, is zero or within [2^-90, 2^90):
    // with ih <= 2^15 a product h * gamma that fp32 does not hold exactly belongs to a smaller y, and one that it takes
    // for zero to a y that is zero.  (A smaller y may round to zero here and not be it.)
    const bool quick = il != 0.f && ih >= 0x1p-30f && ih <= 0x1p15f;
    constexpr uint32_t kLeast = 2u * 0x12800000u - 1, kMost = 0x6C800000u >> 16;   // 2^-90, 2^90
    const float2x ih2 = both(ih, ih), il2 = both(il, il);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = first + v * step;
      if (p < n8) {
        const uint4 gv = reinterpret_cast<const uint4*>(a.gamma)[p];
        const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w};
        uint32_t y[4], least = 0xFFFFFFFFu, most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2x m = bf_mul2(h[v][i], g[i]);
          float r0, r1;
          apart(fma2_rz(m, ih2, mul2(m, il2)), r0, r1);
          y[i] = pack(__uint_as_float(__float_as_uint(r0) | 1u), __uint_as_float(__float_as_uint(r1) | 1u));
          most = __vmaxu2(most, y[i] & 0x7FFF7FFFu);
          least = min(least, min(2 * __float_as_uint(r0) - 1, 2 * __float_as_uint(r1) - 1));   // no sign; zero the largest
        }
        if (!(quick && least >= kLeast && halves_max(most) < kMost)) {
          const uint4 r = normed_any(make_uint4(h[v][0], h[v][1], h[v][2], h[v][3]), gv, ih, il,
                                     wide ? &inv_wide[kWarp ? warp : 0] : nullptr);
          y[0] = r.x;
          y[1] = r.y;
          y[2] = r.z;
          y[3] = r.w;
          most = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) most = __vmaxu2(most, y[i] & 0x7FFF7FFFu);
        }
        amax = __vmaxu2(amax, most);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[v][i] = y[i];
      }
    }
  }

  if (a.y_out) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = first + v * step;
      if (p < n8) reinterpret_cast<uint4*>(a.y_out + t * a.D)[p] = make_uint4(h[v][0], h[v][1], h[v][2], h[v][3]);
    }
  }
  if (a.fmt == MLA_CODES_BF16) return;

  if (!a.gamma) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = __vmaxu2(amax, h[v][i] & 0x7FFF7FFFu);
  }
  amax = halves_max(amax);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (!kWarp) {
    if (lane == 0) part_max[warp] = amax;
    __syncthreads();
    amax = __reduce_max_sync(0xffffffffu, lane < warps ? part_max[lane] : 0u);
  }
  const bool bad = amax >= 0x7F80u;   // a NaN or an infinity: every value of the row reads back as NaN
  const bool int8 = a.fmt == MLA_CODES_INT8;
  float s, rs;
  if (int8) {
    s = amax == 0 ? 1.f : fmaxf(__fmul_rn(__uint_as_float(amax << 16), 1.f / 127.f), 0x1p-126f);
    rs = __frcp_rn(s);
  } else {
    const int e = bad ? 0 : scale_exponent(amax, 8, -126, 127);
    s = pow2(e);
    rs = pow2(-e);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = first + v * step;
    if (p >= n8) continue;
    uint2 w;
    if (bad) w = int8 ? make_uint2(0, 0) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    else w = int8 ? int8_codes(h[v], s, rs) : e4m3_codes(h[v], __float_as_uint(rs) >> 16);
    reinterpret_cast<uint2*>(a.codes + t * a.D)[p] = w;
  }
  if (first == 0) a.scales[t] = bad && int8 ? __uint_as_float(0x7FC00000u) : s;
}

template <int V, bool kWarp, int kThreads>
void start(const Args& a, int threads, cudaStream_t s) {
  const unsigned blocks = kWarp ? ((unsigned)a.T + kWarpRows - 1) / kWarpRows : (unsigned)a.T;
  rmsnorm_kernel<V, kWarp, kThreads><<<blocks, threads, 0, s>>>(a);
}

}  // namespace rq

cudaError_t launch_rmsnorm(int fmt, int rows, int width, const void* x, long long x_stride, const void* residual,
                           void* residual_out, const void* gamma, float eps, void* y_out, void* codes, float* scales,
                           cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  rq::Args a{};
  a.fmt = fmt;
  a.T = rows;
  a.D = width;
  a.x_stride = x_stride;
  a.eps = (double)eps;
  a.eps_wide = eps > 0x1p60f || (eps != 0.f && eps < 0x1p-100f);
  a.inv_h = (float)(1.0 / width);
  a.inv_l = (float)(1.0 / width - (double)a.inv_h);
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.residual = static_cast<const __nv_bfloat16*>(residual);
  a.residual_out = static_cast<__nv_bfloat16*>(residual_out);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.y_out = static_cast<__nv_bfloat16*>(y_out);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  const int n8 = width / 8;
  constexpr int kWarpThreads = 32 * rq::kWarpRows;
  auto threads = [&](int v) { return ((n8 + v - 1) / v + 31) / 32 * 32; };
  // Warps take rows where these fill the device; a few rows have a block each, one piece a thread
  // (64 x 1,536: 4.6 us, with a warp a row 7.2).
  if (rows < 1024 && n8 > 64 && n8 <= 1024) {
    if (n8 <= 256) rq::start<1, false, 256>(a, threads(1), s);
    else rq::start<1, false, 1024>(a, threads(1), s);
  } else if (n8 <= 32) rq::start<1, true, kWarpThreads>(a, kWarpThreads, s);
  else if (n8 <= 64) rq::start<2, true, kWarpThreads>(a, kWarpThreads, s);
  else if (n8 <= 128) rq::start<4, true, kWarpThreads>(a, kWarpThreads, s);
  else if (n8 <= 192) rq::start<6, true, kWarpThreads>(a, kWarpThreads, s);
  else if (n8 <= 256) rq::start<8, true, kWarpThreads>(a, kWarpThreads, s);
  else if (n8 <= 512) rq::start<2, false, 256>(a, threads(2), s);
  else if (n8 <= 1024) rq::start<4, false, 256>(a, threads(4), s);
  else rq::start<4, false, 1024>(a, threads(4), s);
  return cudaGetLastError();
}

}  // namespace mla
