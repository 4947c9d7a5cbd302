// mla_cache_read: rows of the paged latent cache as bf16 values, request after request: token t of
// request b at pos = cache_len - n + i (the addressing of mla_cache_append) gives
//
//   out[t] = [ bf16(code * scale) (L) ; k_rope (R) ]
//
// each value rounded once.
//
// Layout.  A warp takes `per_warp` consecutive tokens.  Its lanes look their tokens up at once, a lane a
// token (request by bisection, length, page), so the chain of dependent reads is paid once a warp and not
// once a row; then the rows are copied, four at a time, all their loads out before the first store, 16 bytes a
// lane each.  Bound by HBM.  199,000 e4m3 rows 58.5 us (6.1 TB/s, 90 % of the copy rate), 278,000 bf16 rows
// 70.4 us (95 %), as many e2m1 rows 54 us (83 %; loaded 4 bytes a lane 70); 4,000 e2m1 rows 3.8 us.
#include "mla_kernels.cuh"
#include "mla_rows.cuh"

namespace mla {
namespace rd {

using namespace rows;

constexpr int kWarps = 4;

struct Args {
  int L, R, ps, num_pages, B, T, bt_stride, per_warp;
  long long row_bytes;
  const uint8_t* pool;
  const float* scales;
  const uint32_t* offsets;
  const uint32_t* cache_lens;
  const int32_t* block_table;
  __nv_bfloat16* out;
  PlanHeader* hdr;
};

// One lane: the cache row of token t, -1 if there is none to read.
__device__ __forceinline__ long long find(const Args& a, int t) {
  if (t >= a.T || (uint32_t)t >= a.offsets[a.B]) return -1;
  int lo = 0, n = a.B;   // the request is the last b with offsets[b] <= t
  while (n > 1) {
    const int half = n >> 1;
    const bool up = a.offsets[lo + half] <= (uint32_t)t;
    lo += up ? half : 0;
    n = up ? n - half : half;
  }
  const uint32_t qb = a.offsets[lo], qe = a.offsets[lo + 1];
  const long long pos = (long long)a.cache_lens[lo] - qe + t;
  if (qb <= (uint32_t)t && (uint32_t)t < qe && pos >= 0 && pos < (long long)a.bt_stride * a.ps) {
    const int page = a.block_table[(size_t)lo * a.bt_stride + pos / a.ps];
    if (page >= 0 && page < a.num_pages) return (long long)page * a.ps + pos % a.ps;
  }
  atomicOr(&a.hdr->status, kDeviceCheckFailed);
  return -1;
}

// x * s rounded to odd.
__device__ __forceinline__ float mul_odd(float x, float s) {
  const float down = __fmul_rd(x, s), up = __fmul_ru(x, s);
  return __float_as_uint(down) & 1u ? down : up;
}

// Eight e4m3 codes times a row scale, each rounded once.  A truncated product with its last bit set rounds
// to bf16 as the exact one does unless that is a tie (or fp32's range ends).  A code has four
// significant bits, so where the scale's last four bits are zero the product is exact and is left alone;
// where they are not it is no tie, whose scale would end in fifteen zeros.
__device__ __forceinline__ uint4 e4m3_values(uint2 codes, float s) {
  uint32_t o[4];
  const bool inner = s >= 0x1p-100f || !(s == s);
  const uint32_t sticky = (__float_as_uint(s) & 15u) != 0 ? 1u : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = ((i < 2 ? codes.x : codes.y) >> (16 * (i & 1))) & 0xFFFFu;
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
    float lo, hi;
    if (inner) {
      apart(mul2_rz(both(v.x, v.y), both(s, s)), lo, hi);
      lo = __uint_as_float(__float_as_uint(lo) | sticky);
      hi = __uint_as_float(__float_as_uint(hi) | sticky);
    } else {
      lo = mul_odd(v.x, s);
      hi = mul_odd(v.y, s);
    }
    o[i] = pack(lo, hi);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight e2m1 codes times a power of two, by bytes: a code's magnitude picks the two bytes of its bf16 value, its
// sign the upper one's top bit; the product of bf16 pairs is exact (or bf16's range ends).
__device__ __forceinline__ uint4 e2m1_values(uint32_t codes, __nv_bfloat162 s) {
  constexpr uint32_t kHi0 = 0x3F3F3F00u, kHi1 = 0x40404040u, kLo0 = 0xC0800000u, kLo1 = 0xC0804000u;   // 0 .5 1 1.5 2 3 4 6
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // four codes: a selector takes four nibbles
    const uint32_t mag = (codes >> (16 * i)) & 0x7777u, sign = (codes >> (16 * i + 3)) & 0x1111u;
    const uint32_t hi = __byte_perm(kHi0, kHi1, mag) | __byte_perm(0x00008000u, 0u, sign);
    const uint32_t lo = __byte_perm(kLo0, kLo1, mag);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t v = __byte_perm(lo, hi, j ? 0x7362 : 0x5140);
      const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), s);
      o[2 * i + j] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Rows of a warp whose loads are out together (199,000 e4m3 rows two 59.9 us, four 58.7; 278,000 bf16 rows 71.2
// and 70.4).  The functions below copy the rows of a warp's tokens from t0 on; `mine`: lane i's is token t0 + i's
// cache row.
constexpr int kRows = 4;

// Of kRows rows from the i-th on, whose `at` each is; -1: none.
__device__ __forceinline__ void rows_at(const Args& a, long long mine, int i, long long (&at)[kRows]) {
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    at[j] = __shfl_sync(0xffffffffu, mine, (i + j) & 31);
    if (i + j >= a.per_warp) at[j] = -1;
  }
}

__device__ __forceinline__ void copy_bf16(const Args& a, long long t0, long long mine, int lane) {
  constexpr int kPieces = 3;   // 16 bytes of a row a lane: L + R <= 640
  const int pieces = (a.L + a.R) / 8;
#pragma unroll 1
  for (int i = 0; i < a.per_warp; i += kRows) {
    uint4 v[kRows][kPieces];
    long long at[kRows];
    rows_at(a, mine, i, at);
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int c = 0; c < kPieces; ++c)
        if (at[j] >= 0 && lane + 32 * c < pieces)
          v[j][c] = reinterpret_cast<const uint4*>(a.pool + at[j] * a.row_bytes)[lane + 32 * c];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int c = 0; c < kPieces; ++c)
        if (at[j] >= 0 && lane + 32 * c < pieces)
          reinterpret_cast<uint4*>(a.out + (t0 + i + j) * (a.L + a.R))[lane + 32 * c] = v[j][c];
  }
}

// 16 codes of the latent part and 8 rope values a lane (8 codes, so that neighbouring lanes store neighbouring 16
// bytes, took 61.3 us).
__device__ __forceinline__ void copy_e4m3(const Args& a, long long t0, long long mine, int lane) {
  const bool latent = lane < a.L / 16, rope = lane < a.R / 8;
#pragma unroll 1
  for (int i = 0; i < a.per_warp; i += kRows) {
    uint4 v[kRows], r[kRows];
    float s[kRows];
    long long at[kRows];
    rows_at(a, mine, i, at);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint8_t* src = a.pool + at[j] * a.row_bytes + 16 * lane;
      if (at[j] >= 0 && latent) {
        v[j] = *reinterpret_cast<const uint4*>(src);
        s[j] = a.scales[at[j]];
      }
      if (at[j] >= 0 && rope) r[j] = *reinterpret_cast<const uint4*>(src + a.L);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (at[j] < 0) continue;
      __nv_bfloat16* out = a.out + (t0 + i + j) * (a.L + a.R);
      if (latent) {
        const uint4 lo = e4m3_values(make_uint2(v[j].x, v[j].y), s[j]), hi = e4m3_values(make_uint2(v[j].z, v[j].w), s[j]);
        reinterpret_cast<uint4*>(out)[2 * lane] = lo;   // one right after the other, or half sectors go to L2 (69 us)
        reinterpret_cast<uint4*>(out)[2 * lane + 1] = hi;
      }
      if (rope) reinterpret_cast<uint4*>(out + a.L)[lane] = r[j];
    }
  }
}

// Rows through shared memory: a lane's 8 values are 4 bytes and a scale, loaded 16 bytes a lane.
__device__ __forceinline__ void copy_e2m1(const Args& a, long long t0, long long mine, int lane) {
  constexpr int kRowBytes = 544;   // rows are at most 528 bytes (L = 512, R = 128)
  __shared__ __align__(16) uint8_t rows[kWarps][kRows][kRowBytes];
  uint8_t(*row)[kRowBytes] = rows[threadIdx.x >> 5];
  const int whole = (int)(a.row_bytes / 16), latent = a.L / 8, pieces = (a.L + a.R) / 8;
#pragma unroll 1
  for (int i = 0; i < a.per_warp; i += kRows) {
    uint4 v[kRows][2];
    long long at[kRows];
    rows_at(a, mine, i, at);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint4* src = reinterpret_cast<const uint4*>(a.pool + at[j] * a.row_bytes);
      if (at[j] >= 0 && lane < whole) v[j][0] = src[lane];
      if (at[j] >= 0 && lane + 32 < whole) v[j][1] = src[lane + 32];
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (at[j] >= 0 && lane < whole) reinterpret_cast<uint4*>(row[j])[lane] = v[j][0];
      if (at[j] >= 0 && lane + 32 < whole) reinterpret_cast<uint4*>(row[j])[lane + 32] = v[j][1];
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (at[j] < 0) continue;
      uint4* out = reinterpret_cast<uint4*>(a.out + (t0 + i + j) * (a.L + a.R));
      for (int c = lane; c < pieces; c += 32) {
        if (c >= latent) {
          out[c] = *reinterpret_cast<const uint4*>(row[j] + a.row_bytes - 2 * (a.L + a.R) + 16 * c);
        } else {
          const uint32_t e = row[j][a.L / 2 + c / 4];   // 2^(e - 127) as a bf16 value, 255 = NaN
          const uint32_t s = e == 255 ? 0x7FC0u : e == 0 ? 0x0040u : e << 7, s2 = s | s << 16;
          out[c] = e2m1_values(*reinterpret_cast<const uint32_t*>(row[j] + 4 * c), *reinterpret_cast<const __nv_bfloat162*>(&s2));
        }
      }
    }
    __syncwarp();
  }
}

template <int kFmt>
__global__ void __launch_bounds__(32 * kWarps) read_kernel(const Args a) {
  const int lane = threadIdx.x & 31;
  const long long t0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * a.per_warp;
  if (t0 >= a.T) return;
  const long long mine = lane < a.per_warp ? find(a, (int)min(t0 + lane, (long long)a.T)) : -1;
  if constexpr (kFmt == MLA_CACHE_BF16) copy_bf16(a, t0, mine, lane);
  else if constexpr (kFmt == MLA_CACHE_E4M3) copy_e4m3(a, t0, mine, lane);
  else copy_e2m1(a, t0, mine, lane);
}

}  // namespace rd

cudaError_t launch_cache_read(const mla_dims_t& d, int fmt, const uint32_t* offsets, int B, int T, const void* pool,
                              const float* scales, const int32_t* block_table, int bt_stride,
                              const uint32_t* cache_lens, void* out, PlanHeader* hdr, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  rd::Args a{};
  a.L = d.kv_lora_rank;
  a.R = d.qk_rope;
  a.ps = d.page_size;
  a.num_pages = d.num_pages;
  a.B = B;
  a.T = T;
  a.bt_stride = bt_stride;
  a.row_bytes = cache_row_bytes(fmt, a.L, a.R);
  a.pool = static_cast<const uint8_t*>(pool);
  a.scales = scales;
  a.offsets = offsets;
  a.cache_lens = cache_lens;
  a.block_table = block_table;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.hdr = hdr;
  // rows of a warp: eight where that leaves every SM some 16 warps, else fewer (4,000 e2m1 rows: two 3.8 us, eight 6.9)
  a.per_warp = T >= 8 * 16 * 152 ? 8 : T >= 4 * 16 * 152 ? 4 : 2;   // at most 32, a lane a row
  const unsigned blocks = (unsigned)(((long long)T + rd::kWarps * a.per_warp - 1) / (rd::kWarps * a.per_warp));
  if (fmt == MLA_CACHE_BF16) rd::read_kernel<MLA_CACHE_BF16><<<blocks, 32 * rd::kWarps, 0, s>>>(a);
  else if (fmt == MLA_CACHE_E4M3) rd::read_kernel<MLA_CACHE_E4M3><<<blocks, 32 * rd::kWarps, 0, s>>>(a);
  else rd::read_kernel<MLA_CACHE_E2M1><<<blocks, 32 * rd::kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
