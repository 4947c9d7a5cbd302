// mla_cache_read: rows of the paged latent cache as bf16 values, request after request: token t of
// request b at pos = cache_len - n + i (the addressing of mla_cache_append) gives
//
//   out[t] = [ bf16(code * scale) (L) ; k_rope (R) ]
//
// each value rounded once.
//
// Layout.  A warp takes `rows_per_warp` consecutive tokens.  Its lanes look their tokens up at
// once, a lane a token (request by bisection, length, page), so the chain of dependent reads is
// paid once a warp and not once a row; then the rows are copied, 16 bytes of output (8 values) a lane.
// bf16 and e4m3 rows are loaded two at a time by the lanes that write them; e2m1 rows, of which a lane's 8
// values are 4 bytes and a scale, whole, 16 bytes a lane, four at a time, through shared memory.  Bound by HBM.
// 199,000 e4m3 rows 61.5 us (5.8 TB/s, 85 % of the copy rate), 278,000 bf16 rows 71.5 us (94 %), as many e2m1
// rows 54 us (83 %; loaded 4 bytes a lane 70); 4,000 e2m1 rows 3.8 us.
#include "mla_kernels.cuh"
#include "mla_rows.cuh"

namespace mla {
namespace rd {

using namespace rows;

constexpr int kWarps = 4;
constexpr int kMaxPieces = 3;        // 8-value pieces of a row a lane: L + R <= 768

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

// What a lane holds of a row: 8 values of the latent part as they are stored, or of the rope part.
template <int kFmt>
struct Piece {
  uint4 raw;
  float scale;
};

template <int kFmt>
__device__ __forceinline__ void load(const Args& a, long long row, int piece, Piece<kFmt>& p) {
  const uint8_t* src = a.pool + row * a.row_bytes;
  const int latent = a.L / 8;
  if (kFmt == MLA_CACHE_BF16 || piece >= latent) {
    p.raw = *reinterpret_cast<const uint4*>(src + (a.row_bytes - 2 * (a.L + a.R)) + 16 * piece);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(src + 8 * piece);
    p.raw.x = v.x;
    p.raw.y = v.y;
    p.scale = a.scales[row];
  }
}

template <int kFmt>
__device__ __forceinline__ uint4 values(const Args& a, int piece, const Piece<kFmt>& p) {
  if (kFmt == MLA_CACHE_BF16 || piece >= a.L / 8) return p.raw;
  return e4m3_values(make_uint2(p.raw.x, p.raw.y), p.scale);
}

// The rows of a warp's tokens from t0 on; `mine`: lane i's is token t0 + i's cache row.
__device__ __forceinline__ void copy_e2m1(const Args& a, long long t0, long long mine, int lane) {
  constexpr int kRows = 4, kRowBytes = 544;   // rows are at most 528 bytes (L = 512, R = 128)
  __shared__ __align__(16) uint8_t rows[kWarps][kRows][kRowBytes];
  uint8_t(*row)[kRowBytes] = rows[threadIdx.x >> 5];
  const int whole = (int)(a.row_bytes / 16), latent = a.L / 8, pieces = (a.L + a.R) / 8;
#pragma unroll 1
  for (int i = 0; i < a.per_warp; i += kRows) {
    uint4 v[kRows][2];
    long long at[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      at[j] = __shfl_sync(0xffffffffu, mine, (i + j) & 31);
      if (i + j >= a.per_warp) at[j] = -1;
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
  const int pieces = (a.L + a.R) / 8;
  if constexpr (kFmt == MLA_CACHE_E2M1) {
    copy_e2m1(a, t0, mine, lane);
    return;
  }
  constexpr int kTogether = 2;   // rows whose loads are out together
  for (int i = 0; i < a.per_warp; i += kTogether) {
    Piece<kFmt> p[kTogether][kMaxPieces];
    long long row[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      row[j] = __shfl_sync(0xffffffffu, mine, (i + j) & 31);
      if (i + j >= a.per_warp) row[j] = -1;
#pragma unroll
      for (int c = 0; c < kMaxPieces; ++c)
        if (row[j] >= 0 && lane + 32 * c < pieces) load<kFmt>(a, row[j], lane + 32 * c, p[j][c]);
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j)
#pragma unroll
      for (int c = 0; c < kMaxPieces; ++c)
        if (row[j] >= 0 && lane + 32 * c < pieces)
          reinterpret_cast<uint4*>(a.out + (t0 + i + j) * (a.L + a.R))[lane + 32 * c] =
              values<kFmt>(a, lane + 32 * c, p[j][c]);
  }
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
