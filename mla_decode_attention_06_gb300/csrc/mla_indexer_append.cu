// mla_indexer_append: the writer of mla_indexer_fp8's inputs.  For token t of request b at
// pos = cache_len - qlen + i, with the new index key k (D values) and the index queries q (H heads):
//
//   k = bf16( (k - mean) / sqrt(var + eps) * gamma + beta )      (with a norm; LayerNorm over D)
//   k, q: the last R values turned by freqs_cis[pos], bf16        (with freqs_cis)
//   e4m3: s = the least 2^e with amax <= 448 s, codes of the exact quotients, a scale a row and head
//   cache row at pos: k's codes and s;  q_codes, q_scales = s * q_weight
//
// Arithmetic as in mla_append.cu: rotations rounded once, codes of exact quotients.  The LayerNorm works
// on unevaluated pairs of floats (mean, deviations, their squares' sum, 1 / sqrt, the result), to some
// 2^-44, and rounds the pair that comes out once; rows at the ends of fp32's range and epsilons below
// 2^-60 take fp64, which for all keys was the longest part of the call (97 us of 8,483 tokens).
//
// Layout.  Neighbouring lanes hold a row, so that its largest magnitude is a few shuffles away and a warp
// reads and writes whole rows.  A query row takes D / 16 lanes of two 8-value pieces half a row apart, so
// that with R = D / 2 all lanes turn one piece of their two together; a block takes the heads of one or
// several tokens, two rows a lane group with all loads out before the tokens' places are looked up.  Keys (a piece a
// lane) have blocks of their own.  8,483 prompt tokens of 64 heads: 58 us, 3.75 TB/s, 55 % of the copy rate, held up
// by loads that a step waits for at its top (the integer pipe is active 51 %); a step of 64 tokens: 4.5 us, bound by
// the chain of dependent reads.
#include "mla_kernels.cuh"
#include "mla_rows.cuh"

namespace mla {
namespace ia {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kBatch = 2;   // rows of queries a lane group
constexpr int kMaxTokens = 32;   // of a block of queries: eight lanes look one up

struct Args {
  int D, H, R, ps, num_pages, B, T, bt_stride;
  int lanes;                       // of a key: 8, 16 or 32, the first D / 8 of them used
  int q_lanes;                     // of a query row, two pieces each
  int key_blocks, q_blocks;        // blocks of keys; blocks of queries for the same tokens
  int together, steps, slots;      // tokens of a block of queries at a time, how many times; head slots of a token
  long long max_seq_len, k_stride;
  double eps;
  float inv_h, inv_l;              // 1 / D as a pair
  const __nv_bfloat16* k_new;      // [T, >= D]
  const __nv_bfloat16* q;          // [T, H, D]
  const float* q_weight;           // [T, H] or NULL
  uint8_t* q_codes;                // [T, H, D]
  float* q_scales;                 // [T, H]
  uint8_t* k_cache;                // [pages, ps, D]
  float* k_scales;                 // [pages, ps]
  const uint32_t* offsets;
  const uint32_t* cache_lens;
  const int32_t* block_table;
  const __nv_bfloat16* freqs;      // [max_seq_len, R] or NULL
  const __nv_bfloat16* gamma;      // [D] or NULL
  const __nv_bfloat16* beta;
  PlanHeader* hdr;
};

// The larger magnitudes of two words of bf16 pairs, half by half.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t largest(uint32_t top, uint4 x) {
  return larger(larger(larger(larger(top, x.x), x.y), x.z), x.w);
}
// The scale of a row whose lanes' largest magnitudes (a word of two halves) lie on `lanes` neighbours: its
// exponent, or a value above 127 where the row holds a NaN or an infinity.  Whole warp.
__device__ __forceinline__ int row_exponent(uint32_t top, int lanes) {
  uint32_t amax = max(top & 0xFFFFu, top >> 16);
  for (int o = lanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  return amax >= 0x7F80u ? 255 : scale_exponent(amax, 8, -126, 127);
}
__device__ __forceinline__ float scale_of(int e) { return e == 255 ? 1.f : pow2(e); }
// Eight values as e4m3 codes under that exponent.
__device__ __forceinline__ uint2 coded(uint4 x, int e) {
  if (e == 255) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);   // every code a NaN
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  return e4m3_codes(w, __float_as_uint(pow2(-e)) >> 16);   // a bf16 value: -e is -127 at least
}

// Whether column `col` lies in the part of a row that is turned, and its rotations.
__device__ __forceinline__ bool in_rope(const Args& a, int col) { return a.R > 0 && col >= a.D - a.R && col < a.D; }
__device__ __forceinline__ uint4 rotations(const Args& a, int col, long long pos) {
  return *reinterpret_cast<const uint4*>(a.freqs + pos * a.R + (col - (a.D - a.R)));
}
__device__ __forceinline__ uint4 turned(uint4 x, uint4 f) {
  uint32_t lost = 0;
  const uint4 y = turn(x, f, lost);
  return lost ? turn_wide(x, f) : y;
}

// LayerNorm of a key, its values on `lanes` neighbours, in fp64.  Whole warp.
__device__ __noinline__ uint4 layer_norm_wide(const Args& a, uint4 x, uint4 gv, uint4 bv, bool have) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  double v[8], sum = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = i & 1 ? hi_f(w[i / 2]) : lo_f(w[i / 2]);
    sum += v[i];
  }
  for (int o = a.lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const double mean = sum / (double)a.D;
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] -= mean;
    sum += have ? v[i] * v[i] : 0.0;
  }
  for (int o = a.lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const double inv = rsqrt(sum / (double)a.D + a.eps);
  const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = pack(double_odd(v[2 * i] * inv * (double)lo_f(g[i]) + (double)lo_f(b[i])),
                double_odd(v[2 * i + 1] * inv * (double)hi_f(g[i]) + (double)hi_f(b[i])));
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// hi + lo rounded to odd: of the floats on either side of the sum the one whose last bit is set.
__device__ __forceinline__ float pair_odd(float hi, float lo) {
  float s, e;
  two_sum(hi, lo, s, e);
  const uint32_t u = __float_as_uint(s);
  if (e == 0.f || (u & 1u)) return s;
  return __uint_as_float((e > 0.f) == (s > 0.f) ? u + 1 : u - 1);
}

// The sum of a pair over a group of `lanes` neighbours, in all of them.
__device__ __forceinline__ void group_sum(int lanes, float& hi, float& lo) {
  for (int o = lanes / 2; o > 0; o >>= 1) {
    const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
    float e;
    two_sum(hi, h2, hi, e);
    lo = __fadd_rn(__fadd_rn(lo, l2), e);
  }
}

// LayerNorm of a key, its values on `lanes` neighbours; as bf16 pairs, zeros in lanes without values.  Whole warp.
__device__ __forceinline__ uint4 layer_norm(const Args& a, uint4 x, int col, bool have) {
  uint4 gv = make_uint4(0, 0, 0, 0), bv = gv;
  if (have) {
    gv = *reinterpret_cast<const uint4*>(a.gamma + col);
    bv = *reinterpret_cast<const uint4*>(a.beta + col);
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w}, g[4] = {gv.x, gv.y, gv.z, gv.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  // lanes whose largest value is below 2^-40 are fine beside larger ones; rows that are all that small are not
  uint32_t row_top = top;
  for (int o = a.lanes / 2; o > 0; o >>= 1) row_top = max(row_top, __shfl_xor_sync(0xffffffffu, row_top, o));
  const bool wide = a.eps < 0x1p-60 || a.eps > 0x1p60 ||
                    (row_top != 0 && !(row_top >= (0x2B800000u >> 16) && row_top <= (0x53800000u >> 16)));
  uint32_t y[4];
  if (__any_sync(0xffffffffu, wide)) {
    const uint4 r = layer_norm_wide(a, x, gv, bv, have);
    return have ? r : make_uint4(0, 0, 0, 0);
  }
  float v[8], hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float e;
    v[i] = i & 1 ? hi_f(w[i / 2]) : lo_f(w[i / 2]);
    two_sum(hi, v[i], hi, e);
    lo = __fadd_rn(lo, e);
  }
  group_sum(a.lanes, hi, lo);
  float mh, ml;
  mean_plus(hi, lo, a.inv_h, a.inv_l, 0.f, mh, ml);
  // what mh leaves of the sum is an fp32 number: divided, not multiplied by 1 / D, a mean that is one of the keys comes
  // out exactly (equal keys of 184 had a deviation of some 2^-49 of theirs, which a beta of zero shows)
  ml = __fdiv_rn(__fadd_rn(__fmaf_rn(-(float)a.D, mh, hi), lo), (float)a.D);
  float dl[8];
  hi = lo = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float e;
    two_sum(v[i], -mh, v[i], e);
    two_sum(v[i], __fsub_rn(e, ml), v[i], dl[i]);
    const float p = __fmul_rn(v[i], v[i]);
    const float pe = __fadd_rn(__fmaf_rn(v[i], v[i], -p), __fmul_rn(__fadd_rn(v[i], v[i]), dl[i]));
    two_sum(hi, have ? p : 0.f, hi, e);
    lo = __fadd_rn(lo, __fadd_rn(e, have ? pe : 0.f));
  }
  group_sum(a.lanes, hi, lo);
  float vh, vl, ih, il;
  mean_plus(hi, lo, a.inv_h, a.inv_l, (float)a.eps, vh, vl);
  rsqrt_pair(vh, vl, ih, il);
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gm = i & 1 ? hi_f(g[i / 2]) : lo_f(g[i / 2]), bt = i & 1 ? hi_f(b[i / 2]) : lo_f(b[i / 2]);
    const float p = __fmul_rn(v[i], ih);
    const float pe = __fadd_rn(__fmaf_rn(v[i], ih, -p), __fmaf_rn(v[i], il, __fmul_rn(dl[i], ih)));
    const float q = __fmul_rn(p, gm), qe = __fmaf_rn(pe, gm, __fmaf_rn(p, gm, -q));
    float s, e;
    two_sum(q, bt, s, e);
    o[i] = pair_odd(s, __fadd_rn(e, qe));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = pack(o[2 * i], o[2 * i + 1]);
  return have ? make_uint4(y[0], y[1], y[2], y[3]) : make_uint4(0, 0, 0, 0);
}

// Whole warp: the keys of 32 / lanes tokens.
__device__ __forceinline__ void new_keys(const Args& a, long long t0, int lane) {
  const int sub = lane & (a.lanes - 1), col = 8 * sub;
  const long long t = t0 + lane / a.lanes;
  const bool have = t < a.T && col < a.D;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (have) x = *reinterpret_cast<const uint4*>(a.k_new + t * a.k_stride + col);
  Place p = locate_groups(a, (int)min(t, a.T - 1ll), a.lanes, sub);
  if (t >= a.T) p.pos = -1;
  if (a.gamma) x = layer_norm(a, x, col, have);
  if (have && p.pos >= 0 && in_rope(a, col)) x = turned(x, rotations(a, col, p.pos));
  const int e = row_exponent(largest(0u, x), a.lanes);
  if (!have || p.pos < 0) return;
  *reinterpret_cast<uint2*>(a.k_cache + p.row * a.D + col) = coded(x, e);
  if (sub == 0) a.k_scales[p.row] = scale_of(e);
}

// The queries of tokens [t0, t0 + a.together * a.steps), `together` at a time: where the heads of one leave lane
// groups free, a block takes several tokens' side by side (slots of a.slots heads, a power of two); else it takes
// heads [part * rows, ...) of one, rows = kBatch times its lane groups.  The tokens' places are
// looked up at once, eight lanes a token, so that the chain of dependent reads is paid once.
// kSide: a.together > 1.
template <bool kSide>
__device__ __forceinline__ void queries(const Args& a, int t0, int part, int lane) {
  __shared__ long long places[kMaxTokens];
  const int per = kThreads / a.q_lanes, sub = (int)threadIdx.x & (a.q_lanes - 1), group = (int)threadIdx.x / a.q_lanes;
  const int col[2] = {8 * sub, 8 * (sub + a.q_lanes)};
  uint4 v[kBatch][2];
  float wt[kBatch];
  int tok[kBatch];       // token of the step
  bool use[kBatch];      // there is a head for it
  size_t row[kBatch];    // of the queries; advanced from step to step
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int slot = group + j * per;
    tok[j] = kSide ? slot / a.slots : 0;
    const int head = kSide ? slot & (a.slots - 1) : part * per * kBatch + slot;
    use[j] = head < a.H && (!kSide || tok[j] < a.together);
    if (!use[j]) tok[j] = 0;
    row[j] = (size_t)(t0 + tok[j]) * a.H + head;
  }
  auto load = [&](int first) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const bool ok = use[j] && t0 + first + tok[j] < a.T;
      wt[j] = ok && a.q_weight && sub == 0 ? a.q_weight[row[j]] : 1.f;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + row[j] * a.D) + sub;
      v[j][0] = ok ? src[0] : make_uint4(0, 0, 0, 0);
      v[j][1] = ok && col[1] < a.D ? src[a.q_lanes] : make_uint4(0, 0, 0, 0);
    }
  };
  load(0);   // on its way while the places are looked up
  const int n = a.together * a.steps;
  if (n == 1) {
    if ((int)threadIdx.x < 32) places[0] = locate(a, t0, lane).pos;
  } else if ((int)(threadIdx.x & ~31u) / 8 < n) {   // whole warps, four tokens each
    const int i = (int)threadIdx.x / 8;
    const long long pos = locate_groups(a, min(t0 + i, a.T - 1), 8, lane & 7).pos;
    places[i] = t0 + i < a.T ? pos : -1;
  }
  __syncthreads();
#pragma unroll 1
  for (int first = 0; first < n; first += a.together) {   // the step's first token, from t0
    if (first > 0) load(first);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!in_rope(a, col[k])) continue;
      uint32_t lost = 0;
      uint4 f = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const long long pos = places[first + tok[j]];
        if ((kSide || j == 0) && pos >= 0) f = rotations(a, col[k], pos);
        v[j][k] = turn(v[j][k], f, lost);   // of a token without a place it is not used
      }
      if (lost) {   // once for all: the rows are read again
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const long long pos = places[first + tok[j]];
          if (use[j] && pos >= 0)
            v[j][k] = turn_wide(*reinterpret_cast<const uint4*>(a.q + row[j] * a.D + col[k]), rotations(a, col[k], pos));
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int e = row_exponent(largest(largest(0u, v[j][0]), v[j][1]), a.q_lanes);
      if (use[j] && places[first + tok[j]] >= 0) {   // no place past the last token
        uint2* dst = reinterpret_cast<uint2*>(a.q_codes + row[j] * a.D) + sub;
        dst[0] = coded(v[j][0], e);
        if (col[1] < a.D) dst[a.q_lanes] = coded(v[j][1], e);
        if (sub == 0) a.q_scales[row[j]] = __fmul_rn(scale_of(e), wt[j]);
      }
      row[j] += (size_t)a.together * a.H;
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kThreads) indexer_append_kernel(const Args a) {
  const int lane = threadIdx.x & 31, blk = (int)blockIdx.x;
  if (blk < a.key_blocks) {
    const long long t0 = ((long long)blk * (kThreads / 32) + (threadIdx.x >> 5)) * (32 / a.lanes);
    if (t0 < a.T) new_keys(a, t0, lane);
  } else {
    const int i = blk - a.key_blocks;
    const int t0 = i / a.q_blocks * a.together * a.steps;
    if (a.together > 1) queries<true>(a, t0, 0, lane);
    else queries<false>(a, t0, i % a.q_blocks, lane);
  }
}

int lanes_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }
int q_lanes_of(int D) {
  int n = 1;
  while (16 * n < D) n *= 2;
  return n;
}

}  // namespace ia

struct QueryCut {
  int together, steps, slots;
  long long parts;   // blocks for the same tokens
};
// Tokens side by side where a block has room for the heads of two and more, as many as fit (5,500 tokens of 4
// heads 7 us, a block each 35); else one after the other, four where that leaves every SM eight blocks
// (8,483 tokens of 64 heads 58 us, two a block 63, eight 72).
static QueryCut query_cut(int H, int D, long long T) {
  const int rows = ia::kThreads / ia::q_lanes_of(D) * ia::kBatch;
  QueryCut c{1, 1, 1, 1};
  while (c.slots < H && c.slots < rows) c.slots *= 2;
  c.together = H <= c.slots ? rows / c.slots : 1;
  if (c.together > ia::kMaxTokens) c.together = ia::kMaxTokens;
  if (c.together == 1) {
    c.parts = ((long long)H + rows - 1) / rows;
    c.steps = T * c.parts >= 4ll * 8 * 152 ? 4 : 1;
  }
  return c;
}

long long indexer_append_blocks(int H, int D, int T, bool queries) {
  const int keys = ia::kThreads / ia::lanes_of(D);
  long long n = ((long long)T + keys - 1) / keys;
  if (queries) {
    const QueryCut c = query_cut(H, D, T);
    n += ((long long)T + c.together * c.steps - 1) / (c.together * c.steps) * c.parts;
  }
  return n;
}

cudaError_t launch_indexer_append(int H, int D, int R, int ps, int num_pages, const void* k_new, long long k_stride,
                                  const uint32_t* offsets, int B, int T, const void* q, const float* q_weight,
                                  void* q_codes, float* q_scales, void* k_cache, float* k_scales,
                                  const int32_t* block_table, int bt_stride, const uint32_t* cache_lens,
                                  const void* freqs, int max_seq_len, const void* gamma, const void* beta, float eps,
                                  PlanHeader* hdr, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  ia::Args a{};
  a.D = D;
  a.H = H;
  a.R = freqs ? R : 0;
  a.ps = ps;
  a.num_pages = num_pages;
  a.B = B;
  a.T = T;
  a.bt_stride = bt_stride;
  a.lanes = ia::lanes_of(D);
  a.q_lanes = ia::q_lanes_of(D);
  a.max_seq_len = freqs ? max_seq_len : INT64_MAX;
  a.k_stride = k_stride;
  a.eps = (double)eps;
  a.inv_h = (float)(1.0 / D);
  a.inv_l = (float)(1.0 / D - (double)a.inv_h);
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_weight = q_weight;
  a.q_codes = static_cast<uint8_t*>(q_codes);
  a.q_scales = q_scales;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.k_scales = k_scales;
  a.offsets = offsets;
  a.cache_lens = cache_lens;
  a.block_table = block_table;
  a.freqs = static_cast<const __nv_bfloat16*>(freqs);
  a.gamma = static_cast<const __nv_bfloat16*>(gamma);
  a.beta = static_cast<const __nv_bfloat16*>(beta);
  a.hdr = hdr;
  const long long blocks = indexer_append_blocks(H, D, T, q != nullptr);
  a.key_blocks = (int)indexer_append_blocks(H, D, T, false);
  const QueryCut c = query_cut(H, D, T);
  a.q_blocks = (int)c.parts;
  a.together = c.together;
  a.steps = c.steps;
  a.slots = c.slots;
  ia::indexer_append_kernel<<<(unsigned)blocks, ia::kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
