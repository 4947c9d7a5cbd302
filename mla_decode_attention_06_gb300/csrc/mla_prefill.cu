// mla_prefill_paged: latent attention in its expanded form, for many query tokens.
//
//   k_j[h] = [ c_j . w_uk[h] ; rope_j ]      v_j[h] = w_uv[h] . c_j
//   out[t,h] = softmax_j(scale q[t,h] . k_j[h]) . v_j[h]
//
// The absorbed form of the decode costs 2 H (2 L + R) operations per (query, key) pair,
// this one 2 H (N + R + V), plus 2 H L (N + V) per cached row: at (N, R, L, V) =
// (128, 64, 512, 128) 320 against 1088 per pair and head, so it is the cheaper one from
// about 170 query tokens per request.
//
// Launches of a call:
//   plan     one block: each request's key range and key tiles (128 keys), the list of
//            query blocks (256 tokens), longest first.
//   gather   cache rows of any format -> bf16 tiles of 128 rows, and which rows are live.
//   expand   K and V of a pass's heads: one GEMM tile (128 rows x (N | V) x L) per key
//            tile and head, tcgen05, written as the attention's shared-memory images.
//   attend   one CTA per SM, taking one (query block, head, key split) after another: running
//            softmax between two tcgen05 products.
//   combine  joins the key splits (only where a call has few query blocks).
//
// Every tile that passes between these kernels is stored as 128-byte-swizzled boxes of
// 128 rows x 64 columns (16 KB), so it moves by plain bulk copies and needs no tensor map.
//
// A row that holds a NaN or an infinity in its latent part would turn every P . V product
// of its tile into NaN, masked queries included (0 * NaN).  The gather stores such a row
// with zeros and a NaN rope part: its scores are NaN where it is visible, and masked
// queries never see it.
//
// Precision.  K, V and P are rounded once each; as bf16 (2^-9) the score's share of that,
// amplified by the softmax, would be most of the error.  They are kept as f16 (2^-12, the
// same tensor rate), which holds what such values are in practice but not what they could
// be: the kernels that write them check the largest magnitude of every row (64 columns of a K
// or V row, a rope row, an e4m3 latent row, 256 neighbouring e4m3 weights) and flag the request
// (for weights the call) where it is above 2^15 or, not being zero, below 2^-15.  At 2^-15 f16's step is 2^-24, so
// each value is off by at most 2^-10 of its row's largest, half of what bf16 may be off by:
// a row small beside its neighbours loses nothing that the second sequence would keep, and
// heads or weights some thousand times smaller than usual stay in the first.  A second
// sequence of the same kernels with bf16 throughout follows in the stream: it takes the flagged
// requests, the first leaves them, so that the other requests of the call keep their bits;
// without flags it returns at once.  Measured, all requests flagged by the gather, all by the
// expansion, the first one by the gather, none: two chunks behind 7,600 e2m1 keys 702, 928, 736 and
// 619 us, seven short prompts 218, 275, 245 and 183, one prompt of 16,384 tokens x 16 heads 962, 986
// and 894.  A flag is raised by one kernel and decides in later ones only: within a launch no two
// threads see it differ.  Queries are converted by the
// CTA that uses them, each row scaled by its own power of two; e4m3 latents and weights
// become f16 before the expansion, bf16 and e2m1 ones enter it as the bf16 values they are.
// Measured on uniform random cases: 1.7e-3 relative to 64 bits with f16, most of it the
// bf16 output itself.
#include <math_constants.h>

#include <algorithm>
#include <cstddef>

#include "mla_prefill.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace pf {

using namespace sm100;

constexpr int kTile = 128;              // keys per tile, query tokens per sub-block
constexpr int kBox = kTile * 128;       // 128 rows x 64 bf16
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr uint32_t kBf16Operands = (1u << 7) | (1u << 10);   // instruction descriptor: types of A and B (0: f16)

// One request of the call.  Keys [lo, lo + nkeys) of its cache are visible to some query;
// they fill tiles [tile0, tile0 + ntiles).
struct Req {
  int32_t q0, qlen;        // query tokens
  int32_t len, lo, nkeys;
  int32_t tile0, ntiles;
  int32_t item0;           // query blocks of the requests before
  int32_t fits;            // 0: no room in the workspace, its outputs are NaN
  int32_t wide[2];         // f16 does not do, found by the gather, by the expansion
  int32_t pad;
};

struct Args {
  mla_dims_t d;
  int fmt, B, T, mask, window, bt_stride, cap_tiles, max_items;
  float scale;
  int nbk, nbv, nbq;               // 64-column boxes of a K (no-rope), V and query row
  int h0, hg, splits;              // heads of this pass, key splits
  int half;                        // 1: f16 sequence, 0: bf16, run only when the flag is up
  const uint32_t* offsets;
  const uint32_t* cache_lens;
  const int32_t* block_table;
  const uint8_t* pool;
  const float* scales;
  PlanHeader* hdr;                 // total_tiles: key tiles; pad[2]: query blocks; pad[3]: f16 does not do;
                                   // pad[4]: blocks that the attention's CTAs took beyond their first
  Req* reqs;
  int2* items;                     // (request, query block)
  uint4* live;                     // per tile: live rows
  uint8_t *rope, *lat;             // boxes per tile: 1, L / 64
  uint8_t* kv;                     // boxes per (head of the pass, tile): nbk + nbv
  float *part_o, *part_lse;        // [splits, T, H, V], [splits, T, H]
  __nv_bfloat16* out;
  float* lse_out;
};

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

constexpr int kWeights = 1, kGathered = 2, kExpanded = 4;   // bits of hdr->pad[3]
__device__ __forceinline__ int raised(const Args& a) { return *reinterpret_cast<const volatile int*>(&a.hdr->pad[3]); }
__device__ __forceinline__ void raise(const Args& a, int bit, int b) {   // b: the request, -1 for weights
  int* w = b < 0 ? &a.hdr->pad[3] : &a.reqs[b].wide[bit == kGathered ? 0 : 1];
  if (__ldcg(w) & bit) return;   // by another thread (all of them at once took three times the call)
  atomicOr(w, bit);
  if (b >= 0) atomicOr(&a.hdr->pad[3], bit);
}
// After the wait on the previous kernel: does this sequence take any request?  (`flags`: one read
// of the word.  What a kernel itself raises it does not look at: the first sequence raises flags,
// the second does not.)
__device__ __forceinline__ bool runs(const Args& a, int flags) { return a.half ? !(flags & kWeights) : flags != 0; }
// Does it take request b, by the gather's flags and (`expanded`) the expansion's?
__device__ __forceinline__ bool takes(const Args& a, int flags, int b, bool expanded) {
  const bool wide = (flags & kWeights) || __ldcg(&a.reqs[b].wide[0]) != 0 || (expanded && __ldcg(&a.reqs[b].wide[1]) != 0);
  return a.half ? !wide : wide;
}
// The request that holds a key tile: the last one with tile0 <= tile that has tiles.
__device__ __forceinline__ int request_of(const Args& a, int tile) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.reqs[mid].tile0 <= tile) lo = mid; else hi = mid - 1;
  }
  while (lo > 0 && a.reqs[lo].ntiles == 0) --lo;
  return lo;
}
// Is a row's largest magnitude (fp32 bits) one that f16 holds well: zero, or within
// [2^-15, 2^15]?  Half a step of f16 then is at most 2^-10 of it.
__device__ __forceinline__ bool f16_holds_row(uint32_t top) {
  return top == 0u || (top >= 0x38000000u && top <= 0x47000000u);
}
// The same for a row that a whole warp holds, `top` the largest of a lane's values.
__device__ __forceinline__ bool f16_holds(uint32_t top) {
  const bool over = __any_sync(0xffffffffu, top > 0x47000000u), some = __any_sync(0xffffffffu, top != 0u);
  return !over && (__any_sync(0xffffffffu, top >= 0x38000000u) || !some);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Keys [lo, hi) that the query at row r of request q sees, relative to q.lo.
__device__ __forceinline__ void row_range(const Args& a, const Req& q, int r, int& lo, int& hi) {
  lo = 0;
  hi = q.nkeys;
  if (a.mask != MLA_MASK_NULL) {
    const int pos = q.len - q.qlen + r;
    hi = max(0, min(hi, pos + 1 - q.lo));
    if (a.mask == MLA_MASK_SLIDING_WINDOW_CAUSAL) lo = max(0, pos + 1 - a.window - q.lo);
  }
}

// Key tiles [j0, j1) of query rows [r0, r1).
__device__ __forceinline__ void tile_range(const Args& a, const Req& q, int r0, int r1, int& j0, int& j1) {
  int lo, hi, x;
  row_range(a, q, r0, lo, x);
  row_range(a, q, r1 - 1, x, hi);
  j0 = lo / kTile;
  j1 = hi > lo ? (hi + kTile - 1) / kTile : j0;
}

// ------------------------------------------------------------------------------ plan

constexpr int kPlanThreads = 512;
constexpr int kBuckets = 1024;

__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {   // exclusive, whole block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = lane < kPlanThreads / 32 ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const int before = warp > 0 ? sums[warp - 1] : 0;
  *total = sums[kPlanThreads / 32 - 1];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Args a) {
  __shared__ int sums[32], hist[kBuckets], any_bad;
  griddep_launch();
  const int tid = threadIdx.x;
  if (tid == 0) any_bad = 0;
  for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  bool bad = false;
  auto request = [&](int b) {
    Req q{};
    const uint32_t qb = min(a.offsets[b], (uint32_t)a.T), qe = min(a.offsets[b + 1], (uint32_t)a.T);
    const long long cap = (long long)a.bt_stride * a.d.page_size;
    long long len = a.cache_lens[b];
    if (a.offsets[b + 1] < a.offsets[b] || a.offsets[b + 1] > (uint32_t)a.T || len > cap) bad = true;
    if (qe > qb && len < (long long)qe - qb) bad = true;   // query tokens that the cache does not count
    q.q0 = (int)qb;
    q.qlen = qe > qb ? (int)(qe - qb) : 0;
    q.len = (int)min(len, min(cap, (long long)INT32_MAX - 2 * kTile));
    q.fits = 1;
    if (a.mask == MLA_MASK_SLIDING_WINDOW_CAUSAL)
      q.lo = (int)max(0ll, (long long)q.len - q.qlen + 1 - a.window);
    q.nkeys = q.qlen > 0 && q.lo < q.len ? q.len - q.lo : 0;
    q.ntiles = (q.nkeys + kTile - 1) / kTile;
    return q;
  };
  int tiles = 0, blocks = 0;
  for (int b = b0; b < b1; ++b) {
    const Req q = request(b);
    // more than there is room for is no room, whatever the sum
    tiles = min(tiles + min(q.ntiles, a.cap_tiles + 1), a.cap_tiles + 1);
    blocks += (q.qlen + 2 * kTile - 1) / (2 * kTile);
  }
  int total_tiles, total_items;
  int tile = block_scan(tiles, sums, &total_tiles);
  int item = block_scan(blocks, sums, &total_items);
  for (int b = b0; b < b1; ++b) {
    Req q = request(b);
    q.tile0 = min(tile, a.cap_tiles);
    q.item0 = item;
    tile = min(tile, a.cap_tiles) + min(q.ntiles, a.cap_tiles + 1);
    item += (q.qlen + 2 * kTile - 1) / (2 * kTile);
    if (q.ntiles > 0 && tile > a.cap_tiles) {
      q.fits = 0;
      q.ntiles = 0;
      bad = true;
    }
    a.reqs[b] = q;
  }
  if (bad) any_bad = 1;
  __syncthreads();
  if (total_items > a.max_items) total_items = a.max_items;   // only for offsets that do not ascend
  if (tid == 0) {
    a.hdr->total_tiles = min(total_tiles, a.cap_tiles);
    a.hdr->status = any_bad ? kDeviceCheckFailed : 0;
    a.hdr->pad[0] = 0;
    a.hdr->pad[1] = 0;
    a.hdr->pad[2] = total_items;
    a.hdr->pad[3] = 0;
  }
  // query blocks by descending number of key tiles (a counting sort; blocks of equal
  // length in any order): the longest start first, the shortest fill the end
  auto block_of = [&](int i, int& b, int& blk) {
    int lo = 0, hi = a.B - 1;   // the last request with item0 <= i that has a block
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.reqs[mid].item0 <= i) lo = mid; else hi = mid - 1;
    }
    b = lo;
    blk = i - a.reqs[lo].item0;
    const Req q = a.reqs[lo];
    int j0 = 0, j1 = 0;
    if (q.qlen > 0) tile_range(a, q, min(blk * 2 * kTile, q.qlen - 1), min((blk + 1) * 2 * kTile, q.qlen), j0, j1);
    return kBuckets - 1 - min(j1 - j0, kBuckets - 1);
  };
  for (int i = tid; i < total_items; i += kPlanThreads) {
    int b, blk;
    atomicAdd(&hist[block_of(i, b, blk)], 1);
  }
  __syncthreads();
  int h[kBuckets / kPlanThreads], sum = 0, unused;
  for (int i = 0; i < kBuckets / kPlanThreads; ++i) sum += h[i] = hist[tid * (kBuckets / kPlanThreads) + i];
  int at = block_scan(sum, sums, &unused);
  for (int i = 0; i < kBuckets / kPlanThreads; ++i) {
    hist[tid * (kBuckets / kPlanThreads) + i] = at;
    at += h[i];
  }
  __syncthreads();
  for (int i = tid; i < total_items; i += kPlanThreads) {
    int b, blk;
    const int k = block_of(i, b, blk);
    a.items[atomicAdd(&hist[k], 1)] = make_int2(b, blk);
  }
}

// ------------------------------------------------------------------------------ gather

// A block takes 32 rows of a tile, a warp four of them, one after the other: 16 values a
// lane.  All of a warp's rows are located before the first is read.
constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 32;

__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const Args a) {
  __shared__ uint32_t word;
  griddep_launch();
  griddep_wait();
  const int flags = raised(a);
  if (!runs(a, flags)) return;
  const int tile = blockIdx.x / (kTile / kGatherRows), part = blockIdx.x % (kTile / kGatherRows);
  if (tile >= a.hdr->total_tiles) return;
  const bool lat_f16 = a.half && a.fmt == MLA_CACHE_E4M3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lo = request_of(a, tile);
  if (!a.half && !takes(a, flags, lo, true)) return;
  const Req q = a.reqs[lo];
  if (threadIdx.x == 0) word = 0;
  __syncthreads();
  const int L = a.d.kv_lora_rank, R = a.d.qk_rope, ps = a.d.page_size;
  const long long row_bytes = a.fmt == MLA_CACHE_BF16   ? 2ll * (L + R)
                              : a.fmt == MLA_CACHE_E4M3 ? (long long)L + 2 * R
                                                        : (long long)((L / 2 + L / 32 + 15) / 16 * 16) + 2 * R;
  constexpr int kPer = kGatherRows / (kGatherThreads / 32);
  long long phys[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = (tile - q.tile0) * kTile + part * kGatherRows + warp * kPer + i;   // key, relative to q.lo
    phys[i] = -1;
    if (tile - q.tile0 < q.ntiles && k < q.nkeys) {
      const int key = q.lo + k;
      const int page = a.block_table[(size_t)lo * a.bt_stride + key / ps];
      if (page >= 0 && page < a.d.num_pages) phys[i] = (long long)page * ps + key % ps;
      else if (lane == 0) atomicOr(&a.hdr->status, kDeviceCheckFailed);
    }
  }
  const int l0 = lane * 16;
  const bool have = l0 < L;
  uint4 w[kPer][2];
  uint4 rp[kPer];
  uint32_t sb[kPer];
  float rs[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    w[i][0] = w[i][1] = rp[i] = make_uint4(0, 0, 0, 0);
    sb[i] = 0;
    rs[i] = 0.f;
    if (phys[i] < 0) continue;
    const uint8_t* src = a.pool + phys[i] * row_bytes;
    if (have) {
      if (a.fmt == MLA_CACHE_BF16) {
        w[i][0] = *reinterpret_cast<const uint4*>(src + 2 * l0);
        w[i][1] = *reinterpret_cast<const uint4*>(src + 2 * l0 + 16);
      } else if (a.fmt == MLA_CACHE_E4M3) {
        w[i][0] = *reinterpret_cast<const uint4*>(src + l0);
        rs[i] = a.scales[phys[i]];
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src + l0 / 2);
        w[i][0].x = v.x;
        w[i][0].y = v.y;
        sb[i] = src[L / 2 + lane / 2];
      }
    }
    if (lane < R / 8) rp[i] = *reinterpret_cast<const uint4*>(src + row_bytes - 2 * R + 16 * lane);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = part * kGatherRows + warp * kPer + i;
    uint32_t o[8] = {}, top = 0;
    if (phys[i] >= 0 && have) {
      const uint32_t x[8] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w, w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
      if (a.fmt == MLA_CACHE_BF16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = x[e];
      } else if (a.fmt == MLA_CACHE_E4M3) {
        // code x scale, rounded once
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
          const float2 f = __half22float2(__half2(h));
          const float fx = f.x * rs[i], fy = f.y * rs[i];
          top = max(top, max(__float_as_uint(fx) & 0x7FFFFFFFu, __float_as_uint(fy) & 0x7FFFFFFFu));
          o[e] = lat_f16 ? pack_f16(fx, fy) : pack_bf16(fx, fy);
        }
      } else {
        const float s = sb[i] == 255u ? CUDART_NAN_F
                                      : (sb[i] == 0u ? 0x1p-127f : __uint_as_float(sb[i] << 23));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __half2_raw h =
              __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(x[e >> 2] >> (8 * (e & 3))), __NV_E2M1);
          const float2 f = __half22float2(__half2(h));
          o[e] = pack_bf16(f.x * s, f.y * s);
        }
      }
    }
    bool odd = false;   // a NaN or an infinity among this lane's values
    if (a.fmt == MLA_CACHE_E4M3) {
      odd = top >= 0x7F800000u;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) odd |= (o[e] & 0x7F80u) == 0x7F80u || (o[e] & 0x7F800000u) == 0x7F800000u;
    }
    odd = __any_sync(0xffffffffu, odd);
    if (odd) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0;
    }
    const bool lat_holds = f16_holds(top);
    uint32_t rt = 0;
    uint32_t rw[4] = {rp[i].x, rp[i].y, rp[i].z, rp[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x0 = (rw[e] << 16) & 0x7FFFFFFFu, x1 = rw[e] & 0x7FFF0000u;
      if (x0 < 0x7F800000u) rt = max(rt, x0);
      if (x1 < 0x7F800000u) rt = max(rt, x1);
      if (a.half) rw[e] = pack_f16(lo_f(rw[e]), hi_f(rw[e]));
      if (odd && lane < R / 8) rw[e] = 0x7FFF7FFFu;   // NaN in either type
    }
    const bool rope_holds = f16_holds(rt);
    if (a.half && lane == 0 && (!rope_holds || (lat_f16 && !odd && !lat_holds))) raise(a, kGathered, lo);
    rp[i] = make_uint4(rw[0], rw[1], rw[2], rw[3]);
    if (have) {
      uint8_t* box = a.lat + ((size_t)tile * (L / 64) + (l0 >> 6)) * kBox + row * 128;
      const int ch = (l0 & 63) >> 3;
      *reinterpret_cast<uint4*>(box + (((ch) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(box + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (lane < 8) *reinterpret_cast<uint4*>(a.rope + (size_t)tile * kBox + row * 128 + ((lane ^ (row & 7)) << 4)) = rp[i];
    if (lane == 0 && phys[i] >= 0) atomicOr(&word, 1u << (warp * kPer + i));
  }
  __syncthreads();
  if (threadIdx.x == 0) reinterpret_cast<uint32_t*>(a.live)[tile * 4 + part] = word;
}

// e4m3 weights x 128 x 128 block scales -> f16 (bf16 in the second sequence), 8 values a thread.
__global__ void __launch_bounds__(256) widen_weights_kernel(const Args a, const uint8_t* w, const float* scale,
                                                            uint16_t* out, int rows, int cols, long long n8) {
  const int nr = (rows + 127) / 128, nc = (cols + 127) / 128;
  griddep_launch();
  griddep_wait();
  if (!a.half && !runs(a, raised(a))) return;
  bool wide = false;
  for (long long i0 = (long long)blockIdx.x * 256; i0 < n8; i0 += (long long)gridDim.x * 256) {
    const long long i = i0 + threadIdx.x;
    uint32_t top = 0;
    if (i < n8) {
      const long long e0 = i * 8;
      const int c = (int)(e0 % cols), r = (int)(e0 / cols % rows), h = (int)(e0 / cols / rows);
      const float s = scale[((size_t)h * nr + r / 128) * nc + c / 128];   // 8 columns lie in one block
      const uint2 v = reinterpret_cast<const uint2*>(w)[i];
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = (e < 2 ? v.x : v.y) >> (16 * (e & 1));
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
        const float2 f = __half22float2(__half2(hr));
        const float fx = f.x * s, fy = f.y * s;
        top = max(top, max(__float_as_uint(fx) & 0x7FFFFFFFu, __float_as_uint(fy) & 0x7FFFFFFFu));
        o[e] = a.half ? pack_f16(fx, fy) : pack_bf16(fx, fy);
      }
      reinterpret_cast<uint4*>(out)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (!f16_holds(top)) wide = true;   // 256 neighbouring weights
  }
  if (a.half && wide && (threadIdx.x & 31) == 0) raise(a, kWeights, -1);
}

// ------------------------------------------------------------------------------ waits

struct Ctl {
  int abort;
  uint32_t tmem_base;
};

__device__ __forceinline__ bool give_up(uint64_t* bar, Ctl* c, PlanHeader* hdr) {
  const int code = (int)(0x80000000u | ((uint32_t)threadIdx.x << 18) | (smem_u32(bar) & 0x3FFFFu));
  if (atomicCAS(&hdr->pad[0], 0, code) == 0) hdr->pad[1] = (int)blockIdx.x;
  atomicOr(&hdr->status, kDeviceTimeout);
  *reinterpret_cast<volatile int*>(&c->abort) = 1;
  return false;
}
// Bounded wait; after one ran out in this CTA the others return at once.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* c, PlanHeader* hdr) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*reinterpret_cast<volatile int*>(&c->abort)) return false;
  if (mbar_wait(bar, parity, kWaitLimitNs)) return true;
  return give_up(bar, c, hdr);
}
// The same for a warp that goes on together.
__device__ __forceinline__ bool wwait(uint64_t* bar, uint32_t parity, Ctl* c, PlanHeader* hdr) {
  return __all_sync(0xffffffffu, wait(bar, parity, c, hdr));
}
// Barrier of 128 threads that also ands their votes.
__device__ __forceinline__ bool all_of_128(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// ------------------------------------------------------------------------------ expand

// Persistent: a CTA walks (head, key tile) pairs, tiles fastest, so neighbours share the
// head's weights in L2.  Warp 0 loads (A = latent boxes, B = 64 rows of w_uk as they lie,
// N contiguous: the MN-major operand, and 64 columns of w_uv: K-major), warp 1 issues the
// MMAs into one of two 256-column accumulators, warps 2-5 round the other to bf16, lay it
// out as the attention's boxes in shared memory and write each 16 KB box by one bulk copy.
constexpr int kExpStages = 4;
constexpr int kExpThreads = 192;
constexpr int kExpStageBytes = kBox + 2 * (kBox / 2) + kBox;   // A | w_uk two 64 x 64 boxes | w_uv 128 x 64
struct ExpSmem {
  uint64_t full[kExpStages], empty[kExpStages], acc_full[2], acc_empty[2];
  Ctl ctl;
};
constexpr int kExpSmem = 1024 + kExpStages * kExpStageBytes + 2 * kBox + (int)sizeof(ExpSmem);
static_assert(kExpSmem <= 232448, "shared memory");

struct ExpMaps {
  CUtensorMap uk, uv;   // [H * L, N] boxes 64 x 64; [H, V, L] boxes 64 x 1 x 128
};

__global__ void __launch_bounds__(kExpThreads, 1) expand_kernel(const __grid_constant__ ExpMaps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* stg = sm + kExpStages * kExpStageBytes;
  ExpSmem* cs = reinterpret_cast<ExpSmem*>(stg + 2 * kBox);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kExpStages; ++i) {
      mbar_init(&cs->full[i], 1);
      mbar_init(&cs->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cs->acc_full[i], 1);
      mbar_init(&cs->acc_empty[i], 128);
    }
    cs->ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&cs->ctl.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = cs->ctl.tmem_base;
  griddep_launch();
  griddep_wait();
  fence_proxy_async_global();
  const int L = a.d.kv_lora_rank, nkb = L / 64, tiles = a.hdr->total_tiles;
  const int flags = raised(a);
  const long long total = runs(a, flags) ? (long long)tiles * a.hg : 0;
  // with no request flagged by the gather the first sequence takes every tile
  const bool choose = !a.half || (flags & kGathered);
  auto skip = [&](int tile) { return choose && !takes(a, flags, request_of(a, tile), !a.half); };
  const bool in_f16 = a.half && a.fmt == MLA_CACHE_E4M3;   // latents and weights
  PlanHeader* hdr = a.hdr;
  if (blockIdx.x == 0 && tid == 0) hdr->pad[4] = 0;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t bytes = kBox + (uint32_t)a.nbk * (kBox / 2) + kBox;
      int c = 0;
      bool ok = true;
      for (long long w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const int h = a.h0 + (int)(w / tiles), tile = (int)(w % tiles);
        if (choose && skip(tile)) continue;
        for (int kb = 0; kb < nkb; ++kb, ++c) {
          const int s = c % kExpStages;
          if (c >= kExpStages && !(ok = wait(&cs->empty[s], ((c / kExpStages) & 1) ^ 1, &cs->ctl, hdr))) break;
          uint8_t* st = sm + s * kExpStageBytes;
          mbar_arrive_expect_tx(&cs->full[s], bytes);
          bulk_copy_g2s(st, a.lat + ((size_t)tile * nkb + kb) * kBox, kBox, &cs->full[s]);
          for (int i = 0; i < a.nbk; ++i)
            tma_load_2d(st + kBox + i * (kBox / 2), &maps.uk, &cs->full[s], 64 * i, h * L + 64 * kb);
          tma_load_3d(st + 2 * kBox, &maps.uv, &cs->full[s], 64 * kb, 0, h);
        }
      }
      for (int j = c > kExpStages ? c - kExpStages : 0; j < c; ++j)   // nothing in flight when the CTA leaves
        mbar_wait(&cs->full[j % kExpStages], (j / kExpStages) & 1, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // The whole warp walks the loop and one lane issues: the descriptors then are warp-uniform
    // values (in a single-lane loop each instruction first has to move them there).
    const uint32_t type = in_f16 ? kBf16Operands : 0u;
    const uint32_t id_k = idesc_bf16_f32(128, 64 * a.nbk, false, true) ^ type;
    const uint32_t id_v = idesc_bf16_f32(128, 64 * a.nbv, false, false) ^ type;
    const uint32_t base = smem_u32(sm);
    int c = 0, it = 0;
    bool ok = true;
    for (long long w = blockIdx.x; w < total && ok; w += gridDim.x) {
      if (choose && skip((int)(w % tiles))) continue;
      const uint32_t acc = tmem + 256 * (it & 1);
      if (it >= 2 && !(ok = wwait(&cs->acc_empty[it & 1], ((it >> 1) & 1) ^ 1, &cs->ctl, hdr))) break;
      for (int kb = 0; kb < nkb; ++kb, ++c) {
        const int s = c % kExpStages;
        if (!(ok = wwait(&cs->full[s], (c / kExpStages) & 1, &cs->ctl, hdr))) break;
        tc_fence_after();
        const uint32_t st = base + s * kExpStageBytes;
        const uint64_t da = smem_desc(st, 16, 1024, kLayoutSw128);
        const uint64_t dk = smem_desc(st + kBox, kBox / 2, 1024, kLayoutSw128);
        const uint64_t dv = smem_desc(st + 2 * kBox, 16, 1024, kLayoutSw128);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_ss(acc, da + 2 * kk, dk + (uint64_t)((kk * 2048) >> 4), id_k, kb > 0 || kk > 0);
            mma_ss(acc + 128, da + 2 * kk, dv + 2 * kk, id_v, kb > 0 || kk > 0);
          }
          mma_commit(&cs->empty[s]);
        }
        __syncwarp();
      }
      if (ok && elect_one()) mma_commit(&cs->acc_full[it & 1]);
      __syncwarp();
      ++it;
    }
    __syncwarp();
  } else {
    const int q = warp & 3, row = 32 * q + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16);
    const int nb = a.nbk + a.nbv;
    const bool first = tid == 64;   // issues the bulk stores
    int it = 0, n = 0;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
      const int h = (int)(w / tiles), tile = (int)(w % tiles);   // h within the pass
      if (choose && skip(tile)) continue;
      bool wide = false;
      const bool ok = wwait(&cs->acc_full[it & 1], (it >> 1) & 1, &cs->ctl, hdr);
      if (!all_of_128(1, ok)) break;
      tc_fence_after();
      uint8_t* dst = a.kv + ((size_t)h * a.cap_tiles + tile) * nb * kBox;
      for (int b = 0; b < nb; ++b, ++n) {
        const uint32_t col = 256 * (it & 1) + (b < a.nbk ? 64 * b : 128 + 64 * (b - a.nbk));
        uint32_t r[64];
        tmem_ld32(trow + col, *reinterpret_cast<uint32_t(*)[32]>(r));
        tmem_ld32(trow + col + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
        tmem_ld_wait();
        if (b + 1 == nb) {
          tc_fence_before();
          mbar_arrive(&cs->acc_empty[it & 1]);
        }
        // the buffer's last bulk store has read it
        if (first) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        all_of_128(2, true);
        uint8_t* box = stg + (n & 1) * kBox + row * 128;
        uint32_t top = 0;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = r[8 * ch + 2 * e], y = r[8 * ch + 2 * e + 1];
            top = max(top, max(x & 0x7FFFFFFFu, y & 0x7FFFFFFFu));
            o[e] = a.half ? pack_f16(__uint_as_float(x), __uint_as_float(y))
                          : pack_bf16(__uint_as_float(x), __uint_as_float(y));
          }
          *reinterpret_cast<uint4*>(box + ((ch ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        wide |= !f16_holds_row(top);
        fence_proxy_async_smem();
        all_of_128(3, true);
        if (first) {
          bulk_copy_s2g(dst + (size_t)b * kBox, stg + (n & 1) * kBox, kBox);
          bulk_commit();
        }
      }
      if (a.half && wide) raise(a, kExpanded, request_of(a, tile));
      ++it;
    }
    if (first) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------ attend

// A block: 256 query tokens of a request (two sub-blocks A and B of 128) for one head, over a
// range of its key tiles.  TMEM holds S of A and B (128 columns each, P over S) and O of A and
// B: all 512 columns.  Per sub-block and key tile the tensor core does P.V of tile j, then Q.K
// of tile j + 1 into the same S; while the softmax warps of one sub-block work, it has the
// other's two products.  Each sub-block has an issuing warp of its own: the tensor core's queue
// is a few instructions deep, so a single one left it idle during each of its waits (150 cycles
// even for a barrier that has completed, eight a tile).  The two take turns: left alone they
// fall into step, both sub-blocks in their softmax at once and then both at the tensor core.
// K (its first box K0 and the others K12, the last of them the rope) and V stream through
// eight places of a box: two for K0 and three pairs.  K12 of tile n lies in pair n % 3, V of
// tile n in the pair that K12 of tile n - 1 left, K0 in place n % 2.  So V(n + 1) and
// K0(n + 2) load when Q.K(n) is done, K12(n + 2) when P.V(n) is: the ten boxes of two tiles do
// not fit beside the queries, and these are the ones needed last.
// A CTA stays on its SM and takes block after block, tiles counted through; a block's queries
// load when the last Q.K of the block before is done, its first keys earlier.
// Warp 0 loads, warps 1 and 2 issue, warp 3 names the blocks, warps 4-7 and 8-11 are the
// softmax of A and B: thread = query token = TMEM lane.  A softmax thread holds a row of 128
// scores: the 168 registers that 384 threads get at launch are split 104 / 200 between the
// warpgroups (384 x 168 = 128 x 104 + 256 x 200).
// Measured, 16,384 tokens x 16 heads: 2,230 us with one barrier a box, 1,184 with one a tile
// and the register split, 1,125 with two issuers, 989 with turns and these places, 978 block
// after block, 895 with the blocks in a better order (1,610 TFLOP/s over the whole call; 3,260
// cycles a step of 256 x 128, of which the products take 96 %).  Those are runs of some 20 calls;
// in longer ones the power cap makes it 967 (1,490 TFLOP/s).  Prompts of 1,500 to 2,300 tokens,
// 128 heads: 718, 690 and 648 us with the last three; what is left there is a block's own start and end, about 13,000 cycles in which
// the queries are converted and the rows of O leave by stores of 16 bytes a row (32-byte
// stores, staging, and the next block's queries converted before this one's O is written were
// all slower).
constexpr int kSlots = 8;
// First byte of a place: K0 of tile n, K12 of tile n, V of tile n.
__device__ __forceinline__ uint32_t place_k0(int n) { return (6 + (n & 1)) * kBox; }
__device__ __forceinline__ uint32_t place_k12(int n) { return n % 3 * 2 * kBox; }
__device__ __forceinline__ uint32_t place_v(int n) { return (n + 2) % 3 * 2 * kBox; }
constexpr int kAttThreads = 384;
constexpr float kRescaleThreshold = 8.0f;   // log2: O is rescaled when a row's maximum grows by more than 2^8

// What a CTA works on: kept in shared memory, read where it is used (the softmax threads
// have no registers to keep it in).
struct Block {
  Req q;
  int r0, nsub, h, split;     // first query row, sub-blocks, head of the pass (-1: no more), key split
  int j0[2], j1[2], js, je;   // key tiles of each sub-block, and of both
};
constexpr long long kGroupBytes = 64ll << 20;   // half the L2
constexpr int kBlocks = 4;      // blocks known ahead
constexpr int kBlockUsers = 11; // warps that read a block: loads, two issuers, eight of the softmax
struct AttSmem {
  uint64_t k0_full[2], k12_full[2], k_empty[2], v_full[2], v_empty[2], turn[2][2], q_full, q_ready[2], s_full[2], p_full[2], o_full[2];
  uint64_t blk_full[kBlocks], blk_empty[kBlocks], want;
  Ctl ctl;
  Block blk[kBlocks];
};
constexpr int kMaxQBoxes = 3;
constexpr int kAttSmem = 1024 + 2 * kMaxQBoxes * kBox + kSlots * kBox + (int)sizeof(AttSmem);
static_assert(kAttSmem <= 232448, "shared memory");

struct AttMaps {
  CUtensorMap qn, qr;   // queries: [T, H, N] and [T, H, R] of rows of N + R, boxes 64 x 1 x 128
};

// Bits [0, n) of a word.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// Block `at`: split fastest, then head, then query block (the longest first, so that the SMs
// finish together), in groups of as many heads as keep their keys and values in half the L2
// (16,384 tokens x 16 heads 978 us head by head, 895 so; 927 and 902 with 16 and 128 MB).
// A block of a request that the other sequence takes becomes one without query tokens.
__device__ __forceinline__ void set_block(const Args& a, int nitems, long long at, int flags, Block& k) {
  const long long head = (long long)max(a.hdr->total_tiles, 1) * (a.nbk + a.nbv) * kBox, i = at / a.splits;
  const int group = (int)min((long long)a.hg, max(1ll, kGroupBytes / head));
  const int h0 = (int)(i / ((long long)group * nitems)) * group, heads = min(group, a.hg - h0);
  const long long in = i - (long long)h0 * nitems;
  const int split = (int)(at % a.splits), item = (int)(in / heads);
  const int2 it = a.items[item];
  Req q = a.reqs[it.x];
  if (flags && !takes(a, flags, it.x, true)) q.qlen = 0;
  const int r0 = it.y * 2 * kTile, nsub = q.qlen > r0 + kTile ? 2 : 1;
  int j0[2] = {0, 0}, j1[2] = {0, 0};
  if (q.fits && q.qlen > 0)
    for (int s = 0; s < nsub; ++s)
      tile_range(a, q, r0 + s * kTile, min(r0 + (s + 1) * kTile, q.qlen), j0[s], j1[s]);
  const bool on0 = j1[0] > j0[0], on1 = j1[1] > j0[1];
  int js = on0 ? (on1 ? min(j0[0], j0[1]) : j0[0]) : j0[1], je = on0 ? (on1 ? max(j1[0], j1[1]) : j1[0]) : max(j1[1], js);
  if (a.splits > 1) {   // this split's share of the block's key tiles
    const int n = je - js, b = js;
    js = b + (int)((long long)n * split / a.splits);
    je = b + (int)((long long)n * (split + 1) / a.splits);
    for (int s = 0; s < 2; ++s) {
      j0[s] = max(j0[s], js);
      j1[s] = max(j0[s], min(j1[s], je));
    }
  }
  k.q = q;
  k.r0 = r0;
  k.nsub = nsub;
  k.h = h0 + (int)(in % heads);
  k.split = split;
  for (int s = 0; s < 2; ++s) {
    k.j0[s] = j0[s];
    k.j1[s] = j1[s];
  }
  k.js = js;
  k.je = je;
}

template <bool kHalf>
__global__ void __launch_bounds__(kAttThreads, 1) attend_kernel(const __grid_constant__ AttMaps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = sm;
  uint8_t* ring = sQ + 2 * kMaxQBoxes * kBox;
  AttSmem* cs = reinterpret_cast<AttSmem*>(ring + kSlots * kBox);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  PlanHeader* hdr = a.hdr;
  griddep_launch();
  griddep_wait();
  fence_proxy_async_global();
  const int flags = raised(a);
  if (!runs(a, flags)) return;
  const int nitems = hdr->pad[2];
  const long long nblocks = (long long)a.splits * nitems * a.hg;
  if (warp == 1) {
    tmem_alloc(&cs->ctl.tmem_base, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    cs->ctl.abort = 0;
    mbar_init(&cs->q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cs->k0_full[i], 1);
      mbar_init(&cs->k12_full[i], 1);
      mbar_init(&cs->k_empty[i], 2);
      mbar_init(&cs->v_full[i], 1);
      mbar_init(&cs->v_empty[i], 2);
      mbar_init(&cs->turn[i][0], 1);
      mbar_init(&cs->turn[i][1], 1);
      mbar_init(&cs->q_ready[i], 128);
      mbar_init(&cs->s_full[i], 1);
      mbar_init(&cs->p_full[i], 128);
      mbar_init(&cs->o_full[i], 1);
    }
    mbar_init(&cs->want, 1);
    for (int i = 0; i < kBlocks; ++i) {
      mbar_init(&cs->blk_full[i], 1);
      mbar_init(&cs->blk_empty[i], kBlockUsers);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = cs->ctl.tmem_base;
  // Block i of this CTA, for a warp that uses it; its place is given back by `done_with`.
  // A role that has nothing to do in a block waits it out: 2^28 keys take 4 seconds.
  auto long_wait = [&](uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < 20; ++i) {
      if (mbar_wait(bar, parity, kWaitLimitNs)) return true;
      if (*reinterpret_cast<volatile int*>(&cs->ctl.abort)) return false;
    }
    return give_up(bar, &cs->ctl, hdr);
  };
  auto block = [&](int i) {
    return __all_sync(0xffffffffu, long_wait(&cs->blk_full[i % kBlocks], (i / kBlocks) & 1));
  };
  auto done_with = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&cs->blk_empty[i % kBlocks]);
  };

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (warp == 3) {
    // Which blocks: the first by the CTA's number, then whatever nobody took yet, one at a time
    // and as late as the loads allow (with four taken ahead the last ones were spread badly:
    // 16,384 tokens x 16 heads 1,159 instead of 978 us).
    if (lane == 0) {
      for (int i = 0;; ++i) {
        if (i > 0 && !long_wait(&cs->want, (i - 1) & 1)) break;
        if (i >= kBlocks && !wait(&cs->blk_empty[i % kBlocks], ((i / kBlocks) & 1) ^ 1, &cs->ctl, hdr)) break;
        const long long at = i == 0 ? blockIdx.x : (long long)gridDim.x + atomicAdd(&hdr->pad[4], 1);
        Block& k = cs->blk[i % kBlocks];
        if (at < nblocks) set_block(a, nitems, at, flags, k);
        else k.h = -1;
        mbar_arrive(&cs->blk_full[i % kBlocks]);
        if (at >= nblocks) break;
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    if (lane == 0) {
      // Key tiles are counted through the CTA's blocks.  Step n: V of tile n + 1, K of tile n + 2,
      // and the queries of a block as its first tile becomes n + 1, when the block before has
      // done its last Q.K.  A: the block of tile n + 1, B: the one after it, once it is known.
      const int nb = a.nbk + a.nbv;
      const uint8_t *kv_a = nullptr, *kv_b = nullptr, *rope_a = nullptr, *rope_b = nullptr;   // of its tile 0, were it the CTA's first
      int end_a = 0, end_b = 0, t_b = 0, h_b = 0, two_b = 0;
      bool have_b = false, stop = false, ok = true;
      int nblk = 0, nq = 0, nk0 = 0, nk12 = 0, nv = 0;   // blocks read; loads of each kind
      int nasked = 1;                                    // blocks asked for, the first by itself
      auto ask = [&]() {
        if (nasked > nblk) return;
        mbar_arrive(&cs->want);
        ++nasked;
      };
      auto next_block = [&]() {
        for (; !have_b && !stop && ok; ++nblk) {
          ask();
          if (!(ok = wait(&cs->blk_full[nblk % kBlocks], (nblk / kBlocks) & 1, &cs->ctl, hdr))) return;
          const Block& k = cs->blk[nblk % kBlocks];
          if ((stop = k.h < 0)) return;
          if (k.je > k.js) {
            have_b = true;
            h_b = k.h;
            t_b = k.q.q0 + k.r0;
            two_b = k.nsub > 1;
            end_b = end_a + (k.je - k.js);
            const long long first = (long long)k.q.tile0 + k.js;
            kv_b = a.kv + ((long long)h_b * a.cap_tiles + first - end_a) * nb * kBox;
            rope_b = a.rope + (first - end_a) * kBox;
          }
          mbar_arrive(&cs->blk_empty[nblk % kBlocks]);
        }
      };
      for (int n = -2; ok; ++n) {
        if (n >= 0 && !(ok = wait(&cs->k_empty[n & 1], (n >> 1) & 1, &cs->ctl, hdr))) break;
        if (n >= -1) {
          if (n + 1 == end_a) {
            if (!have_b) break;   // no more
            kv_a = kv_b;
            rope_a = rope_b;
            end_a = end_b;
            have_b = false;
            mbar_arrive_expect_tx(&cs->q_full, (uint32_t)(2 * a.nbq * kBox));
            for (int s = 0; s < 2; ++s)
              for (int i = 0; i < a.nbq; ++i) {
                uint8_t* dst = sQ + (s * a.nbq + i) * kBox;
                const int t = t_b + (s & two_b) * kTile;   // a block of one sub-block loads it twice
                if (i < a.nbk) tma_load_3d(dst, &maps.qn, &cs->q_full, 64 * i, a.h0 + h_b, t);
                else tma_load_3d(dst, &maps.qr, &cs->q_full, 0, a.h0 + h_b, t);
              }
            ++nq;
          }
          mbar_arrive_expect_tx(&cs->v_full[nv & 1], (uint32_t)(a.nbv * kBox));
          bulk_copy_g2s(ring + place_v(nv), kv_a + ((long long)nv * nb + a.nbk) * kBox, (uint32_t)(a.nbv * kBox),
                        &cs->v_full[nv & 1]);
          ++nv;
        }
        if (n + 5 >= end_a && !have_b && !stop) ask();
        const uint8_t *kv = kv_a, *rope = rope_a;
        if (n + 2 >= end_a) {
          next_block();
          if (!have_b) continue;
          kv = kv_b;
          rope = rope_b;
        }
        mbar_arrive_expect_tx(&cs->k0_full[nk0 & 1], kBox);
        bulk_copy_g2s(ring + place_k0(nk0), kv + (long long)nk0 * nb * kBox, kBox, &cs->k0_full[nk0 & 1]);
        ++nk0;
        if (n >= 0 && !(ok = wait(&cs->v_empty[n & 1], (n >> 1) & 1, &cs->ctl, hdr))) break;
        mbar_arrive_expect_tx(&cs->k12_full[nk12 & 1], (uint32_t)(a.nbk * kBox));
        if (a.nbk > 1)
          bulk_copy_g2s(ring + place_k12(nk12), kv + ((long long)nk12 * nb + 1) * kBox, kBox, &cs->k12_full[nk12 & 1]);
        bulk_copy_g2s(ring + place_k12(nk12) + (a.nbk - 1) * kBox, rope + (long long)nk12 * kBox, kBox,
                      &cs->k12_full[nk12 & 1]);
        ++nk12;
      }
      // nothing in flight when the CTA leaves: the last loads of each kind
      for (int i = max(nk0 - 2, 0); i < nk0; ++i) mbar_wait(&cs->k0_full[i & 1], (i >> 1) & 1, kWaitLimitNs);
      for (int i = max(nk12 - 2, 0); i < nk12; ++i) mbar_wait(&cs->k12_full[i & 1], (i >> 1) & 1, kWaitLimitNs);
      for (int i = max(nv - 2, 0); i < nv; ++i) mbar_wait(&cs->v_full[i & 1], (i >> 1) & 1, kWaitLimitNs);
      if (nq > 0) mbar_wait(&cs->q_full, (nq - 1) & 1, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // One sub-block's products.  The whole warp walks the loop, one lane issues (as in the
    // expansion).  For a key tile that this sub-block does not use it only passes the data on.
    const int s = warp - 1;
    const uint32_t type = kHalf ? kBf16Operands : 0u;
    const uint32_t id_s = idesc_bf16_f32(128, 128, false, false) ^ type;
    const uint32_t id_o = idesc_bf16_f32(128, 64 * a.nbv, false, true) ^ type;
    const uint64_t dq0 = smem_desc(smem_u32(sQ) + s * a.nbq * kBox, 16, 1024, kLayoutSw128);
    const uint64_t dr0 = smem_desc(smem_u32(ring), 16, 1024, kLayoutSw128);
    const uint64_t dv0 = smem_desc(smem_u32(ring), kBox, 1024, kLayoutSw128);
    constexpr uint64_t kBoxStep = kBox >> 4;
    const int nbq = a.nbq;
    const uint32_t ts = tmem + 128 * s, to = tmem + 256 + 128 * s;
    bool ok = true;
    int n0 = 0, np = 0, nblk = 0;      // key tiles of the blocks before, P tiles taken, blocks with tiles
    // A may be in the next block while B has its last turn of this one before it, so blocks
    // alternate between two barriers each
    int par = 0, nturn[2] = {0, 0};
    for (int i = 0; ok; ++i) {
      if (!(ok = block(i))) break;
      const Block& blk = cs->blk[i % kBlocks];
      if (blk.h < 0) break;
      const int js = blk.js, je = blk.je, ja = blk.j0[s], jb = blk.j1[s];
      const bool both = jb > ja && blk.j1[s ^ 1] > blk.j0[s ^ 1];
      done_with(i);
      if (je <= js) continue;
      // waited for in every block with tiles, used or not: a barrier's parity tells one phase from
      // the next only, so neither side may be two ahead
      if (!(ok = wwait(&cs->q_ready[s], nblk++ & 1, &cs->ctl, hdr))) break;
      bool add = false;   // O holds something
      // Group n: O (+)= P V of key tile n - 1, then S = Q K^T of key tile n
      int n = n0;
      for (int j = js; j <= je && ok; ++j, ++n) {
        const bool use_v = j > js && j - 1 >= ja && j - 1 < jb, use_k = j >= ja && j < jb;
        const int v = n - 1;
        if (j < je && !(ok = wwait(&cs->k0_full[n & 1], (n >> 1) & 1, &cs->ctl, hdr))) break;
        if (j > js && !(ok = wwait(&cs->v_full[v & 1], (v >> 1) & 1, &cs->ctl, hdr))) break;
        if (use_v && !(ok = wwait(&cs->p_full[s], np & 1, &cs->ctl, hdr))) break;
        // the sub-blocks take turns, A first in each block
        if (both && (s == 1 || j > js)) {
          const int t = par ? nturn[1]++ : nturn[0]++;
          if (!(ok = wwait(&cs->turn[s][par], t & 1, &cs->ctl, hdr))) break;
        }
        tc_fence_after();
        const uint64_t dv = dv0 + (place_v(v + 3) >> 4), dk0 = dr0 + (place_k0(n) >> 4), dk12 = dr0 + (place_k12(n) >> 4);
        if (elect_one()) {
          if (use_v) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(to, ts + 8 * kk, dv + (uint64_t)((kk * 2048) >> 4), id_o, add || kk > 0);
            if (j == jb) mma_commit(&cs->o_full[s]);
            mma_commit(&cs->v_empty[v & 1]);
          } else if (j > js) {
            mbar_arrive(&cs->v_empty[v & 1]);
          }
          // columns past a row's end are zero on both sides
          if (use_k) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss(ts, dq0 + 2 * kk, dk0 + 2 * kk, id_s, kk > 0);
          }
        }
        __syncwarp();
        if (j < je && !(ok = wwait(&cs->k12_full[n & 1], (n >> 1) & 1, &cs->ctl, hdr))) break;
        tc_fence_after();
        if (elect_one()) {
          for (int b = 1; b < nbq && use_k; ++b) {
            const uint64_t dq = dq0 + b * kBoxStep, dk = dk12 + (b - 1) * kBoxStep;
            if (b == nbq - 1 && both) mbar_arrive(&cs->turn[s ^ 1][par]);   // its wait passes under the last box
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss(ts, dq + 2 * kk, dk + 2 * kk, id_s, 1u);
          }
          if (use_k) {
            mma_commit(&cs->s_full[s]);
            mma_commit(&cs->k_empty[n & 1]);
          } else {
            if (both && (s == 0 || j < je)) mbar_arrive(&cs->turn[s ^ 1][par]);
            if (j < je) mbar_arrive(&cs->k_empty[n & 1]);
          }
        }
        __syncwarp();
        if (use_v) {
          ++np;
          add = true;
        }
      }
      n0 += je - js;
      par ^= both;
    }
    // the last signals have arrived before the barriers go away
    if (ok && n0 > 0) wwait(&cs->v_empty[(n0 - 1) & 1], ((n0 - 1) >> 1) & 1, &cs->ctl, hdr);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int s = warp >= 8 ? 1 : 0;
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * quad) << 16), ts = trow + 128 * s, to = trow + 256 + 128 * s;
    uint32_t phase = 0;   // bit 0: of s_full, bit 1: of q_full, bit 2: of o_full
    bool ok = true;
    for (int at = 0; ok; ++at) {
    if (!(ok = block(at))) break;
    const Block& blk = cs->blk[at % kBlocks];
    if (blk.h < 0) break;
    const int ja = blk.j0[s], jb = blk.j1[s];
    const bool live = jb > ja;
    // this row's keys [lo, hi); the sub-block's first and last row bound what needs no mask
    int lo, hi, lo_last, hi_first;
    {
      const int r = blk.r0 + s * kTile, last = blk.q.qlen - 1;
      int unused;
      row_range(a, blk.q, min(r + row, last), lo, hi);
      row_range(a, blk.q, min(r + kTile - 1, last), lo_last, unused);
      row_range(a, blk.q, min(r, last), unused, hi_first);
    }
    float sl2 = a.scale * 1.4426950408889634f;
    if (blk.je > blk.js) {   // waited for whether used or not, as q_ready is
      ok = wwait(&cs->q_full, (phase >> 1) & 1, &cs->ctl, hdr);
      phase ^= 2;
    }
    if (live) {
      // this thread's query row: bf16 -> f16, scaled to a largest magnitude in [2^10, 2^11);
      // a scale below zero turns its sign, a scale of zero its values to zero
      if (ok && (kHalf || !(sl2 > 0.f))) {
        uint8_t* qr = sQ + s * a.nbq * kBox + row * 128;
        __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);   // a NaN does not count: its row is NaN anyhow
        for (int i = 0; i < a.nbq && kHalf; ++i)
#pragma unroll 4
          for (int ch = 0; ch < 8; ++ch) {
            const uint4 v = *reinterpret_cast<const uint4*>(qr + i * kBox + ((ch ^ (row & 7)) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
          }
        const uint32_t tw = *reinterpret_cast<const uint32_t*>(&top2), top = max(tw & 0xFFFFu, tw >> 16);
        const int k = (top >= 0x7F80u || top == 0u ? 10 : max((int)(top >> 7) - 127, -110)) - 10;
        const float f = (sl2 > 0.f ? 1.f : (sl2 < 0.f ? -1.f : 0.f)) * __uint_as_float((uint32_t)(127 - k) << 23);
        auto put = [&](uint32_t v) {
          return kHalf ? pack_f16(lo_f(v) * f, hi_f(v) * f) : pack_bf16(lo_f(v) * f, hi_f(v) * f);
        };
        for (int i = 0; i < a.nbq; ++i)
#pragma unroll 4
          for (int ch = 0; ch < 8; ++ch) {
            uint4* p = reinterpret_cast<uint4*>(qr + i * kBox + ((ch ^ (row & 7)) << 4));
            const uint4 v = *p;
            *p = make_uint4(put(v.x), put(v.y), put(v.z), put(v.w));
          }
        sl2 = sl2 == 0.f ? 1.f : fabsf(sl2);
        // times 2^k in two steps: 2^k alone may leave the normal range
        sl2 = sl2 * __uint_as_float((uint32_t)(k / 2 + 127) << 23) * __uint_as_float((uint32_t)(k - k / 2 + 127) << 23);
        fence_proxy_async_smem();
      }
    }
    if (blk.je > blk.js) mbar_arrive(&cs->q_ready[s]);
    float m = -CUDART_INF_F, l = 0.f;
    const uint4* live_rows = a.live + blk.q.tile0;
    if (ok && s < blk.nsub) {
      for (int j = ja; j < jb; ++j) {
        const uint4 lv = __ldcg(live_rows + j);   // its latency passes in the wait
        if (!(ok = wwait(&cs->s_full[s], phase & 1, &cs->ctl, hdr))) break;
        phase ^= 1;
        tc_fence_after();
        float x[128];
        const int k0 = j * kTile;
        const bool all = (lv.x & lv.y & lv.z & lv.w) == ~0u && k0 + kTile <= hi_first && k0 >= lo_last;
        auto scores = [&]() {   // S of this row, -inf where the key is not visible
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * i));
          tmem_ld_wait();
          if (!all) {
            const uint32_t lw[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t see = lw[w] & low_bits(hi - k0 - 32 * w) & ~low_bits(lo - k0 - 32 * w);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[32 * w + i] = (see >> i) & 1u ? x[32 * w + i] : -CUDART_INF_F;
            }
          }
        };
        scores();
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = fmaxf(fmaxf(m4[e], x[i + e]), x[i + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], x[124 + e]);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
        const bool want = m != -CUDART_INF_F && mx > m + kRescaleThreshold;
        if (__any_sync(0xffffffffu, want)) {
          // S of this tile is complete, so P.V of the last one is too (same issuing thread)
          const float alpha = want ? ex2(m - mx) : 1.f;
#pragma unroll 1
          for (int col = 0; col < 64 * a.nbv; col += 32) {
            uint32_t o[32];
            tmem_ld32(to + col, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(to + col, o);
          }
          if (want) {
            l *= alpha;
            m = mx;
          }
          scores();   // read again: a row of scores and one of O do not fit the registers together
        }
        if (m == -CUDART_INF_F) m = mx;   // the row's first visible key
        const float neg = m == -CUDART_INF_F ? 0.f : -m;
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float* v = x + 32 * i + 2 * e;
            fma_pair(v[0], v[1], sl2, neg);
            fma_pair(v[2], v[3], sl2, neg);
            v[0] = ex2(v[0]);
            v[1] = ex2(v[1]);
            v[2] = ex2(v[2]);
            v[3] = ex2(v[3]);
            add_pair(l0, l1, v[0], v[1]);
            add_pair(l2, l3, v[2], v[3]);
            p[e] = kHalf ? pack_f16(v[0], v[1]) : pack_bf16(v[0], v[1]);
            p[e + 1] = kHalf ? pack_f16(v[2], v[3]) : pack_bf16(v[2], v[3]);
          }
          tmem_st16(ts + 16 * i, p);
        }
        l += (l0 + l1) + (l2 + l3);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&cs->p_full[s]);
      }
      // epilogue
      if (ok && live) ok = wwait(&cs->o_full[s], (phase >> 2) & 1, &cs->ctl, hdr);
      if (live) phase ^= 4;
      tc_fence_after();
      const volatile Block* vb = &cs->blk[at % kBlocks];   // read again: nothing of it was kept
      const int r = vb->r0 + s * kTile + row;
      const bool mine = ok && r < vb->q.qlen, fits = vb->q.fits != 0;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : CUDART_NAN_F);
      const float lse = !fits ? CUDART_NAN_F : (l == 0.f ? -CUDART_INF_F : (m + __log2f(l)) * 0.6931471805599453f);
      const size_t th = (size_t)(vb->q.q0 + r) * a.d.num_heads + a.h0 + vb->h;
      const size_t sp = (size_t)vb->split * a.T * a.d.num_heads;
      const int V = a.d.v_head;
      // This code and the queries' conversion run once a block, from a cold instruction cache:
      // few instructions and rolled loops (one prompt of 1,900 tokens 257 -> 245 us).
      const bool some = live && fits && l != 0.f;
      const float fill = fits ? 0.f : CUDART_NAN_F;
#pragma unroll 1
      for (int col = 0; col < V; col += 32) {
        uint32_t o[32];
        if (live) {
          tmem_ld32(to + col, o);
          tmem_ld_wait();
        }
        if (!mine) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(some ? __uint_as_float(o[i]) * inv : fill);
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          if (col + i >= V) break;
          if (a.splits == 1) {
            *reinterpret_cast<uint4*>(a.out + th * V + col + i) =
                make_uint4(pack_bf16(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                           pack_bf16(__uint_as_float(o[i + 2]), __uint_as_float(o[i + 3])),
                           pack_bf16(__uint_as_float(o[i + 4]), __uint_as_float(o[i + 5])),
                           pack_bf16(__uint_as_float(o[i + 6]), __uint_as_float(o[i + 7])));
          } else {
            uint4* d = reinterpret_cast<uint4*>(a.part_o + (sp + th) * V + col + i);
            d[0] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            d[1] = make_uint4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
          }
        }
      }
      if (mine) {
        if (a.splits > 1) a.part_lse[sp + th] = lse;
        else if (a.lse_out) a.lse_out[th] = lse;
      }
    }
    tc_fence_before();   // O is read
    done_with(at);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------ combine

// A warp per (token, head): lse = ln sum_s e^lse_s, out = sum_s e^(lse_s - lse) o_s, in order.
__global__ void __launch_bounds__(256) combine_kernel(const Args a) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31, H = a.d.num_heads, V = a.d.v_head;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5), n = (long long)a.T * H;
  const int last = (int)min(a.offsets[a.B], (uint32_t)a.T);   // tokens behind the last request stay as they were
  if (i >= n || i / H >= last) return;
  float mx = -CUDART_INF_F;
  bool nan = false;
  for (int s = 0; s < a.splits; ++s) {
    const float v = a.part_lse[s * n + i];
    nan |= v != v;
    mx = fmaxf(mx, v);
  }
  float sum = 0.f;
  if (mx != -CUDART_INF_F)
    for (int s = 0; s < a.splits; ++s) sum += __expf(a.part_lse[s * n + i] - mx);
  for (int c = 4 * lane; c < V; c += 128) {
    float o[4] = {};
    if (mx != -CUDART_INF_F)
      for (int s = 0; s < a.splits; ++s) {
        const float w = __expf(a.part_lse[s * n + i] - mx) / sum;
        const float4 v = *reinterpret_cast<const float4*>(a.part_o + (s * n + i) * V + c);
        o[0] = fmaf(w, v.x, o[0]);
        o[1] = fmaf(w, v.y, o[1]);
        o[2] = fmaf(w, v.z, o[2]);
        o[3] = fmaf(w, v.w, o[3]);
      }
    if (nan) o[0] = o[1] = o[2] = o[3] = CUDART_NAN_F;
    *reinterpret_cast<uint2*>(a.out + i * V + c) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
  }
  if (lane == 0 && a.lse_out)
    a.lse_out[i] = nan ? CUDART_NAN_F : (mx == -CUDART_INF_F ? mx : mx + __logf(sum));
}

// ------------------------------------------------------------------------------ host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// bf16, 128-byte swizzle, boxes 64 columns wide; `rank` sizes innermost first, strides in bytes.
bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const cuuint32_t es[3] = {1, 1, 1};
  EncodeTiledFn fn = encode_fn();
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class... P, class... A>
cudaError_t start(void (*kernel)(P...), unsigned grid, int threads, int smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set-up overlaps the previous kernel's end
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pf

bool prefill_supported(const mla_dims_t& d) {
  return d.kv_lora_rank % 64 == 0 && d.kv_lora_rank >= 64 && d.kv_lora_rank <= 512 && d.qk_nope % 8 == 0 &&
         d.qk_nope >= 8 && d.qk_nope <= 128 && d.qk_rope % 8 == 0 && d.qk_rope >= 8 && d.qk_rope <= 64 &&
         d.v_head % 8 == 0 && d.v_head >= 8 && d.v_head <= 128;
}

PrefillLayout prefill_layout(const mla_dims_t& d, int B, int T, long long total_keys, int splits, bool fp8) {
  auto up = [](size_t x) { return (x + 1023) & ~size_t(1023); };
  PrefillLayout w{};
  // every request rounds its keys up to whole tiles: at most one tile each
  w.cap_tiles = total_keys / pf::kTile + B;
  w.max_items = (long long)T / (2 * pf::kTile) + B;
  const size_t L = d.kv_lora_rank, H = d.num_heads, tiles = (size_t)w.cap_tiles;
  size_t o = 0;
  w.header = o; o = up(o + sizeof(PlanHeader));
  w.reqs = o;   o = up(o + sizeof(pf::Req) * B);
  w.items = o;  o = up(o + sizeof(int2) * (size_t)w.max_items);
  w.live = o;   o = up(o + 16 * tiles);
  w.rope = o;   o = up(o + tiles * pf::kBox);
  w.lat = o;    o = up(o + tiles * (L / 64) * pf::kBox);
  w.w_uk = o;   o = up(o + (fp8 ? H * L * d.qk_nope * 2 : 0));
  w.w_uv = o;   o = up(o + (fp8 ? H * L * d.v_head * 2 : 0));
  w.part_o = o; o = up(o + (splits > 1 ? (size_t)splits * T * H * d.v_head * 4 : 0));
  w.part_lse = o; o = up(o + (splits > 1 ? (size_t)splits * T * H * 4 : 0));
  w.kv = o;
  w.head_bytes = tiles * ((d.qk_nope + 63) / 64 + (d.v_head + 63) / 64) * pf::kBox;
  return w;
}

// Key splits: one, unless the query blocks of a call leave SMs idle; then as many as fill
// them, each of at least four key tiles on average (a split's start, its first load and
// its partial result cost about as much as two).
int prefill_splits(const mla_dims_t& d, int B, int T, long long total_keys, int sms) {
  const long long ctas = ((long long)T + 2 * pf::kTile - 1) / (2 * pf::kTile) * d.num_heads;
  if (ctas <= 0 || ctas * 2 > sms) return 1;
  const long long tiles = total_keys / pf::kTile / std::min(B, T);
  return (int)std::max(1ll, std::min((long long)sms / ctas, tiles / 4));
}

cudaError_t launch_prefill(const PrefillCall& c, const PrefillLayout& lay, int heads, int splits, cudaStream_t s) {
  using namespace pf;
  if (c.T == 0) return cudaSuccess;
  const mla_dims_t& d = c.d;
  const int N = d.qk_nope, R = d.qk_rope, L = d.kv_lora_rank, V = d.v_head, H = d.num_heads;
  char* ws = static_cast<char*>(c.ws);
  Args a{};
  a.d = d;
  a.fmt = c.fmt;
  a.B = c.B;
  a.T = c.T;
  a.mask = c.mask;
  a.window = std::min(c.window, 1 << 30);   // more than a call can hold keys; positions less a window stay in 32 bits
  a.scale = c.scale;
  a.bt_stride = c.bt_stride;
  a.cap_tiles = (int)lay.cap_tiles;
  a.max_items = (int)lay.max_items;
  a.nbk = (N + 63) / 64;
  a.nbv = (V + 63) / 64;
  a.nbq = a.nbk + 1;
  a.splits = splits;
  a.offsets = c.offsets;
  a.cache_lens = c.cache_lens;
  a.block_table = c.block_table;
  a.pool = static_cast<const uint8_t*>(c.pool);
  a.scales = c.kv_scales;
  a.hdr = reinterpret_cast<PlanHeader*>(ws + lay.header);
  a.reqs = reinterpret_cast<Req*>(ws + lay.reqs);
  a.items = reinterpret_cast<int2*>(ws + lay.items);
  a.live = reinterpret_cast<uint4*>(ws + lay.live);
  a.rope = reinterpret_cast<uint8_t*>(ws + lay.rope);
  a.lat = reinterpret_cast<uint8_t*>(ws + lay.lat);
  a.kv = reinterpret_cast<uint8_t*>(ws + lay.kv);
  a.part_o = reinterpret_cast<float*>(ws + lay.part_o);
  a.part_lse = reinterpret_cast<float*>(ws + lay.part_lse);
  a.out = static_cast<__nv_bfloat16*>(c.out);
  a.lse_out = c.lse_out;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;

  const void *w_uk = c.w_uk, *w_uv = c.w_uv;
  if (c.w_uk_scale) {
    w_uk = ws + lay.w_uk;
    w_uv = ws + lay.w_uv;
  }
  ExpMaps em;
  AttMaps am;
  {
    const cuuint64_t dk[2] = {(cuuint64_t)N, (cuuint64_t)H * L}, sk[1] = {(cuuint64_t)N * 2};
    const cuuint32_t bk[2] = {64, 64};
    const cuuint64_t dv[3] = {(cuuint64_t)L, (cuuint64_t)V, (cuuint64_t)H};
    const cuuint64_t sv[2] = {(cuuint64_t)L * 2, (cuuint64_t)L * V * 2};
    const cuuint32_t bv[3] = {64, 128, 1};
    const cuuint64_t sq[2] = {(cuuint64_t)(N + R) * 2, (cuuint64_t)H * (N + R) * 2};
    const cuuint64_t dn[3] = {(cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)c.T};
    const cuuint64_t dr[3] = {(cuuint64_t)R, (cuuint64_t)H, (cuuint64_t)c.T};
    const cuuint32_t bq[3] = {64, 1, 128};
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(c.q);
    if (!encode(&em.uk, w_uk, 2, dk, sk, bk) || !encode(&em.uv, w_uv, 3, dv, sv, bv) ||
        !encode(&am.qn, q, 3, dn, sq, bq) || !encode(&am.qr, q + N, 3, dr, sq, bq))
      return cudaErrorInvalidValue;
  }
  if ((e = ensure_smem_limit(reinterpret_cast<const void*>(expand_kernel), kExpSmem)) != cudaSuccess) return e;
  if ((e = ensure_smem_limit(reinterpret_cast<const void*>(attend_kernel<true>), kAttSmem)) != cudaSuccess) return e;
  if ((e = ensure_smem_limit(reinterpret_cast<const void*>(attend_kernel<false>), kAttSmem)) != cudaSuccess) return e;

  // the first kernel follows whatever wrote the inputs, so it is launched plainly
  plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  for (a.half = 1; a.half >= 0 && e == cudaSuccess; --a.half) {
    if (c.w_uk_scale) {
      const long long nk = (long long)H * L * N / 8, nv = (long long)H * L * V / 8;
      const int most = 8 * sms;
      e = start(widen_weights_kernel, (unsigned)std::min<long long>((nk + 255) / 256, most), 256, 0, s, a,
                static_cast<const uint8_t*>(c.w_uk), c.w_uk_scale, reinterpret_cast<uint16_t*>(ws + lay.w_uk), L, N, nk);
      if (e == cudaSuccess)
        e = start(widen_weights_kernel, (unsigned)std::min<long long>((nv + 255) / 256, most), 256, 0, s, a,
                  static_cast<const uint8_t*>(c.w_uv), c.w_uv_scale, reinterpret_cast<uint16_t*>(ws + lay.w_uv), V, L,
                  nv);
    }
    const long long parts = lay.cap_tiles * (kTile / kGatherRows);
    if (e == cudaSuccess) e = start(gather_kernel, (unsigned)parts, kGatherThreads, 0, s, a);
    for (int h0 = 0; h0 < H && e == cudaSuccess; h0 += heads) {
      a.h0 = h0;
      a.hg = std::min(heads, H - h0);
      const long long pairs = lay.cap_tiles * a.hg, blocks = lay.max_items * a.hg * splits;
      e = start(expand_kernel, (unsigned)std::min<long long>(pairs, sms), kExpThreads, kExpSmem, s, em, a);
      if (e == cudaSuccess)
        e = start(a.half ? attend_kernel<true> : attend_kernel<false>, (unsigned)std::min<long long>(blocks, sms), kAttThreads,
                  kAttSmem, s, am, a);
    }
  }
  if (e == cudaSuccess && splits > 1)
    e = start(combine_kernel, (unsigned)(((long long)c.T * H + 7) / 8), 256, 0, s, a);
  return e;
}

}  // namespace mla
