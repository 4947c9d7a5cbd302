// mla_linear_fp8, mla_linear_int8: projections over 8-bit codes,
//
//   out[t, n] = bf16( (sum_k x[t, k] * w[n, k]) * x_scale[t] * w_scale[n] )
//
// on tcgen05, fp32 accumulators in tensor memory.  e4m3 codes are the operands of kind::f8f6f4 as
// they lie in memory.  The GB300 has no fast integer tensor path (its int8 rate is a tenth of its
// f16 rate), so int8 codes are widened to f16 on the SM: every int8 value is an f16 value, every
// product of two is exact in the fp32 accumulator.  Four kernels, chosen by estimated time:
//
// Few tokens (split kernel).  The weights are the A operand (128 output channels a tile), the
// tokens the B operand (16 to 128), so that one token costs no more than a tile's weights, and the
// call is bound by reading those once.  int8: the weights are widened into tensor memory, the tokens into
// shared memory (both there cost a sixth more).  Where the tiles are fewer than the SMs, a cluster of CTAs
// splits K: each leaves its fp32 partial in its shared memory and sums a share of the tokens over the
// cluster, in rank order (the result does not depend on timing).  Times of a call among others, inputs out
// of L2: 64 x 24,576 x 1,536 e4m3 10.8 us (6.0 at the copy rate; launch, first bytes and end of a
// block take 5), int8 16.6 (a stage waits for its widening: 400 ns of two blocks side by side, e4m3 200), 16 x
// 2,112 x 8,192 e4m3 8.4 us.
//
// Up to 32 tokens of int8 (mma kernel).  Widening costs the split kernel more than the weights' way from memory
// does, and tensor memory, clusters and copies take time to begin and end, so here warps take the codes from memory
// into registers and multiply there, with the warp-wide instruction: nothing is handed on but the sums at the end.
// Up to eight tokens the codes themselves, summed in integers (exact); more than that would wait for that
// slow path (32 x 8,192 x 16,384 75 us, widened 52), so they are widened in registers.  8 and 16 x 2,112 x 8,192
// 7.2 and 8.0 us (split kernel 12.6, 12.7), 8 and 16 x 24,576 x 1,536 10.3 and 12.3 (15.9, 16.2).
//
// One token, and two of int8 (dot kernel).  Dot products straight from registers, of int8 on the integer units
// (four products a lane and instruction, exact), of e4m3 in fp32; K is split over a block's warps where rows
// are few.  1 x 2,112 x 8,192 int8 4.5, e4m3 6.0 us (2.5 at the copy rate), 1 x 8,192 x 16,384
// 23 and 25.5 us (20).
//
// Many tokens (pair kernel).  A pair of CTAs a pair of SMs, cta_group::2: 256 tokens (A) by 256, 192 or 128
// channels (B), each CTA loading half of either operand, one tile after another.  Tiles go group by
// group of token tiles, so that those in flight share operands in L2.  The accumulator is double: while
// a tile's products run, other warps scale the last one, lay it out in shared memory and store it by TMA,
// which also cuts off what lies past the last token or channel.  int8: for either half of a stage four
// warps widen the tokens' codes into tensor memory, four the weights' into shared memory (both there would
// cost more of its bandwidth than the products leave).  8,192 x 8,192 x 16,384 e4m3: 600 us, 670 under the
// power cap, 95 % of twice the measured bf16 rate of either; the tensor pipe is active 98 % of the time.
// 4,096 x 24,576 x 1,536: e4m3 95 us (80), int8 188 us (161).
#include <algorithm>
#include <type_traits>

#include "mla_kernels.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace wg {
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();
}  // namespace wg

namespace lin {

using namespace sm100;

constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kStepK = 128;            // codes of a stage along K
constexpr int kRowsW = 128;            // output channels of a tile
constexpr int kMaxTokens = 128;        // tokens of a split tile (MMA N)
constexpr int kMaxStages = 12;
constexpr int kHalfSm = 108 * 1024;    // shared memory for the stages of a block that shares an SM
constexpr int kConvWarps = 8;          // split kernel, int8: warps that widen codes, four for either half of a stage
constexpr int kPlaces = 4;             // ... of widened operands (even: the warps of either half wait for places of their own)
constexpr int kColW = kMaxTokens;      // ... the weights' in tensor memory, 32 columns each, behind the accumulator

struct Maps {
  CUtensorMap w, x, out;
};

struct Args {
  int T, N, K;
  int TN;                 // tokens of a tile
  int S;                  // stages of the ring the copies fill
  int C;                  // CTAs that split K
  long long out_stride;
  const float* x_scale;
  const float* w_scale;
  __nv_bfloat16* out;
  PlanHeader* hdr;
};

// The issuing warps spin on a phase (a suspended waiter wakes later, between products); all others are
// suspended by the hardware for a while, or two dozen spinning warps would take the issue slots of those
// that work.  The clock is looked at now and then.
template <bool kSpin, bool kCluster>
__device__ __forceinline__ bool wait_any(uint64_t* bar, uint32_t parity, PlanHeader* hdr) {
  auto there = [&]() {
    if (kCluster) return kSpin ? mbar_test_wait_cluster(bar, parity) : mbar_try_wait_cluster(bar, parity);
    return kSpin ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
  };
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !there(); ++i) {
    if ((i & (kSpin ? 255u : 15u)) != 0) continue;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      atomicOr(&hdr->status, kDeviceTimeout);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, PlanHeader* hdr) {
  return wait_any<false, false>(bar, parity, hdr);
}
__device__ __forceinline__ bool spin_bar(uint64_t* bar, uint32_t parity, PlanHeader* hdr) {
  return wait_any<true, false>(bar, parity, hdr);
}
// The same for barriers on which the other CTA of a pair arrives: what it did before is there (acquire at cluster scope).
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, PlanHeader* hdr) {
  return wait_any<false, true>(bar, parity, hdr);
}
__device__ __forceinline__ bool spin_pair(uint64_t* bar, uint32_t parity, PlanHeader* hdr) {
  return wait_any<true, true>(bar, parity, hdr);
}

// Place in a ring of `n` stages, and the parity of the round.
struct Ring {
  int s = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++s == n) {
      s = 0;
      round ^= 1;
    }
  }
};

// Sixteen int8 codes as sixteen f16 values: a code with its sign bit flipped, in the low bits of
// 1024, is 1024 + 128 + code.
__device__ __forceinline__ void widen(uint4 raw, uint4& lo, uint4& hi) {
  const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
  const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = in[i] ^ 0x80808080u;
    const uint32_t p = __byte_perm(b, 0x64646464u, 0x4140), q = __byte_perm(b, 0x64646464u, 0x4342);
    const __half2 u = __hsub2(*reinterpret_cast<const __half2*>(&p), off);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&q), off);
    o[2 * i] = *reinterpret_cast<const uint32_t*>(&u);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&v);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Piece q (of four) of half `h` of row r: 16 of the row's 128 codes, which lie in the 128-byte swizzle.
__device__ __forceinline__ uint4 codes_at(const uint8_t* raw, int r, int h, int q) {
  return *reinterpret_cast<const uint4*>(raw + r * 128 + (((4 * h + q) ^ (r & 7)) << 4));
}
// ... widened into a row of 64 f16 values, in the same swizzle.  Neighbouring lanes take neighbouring
// rows, so that the reads and the writes of eight meet each bank once.
__device__ __forceinline__ void store_widened(uint4 codes, uint8_t* dst, int r, int q) {
  uint4 lo, hi;
  widen(codes, lo, hi);
  *reinterpret_cast<uint4*>(dst + r * 128 + (((2 * q) ^ (r & 7)) << 4)) = lo;
  *reinterpret_cast<uint4*>(dst + r * 128 + (((2 * q + 1) ^ (r & 7)) << 4)) = hi;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

template <bool kInt8>
constexpr int kSplitThreads = kInt8 ? 128 + 32 * kConvWarps : 256;

// Threads: warp 0 copies, warp 1 issues the products and owns the tensor memory, warps 4 on widen
// (int8); all of them take part in the epilogue.
template <bool kInt8>
__global__ void __launch_bounds__(kSplitThreads<kInt8>, 2)
    split_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int TN = a.TN, S = a.S;
  const int stage = (kRowsW + TN) * 128, stage2 = TN * 128;   // rows of 128 codes; of 64 widened ones
  uint8_t* ring2 = sm;                                          // int8: widened tokens, then the codes
  uint8_t* ring = kInt8 ? sm + kPlaces * stage2 : sm;
  const int ring_bytes = max(S * stage + (kInt8 ? kPlaces * stage2 : 0), TN * kRowsW * 4);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + ring_bytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* full2 = empty + kMaxStages;
  uint64_t* empty2 = full2 + kMaxStages;
  uint64_t* done = empty2 + kMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = (int)blockDim.x >> 5;
  const uint32_t rank = a.C > 1 ? cluster_ctarank() : 0;
  const int n0 = ((int)blockIdx.x / a.C) * kRowsW, t0 = (int)blockIdx.y * TN;
  const int nkb = (a.K + kStepK - 1) / kStepK;
  const int kb0 = (int)((long long)nkb * rank / a.C), kn = (int)((long long)nkb * (rank + 1) / a.C) - kb0;
  const uint32_t tcols = kInt8 ? kColW + 32 * kPlaces : TN <= 32 ? 32 : TN <= 64 ? 64 : 128;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kInt8 ? kConvWarps : 1);
    }
    if (kInt8)
      for (int s = 0; s < kPlaces; ++s) {
        mbar_init(&full2[s], kConvWarps / 2);
        mbar_init(&empty2[s], 1);
      }
    mbar_init(done, 1);
    fence_mbar_init();
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // A whole warp walks each loop and elects the lane that issues (in a loop of one lane the operands of
  // copies and products, which are warp-uniform, cost hundreds of cycles a stage).
  if (warp == 0) {
    Ring at;
    int i = 0;
    for (; i < kn; ++i, at.next(S)) {
      if (i >= S && !wait_bar(&empty[at.s], at.round ^ 1, a.hdr)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[at.s], stage);
        tma_load_2d(ring + at.s * stage, &maps.w, &full[at.s], (kb0 + i) * kStepK, n0);
        tma_load_2d(ring + at.s * stage + kRowsW * 128, &maps.x, &full[at.s], (kb0 + i) * kStepK, t0);
      }
      __syncwarp();
    }
    // no copy outlives the block, whatever became of those who read them
    for (int j = max(0, i - S); j < i; ++j) wait_bar(&full[j % S], (j / S) & 1, a.hdr);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f32(128, TN, 0);   // f16 and e4m3 are both type 0 of their kinds
    const int steps = kInt8 ? 2 * kn : kn;          // int8: half a stage of codes at a time
    const int stages = kInt8 ? kPlaces : S;
    uint64_t* landed = kInt8 ? full2 : full;
    uint64_t* read = kInt8 ? empty2 : empty;
    const uint64_t d0 = smem_desc(smem_u32(kInt8 ? ring2 : ring), 16, 1024, kLayoutSw128);
    Ring at;
    for (int i = 0; i < steps; ++i, at.next(stages)) {
      if (!spin_bar(&landed[at.s], at.round, a.hdr)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t wd = d0 + (uint64_t)(at.s * ((kInt8 ? stage2 : stage) >> 4)), xd = kInt8 ? wd : wd + (kRowsW * 128 >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {   // 32 bytes of K at a time
          if (kInt8) mma_ts(tmem, tmem + kColW + 32 * at.s + 8 * kk, xd + 2 * kk, idesc, (i | kk) != 0);
          else mma_ss_f8(tmem, wd + 2 * kk, xd + 2 * kk, idesc, (i | kk) != 0);
        }
        mma_commit(&read[at.s]);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(done);
    __syncwarp();
  } else if (kInt8 && warp >= 4) {
    // its half of every stage; its row of the weights (= TMEM lane), its piece of every token
    const int h = (warp - 4) >> 2, q = warp & 3, row = 32 * q + lane;
    Ring from, to;
    if (h) to.next(kPlaces);
    for (int i = h; i < 2 * kn; i += 2, from.next(S)) {
      bool ok = wait_bar(&full[from.s], from.round, a.hdr);
      if (ok && i >= kPlaces) ok = wait_bar(&empty2[to.s], to.round ^ 1, a.hdr);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint8_t* raw = ring + from.s * stage;
      uint4 v[4], x[4];
      uint32_t o[32];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = codes_at(raw, row, h, j);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (32 * j + lane < TN) x[j] = codes_at(raw + kRowsW * 128, 32 * j + lane, h, q);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 lo, hi;
        widen(v[j], lo, hi);
        o[8 * j] = lo.x; o[8 * j + 1] = lo.y; o[8 * j + 2] = lo.z; o[8 * j + 3] = lo.w;
        o[8 * j + 4] = hi.x; o[8 * j + 5] = hi.y; o[8 * j + 6] = hi.z; o[8 * j + 7] = hi.w;
      }
      tmem_st32(tmem + kColW + 32 * to.s + ((uint32_t)(32 * q) << 16), o);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (32 * j + lane < TN) store_widened(x[j], ring2 + to.s * stage2, 32 * j + lane, q);
      fence_proxy_async_smem();
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (elect_one()) {
        mbar_arrive(&empty[from.s]);
        mbar_arrive(&full2[to.s]);
      }
      __syncwarp();
      to.next(kPlaces);
      to.next(kPlaces);
    }
  }
  __syncwarp();
  bool ok = wait_bar(done, 0, a.hdr);
  ok = __syncthreads_and(ok);
  tc_fence_after();

  // the partial, [token][channel] fp32, over the idle rings (TMEM lane = channel, column = token)
  float* part = reinterpret_cast<float*>(sm);
  for (int c = 32 * (warp >> 2); c < TN; c += 8 * warps) {   // warps / 4 groups of 32 columns at a time
    const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + c;
    uint32_t r[32];
    if (c + 32 <= TN) tmem_ld32(at, r);
    else tmem_ld16(at, *reinterpret_cast<uint32_t(*)[16]>(r));
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c + j < TN) part[(c + j) * kRowsW + 32 * (warp & 3) + lane] = __uint_as_float(r[j]);
  }
  tc_fence_before();
  if (a.C > 1) cluster_sync();
  else __syncthreads();

  // a share of the tokens, summed over the cluster in rank order
  if (ok && n0 + 4 * lane < a.N) {
    const float4 ws = *reinterpret_cast<const float4*>(a.w_scale + n0 + 4 * lane);
    const int tokens = min(TN, a.T - t0);
    const int lo = tokens * (int)rank / a.C, hi = tokens * ((int)rank + 1) / a.C;
    // eight partials at a time, of 8 / C tokens (C a power of two up to 8), all loads out before the first sum
    const int cmask = a.C - 1, cshift = 31 - __clz(a.C);
    for (int t1 = lo + warp; t1 < hi; t1 += (8 >> cshift) * warps) {
      float4 u[8], v = make_float4(0.f, 0.f, 0.f, 0.f);
      float xs[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = min(t1 + (j >> cshift) * warps, hi - 1);
        const uint32_t at = smem_u32(part + t * kRowsW + 4 * lane);
        u[j] = ld_cluster_f4(a.C > 1 ? mapa_shared(at, j & cmask) : at);
        xs[j] = a.x_scale[t0 + t];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool first = (j & cmask) == 0;
        v.x = (first ? 0.f : v.x) + u[j].x;
        v.y = (first ? 0.f : v.y) + u[j].y;
        v.z = (first ? 0.f : v.z) + u[j].z;
        v.w = (first ? 0.f : v.w) + u[j].w;
        const int t = t1 + (j >> cshift) * warps;
        if ((j & cmask) != cmask || t >= hi) continue;
        const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * xs[j] * ws.x, v.y * xs[j] * ws.y);
        const __nv_bfloat162 q = __floats2bfloat162_rn(v.z * xs[j] * ws.z, v.w * xs[j] * ws.w);
        *reinterpret_cast<uint2*>(a.out + (t0 + t) * a.out_stride + n0 + 4 * lane) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
      }
    }
  }
  __syncwarp();
  if (a.C > 1) cluster_sync();   // partials stay until all have read them
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

// ------------------------------------------------------------------ one token, or two

constexpr int kDotWarps = 8;
constexpr int kDotMaxK = 1 << 16;    // int8: 2^16 products of up to 2^14 each stay within 32 bits

// Sixteen products of codes added to s: int8 exactly, four an instruction; e4m3 in fp32, each product exact.
__device__ __forceinline__ void dot16(uint4 w, uint4 x, int& s) {
  s = __dp4a((int)w.x, (int)x.x, s);
  s = __dp4a((int)w.y, (int)x.y, s);
  s = __dp4a((int)w.z, (int)x.z, s);
  s = __dp4a((int)w.w, (int)x.w, s);
}
struct E4m3x16 {
  float2 v[8];
};
__device__ __forceinline__ E4m3x16 e4m3x16(uint4 c) {
  const uint32_t u[4] = {c.x, c.y, c.z, c.w};
  E4m3x16 r;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    r.v[i] = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i / 2] >> (16 * (i & 1))), __NV_E4M3)));
  return r;
}
// The sums of the codes' even and odd places, side by side.
__device__ __forceinline__ void dot16(const E4m3x16& w, const E4m3x16& x, float2& s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s.x = fmaf(w.v[i].x, x.v[i].x, s.x);
    s.y = fmaf(w.v[i].y, x.v[i].y, s.y);
  }
}
__device__ __forceinline__ int warp_sum(int s) { return __reduce_add_sync(0xffffffffu, s); }
__device__ __forceinline__ float warp_sum(float2 v) {
  float s = v.x + v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// TT: tokens, R: rows of weights (channels) of a warp.  `along` of a block's warps (a power of two) share the
// rows and split K.
template <bool kInt8, int TT, int R>
__global__ void __launch_bounds__(32 * kDotWarps) dot_kernel(const uint8_t* __restrict__ x, const uint8_t* __restrict__ w,
                                                             const Args a, int along) {
  using Sum = std::conditional_t<kInt8, int, float>;
  using Acc = std::conditional_t<kInt8, int, float2>;
  constexpr int kAhead = R * TT >= 16 ? 1 : 8 / (R + TT) > 1 ? 8 / (R + TT) : 2;   // steps whose loads are out together
  __shared__ Sum part[kDotWarps][R * TT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = ((int)blockIdx.x * (kDotWarps / along) + warp / along) * R;
  const int pieces = a.K / 16, step = 32 * along;
  const uint4* xp[TT];
  const uint4* wp[R];
#pragma unroll
  for (int t = 0; t < TT; ++t) xp[t] = reinterpret_cast<const uint4*>(x + (size_t)min(t, a.T - 1) * a.K);
#pragma unroll
  for (int r = 0; r < R; ++r) wp[r] = reinterpret_cast<const uint4*>(w + (size_t)min(n0 + r, a.N - 1) * a.K);
  Acc acc[R * TT] = {};
#pragma unroll 1
  for (int c = (warp & (along - 1)) * 32 + lane; c < pieces; c += kAhead * step) {
    uint4 wv[kAhead][R], xv[kAhead][TT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool in = c + u * step < pieces;
#pragma unroll
      for (int r = 0; r < R; ++r) wv[u][r] = in ? __ldcs(wp[r] + c + u * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[u][t] = in ? __ldg(xp[t] + c + u * step) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if constexpr (kInt8) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < TT; ++t) dot16(wv[u][r], xv[u][t], acc[r * TT + t]);
      } else {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const E4m3x16 xf = e4m3x16(xv[u][t]);
#pragma unroll
          for (int r = 0; r < R; ++r) dot16(e4m3x16(wv[u][r]), xf, acc[r * TT + t]);
        }
      }
    }
  }
  Sum mine = 0;
#pragma unroll
  for (int i = 0; i < R * TT; ++i) {
    const Sum s = warp_sum(acc[i]);
    if (lane == i) mine = s;
  }
  if (along > 1) {
    if (lane < R * TT) part[warp][lane] = mine;
    __syncthreads();
    if (warp & (along - 1)) return;
    if (lane < R * TT)
      for (int i = 1; i < along; ++i) mine += part[warp + i][lane];
  }
  const int n = n0 + lane / TT, t = lane % TT;
  if (lane < R * TT && n < a.N && t < a.T)
    a.out[t * a.out_stride + n] = __float2bfloat16_rn((float)mine * a.x_scale[t] * a.w_scale[n]);
}

// ------------------------------------------------------------------ a few tokens of int8

constexpr int kMmaWarps = 16;   // at most, of a block

__device__ __forceinline__ void mma_warp(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_warp(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A lane's 16 codes of a row as operand registers: the codes, or their f16 values.
template <bool kExact>
struct Operand {
  uint32_t v[kExact ? 4 : 8];
  __device__ __forceinline__ explicit Operand(uint4 c) {
    uint4 lo = c, hi;
    if constexpr (!kExact) {
      widen(c, lo, hi);
      v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    }
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
  }
};

// NT * 8 tokens a block, 16 channels a warp, U steps of 64 codes along K whose loads are out together.  `along` of
// a block's warps (a power of two) share the channels and split K.  The lanes of a row take 16 neighbouring
// codes each: which of them an instruction takes for its place along K is free, as long as it is the same ones
// of the weights and of the tokens.
template <bool kExact, int NT, int U>
__global__ void __launch_bounds__(32 * kMmaWarps) mma_kernel(const uint8_t* __restrict__ x, const uint8_t* __restrict__ w,
                                                             const Args a, int along) {
  using Sum = std::conditional_t<kExact, int, float>;
  constexpr int kPitch = 20;   // 16 channels; the lanes' stores meet each bank once
  extern __shared__ uint8_t smem_raw[];
  Sum* part = reinterpret_cast<Sum*>(smem_raw);   // [warp][token][kPitch]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int per = ((int)blockDim.x >> 5) / along;
  const int n0 = ((int)blockIdx.x * per + warp / along) * 16;
  const uint8_t* wp[2];
  const uint8_t* xp[NT];
#pragma unroll
  for (int r = 0; r < 2; ++r) wp[r] = w + (size_t)min(n0 + 8 * r + g, a.N - 1) * a.K + 16 * c;
#pragma unroll
  for (int t = 0; t < NT; ++t) xp[t] = x + (size_t)min(8 * t + g, a.T - 1) * a.K + 16 * c;
  Sum acc[NT][4] = {};
#pragma unroll 1
  for (int k = (warp & (along - 1)) * 64 * U; k < a.K; k += 64 * U * along) {
    uint4 wv[U][2], xv[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = k + 64 * u + 16 * c < a.K;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        wv[u][r] = in ? __ldcs(reinterpret_cast<const uint4*>(wp[r] + k + 64 * u)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xv[u][t] = in ? __ldg(reinterpret_cast<const uint4*>(xp[t] + k + 64 * u)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Operand<kExact> w0(wv[u][0]), w1(wv[u][1]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Operand<kExact> xo(xv[u][t]);
#pragma unroll
        for (int j = 0; j < (kExact ? 4 : 8); j += 2)
          mma_warp(acc[t], w0.v[j], w1.v[j], w0.v[j + 1], w1.v[j + 1], xo.v[j], xo.v[j + 1]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      part[(warp * NT * 8 + 8 * t + 2 * c + (i & 1)) * kPitch + 8 * (i >> 1) + g] = acc[t][i];
  __syncthreads();
  // eight channels of a token a thread, the warps' sums in their order
  for (int i = threadIdx.x; i < per * NT * 16; i += blockDim.x) {
    const int half = i & 1, group = (i >> 1) % per, t = (i >> 1) / per;
    const int n = ((int)blockIdx.x * per + group) * 16 + 8 * half;
    if (t >= a.T || n >= a.N) continue;
    Sum s[8] = {};
    for (int j = 0; j < along; ++j) {
      const Sum* p = part + ((group * along + j) * NT * 8 + t) * kPitch + 8 * half;
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += p[q];
    }
    const float xs = a.x_scale[t];
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 ws = *reinterpret_cast<const float2*>(a.w_scale + n + 2 * q);
      const __nv_bfloat162 v = __floats2bfloat162_rn((float)s[2 * q] * xs * ws.x, (float)s[2 * q + 1] * xs * ws.y);
      o[q] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(a.out + t * a.out_stride + n) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------------ many tokens

// kW: channels of a tile.  int8 tiles of 256 leave no room for a second accumulator beside the widened tokens.
template <bool kInt8, int kW>
struct Pair {
  static constexpr int kN = kW;
  static constexpr int kRows = 128 + kN / 2;                // rows of a stage in a CTA: its tokens, its channels
  static constexpr int kStage = kRows * 128;
  static constexpr int kStages = kInt8 ? (kN == 256 ? 3 : 4) : (kN == 128 ? 8 : 6);
  static constexpr int kStages2 = 4;                        // int8, widened: tokens 32 TMEM columns, channels a box
  static constexpr int kStage2 = kN / 2 * 128;
  static constexpr int kAccs = kInt8 && kN == 256 ? 1 : 2;  // accumulators
  static constexpr int kColA = 384;                         // int8: TMEM columns of the widened tokens
  static constexpr int kGroups = kInt8 ? 1 : 2;             // of four warps that read and store a tile
  static constexpr int kBoxes = kInt8 ? 2 : 1;              // boxes of a group
  static constexpr int kBoxOut = 128 * 128;                 // 128 tokens x 64 channels bf16
  static constexpr int kRing2 = kStages * kStage;
  static constexpr int kOut = kRing2 + (kInt8 ? kStages2 * kStage2 : 0);
  static constexpr int kScales = kOut + 2 * kBoxOut;        // [kN] channel scales
  static constexpr int kBars = kScales + kN * 4;
  static constexpr int kSmem = 1024 + kBars + 8 * (2 * kStages + 2 * kStages2 + 4) + 16;
  static_assert(kSmem <= 232448 && (!kInt8 || kAccs * kN <= kColA));
  static constexpr int kThreads = kInt8 ? 768 : 384;
};

// Tile i of a call: tokens from m0, channels from n0.  Groups of 8 token tiles, channel tiles in turn
// within a group, the group's token tiles one after the other.
struct Tile {
  int m0, n0;
};
__device__ __forceinline__ Tile tile_of(int i, int mtiles, int ntiles, int kn) {
  const int group = i / (8 * ntiles), in = i - group * 8 * ntiles;
  const int gm = min(8, mtiles - 8 * group);
  return Tile{(8 * group + in % gm) * 256, in / gm * kn};
}

// Warp 0 copies, warp 1 of the pair's first CTA issues the products, warp 2 owns the tensor memory, warps 4-7 (e4m3:
// 4-11) are the epilogue; int8: warps 8-11 widen the first half of a stage's tokens (thread = row = TMEM lane), 12-15
// of its channels, 16-23 the second half's, and warp 1 of the second CTA says that they are there.
template <bool kInt8, int kW>
__global__ void __launch_bounds__(Pair<kInt8, kW>::kThreads, 1) __cluster_dims__(2, 1, 1)
    pair_kernel(const __grid_constant__ Maps maps, const Args a) {
  using P = Pair<kInt8, kW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + P::kBars);   // e4m3: the first CTA's, for both; int8: each its own
  uint64_t* empty = full + P::kStages;
  uint64_t* full2 = empty + P::kStages;      // int8: widened in this CTA; the first's: in both
  uint64_t* empty2 = full2 + P::kStages2;
  uint64_t* acc_full = empty2 + P::kStages2;           // a tile's products are done
  uint64_t* acc_empty = acc_full + 2;        // ... and read, in the first CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int mtiles = (a.T + 255) / 256, ntiles = (a.N + P::kN - 1) / P::kN;
  const int tiles = mtiles * ntiles, pairs = (int)gridDim.x / 2, first = (int)blockIdx.x / 2;
  const int nkb = (a.K + kStepK - 1) / kStepK;

  if (tid == 0) {
    for (int s = 0; s < P::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kInt8 ? 16 : 1);
    }
    for (int s = 0; s < P::kStages2; ++s) {
      mbar_init(&full2[s], rank == 0 ? 9 : 8);   // its CTA's warps, and in the first what the second hands over
      mbar_init(&empty2[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 8 * P::kGroups);
    }
    fence_mbar_init();
    prefetch_tensormap(&maps.x);
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.out);
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    bool ok = true;
    Ring pos;
    int i = 0;
    for (int tile = first; tile < tiles && ok; tile += pairs) {
      const Tile at = tile_of(tile, mtiles, ntiles, P::kN);
      for (int kb = 0; kb < nkb; ++kb, ++i, pos.next(P::kStages)) {
        if (i >= P::kStages && !(ok = wait_bar(&empty[pos.s], pos.round ^ 1, a.hdr))) break;
        if (elect_one()) {
          uint8_t* dst = sm + pos.s * P::kStage;
          if (kInt8) {
            mbar_arrive_expect_tx(&full[pos.s], P::kStage);
            tma_load_2d(dst, &maps.x, &full[pos.s], kb * kStepK, at.m0 + 128 * rank);
            tma_load_2d(dst + 128 * 128, &maps.w, &full[pos.s], kb * kStepK, at.n0 + P::kN / 2 * rank);
          } else {
            const uint32_t bar = mapa_shared(smem_u32(&full[pos.s]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[pos.s], 2 * P::kStage);
            tma_load_2d_pair(dst, &maps.x, bar, kb * kStepK, at.m0 + 128 * rank);
            tma_load_2d_pair(dst + 128 * 128, &maps.w, bar, kb * kStepK, at.n0 + P::kN / 2 * rank);
          }
        }
        __syncwarp();
      }
    }
    // no copy and no arrival outlives the pair, whatever became of those who wait for them
    for (int j = max(0, i - P::kStages); j < i; ++j) {
      if (kInt8 || rank == 0) wait_bar(&full[j % P::kStages], (j / P::kStages) & 1, a.hdr);
      wait_bar(&empty[j % P::kStages], (j / P::kStages) & 1, a.hdr);
    }
  } else if (warp == 1 && rank == 0) {
    const uint32_t idesc = idesc_f32(256, P::kN, 0);   // f16 and e4m3 are both type 0 of their kinds
    const uint64_t d0 = smem_desc(smem_u32(sm + (kInt8 ? P::kRing2 : 0)), 16, 1024, kLayoutSw128);
    bool ok = true;
    Ring pos, acc;
    int n = 0;
    for (int tile = first; tile < tiles && ok; tile += pairs, ++n, acc.next(P::kAccs)) {
      const uint32_t d = tmem + acc.s * P::kN;
      if (n >= P::kAccs && !(ok = wait_pair(&acc_empty[acc.s], acc.round ^ 1, a.hdr))) break;
      tc_fence_after();
      for (int kb = 0; kb < (kInt8 ? 2 * nkb : nkb); ++kb, pos.next(kInt8 ? P::kStages2 : P::kStages)) {
        if (!(ok = spin_pair(kInt8 ? &full2[pos.s] : &full[pos.s], pos.round, a.hdr))) break;
        tc_fence_after();
        if (elect_one()) {
          if (kInt8) {
            const uint64_t wd = d0 + (uint64_t)(pos.s * (P::kStage2 >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts_pair(d, tmem + P::kColA + 32 * pos.s + 8 * kk, wd + 2 * kk, idesc, (kb | kk) != 0);
            mma_commit_pair(&empty2[pos.s]);
          } else {
            const uint64_t xd = d0 + (uint64_t)(pos.s * (P::kStage >> 4)), wd = xd + (128 * 128 >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss_f8_pair(d, xd + 2 * kk, wd + 2 * kk, idesc, (kb | kk) != 0);
            mma_commit_pair(&empty[pos.s]);
          }
        }
        __syncwarp();
      }
      if (elect_one()) mma_commit_pair(&acc_full[acc.s]);
      __syncwarp();
    }
  } else if (kInt8 && warp == 1) {
    // What the second CTA's warps widened: they arrive here, and this warp hands it on to the first CTA.  The release to the
    // cluster takes a warp that widens a twelfth of its time (4,096 x 24,576 x 1,536 196 us against 185); here
    // nothing waits for it.
    Ring pos;
    bool ok = true;
    for (int tile = first; tile < tiles && ok; tile += pairs)
      for (int kb = 0; kb < 2 * nkb; ++kb, pos.next(P::kStages2)) {
        if (!(ok = wait_bar(&full2[pos.s], pos.round, a.hdr))) break;
        tc_fence_after();
        tc_fence_before();
        if (elect_one()) mbar_arrive_remote(mapa_shared(smem_u32(&full2[pos.s]), 0));
        __syncwarp();
      }
  } else if (warp >= 4 && warp < 4 + 4 * P::kGroups) {
    // Groups of four warps share the accumulator's chunks of 64 channels.
    const int row = tid & 127, g4 = (warp - 4) >> 2;   // token of the CTA's half = TMEM lane; group
    uint8_t* box = sm + P::kOut + g4 * P::kBoxes * P::kBoxOut;
    float* ws = reinterpret_cast<float*>(sm + P::kScales);   // a group's own channels, read between its barriers
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + g4) : "memory"); };
    auto group_and = [&](bool ok) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "r"((uint32_t)ok), "r"(1 + g4)
          : "memory");
      return r != 0;
    };
    int chunk = 0;
    Ring acc;
    for (int tile = first; tile < tiles; tile += pairs, acc.next(P::kAccs)) {
      const Tile at = tile_of(tile, mtiles, ntiles, P::kN);
      const int m0 = at.m0 + 128 * rank;
      for (int c = 64 * g4 + (row & 63) + 64 * P::kGroups * (row >> 6); c < P::kN; c += 128 * P::kGroups)
        ws[c] = at.n0 + c < a.N ? a.w_scale[at.n0 + c] : 0.f;
      const float xs = m0 + row < a.T ? a.x_scale[m0 + row] : 0.f;
      // the group goes on or gives up together: its barriers count all of its warps
      if (!group_and(wait_bar(&acc_full[acc.s], acc.round, a.hdr))) break;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 64 * g4; c0 < P::kN; c0 += 64 * P::kGroups, ++chunk) {
        uint8_t* dst = box + (chunk & (P::kBoxes - 1)) * P::kBoxOut;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32];
          tmem_ld32(tmem + acc.s * P::kN + c0 + 32 * half + lanes, r);
          if (half == 0) {
            if (row == 0) bulk_wait_read<P::kBoxes - 1>();   // what the box held has left
            group_sync();                                      // ... and the scales are there
          }
          tmem_ld_wait();
          if (half == 1 && c0 + 64 * P::kGroups >= P::kN) {   // this warp has read its part of the accumulator
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive_remote(mapa_shared(smem_u32(&acc_empty[acc.s]), 0));
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const int c = 8 * g + 2 * j;
              const float4 w4 = *reinterpret_cast<const float4*>(ws + c0 + 32 * half + c);
              const __nv_bfloat162 p =
                  __floats2bfloat162_rn(__uint_as_float(r[c]) * xs * w4.x, __uint_as_float(r[c + 1]) * xs * w4.y);
              const __nv_bfloat162 q =
                  __floats2bfloat162_rn(__uint_as_float(r[c + 2]) * xs * w4.z, __uint_as_float(r[c + 3]) * xs * w4.w);
              o[j] = *reinterpret_cast<const uint32_t*>(&p);
              o[j + 1] = *reinterpret_cast<const uint32_t*>(&q);
            }
            *reinterpret_cast<uint4*>(dst + row * 128 + (((4 * half + g) ^ (row & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        fence_proxy_async_smem();
        group_sync();
        if (row == 0) {
          if (m0 < a.T && at.n0 + c0 < a.N) tma_store_2d(&maps.out, dst, at.n0 + c0, m0);
          bulk_commit();
        }
      }
    }
    if (row == 0) bulk_wait_all();
  } else if (kInt8 && warp >= 8) {
    const bool tokens = (warp & 4) == 0;
    const int row = tid & 127, h = (warp - 8) >> 3;   // its half of every stage
    int i = h;
    bool ok = true;
    Ring from, to;
    if (h) to.next(P::kStages2);
    for (int tile = first; tile < tiles && ok; tile += pairs)
      for (int kb = 0; kb < nkb; ++kb, i += 2) {
        ok = wait_bar(&full[from.s], from.round, a.hdr);
        if (ok && i >= P::kStages2) ok = wait_bar(&empty2[to.s], to.round ^ 1, a.hdr);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const uint8_t* raw = sm + from.s * P::kStage;
        if (tokens) {
          tc_fence_after();
          uint4 v[4];
          uint32_t o[32];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = codes_at(raw, row, h, q);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 lo, hi;
            widen(v[q], lo, hi);
            o[8 * q] = lo.x; o[8 * q + 1] = lo.y; o[8 * q + 2] = lo.z; o[8 * q + 3] = lo.w;
            o[8 * q + 4] = hi.x; o[8 * q + 5] = hi.y; o[8 * q + 6] = hi.z; o[8 * q + 7] = hi.w;
          }
          tmem_st32(tmem + P::kColA + 32 * to.s + ((uint32_t)(32 * (warp & 3)) << 16), o);
          tmem_st_wait();
          tc_fence_before();
        } else {
          // each of four warps takes a piece of the CTA's channels
          uint4 v[P::kN / 64];
#pragma unroll
          for (int j = 0; j < P::kN / 64; ++j) v[j] = codes_at(raw + 128 * 128, 32 * j + lane, h, warp & 3);
#pragma unroll
          for (int j = 0; j < P::kN / 64; ++j)
            store_widened(v[j], sm + P::kRing2 + to.s * P::kStage2, 32 * j + lane, warp & 3);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (elect_one()) {
          mbar_arrive(&empty[from.s]);
          mbar_arrive(&full2[to.s]);
        }
        __syncwarp();
        from.next(P::kStages);
        to.next(P::kStages2);
        to.next(P::kStages2);
      }
    // the pair's last arrivals on this CTA's barriers
    if (warp == 16)   // half 1: i is one past the last
      for (int j = max(0, i - 1 - P::kStages2); j < i - 1; ++j) wait_bar(&empty2[j % P::kStages2], (j / P::kStages2) & 1, a.hdr);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves while the other's products use its memory
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Rows of K codes as a tensor map, boxes of `rows` rows of 128 codes.  (Boxes of 64 codes took three
// times as long a byte.)
bool encode_codes(CUtensorMap* m, const void* p, int K, int rows_total, int rows) {
  const wg::EncodeTiledFn fn = wg::encode_fn();
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows_total};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {kStepK, (cuuint32_t)rows};
  cuuint32_t es[2] = {1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output, boxes of 128 tokens by 64 channels.
bool encode_out(CUtensorMap* m, void* p, int T, int N, long long stride) {
  const wg::EncodeTiledFn fn = wg::encode_fn();
  cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)T};
  cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  cuuint32_t box[2] = {64, 128};
  cuuint32_t es[2] = {1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the split kernel cuts a call, and what that takes, in ns: 3.5 us, and for each block of an SM 1.7 and its
// stages (e4m3 200 ns and half a one a token of the tile, int8 540 and 1.5; of two int8 blocks side by side 1.3 us,
// 400 ns and one a token).
template <bool kInt8>
long long split_ns(Args* a, int sms) {
  const int ttiles = (a->T + kMaxTokens - 1) / kMaxTokens;   // as even as they come, in 16s
  a->TN = ((a->T + ttiles - 1) / ttiles + 15) / 16 * 16;
  const long long tiles = (long long)((a->N + kRowsW - 1) / kRowsW) * ((a->T + a->TN - 1) / a->TN);
  const int nkb = (a->K + kStepK - 1) / kStepK;
  const int stage = (kRowsW + a->TN) * 128, places = kInt8 ? kPlaces * a->TN * 128 : 0;
  const bool pairable = places + 2 * stage <= kHalfSm;   // two blocks fit an SM
  // K is split while there are SMs for the blocks and two stages left for each (16 x 576 x 2,048, eight blocks and
  // two: int8 5.7 us and 6.9, e4m3 4.8 and 5.4).  int8 blocks wait for their own widening, so two an SM are taken
  // where either keeps 16 stages: 16 x 8,192 x 16,384 32.8 us against 40.5, but 64 x 7,168 x 2,048 (4 stages) 12.6
  // against 11.5.  Of clusters whose blocks fill an SM each the device holds 16 of eight and some 36 of four.
  const auto fits = [&](int C) {
    if (tiles * C > sms) return kInt8 && pairable && tiles * C <= 2 * sms && nkb >= 16 * C;
    return nkb >= 2 * C && (pairable || C < 4 || tiles * C <= 128);
  };
  a->C = 1;
  while (a->C < 8 && fits(2 * a->C)) a->C *= 2;
  const long long blocks = tiles * a->C, stages = (nkb + a->C - 1) / a->C;
  // blocks an SM (clusters of eight do not fill all SMs: 136 blocks of 17 share some)
  const long long rounds = a->C == 8 && blocks > 128 ? 2 : (blocks + sms - 1) / sms;
  const bool two = pairable && (rounds > 1 || a->C > 2);
  a->S = std::min({kMaxStages, ((two ? kHalfSm : 200 * 1024) - places) / stage, nkb});
  if (!kInt8) return 3500 + rounds * (1700 + stages * (200 + a->TN / 2));
  return 3500 + rounds * (two && rounds > 1 ? 1300 + stages * (400 + a->TN) : 1700 + stages * (540 + a->TN * 3 / 2));
}

template <bool kInt8>
cudaError_t launch_split(const Args& a, const void* x, const void* w, cudaStream_t s) {
  Maps maps;
  const int tiles = (a.N + kRowsW - 1) / kRowsW, ttiles = (a.T + a.TN - 1) / a.TN;
  const int stage = (kRowsW + a.TN) * 128, places = kInt8 ? kPlaces * a.TN * 128 : 0;
  if (!encode_codes(&maps.w, w, a.K, a.N, kRowsW) || !encode_codes(&maps.x, x, a.K, a.T, a.TN))
    return cudaErrorInvalidValue;
  const size_t ring = std::max((size_t)a.S * stage + places, (size_t)a.TN * kRowsW * 4);
  // int8: more than a third of an SM's, whose tensor memory holds the columns of two blocks
  const size_t smem = std::max<size_t>(1024 + ring + (4 * kMaxStages + 2) * 8, kInt8 ? 78 * 1024 : 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * a.C, ttiles);
  cfg.blockDim = dim3(kSplitThreads<kInt8>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.C > 1 ? 1 : 0;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(split_kernel<kInt8>), (int)smem);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, split_kernel<kInt8>, maps, a);
  return e;
}

template <bool kInt8, int TT, int R>
cudaError_t launch_dot(const Args& a, const void* x, const void* w, int sms, cudaStream_t s) {
  const long long groups = (a.N + R - 1) / R;
  int along = 1;   // some 24 warps an SM, each with two steps along K and more
  while (along < kDotWarps && groups * along < 24ll * sms && a.K >= 2048 * along) along *= 2;
  const int per = kDotWarps / along;
  dot_kernel<kInt8, TT, R><<<(unsigned)((groups + per - 1) / per), 32 * kDotWarps, 0, s>>>(
      static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(w), a, along);
  return cudaGetLastError();
}

// What the mma kernel takes, in ns: 3.5 us, and for a million codes of weights 230, for more than 16 tokens 380.
long long mma_ns(const Args& a) { return 3500 + (long long)a.N * a.K / 1000 * (a.T <= 16 ? 230 : 380) / 1000; }

template <bool kExact, int NT>
cudaError_t launch_mma(const Args& a, const void* x, const void* w, int sms, cudaStream_t s) {
  constexpr int kU = NT <= 2 ? 4 : 2;   // 24,576 x 1,536: 8 tokens 10.3 us with 4 and 11.2 with 2, 32 26.9 and 17.8
  const long long groups = (a.N + 15) / 16;
  int along = 1;   // some 16 warps an SM (24: 8 x 24,576 x 1,536 13.3 us), each with work for its loads
  while (along < kMmaWarps && groups * along < 16ll * sms && a.K >= 64 * kU * along) along *= 2;
  const int warps = std::max(8, along), per = warps / along;
  mma_kernel<kExact, NT, kU><<<(unsigned)((groups + per - 1) / per), 32 * warps, warps * NT * 8 * 20 * 4, s>>>(
      static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(w), a, along);
  return cudaGetLastError();
}

template <bool kInt8, int kW>
cudaError_t launch_pair(const Args& a, const void* x, const void* w, int sms, cudaStream_t s) {
  using P = Pair<kInt8, kW>;
  Maps maps;
  if (!encode_codes(&maps.x, x, a.K, a.T, 128) || !encode_codes(&maps.w, w, a.K, a.N, P::kN / 2) ||
      !encode_out(&maps.out, a.out, a.T, a.N, a.out_stride))
    return cudaErrorInvalidValue;
  const long long tiles = (long long)((a.T + 255) / 256) * ((a.N + P::kN - 1) / P::kN);
  const int pairs = (int)std::min<long long>(tiles, sms / 2);
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(pair_kernel<kInt8, kW>), P::kSmem);
  if (e != cudaSuccess) return e;
  pair_kernel<kInt8, kW><<<2 * pairs, P::kThreads, P::kSmem, s>>>(maps, a);
  return cudaGetLastError();
}

// What a call takes by the pair kernel, in ns, and the width of its tiles: rounds of tiles over the pairs of SMs
// by stages of K by a stage's time (measured at 16,384 of K: tiles of 256, 192, 128 channels 340, 260, 200 ns,
// int8 660, 550, 530 - there the widening of the tokens' codes holds up narrow tiles, and the end of
// a tile of 256, without a second accumulator, is not overlapped), and 8 us.
template <bool kInt8>
long long pair_ns(const Args& a, int sms, int* width) {
  long long least = 0;
  for (int w : {256, 192, 128}) {
    const long long tiles = (long long)((a.T + 255) / 256) * ((a.N + w - 1) / w), nkb = (a.K + kStepK - 1) / kStepK;
    const int stage = kInt8 ? (w == 256 ? 660 : w == 192 ? 550 : 530) : (w == 256 ? 340 : w == 192 ? 260 : 200);
    const long long ns = 8000 + (tiles + sms / 2 - 1) / (sms / 2) * (nkb * stage + (kInt8 && w == 256 ? 1800 : 400));
    if (least == 0 || ns < least) {
      *width = w;
      least = ns;
    }
  }
  return least;
}

template <bool kInt8>
cudaError_t launch(const Args& a, const void* x, const void* w, int sms, cudaStream_t s) {
  // dot kernel against split kernel: one token, 2,112 x 8,192 and 24,576 x 1,536, int8 4.7 and 8.2 us against 12 and 15,
  // e4m3 5.8 and 11 against 7.5 and 10.4 (576 x 2,048: 2.9 against 5.1); two of e4m3 7.6 and 15 against 7.9 and 10.5.
  if (a.T == 1 && a.K <= kDotMaxK) return launch_dot<kInt8, 1, 4>(a, x, w, sms, s);
  if constexpr (kInt8) {
    // mma kernel, eight tokens: 7.3 and 10.3 us (dot products 8.5 and 12, split kernel 12.6 and 15.9)
    if (a.T == 2 && a.K <= kDotMaxK) return launch_dot<true, 2, 2>(a, x, w, sms, s);
    if (a.T <= 8 && a.K <= kDotMaxK) return launch_mma<true, 1>(a, x, w, sms, s);
  }
  // The estimates follow what was measured within a fifth where two kernels are close: 128 tokens, 8,192 x 16,384,
  // pair 68 us and split 50 (int8), 33 and 30; 64 of 24,576 x 1,536 19.3 and 16.6; 192 of 8,192 x 16,384 68 and 66,
  // 33 and 34; 32 of 2,112 x 8,192 mma 11 and split 13, of 8,192 x 8,192 28 and 20 (int8).
  int width = 0;
  const long long pair = pair_ns<kInt8>(a, sms, &width);
  Args b = a;
  const long long split = split_ns<kInt8>(&b, sms);
  if constexpr (kInt8)
    if (a.T <= 32 && mma_ns(a) < std::min(split, pair))
      return a.T <= 16 ? launch_mma<false, 2>(a, x, w, sms, s) : launch_mma<false, 4>(a, x, w, sms, s);
  if (split <= pair) return launch_split<kInt8>(b, x, w, s);
  switch (width) {
    case 256: return launch_pair<kInt8, 256>(a, x, w, sms, s);
    case 192: return launch_pair<kInt8, 192>(a, x, w, sms, s);
    default: return launch_pair<kInt8, 128>(a, x, w, sms, s);
  }
}

}  // namespace lin

cudaError_t launch_linear(bool int8, int T, int N, int K, const void* x, const float* x_scale, const void* w,
                          const float* w_scale, void* out, long long out_stride, PlanHeader* hdr, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  lin::Args a{};
  a.T = T;
  a.N = N;
  a.K = K;
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_stride = out_stride;
  a.hdr = hdr;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return int8 ? lin::launch<true>(a, x, w, sms, s) : lin::launch<false>(a, x, w, sms, s);
}

}  // namespace mla
