// mla_linear_fp8, mla_linear_int8: projections over 8-bit codes,
//
//   out[t, n] = bf16( (sum_k x[t, k] * w[n, k]) * x_scale[t] * w_scale[n] )
//
// on tcgen05, fp32 accumulators in tensor memory.  e4m3 codes are the operands of kind::f8f6f4 as
// they lie in memory.  The GB300 has no fast integer tensor path (its int8 rate is a tenth of its
// f16 rate), so int8 codes are widened to f16 in shared memory: every int8 value is an f16 value, every
// product of two is exact in the fp32 accumulator.
//
// Few tokens (split kernel).  The weights are the A operand (128 output channels a tile), the
// tokens the B operand (up to 256), so that one token costs no more than a tile's weights, and the
// call is bound by reading those once.  Where the tiles are fewer than the SMs, a cluster of CTAs
// splits K: each leaves its fp32 partial in its shared memory and sums a share of the tokens over the
// cluster, in rank order (the result does not depend on timing).
//
// Many tokens (pair kernel).  One pair of CTAs a pair of SMs, cta_group::2: 256 tokens (A) by 256
// channels (B; int8 192), each CTA loading half of either operand, one tile after another.  Tiles go
// group by group of token tiles, so that those in flight share operands in L2.  The accumulator is
// double: while a tile's products run, four warps scale the last one, lay it out in shared memory
// and store it by TMA, which also cuts off what lies past the last token or channel.  int8: four
// warps widen the tokens' codes into tensor memory, four the weights' into shared memory (both
// there would cost more of its bandwidth than the products leave).
#include <algorithm>

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
constexpr int kRowsW = 128;            // output channels of a tile
constexpr int kMaxTokens = 256;        // tokens of a tile (MMA N)
constexpr int kMaxStages = 12;
constexpr int kConvWarps = 8;          // int8: warps that widen codes

struct Maps {
  CUtensorMap w, x, out;
};

struct Args {
  int T, N, K;
  int TN;                 // tokens of a tile
  int S, S2;              // stages of the ring the copies fill; int8: of the ring of widened operands
  int C;                  // CTAs that split K
  long long out_stride;
  const float* x_scale;
  const float* w_scale;
  __nv_bfloat16* out;
  PlanHeader* hdr;
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, PlanHeader* hdr) {
  if (mbar_wait(bar, parity, kWaitLimitNs)) return true;
  atomicOr(&hdr->status, kDeviceTimeout);
  return false;
}

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

// A thread's share of widening `rows` rows of 64 codes (64 bytes apart) into rows of 64 f16 values in
// the 128-byte swizzle.  Four neighbours take a row: reads are contiguous, the writes of eight
// neighbours meet each bank once.
__device__ __forceinline__ void widen_rows(const uint8_t* raw, uint8_t* dst, int rows, int i0, int step) {
  for (int i = i0; i < rows * 4; i += step) {
    const int r = i >> 2, q = i & 3;
    uint4 lo, hi;
    widen(*reinterpret_cast<const uint4*>(raw + 16 * i), lo, hi);
    uint8_t* d = dst + r * 128;
    *reinterpret_cast<uint4*>(d + (((2 * q) ^ (r & 7)) << 4)) = lo;
    *reinterpret_cast<uint4*>(d + (((2 * q + 1) ^ (r & 7)) << 4)) = hi;
  }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// Threads: warp 0 copies, warp 1 issues the products and owns the tensor memory, warps 4 on widen
// (int8); all of them take part in the epilogue.
template <bool kInt8>
__global__ void __launch_bounds__(kInt8 ? 128 + 32 * kConvWarps : 128)
    split_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  constexpr int kStepK = kInt8 ? 64 : 128;     // codes of a stage along K
  const int TN = a.TN, S = a.S, S2 = a.S2;
  const int stage = (kRowsW + TN) * kStepK;    // what the copies fill
  const int stage2 = (kRowsW + TN) * 128;      // operands: rows of 128 bytes
  uint8_t* ring2 = kInt8 ? sm : nullptr;       // widened operands, then the codes
  uint8_t* ring = kInt8 ? sm + S2 * stage2 : sm;
  const int ring_bytes = max(S * stage + (kInt8 ? S2 * stage2 : 0), TN * kRowsW * 4);
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
  const uint32_t tcols = TN <= 32 ? 32 : TN <= 64 ? 64 : TN <= 128 ? 128 : 256;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kInt8 ? kConvWarps : 1);
    }
    if (kInt8)
      for (int s = 0; s < S2; ++s) {
        mbar_init(&full2[s], kConvWarps);
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

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int i = 0;
      for (; i < kn; ++i) {
        const int s = i % S;
        if (i >= S && !(ok = wait_bar(&empty[s], ((i / S) & 1) ^ 1, a.hdr))) break;
        mbar_arrive_expect_tx(&full[s], stage);
        tma_load_2d(ring + s * stage, &maps.w, &full[s], (kb0 + i) * kStepK, n0);
        tma_load_2d(ring + s * stage + kRowsW * kStepK, &maps.x, &full[s], (kb0 + i) * kStepK, t0);
      }
      // no copy outlives the block, whatever became of those who read them
      for (int j = max(0, i - S); j < i; ++j) wait_bar(&full[j % S], (j / S) & 1, a.hdr);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f32(128, TN, 0);   // f16 and e4m3 are both type 0 of their kinds
      for (int i = 0; i < kn; ++i) {
        const int s = kInt8 ? i % S2 : i % S;
        if (!wait_bar(kInt8 ? &full2[s] : &full[s], (kInt8 ? i / S2 : i / S) & 1, a.hdr)) break;
        tc_fence_after();
        const uint8_t* w = kInt8 ? ring2 + s * stage2 : ring + s * stage;
        const uint64_t wd = smem_desc(smem_u32(w), 16, 1024, kLayoutSw128);
        const uint64_t xd = smem_desc(smem_u32(w + kRowsW * 128), 16, 1024, kLayoutSw128);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {   // 32 bytes of K at a time
          if (kInt8) mma_ss(tmem, wd + 2 * kk, xd + 2 * kk, idesc, (i | kk) != 0);
          else mma_ss_f8(tmem, wd + 2 * kk, xd + 2 * kk, idesc, (i | kk) != 0);
        }
        mma_commit(kInt8 ? &empty2[s] : &empty[s]);
      }
      mma_commit(done);
    }
  } else if (kInt8 && warp >= 4) {
    for (int i = 0; i < kn; ++i) {
      const int s = i % S, s2 = i % S2;
      bool ok = wait_bar(&full[s], (i / S) & 1, a.hdr);
      if (ok && i >= S2) ok = wait_bar(&empty2[s2], ((i / S2) & 1) ^ 1, a.hdr);
      if (!__all_sync(0xffffffffu, ok)) break;
      widen_rows(ring + s * stage, ring2 + s2 * stage2, kRowsW + TN, tid - 128, 32 * kConvWarps);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&empty[s]);
        mbar_arrive(&full2[s2]);
      }
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
    for (int t = lo + warp; t < hi; t += warps) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t at = smem_u32(part + t * kRowsW + 4 * lane);
      for (int c = 0; c < a.C; ++c) {
        const float4 u = ld_cluster_f4(a.C > 1 ? mapa_shared(at, c) : at);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      const float xs = a.x_scale[t0 + t];
      const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * xs * ws.x, v.y * xs * ws.y);
      const __nv_bfloat162 q = __floats2bfloat162_rn(v.z * xs * ws.z, v.w * xs * ws.w);
      *reinterpret_cast<uint2*>(a.out + (t0 + t) * a.out_stride + n0 + 4 * lane) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
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

// ------------------------------------------------------------------ many tokens

template <bool kInt8>
struct Pair {
  static constexpr int kN = kInt8 ? 192 : 256;              // channels of a tile
  static constexpr int kStepK = kInt8 ? 64 : 128;           // codes of a stage
  static constexpr int kRows = 128 + kN / 2;                // rows of a stage in a CTA: its tokens, its channels
  static constexpr int kStage = kRows * kStepK;
  static constexpr int kStages = 6;
  static constexpr int kStages2 = 4;                        // int8, widened: tokens 32 TMEM columns, channels a box
  static constexpr int kStage2 = kN / 2 * 128;
  static constexpr int kBoxOut = 128 * 128;                 // 128 tokens x 64 channels bf16
  static constexpr int kRing2 = kStages * kStage;
  static constexpr int kOut = kRing2 + (kInt8 ? kStages2 * kStage2 : 0);
  static constexpr int kScales = kOut + 2 * kBoxOut;        // [kN] channel scales
  static constexpr int kBars = kScales + kN * 4;
  static constexpr int kSmem = 1024 + kBars + 8 * (2 * kStages + 2 * kStages2 + 4) + 16;
  static_assert(kSmem <= 232448);
  static constexpr int kThreads = kInt8 ? 512 : 256;
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

__device__ __forceinline__ bool wait_bar_cluster(uint64_t* bar, uint32_t parity, PlanHeader* hdr) {
  if (mbar_wait<true>(bar, parity, kWaitLimitNs)) return true;
  atomicOr(&hdr->status, kDeviceTimeout);
  return false;
}

// Warp 0 copies, warp 1 (of the pair's first CTA) issues the products, warp 2 owns the tensor memory,
// warps 4-7 are the epilogue; int8: warps 8-11 widen tokens (thread = row = TMEM lane), 12-15 channels.
template <bool kInt8>
__global__ void __launch_bounds__(Pair<kInt8>::kThreads, 1) __cluster_dims__(2, 1, 1)
    pair_kernel(const __grid_constant__ Maps maps, const Args a) {
  using P = Pair<kInt8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + P::kBars);   // e4m3: the first CTA's, for both; int8: each its own
  uint64_t* empty = full + P::kStages;
  uint64_t* full2 = empty + P::kStages;      // int8: widened, in the first CTA
  uint64_t* empty2 = full2 + P::kStages2;
  uint64_t* acc_full = empty2 + P::kStages2;           // a tile's products are done
  uint64_t* acc_empty = acc_full + 2;        // ... and read, in the first CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int mtiles = (a.T + 255) / 256, ntiles = (a.N + P::kN - 1) / P::kN;
  const int tiles = mtiles * ntiles, pairs = (int)gridDim.x / 2, first = (int)blockIdx.x / 2;
  const int nkb = (a.K + P::kStepK - 1) / P::kStepK;

  if (tid == 0) {
    for (int s = 0; s < P::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kInt8 ? 8 : 1);
    }
    for (int s = 0; s < P::kStages2; ++s) {
      mbar_init(&full2[s], 16);
      mbar_init(&empty2[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 8);
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
  constexpr uint32_t kColA = 2 * P::kN;   // int8: columns of the widened tokens

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int i = 0;
      for (int tile = first; tile < tiles && ok; tile += pairs) {
        const Tile at = tile_of(tile, mtiles, ntiles, P::kN);
        for (int kb = 0; kb < nkb; ++kb, ++i) {
          const int s = i % P::kStages;
          if (i >= P::kStages && !(ok = wait_bar(&empty[s], ((i / P::kStages) & 1) ^ 1, a.hdr))) break;
          uint8_t* dst = sm + s * P::kStage;
          if (kInt8) {
            mbar_arrive_expect_tx(&full[s], P::kStage);
            tma_load_2d(dst, &maps.x, &full[s], kb * P::kStepK, at.m0 + 128 * rank);
            tma_load_2d(dst + 128 * P::kStepK, &maps.w, &full[s], kb * P::kStepK, at.n0 + P::kN / 2 * rank);
          } else {
            const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * P::kStage);
            tma_load_2d_pair(dst, &maps.x, bar, kb * P::kStepK, at.m0 + 128 * rank);
            tma_load_2d_pair(dst + 128 * P::kStepK, &maps.w, bar, kb * P::kStepK, at.n0 + P::kN / 2 * rank);
          }
        }
      }
      // no copy and no arrival outlives the pair, whatever became of those who wait for them
      for (int j = max(0, i - P::kStages); j < i; ++j) {
        if (kInt8 || rank == 0) wait_bar(&full[j % P::kStages], (j / P::kStages) & 1, a.hdr);
        wait_bar(&empty[j % P::kStages], (j / P::kStages) & 1, a.hdr);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_f32(256, P::kN, 0);   // f16 and e4m3 are both type 0 of their kinds
      bool ok = true;
      int i = 0, n = 0;
      for (int tile = first; tile < tiles && ok; tile += pairs, ++n) {
        const int b = n & 1;
        const uint32_t d = tmem + b * P::kN;
        if (n >= 2 && !(ok = wait_bar_cluster(&acc_empty[b], ((n >> 1) & 1) ^ 1, a.hdr))) break;
        tc_fence_after();
        for (int kb = 0; kb < nkb; ++kb, ++i) {
          if (kInt8) {
            const int s = i % P::kStages2;
            if (!(ok = wait_bar_cluster(&full2[s], (i / P::kStages2) & 1, a.hdr))) break;
            tc_fence_after();
            const uint64_t wd = smem_desc(smem_u32(sm + P::kRing2 + s * P::kStage2), 16, 1024, kLayoutSw128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts_pair(d, tmem + kColA + 32 * s + 8 * kk, wd + 2 * kk, idesc, (kb | kk) != 0);
            mma_commit_pair(&empty2[s]);
          } else {
            const int s = i % P::kStages;
            if (!(ok = wait_bar_cluster(&full[s], (i / P::kStages) & 1, a.hdr))) break;
            tc_fence_after();
            const uint64_t xd = smem_desc(smem_u32(sm + s * P::kStage), 16, 1024, kLayoutSw128);
            const uint64_t wd = smem_desc(smem_u32(sm + s * P::kStage + 128 * 128), 16, 1024, kLayoutSw128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss_f8_pair(d, xd + 2 * kk, wd + 2 * kk, idesc, (kb | kk) != 0);
            mma_commit_pair(&empty[s]);
          }
        }
        mma_commit_pair(&acc_full[b]);
      }
    }
  } else if (warp >= 4 && warp < 8) {
    const int row = tid - 128;                       // token of the CTA's half = TMEM lane
    uint8_t* box = sm + P::kOut;
    float* ws = reinterpret_cast<float*>(sm + P::kScales);   // read between a chunk's two barriers only
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    int n = 0, chunk = 0;
    for (int tile = first; tile < tiles; tile += pairs, ++n) {
      const Tile at = tile_of(tile, mtiles, ntiles, P::kN);
      const int b = n & 1, m0 = at.m0 + 128 * rank;
      for (int c = row; c < P::kN; c += 128) ws[c] = at.n0 + c < a.N ? a.w_scale[at.n0 + c] : 0.f;
      const float xs = m0 + row < a.T ? a.x_scale[m0 + row] : 0.f;
      bool ok = wait_bar(&acc_full[b], (n >> 1) & 1, a.hdr);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < P::kN; c0 += 64, ++chunk) {
        uint32_t r[2][32];
        tmem_ld32(tmem + b * P::kN + c0 + lanes, r[0]);
        tmem_ld32(tmem + b * P::kN + c0 + 32 + lanes, r[1]);
        tmem_ld_wait();
        if (c0 + 64 == P::kN) {   // the tile's accumulator is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[b]), 0));
        }
        // the box written two chunks ago has left (its writer waits), the scales are there
        uint8_t* dst = box + (chunk & 1) * P::kBoxOut;
        if (row == 0) bulk_wait_read<1>();
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const int c = 8 * g + 2 * j;
            const float4 w4 = *reinterpret_cast<const float4*>(ws + c0 + c);
            const uint32_t* v = &r[c >> 5][c & 31];
            const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(v[0]) * xs * w4.x, __uint_as_float(v[1]) * xs * w4.y);
            const __nv_bfloat162 q = __floats2bfloat162_rn(__uint_as_float(v[2]) * xs * w4.z, __uint_as_float(v[3]) * xs * w4.w);
            o[j] = *reinterpret_cast<const uint32_t*>(&p);
            o[j + 1] = *reinterpret_cast<const uint32_t*>(&q);
          }
          *reinterpret_cast<uint4*>(dst + row * 128 + ((g ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (row == 0) {
          if (m0 < a.T && at.n0 + c0 < a.N) tma_store_2d(&maps.out, dst, at.n0 + c0, m0);
          bulk_commit();
        }
      }
    }
    if (row == 0) bulk_wait_all();
  } else if (kInt8 && warp >= 8) {
    const bool tokens = warp < 12;
    const int row = tid & 127;
    int i = 0;
    bool ok = true;
    for (int tile = first; tile < tiles && ok; tile += pairs)
      for (int kb = 0; kb < nkb; ++kb, ++i) {
        const int s = i % P::kStages, s2 = i % P::kStages2;
        ok = wait_bar(&full[s], (i / P::kStages) & 1, a.hdr);
        if (ok && i >= P::kStages2) ok = wait_bar(&empty2[s2], ((i / P::kStages2) & 1) ^ 1, a.hdr);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const uint8_t* raw = sm + s * P::kStage;
        if (tokens) {
          tc_fence_after();
          uint32_t o[32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {   // 64-byte rows in the 64-byte swizzle
            uint4 lo, hi;
            widen(*reinterpret_cast<const uint4*>(raw + row * 64 + ((q ^ ((row >> 1) & 3)) << 4)), lo, hi);
            o[8 * q] = lo.x; o[8 * q + 1] = lo.y; o[8 * q + 2] = lo.z; o[8 * q + 3] = lo.w;
            o[8 * q + 4] = hi.x; o[8 * q + 5] = hi.y; o[8 * q + 6] = hi.z; o[8 * q + 7] = hi.w;
          }
          tmem_st32(tmem + kColA + 32 * s2 + ((uint32_t)(32 * (warp & 3)) << 16), o);
          tmem_st_wait();
          tc_fence_before();
        } else {
          uint8_t* dst = sm + P::kRing2 + s2 * P::kStage2;
          for (int j = row; j < P::kN / 2 * 4; j += 128) {
            const int r = j >> 2, q = j & 3;   // place q of row r holds the codes of piece p
            const int p = q ^ ((r >> 1) & 3);
            uint4 lo, hi;
            widen(*reinterpret_cast<const uint4*>(raw + 128 * 64 + 16 * j), lo, hi);
            *reinterpret_cast<uint4*>(dst + r * 128 + (((2 * p) ^ (r & 7)) << 4)) = lo;
            *reinterpret_cast<uint4*>(dst + r * 128 + (((2 * p + 1) ^ (r & 7)) << 4)) = hi;
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&empty[s]);
          mbar_arrive_cluster(mapa_shared(smem_u32(&full2[s2]), 0));
        }
      }
    // the pair's last arrivals on this CTA's barriers
    if (warp == 8 && lane == 0)
      for (int j = max(0, i - P::kStages2); j < i; ++j) wait_bar(&empty2[j % P::kStages2], (j / P::kStages2) & 1, a.hdr);
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

// Rows of K codes as a tensor map with boxes of `rows` rows and `step` codes.
bool encode_codes(CUtensorMap* m, const void* p, int K, int rows_total, int step, int rows, CUtensorMapSwizzle swizzle) {
  const wg::EncodeTiledFn fn = wg::encode_fn();
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows_total};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {(cuuint32_t)step, (cuuint32_t)rows};
  cuuint32_t es[2] = {1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

template <bool kInt8>
cudaError_t launch_split(Args a, const void* x, const void* w, int sms, cudaStream_t s) {
  constexpr int kStepK = kInt8 ? 64 : 128;
  Maps maps;
  a.TN = a.T >= kMaxTokens ? kMaxTokens : (a.T + 15) / 16 * 16;
  const int tiles = (a.N + kRowsW - 1) / kRowsW, ttiles = (a.T + a.TN - 1) / a.TN;
  const int nkb = (a.K + kStepK - 1) / kStepK;
  a.C = 1;
  while (a.C < 8 && (long long)tiles * ttiles * a.C * 2 <= sms && nkb >= 8 * a.C) a.C *= 2;
  const int rows = kRowsW + a.TN, budget = 200 * 1024;
  if (kInt8) {
    a.S2 = std::min(4, budget * 2 / 3 / (rows * 128));
    a.S = std::min(kMaxStages, (budget - a.S2 * rows * 128) / (rows * kStepK));
  } else {
    a.S2 = 0;
    a.S = std::min(kMaxStages, budget / (rows * kStepK));
  }
  const CUtensorMapSwizzle swizzle = kInt8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_codes(&maps.w, w, a.K, a.N, kStepK, kRowsW, swizzle) ||
      !encode_codes(&maps.x, x, a.K, a.T, kStepK, a.TN, swizzle))
    return cudaErrorInvalidValue;
  const size_t ring = std::max((size_t)a.S * rows * kStepK + (size_t)a.S2 * rows * 128, (size_t)a.TN * kRowsW * 4);
  const size_t smem = 1024 + ring + (4 * kMaxStages + 2) * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * a.C, ttiles);
  cfg.blockDim = dim3(kInt8 ? 128 + 32 * kConvWarps : 128);
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

template <bool kInt8>
cudaError_t launch_pair(const Args& a, const void* x, const void* w, int sms, cudaStream_t s) {
  using P = Pair<kInt8>;
  Maps maps;
  const CUtensorMapSwizzle swizzle = kInt8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_codes(&maps.x, x, a.K, a.T, P::kStepK, 128, swizzle) ||
      !encode_codes(&maps.w, w, a.K, a.N, P::kStepK, P::kN / 2, swizzle) ||
      !encode_out(&maps.out, a.out, a.T, a.N, a.out_stride))
    return cudaErrorInvalidValue;
  const long long tiles = (long long)((a.T + 255) / 256) * ((a.N + P::kN - 1) / P::kN);
  const int pairs = (int)std::min<long long>(tiles, sms / 2);
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(pair_kernel<kInt8>), P::kSmem);
  if (e != cudaSuccess) return e;
  pair_kernel<kInt8><<<2 * pairs, P::kThreads, P::kSmem, s>>>(maps, a);
  return cudaGetLastError();
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
  if (T > lin::kMaxTokens) return int8 ? lin::launch_pair<true>(a, x, w, sms, s) : lin::launch_pair<false>(a, x, w, sms, s);
  return int8 ? lin::launch_split<true>(a, x, w, sms, s) : lin::launch_split<false>(a, x, w, sms, s);
}

}  // namespace mla
