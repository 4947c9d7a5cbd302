// Launcher of the expanded-form prefill (internal to libmla_decode.so).
#pragma once
#include <cuda_fp4.h>

#include "mla_kernels.cuh"

namespace mla {

struct PrefillCall {
  mla_dims_t d;
  int fmt, B, T, mask, window, bt_stride;
  float scale;
  const void* q;
  const uint32_t* offsets;
  const void* pool;
  const float* kv_scales;                    // e4m3 cache
  const int32_t* block_table;
  const uint32_t* cache_lens;
  const void *w_uk, *w_uv;                   // bf16, or e4m3 with scales
  const float *w_uk_scale, *w_uv_scale;      // NULL for bf16 weights
  void* out;
  float* lse_out;
  void* ws;
};

// Byte offsets of the workspace: plan header, requests, query blocks, live rows of each
// key tile, rope and latent boxes of each tile, widened weights (e4m3), partial results
// (several key splits), then K and V boxes, head_bytes per head of a pass.
struct PrefillLayout {
  size_t header, reqs, items, live, rope, lat, w_uk, w_uv, part_o, part_lse, kv, head_bytes;
  long long cap_tiles, max_items;
};

bool prefill_supported(const mla_dims_t& d);
PrefillLayout prefill_layout(const mla_dims_t& d, int B, int T, long long total_keys, int splits, bool fp8);
int prefill_splits(const mla_dims_t& d, int B, int T, long long total_keys, int sms);
// `heads` heads per pass through the K and V boxes.
cudaError_t launch_prefill(const PrefillCall& c, const PrefillLayout& lay, int heads, int splits, cudaStream_t s);

}  // namespace mla
