// What the chunked-prefill kernels share: their arguments, the partial rows
// they hand to the un-rotation, and the split of the key positions.
#pragma once

#include "okv_common.cuh"
#include "okv_internal.h"

namespace okv {

struct PrefillArgs {
  const __nv_bfloat16* q;  // [T][Hq][128]
  const int32_t* block_table;
  const uint8_t* pages;
  const __half* ring;
  const __half* sink;
  const float* u_k;
  const float* u_v;
  uint32_t* status;
  __half* qhi;   // [T][Hq][128]: hi half of q~ 2^-e
  __half* qlo;   // [T][Hq][128]: lo half
  float* qaux;   // [T][Hq][8]: sum of q~ per group (4), 2^e, spare
  float* obuf;   // [splits][T][Hq][kOStride]: o' (128), l, running maximum (log2 units)
  void* out;     // [T][Hq][128], fp32 or bf16
  int out_bf16;
  int q_order;   // qhi in prefill_int4.cu's channel order, no qlo
  int splits;    // key ranges per row, merged by the un-rotation
  int T, hq, hkv, g, ng, bhb, slot, L, first, mbps, num_blocks, nsink;
};

constexpr int kQaux = 8;
constexpr int kOStride = 132;

// The 4-bit cache's attention with bf16 output (prefill_int4.cu): 256 query
// rows of a KV head per CTA.
constexpr int kP4Rows = 256;
okv_status launch_prefill_int4_bf16(const PrefillArgs& a, cudaStream_t s);

}  // namespace okv
