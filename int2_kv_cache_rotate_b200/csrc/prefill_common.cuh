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
  float* obuf;   // [T][Hq][kOStride]: o' (128), l, running maximum (log2 units)
  void* out;     // [T][Hq][128], fp32 or bf16
  int out_bf16;
  int q_order;   // qhi in prefill_int4.cu's channel order, no qlo
  int T, hq, hkv, g, ng, bhb, slot, L, first, mbps, num_blocks, nsink;
};

constexpr int kQaux = 8;
constexpr int kOStride = 132;

// The 4-bit cache's attention with bf16 output (prefill_int4.cu): tiles of 256
// query rows of a KV head, each over the keys its last row sees, in chunks of
// 128.  The tiles (KV head hk, tile x: index hk tiles + x), laid end to end, are
// cut into `ctas` ranges of about the same work, one per CTA, so no SM idles when
// the tiles do not divide evenly among them.  A tile that one range holds whole
// goes to obuf; the pieces of a cut tile go to `part`, slot 1 of the range where
// the tile begins and slot 0 of the others, and the un-rotation merges them.
constexpr int kP4Rows = 256;
constexpr int kP4Keys = 128;       // key positions per chunk
constexpr int kP4MostPieces = 32;  // of a tile: a warp's lanes in the merge
constexpr int kP4MostCtas = 256;
struct P4Split {
  int tiles;     // per head
  int ctas;
  int prow;      // rows of a piece in `part`
  float* part;   // [ctas][2][prow][kOStride]
  int2 start[kP4MostCtas + 1];  // first tile and chunk of each range, and the end; strictly increasing

  __device__ float* piece(int j, int slot) const { return part + ((size_t)(2 * j + slot) * prow) * kOStride; }
  // the ranges with a piece of tile t: returns the first, sets how many
  __device__ int ranges_of(int t, int& pieces) const {
    int cut[2];  // the first range that starts inside the tile, the first that starts behind it
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int lo = 1, hi = ctas;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const int2 s = start[mid];
        if (s.x > t || (k == 0 && s.x == t && s.y > 0)) hi = mid;
        else lo = mid + 1;
      }
      cut[k] = lo;
    }
    // (a range that starts at tile t + 1's first chunk is behind, one at tile t's first is not inside)
    pieces = 1 + max(cut[1] - cut[0], 0);
    return cut[0] - 1;
  }
};
__host__ __device__ inline int prefill_last_pos(const PrefillArgs& a, int x) {  // of any row of tile x
  const long long rows = (long long)a.T * a.g, end = (long long)kP4Rows * (x + 1);
  return a.first + (int)((end < rows ? end : rows) - 1) / a.g;
}
okv_status launch_prefill_int4_bf16(const PrefillArgs& a, const P4Split& sp, cudaStream_t s);

// Its rotations on the tensor cores (prefill_rotate.cu): q~ from the cache's
// staged image of R, and the output (16-byte aligned) from U_V.
okv_status launch_prefill_qrot_int4(const PrefillArgs& a, const void* r_image, cudaStream_t s);
okv_status launch_prefill_unrotate_int4(const PrefillArgs& a, const P4Split& sp, cudaStream_t s);

}  // namespace okv
