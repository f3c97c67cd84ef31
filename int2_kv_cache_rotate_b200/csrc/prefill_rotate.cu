// The rotations around the 4-bit cache's bf16 prefill (prefill_int4.cu) on the
// tcgen05 tensor cores: q~ = q R_K before it, o = (o' / l) R_V^T behind it.
//
// One CTA per 128 rows (token, query head) of a KV head; two fit an SM.  Both
// are one M 128, N 128, K 128 product with the head's 128 x 128 matrix in two
// 16-bit parts (32 MMAs of K 16 per 256 rows), and both round their result's
// or their input's rows once:
//   query  A = q (bf16, exact), B = R_K as the first two bf16 parts of the
//          cache's staged image (2^-16 of it); the row is scaled by 2^-e and
//          rounded to fp16, which is what the attention takes;
//   output the merged row is normalised, goes through the butterfly in
//          registers in fp32 and, scaled by 2^-e, to fp16 (2^-11 of a value,
//          an eighth of a bf16 output's rounding), B = U_V as two fp16 parts.
// Bound: the latency of load, product and store one after the other, and behind
// the attention the bytes (32768 rows: 17 MB, and up to three pieces of each).
// 32768 rows take 10 us before the attention (39 on the CUDA cores) and 36
// behind it (45 and more); fp32 output and the 2-bit cache keep the CUDA cores,
// whose fp32 products their smaller tolerances count on.
#include "okv_common.cuh"
#include "okv_internal.h"
#include "prefill_common.cuh"
#include "umma.cuh"

namespace okv {
namespace {

constexpr int kRoRows = 128;
constexpr uint32_t kRoRegion = 16384;             // 128 rows x 128 B: one K-block of 64
constexpr uint32_t kRoOffA = 4 * kRoRegion;       // B before it: parts hi and lo, two K-blocks each
constexpr uint32_t kRoIdescBf16 = um_idesc(128, true, true), kRoIdescFp16 = um_idesc(128, false, false);
constexpr uint32_t kRoOffCtl = 6 * kRoRegion;
struct RoCtl {
  uint64_t b_full, done;
  uint32_t tmem_slot;
  float scale[kRoRows];
};
constexpr size_t kRoSmem = 1024 + kRoOffCtl + sizeof(RoCtl);

// row rk (0 .. T g - 1) of KV head hk: token rk / g, query head hk g + rk % g
__device__ __forceinline__ size_t ro_row(const PrefillArgs& a, int hk, int rk) {
  return (size_t)(rk / a.g) * a.hq + hk * a.g + rk % a.g;
}

// 2^-e with amax 2^-e in [1, 2)
__device__ __forceinline__ int ro_exponent(float amax) {
  const int e = amax > 0.f ? ((__float_as_int(amax) >> 23) & 0xff) - 127 : 0;
  return max(-100, min(100, e));
}
__device__ __forceinline__ float ro_pow2(int e) { return __int_as_float((127 + e) << 23); }

__device__ __forceinline__ uint32_t ro_pack(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// D = A B^T over both parts of B, committed to bar (one elected thread)
__device__ __forceinline__ void ro_product(uint32_t tmem, uint32_t base, uint32_t idesc, uint64_t* bar) {
#pragma unroll
  for (int pt = 0; pt < 2; ++pt)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t at = (uint32_t)(k >> 2) * kRoRegion + (uint32_t)(k & 3) * 32u;
      um_mma(tmem, um_desc(base + kRoOffA + at), um_desc(base + 2 * pt * kRoRegion + at), idesc, pt + k > 0 ? 1u : 0u);
    }
  um_commit(bar);
}

__global__ void __launch_bounds__(128, 2) prefill_qrot_int4_kernel(const __grid_constant__ PrefillArgs a,
                                                                  const uint8_t* r_image) {
  extern __shared__ unsigned char ro_raw[];
  const uint32_t raw_u32 = smem_u32(ro_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;
  unsigned char* gb = ro_raw + (base - raw_u32);
  RoCtl& ctl = *reinterpret_cast<RoCtl*>(gb + kRoOffCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.y, nrows = a.T * a.g, r0 = blockIdx.x * kRoRows;
  grid_dep_launch();  // the attention may start fetching codes
  if (tid == 0) {
    mbar_init(&ctl.b_full, 1);
    mbar_init(&ctl.done, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&ctl.b_full, 4 * kRoRegion);
    bulk_g2s(gb, r_image + (size_t)2 * hk * kRImageBytesPerHead, 4 * kRoRegion, &ctl.b_full);
  }
  __syncwarp();
  if (warp == 0) um_alloc(&ctl.tmem_slot, 128);
  uint4 v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int at = tid + 128 * i;
    v[i] = __ldg(reinterpret_cast<const uint4*>(a.q + ro_row(a, hk, min(r0 + (at >> 4), nrows - 1)) * kD) + (at & 15));
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t at = (uint32_t)(tid + 128 * i), c = at & 15u;
    *reinterpret_cast<uint4*>(gb + kRoOffA + (c >> 3) * kRoRegion + um_swz(at >> 4, (c & 7u) * 16u)) = v[i];
  }
  um_fence_proxy_async();
  um_fence_before();
  __syncthreads();
  um_fence_after();
  const uint32_t tmem = ctl.tmem_slot;
  bool issued = false;
  if (warp == 0) {
    issued = __all_sync(0xffffffffu, mbar_wait_bounded(&ctl.b_full, 0u)) != 0;
    if (issued && um_elect()) ro_product(tmem, base, kRoIdescBf16, &ctl.done);
    __syncwarp();
  }
  const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(&ctl.done, 0u)) != 0;
  if (ok) {
    um_fence_after();
    const uint32_t t = tmem + ((uint32_t)(32 * warp) << 16);
    float amax = 0.f;
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      float x[32];
      um_ld32(t + 32u * b, x);
      um_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(x[j]));
    }
    const int e = ro_exponent(amax);
    const float down = ro_pow2(-e);
    const int rk = r0 + 32 * warp + lane;
    const size_t row = ro_row(a, hk, min(rk, nrows - 1));
    uint4* dst = reinterpret_cast<uint4*>(a.qhi + row * kD);
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      float x[32];
      um_ld32(t + 32u * b, x);
      um_wait_ld();
      if (rk < nrows) {
#pragma unroll
        for (int j = 0; j < 32; j += 8)  // channels in the order 0 4 1 5 2 6 3 7 of the key tiles
          dst[4 * b + (j >> 3)] = make_uint4(ro_pack(x[j] * down, x[j + 4] * down), ro_pack(x[j + 1] * down, x[j + 5] * down),
                                             ro_pack(x[j + 2] * down, x[j + 6] * down), ro_pack(x[j + 3] * down, x[j + 7] * down));
      }
    }
    if (rk < nrows) a.qaux[row * kQaux + 4] = ro_pow2(e);
  } else if (lane == 0) {
    raise_flag(a.status, OKV_DEV_TIMEOUT);
  }
  // nothing in flight may reach this shared memory or TMEM later
  if (warp == 0) {
    mbar_drain_bounded(&ctl.b_full, 0u);
    if (issued) mbar_drain_bounded(&ctl.done, 0u);
  }
  um_fence_before();
  __syncthreads();
  if (warp == 0) {
    um_fence_after();
    um_dealloc(tmem, 128);
  }
}

constexpr int kRoBatch = 4;  // rows a warp merges at a time

__global__ void __launch_bounds__(256, 2)
    prefill_unrotate_int4_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ P4Split sp) {
  extern __shared__ unsigned char ro_raw[];
  const uint32_t raw_u32 = smem_u32(ro_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;
  unsigned char* gb = ro_raw + (base - raw_u32);
  RoCtl& ctl = *reinterpret_cast<RoCtl*>(gb + kRoOffCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.y, nrows = a.T * a.g, r0 = blockIdx.x * kRoRows;
  if (tid == 0) {
    mbar_init(&ctl.done, 1);
    fence_mbar_init();
  }
  {
    // B = U_V, row i K-major: 8 channels of a row per piece, hi and lo
    const float4* U = reinterpret_cast<const float4*>(a.u_v + (size_t)hk * kD * kD);
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += 4) {
      float4 u[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = tid + 256 * (i0 + i);
        u[i][0] = __ldg(U + 2 * at);
        u[i][1] = __ldg(U + 2 * at + 1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = (uint32_t)(tid + 256 * (i0 + i)), c = at & 15u;
        const float x[8] = {u[i][0].x, u[i][0].y, u[i][0].z, u[i][0].w, u[i][1].x, u[i][1].y, u[i][1].z, u[i][1].w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 hh = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
          const float2 f = __half22float2(hh);
          h[j] = *reinterpret_cast<const uint32_t*>(&hh);
          l[j] = ro_pack(x[2 * j] - f.x, x[2 * j + 1] - f.y);
        }
        unsigned char* dst = gb + (c >> 3) * kRoRegion + um_swz(at >> 4, (c & 7u) * 16u);
        *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(dst + 2 * kRoRegion) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  }
  grid_dep_wait();  // the attention's outputs are read from here on
  if (warp == 0) um_alloc(&ctl.tmem_slot, 128);  // (behind the wait: no CTA holds TMEM while it waits for a grid)
  const int t0 = r0 / kP4Rows * kP4Rows;
  int pieces;
  const int j0 = sp.ranges_of(hk * sp.tiles + r0 / kP4Rows, pieces);
  const int r = rev5(lane);
#pragma unroll 1
  for (int q = 0; q < 16; q += kRoBatch) {
    const int rb = 16 * warp + q;  // the batch's rows of the tile
    float4 o4[kRoBatch];
    float l[kRoBatch];
    if (pieces > 1) {
      const float* first = sp.piece(j0, 1);
      const float* others = sp.piece(j0, 0);
      const size_t next = (size_t)2 * sp.prow * kOStride;
      auto piece_row = [&](int s, int k) {
        return (s == 0 ? first : others + s * next) + (size_t)(min(r0 + rb + k, nrows - 1) - t0) * kOStride;
      };
      // lane s holds (l, maximum) of piece s (at most 32), then its weight 2^(m_s - m)
      float w[kRoBatch];
#pragma unroll
      for (int k = 0; k < kRoBatch; ++k) {
        const float2 lm =
            lane < pieces ? *reinterpret_cast<const float2*>(piece_row(lane, k) + 128) : make_float2(0.f, 0.f);
        l[k] = lm.x;
        w[k] = lm.y;
        o4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kRoBatch; ++k) {
        // (a piece without a key has l = 0; an l that is NaN goes on to the output)
        const float top = warp_max(l[k] != 0.f ? w[k] : -INFINITY);
        w[k] = l[k] != 0.f ? exp2f(w[k] - top) : 0.f;
        l[k] = warp_sum(w[k] * l[k]);
      }
#pragma unroll 2
      for (int s = 0; s < pieces; ++s) {  // the batch's rows' loads in flight together
        float4 x[kRoBatch];
        float ws[kRoBatch];
#pragma unroll
        for (int k = 0; k < kRoBatch; ++k) {
          ws[k] = __shfl_sync(0xffffffffu, w[k], s);
          x[k] = ws[k] != 0.f ? *reinterpret_cast<const float4*>(piece_row(s, k) + 4 * r) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kRoBatch; ++k)
          o4[k] = make_float4(fmaf(ws[k], x[k].x, o4[k].x), fmaf(ws[k], x[k].y, o4[k].y), fmaf(ws[k], x[k].z, o4[k].z),
                              fmaf(ws[k], x[k].w, o4[k].w));
      }
    } else {
#pragma unroll
      for (int k = 0; k < kRoBatch; ++k) {
        const float* src = a.obuf + ro_row(a, hk, min(r0 + rb + k, nrows - 1)) * kOStride;
        o4[k] = *reinterpret_cast<const float4*>(src + 4 * r);  // rotated channels 4 r .. 4 r + 3
        l[k] = src[128];
      }
    }
#pragma unroll
    for (int k = 0; k < kRoBatch; ++k) {
      const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
      // lane l: pre-permutation channels l + 32 aa = rotated channels 4 rev5(l) + rev2(aa)
      float y[4] = {o4[k].x * inv, o4[k].z * inv, o4[k].y * inv, o4[k].w * inv};
      wht128_warp(y, lane);
      const float amax = warp_max(fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3]))));
      const int e = ro_exponent(amax);
      const float down = ro_pow2(-e);
#pragma unroll
      for (int aa = 0; aa < 4; ++aa)
        *reinterpret_cast<__half*>(gb + kRoOffA + (uint32_t)(aa >> 1) * kRoRegion +
                                   um_swz((uint32_t)(rb + k), (uint32_t)(32 * (aa & 1) + lane) * 2u)) =
            __float2half_rn(y[aa] * down);
      if (lane == 0) ctl.scale[rb + k] = ro_pow2(e) * kInvSqrtD;
    }
  }
  um_fence_proxy_async();
  um_fence_before();
  __syncthreads();
  um_fence_after();
  const uint32_t tmem = ctl.tmem_slot;
  if (warp == 0) {
    if (um_elect()) ro_product(tmem, base, kRoIdescFp16, &ctl.done);
    __syncwarp();
  }
  const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(&ctl.done, 0u)) != 0;
  if (ok) {
    um_fence_after();
    const int tr = 32 * (warp & 3) + lane, rk = r0 + tr;  // the thread's row, and half of its channels
    const uint32_t t = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 64u * (uint32_t)(warp >> 2);
    const float s = ctl.scale[tr];
    uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + ro_row(a, hk, min(rk, nrows - 1)) * kD + 64 * (warp >> 2));
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      float x[32];
      um_ld32(t + 32u * b, x);
      um_wait_ld();
      if (rk < nrows) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[j + 2 * i] * s, x[j + 2 * i + 1] * s);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
          }
          dst[4 * b + (j >> 3)] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  } else if (lane == 0) {
    raise_flag(a.status, OKV_DEV_TIMEOUT);
  }
  if (warp == 0) mbar_drain_bounded(&ctl.done, 0u);
  um_fence_before();
  __syncthreads();
  if (warp == 0) {
    um_fence_after();
    um_dealloc(tmem, 128);
  }
}

}  // namespace

okv_status launch_prefill_qrot_int4(const PrefillArgs& a, const void* r_image, cudaStream_t s) {
  static std::atomic<uint32_t> attr{0};
  const cudaError_t e = set_smem_limit_once((const void*)prefill_qrot_int4_kernel, (int)kRoSmem, attr);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "prefill rotation smem attribute: %s", cudaGetErrorString(e));
  const dim3 grid((unsigned)((a.T * a.g + kRoRows - 1) / kRoRows), (unsigned)a.hkv);
  prefill_qrot_int4_kernel<<<grid, 128, kRoSmem, s>>>(a, (const uint8_t*)r_image);
  return check_launch("prefill query rotation");
}

okv_status launch_prefill_unrotate_int4(const PrefillArgs& a, const P4Split& sp, cudaStream_t s) {
  static std::atomic<uint32_t> attr{0};
  cudaError_t e = set_smem_limit_once((const void*)prefill_unrotate_int4_kernel, (int)kRoSmem, attr);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "prefill rotation smem attribute: %s", cudaGetErrorString(e));
  const dim3 grid((unsigned)((a.T * a.g + kRoRows - 1) / kRoRows), (unsigned)a.hkv);
  e = launch_pdl(prefill_unrotate_int4_kernel, grid, dim3(256), kRoSmem, s, true, a, sp);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "prefill un-rotation launch: %s", cudaGetErrorString(e));
  return check_launch("prefill un-rotation");
}

}  // namespace okv
