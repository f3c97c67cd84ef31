// Norms of queries and keys for each head with the position rotation in the
// same pass (okv_qk_norm_rope): the step between a model's fused projection
// and this library's append and attention calls.
//
//   y = x / sqrt(mean(x^2) + eps) * w                (128 channels of a head)
//   (a, b) -> (a cos - b sin, b cos + a sin) of the channel pairs inside
//   rot_dim, angle = position * inv_freq
//
// Bound: bytes.  A row (one token's head) is read once and written once.  A
// half-warp takes a row.  A lane holds two runs of four channels, chosen so
// that the pairs it rotates lie in it: runs j and j + rot_dim / 8 (pairs i, i +
// rot_dim / 2), or two neighbouring runs (adjacent pairs, and the channels past
// rot_dim).  So the only exchange between lanes is the sum of squares, four
// shuffles; the arithmetic is on the paired fp32 instructions.  (With eight
// consecutive channels a lane and the partner fetched by eight more shuffles,
// 8192 tokens of 48 heads took 53.5 us: 75 % of the shared-memory pipe, 67 % of
// the issue slots, 34 % of DRAM.)  A half-warp keeps one head and walks tokens,
// so that its pointers step by a stride and its weights stay in registers; the
// angles of a token do not depend on the head and are computed once per CTA
// into shared memory.  (The other way round, one token per half-warp walking
// the heads, took 40.5 us: looking up the tensor of every row made 150
// instructions of 60.)
//
// Rounding: the product position * inv_freq and its reduction to one turn are
// fp64 (in fp32 a position of 10^5 would leave an angle error of 4e-3); the
// sums and products are fp32; each output is rounded once, to bf16, the type
// that the append and the attention take.
#include <algorithm>
#include <type_traits>

#include "okv_common.cuh"
#include "okv_internal.h"

namespace okv {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrHalves = kNrThreads / 16;  // rows in flight per CTA
constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr double kTwoPi = 6.28318530717958647693;
constexpr double kTwoPiLo = 2.4492935982947064e-16;  // 2 pi - kTwoPi

struct NormRopeArgs {
  okv_norm_rope p;
};

// four consecutive channels of an input row, as loaded, as fp32 pairs and as stored
template <typename T>
using Raw4 = std::conditional_t<sizeof(T) == 4, uint4, uint2>;

template <typename T>
__device__ __forceinline__ void unpack4(const Raw4<T>& r, float2& lo, float2& hi) {
  if constexpr (sizeof(T) == 4) {
    lo = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    hi = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  } else if constexpr (std::is_same<T, __half>::value) {
    lo = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
    hi = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
  } else {
    lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
    hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
  }
}

__device__ __forceinline__ void store4(__nv_bfloat16* dst, float2 lo, float2 hi) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(lo.x, lo.y), b = __floats2bfloat162_rn(hi.x, hi.y);
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// CTA (x, y) takes tokens x * tokens .. + tokens - 1 (tokens <= kNrMaxTokens)
// and, of the rows of a token (query heads, then key heads, then value heads),
// y * 16 + half-warp, + 16 gridDim.y, ...; kAhead tokens' loads of a row are in
// flight before the first is used.
constexpr int kNrMaxTokens = 16;
// (8192 tokens of 48 heads: 3 rows ahead at 4 CTAs per SM 40.6 us, 4 ahead 45.0
// with spills, 4 ahead at 3 CTAs 42.9, 2 ahead at 5 CTAs 57, 8 ahead at 2 CTAs 48)
constexpr int kAhead = 3;

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads, sizeof(T) == 4 ? 3 : 4) norm_rope_kernel(NormRopeArgs args, int tokens) {
  const okv_norm_rope& p = args.p;
  __shared__ __align__(16) float cs[2][kNrMaxTokens * (kD / 2)];  // cosines, sines: [token][pair]
  __shared__ int live[kNrMaxTokens];                               // a negative position marks a padding row
  const int t0 = blockIdx.x * tokens;
  const int half = p.rot_dim >> 1;
  const int nt = min(tokens, p.num_tokens - t0);
  const int sub = threadIdx.x & 15;  // lane in the half-warp
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const int rows = hq + hkv + (p.v != nullptr ? hkv : 0);
  // this lane's two runs of four channels (first channels ca and cb), and whether they are rotated
  const bool turned = kInterleaved ? 8 * sub < p.rot_dim : 4 * sub < half;
  const int ca = kInterleaved ? 8 * sub : turned ? 4 * sub : p.rot_dim + 8 * (sub - (half >> 2));
  const int cb = kInterleaved || !turned ? ca + 4 : ca + half;
  const float* angles = turned ? &cs[0][4 * sub] : &cs[0][0];
  const int a_step = turned ? half : 0;
  bool first = true;
  // every half-warp runs the first round (it holds the CTA's barrier), and both
  // of a warp run the same rounds (the shuffles are warp-wide)
  const int row0 = blockIdx.y * kNrHalves + (threadIdx.x >> 4);
  for (int row = row0; first || (row & ~1) < rows; row += gridDim.y * kNrHalves) {
    const bool mine = row < rows;
    const int r = min(row, rows - 1);
    const bool is_q = r < hq, is_k = !is_q && r < hq + hkv;
    const int h = r - (is_q ? 0 : is_k ? hq : hq + hkv);
    const T* src = (const T*)(is_q ? p.q : is_k ? p.k : p.v);
    const long long ts = is_q ? p.q_token_stride : is_k ? p.k_token_stride : p.v_token_stride;
    src += t0 * ts + h * (is_q ? p.q_head_stride : is_k ? p.k_head_stride : p.v_head_stride);
    const int dh = is_q ? hq : hkv;
    __nv_bfloat16* dst = (__nv_bfloat16*)(is_q ? p.q_out : is_k ? p.k_out : p.v_out) + ((size_t)t0 * dh + h) * kD;
    Raw4<T> xa[kAhead], xb[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < nt) {
        xa[i] = __ldcs(reinterpret_cast<const Raw4<T>*>(src + i * ts + ca));
        xb[i] = __ldcs(reinterpret_cast<const Raw4<T>*>(src + i * ts + cb));
      }
    src += kAhead * ts;
    const bool normed = p.norm != 0 && (is_q || is_k);
    const bool rotated = turned && (is_q || is_k);  // channels past rot_dim and the values pass as they are
    const float* wp = is_q ? p.q_weight : p.k_weight;
    float4 wa = make_float4(1.f, 1.f, 1.f, 1.f), wb = wa;
    if (normed && wp != nullptr) {
      wa = make_float4(wp[ca], wp[ca + 1], wp[ca + 2], wp[ca + 3]);
      wb = make_float4(wp[cb], wp[cb + 1], wp[cb + 2], wp[cb + 3]);
    }
    if (first) {  // the CTA's angles, while the first rows are on their way
      for (int i = threadIdx.x; i < nt * half; i += kNrThreads) {
        const int ti = i / half, j = i - ti * half;
        const double angle = (double)p.positions[t0 + ti] * (double)p.inv_freq[j];
        const double full = rint(angle * kInvTwoPi);
        const float x = (float)fma(-full, kTwoPiLo, fma(-full, kTwoPi, angle));  // within half a turn of 0
        float sn, c;
        sincosf(x, &sn, &c);
        cs[0][i] = c * p.rope_scale;
        cs[1][i] = sn * p.rope_scale;
      }
      if (threadIdx.x < nt) live[threadIdx.x] = p.positions[t0 + threadIdx.x] >= 0;
      first = false;
      __syncthreads();
    }
    for (int tb = 0; tb < nt; tb += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = tb + i;
        if (t >= nt) break;
        float2 x[4];
        unpack4<T>(xa[i], x[0], x[1]);
        unpack4<T>(xb[i], x[2], x[3]);
        if (t + kAhead < nt) {
          xa[i] = __ldcs(reinterpret_cast<const Raw4<T>*>(src + ca));
          xb[i] = __ldcs(reinterpret_cast<const Raw4<T>*>(src + cb));
        }
        src += ts;
        float2 q2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) q2 = __ffma2_rn(x[j], x[j], q2);
        float ss = q2.x + q2.y;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (normed) {
          const float inv = rsqrtf(fmaf(ss, 1.f / kD, p.eps));
          const float2 i2 = make_float2(inv, inv);
          x[0] = __fmul2_rn(__fmul2_rn(x[0], i2), make_float2(wa.x, wa.y));
          x[1] = __fmul2_rn(__fmul2_rn(x[1], i2), make_float2(wa.z, wa.w));
          x[2] = __fmul2_rn(__fmul2_rn(x[2], i2), make_float2(wb.x, wb.y));
          x[3] = __fmul2_rn(__fmul2_rn(x[3], i2), make_float2(wb.z, wb.w));
        }
        if (rotated) {
          // the four angles of this lane's pairs (pairs 4 sub .. 4 sub + 3 either way)
          const float4 c4 = *reinterpret_cast<const float4*>(angles + t * a_step);
          const float4 s4 = *reinterpret_cast<const float4*>(angles + t * a_step + kNrMaxTokens * (kD / 2));
          if constexpr (kInterleaved) {  // pairs (x[j].x, x[j].y)
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[j] = make_float2(fmaf(x[j].x, c[j], -x[j].y * sn[j]), fmaf(x[j].y, c[j], x[j].x * sn[j]));
          } else {  // pairs (x[j], x[j + 2])
            const float2 c[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
            const float2 sn[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 a = x[j], b = x[j + 2];
              x[j] = __ffma2_rn(a, c[j], __fmul2_rn(b, make_float2(-sn[j].x, -sn[j].y)));
              x[j + 2] = __ffma2_rn(b, c[j], __fmul2_rn(a, sn[j]));
            }
          }
        }
        if (mine && live[t]) {
          store4(dst + ca, x[0], x[1]);
          store4(dst + cb, x[2], x[3]);
        }
        dst += dh * kD;
      }
    }
  }
}

template <typename T>
static void launch_norm_rope(const okv_norm_rope& p, int tokens, int row_ctas, cudaStream_t s) {
  NormRopeArgs a{p};
  const dim3 grid((unsigned)((p.num_tokens + tokens - 1) / tokens), (unsigned)row_ctas);
  if (p.interleaved) norm_rope_kernel<T, true><<<grid, kNrThreads, 0, s>>>(a, tokens);
  else norm_rope_kernel<T, false><<<grid, kNrThreads, 0, s>>>(a, tokens);
}

}  // namespace
}  // namespace okv

using namespace okv;

extern "C" okv_status okv_qk_norm_rope(const okv_norm_rope* args, void* stream) {
  if (args == nullptr) return fail(OKV_ERR_INVALID_ARG, "args is NULL");
  const okv_norm_rope& p = *args;
  if (p.head_dim != kD) return fail(OKV_ERR_UNSUPPORTED, "only head_dim = 128 is built (got %d)", p.head_dim);
  if (p.num_tokens < 0) return fail(OKV_ERR_INVALID_ARG, "num_tokens must be >= 0");
  if (p.num_q_heads < 1 || p.num_kv_heads < 1 || p.num_q_heads > 65535 || p.num_kv_heads > 65535)
    return fail(OKV_ERR_INVALID_ARG, "num_q_heads and num_kv_heads must be in [1, 65535]");
  if (p.rot_dim < 0 || p.rot_dim > kD || p.rot_dim % 16 != 0)
    return fail(OKV_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16 in [0, 128] (got %d)", p.rot_dim);
  if (p.in_type != OKV_TYPE_BF16 && p.in_type != OKV_TYPE_FP16 && p.in_type != OKV_TYPE_FP32)
    return fail(OKV_ERR_UNSUPPORTED, "in_type must be OKV_TYPE_BF16, OKV_TYPE_FP16 or OKV_TYPE_FP32 (got %d)", p.in_type);
  if (!(p.eps >= 0.f) || !(p.eps <= 1.f)) return fail(OKV_ERR_INVALID_ARG, "eps must be in [0, 1]");
  if (!(p.rope_scale > 0.f) || !(p.rope_scale < 1e6f)) return fail(OKV_ERR_INVALID_ARG, "rope_scale must be positive");
  if ((p.v == nullptr) != (p.v_out == nullptr)) return fail(OKV_ERR_INVALID_ARG, "pass both v and v_out, or neither");
  if (p.num_tokens == 0) return OKV_OK;
  if (!p.q || !p.k || !p.q_out || !p.k_out || !p.positions)
    return fail(OKV_ERR_INVALID_ARG, "q, k, q_out, k_out and positions must be non-NULL");
  if (p.rot_dim > 0 && !p.inv_freq) return fail(OKV_ERR_INVALID_ARG, "inv_freq must be non-NULL when rot_dim > 0");
  if (((uintptr_t)p.positions | (uintptr_t)p.inv_freq | (uintptr_t)p.q_weight | (uintptr_t)p.k_weight) % 4)
    return fail(OKV_ERR_INVALID_ARG, "positions, inv_freq and the weights must be 4-byte aligned");
  const int size = p.in_type == OKV_TYPE_FP32 ? 4 : 2;
  const void* in[3] = {p.q, p.k, p.v};
  const void* out[3] = {p.q_out, p.k_out, p.v_out};
  const int64_t ts[3] = {p.q_token_stride, p.k_token_stride, p.v_token_stride};
  const int64_t hs[3] = {p.q_head_stride, p.k_head_stride, p.v_head_stride};
  for (int i = 0; i < (p.v != nullptr ? 3 : 2); ++i) {
    if ((uintptr_t)in[i] % 16 || (uintptr_t)out[i] % 16 || (ts[i] * size) % 16 || (hs[i] * size) % 16)
      return fail(OKV_ERR_INVALID_ARG, "rows of q, k and v must start on 16-byte boundaries (addresses and strides)");
    if (ts[i] < 0 || hs[i] < 0) return fail(OKV_ERR_INVALID_ARG, "strides must be >= 0");
  }
  // Tokens and rows per CTA.  Long calls: 16 tokens and every row, so that a
  // token's angles are computed once (8192 tokens of 48 heads: 40.6 us; 16 rows
  // per CTA 41.1).  Short ones (fewer than two such CTAs per SM): 16 rows per
  // CTA, each half-warp one row, and as many tokens as leave four CTAs per SM
  // (64 tokens of 48 heads: 1 token 2.9 us, 4 tokens 3.7; every row 4.3.  1021
  // tokens of 80 rows: 8 tokens 11.1 us, 1 token 19.1; every row 13.2 or more).
  const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
  const int rows = p.num_q_heads + p.num_kv_heads * (p.v != nullptr ? 2 : 1);
  int tokens = kNrMaxTokens, row_ctas = 1;
  if (p.num_tokens < 2 * kNrMaxTokens * sms) {
    row_ctas = (rows + kNrHalves - 1) / kNrHalves;
    tokens = std::max(1, std::min(kNrMaxTokens, (int)((long long)p.num_tokens * row_ctas / (4 * sms))));
  }
  const cudaStream_t s = (cudaStream_t)stream;
  if (p.in_type == OKV_TYPE_BF16) launch_norm_rope<__nv_bfloat16>(p, tokens, row_ctas, s);
  else if (p.in_type == OKV_TYPE_FP16) launch_norm_rope<__half>(p, tokens, row_ctas, s);
  else launch_norm_rope<float>(p, tokens, row_ctas, s);
  return check_launch("norm and rotation");
}
