// Norms of queries and keys for each head with the position rotation in the
// same pass (okv_qk_norm_rope): the step between a model's fused projection
// and this library's append and attention calls.
//
//   y = x / sqrt(mean(x^2) + eps) * w                (128 channels of a head)
//   (a, b) -> (a cos - b sin, b cos + a sin) of the channel pairs inside
//   rot_dim, angle = position * inv_freq
//
// Bound: bytes.  A row (one token's head) is read once and written once; its
// arithmetic is ~25 instructions per 8 channels.  A half-warp takes a row, 8
// consecutive channels (16 bytes of a 16-bit type) per lane, so that a row is
// one coalesced access each way, the sum of squares is four shuffles, and a
// pair's partner sits in another lane of the half-warp (first half with
// second half) or in the lane itself (adjacent pairs).  The angles of a token
// do not depend on the head: a CTA computes the cosines and sines of its
// tokens once, in shared memory, and every half-warp keeps one token's in
// registers while it walks that token's heads.
//
// Rounding: the product position * inv_freq and its reduction to one turn are
// fp64 (in fp32 a position of 10^5 would leave an angle error of 4e-3); the
// sums and products are fp32; each output is rounded once, to bf16, the type
// that the append and the attention take.
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

// 8 consecutive channels as fp32
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(src));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(src) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (std::is_same<T, __half>::value) f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
}

// A CTA takes `tokens` (<= 16) consecutive tokens; half-warp j serves token
// j % tokens and heads j / tokens, + 16 / tokens, ...
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(NormRopeArgs args, int tokens) {
  const okv_norm_rope& p = args.p;
  __shared__ float2 cs[kNrHalves * (kD / 2)];  // [token][pair]: cosine, sine
  const int t0 = blockIdx.x * tokens;
  const int half = p.rot_dim >> 1;
  const int nt = min(tokens, p.num_tokens - t0);
  for (int i = threadIdx.x; i < nt * half; i += kNrThreads) {
    const int t = i / half, j = i - t * half;
    const int pos = p.positions[t0 + t];
    const double angle = (double)pos * (double)p.inv_freq[j];
    const double full = rint(angle * kInvTwoPi);
    const float r = (float)fma(-full, kTwoPiLo, fma(-full, kTwoPi, angle));  // within half a turn of 0
    float s, c;
    sincosf(r, &s, &c);
    cs[t * half + j] = make_float2(c * p.rope_scale, s * p.rope_scale);
  }
  const int sub = threadIdx.x & 15, hw = threadIdx.x >> 4;  // lane in the half-warp, half-warp in the CTA
  const int t = hw % tokens, step = kNrHalves / tokens;
  const bool live = t < nt && p.positions[t0 + min(t, nt - 1)] >= 0;  // a negative position marks a padding row
  const int tok = t0 + t;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const int rows = hq + hkv + (p.v != nullptr ? hkv : 0);
  const float eps = p.eps;
  __syncthreads();
  // this lane's rotation: channel 8 sub + i pairs with another of the row
  float2 rot[8];
  int partner = 0;
  float sign = 0.f;
  const bool turns = 8 * sub < p.rot_dim;
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rot[i] = live && turns ? cs[t * half + 4 * sub + i] : make_float2(1.f, 0.f);
  } else {
    const bool upper = 8 * sub >= half;
    const int j0 = 8 * sub - (upper ? half : 0);
    partner = turns ? (8 * sub + (upper ? -half : half)) >> 3 : sub;
    sign = upper ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) rot[i] = live && turns ? cs[t * half + j0 + i] : make_float2(1.f, 0.f);
  }
  partner |= (threadIdx.x & 16);
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wq[i] = p.q_weight != nullptr ? p.q_weight[8 * sub + i] : 1.f;
    wk[i] = p.k_weight != nullptr ? p.k_weight[8 * sub + i] : 1.f;
  }
  // every lane of the warp runs the same number of rounds (the shuffles are warp-wide)
  const int rounds = (rows + step - 1) / step;
  for (int r = 0; r < rounds; ++r) {
    const int row = r * step + hw / tokens;
    const bool mine = live && row < rows;
    const bool is_q = row < hq, is_k = !is_q && row < hq + hkv;
    const int h = is_q ? row : is_k ? row - hq : row - hq - hkv;
    const void* src = is_q ? p.q : is_k ? p.k : p.v;
    const long long ts = is_q ? p.q_token_stride : is_k ? p.k_token_stride : p.v_token_stride;
    const long long hs = is_q ? p.q_head_stride : is_k ? p.k_head_stride : p.v_head_stride;
    void* out = is_q ? p.q_out : is_k ? p.k_out : p.v_out;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (mine) load8((const T*)src + tok * ts + h * hs + 8 * sub, x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (p.norm != 0 && (is_q || is_k)) {
      const float inv = 1.f / sqrtf(fmaf(ss, 1.f / kD, eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * (is_q ? wq[i] : wk[i]);
    }
    float y[8];
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = fmaf(x[2 * i], rot[i].x, -x[2 * i + 1] * rot[i].y);
        y[2 * i + 1] = fmaf(x[2 * i + 1], rot[i].x, x[2 * i] * rot[i].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_sync(0xffffffffu, x[i], partner);
        y[i] = fmaf(x[i], rot[i].x, sign * other * rot[i].y);
      }
    }
    if (mine) {
      // channels past rot_dim and the values pass as they are (an infinity times sin = 0 would be NaN)
      const bool turned = turns && (is_q || is_k);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = turned ? y[i] : x[i];
      store8((__nv_bfloat16*)out + ((size_t)tok * (is_q ? hq : hkv) + h) * kD + 8 * sub, y);
    }
  }
}

template <typename T>
static void launch_norm_rope(const okv_norm_rope& p, int tokens, cudaStream_t s) {
  NormRopeArgs a{p};
  const unsigned grid = (unsigned)((p.num_tokens + tokens - 1) / tokens);
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
  // Tokens per CTA.  One token per CTA fills the GPU first (a decode step);
  // with enough tokens for four CTAs per SM, four tokens share a CTA.
  const int sms = device_sm_count();
  const int tokens = p.num_tokens >= 16 * (sms > 0 ? sms : 148) ? 4 : 1;
  const cudaStream_t s = (cudaStream_t)stream;
  if (p.in_type == OKV_TYPE_BF16) launch_norm_rope<__nv_bfloat16>(p, tokens, s);
  else if (p.in_type == OKV_TYPE_FP16) launch_norm_rope<__half>(p, tokens, s);
  else launch_norm_rope<float>(p, tokens, s);
  return check_launch("norm and rotation");
}
