// Decode attention over the paged INT2 or INT4 cache: query rotation, split-K
// attention with online softmax (decode_heads.cuh; here its CUDA-core form for
// other KV head counts), and the split combine with the value un-rotation.
#include "append_warp.cuh"
#include "decode_heads.cuh"
#include "okv_common.cuh"
#include "okv_internal.h"

namespace okv {

// ---------------------------------------------------------------------------
// Kernel 1: q~ = q R_K for one (b, query head) per CTA: warp w holds rows
// 16w..16w+15 of U_K (lane l columns 4l..4l+3, all loads in flight
// together), the eight warps' partial sums meet in shared memory and warp 0
// runs the butterfly.  CTA 0 also writes the cost prefix.
// Also emits the query in the two forms the split-K kernel consumes:
// signed 8-bit limbs in MMA-fragment order and fp16 hi/lo halves.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
static_assert(kPrepThreads == kAppThreads, "the fused step kernel runs append tiles and query rotations alike");

__device__ __forceinline__ void qrot_cta(const DecodeArgs& a, int cta) {
  __shared__ float red[8][kD];
  const int b = cta / a.hq, head = cta % a.hq;
  const int hk = head / a.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float* U = a.u_k + (size_t)hk * kD * kD;
  float4 u[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) u[r] = __ldg(reinterpret_cast<const float4*>(U + (size_t)(16 * warp + r) * kD) + lane);
  const float xv = __bfloat162float(a.q[((size_t)b * a.hq + head) * kD + 16 * warp + (lane & 15)]);
  if (cta == 0) {
    // cost prefix: thread i sums its chunk of consecutive entries, then a
    // block-wide exclusive scan (warp shuffles, then the eight warp totals)
    __shared__ int warp_tot[kPrepThreads / 32];
    const int per = (a.batch + kPrepThreads - 1) / kPrepThreads;
    const int lo = threadIdx.x * per, hi = min(a.batch, lo + per);
    int own = 0;
    for (int i = lo; i < hi; ++i) own += unit_shape(clamp_len(a.context_lens, i, a.mbps, a.status, true), a.nsink).cost;
    int inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += v;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPrepThreads / 32; ++w) {
      before += w < warp ? warp_tot[w] : 0;
      total += warp_tot[w];
    }
    int run = before + inc - own;
    for (int i = lo; i < hi; ++i) {
      a.prefix[i] = run;
      run += unit_shape(clamp_len(a.context_lens, i, a.mbps, a.status, false), a.nsink).cost;
    }
    if (threadIdx.x == 0) a.prefix[a.batch] = total;
  }
  {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float x = __shfl_sync(0xffffffffu, xv, r);
      acc.x = fmaf(x, u[r].x, acc.x);
      acc.y = fmaf(x, u[r].y, acc.y);
      acc.z = fmaf(x, u[r].z, acc.z);
      acc.w = fmaf(x, u[r].w, acc.w);
    }
    *reinterpret_cast<float4*>(&red[warp][4 * lane]) = acc;
  }
  __syncthreads();
  if (warp == 0) {
    float y[4];
#pragma unroll
    for (int aa = 0; aa < 4; ++aa) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += red[w][lane + 32 * aa];
      y[aa] = s;
    }
    wht128_warp(y, lane);
#pragma unroll
    for (int aa = 0; aa < 4; ++aa) y[aa] *= kInvSqrtD;
    const int r = rev5(lane);
    const size_t bh = (size_t)b * a.hq + head;
    *reinterpret_cast<float4*>(a.qrot + bh * kD + 4 * r) = make_float4(y[0], y[2], y[1], y[3]);
    // Integer limbs for the tensor-core score tiles: Q = rint(q~/sigma) in
    // [-32000, 32000] = 256*hi + lo with hi, lo signed 8-bit.  Bytes are stored
    // in MMA-fragment order, so that a lane of quad t reads its 32 bytes in one
    // go; the order follows the K-columns each score MMA gives a lane (code
    // byte b = c / 4 holds channel c in field f = c % 4):
    //   ng = 1: one MMA per field f; quad t holds bytes 8t .. 8t + 7:
    //           c = 32t + 16h + 4i + f goes to 32t + 8f + 4h + i;
    //   ng = 2: one MMA per (group k, field pair p); quad t holds bytes
    //           16k + 4t .. + 3 in fields 2p (K-columns 4t..) and 2p + 1
    //           (16 + 4t..): c = 4 (16k + 4t + i) + 2p + h goes to
    //           32t + 16k + 8p + 4h + i;
    //   ng = 4: one MMA per group k; quad t holds field t of the group's
    //           bytes 8k .. 8k + 7: c = 4 (8k + j) + t goes to 32t + 8k + j.
    // 4-bit codes: score MMA s takes words 4 s + t of the row, low halves of
    // the four bytes at K-columns 4t.., high halves at 16 + 4t..: c = 32 s + 8 t
    // + 2 i + h goes to 32 t + 8 s + 4 h + i, for every group size.
    const float zc[4] = {y[0], y[2], y[1], y[3]};  // rotated channels 4r + e
    float amax = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
    amax = warp_max(amax);
    const float own = (y[0] + y[1]) + (y[2] + y[3]);
    const float sum = warp_sum(own);
    const float sigma = amax > 0.f ? amax / 32000.f : 1.f;
    const float inv = amax > 0.f ? 32000.f / amax : 0.f;
    int8_t* lim = a.qlimb + bh * 2 * kD;
    __half* qw = a.qwin + bh * 2 * kD;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = 4 * r + e;
      const float x = zc[e] * inv;
      const int q = max(-32000, min(32000, __float2int_rn(x)));
      const int hi = ((q + 32896) >> 8) - 128;
      const int lo = q - 256 * hi;
      const int cb = c >> 2, f = c & 3;
      const int pos = a.bits == 4 ? ((c >> 3) & 3) * 32 + (c >> 5) * 8 + (c & 1) * 4 + ((c >> 1) & 3)
                      : a.ng == 1 ? (c >> 5) * 32 + f * 8 + ((c >> 4) & 1) * 4 + ((c >> 2) & 3)
                      : a.ng == 2 ? ((cb >> 2) & 3) * 32 + (cb >> 4) * 16 + (f >> 1) * 8 + (f & 1) * 4 + (cb & 3)
                                  : f * 32 + cb;
      lim[pos] = (int8_t)hi;
      lim[kD + pos] = (int8_t)lo;
      const __half hx = __float2half_rn(x);
      qw[c] = hx;
      qw[kD + c] = __float2half_rn(x - __half2float(hx));
    }
    // per-group sums of q~ (a lane's four channels 4r .. 4r + 3 share a group)
    float gsum[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.ng > 1) {
      const int my = (4 * r) / (kD / a.ng);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < a.ng) gsum[k] = warp_sum(k == my ? own : 0.f);
    }
    if (lane == 0) {
      float4 qs4 = make_float4(sigma * (kInvSqrtD * kLog2e), sum * (kInvSqrtD * kLog2e), sigma, sum);
      *reinterpret_cast<float4*>(a.qscale + bh * kQsStride) = qs4;
      *reinterpret_cast<float4*>(a.qscale + bh * kQsStride + 4) =
          make_float4(gsum[0] * (kInvSqrtD * kLog2e), gsum[1] * (kInvSqrtD * kLog2e), gsum[2] * (kInvSqrtD * kLog2e),
                      gsum[3] * (kInvSqrtD * kLog2e));
    }
  }
}

__global__ void __launch_bounds__(kPrepThreads) qrot_kernel(DecodeArgs a) {
  grid_dep_launch();  // the split-K kernel may start its partition and first copies now
  qrot_cta(a, blockIdx.x);
}

// One launch for the start of a decode step: CTAs [0, n_app) append the
// step's new tokens (one 8-token tile of one (KV head, K|V) each), the rest
// rotate the queries.  The two halves touch disjoint data.
__global__ void __launch_bounds__(kPrepThreads) step_prep_kernel(AppendArgs aa, int T, int n_tiles, DecodeArgs a) {
  grid_dep_launch();
  const int n_app = n_tiles * aa.hkv * 2;
  const int x = blockIdx.x;
  if (x < n_app) {
    append_tile<false>(aa, T, x % n_tiles, (x / n_tiles) % aa.hkv, x / (n_tiles * aa.hkv));
  } else {
    qrot_cta(a, x - n_app);
  }
}

// ---------------------------------------------------------------------------
// Kernel 2 (SIMT fallback, for head groupings the tensor-core kernel does not
// cover): 4 warps per CTA; a warp takes whole 16-token chunks (an INT2 block,
// or 16 window rows) of one KV head and keeps its own online-softmax state;
// warps merge through shared memory.  Lane l scores token l/2 over channels
// 64*(l&1)..+63 and accumulates output channels 4l..4l+3.
// ---------------------------------------------------------------------------
constexpr int kDecWarps = 4;

template <int G>
struct WarpState {
  float m[G], l[G], o[G][4];
};

// kWindow: fp16 rows of positions first_row + t of krow0 / vrow0: the window
// ring (kRing, row = position % W) or the sink rows (row = position);
// otherwise the INT2 block at blockp.
template <int G, int BITS, bool kWindow, bool kRing = true>
__device__ __forceinline__ void simt_chunk(const DecodeArgs& a, const float* qs /*smem [G][128]*/,
                                           const uint8_t* blockp, const __half* krow0,
                                           const __half* vrow0, int win_first_row, int ntok,
                                           WarpState<G>& st, int lane) {
  const int tt = lane >> 1, half = lane & 1;
  const bool valid = tt < ntok;
  float sc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) sc[g] = 0.f;
  if (valid) {
    if constexpr (!kWindow && BITS == 4) {
#pragma unroll
      for (int wi = 0; wi < 8; ++wi) {
        // word 8 half + wi: channels 64 half + 8 wi .. + 7, group (8 half + wi) ng / 16
        const uint32_t w = *reinterpret_cast<const uint32_t*>(blockp + k4_code_offset(tt, 32 * half + 4 * wi));
        const uint32_t smk =
            *reinterpret_cast<const uint32_t*>(blockp + sm_offset(a.ng, 0, tt, (8 * half + wi) * a.ng / 16, BITS));
        const float s = __half2float(__ushort_as_half((unsigned short)(smk & 0xffff)));
        const float m = __half2float(__ushort_as_half((unsigned short)(smk >> 16)));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = fmaf(s, (float)((w >> (4 * j)) & 15u), m);
#pragma unroll
          for (int g = 0; g < G; ++g) sc[g] = fmaf(qs[g * kD + 64 * half + 8 * wi + j], x, sc[g]);
        }
      }
    } else if constexpr (!kWindow) {
      const uint4 w = *reinterpret_cast<const uint4*>(blockp + kKcOff + tt * 32 + 16 * half);
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int wi = 0; wi < 4; ++wi) {
        // channels 64 half + 16 wi .. + 15: group (4 half + wi) ng / 8
        const uint32_t smk =
            *reinterpret_cast<const uint32_t*>(blockp + sm_offset(a.ng, 0, tt, (4 * half + wi) * a.ng / 8, BITS));
        const float s = __half2float(__ushort_as_half((unsigned short)(smk & 0xffff)));
        const float m = __half2float(__ushort_as_half((unsigned short)(smk >> 16)));
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int c = 64 * half + 16 * wi + j;
          const float x = fmaf(s, (float)((words[wi] >> (2 * j)) & 3u), m);
#pragma unroll
          for (int g = 0; g < G; ++g) sc[g] = fmaf(qs[g * kD + c], x, sc[g]);
        }
      }
    } else {
      const int row = kRing ? (win_first_row + tt) % kWin : win_first_row + tt;
      const __half* kr = krow0 + (size_t)row * kD + 64 * half;
#pragma unroll 4
      for (int c8 = 0; c8 < 8; ++c8) {
        const uint4 w = *reinterpret_cast<const uint4*>(kr + 8 * c8);
        const __half2* hp = reinterpret_cast<const __half2*>(&w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(hp[j]);
          const int c = 64 * half + 8 * c8 + 2 * j;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            sc[g] = fmaf(qs[g * kD + c], f.x, sc[g]);
            sc[g] = fmaf(qs[g * kD + c + 1], f.y, sc[g]);
          }
        }
      }
    }
  }
  float p[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float v = sc[g] + __shfl_xor_sync(0xffffffffu, sc[g], 1);
    v = valid ? v * (kInvSqrtD * kLog2e) : -INFINITY;
    const float cmax = warp_max(v);
    const float mnew = fmaxf(st.m[g], cmax);
    const float alpha = (st.m[g] == -INFINITY) ? 0.f : exp2f(st.m[g] - mnew);
    p[g] = valid ? exp2f(v - mnew) : 0.f;
    const float psum = warp_sum(half ? 0.f : p[g]);
    st.l[g] = st.l[g] * alpha + psum;
    st.m[g] = mnew;
#pragma unroll
    for (int j = 0; j < 4; ++j) st.o[g][j] *= alpha;
  }
  // P V: lane owns channels 4*lane .. 4*lane+3
  for (int t = 0; t < ntok; ++t) {
    float x[4];
    if constexpr (!kWindow) {
      uint32_t byte;  // the codes of channels 4 lane .. + 3: one byte, or two
      if constexpr (BITS == 4)
        byte = (uint32_t)blockp[v4_code_offset(t, 2 * lane)] | ((uint32_t)blockp[v4_code_offset(t, 2 * lane + 1)] << 8);
      else byte = blockp[v_code_offset(t, lane)];
      const uint32_t smv = *reinterpret_cast<const uint32_t*>(blockp + sm_offset(a.ng, 1, t, lane * a.ng / 32, BITS));
      const float s = __half2float(__ushort_as_half((unsigned short)(smv & 0xffff)));
      const float m = __half2float(__ushort_as_half((unsigned short)(smv >> 16)));
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = fmaf(s, (float)((byte >> (BITS * j)) & ((1u << BITS) - 1u)), m);
    } else {
      const int row = kRing ? (win_first_row + t) % kWin : win_first_row + t;
      const uint2 w = *reinterpret_cast<const uint2*>(vrow0 + (size_t)row * kD + 4 * lane);
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
      x[0] = f0.x;
      x[1] = f0.y;
      x[2] = f1.x;
      x[3] = f1.y;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float pt = __shfl_sync(0xffffffffu, p[g], 2 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[g][j] = fmaf(pt, x[j], st.o[g][j]);
    }
  }
}

template <int G, int BITS>
__global__ void __launch_bounds__(kDecWarps * 32) decode_simt_kernel(DecodeArgs a) {
  extern __shared__ float smem[];
  float* qs = smem;                               // [G][128]
  float* mo = qs + G * kD;                        // [warps][G][128]
  float* ml = mo + kDecWarps * G * kD;            // [warps][G][2]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long total = a.prefix[a.batch];
  if (total == 0) return;
  const int nc = working_ctas(a, total);
  const int c = blockIdx.x;
  if (c >= nc) return;
  const long long start = (long long)c * total / nc;
  const long long end = (long long)(c + 1) * total / nc;
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.prefix[mid] <= start) lo = mid; else hi = mid - 1;
  }
  for (int b = lo; b < a.batch && a.prefix[b] < end; ++b) {
    const UnitShape us = unit_shape(clamp_len(a.context_lens, b, a.mbps, a.status, false), a.nsink);
    if (us.cost == 0) continue;
    const int slot = a.seq_slot[b];
    const bool slot_ok = slot >= 0 && slot < a.num_slots;
    const long long pu = a.prefix[b];
    const int l0 = (int)(max(start, pu) - pu), l1 = (int)(min(end, pu + us.cost) - pu);
    for (int hk = 0; hk < a.hkv; ++hk) {
      __syncthreads();
      for (int i = threadIdx.x; i < G * kD; i += blockDim.x)
        qs[i] = a.qrot[((size_t)b * a.hq + hk * G) * kD + i];
      __syncthreads();
      WarpState<G> st;
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
        st.m[gg] = -INFINITY;
        st.l[gg] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) st.o[gg][j] = 0.f;
      }
      if (slot_ok) {
        {
          const __half* kbase = a.ring + (((size_t)slot * a.hkv + hk) * 2 + 0) * kWin * kD;
          const __half* vbase = a.ring + (((size_t)slot * a.hkv + hk) * 2 + 1) * kWin * kD;
          const __half* ksink = a.sink + (((size_t)slot * a.hkv + hk) * 2 + 0) * a.nsink * kD;
          const __half* vsink = a.sink + (((size_t)slot * a.hkv + hk) * 2 + 1) * a.nsink * kD;
          const int ci0 = (l0 + kWinCost - 1) / kWinCost;
          const int ci1 = min(us.n_wchunk + us.n_schunk, (l1 + kWinCost - 1) / kWinCost);
          for (int ci = ci0 + warp; ci < ci1; ci += kDecWarps) {
            if (ci < us.n_wchunk) {  // window positions win_first + 16 ci .. at ring rows pos % W
              const int ntok = min(kBlock, us.n_win - ci * kBlock);
              simt_chunk<G, BITS, true>(a, qs, nullptr, kbase, vbase, us.win_first + ci * kBlock, ntok, st, lane);
            } else {  // sink positions 16 (ci - n_wchunk) .. at sink rows pos
              const int f = (ci - us.n_wchunk) * kBlock;
              simt_chunk<G, BITS, true, false>(a, qs, nullptr, ksink, vsink, f, min(kBlock, us.n_sink - f), st, lane);
            }
          }
        }
        const int p0 = max(l0, us.win_cost) - us.win_cost;
        const int p1 = l1 - us.win_cost;
        for (int pi = p0 + warp; pi < p1; pi += kDecWarps) {
          const int blk = a.block_table[(size_t)slot * a.mbps + (a.nsink >> 4) + pi];
          if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) raise_flag(a.status, OKV_DEV_BAD_BLOCK);
            continue;
          }
          const uint8_t* bp = a.pages + ((size_t)blk * a.hkv + hk) * block_head_bytes(a.ng, BITS);
          const int ntok = min(kBlock, us.n_int2 - pi * kBlock);
          simt_chunk<G, BITS, false>(a, qs, bp, nullptr, nullptr, 0, ntok, st, lane);
        }
      } else if (lane == 0 && warp == 0) {
        raise_flag(a.status, OKV_DEV_BAD_SLOT);
      }
#pragma unroll
      for (int gg = 0; gg < G; ++gg) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mo[(warp * G + gg) * kD + 4 * lane + j] = st.o[gg][j];
        if (lane == 0) {
          ml[(warp * G + gg) * 2 + 0] = merge_max(st.m[gg], st.l[gg]);
          ml[(warp * G + gg) * 2 + 1] = st.l[gg];
        }
      }
      __syncthreads();
      float* dst = a.part + ((size_t)(c + b) * a.hq + (size_t)hk * G) * kPartStride;
      for (int i = threadIdx.x; i < G * kD; i += blockDim.x) {
        const int gg = i / kD, ch = i % kD;
        float mx = -INFINITY;
        for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, ml[(w * G + gg) * 2]);
        float o = 0.f, l = 0.f;
        if (mx != -INFINITY) {
          for (int w = 0; w < kDecWarps; ++w) {
            const float mw = ml[(w * G + gg) * 2];
            const float sc = (mw == -INFINITY) ? 0.f : exp2f(mw - mx);
            o = fmaf(mo[(w * G + gg) * kD + ch], sc, o);
            l = fmaf(ml[(w * G + gg) * 2 + 1], sc, l);
          }
        }
        dst[gg * kPartStride + ch] = o;
        if (ch == 0) {
          dst[gg * kPartStride + 128] = mx;
          dst[gg * kPartStride + 129] = l;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Kernel 3: merge the splits of one (b, query head), normalise, undo the
// value rotation (un-permute, Hadamard, U_V^T) and write the fp32 output.
// One CTA per (b, query head) so that enough loads are in flight: before any
// reduction a CTA starts async copies of U_V into shared memory and loads the
// o' rows of the first 128 splits into registers (warp w: splits w, w+8, ...;
// lane l: channels 4l..4l+3).
// ---------------------------------------------------------------------------
constexpr int kCombThreads = 256;
constexpr int kCombWarps = kCombThreads / 32;
constexpr int kCombPre = 16;      // o' rows per warp loaded ahead of the weights
constexpr int kMaxSplits = 1024;  // >= split-K CTAs (at most 4 per SM)
constexpr size_t kCombSmem = (size_t)(kD * kD + kMaxSplits + kCombWarps * kD + kD + 2 * kCombWarps) * sizeof(float);

__device__ __forceinline__ void cp_async16(void* smem_dst, const void* gsrc) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(smem_dst)), "l"(gsrc) : "memory");
}

__global__ void __launch_bounds__(kCombThreads) combine_kernel(DecodeArgs a) {
  extern __shared__ __align__(16) float csm[];
  float* us_ = csm;                        // U_V [128][128]
  float* ml = us_ + kD * kD;               // [kMaxSplits] split maxima, then weights 2^(m_c - M)
  float* wsum = ml + kMaxSplits;           // [warps][128] per-warp partial sums
  float* xs = wsum + kCombWarps * kD;      // [128] merged, normalised, un-rotated o
  float* redm = xs + kD;                   // [warps]
  float* redl = redm + kCombWarps;         // [warps]
  const int b = blockIdx.x / a.hq, head = blockIdx.x % a.hq;
  const int hk = head / a.g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  {
    const float* U = a.u_v + (size_t)hk * kD * kD;
#pragma unroll
    for (int k = 0; k < kD * kD / 4 / kCombThreads; ++k) {
      const int i = tid + kCombThreads * k;
      cp_async16(us_ + 4 * i, U + 4 * i);
    }
    cp_async_commit();
  }
  grid_dep_wait();  // the split partials (and the cost prefix) are read from here on
  const UnitShape sh = unit_shape(clamp_len(a.context_lens, b, a.mbps, a.status, false), a.nsink);
  const long long total = a.prefix[a.batch];
  const size_t outp = ((size_t)b * a.hq + head) * kD;
  auto put = [&](int ch, float x) {
    if (a.out_bf16) ((__nv_bfloat16*)a.out)[outp + ch] = __float2bfloat16_rn(x);
    else ((float*)a.out)[outp + ch] = x;
  };
  if (sh.cost == 0 || total == 0) {
    if (tid < kD) put(tid, 0.f);
    cp_async_wait_all();
    return;
  }
  const long long pu = a.prefix[b];
  const int nc = working_ctas(a, total);
  const int c0 = cta_of(pu, total, nc);
  const int ns = cta_of(pu + sh.cost - 1, total, nc) - c0 + 1;  // splits of this entry
  const size_t split_stride = (size_t)a.hq * kPartStride;
  const float* base = a.part + ((size_t)(c0 + b) * a.hq + head) * kPartStride;
  // o' rows of the first kCombPre splits of this warp
  float4 pre[kCombPre];
#pragma unroll
  for (int j = 0; j < kCombPre; ++j) {
    const int c = warp + kCombWarps * j;
    pre[j] = c < ns ? *reinterpret_cast<const float4*>(base + (size_t)c * split_stride + 4 * lane)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // split maxima and sums, and the global maximum
  float mx = -INFINITY;
  for (int c = tid; c < ns; c += kCombThreads) {
    const float2 m2 = *reinterpret_cast<const float2*>(base + (size_t)c * split_stride + 128);
    ml[c] = m2.x;
    wsum[c] = m2.y;  // the sums borrow the partial-sum buffer until the weights are known
    mx = fmaxf(mx, m2.x);
  }
  mx = warp_max(mx);
  if (lane == 0) redm[warp] = mx;
  __syncthreads();
  mx = redm[0];
#pragma unroll
  for (int w = 1; w < kCombWarps; ++w) mx = fmaxf(mx, redm[w]);
  float l = 0.f;
  for (int c = tid; c < ns; c += kCombThreads) {
    const float m = ml[c];
    const float w = (mx == -INFINITY || m == -INFINITY) ? 0.f : exp2f(m - mx);
    ml[c] = w;
    l = fmaf(wsum[c], w, l);
  }
  l = warp_sum(l);
  if (lane == 0) redl[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kCombWarps; ++w) l += redl[w];
  const float inv_l = l == 0.f ? 0.f : 1.f / l;
  // weighted sum of the splits
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < kCombPre; ++j) {
    const int c = warp + kCombWarps * j;
    const float w = c < ns ? ml[c] : 0.f;
    acc.x = fmaf(pre[j].x, w, acc.x);
    acc.y = fmaf(pre[j].y, w, acc.y);
    acc.z = fmaf(pre[j].z, w, acc.z);
    acc.w = fmaf(pre[j].w, w, acc.w);
  }
  for (int c0w = warp + kCombWarps * kCombPre; c0w < ns; c0w += kCombWarps * kCombPre) {
#pragma unroll
    for (int j = 0; j < kCombPre; ++j) {
      const int c = c0w + kCombWarps * j;
      pre[j] = c < ns ? *reinterpret_cast<const float4*>(base + (size_t)c * split_stride + 4 * lane)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < kCombPre; ++j) {
      const int c = c0w + kCombWarps * j;
      const float w = c < ns ? ml[c] : 0.f;
      acc.x = fmaf(pre[j].x, w, acc.x);
      acc.y = fmaf(pre[j].y, w, acc.y);
      acc.z = fmaf(pre[j].z, w, acc.z);
      acc.w = fmaf(pre[j].w, w, acc.w);
    }
  }
  __syncthreads();  // every thread is done with the sums borrowed in wsum
  *reinterpret_cast<float4*>(&wsum[warp * kD + 4 * lane]) = acc;
  cp_async_wait_all();
  __syncthreads();
  // un-permute + Hadamard in warp 0: lane holds pre-permutation channels
  // l + 32a = rotated channels 4*rev5(l) + rev2(a)
  if (warp == 0) {
    const int r = rev5(lane);
    float y[4];
#pragma unroll
    for (int aa = 0; aa < 4; ++aa) {
      const int ch = 4 * r + rev2(aa);
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kCombWarps; ++w) o += wsum[w * kD + ch];
      y[aa] = o * inv_l;
    }
    wht128_warp(y, lane);
#pragma unroll
    for (int aa = 0; aa < 4; ++aa) xs[lane + 32 * aa] = y[aa] * kInvSqrtD;
  }
  __syncthreads();
  // o_c = sum_i x_i U_V[c][i]: warp w, channels 16w..16w+15; lane l inputs 4l..4l+3
  const float4 xv = *reinterpret_cast<const float4*>(&xs[4 * lane]);
  float part[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float4 u = *reinterpret_cast<const float4*>(us_ + (16 * warp + r) * kD + 4 * lane);
    part[r] = fmaf(xv.x, u.x, fmaf(xv.y, u.y, fmaf(xv.z, u.z, xv.w * u.w)));
  }
  // transpose-reduce: after the four halving steps lane l holds the partial of
  // channel 16w + (l & 15) summed over 16 lanes; one more step finishes it
#pragma unroll
  for (int step = 8; step >= 1; step >>= 1) {
    const bool upper = (lane & step) != 0;
#pragma unroll
    for (int r = 0; r < step; ++r) {
      const float send = upper ? part[r] : part[r + step];
      const float keep = upper ? part[r + step] : part[r];
      part[r] = keep + __shfl_xor_sync(0xffffffffu, send, step);
    }
  }
  const float o = part[0] + __shfl_xor_sync(0xffffffffu, part[0], 16);
  if (lane < 16) put(16 * warp + lane, o);
}

template <int G, int BITS>
static okv_status launch_decode_simt(const DecodeArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)(G * kD + kDecWarps * G * kD + kDecWarps * G * 2) * sizeof(float);
  static std::atomic<uint32_t> attr_set{0};
  cudaError_t e = set_smem_limit_once((const void*)decode_simt_kernel<G, BITS>, (int)smem, attr_set);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "decode smem attribute: %s", cudaGetErrorString(e));
  decode_simt_kernel<G, BITS><<<a.nc, kDecWarps * 32, smem, s>>>(a);
  return check_launch("decode");
}


bool decode_uses_tensor_cores(int g, int hkv, int ng) {
  const bool hkv_ok = hkv == 1 || hkv == 2 || hkv == 4 || hkv == 8;
  return hkv_ok && (ng == 1 || ng == 2 || ng == 4) && (g == 1 || g == 2 || g == 4 || g == 8 || g == 16);
}

// split-K cost ranges for a device of `sms` SMs: two CTAs per SM for the
// tensor-core kernel (one at G = 8 with one group per vector, whose CTA holds
// both n-tiles), with a range split over two (G = 8 grouped) or four (G = 16)
// CTAs of four query heads; four CTAs per SM for the CUDA-core kernel
int decode_ranges(int sms, int g, int hkv, int ng) {
  if (!decode_uses_tensor_cores(g, hkv, ng)) return 4 * sms;
  if (g <= 4) return 2 * sms;
  if (g == 8) return sms;
  return sms / 2;  // g = 16
}

static DecodeArgs make_decode_args(const okv_cache_desc* d, const void* q, int B, const int32_t* seq_slot,
                                   const int32_t* block_table, const int32_t* context_lens, void* out, void* ws,
                                   const DecodePlan& plan) {
  DecodeArgs a;
  a.q = (const __nv_bfloat16*)q;
  a.seq_slot = seq_slot;
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.u_k = d->u_k;
  a.u_v = d->u_v;
  a.pages = (const uint8_t*)d->pages;
  a.ring = (const __half*)d->window_ring;
  a.sink = (const __half*)d->sink_rows;
  a.nsink = d->num_sink;
  a.out = out;
  a.status = d->status_word;
  uint8_t* w = (uint8_t*)ws;
  a.qrot = (float*)(w + plan.qrot_off);
  a.qlimb = (int8_t*)(w + plan.qlimb_off);
  a.qscale = (float*)(w + plan.qscale_off);
  a.qwin = (__half*)(w + plan.qwin_off);
  a.prefix = (int32_t*)(w + plan.prefix_off);
  a.part = (float*)(w + plan.part_off);
  a.batch = B;
  a.hq = d->num_q_heads;
  a.hkv = d->num_kv_heads;
  a.g = plan.g;
  a.nc = plan.num_ctas;
  a.num_blocks = d->num_blocks;
  a.num_slots = d->num_seq_slots;
  a.mbps = d->max_blocks_per_seq;
  a.ng = kD / group_channels(d);
  a.bits = code_bits(d);
  a.out_bf16 = out_bf16(d);
  // grouped layouts at G = 8, and every layout at G = 16: two or four CTAs per
  // cost range, four query heads each
  a.hsplit = a.g == 16 ? 4 : (a.ng > 1 && a.g == 8) ? 2 : 1;
  a.new_slot = a.new_pos = a.slot_lens = nullptr;
  a.new_tokens = 0;
  return a;
}

// split-K attention and the combine, after the queries have been rotated
static okv_status launch_decode_tail(const DecodeArgs& a, int B, cudaStream_t s) {
  okv_status st = OKV_OK;
  cudaEvent_t ev0, ev1;
  take_decode_events(&ev0, &ev1);
  // inside a stream capture the events become external event nodes of the
  // graph, so that each replay records them; outside one they are recorded
  // as usual
  unsigned ev_flags = cudaEventRecordDefault;
  if (ev0 != nullptr) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) return fail(OKV_ERR_CUDA, "cudaStreamIsCapturing failed");
    if (cs == cudaStreamCaptureStatusActive) ev_flags = cudaEventRecordExternal;
  }
  if (ev0 != nullptr && cudaEventRecordWithFlags(ev0, s, ev_flags) != cudaSuccess)
    return fail(OKV_ERR_CUDA, "cudaEventRecord failed");
  // Early (programmatic) launches overlap each kernel's start with its
  // predecessor; they are left out when the split-K kernel is being timed, so
  // that the events bracket it alone.
  const bool early = ev0 == nullptr;
  const bool tc = decode_uses_tensor_cores(a.g, a.hkv, a.ng);
  if (tc && a.bits == 4) {
    st = launch_decode_heads_int4(a, s, early);
  } else if (tc && a.ng == 2) {
    switch (a.g) {
      case 1: st = launch_decode_heads<1, 2>(a, s, early); break;
      case 2: st = launch_decode_heads<2, 2>(a, s, early); break;
      case 4: st = launch_decode_heads<4, 2>(a, s, early); break;
      case 8: st = launch_decode_heads<4, 2, 2>(a, s, early); break;  // G = 8 as two halves
      default: st = launch_decode_heads<4, 2, 4>(a, s, early); break;  // G = 16 as four quarters
    }
  } else if (tc && a.ng == 4) {
    switch (a.g) {
      case 1: st = launch_decode_heads<1, 4>(a, s, early); break;
      case 2: st = launch_decode_heads<2, 4>(a, s, early); break;
      case 4: st = launch_decode_heads<4, 4>(a, s, early); break;
      case 8: st = launch_decode_heads<4, 4, 2>(a, s, early); break;  // G = 8 as two halves
      default: st = launch_decode_heads<4, 4, 4>(a, s, early); break;  // G = 16 as four quarters
    }
  } else if (tc) {
    switch (a.g) {
      case 1: st = launch_decode_heads<1>(a, s, early); break;
      case 2: st = launch_decode_heads<2>(a, s, early); break;
      case 4: st = launch_decode_heads<4>(a, s, early); break;
      case 8: st = launch_decode_heads<8>(a, s, early); break;
      default: st = launch_decode_heads<4, 1, 4>(a, s, early); break;  // G = 16 as four quarters
    }
  } else {
    switch (a.g) {
      case 1: st = a.bits == 4 ? launch_decode_simt<1, 4>(a, s) : launch_decode_simt<1, 2>(a, s); break;
      case 2: st = a.bits == 4 ? launch_decode_simt<2, 4>(a, s) : launch_decode_simt<2, 2>(a, s); break;
      case 4: st = a.bits == 4 ? launch_decode_simt<4, 4>(a, s) : launch_decode_simt<4, 2>(a, s); break;
      case 8: st = a.bits == 4 ? launch_decode_simt<8, 4>(a, s) : launch_decode_simt<8, 2>(a, s); break;
      case 16: st = a.bits == 4 ? launch_decode_simt<16, 4>(a, s) : launch_decode_simt<16, 2>(a, s); break;
      default: return fail(OKV_ERR_UNSUPPORTED, "group size %d (Hq/Hkv) not in {1,2,4,8,16}", a.g);
    }
  }
  if (st != OKV_OK) return st;
  if (ev1 != nullptr && cudaEventRecordWithFlags(ev1, s, ev_flags) != cudaSuccess)
    return fail(OKV_ERR_CUDA, "cudaEventRecord failed");
  static std::atomic<uint32_t> attr_set{0};
  cudaError_t e = set_smem_limit_once((const void*)combine_kernel, (int)kCombSmem, attr_set);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "combine smem attribute: %s", cudaGetErrorString(e));
  e = launch_pdl(combine_kernel, dim3(B * a.hq), dim3(kCombThreads), kCombSmem, s, early && tc, a);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "combine launch: %s", cudaGetErrorString(e));
  return check_launch("combine");
}

okv_status launch_decode(const okv_cache_desc* d, const void* q, int B, const int32_t* seq_slot,
                         const int32_t* block_table, const int32_t* context_lens, void* out,
                         void* ws, const DecodePlan& plan, cudaStream_t s) {
  const DecodeArgs a = make_decode_args(d, q, B, seq_slot, block_table, context_lens, out, ws, plan);
  qrot_kernel<<<B * a.hq, kPrepThreads, 0, s>>>(a);
  const okv_status st = check_launch("query rotation");
  if (st != OKV_OK) return st;
  return launch_decode_tail(a, B, s);
}

okv_status launch_decode_step(const okv_cache_desc* d, const void* k, const void* v, int T, const int32_t* new_slot,
                              const int32_t* new_pos, const int32_t* slot_lens, const void* q, int B,
                              const int32_t* seq_slot, const int32_t* block_table, const int32_t* context_lens,
                              void* out, void* ws, const DecodePlan& plan, cudaStream_t s) {
  DecodeArgs a = make_decode_args(d, q, B, seq_slot, block_table, context_lens, out, ws, plan);
  a.new_slot = new_slot;
  a.new_pos = new_pos;
  a.slot_lens = slot_lens;
  a.new_tokens = T;
  const AppendArgs aa = make_append_args(d, k, v, new_slot, new_pos, block_table, slot_lens, nullptr);
  const int n_tiles = (T + kAppTokens - 1) / kAppTokens;
  const long long ctas = (long long)n_tiles * d->num_kv_heads * 2 + (long long)B * a.hq;
  step_prep_kernel<<<(unsigned)ctas, kPrepThreads, 0, s>>>(aa, T, n_tiles, a);
  const okv_status st = check_launch("decode step (append + query rotation)");
  if (st != OKV_OK) return st;
  return launch_decode_tail(a, B, s);
}

}  // namespace okv
