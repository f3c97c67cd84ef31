// Chunked-prefill attention over the 4-bit cache with bf16 output, on the
// tcgen05 tensor cores.
//
// bf16 output leaves 2^-8 of a value, so one fp16 operand per factor is
// enough: q~ 2^-e is rounded to fp16 once, keys and values are dequantised
// once, s c + m rounded to fp16 by one half-precision FMA, and the softmax
// weight p 2^11 is rounded to fp16.  Each rounding is 2^-11 of its operand at
// most and independent from key to key.  (fp32 output takes the kernel of
// prefill.cu: two fp16 halves of q~ and of p s against exact codes.)  The
// group's scale and minimum are gone after staging, so the softmax has no
// per-key factor and one kernel body serves every group size.  Values past
// fp16's +-65504 saturate, like the cache's fp16 rows.
//
// A CTA takes its range of the work (P4Split): piece by piece, 256 query rows
// (two tiles of 128, the MMA's M) of one KV head against a run of 128-key chunks:
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread owns a row (TMEM lane);
//   warps 8-11      keys into shared memory, [token][channel] fp16, and values,
//                   [channel][token] fp16, both K-major (13 warps leave 128
//                   registers a thread; 17, with keys and values apart, 96);
//   warp 12         TMEM allocation; one lane issues the MMAs:
//                   S_t = Q_t K^T (M 128, N 128, K 128; Q_t in shared memory)
//                   and O_t += P_t V (P_t in TMEM over the columns of S_t).
// TMEM: S_0, S_1, O_0, O_1, 128 columns each (all 512).  The two tiles keep
// the tensor pipe and the softmax warps busy in turn: while a tile's scores
// become weights, the other tile's MMAs run.
// Per row the softmax goes through its 128 scores once, 32 at a time: maximum,
// weights, sum, and the fp16 weights back into TMEM (columns 16 b .. of the
// batch b, never past scores still to be read).  The running maximum is lazy:
// it moves only when a batch passes it by more than 4 (log2 units); then O_t
// and the chunk's weights written so far are scaled in TMEM.
// Staging costs the fewest instructions where two codes of one word are masked
// out together without moving bytes, which gives channels c and c + 4 of a key
// word, and tokens t and t + 2 of a value word.  So the channels of a key row
// (and of q~, which the rotation writes the same way) lie in the order 0 4 1 5 2
// 6 3 7 within eight, and keys in the order 0 2 1 3 within four, in the score
// columns and in the value tile alike.
// Bound: 128 keys x 256 rows cost 32 MMAs of 64 cycles and 32768 exponentials
// at 16 a cycle, 2048 cycles each; a chunk takes 5250 (1024 tokens over 32K keys,
// 32/8 heads: 640 us, 845 TFLOP/s), so that either unit is 39 % busy, which is
// also what the counters say, and issue slots 45 %: what is left is the latency
// of each tile's chain of scores, softmax and value MMA.  64-channel groups take
// the same time (694 us a call against 688); with 32 channels the staging's
// pairs push the kernel past 128 registers (112 bytes of spills) and a call
// takes 846.  One range of work per SM against one tile
// per CTA (128 of them): 762 against 873 us a call.  Not taken (same call, 762):
// the value MMA of the first 64 keys started while the softmax does the others
// 847 (the issuing warp then waits where the other tile could go on), a warp of
// MMAs per tile 785 (the tiles fall into step), both 785, the next batch's
// scores loaded ahead 768.
#include <type_traits>

#include "okv_common.cuh"
#include "okv_internal.h"
#include "prefill_common.cuh"
#include "umma.cuh"

namespace okv {
namespace {

constexpr int kP4Threads = 32 * 13;
constexpr uint32_t kP4Tile = 32768;           // a 128 x 128 fp16 tile: two K-blocks of 128 rows x 128 B
constexpr uint32_t kP4OffQ = 0;               // Q_0, Q_1
constexpr uint32_t kP4OffK = 2 * kP4Tile;     // two stages
constexpr uint32_t kP4OffV = 4 * kP4Tile;     // two stages
constexpr uint32_t kP4OffMisc = 6 * kP4Tile;
struct P4Misc {
  uint64_t q_full[2], k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], pv_done[2];
  int bad[4][4];               // per chunk mod 4, key warp: a block id was out of range
  int kval[4][kP4Keys];        // then: 1 where the token was staged
  uint32_t tmem_slot;
};
constexpr size_t kP4Smem = 1024 + kP4OffMisc + sizeof(P4Misc);
constexpr uint32_t kP4Idesc = um_idesc(128, false, false);
constexpr float kP4Slack = 4.f;    // log2 units a score may pass the running maximum
constexpr float kP4Offset = 11.f;  // weights are stored as p 2^11: at most 2^15, and full precision 25 bits down

__device__ __forceinline__ float p4_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }

// Codes to values s c + m, two at a time: of a word with the nibbles n0 .. n7,
// the even form takes n0 and n4, the odd form n1 and n5.  The code goes under an
// exponent that makes its unit one mantissa step (1024 + c, or 64 + c for the
// upper nibble), the bias comes off exactly, and the FMA rounds once.
__device__ __forceinline__ uint32_t p4_even(uint32_t x, __half2 s, __half2 m) {
  return h2_bits(__hfma2(__hsub2(bits_h2((x & 0x000F000Fu) | 0x64006400u), bits_h2(0x64006400u)), s, m));
}
__device__ __forceinline__ uint32_t p4_odd(uint32_t x, __half2 s, __half2 m) {
  return h2_bits(__hfma2(__hsub2(bits_h2((x & 0x00F000F0u) | 0x54005400u), bits_h2(0x54005400u)), s, m));
}
__device__ __forceinline__ uint32_t sat_h2(uint32_t x) {  // infinities to the largest finite values
  const __half2 top = bits_h2(0x7BFF7BFFu);
  return h2_bits(__hmin2(__hmax2(bits_h2(x), __hneg2(top)), top));
}

template <int NG>
__global__ void __launch_bounds__(kP4Threads, 1)
    prefill_int4_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ P4Split sp) {
  extern __shared__ unsigned char p4_raw[];
  const uint32_t raw_u32 = smem_u32(p4_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;  // swizzle atoms need 1024-byte alignment
  unsigned char* gb = p4_raw + (base - raw_u32);
  P4Misc& ms = *reinterpret_cast<P4Misc*>(gb + kP4OffMisc);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nrows = a.T * a.g;
  const int32_t* table = a.block_table + (size_t)a.slot * a.mbps;
  grid_dep_launch();  // the un-rotation may start staging U_V

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.q_full[i], 128);
      mbar_init(&ms.k_full[i], 128);
      mbar_init(&ms.k_free[i], 1);
      mbar_init(&ms.v_full[i], 128);
      mbar_init(&ms.v_free[i], 1);
      mbar_init(&ms.s_full[i], 2);  // the MMAs' commit, and the issuing thread (for bad and kval)
      mbar_init(&ms.p_full[i], 128);
      mbar_init(&ms.pv_done[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 12) um_alloc(&ms.tmem_slot, 512);

  // this CTA's pieces, the same for every role
  struct Piece {
    int hk, x;  // KV head, tile of the head
    int c0, n;  // chunks c0 .. c0 + n - 1
    int nt;     // 128-row tiles with any row
    int slot;   // where the rows go: -1 obuf (the whole tile), else the slot of `part`
  };
  const int2 u_begin = sp.start[blockIdx.x], u_end = sp.start[blockIdx.x + 1];
  auto more = [&](int2 u) { return u.x < u_end.x || u.y < u_end.y; };
  auto next_piece = [&](int2 u, Piece& pc) -> int2 {
    pc.hk = u.x / sp.tiles;
    pc.x = u.x - pc.hk * sp.tiles;
    pc.c0 = u.y;
    const bool cut = u.x == u_end.x;
    pc.n = (cut ? u_end.y : prefill_last_pos(a, pc.x) / kP4Keys + 1) - pc.c0;
    pc.nt = pc.x * kP4Rows + 128 < nrows ? 2 : 1;
    pc.slot = pc.c0 > 0 ? 0 : cut ? 1 : -1;
    return cut ? u_end : make_int2(u.x + 1, 0);
  };

  const int tile = (warp >> 2) & 1, quarter = warp & 3;
  const int trow = 32 * quarter + lane;  // row in the tile (TMEM lane) of a softmax thread
  um_fence_before();
  __syncthreads();
  um_fence_after();
  const uint32_t tmem = ms.tmem_slot;
  const uint32_t tS = tmem + 128u * (uint32_t)tile, tO = tmem + 256u + 128u * (uint32_t)tile;

  // key order within a quad: token t sits at row swap_mid(t), row r holds token swap_mid(r)
  auto swap_mid = [](int t) { return (t & ~3) | ((t & 1) << 1) | ((t & 2) >> 1); };
  constexpr int kSm = 2048;  // (scale, min) pairs of the keys; the values' follow 64 NG bytes on

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const uint32_t lb = (uint32_t)(32 * quarter) << 16;
    grid_dep_wait();  // q~ is read from here on (the staging warps read the cache only)
    bool alive = true;
    int done = 0, seen = 0;  // chunks of the pieces before: staged, and those with this tile
    Piece pc;
#pragma unroll 1
    for (int2 u = u_begin; more(u); done += pc.n) {
      u = next_piece(u, pc);
      if (tile >= pc.nt) continue;
      // the thread's row, and its q~ into the Q tile (the MMAs that read the last one are done: pv_done)
      const int r = pc.x * kP4Rows + 128 * tile + trow;
      const bool rok = r < nrows;
      const int rr = rok ? r : nrows - 1;
      const int rtok = rr / a.g, rpos = a.first + rtok;
      const size_t rrow = (size_t)rtok * a.hq + pc.hk * a.g + rr % a.g;
      {
        const uint4* src = reinterpret_cast<const uint4*>(a.qhi + rrow * kD);
        unsigned char* dst = gb + kP4OffQ + (uint32_t)tile * kP4Tile;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          *reinterpret_cast<uint4*>(dst + (j >> 3) * 16384 + um_swz((uint32_t)trow, (uint32_t)(j & 7) * 16u)) = src[j];
        um_fence_proxy_async();
        mbar_arrive(&ms.q_full[tile]);
      }
      const float sc = a.qaux[rrow * kQaux + 4] * (kInvSqrtD * kLog2e);  // score scale, log2 units: 2^e log2(e) / sqrt(d)
      const float2 sc2 = make_float2(sc, sc);
      float m_use = -INFINITY;
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // partial sums of the weights
      for (int i = 0; i < pc.n && alive; ++i) {
        const uint32_t ph = (uint32_t)(seen + i) & 1u;
        alive = __all_sync(0xffffffffu, mbar_wait_bounded(&ms.s_full[tile], ph));
        if (!alive) break;
        um_fence_after();
        const int kb = (done + i) & 3;
        const int lim = min(rpos + 1, a.L) - kP4Keys * (pc.c0 + i);  // columns below it are visible
        const int* bd = ms.bad[kb];
        const bool bad = (bd[0] | bd[1] | bd[2] | bd[3]) != 0;
        // A batch of 32 columns at a time, rolled up: the loops of the three roles
        // share the instruction cache, and the smallest body was the fastest (one
        // batch per turn 791 us a call, two with the second's loads ahead 806, all
        // four unrolled 836; with the causal mask's selects inside, 860).
        auto weights = [&](auto masked) {
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            float x[32];
            um_ld32(tS + lb + 32u * b, x);
            um_wait_ld();
            if constexpr (decltype(masked)::value) {
              const int* kv = &ms.kval[kb][32 * b];
#pragma unroll
              for (int j = 0; j < 32; ++j)
                x[j] = (32 * b + swap_mid(j) < lim && (!bad || kv[j] != 0)) ? x[j] : -INFINITY;
            }
            float mx[2] = {fmaxf(x[0], x[1]), fmaxf(x[2], x[3])};
#pragma unroll
            for (int j = 4; j < 32; j += 4) {
              mx[0] = max3(mx[0], x[j], x[j + 1]);
              mx[1] = max3(mx[1], x[j + 2], x[j + 3]);
            }
            const float bm = fmaxf(mx[0], mx[1]) * sc;
            const bool need = bm > m_use + kP4Slack;
            if (__any_sync(0xffffffffu, need)) {
              // O_t holds every earlier chunk (S_t of this one was issued after its MMAs were done).
              // The weights read back below are this thread's own stores of the batches before:
              // a load from TMEM is ordered behind them by this wait alone.
              if (b > 0) um_wait_st();
              const float alpha = need ? p4_ex2(m_use - bm) : 1.f;  // 0 while the row has seen nothing
              if (i > 0) {
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {
                  uint32_t o[16];
                  um_ld16(tO + lb + 16u * q, o);
                  um_wait_ld();
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                  um_st16(tO + lb + 16u * q, o);
                }
              }
#pragma unroll 1
              for (int q = 0; q < b; ++q) {  // weights of this chunk's batches before: columns 16 q ..
                uint32_t u[16];
                um_ld16(tS + lb + 16u * q, u);
                um_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float2 f = __half22float2(bits_h2(u[j]));
                  u[j] = h2_bits(__floats2half2_rn(f.x * alpha, f.y * alpha));
                }
                um_st16(tS + lb + 16u * q, u);
              }
              um_wait_st();
              ls[0] = __fmul2_rn(ls[0], make_float2(alpha, alpha));
              ls[1] = __fmul2_rn(ls[1], make_float2(alpha, alpha));
              if (need) m_use = bm;
            }
            const float nm = kP4Offset - (m_use == -INFINITY ? 0.f : m_use);
            const float2 nm2 = make_float2(nm, nm);
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 d = __ffma2_rn(make_float2(x[2 * j], x[2 * j + 1]), sc2, nm2);
              const float2 p = make_float2(p4_ex2(d.x), p4_ex2(d.y));
              ls[j & 1] = __fadd2_rn(ls[j & 1], p);
              w[j] = h2_bits(__floats2half2_rn(p.x, p.y));
            }
            um_st16(tS + lb + 16u * b, w);
          }
        };
        // (the whole warp one way: the bodies are warp-collective)
        if (__builtin_expect(__any_sync(0xffffffffu, lim < kP4Keys || bad), 0)) weights(std::true_type{});
        else weights(std::false_type{});
        um_wait_st();
        um_fence_before();
        mbar_arrive(&ms.p_full[tile]);
      }
      seen += pc.n;
      if (alive) {
        alive = mbar_wait_bounded(&ms.pv_done[tile], (uint32_t)(seen - 1) & 1u);
        alive = __all_sync(0xffffffffu, alive);
      }
      {
        float* dst = pc.slot < 0 ? a.obuf + rrow * kOStride
                                 : sp.piece(blockIdx.x, pc.slot) + (size_t)(128 * tile + trow) * kOStride;
        if (alive) {
          um_fence_after();
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float o[32];
            um_ld32(tO + lb + 32u * q, o);
            um_wait_ld();
            if (rok) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4*>(dst + 32 * q + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
          }
        }
        // a piece without a visible key has l = 0 and is skipped by the merge
        const float l = alive ? (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y) : 0.f;
        if (rok) *reinterpret_cast<float2*>(dst + 128) = make_float2(l, m_use);
      }
    }
    if (!alive && lane == 0) raise_flag(a.status, OKV_DEV_TIMEOUT);
  } else if (warp < 12) {
    // ------------------------------------------------------------ staging
    int hk = 0, pmax = 0;
    // fp16 row (sink or window ring) of position p
    auto fp16_row = [&](int p, int kind) -> const __half* {
      const bool sink = p < a.nsink;
      const size_t rows = sink ? (size_t)a.nsink : (size_t)kWin;
      const size_t row = sink ? (size_t)p : (size_t)(p % kWin);
      return (sink ? a.sink : a.ring) + ((((size_t)a.slot * a.hkv + hk) * 2 + kind) * rows + row) * kD;
    };
    // where position p is read from: 0 nowhere, 1 codes (block blk), 2 an fp16 row
    auto source = [&](int p, int blk) -> int {
      if (p > pmax || p >= a.L) return 0;
      if (p < a.nsink || p >= a.L - kWin) return 2;
      if (blk < 0 || blk >= a.num_blocks) {
        raise_flag(a.status, OKV_DEV_BAD_BLOCK);
        return 0;
      }
      return 1;
    };
    auto block_of = [&](int p) -> int { return p <= pmax && p < a.L ? __ldg(table + (p >> 4)) : -1; };
    auto head_of = [&](int blk) { return a.pages + ((size_t)blk * a.hkv + hk) * a.bhb; };
    // keys: thread = token of the chunk
    const int kt = tid - 256, krow = swap_mid(kt);
    struct FetchedK {
      int src;
      uint4 w[4];
      uint32_t sm[NG];
    } fk;
    auto fetch_k = [&](int c, int blk) {
      const int p = kP4Keys * c + kt;
      fk.src = source(p, blk);
      if (fk.src == 1) {
        const uint8_t* bp = head_of(blk);
        const uint4* cp = reinterpret_cast<const uint4*>(bp + (p & 15) * 64);
#pragma unroll
        for (int j = 0; j < 4; ++j) fk.w[j] = __ldg(cp + j);
        const uint32_t* sp = reinterpret_cast<const uint32_t*>(bp + kSm) + (p & 15) * NG;
#pragma unroll
        for (int k = 0; k < NG; ++k) fk.sm[k] = __ldg(sp + k);
      }
    };
    // values: thread = (token quad, code byte mod 8) of two blocks
    const int vg = lane >> 2, tq = lane & 3, vw = warp - 8;  // blocks 2 vw, 2 vw + 1 of the chunk
    struct FetchedV {
      int src[2];       // per block: 1 all four tokens from codes, 0 none read, else token by token (2: no codes)
      uint4 w[2][2];    // words 0-3 and 4-7: byte 8 mt + vg of tokens 4 tq .. + 3
      uint4 sm[2][NG];  // (scale, min) of the four tokens, NG pairs each
    } fv;
    auto quad_pos = [&](int c, int bb) { return kP4Keys * c + 16 * (2 * vw + bb) + 4 * tq; };
    auto fetch_block = [&](const uint8_t* bp, int bb) {
      fv.w[bb][0] = __ldg(reinterpret_cast<const uint4*>(bp + kVcOff4 + 16 * lane));
      fv.w[bb][1] = __ldg(reinterpret_cast<const uint4*>(bp + kVcOff4 + 512 + 16 * lane));
      const uint4* sp = reinterpret_cast<const uint4*>(bp + kSm + 64 * NG) + tq * NG;
#pragma unroll
      for (int k = 0; k < NG; ++k) fv.sm[bb][k] = __ldg(sp + k);
    };
    static_assert(NG == 1 || NG == 2 || NG == 4, "groups per vector");
    auto fetch_v = [&](int c, const int (&blk)[2]) {
#pragma unroll
      for (int bb = 0; bb < 2; ++bb) {
        const int p = quad_pos(c, bb);
        const int first = source(p, blk[bb]), last = p + 3 > pmax || p + 3 >= a.L ? 0 : source(p + 3, blk[bb]);
        // a quad lies on one side of the sinks' end (a multiple of 16); only the window's start and pmax cut it
        // (a bad block id skips the quad's code positions; window positions in it are still read)
        fv.src[bb] = first == 1 && last == 1 ? 1 : first == 1 ? 3 : first == 2 || last == 2 ? 2 : 0;
        if (first == 1) fetch_block(head_of(blk[bb]), bb);
      }
    };
    // lane's (chunk lane = 4 vg + tq) pair words: token i, group k at word i NG + k of the quad's 16 NG bytes
    auto pair_word = [&](int bb, int i, int k) -> uint32_t {
      const int w = i * NG + k;
      const uint4& q = fv.sm[bb][w >> 2];
      return (w & 3) == 0 ? q.x : (w & 3) == 1 ? q.y : (w & 3) == 2 ? q.z : q.w;
    };
    int done = 0;  // chunks of the pieces before
    bool alive = true;
    Piece pc;
#pragma unroll 1
    for (int2 u = u_begin; more(u) && alive; done += pc.n) {
      u = next_piece(u, pc);
      hk = pc.hk;
      pmax = prefill_last_pos(a, pc.x);
      int kblk = block_of(kP4Keys * pc.c0 + kt), vblk[2];  // block ids one chunk ahead of the codes
#pragma unroll
      for (int bb = 0; bb < 2; ++bb) vblk[bb] = block_of(quad_pos(pc.c0, bb));
      fetch_k(pc.c0, kblk);
      fetch_v(pc.c0, vblk);
      kblk = block_of(kP4Keys * (pc.c0 + 1) + kt);
#pragma unroll
      for (int bb = 0; bb < 2; ++bb) vblk[bb] = block_of(quad_pos(pc.c0 + 1, bb));
      for (int i = 0; i < pc.n; ++i) {
        const int c = pc.c0 + i, at = done + i, st = at & 1;
        const uint32_t ph = (uint32_t)((at >> 1) - 1) & 1u;
        if (at >= 2 && !(alive = __all_sync(0xffffffffu, mbar_wait_bounded(&ms.k_free[st], ph)) != 0)) {
          raise_flag(a.status, OKV_DEV_TIMEOUT);
          break;
        }
        {
          unsigned char* dst = gb + kP4OffK + (uint32_t)st * kP4Tile;
          bool easy = fk.src == 1;  // codes, and no |s c + m| past fp16's range
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            const __half2 sm = bits_h2(fk.sm[k]);
            easy = easy && 15.f * __low2float(sm) + fabsf(__high2float(sm)) <= 65504.f;
          }
          if (__builtin_expect(easy, 1)) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const __half2 sm = bits_h2(fk.sm[s * NG / 4]);
              const __half2 s2 = __low2half2(sm), m2 = __high2half2(sm);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // word s of chunk j: channels 32 s + 8 j .. + 7, low halves even
                const uint32_t w = s == 0 ? fk.w[j].x : s == 1 ? fk.w[j].y : s == 2 ? fk.w[j].z : fk.w[j].w;
                const uint32_t y = w >> 8;
                *reinterpret_cast<uint4*>(dst + (s >> 1) * 16384 +
                                          um_swz((uint32_t)krow, (uint32_t)(4 * (s & 1) + j) * 16u)) =
                    make_uint4(p4_even(w, s2, m2), p4_odd(w, s2, m2), p4_even(y, s2, m2), p4_odd(y, s2, m2));
              }
            }
          } else if (fk.src != 1) {  // an fp16 row, or a key nobody reads
            const uint4* row = fk.src == 2 ? reinterpret_cast<const uint4*>(fp16_row(kP4Keys * c + kt, 0)) : nullptr;
#pragma unroll 1
            for (int h = 0; h < 16; h += 8) {
              uint4 y[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = row != nullptr ? row[h + j] : make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int j = 0; j < 8; ++j)  // into the order 0 4 1 5 2 6 3 7
                *reinterpret_cast<uint4*>(dst + h * 2048 + um_swz((uint32_t)krow, (uint32_t)j * 16u)) =
                    make_uint4(__byte_perm(y[j].x, y[j].z, 0x5410u), __byte_perm(y[j].x, y[j].z, 0x7632u),
                               __byte_perm(y[j].y, y[j].w, 0x5410u), __byte_perm(y[j].y, y[j].w, 0x7632u));
            }
          } else {  // values that saturate, from global memory; rolled up, as what is rare stays out of the instruction cache
            const int p = kP4Keys * c + kt;
            const uint8_t* bp = head_of(__ldg(table + (p >> 4)));
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {  // channels 8 j .. + 7
              const uint32_t w = *reinterpret_cast<const uint32_t*>(bp + (p & 15) * 64 + (j & 3) * 16 + (j >> 2) * 4);
              const __half2 sm = *reinterpret_cast<const __half2*>(bp + kSm + ((p & 15) * NG + (j >> 2) * NG / 4) * 4);
              const __half2 s2 = __low2half2(sm), m2 = __high2half2(sm);
              const uint32_t y = w >> 8;
              *reinterpret_cast<uint4*>(dst + (j >> 3) * 16384 + um_swz((uint32_t)krow, (uint32_t)(j & 7) * 16u)) =
                  make_uint4(sat_h2(p4_even(w, s2, m2)), sat_h2(p4_odd(w, s2, m2)), sat_h2(p4_even(y, s2, m2)),
                             sat_h2(p4_odd(y, s2, m2)));
            }
          }
          const int p = kP4Keys * c + kt;
          const bool lost = fk.src == 0 && p <= pmax && p < a.L;  // a visible position without its block
          ms.kval[at & 3][krow] = !lost;
          const int any = __any_sync(0xffffffffu, lost);
          if (lane == 0) ms.bad[at & 3][warp - 8] = any;
        }
        um_fence_proxy_async();
        mbar_arrive(&ms.k_full[st]);
        if (at >= 2 && !(alive = __all_sync(0xffffffffu, mbar_wait_bounded(&ms.v_free[st], ph)) != 0)) {
          raise_flag(a.status, OKV_DEV_TIMEOUT);
          break;
        }
        unsigned char* dst = gb + kP4OffV + (uint32_t)st * kP4Tile;
        // the quad's four tokens of channel ch, of the thread's block bb
        auto put = [&](int bb, int ch, uint32_t t02, uint32_t t13) {
          const int blk16 = 2 * vw + bb;  // block of the chunk
          *reinterpret_cast<uint2*>(dst + (blk16 >> 2) * 16384 +
                                    um_swz((uint32_t)ch, (uint32_t)(16 * (blk16 & 3) + 4 * tq) * 2u)) = make_uint2(t02, t13);
        };
        uint32_t rare = 0;  // blocks left to the loop below
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          bool easy = fv.src[bb] == 1;
#pragma unroll
          for (int k = 0; k < NG; ++k)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const __half2 sm = bits_h2(pair_word(bb, t, k));
              easy = easy && 15.f * __low2float(sm) + fabsf(__high2float(sm)) <= 65504.f;
            }
          if (__builtin_expect(easy, 1)) {
#pragma unroll
            for (int k = 0; k < NG; ++k) {
              const uint32_t q0 = pair_word(bb, 0, k), q1 = pair_word(bb, 1, k), q2 = pair_word(bb, 2, k),
                             q3 = pair_word(bb, 3, k);
              const __half2 s02 = bits_h2(__byte_perm(q0, q2, 0x5410u)), m02 = bits_h2(__byte_perm(q0, q2, 0x7632u));
              const __half2 s13 = bits_h2(__byte_perm(q1, q3, 0x5410u)), m13 = bits_h2(__byte_perm(q1, q3, 0x7632u));
#pragma unroll
              for (int mt = 8 / NG * k; mt < 8 / NG * (k + 1); ++mt) {
                const uint4& q = fv.w[bb][mt >> 2];
                const uint32_t w = (mt & 3) == 0 ? q.x : (mt & 3) == 1 ? q.y : (mt & 3) == 2 ? q.z : q.w;
                const uint32_t y = w >> 8;  // tokens 1 and 3
                put(bb, 16 * mt + 2 * vg, p4_even(w, s02, m02), p4_even(y, s13, m13));
                put(bb, 16 * mt + 2 * vg + 1, p4_odd(w, s02, m02), p4_odd(y, s13, m13));
              }
            }
          } else {
            rare |= 1u << bb;
          }
        }
        if (__builtin_expect(rare != 0, 0)) {
#pragma unroll 1
          for (int bb = 0; bb < 2; ++bb) {
            if (((rare >> bb) & 1u) == 0) continue;
            const int p = quad_pos(c, bb), src = bb == 0 ? fv.src[0] : fv.src[1];
            const __half* row[4];  // of the quad's tokens: fp16 rows, null for codes and for tokens nobody reads
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int pt = p + t;
              const bool fp16 = src != 0 && pt <= pmax && pt < a.L && (pt < a.nsink || pt >= a.L - kWin);
              row[t] = fp16 ? fp16_row(pt, 1) : nullptr;
            }
            if ((src & 1) == 0) {  // no codes: 8 channels of the four rows at a time
#pragma unroll 1
              for (int h = 0; h < 128; h += 64) {
                const int ch = h + 8 * vg;
                uint4 y[4];
#pragma unroll
                for (int t = 0; t < 4; ++t)
                  y[t] = row[t] != nullptr ? *reinterpret_cast<const uint4*>(row[t] + ch) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t e0 = (&y[0].x)[k], e1 = (&y[1].x)[k], e2 = (&y[2].x)[k], e3 = (&y[3].x)[k];
                  put(bb, ch + 2 * k, __byte_perm(e0, e2, 0x5410u), __byte_perm(e1, e3, 0x5410u));
                  put(bb, ch + 2 * k + 1, __byte_perm(e0, e2, 0x7632u), __byte_perm(e1, e3, 0x7632u));
                }
              }
              continue;
            }
            // codes beside fp16 rows, or values that saturate: token by token
            const uint8_t* bp = head_of(__ldg(table + (p >> 4)));
#pragma unroll 1
            for (int mt = 0; mt < 8; ++mt) {
              const uint8_t* wp = bp + kVcOff4 + (mt >> 2) * 512 + 16 * lane + 4 * (mt & 3);
              const uint32_t w = *reinterpret_cast<const uint32_t*>(wp);
              uint32_t e[4];  // token t: channels 16 mt + 2 vg, + 1
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const uint8_t* mp = bp + kSm + 64 * NG + ((4 * tq + t) * NG + mt * NG / 8) * 4;
                const __half2 sm = *reinterpret_cast<const __half2*>(mp);
                const uint32_t byte = (w >> (8 * t)) & 0xFFu;
                e[t] = sat_h2(p4_even((byte & 15u) | (byte << 12), __low2half2(sm), __high2half2(sm)));
                if (row[t] != nullptr) e[t] = *reinterpret_cast<const uint32_t*>(row[t] + 16 * mt + 2 * vg);
                else if (p + t > pmax || p + t >= a.L) e[t] = 0u;
              }
              put(bb, 16 * mt + 2 * vg, __byte_perm(e[0], e[2], 0x5410u), __byte_perm(e[1], e[3], 0x5410u));
              put(bb, 16 * mt + 2 * vg + 1, __byte_perm(e[0], e[2], 0x7632u), __byte_perm(e[1], e[3], 0x7632u));
            }
          }
        }
        um_fence_proxy_async();
        mbar_arrive(&ms.v_full[st]);
        // The next chunk's loads go out here, behind the second fence: a fence
        // waits for the loads in flight, so keys fetched between the two fences
        // (and values before the first) left their latency bare twice per chunk.
        if (i + 1 < pc.n) {
          fetch_k(c + 1, kblk);
          fetch_v(c + 1, vblk);
          kblk = block_of(kP4Keys * (c + 2) + kt);
#pragma unroll
          for (int bb = 0; bb < 2; ++bb) vblk[bb] = block_of(quad_pos(c + 2, bb));
        }
      }
    }
  } else {
    // ------------------------------------------------------------ MMA issue
    // Per piece S_0(0), S_1(0), then per chunk: O_0 += P_0 V, S_0 of the next chunk, O_1 += P_1 V, S_1 of the next.
    // The whole warp runs the loop and one elected lane issues: descriptors and
    // TMEM addresses then stay in uniform registers.  (Issued by `lane == 0`,
    // an MMA cost the thread 130 cycles, twice its time on the tensor pipe.)
    uint64_t* last_bar = nullptr;  // the latest commit: it completes after every MMA issued before it
    uint32_t last_par = 0;
    const uint64_t dQ = um_desc(base + kP4OffQ), dK = um_desc(base + kP4OffK), dV = um_desc(base + kP4OffV);
    // phase `k` of a barrier, the same answer in every lane
    auto wait = [&](uint64_t* bar, int k) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(bar, (uint32_t)k & 1u)) != 0;
    };
    int nt = 0;
    int done = 0, seen[2] = {0, 0}, pieces[2] = {0, 0};  // before this piece: chunks; those, and pieces, with tile t
    auto issue_s = [&](int t, int i) -> bool {
      const int at = done + i, st = at & 1, own = (t == 0 ? seen[0] : seen[1]) + i;
      if (!wait(&ms.k_full[st], at >> 1)) return false;
      // the weights of the chunk before lie over the score columns until its value MMA is done
      if (own >= 1 && !wait(&ms.pv_done[t], own - 1)) return false;
      if (i == 0 && !wait(&ms.q_full[t], t == 0 ? pieces[0] : pieces[1])) return false;
      um_fence_after();
      const uint64_t qd = dQ + (uint64_t)((t * kP4Tile) >> 4), kd = dK + (uint64_t)((st * kP4Tile) >> 4);
      if (um_elect()) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t off = (uint64_t)(((k >> 2) * 16384 + (k & 3) * 32) >> 4);
          um_mma(tmem + 128u * (uint32_t)t, qd + off, kd + off, kP4Idesc, k > 0 ? 1u : 0u);
        }
        mbar_arrive(&ms.s_full[t]);  // passes on what the key warps wrote before k_full
        um_commit(&ms.s_full[t]);
        if (t == nt - 1) um_commit(&ms.k_free[st]);
      }
      __syncwarp();
      last_bar = t == nt - 1 ? &ms.k_free[st] : &ms.s_full[t];
      last_par = (uint32_t)(t == nt - 1 ? at >> 1 : own) & 1u;
      return true;
    };
    auto issue_pv = [&](int t, int i) -> bool {
      const int at = done + i, st = at & 1, own = (t == 0 ? seen[0] : seen[1]) + i;
      if (!wait(&ms.v_full[st], at >> 1)) return false;
      if (!wait(&ms.p_full[t], own)) return false;
      um_fence_after();
      const uint64_t vd = dV + (uint64_t)((st * kP4Tile) >> 4);
      if (um_elect()) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t off = (uint64_t)(((k >> 2) * 16384 + (k & 3) * 32) >> 4);
          um_mma_ts(tmem + 256u + 128u * (uint32_t)t, tmem + 128u * (uint32_t)t + 8u * (uint32_t)k, vd + off, kP4Idesc,
                    (i > 0 || k > 0) ? 1u : 0u);
        }
        um_commit(&ms.pv_done[t]);
        if (t == nt - 1) um_commit(&ms.v_free[st]);
      }
      __syncwarp();
      last_bar = t == nt - 1 ? &ms.v_free[st] : &ms.pv_done[t];
      last_par = (uint32_t)(t == nt - 1 ? at >> 1 : own) & 1u;
      return true;
    };
    bool alive = true;
    Piece pc;
#pragma unroll 1
    for (int2 u = u_begin; more(u) && alive;) {
      u = next_piece(u, pc);
      nt = pc.nt;
#pragma unroll 1
      for (int i = -1; i < pc.n && alive; ++i)
#pragma unroll 1
        for (int t = 0; t < nt && alive; ++t)
          alive = (i < 0 || issue_pv(t, i)) && (i + 1 >= pc.n || issue_s(t, i + 1));
      done += pc.n;
      for (int t = 0; t < nt; ++t) {
        (t == 0 ? seen[0] : seen[1]) += pc.n;
        (t == 0 ? pieces[0] : pieces[1]) += 1;
      }
    }
    if (!alive && lane == 0) raise_flag(a.status, OKV_DEV_TIMEOUT);
    // the MMAs already issued finish before TMEM is freed: the last commit covers them all
    if (last_bar != nullptr) mbar_drain_bounded(last_bar, last_par);
  }
  um_fence_before();
  __syncthreads();
  if (warp == 12) {
    um_fence_after();
    um_dealloc(tmem, 512);
  }
}

}  // namespace

okv_status launch_prefill_int4_bf16(const PrefillArgs& a, const P4Split& sp, cudaStream_t s) {
  using Kernel = void (*)(PrefillArgs, P4Split);
  static const Kernel kernels[3] = {prefill_int4_kernel<1>, prefill_int4_kernel<2>, prefill_int4_kernel<4>};
  static std::atomic<uint32_t> attr[3];
  const int gi = a.ng >> 1;  // ng = 1, 2, 4 -> 0, 1, 2
  cudaError_t e = set_smem_limit_once((const void*)kernels[gi], (int)kP4Smem, attr[gi]);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "prefill attention smem attribute: %s", cudaGetErrorString(e));
  // Programmatic launch: staging starts while the query rotation runs (the calls before that are done, as it is
  // launched behind them); 203 tokens over 2999 keys 54.4 against 57.0 us, 1024 over 32K 685 against 687.
  e = launch_pdl(kernels[gi], dim3(sp.ctas), dim3(kP4Threads), kP4Smem, s, true, a, sp);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "prefill attention launch: %s", cudaGetErrorString(e));
  return check_launch("prefill attention");
}

}  // namespace okv
