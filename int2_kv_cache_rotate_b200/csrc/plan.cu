// Block tables and slot maps of a serving step, built on the GPU from request
// lengths (okv_plan_append).
//
// Request b holds old_b tokens and gains new_b.  With need_b =
// ceil((old_b + new_b) / 16) - ceil(old_b / 16) and the inclusive sums
// NB_b = sum need, NT_b = sum new over the requests up to b, request b is
// served when NB_b fits the pool and NT_b the token rows; its tokens take rows
// NT_{b-1} .. NT_b - 1 and its new table columns the pool's blocks
// count - 1 - NB_{b-1}, downwards.  A new column c has exactly one new token
// at position 16 c, so the thread that writes that token's row also writes
// the column: one pass over token rows does everything but the scan.  The row
// of a request's last new token also gets the request's length, every other row
// 0: with them a decode call takes token rows as its entries.
//
// Bound: the scan is latency (a few loads and a block-wide scan), the rows are
// 8 bytes written per token.
#include "okv_common.cuh"
#include "okv_internal.h"

namespace okv {
namespace {

constexpr int kPlThreads = 1024;
constexpr int kPlWarps = kPlThreads / 32;
constexpr uint32_t kPlSat = 1u << 30;  // sums saturate here, above every capacity

struct PlanArgs {
  okv_plan p;
  // per request, between the two kernels of the split form (workspace): tokens
  // held before, blocks taken by the requests before it; then the pool's count
  int32_t* old_len;
  int32_t* blk_off;
  int32_t* pool;
};

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kPlSat); }

// Block-wide inclusive scan of two saturating sums (non-negative operands up
// to 2^30 each, so a + b stays below 2^31 and saturation is associative).
__device__ __forceinline__ void scan2(uint32_t& x, uint32_t& y, uint2* warp_tot, uint2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, x, d), b = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x = sat_add(x, a);
      y = sat_add(y, b);
    }
  }
  if (lane == 31) warp_tot[warp] = make_uint2(x, y);
  __syncthreads();
  uint2 w = warp_tot[lane];  // kPlWarps = 32 totals: every warp scans them itself
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, w.x, d), b = __shfl_up_sync(0xffffffffu, w.y, d);
    if (lane >= d) {
      w.x = sat_add(w.x, a);
      w.y = sat_add(w.y, b);
    }
  }
  total = make_uint2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
  const uint32_t px = __shfl_sync(0xffffffffu, w.x, max(warp - 1, 0)), py = __shfl_sync(0xffffffffu, w.y, max(warp - 1, 0));
  if (warp > 0) {
    x = sat_add(x, px);
    y = sat_add(y, py);
  }
  __syncthreads();  // warp_tot may be written again
}
static_assert(kPlWarps == 32, "scan2 lets one warp hold every warp's total");

// Row `row` of the token maps: its request is the one with cu[b] <= row <
// cu[b + 1] (n_req requests, cu[n_req] = total); `old_of` and `off_of` give a
// request's tokens before this step and its first block's distance from the
// pool's end.  len: the request's tokens after the step in the row of its last
// new token, else 0.
template <typename Cu, typename Slot, typename Old, typename Off>
__device__ __forceinline__ void plan_row(const okv_plan& p, int row, int lo, int hi, int total, int count, const Cu& cu,
                                         const Slot& slot_of, const Old& old_of, const Off& off_of, int& slot, int& pos, int& len) {
  slot = pos = -1;
  len = 0;
  if (row >= total) return;
  while (lo < hi) {  // the last request whose first row is <= row
    const int mid = (lo + hi + 1) >> 1;
    if (cu(mid) <= row) lo = mid;
    else hi = mid - 1;
  }
  slot = slot_of(lo);
  const int old = old_of(lo);
  pos = old + row - cu(lo);
  len = row + 1 == cu(lo + 1) ? pos + 1 : 0;
  if ((pos & (kBlock - 1)) == 0) {
    const int col = pos >> 4, first = (old + kBlock - 1) >> 4;
    p.block_table[(size_t)slot * p.max_blocks_per_seq + col] = p.free_blocks[count - 1 - off_of(lo) - (col - first)];
  }
}

// The scan, by one CTA; with kFill also the token rows (small steps: one
// launch).  Shared memory: two bits per sequence slot (seen, seen twice), then
// with kFill four ints per request (first row, slot, old length, block offset).
template <bool kFill>
__global__ void __launch_bounds__(kPlThreads) plan_scan_kernel(PlanArgs a) {
  extern __shared__ uint32_t pl_smem[];
  __shared__ uint2 warp_tot[kPlWarps];
  const okv_plan& p = a.p;
  const int B = p.num_requests, tid = threadIdx.x;
  const int words = (p.num_seq_slots + 31) >> 5;
  uint32_t* seen = pl_smem;
  uint32_t* twice = pl_smem + words;
  int* s_cu = reinterpret_cast<int*>(pl_smem + 2 * words);
  int* s_slot = s_cu + (B + 1);
  int* s_old = s_slot + B;
  int* s_off = s_old + B;
  grid_dep_launch();
  const int count = min(max(*p.free_count, 0), p.num_free);
  for (int i = tid; i < 2 * words; i += kPlThreads) pl_smem[i] = 0u;
  __syncthreads();
  // a slot named by two requests: both are dropped, whatever the order
  for (int b = tid; b < B; b += kPlThreads) {
    const int slot = p.seq_slot[b];
    if (slot >= 0 && slot < p.num_seq_slots) {
      const uint32_t bit = 1u << (slot & 31);
      if (atomicOr(&seen[slot >> 5], bit) & bit) atomicOr(&twice[slot >> 5], bit);
    }
  }
  __syncthreads();
  uint32_t base_b = 0, base_t = 0;      // inclusive sums of the tiles before
  uint32_t used_b = 0, used_t = 0;      // of the requests served (tile-wide, the same in every thread)
  uint32_t flags = 0;
  __shared__ uint32_t s_used[2];
  if (tid == 0) s_used[0] = s_used[1] = 0u;
  for (int b0 = 0; b0 < B; b0 += kPlThreads) {
    const int b = b0 + tid;
    int slot = -1, old = 0;
    uint32_t nb = 0, nt = 0;
    bool live = false;
    if (b < B) {
      slot = p.seq_slot[b];
      old = p.cached_lens[b];
      const int add = p.new_lens[b];
      if (slot < 0 || slot >= p.num_seq_slots || ((twice[slot >> 5] >> (slot & 31)) & 1u)) {
        if (slot != -1) flags |= OKV_DEV_BAD_SLOT;  // -1: a padding entry
      } else if (old < 0 || add < 0 || (long long)old + add > (long long)p.max_blocks_per_seq * kBlock) {
        flags |= OKV_DEV_BAD_POS;
      } else {
        live = true;
        nt = (uint32_t)add;
        nb = (uint32_t)(((old + add + kBlock - 1) >> 4) - ((old + kBlock - 1) >> 4));
      }
    }
    uint32_t sb = nb, st = nt;
    uint2 total;
    scan2(sb, st, warp_tot, total);
    sb = sat_add(sb, base_b);
    st = sat_add(st, base_t);
    const bool took = live && sb <= (uint32_t)count && st <= (uint32_t)p.max_tokens;
    if (live && !took) flags |= (sb > (uint32_t)count ? OKV_DEV_NO_BLOCKS : 0u) |
                               (st > (uint32_t)p.max_tokens ? OKV_DEV_NO_ROWS : 0u);
    // The sums grow with b, so the requests served are a prefix of the live
    // ones, and a served request's sums hold served requests only.
    const uint32_t top_b = __reduce_max_sync(0xffffffffu, took ? sb : 0u);
    const uint32_t top_t = __reduce_max_sync(0xffffffffu, took ? st : 0u);
    if ((tid & 31) == 0) {
      atomicMax(&s_used[0], top_b);
      atomicMax(&s_used[1], top_t);
    }
    __syncthreads();
    used_b = s_used[0];
    used_t = s_used[1];
    if (b < B) {
      const int first = (int)(took ? st - nt : used_t);  // an unserved request is an empty range
      const int off = (int)(took ? sb - nb : 0u);
      const int len = live ? old + (took ? (int)nt : 0) : 0;
      // dead requests between served ones: their range must keep the order of cu
      const int at = took ? first : (int)min(st, used_t);
      p.cu_tokens[b] = at;
      p.context_lens[b] = len;
      if (live) p.slot_lens[slot] = len;
      if constexpr (kFill) {
        s_cu[b] = at;
        s_slot[b] = slot;
        s_old[b] = old;
        s_off[b] = off;
      } else {
        a.old_len[b] = old;
        a.blk_off[b] = off;
      }
    }
    base_b = sat_add(base_b, total.x);
    base_t = sat_add(base_t, total.y);
  }
  flags = __reduce_or_sync(0xffffffffu, flags);  // (one atomic per warp: 300 of one word took 10 us)
  if (flags != 0u && (tid & 31) == 0) raise_flag(p.status_word, flags);
  const int total_rows = (int)used_t;
  if (tid == 0) {
    p.cu_tokens[B] = total_rows;
    *p.free_count_out = count - (int)used_b;
    if constexpr (!kFill) *a.pool = count;
  }
  if constexpr (kFill) {
    if (tid == 0) s_cu[B] = total_rows;
    __syncthreads();
    for (int row = tid; row < p.max_tokens; row += kPlThreads) {
      int slot, pos, len;
      plan_row(p, row, 0, B - 1, total_rows, count, [&](int i) { return s_cu[i]; }, [&](int i) { return s_slot[i]; },
               [&](int i) { return s_old[i]; }, [&](int i) { return s_off[i]; }, slot, pos, len);
      p.tok_slot[row] = slot;
      p.tok_pos[row] = pos;
      if (p.tok_lens != nullptr) p.tok_lens[row] = len;
    }
  }
}

constexpr int kPlRows = 4;  // consecutive rows per thread of the fill kernel
constexpr int kPlFillThreads = 256;

__global__ void __launch_bounds__(kPlFillThreads) plan_fill_kernel(PlanArgs a) {
  grid_dep_wait();  // the scan's results
  const okv_plan& p = a.p;
  const int B = p.num_requests;
  const int total = p.cu_tokens[B], count = *a.pool;
  const long long r0 = ((long long)blockIdx.x * kPlFillThreads + threadIdx.x) * kPlRows;
  if (r0 >= p.max_tokens) return;
  int lo = 0, hi = B - 1;
  while (lo < hi) {  // the request of row r0
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_tokens[mid] <= r0) lo = mid;
    else hi = mid - 1;
  }
  int slot[kPlRows], pos[kPlRows], len[kPlRows];
#pragma unroll
  for (int i = 0; i < kPlRows; ++i) {
    const int row = (int)r0 + i;
    // rows of one thread nearly always share a request: step on from the last one's
    // (not past the last token: the requests behind it all start there)
    if (row < total)
      while (lo + 1 < B && p.cu_tokens[lo + 1] <= row) ++lo;
    plan_row(p, row, lo, lo, total, count, [&](int b) { return p.cu_tokens[b]; }, [&](int b) { return p.seq_slot[b]; },
             [&](int b) { return a.old_len[b]; }, [&](int b) { return a.blk_off[b]; }, slot[i], pos[i],
             len[i]);
  }
  const bool lens = p.tok_lens != nullptr;
  if (r0 + kPlRows <= p.max_tokens &&
      ((((uintptr_t)p.tok_slot | (uintptr_t)p.tok_pos | (uintptr_t)p.tok_lens) & 15u) == 0)) {
    *reinterpret_cast<int4*>(p.tok_slot + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(p.tok_pos + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    if (lens) *reinterpret_cast<int4*>(p.tok_lens + r0) = make_int4(len[0], len[1], len[2], len[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kPlRows; ++i)
      if (r0 + i < p.max_tokens) {
        p.tok_slot[r0 + i] = slot[i];
        p.tok_pos[r0 + i] = pos[i];
        if (lens) p.tok_lens[r0 + i] = len[i];
      }
  }
}

// One launch up to this many requests and token rows, else the scan and a
// fill over the whole GPU.  Measured in a graph, one launch against two:
// 256 requests with 256 rows 3.6 and 6.4 us, 8 with 4096 rows 5.5 and 5.7, 256
// with 4096 rows 6.6 and 6.5, 4096 with 4096 rows 13.0 and 14.3; but 8 with
// 8192 rows 7.5 and 5.8, 256 with 8192 rows 9.7 and 6.8, 8 with 32768 rows
// 19.6 and 5.8.  So rows decide; more requests than this would not fit the
// shared memory beside the largest slot bitmap.
constexpr int kPlOneCtaRequests = 4096;
constexpr int kPlOneCtaRows = 4096;

}  // namespace
}  // namespace okv

using namespace okv;

extern "C" {

size_t okv_plan_workspace_bytes(int32_t num_requests) {
  return num_requests < 0 ? 0 : (size_t)(2 * (long long)num_requests + 1) * sizeof(int32_t);
}

okv_status okv_plan_append(const okv_plan* plan, void* workspace, size_t workspace_bytes, void* stream) {
  if (plan == nullptr) return fail(OKV_ERR_INVALID_ARG, "plan is NULL");
  const okv_plan& p = *plan;
  if (p.num_requests < 0 || p.max_tokens < 0 || p.num_free < 0)
    return fail(OKV_ERR_INVALID_ARG, "num_requests, max_tokens and num_free must be >= 0");
  if (p.num_seq_slots < 1 || p.max_blocks_per_seq < 1)
    return fail(OKV_ERR_INVALID_ARG, "num_seq_slots and max_blocks_per_seq must be >= 1");
  if ((long long)p.max_blocks_per_seq * kBlock > 0x3fffffffLL)
    return fail(OKV_ERR_INVALID_ARG, "max_blocks_per_seq too large");
  if (p.num_seq_slots > OKV_PLAN_MAX_SLOTS)
    return fail(OKV_ERR_UNSUPPORTED, "num_seq_slots > %d", OKV_PLAN_MAX_SLOTS);
  if (p.max_tokens >= (int)kPlSat || p.num_free >= (int)kPlSat || p.num_requests >= (int)kPlSat)
    return fail(OKV_ERR_INVALID_ARG, "max_tokens, num_free and num_requests must be below 2^30");
  if (!p.cu_tokens || !p.free_count || !p.free_count_out)
    return fail(OKV_ERR_INVALID_ARG, "cu_tokens, free_count and free_count_out must be non-NULL");
  if (p.num_requests > 0 && (!p.seq_slot || !p.cached_lens || !p.new_lens || !p.context_lens))
    return fail(OKV_ERR_INVALID_ARG, "seq_slot, cached_lens, new_lens and context_lens must be non-NULL");
  if (!p.block_table || !p.slot_lens || (p.num_free > 0 && !p.free_blocks))
    return fail(OKV_ERR_INVALID_ARG, "block_table, slot_lens and free_blocks must be non-NULL");
  if (p.max_tokens > 0 && (!p.tok_slot || !p.tok_pos))
    return fail(OKV_ERR_INVALID_ARG, "tok_slot and tok_pos must be non-NULL");
  for (const void* x : {(const void*)p.seq_slot, (const void*)p.cached_lens, (const void*)p.new_lens,
                        (const void*)p.free_blocks, (const void*)p.free_count, (const void*)p.block_table,
                        (const void*)p.slot_lens, (const void*)p.context_lens, (const void*)p.cu_tokens,
                        (const void*)p.tok_slot, (const void*)p.tok_pos, (const void*)p.free_count_out,
                        (const void*)p.status_word, (const void*)p.tok_lens})
    if ((uintptr_t)x % 4) return fail(OKV_ERR_INVALID_ARG, "every array must be 4-byte aligned");
  const cudaStream_t s = (cudaStream_t)stream;
  const size_t bitmap = (size_t)2 * ((p.num_seq_slots + 31) / 32) * sizeof(uint32_t);
  PlanArgs a;
  a.p = p;
  a.old_len = a.blk_off = a.pool = nullptr;
  static std::atomic<uint32_t> one_attr{0}, scan_attr{0};
  constexpr int kBitmapMost = 2 * ((OKV_PLAN_MAX_SLOTS + 31) / 32) * 4;
  if (p.num_requests <= kPlOneCtaRequests && p.max_tokens <= kPlOneCtaRows) {
    constexpr int kMost = kBitmapMost + (4 * kPlOneCtaRequests + 1) * 4;
    cudaError_t e = set_smem_limit_once((const void*)plan_scan_kernel<true>, kMost, one_attr);
    if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "plan smem attribute: %s", cudaGetErrorString(e));
    plan_scan_kernel<true><<<1, kPlThreads, bitmap + (4 * (size_t)p.num_requests + 1) * sizeof(int), s>>>(a);
    return check_launch("plan");
  }
  if (workspace == nullptr || (uintptr_t)workspace % 4)
    return fail(OKV_ERR_INVALID_ARG, "workspace must be a 4-byte aligned device buffer");
  if (workspace_bytes < okv_plan_workspace_bytes(p.num_requests))
    return fail(OKV_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes,
                okv_plan_workspace_bytes(p.num_requests));
  a.old_len = (int32_t*)workspace;
  a.blk_off = a.old_len + p.num_requests;
  a.pool = a.blk_off + p.num_requests;
  cudaError_t e = set_smem_limit_once((const void*)plan_scan_kernel<false>, kBitmapMost, scan_attr);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "plan smem attribute: %s", cudaGetErrorString(e));
  plan_scan_kernel<false><<<1, kPlThreads, bitmap, s>>>(a);
  okv_status st = check_launch("plan scan");
  if (st != OKV_OK || p.max_tokens == 0) return st;
  const long long per = (long long)kPlFillThreads * kPlRows;
  e = launch_pdl(plan_fill_kernel, dim3((unsigned)((p.max_tokens + per - 1) / per)), dim3(kPlFillThreads), 0, s, true, a);
  if (e != cudaSuccess) return fail(OKV_ERR_CUDA, "plan fill launch: %s", cudaGetErrorString(e));
  return check_launch("plan fill");
}

}  // extern "C"
