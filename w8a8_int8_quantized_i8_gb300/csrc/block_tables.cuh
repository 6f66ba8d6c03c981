// block_tables.cuh -- block tables, slot map, positions and offsets of one
// serving step, from the requests' lengths, on the device.
//
// Request r holds context[r] tokens in ceil(context[r] / B) blocks and brings
// news[r] new ones.  With exclusive sums over the requests,
//   cu_new[r]    = sum of news before r
//   first[r]     = taken + sum of fresh blocks before r,
//   fresh[r]     = ceil((context + news) / B) - ceil(context / B),
// the request's fresh block c (counted from its first) is
// free_blocks[first[r] + c], and the new token at position p gets the slot
// table[r][p / B] * B + p % B.
//
// The work is a few bytes a token: a launch's latency bounds it.  So it is one
// launch without a grid-wide wait: every CTA scans all requests by itself (two
// loads a request, from L2) into shared memory, then writes its share of the
// tokens and of the tables.  A fresh block is taken from the free list, not
// from the table that another CTA may still be writing.  5.1 us for 64 decoding
// requests, 7.0 us for 2048 requests with 104236 tokens (1.3 MB); one scan over
// consecutive requests a thread instead of one a 512 requests took 2 us off the
// latter, shifts instead of 64-bit divisions 1 us off the former.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace i8 {

constexpr int kTableThreads = 1024;
constexpr int kTableMaxRequests = 16384;  // three words a request in shared memory: 192 KB

struct TableArgs {
  const int32_t* context;
  const int32_t* news;
  int32_t* table;
  const int32_t* free_blocks;
  const int32_t* taken;
  int32_t* cu_new;
  int32_t* seq_lens;
  int64_t* slots;
  int32_t* positions;
  int32_t* counts;
  int64_t ld_table;
  int64_t n_free;
  int64_t max_tokens;
  int32_t requests;
  int32_t width;
  int32_t block;
  int32_t shift;  // log2 of block, or -1
};

// Lengths are below 2^31, so positions fit 32 unsigned bits.
__device__ __forceinline__ uint32_t table_column(const TableArgs& p, uint32_t position) {
  return p.shift >= 0 ? position >> p.shift : position / static_cast<uint32_t>(p.block);
}
// Blocks that n tokens take, at most the table's width.
__device__ __forceinline__ int table_blocks(const TableArgs& p, uint32_t n) {
  const uint32_t whole = table_column(p, n);
  return static_cast<int>(min(whole + (whole * static_cast<uint32_t>(p.block) < n ? 1u : 0u),
                              static_cast<uint32_t>(p.width)));
}

__device__ __forceinline__ int32_t saturate_i32(int64_t v) {
  return static_cast<int32_t>(v > INT32_MAX ? INT32_MAX : v);
}

// Exclusive sums of (a, b) over the CTA; the totals come back in ta, tb.
__device__ __forceinline__ void scan_pair(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb,
                                          int64_t (*sm)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, a, o);
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  __syncthreads();  // the previous round's sums have been read
  if (lane == 31) {
    sm[warp][0] = a;
    sm[warp][1] = b;
  }
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kTableThreads / 32; ++w) {
    if (w < warp) {
      pa += sm[w][0];
      pb += sm[w][1];
    }
    ta += sm[w][0];
    tb += sm[w][1];
  }
  a += pa - a0;
  b += pb - b0;
}

__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const TableArgs p) {
  extern __shared__ int32_t sm_dyn[];
  __shared__ int64_t sm_scan[kTableThreads / 32][2];
  __shared__ int sm_lost;
  int32_t* cu = sm_dyn;                      // [requests + 1]
  int32_t* first = cu + p.requests + 1;      // [requests]: free-list index of column 0, were it fresh
  int32_t* ctxs = first + p.requests;        // [requests]
  const int tid = threadIdx.x;
  if (tid == 0) sm_lost = 0;

  pdl_wait();
  const int64_t taken = p.taken ? max(0, *p.taken) : 0;
  // consecutive requests a thread, one scan of the threads' sums
  const int each = (p.requests + kTableThreads - 1) / kTableThreads;
  const int r_lo = min(p.requests, tid * each), r_hi = min(p.requests, r_lo + each);
  int64_t t = 0, b = 0, base_t, base_b;
  for (int r = r_lo; r < r_hi; ++r) {
    const int ctx = max(0, p.context[r]), nw = max(0, p.news[r]);
    ctxs[r] = ctx;
    cu[r] = nw;
    t += nw;
    b += table_blocks(p, static_cast<uint32_t>(ctx) + nw) - table_blocks(p, ctx);
  }
  scan_pair(t, b, base_t, base_b, sm_scan);
  b += taken;
  base_b += taken;
  for (int r = r_lo; r < r_hi; ++r) {
    const int ctx = ctxs[r], nw = cu[r];
    const int held = table_blocks(p, ctx), need = table_blocks(p, static_cast<uint32_t>(ctx) + nw);
    cu[r] = saturate_i32(t);
    // clamped to the free list's end: beyond it every index is out of blocks
    first[r] = static_cast<int32_t>(min(b, p.n_free) - held);
    if (blockIdx.x == 0) {
      p.cu_new[r] = saturate_i32(t);
      const int64_t len = static_cast<int64_t>(ctx) + nw;
      p.seq_lens[r] = saturate_i32(len);
      const int64_t have = held + min(static_cast<int64_t>(need - held), max(static_cast<int64_t>(0), p.n_free - b));
      const int64_t lost = len - max(static_cast<int64_t>(ctx), min(len, have * p.block));
      if (lost > 0) atomicAdd(&sm_lost, saturate_i32(lost));
    }
    t += nw;
    b += need - held;
  }
  if (tid == 0) cu[p.requests] = saturate_i32(base_t);
  __syncthreads();
  pdl_trigger();
  if (blockIdx.x == 0 && tid == 0) {
    p.cu_new[p.requests] = saturate_i32(base_t);
    p.counts[0] = saturate_i32(base_t);
    p.counts[1] = saturate_i32(min(base_b, max(taken, p.n_free)));
    p.counts[2] = sm_lost;
  }

  // the tables' fresh columns: a warp a request
  const int lane = tid & 31;
  const int warps = static_cast<int>(gridDim.x) * (kTableThreads / 32);
  for (int r = blockIdx.x * (kTableThreads / 32) + (tid >> 5); r < p.requests; r += warps) {
    const int held = table_blocks(p, ctxs[r]);
    const int need = table_blocks(p, static_cast<uint32_t>(ctxs[r]) + (cu[r + 1] - cu[r]));
    for (int c = held + lane; c < need; c += 32) {
      const int64_t at = static_cast<int64_t>(first[r]) + c;
      p.table[r * p.ld_table + c] = at < p.n_free ? p.free_blocks[at] : -1;
    }
  }

  // the tokens, one a thread
  const int total = cu[p.requests];
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTableThreads;
  for (int64_t tk = static_cast<int64_t>(blockIdx.x) * kTableThreads + tid; tk < p.max_tokens; tk += stride) {
    int64_t slot = -1;
    int pos = 0;
    if (tk < total) {
      int r = 0, hi = p.requests;  // the last request with cu[r] <= tk: it has tokens
      for (int step = 0; step < 32 && hi - r > 1; ++step) {
        const int mid = (r + hi) >> 1;
        if (cu[mid] <= tk) r = mid;
        else hi = mid;
      }
      const uint32_t ctx = ctxs[r], at = ctx + static_cast<uint32_t>(tk - cu[r]);
      pos = saturate_i32(at);
      const uint32_t c = table_column(p, at);
      if (c < static_cast<uint32_t>(p.width)) {
        int64_t blk;
        if (c < static_cast<uint32_t>(table_blocks(p, ctx))) {
          blk = p.table[r * p.ld_table + c];
        } else {
          const int64_t f = static_cast<int64_t>(first[r]) + c;
          blk = f < p.n_free ? p.free_blocks[f] : -1;
        }
        if (blk >= 0) slot = blk * p.block + (at - c * static_cast<uint32_t>(p.block));
      }
    }
    p.slots[tk] = slot;
    p.positions[tk] = pos;
  }
}

}  // namespace i8
