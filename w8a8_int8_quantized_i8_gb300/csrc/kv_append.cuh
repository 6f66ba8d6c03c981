// kv_append.cuh -- new keys and values into a paged cache held in 8 bits, one
// scale for each block of tokens and head.
//
// The cache holds codes [blocks, heads, B, D] and scales [blocks, heads].  The
// step's tokens come with their slots (block * B + offset, negative: skipped).
// The tokens of one block follow one another, but for skipped ones, and have
// consecutive offsets: a "run" of `count` tokens from offset o, which spans
// `span` >= count tokens of the step.  A run appends: the block's first o tokens are older ones.  Per run, head
// and tensor, with L = 127 (int8) or 448 (E4M3):
//   m     = max |x| over the run's tokens
//   s_new = max(o > 0 ? s_old : 0, m / L)
//   older codes:  q' = rne(q * fl(s_old / s_new))   where s_new > s_old
//   new codes:    q  = rne(fl(x / s_new))           (0 where s_new is 0 or NaN)
// where a NaN wins a maximum: it makes the block's scale NaN until the block is
// begun again.
// A block whose scale does not grow keeps its codes, so appending a token
// costs that token only, except when it is the loudest of its block yet.
//
// Every run is handled by one warp (short runs, a decode step) or one CTA
// (long runs, a prefill), whole: no two CTAs write a block, no atomics.  A run
// of up to 4 vectors a thread stays in registers between the maximum and the
// codes; of a longer one the rest is read again (from L1 / L2).
//
// Finding the runs is a chain of short dependent steps, so the slots that they
// need go to shared memory first, in one load a thread.
//
// Bound by latency (slots, rows, maximum, codes): 128 tokens of 8 heads of 128
// take 4.6 us; 4767 tokens of prompts (29 MB) 15.7 us, in two waves of CTAs.
// 8 vectors a thread with 6 CTAs an SM, or 256 threads, measured no faster.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "quant.cuh"
#include "rmsnorm.cuh"

namespace i8 {

constexpr int kAppendThreads = 128;
constexpr int kAppendMaxWindow = 32;  // tokens a CTA looks for runs in
constexpr int kAppendShortRun = 8;    // runs up to this are one warp's work
constexpr int kAppendKeep = 4;        // vectors a thread keeps
constexpr int kAppendSlots = 256;     // slots in shared memory: the one before the window, then on

struct AppendSide {
  const uint16_t* src;        // bf16 [tokens, heads, D]
  int64_t ld_token, ld_head;  // elements between tokens and between heads
  uint8_t* codes;             // [blocks, heads, B, D]
  float* scale;               // [blocks, heads]
};

struct AppendArgs {
  AppendSide k, v;
  const int64_t* slots;
  int64_t tokens;
  int64_t blocks;
  int32_t heads;
  int32_t block;
  int32_t dim_shift;   // log2 of the head dimension
  int32_t window;
};

// Four int8 codes times a ratio <= 1, rounded back to int8 (ties to even).
__device__ __forceinline__ uint32_t rescale_s8x4(uint32_t w, float ratio) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
    b[i] = __float_as_uint(__fadd_rn(__fmul_rn(x, ratio), kRoundMagic));
  }
  return low_bytes4(b[0], b[1], b[2], b[3]);
}

// Two E4M3 codes (a 16-bit word) as fp32 values, exactly.
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t two, float& lo, float& hi) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(two)));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h2));
}
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float ratio) {
  float a, b, c, d;
  e4m3x2_to_f32(w & 0xFFFFu, a, b);
  e4m3x2_to_f32(w >> 16, c, d);
  return e4m3x2(__fmul_rn(a, ratio), __fmul_rn(b, ratio)) |
         (e4m3x2(__fmul_rn(c, ratio), __fmul_rn(d, ratio)) << 16);
}

// Lane-wise max of |a| and |b| over bf16 pairs, as absmax_bf16x2, but a NaN wins:
// it has to show in the block's scale, since an int8 code cannot hold it.
__device__ __forceinline__ uint32_t loudest_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

struct AppendRun {
  int64_t slot;  // of its first token
  int64_t at;    // its first token
  int64_t block;
  int off;       // its first offset in the block
  int span;
  int count;
};

// The step's slots: the window's neighbourhood from shared memory.
struct AppendSlots {
  const int64_t* all;
  const int64_t* near;  // [kAppendSlots] from token w0 - 1 on
  int64_t w0;
  __device__ __forceinline__ int64_t operator[](int64_t t) const {
    const int64_t i = t - w0 + 1;
    return i >= 0 && i < kAppendSlots ? near[i] : all[t];
  }
};

// The first token from t on that is not skipped, or T (the whole warp calls).
__device__ __forceinline__ int64_t next_token(const AppendSlots& slots, int64_t t, int64_t T,
                                              int lane) {
  for (; t < T; t += 256) {
    int first = 256;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      const int64_t u = t + 32 * j + lane;
      if (u < T && slots[u] >= 0) first = 32 * j + lane;
    }
    first = __reduce_min_sync(0xFFFFFFFFu, first);
    if (first < 256) return t + first;
  }
  return T;
}

// The slot of the last token before t that is not skipped, or -1 (the whole
// warp calls).
__device__ __forceinline__ int64_t slot_before(const AppendSlots& slots, int64_t t, int lane) {
  for (; t > 0; t -= 256) {
    int back = 256;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      const int64_t u = t - 1 - (32 * j + lane);
      if (u >= 0 && slots[u] >= 0) back = 32 * j + lane;
    }
    back = __reduce_min_sync(0xFFFFFFFFu, back);
    if (back < 256) return slots[t - 1 - back];
  }
  return -1;
}

// Extends a run from its first token to its last (the whole warp calls).
// Every round finds tokens of the run or ends, so there are at most `most`.
__device__ __forceinline__ void run_extent(const AppendSlots& slots, int64_t T, AppendRun& r,
                                           int most, int lane) {
  int64_t t = r.at + 1;
  for (int round = 0; round < most && r.count < most && t < T; ++round) {
    const bool goes_on = r.count + lane < most && t + lane < T &&
                         slots[t + lane] == r.slot + r.count + lane;
    const unsigned on = __ballot_sync(0xFFFFFFFFu, goes_on);
    const int n = __popc(on & ~(on + 1));  // the low ones of `on`
    r.count += n;
    t += n;
    if (n > 0) r.span = static_cast<int>(t - r.at);
    if (n == 32 || r.count == most) continue;
    if (t >= T || slots[t] >= 0) break;    // another block's token
    t = next_token(slots, t, T, lane);
    if (t >= T || slots[t] != r.slot + r.count) break;
  }
}

// One run for one head of one tensor, by `threads` consecutive threads of
// which this is number `me`: a warp (red == nullptr) or the CTA.
template <bool E4M3>
__device__ __forceinline__ void append_run(const AppendArgs& p, const AppendSide& a, int head,
                                           const AppendRun& run, int me, int threads,
                                           uint32_t* red) {
  const int64_t s0 = run.slot;
  const int64_t* slots = p.slots + run.at;
  const bool gaps = run.span != run.count;
  const int64_t blk = run.block;
  const int off = run.off;
  const int vs = p.dim_shift - 3;  // 16-byte vectors a token: 1 << vs
  const uint16_t* src = a.src + run.at * a.ld_token + head * a.ld_head;
  float* sp = a.scale + blk * p.heads + head;
  uint8_t* dst = a.codes + (((blk * p.heads + head) * p.block) << p.dim_shift);
  const float s_old = off > 0 ? *sp : 0.0f;

  uint32_t amax2 = 0;
  // (a run with many skipped tokens may span more vectors than 32 bits count)
  const int64_t n = static_cast<int64_t>(run.span) << vs;
  uint4 keep[kAppendKeep];
#pragma unroll
  for (int q = 0; q < kAppendKeep; ++q) {
    const int i = me + q * threads, t = i >> vs, c = i - (t << vs);
    keep[q] = make_uint4(0u, 0u, 0u, 0u);  // (skipped tokens and the run's end: nothing louder)
    if (i < n && !(gaps && slots[t] < 0))
      keep[q] = *reinterpret_cast<const uint4*>(src + t * a.ld_token + c * 8);
  }
#pragma unroll
  for (int q = 0; q < kAppendKeep; ++q) {
    amax2 = loudest_bf16x2(amax2, keep[q].x);
    amax2 = loudest_bf16x2(amax2, keep[q].y);
    amax2 = loudest_bf16x2(amax2, keep[q].z);
    amax2 = loudest_bf16x2(amax2, keep[q].w);
  }
#pragma unroll 4
  for (int64_t i = me + kAppendKeep * threads; i < n; i += threads) {
    const int t = static_cast<int>(i >> vs), c = static_cast<int>(i) & ((1 << vs) - 1);
    if (gaps && slots[t] < 0) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(src + t * a.ld_token + c * 8);
    amax2 = loudest_bf16x2(amax2, v.x);
    amax2 = loudest_bf16x2(amax2, v.y);
    amax2 = loudest_bf16x2(amax2, v.z);
    amax2 = loudest_bf16x2(amax2, v.w);
  }
  amax2 &= 0x7FFF7FFFu;
  uint32_t abits = __reduce_max_sync(0xFFFFFFFFu, max(amax2 & 0xFFFFu, amax2 >> 16));
  if (red) {
    __syncthreads();  // the previous run's maxima have been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = abits;
    __syncthreads();
    abits = 0;
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) abits = max(abits, red[w]);
  } else {
    __syncwarp();
  }
  const float s_run = __fdiv_rn(__uint_as_float(abits << 16), E4M3 ? 448.0f : 127.0f);
  const float s = max_or_nan(s_old, s_run);
  if (me == 0) *sp = s;  // every thread has read s_old before the barrier above
  if (s > s_old && off > 0) {
    const float ratio = __fdiv_rn(s_old, s);
    uint2* old = reinterpret_cast<uint2*>(dst);
    for (int i = me; i < off << vs; i += threads) {
      uint2 w = old[i];
      w.x = E4M3 ? rescale_e4m3x4(w.x, ratio) : rescale_s8x4(w.x, ratio);
      w.y = E4M3 ? rescale_e4m3x4(w.y, ratio) : rescale_s8x4(w.y, ratio);
      old[i] = w;
    }
  }
  const bool fast = s >= 0x1p-126f;
  const float r = __frcp_rn(s);
  const unsigned long long rr = f2(r, r);
  uint2* out = reinterpret_cast<uint2*>(dst + (off << p.dim_shift));
  auto code = [&](int64_t i, const uint4& v) {
    const int t = static_cast<int>(i >> vs);
    int to = static_cast<int>(i);
    if (gaps) {
      if (slots[t] < 0) return;
      to = (static_cast<int>(slots[t] - s0) << vs) + (static_cast<int>(i) & ((1 << vs) - 1));
    }
    uint2 w = make_uint2(0u, 0u);
    if (s > 0.0f) {
      if constexpr (E4M3) {
        const float x[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                            bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
        w = quant_f32x8_e4m3(x, s, r, fast);
      } else {
        w = quant_vec8(v, s, rr, fast);
      }
    }
    out[to] = w;
  };
#pragma unroll
  for (int q = 0; q < kAppendKeep; ++q)
    if (me + q * threads < n) code(me + q * threads, keep[q]);
  for (int64_t i = me + kAppendKeep * threads; i < n; i += threads) {
    const int t = static_cast<int>(i >> vs), c = static_cast<int>(i) & ((1 << vs) - 1);
    if (gaps && slots[t] < 0) continue;
    code(i, *reinterpret_cast<const uint4*>(src + t * a.ld_token + c * 8));
  }
}

// grid (windows of tokens, 2 * heads).
template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, 8) kv_append_kernel(const AppendArgs p) {
  __shared__ uint32_t red[kAppendThreads / 32];
  __shared__ AppendRun run[kAppendMaxWindow];
  __shared__ int n_runs;
  __shared__ int64_t near[kAppendSlots];
  const bool values = blockIdx.y & 1;
  const int head = blockIdx.y >> 1;
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * p.window;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  pdl_wait();
  for (int i = threadIdx.x; i < kAppendSlots; i += kAppendThreads) {
    const int64_t t = w0 - 1 + i;
    near[i] = t >= 0 && t < p.tokens ? p.slots[t] : -1;
  }
  __syncthreads();
  // warp 0 finds the runs that start in this window: lane j looks at token j
  if (warp == 0) {
    const AppendSlots slots{p.slots, near, w0};
    const int64_t t = w0 + lane;
    bool starts = false;
    int64_t s = -1, blk = 0;
    if (lane < p.window && t < p.tokens) s = near[lane + 1];
    // the slot of the last token before it that is not skipped: a lane's of the
    // window, or for the first one what lies before the window
    int64_t before = near[lane];
    if (__any_sync(0xFFFFFFFFu, s >= 0 && before < 0)) {
      const unsigned held = __ballot_sync(0xFFFFFFFFu, s >= 0);
      const unsigned earlier = held & ((1u << lane) - 1u);
      const int64_t inside = __shfl_sync(0xFFFFFFFFu, s, earlier ? 31 - __clz(earlier) : 0);
      const int64_t outside = slot_before(slots, w0, lane);
      before = earlier ? inside : outside;
    }
    if (s >= 0) {
      blk = s / p.block;
      starts = true;
      if (before >= 0 && before >= blk * p.block && before < (blk + 1) * p.block) {
        starts = false;  // inside a run
        if (before + 1 != s) atomicOr(&g_status, 1u << 7);  // out of order: not written
      }
      if (starts && blk >= p.blocks) {
        starts = false;
        atomicOr(&g_status, 1u << 7);
      }
    }
    const unsigned mask = __ballot_sync(0xFFFFFFFFu, starts);
    int i = 0;
    for (unsigned left = mask; left != 0; left &= left - 1, ++i) {
      const int at = __ffs(left) - 1;
      AppendRun r;
      r.slot = __shfl_sync(0xFFFFFFFFu, s, at);
      r.block = __shfl_sync(0xFFFFFFFFu, blk, at);
      r.off = static_cast<int>(r.slot - r.block * p.block);
      r.at = w0 + at;
      r.span = r.count = 1;
      run_extent(slots, p.tokens, r, p.block - r.off, lane);
      if (lane == 0) run[i] = r;
    }
    if (lane == 0) n_runs = __popc(mask);
  }
  __syncthreads();
  pdl_trigger();
  const int runs = n_runs;
  AppendSide a;
  a.src = values ? p.v.src : p.k.src;
  a.ld_token = values ? p.v.ld_token : p.k.ld_token;
  a.ld_head = values ? p.v.ld_head : p.k.ld_head;
  a.codes = values ? p.v.codes : p.k.codes;
  a.scale = values ? p.v.scale : p.k.scale;
  // the short runs first, a warp each, then the long ones, the CTA together:
  // one call of append_run for both, so that it is in the code once
  bool solo = true;
  int i = warp;
  for (int step = 0; step < 2 * kAppendMaxWindow + 2; ++step) {
    for (; i < runs && (run[i].span <= kAppendShortRun) != solo;) i += solo ? kAppendThreads / 32 : 1;
    if (i >= runs) {
      if (!solo) break;
      solo = false;
      i = 0;
      continue;
    }
    append_run<E4M3>(p, a, head, run[i], solo ? lane : threadIdx.x, solo ? 32 : kAppendThreads,
                     solo ? nullptr : red);
    i += solo ? kAppendThreads / 32 : 1;
  }
}

}  // namespace i8
