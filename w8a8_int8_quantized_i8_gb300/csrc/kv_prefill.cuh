// kv_prefill.cuh -- the paged attention of kv_attention.cuh for requests with
// many rows (chunks of prompts), on the tensor cores of tcgen05.
//
// The same formula and cache.  An item is 256 rows of a request (new token x
// query head of one kv head, token-major) as two tiles of 128; a CTA goes over
// its keys 128 tokens at a time:
//   S_t = Q_t K^T  -> TMEM      (fp16 x fp16, exact products, fp32 sums)
//   P_t = 2^(s + log2 sv - R)   softmax threads, P back to TMEM
//   O_t += P_t V   -> TMEM      (A operand from TMEM, V as it lies: N-major)
// with s = S * sk * scale * log2 e and sv, sk the block's scales.  The two
// tiles take turns: while one tile's softmax runs, the tensor cores do the
// other's O and next S.
//
// Codes are converted to fp16, exactly, once a CTA and serve all 256 rows.  q is
// scaled per row by a power of two as in kv_attention.cuh.  R is a row's running
// maximum of s + log2 sv, the log of a term's weight in O; it moves only when it
// grows by more than 8 (2^8 in weight), so that O in TMEM is rarely rescaled,
// and P, held in fp16 as 2^(6 + s + log2 sv - R), stays below 2^14.  The sum of
// exponentials is kept in fp32 beside it, each 16 tokens' sum of P times
// 2^(Lr - log2 sv), Lr a segment's fixed reference; from the first tile on that
// holds a log2 sv further than 40 from Lr, or a block of zeros, it has a maximum X
// of its own, as in kv_attention.cuh.
//
// Bound by a row tile's chain: S, softmax (about 2400 cycles and the barriers
// around it), P, O.  TMEM is full, so a tile has one S buffer and its next S
// waits for its P to be used; the two tiles in turn take about 4700 cycles a
// tile of keys, of which the products take 2950 (2048 at the nominal rate: S
// reads both operands from shared memory, which the conversion uses too).  Four
// requests, 5357 new tokens, contexts to 8000, 32 query and 8 kv heads of 128:
// 560 us, 46 % of the measured bf16 rate (warp MMA: 4224 us).  Two softmax
// threads a row against one: 510 against 543 us; 8 converting warps against 6:
// 528 against 510.
//
// Every CTA stays and takes an equal share of the line of all items' tiles, as
// in kv_attention.cuh; cut items meet in a join.
//
// Roles: warps 0-15 softmax (tile = warp / 8; a row has two threads, each for
// half of the keys, which agree on R once a tile; a warp reads the 32 TMEM
// lanes of its place in the warpgroup), warp 16 copies by TMA and prepares the
// scales, warp 17 issues the MMAs, warps 18-23 convert.  At 128 head dimensions
// 208 KB of shared memory (Q 64, three fp16 tiles 96, three tiles of codes 48)
// and all of TMEM (S 2 x 128, O 2 x 128 columns): one CTA an SM.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "kv_attention.cuh"
#include "ptx.cuh"

namespace i8 {

constexpr int kPreThreads = 768;
constexpr int kPreSoftWarps = 16;
constexpr int kPreRows = 256;      // rows of an item
constexpr int kPreTokens = 128;    // tokens of a tile of keys
constexpr int kPreConvWarps = 6;
constexpr int kPreSlots = 3;       // stages of codes, and of fp16 tiles
constexpr int kPreScales = 4;      // stages of block scales
constexpr int kPreGranules = kPreTokens / 16;
constexpr int kPreJoinRows = 8;    // rows of an item that a CTA of the join takes

template <int D>
struct PrefillSmem {
  static constexpr int SUB = D / 64;                    // 64 head dimensions, 128 bytes a row
  static constexpr int TILE = SUB * 128 * 128;          // 128 rows in fp16
  static constexpr int RAW = kPreTokens * D;
  static constexpr int Q = 0;
  static constexpr int KV = 2 * TILE;
  static constexpr int CODES = KV + kPreSlots * TILE;
  static constexpr int BYTES = CODES + kPreSlots * RAW;
};

struct PrefillScales {   // of the 16-token granules of a tile, and its place
  float k[kPreGranules];
  float lv[kPreGranules];     // log2 of V's
  float back[kPreGranules];   // 2^(Lr - lv), or 0 where `far`
  float ref;                  // Lr
  int far;                    // the segment's lv has left Lr's neighbourhood
  int there;                  // a bit for each granule that holds tokens
  int ends;                   // it is a segment's last
  int at;                     // its first token
  int tokens;                 // tokens that some row of the item sees
  int strange;                // there are places that not every row sees
};

// The part of an item in a CTA's share, written down by the warp that copies:
// the softmax threads have no registers to spare for finding it themselves.
struct PrefillSegment {
  int q0, fresh, pos0, len;  // of the request
  int head, row0;
  int first, last, n;      // its units, of the item's n
  int64_t item_u;          // the item's first unit
  int nan;                 // NaN codes were taken out of its values
};
constexpr int kPreSegments = 8;  // stages of them: the copies run at most three tiles ahead

// Where a CTA stands in the line of all items' tiles of keys (the units).  An
// item's keys end with its last row's; its row tiles go from the last to the
// first, head after head, request after request.
struct PrefillCursor {
  AttnRequest rq;
  int req, head, tile, n;     // the item and its units
  int64_t item_u;             // its first unit
};

// The tokens that a row tile sees.
__device__ __forceinline__ int prefill_end(const AttnRequest& rq, int group, int tile) {
  const int last = min((tile + 1) * kPreRows, rq.fresh * group) - 1;
  return min(max(rq.pos0 + last / group + 1, 0), rq.len);
}
// Units of a row tile: one even where it sees nothing.
__device__ __forceinline__ int prefill_units(const AttnRequest& rq, int group, int tile) {
  return max(1, (prefill_end(rq, group, tile) + kPreTokens - 1) / kPreTokens);
}
__device__ __forceinline__ AttnRequest prefill_request(const AttnArgs& p, int r) {
  AttnRequest rq = attn_request<kPreRows, kPreTokens>(p, r);
  const int group = p.q_heads / p.kv_heads;
  rq.units = 0;
  if (static_cast<int64_t>(rq.fresh) * group < p.split_rows) rq.tiles = 0;
  for (int t = 0; t < rq.tiles; ++t) rq.units += prefill_units(rq, group, t);
  rq.units *= p.kv_heads;
  return rq;
}
// Moves the cursor to the item that holds unit u, at or behind the cursor's.
__device__ __forceinline__ void prefill_seek(const AttnArgs& p, PrefillCursor& c, int64_t u) {
  const int group = p.q_heads / p.kv_heads;
  for (; u >= c.item_u + c.n;) {
    c.item_u += c.n;
    if (--c.tile < 0) {
      if (++c.head == p.kv_heads) {
        c.head = 0;
        for (++c.req; c.req < p.requests; ++c.req) {  // (a unit behind it: there is one)
          c.rq = prefill_request(p, c.req);
          if (c.rq.tiles > 0) break;
        }
      }
      c.tile = c.rq.tiles - 1;
    }
    c.n = prefill_units(c.rq, group, c.tile);
  }
}

// An N-major (transposed) operand stored with the 128-byte swizzle: rows of
// 128 bytes (64 values along N) for each k, 8-row groups 1024 bytes apart along
// K, 64-value groups `n_stride` bytes apart along N.
__device__ __forceinline__ uint64_t smem_desc_sw128_n(uint32_t saddr, uint32_t n_stride) {
  uint64_t d = smem_desc_sw128(saddr) & ~(static_cast<uint64_t>(0x3FFFu) << 16);
  return d | (static_cast<uint64_t>(n_stride >> 4) << 16);
}

// A product of 128 rows, kind::f16, one CTA: D[tmem] (+)= A * B[smem]^T over
// D / 16 steps of K (A in shared memory, both K-major in 64-value groups 16 KB
// apart) or over 8 (A in TMEM, B N-major); and the commit that arrives on `bar`
// when what was issued is done.  The whole warp calls, its elected lane (the
// same one every time) issues: in converged code, and a product in one piece,
// the operands stay in the uniform registers that the instruction wants.
// Issued step by step from a lane's own branch a product took 980 cycles
// instead of 512.
#define I8_MMA_SS(OFF, P)                                                                  \
  "add.s64 a, %1, " OFF ";\n\tadd.s64 b, %2, " OFF ";\n\t"                                \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " P ";\n\t"
#define I8_MMA_TS(OFF_A, OFF_B, P)                                                         \
  "add.s32 a, %1, " OFF_A ";\n\tadd.s64 b, %2, " OFF_B ";\n\t"                            \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, " P ";\n\t"
template <int D>
__device__ __forceinline__ void mma_product_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                               uint32_t idesc) {
  if constexpr (D == 128)
    asm volatile("{\n\t.reg .pred n, y, q;\n\t.reg .b64 a, b;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
                 "setp.ne.u32 n, 0, 0;\n\tsetp.eq.u32 y, 0, 0;\n\t"
                 I8_MMA_SS("0", "n") I8_MMA_SS("2", "y") I8_MMA_SS("4", "y") I8_MMA_SS("6", "y")
                 I8_MMA_SS("1024", "y") I8_MMA_SS("1026", "y") I8_MMA_SS("1028", "y")
                 I8_MMA_SS("1030", "y") "}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred n, y, q;\n\t.reg .b64 a, b;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
                 "setp.ne.u32 n, 0, 0;\n\tsetp.eq.u32 y, 0, 0;\n\t"
                 I8_MMA_SS("0", "n") I8_MMA_SS("2", "y") I8_MMA_SS("4", "y") I8_MMA_SS("6", "y")
                 "}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc)
                 : "memory");
}
__device__ __forceinline__ void mma_product_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                               uint32_t idesc, bool accumulate) {
  asm volatile("{\n\t.reg .pred n, y, q;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
               "setp.ne.u32 n, %4, 0;\n\tsetp.eq.u32 y, 0, 0;\n\t"
               I8_MMA_TS("0", "0", "n") I8_MMA_TS("8", "128", "y") I8_MMA_TS("16", "256", "y")
               I8_MMA_TS("24", "384", "y") I8_MMA_TS("32", "512", "y") I8_MMA_TS("40", "640", "y")
               I8_MMA_TS("48", "768", "y") I8_MMA_TS("56", "896", "y") "}" ::"r"(d_tmem),
               "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
               : "memory");
}
#undef I8_MMA_SS
#undef I8_MMA_TS
__device__ __forceinline__ void mma_commit_warp(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Waits for the tcgen05.ld that fills r; naming the registers keeps their uses
// behind the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ unsigned long long f2_fma(unsigned long long a, unsigned long long b,
                                                     unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 lanes x 16 consecutive 32-bit columns, to and from the warp's registers.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void sts_16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kPreThreads, 1)
    kv_prefill_kernel(const AttnArgs p, const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map) {
  using Sm = PrefillSmem<D>;
  constexpr int PIECE = kPreRows * (D + 2);
  extern __shared__ uint8_t sm_pre[];
  __shared__ __align__(8) uint64_t raw_full[kPreSlots], raw_empty[kPreSlots], kv_full[kPreSlots],
      kv_empty[kPreSlots], sc_full[kPreScales], s_full[2], p_full[2], sum_full[2], q_full,
      o_full, drained;
  __shared__ PrefillScales sc[kPreScales];
  __shared__ PrefillSegment segs[kPreSegments];
  // the first token with a NaN code, of those taken out, by head dimension
  __shared__ int first_nan[E4M3 ? kPreSegments : 1][E4M3 ? D : 1];
  __shared__ float sm_top[2][2][128], sm_sum[2][2][128];  // [tile][half of the keys][row]
  __shared__ int64_t sm_scan[kAttnWarps], sm_base;
  __shared__ int sm_req;
  __shared__ uint32_t sm_tmem;
  __shared__ int abort_flag;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int group = p.q_heads / p.kv_heads;
  const uint32_t base = (smem_u32(sm_pre) + 1023u) & ~1023u;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kPreSlots; ++i) {
      mbar_init(smem_u32(&raw_full[i]), 1);
      mbar_init(smem_u32(&raw_empty[i]), kPreConvWarps);
      mbar_init(smem_u32(&kv_full[i]), kPreConvWarps);
      mbar_init(smem_u32(&kv_empty[i]), 1);
    }
    for (int i = 0; i < kPreScales; ++i) mbar_init(smem_u32(&sc_full[i]), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), kPreSoftWarps / 2);
      mbar_init(smem_u32(&sum_full[i]), kPreSoftWarps / 2);
    }
    mbar_init(smem_u32(&q_full), kPreSoftWarps);
    mbar_init(smem_u32(&o_full), 2);
    mbar_init(smem_u32(&drained), 1);
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
    fence_mbarrier_init();
  }

  pdl_wait();
  // ---- this CTA's share of the units
  int64_t mine = 0, total, before = 0;
  const int chunk = (p.requests + kAttnThreads - 1) / kAttnThreads;
  const int r_lo = min(p.requests, static_cast<int>(threadIdx.x) * chunk);
  const int r_hi = min(p.requests, r_lo + chunk);
  if (threadIdx.x < kAttnThreads)
    for (int r = r_lo; r < r_hi; ++r) mine += prefill_request(p, r).units;
  {
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (warp < kAttnWarps && lane == 31) sm_scan[warp] = x;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      if (w < warp) before += sm_scan[w];
      total += sm_scan[w];
    }
    before += x - mine;
  }
  const int64_t workers = min(total, static_cast<int64_t>(gridDim.x));
  if (threadIdx.x == 0) p.cut[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (blockIdx.x >= workers) return;  // (the whole CTA)
  const int64_t u_begin = blockIdx.x * total / workers;
  const int64_t u_end = (blockIdx.x + 1) * total / workers;
  const int tiles = static_cast<int>(u_end - u_begin);
  if (threadIdx.x < kAttnThreads && before <= u_begin && u_begin < before + mine) {
    int r = r_lo;
    for (; r < r_hi - 1; ++r) {
      const int64_t n = prefill_request(p, r).units;
      if (u_begin < before + n) break;
      before += n;
    }
    sm_req = r;
    sm_base = before;
  }
  if (warp == kPreSoftWarps + 1) {
    tmem_alloc(smem_u32(&sm_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm_tmem;
  // the first item: over the request's heads that lie before it at once
  auto first_item = [&](PrefillCursor& c) {
    c.req = sm_req;
    c.rq = prefill_request(p, c.req);
    const int64_t per_head = c.rq.units / p.kv_heads;
    c.head = static_cast<int>((u_begin - sm_base) / per_head);
    c.item_u = sm_base + c.head * per_head;
    c.tile = c.rq.tiles - 1;
    c.n = prefill_units(c.rq, group, c.tile);
    prefill_seek(p, c, u_begin);
  };

  int copied = 0;  // tiles of K or V whose copies the copying warp has begun
  if (warp < kPreSoftWarps) {
    // =================================================================== softmax
    regs_inc<96>();
    const int t = warp >> 3, half = (warp >> 2) & 1;
    const int r = (warp & 3) * 32 + lane;  // row of the tile
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t s_at = tmem + lanes + t * 128 + half * 64;  // this half's S
    const uint32_t p_at = tmem + lanes + t * 128 + half * 32;  // and P
    const uint32_t o_at = tmem + lanes + 256 + t * D + half * (D / 2);
    bool ok = true;
    int jt = 0;  // tiles done
    // whatever happens, every warp of the tile passes its barrier `tiles` times
#pragma unroll 1
    for (int seg = 0; jt < tiles; ++seg) {
      // the first tile's scales say that the segment is written down
      ok = __all_sync(0xFFFFFFFFu,
                      ok && mbar_wait(smem_u32(&sc_full[jt & 3]), (jt >> 2) & 1, &abort_flag));
      if (!ok) {
        for (; jt < tiles; ++jt) named_bar_sync(1 + t, 256);
        break;
      }
      const PrefillSegment& sg = segs[seg & (kPreSegments - 1)];
      const int first = sg.first, last = sg.last;
      const int row = sg.row0 + t * 128 + r;
      const bool real = row < sg.fresh * group;
      const int i = real ? row / group : 0;
      float rowfac;
      {
        // q's row: its power of two, then this thread's half in fp16 into the
        // swizzled tile (which the segment before has been done with since its
        // o_full)
        const int hq = sg.head * group + (real ? row - i * group : 0);
        const uint4* qp = reinterpret_cast<const uint4*>(
            p.q + (static_cast<int64_t>(sg.q0) + i) * p.ldq_token + hq * p.ldq_head);
        uint32_t amax = 0;
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = real ? qp[c] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a = x[k] & 0x7FFF7FFFu;
            amax = max(amax, max(a & 0xFFFFu, a >> 16));
          }
        }
        const int e = 14 - max(static_cast<int>(amax >> 7) - 127, -100);
        float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        rowfac = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * fabsf(p.scale_log2);
        if (p.scale_log2 < 0.0f) up = -up;  // the factor of S is never negative
        const uint32_t to = base + Sm::Q + t * Sm::TILE + r * 128;
#pragma unroll 4
        for (int c = half * (D / 16); c < (half + 1) * (D / 16); ++c) {
          const uint4 w = real ? qp[c] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = pack_f16x2(__uint_as_float(x[k] << 16) * up, __uint_as_float(x[k] & 0xFFFF0000u) * up);
          sts_16(to + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&q_full));
      }
      const int limit =
          real ? min(max(sg.pos0 + i + 1, 0), sg.len) : 0x7FFFFFFF;
      float R = -INFINITY, l = 0.0f, Lr = 0.0f, X = -INFINITY;
      int j = first;
      // the segment's tiles; without FAR, up to the first one that is far (two
      // loops, so that the usual one pays nothing for the other)
      auto go_over = [&](auto kind) {
      constexpr bool FAR = decltype(kind)::value;
#pragma unroll 1
      for (; j < last; ++j, ++jt) {
        ok = ok && mbar_wait(smem_u32(&sc_full[jt & 3]), (jt >> 2) & 1, &abort_flag) &&
             mbar_wait(smem_u32(&s_full[t]), jt & 1, &abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) {  // given up: only keep the tile's barrier company
          named_bar_sync(1 + t, 256);
          continue;
        }
        tc_fence_after();
        const PrefillScales& z = sc[jt & 3];
        if (!FAR && j == first) Lr = z.ref;
        const int seen = limit - j * kPreTokens - 64 * half;  // columns below this are seen
        const bool masked = __any_sync(0xFFFFFFFFu, seen < 64 || (!FAR && z.far));
        if constexpr (FAR) {
          // this thread's exponentials by themselves: their maximum, their sum
          float x = X, sum = 0.0f;
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const int gr = 4 * half + (g & 3);
            const int lim = (z.there >> gr) & 1 ? seen - 16 * (g & 3) : 0;
            const float f = z.k[gr] * rowfac;
            uint32_t v[16];
            tmem_ld_32x32b_x16(s_at + 16 * (g & 3), v);
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float y = k < lim ? __uint_as_float(v[k]) * f : -INFINITY;
              if (g < 4) x = fmaxf(x, y);
              else sum += ex2(y - exp_ref(x));
            }
          }
          l = fmaf(l, ex2(X - exp_ref(x)), sum);
          X = x;
        }
        uint32_t s[2][32];
        tmem_ld_32x32b_x32(s_at, s[0]);
        tmem_ld_32x32b_x32(s_at + 32, s[1]);
        tmem_wait_ld(s[0]);
        tmem_wait_ld(s[1]);
        if (!FAR && masked && z.far) return;
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t* v = &s[g >> 1][16 * (g & 1)];
          const float f = z.k[4 * half + g] * rowfac, b = z.lv[4 * half + g];
          if (masked) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float x = fmaf(__uint_as_float(v[k]), f, b);
              top = fmaxf(top, 16 * g + k < seen ? x : -INFINITY);
            }
          } else {
            float x = max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
            float y = max3(__uint_as_float(v[3]), __uint_as_float(v[4]), __uint_as_float(v[5]));
#pragma unroll
            for (int k = 6; k < 14; k += 4) {
              x = max3(x, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
              y = max3(y, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
            }
            x = max3(x, __uint_as_float(v[14]), __uint_as_float(v[15]));
            top = fmaxf(top, fmaf(fmaxf(x, y), f, b));
          }
        }
        // the row's two threads agree on the maximum.  Both have read their S
        // after the barrier, so that either may overwrite any of it with P.
        sm_top[t][half][r] = top;
        named_bar_sync(1 + t, 256);
        top = fmaxf(top, sm_top[t][half ^ 1][r]);
        float alpha = 1.0f;
        if (top > R + 8.0f) {  // (-inf + 8 is -inf)
          alpha = ex2(R - top);
          R = top;
          if (!FAR) l *= alpha;
        }
        if (__any_sync(0xFFFFFFFFu, alpha != 1.0f) && j > first) {
          // S of this tile was committed after the last product into O, so O
          // is complete; each thread rescales its half of the head dimensions
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_at + 16 * q, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st_32x32b_x16(o_at + 16 * q, o);
          }
        }
        const float ref = exp_ref(R) - 6.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint32_t* v = &s[q][16 * g];
            const int gr = 4 * half + 2 * q + g;
            const float f = z.k[gr] * rowfac, b = z.lv[gr] - ref;
            const unsigned long long ff = f2(f, f), bb = f2(b, b);
            unsigned long long sum[2];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float e0, e1;
              f2_split(f2_fma(f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), ff, bb), e0, e1);
              if (masked) {
                e0 = 32 * q + 16 * g + k < seen ? e0 : -INFINITY;
                e1 = 32 * q + 16 * g + k + 1 < seen ? e1 : -INFINITY;
              }
              e0 = ex2(e0);
              e1 = ex2(e1);
              const unsigned long long e = f2(e0, e1);
              sum[(k >> 1) & 1] = k < 4 ? e : f2_add(sum[(k >> 1) & 1], e);
              pk[8 * g + (k >> 1)] = pack_f16x2(e0, e1);
            }
            float s0, s1;
            f2_split(f2_add(sum[0], sum[1]), s0, s1);
            if constexpr (!FAR) l = fmaf(s0 + s1, z.back[gr], l);
          }
          tmem_st_32x32b_x16(p_at + 16 * q, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[t]));
      }
      };
      go_over(std::false_type{});
      X = R - 6.0f - Lr;  // l is the sum of 2^(s - X)
      if (j < last) go_over(std::true_type{});
      // ---- out: each thread its half of the head dimensions
      sm_sum[t][half][r] = attn_log(X, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sum_full[t]));
      ok = ok && mbar_wait(smem_u32(&sum_full[t]), seg & 1, &abort_flag) &&
           mbar_wait(smem_u32(&o_full), seg & 1, &abort_flag);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok) {
        tc_fence_after();
        const float l0 = sm_sum[t][0][r], l1 = sm_sum[t][1][r], most = fmaxf(l0, l1);
        const float L = attn_log(most, ex2(l0 - exp_ref(most)) + ex2(l1 - exp_ref(most)));
        const int hq = sg.head * group + (real ? row - i * group : 0);
        const int64_t token = static_cast<int64_t>(sg.q0) + i;
        const bool whole = first == 0 && last == sg.n;
        const float fac = attn_factor(exp_ref(R) - 6.0f, L);
        uint16_t* to = p.out + token * p.ldo_token + hq * p.ldo_head + half * (D / 2);
        // a piece of an item begun earlier goes to the first slot, of one that
        // goes on to the second
        float* piece = p.pieces + (2 * static_cast<int64_t>(blockIdx.x) + (first == 0 ? 1 : 0)) * PIECE;
        float* part = piece + (t * 128 + r) * D + half * (D / 2);
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[16];
          tmem_ld_32x32b_x16(o_at + 16 * q, o);
          tmem_wait_ld(o);
          if (E4M3 && sg.nan) {
            const int* at = first_nan[seg & (kPreSegments - 1)] + half * (D / 2) + 16 * q;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (limit > at[k]) o[k] = 0x7FFFFFFFu;  // the row sees it
          }
          if (whole && real) {
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
              uint32_t y[4];
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const float lo = __uint_as_float(o[k + 2 * m]) * fac * fac;
                const float hi = __uint_as_float(o[k + 2 * m + 1]) * fac * fac;
                const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
                y[m] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(to + 16 * q + k) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (!whole) {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<uint4*>(part + 16 * q + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        if (half == 0) {
          if (!whole) {
            piece[kPreRows * D + 2 * (t * 128 + r)] = R;
            piece[kPreRows * D + 2 * (t * 128 + r) + 1] = L;
          } else if (real && p.lse) {
            p.lse[token * p.q_heads + hq] = L * 0.69314718055994531f;
          }
        }
        if (!whole && first == 0 && threadIdx.x == 0) {
          // the worker that holds the item's last unit
          const int64_t w_end = ((sg.item_u + sg.n) * workers - 1) / total;
          p.cut[2 * blockIdx.x] = make_int4(static_cast<int>(w_end), sg.head, sg.row0, sg.fresh * group);
          p.cut[2 * blockIdx.x + 1] = make_int4(sg.q0, 0, 0, 0);
        }
      }
      tc_fence_before();
    }
  } else {
    regs_dec<48>();
    if (warp == kPreSoftWarps) {
      // ================================================================= copies
      const int boxes = kPreTokens / p.box_rows;
      PrefillCursor cur;
      first_item(cur);
      int item = 0, jt = 0, seg = -1;
      float ref = 0.0f;
      bool far = false, ok = true;
#pragma unroll 1
      for (int64_t u = u_begin; u < u_end && ok; ++u, ++jt) {
        prefill_seek(p, cur, u);
        const int j = static_cast<int>(u - cur.item_u);
        const int end = prefill_end(cur.rq, group, cur.tile);
        const int32_t* table = p.table + cur.req * p.ld_table;
        const bool begins = u == u_begin || j == 0, ends = u + 1 == u_end || j + 1 == cur.n;
        // scales, a lane a granule
        float sk = 0.0f, lv = -INFINITY;  // (-inf: no tokens, or a block of zeros)
        bool there = false;
        if (lane < kPreGranules) {
          const int tk = j * kPreTokens + 16 * lane;
          if (tk < end) {
            const int64_t blk = table[tk / p.block];  // end lies within the table's width
            if (blk >= 0 && blk < p.blocks) {
              sk = scale_value(p.k_scale[blk * p.kv_heads + cur.head]);
              const float sv = p.v_scale[blk * p.kv_heads + cur.head];
              lv = log2f(sv);
              there = true;
            } else {
              atomicOr(&g_status, 1u << 7);
            }
          }
        }
        if (begins) {
          float x = lv;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
          x = __shfl_sync(0xFFFFFFFFu, x, 0);
          ref = x > -INFINITY ? x : 0.0f;
          far = false;
          ++seg;
          if (lane == 0)
            segs[seg & (kPreSegments - 1)] = {
                cur.rq.q0, cur.rq.fresh, cur.rq.pos0, cur.rq.len, cur.head, cur.tile * kPreRows, j,
                static_cast<int>(min(static_cast<int64_t>(cur.n), u_end - cur.item_u)), cur.n, cur.item_u, 0};
          if constexpr (E4M3)
            for (int d = lane; d < D; d += 32) first_nan[seg & (kPreSegments - 1)][d] = 0x7FFFFFFF;
        }
        const unsigned held = __ballot_sync(0xFFFFFFFFu, there);
        far = far || __any_sync(0xFFFFFFFFu, there && !(fabsf(lv - ref) <= 40.0f));
        PrefillScales& z = sc[jt & 3];
        if (lane < kPreGranules) {
          z.k[lane] = sk;
          z.lv[lane] = lv;
          z.back[lane] = !there || far ? 0.0f : ex2(ref - lv);
        }
        if (lane == 0) {
          z.ref = ref;
          z.ends = ends;
          z.far = far;
          z.there = static_cast<int>(held);
          z.at = j * kPreTokens;
          z.tokens = min(end - j * kPreTokens, kPreTokens);
          const int least = cur.rq.pos0 + cur.tile * kPreRows / group + 1;  // what the first row sees
          z.strange = held != (1u << kPreGranules) - 1u || (j + 1) * kPreTokens > min(least, end);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sc_full[jt & 3]));
        // the codes, a lane a box
        const int tb = j * kPreTokens + lane * p.box_rows;
        int64_t blk = -1;
        int off = 0;
        if (lane < boxes && tb < end) {
          const int col = tb / p.block;
          off = tb - col * p.block;
          blk = table[col];
          if (blk >= p.blocks) blk = -1;
        }
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, blk >= 0)) * p.box_rows * D;
#pragma unroll
        for (int side = 0; side < 2; ++side, ++item) {
          const int slot = item % kPreSlots, round = item / kPreSlots;
          if (round > 0) ok = mbar_wait(smem_u32(&raw_empty[slot]), (round - 1) & 1, &abort_flag);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          const uint32_t bar = smem_u32(&raw_full[slot]);
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (blk >= 0)
            tma_load_3d(base + Sm::CODES + slot * Sm::RAW + lane * p.box_rows * D,
                        side ? static_cast<const void*>(&v_map) : &k_map, bar, 0, off,
                        static_cast<int>(blk) * p.kv_heads + cur.head);
        }
      }
      copied = item;
    } else if (warp == kPreSoftWarps + 1) {
      // ================================================================= products
      constexpr uint32_t kIdS = idesc_f16_f32(128, kPreTokens);
      constexpr uint32_t kIdO = idesc_f16_f32(128, D) | (1u << 16);  // B is N-major
      const uint32_t kv0 = base + Sm::KV;
      auto product_s = [&](int t, int slot) {
        mma_product_ss<D>(tmem + t * 128, smem_desc_sw128(base + Sm::Q + t * Sm::TILE),
                          smem_desc_sw128(kv0 + slot * Sm::TILE), kIdS);
      };
      auto product_o = [&](int t, int slot, bool first) {
        mma_product_ts(tmem + 256 + t * D, tmem + t * 128,
                       smem_desc_sw128_n(kv0 + slot * Sm::TILE, 16384), kIdO, !first);
      };
      auto wait = [&](uint64_t* bar, int parity) {
        return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(bar), parity, &abort_flag)) != 0;
      };
      auto wait_kv = [&](int it) { return wait(&kv_full[it % kPreSlots], (it / kPreSlots) & 1); };
      auto flag = [&](int v) { return __any_sync(0xFFFFFFFFu, v != 0) != 0; };  // uniform
      int seg = 0;
      bool ok = true, begins = true;  // (tile 0 begins a segment)
#pragma unroll 1
      for (int j = 0; j < tiles && ok; ++j) {
        // K's arrival says that the tile's place has been written down
        const int k_slot = (2 * j) % kPreSlots, v_slot = (2 * j + 1) % kPreSlots;
        const int next_slot = (2 * j + 2) % kPreSlots;
        if (begins) {
          // a segment's first S: its q has come, and the last one's O was read before that
          ok = wait_kv(2 * j) && wait(&q_full, seg & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            product_s(t, k_slot);
            mma_commit_warp(smem_u32(&s_full[t]));
          }
          mma_commit_warp(smem_u32(&kv_empty[k_slot]));
        }
        const bool ends = flag(sc[j & 3].ends);
        ok = wait_kv(2 * j + 1) && (ends || wait_kv(2 * j + 2));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          ok = ok && wait(&p_full[t], j & 1);
          if (!ok) break;
          tc_fence_after();
          product_o(t, v_slot, begins);
          if (t == 1) mma_commit_warp(smem_u32(&kv_empty[v_slot]));
          if (!ends) {
            product_s(t, next_slot);
            mma_commit_warp(smem_u32(&s_full[t]));
          }
        }
        if (!ok) break;
        if (ends) {
          // (the commit says that O is complete, the arrival passes on what the
          // converting warps wrote down)
          mma_commit_warp(smem_u32(&o_full));
          if (lane == 0) mbar_arrive(smem_u32(&o_full));
          ++seg;
        } else {
          mma_commit_warp(smem_u32(&kv_empty[next_slot]));
        }
        begins = ends;
      }
    } else {
      // ================================================================= conversion
      const int cw = warp - kPreSoftWarps - 2;
      int seg = 0;
      bool ok = true;
#pragma unroll 1
      for (int item = 0; item < 2 * tiles && ok; ++item) {
        const int slot = item % kPreSlots, round = item / kPreSlots;
        ok = mbar_wait(smem_u32(&raw_full[slot]), round & 1, &abort_flag) &&
             (round == 0 || mbar_wait(smem_u32(&kv_empty[slot]), (round - 1) & 1, &abort_flag));
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const uint32_t from = base + Sm::CODES + slot * Sm::RAW;
        const uint32_t to = base + Sm::KV + slot * Sm::TILE;
        // Places that hold no token may hold NaN codes, and 0 * NaN is NaN: what
        // is not there goes in as zeros, and so do the NaN codes of V where not
        // every row sees its token; those of tokens are written down.
        const PrefillScales& z = sc[(item >> 1) & 3];
        const bool strange = E4M3 && z.strange != 0;
        const int there = z.there, tokens = z.tokens, at = z.at;
        // 8 rows a step (16 at 64 head dimensions).  Eight neighbouring lanes
        // read 128 bytes on different banks and write eight different chunks
        // of the swizzle: at 128 head dimensions the lanes of the row's second
        // half take the pair's other row.
        constexpr int STEP = D == 128 ? 8 : 16;
        for (int r0 = cw * STEP; r0 < kPreTokens; r0 += kPreConvWarps * STEP) {
#pragma unroll
          for (int pass = 0; pass < 2; ++pass) {
            int r, c;  // row, 16-code chunk
            if constexpr (D == 128) {
              c = lane & 7;
              r = r0 + 2 * (lane >> 3) + (((c >> 2) ^ pass) & 1);
            } else {
              c = lane & 3;
              r = r0 + 8 * pass + (lane >> 2);
            }
            uint4 w = lds_16(from + r * D + c * 16);
            if (strange) {
              if (!((there >> (r >> 4)) & 1)) {
                w = make_uint4(0u, 0u, 0u, 0u);
              } else if (item & 1) {
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
                if ((nan_codes(x[0]) | nan_codes(x[1]) | nan_codes(x[2]) | nan_codes(x[3])) != 0) {
                  w = make_uint4(x[0] & ~nan_codes(x[0]), x[1] & ~nan_codes(x[1]), x[2] & ~nan_codes(x[2]),
                                 x[3] & ~nan_codes(x[3]));
                  if (r < tokens) {
                    segs[seg & (kPreSegments - 1)].nan = 1;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      if ((nan_codes(x[i >> 2]) >> (8 * (i & 3))) & 1u)
                        atomicMin(&first_nan[seg & (kPreSegments - 1)][c * 16 + i], at + r);
                  }
                }
              }
            }
            uint32_t h[8];
            codes_to_f16<E4M3>(w.x, h[0], h[1]);
            codes_to_f16<E4M3>(w.y, h[2], h[3]);
            codes_to_f16<E4M3>(w.z, h[4], h[5]);
            codes_to_f16<E4M3>(w.w, h[6], h[7]);
            const uint32_t row = to + (c >> 2) * 16384 + r * 128;
            const int at = 2 * (c & 3);
            sts_16(row + ((at ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
            sts_16(row + (((at + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
          }
        }
        if (E4M3 && (item & 1) && z.ends) ++seg;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&raw_empty[slot]));
          mbar_arrive(smem_u32(&kv_full[slot]));
        }
      }
    }
  }
  __syncthreads();
  if (abort_flag) {
    // given up, whoever did: what is on its way ends (bounded) before shared
    // memory and TMEM go
    if (warp == kPreSoftWarps) {
      for (int at = max(0, copied - kPreSlots); at < copied; ++at)
        mbar_wait_bounded(smem_u32(&raw_full[at % kPreSlots]), (at / kPreSlots) & 1, kDrainLimitNs);
    } else if (warp == kPreSoftWarps + 1) {
      mma_commit_warp(smem_u32(&drained));
      mbar_wait_bounded(smem_u32(&drained), 0, kDrainLimitNs);
    }
  }
  pdl_trigger();
  if (warp == kPreSoftWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the items that workers began and did not end, in the
// order of the keys: CTA (w, i) rows kPreJoinRows * i .. of worker w's item, a
// warp a row.
template <int D>
__global__ void __launch_bounds__(32 * kPreJoinRows) kv_prefill_join_kernel(const AttnArgs p) {
  constexpr int PIECE = kPreRows * (D + 2);
  constexpr int V = D / 32;
  const int w0 = blockIdx.x, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kPreJoinRows + (threadIdx.x >> 5);
  pdl_wait();
  const int4 cut = p.cut[2 * w0];
  pdl_trigger();
  const int r = cut.z + row;
  if (cut.x < 0 || r >= cut.w) return;
  const int q0 = p.cut[2 * w0 + 1].x;
  const int pieces = cut.x - w0 + 1;
  float m = -INFINITY, xm = -INFINITY, l = 0.0f, o[V];
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = 0.0f;
  // two pieces at a time, both on their way before either is used (most items
  // are cut once)
#pragma unroll 1
  for (int i = 0; i < pieces; i += 2) {
    float2 ml[2];  // R, L
    float v[2][V];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      ml[x] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
      for (int k = 0; k < V; ++k) v[x][k] = 0.0f;
      if (i + x < pieces) {
        const int64_t slot = i + x == 0 ? 2 * static_cast<int64_t>(w0) + 1 : 2 * (static_cast<int64_t>(w0) + i + x);
        const float* piece = p.pieces + slot * PIECE;
        ml[x] = __ldcg(reinterpret_cast<const float2*>(piece + kPreRows * D) + row);
        if constexpr (V == 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4*>(piece + row * D) + lane);
          v[x][0] = y.x, v[x][1] = y.y, v[x][2] = y.z, v[x][3] = y.w;
        } else {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(piece + row * D) + lane);
          v[x][0] = y.x, v[x][1] = y.y;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float top = fmaxf(m, ml[x].x), most = fmaxf(xm, ml[x].y);
      const float keep = ex2(m - exp_ref(top)), add = ex2(ml[x].x - exp_ref(top));
      l = l * ex2(xm - exp_ref(most)) + ex2(ml[x].y - exp_ref(most));
      m = top;
      xm = most;
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = o[k] * keep + v[x][k] * add;
    }
  }
  const int group = p.q_heads / p.kv_heads;
  const int i = r / group, hq = cut.y * group + r - i * group;
  const int64_t token = static_cast<int64_t>(q0) + i;
  const float L = attn_log(xm, l), fac = attn_factor(exp_ref(m) - 6.0f, L);
  uint16_t* to = p.out + token * p.ldo_token + hq * p.ldo_head + lane * V;
  uint32_t y[V / 2];
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * k] * fac * fac, o[2 * k + 1] * fac * fac);
    y[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if constexpr (V == 4) *reinterpret_cast<uint2*>(to) = make_uint2(y[0], y[1]);
  else *reinterpret_cast<uint32_t*>(to) = y[0];
  if (p.lse && lane == 0) p.lse[token * p.q_heads + hq] = L * 0.69314718055994531f;
}

}  // namespace i8
