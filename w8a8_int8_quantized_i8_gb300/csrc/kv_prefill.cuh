// kv_prefill.cuh -- the paged attention of kv_attention.cuh for requests with
// many rows (chunks of prompts), on the tensor cores of tcgen05.
//
// The same formula and cache.  A CTA takes 256 rows of a request (new token x
// query head of one kv head, token-major) as two tiles of 128, and goes over
// the keys 128 tokens at a time:
//   S_t = Q_t K^T  -> TMEM      (fp16 x fp16, exact products, fp32 sums)
//   P_t = 2^(s + log2 sv - R)   softmax threads, P back to TMEM
//   O_t += P_t V   -> TMEM      (A operand from TMEM, V as it lies: N-major)
// with s = S * sk * scale * log2 e and sv, sk the block's scales.  The two
// tiles take turns: while one tile's softmax runs, the tensor cores do the
// other's O and next S.
//
// Codes are converted to fp16, exactly, once a CTA and serve all 256 rows.  q is scaled per row by a power of two as in
// kv_attention.cuh.  R is a row's running maximum of s + log2 sv, the log of a
// term's weight in O; it moves only when it grows by more than 2^8, so that O
// in TMEM is rarely rescaled, and P, held in fp16 as 2^(6 + s + log2 sv - R),
// stays below 2^14.  The sum of exponentials is kept in fp32 beside it, each
// 16 tokens' sum of P times 2^(Lr - log2 sv), Lr a fixed reference.
//
// Roles: warps 0-15 softmax (tile = warp / 8; a row has two threads, each for
// half of the keys, which agree on R once a tile; a warp reads the 32 TMEM
// lanes of its place in the warpgroup), warp 16 copies by TMA and prepares the
// scales, warp 17 issues the MMAs, warps 18-23 convert.  At 128 head dimensions 208 KB
// of shared memory (Q 64, three fp16 tiles 96, three tiles of codes 48) and all
// of TMEM (S 2 x 128, O 2 x 128 columns): one CTA an SM.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

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

struct PrefillScales {   // of the 16-token granules of a tile
  float k[kPreGranules];
  float lv[kPreGranules];     // log2 of V's
  float back[kPreGranules];   // 2^(Lr - lv)
};

// An N-major (transposed) operand stored with the 128-byte swizzle: rows of
// 128 bytes (64 values along N) for each k, 8-row groups 1024 bytes apart along
// K, 64-value groups `n_stride` bytes apart along N.
__device__ __forceinline__ uint64_t smem_desc_sw128_n(uint32_t saddr, uint32_t n_stride) {
  uint64_t d = smem_desc_sw128(saddr) & ~(static_cast<uint64_t>(0x3FFFu) << 16);
  return d | (static_cast<uint64_t>(n_stride >> 4) << 16);
}

// D[tmem] (+)= A * B[smem]^T, kind::f16, one CTA, A in shared memory or in
// TMEM; and the commit that arrives on `bar` when what was issued is done.  The
// whole warp calls, its elected lane (the same one every time) issues: kept in
// converged code the operands stay in uniform registers, where the instruction
// wants them.  Issued by one lane of a divergent branch, each product of eight
// took about 980 cycles instead of 512.
__device__ __forceinline__ void mma_f16_ss_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
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
  extern __shared__ uint8_t sm_pre[];
  __shared__ __align__(8) uint64_t raw_full[kPreSlots], raw_empty[kPreSlots], kv_full[kPreSlots],
      kv_empty[kPreSlots], sc_full[kPreScales], s_full[2], p_full[2], q_full, o_full, drained;
  __shared__ PrefillScales sc[kPreScales];
  __shared__ float sm_ref;
  __shared__ float sm_top[2][2][128], sm_sum[2][2][128];  // [tile][half of the keys][row]
  __shared__ uint32_t sm_tmem;
  __shared__ int abort_flag, sm_gaps;  // sm_gaps: some block was missing so far
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int group = p.q_heads / p.kv_heads;
  const uint32_t base = (smem_u32(sm_pre) + 1023u) & ~1023u;

  if (threadIdx.x == 0) {
    abort_flag = sm_gaps = 0;
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
    }
    mbar_init(smem_u32(&q_full), kPreSoftWarps);
    mbar_init(smem_u32(&o_full), 1);
    mbar_init(smem_u32(&drained), 1);
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
    fence_mbarrier_init();
  }

  pdl_wait();
  // ---- the item: row tiles of a request from the last (the longest) to the first
  const int tiles_max = static_cast<int>((static_cast<int64_t>(p.max_new) * group + kPreRows - 1) / kPreRows);
  const int head = blockIdx.x % p.kv_heads;
  const int req = static_cast<int>(blockIdx.x / p.kv_heads) % p.requests;
  const int back = static_cast<int>(blockIdx.x / p.kv_heads) / p.requests;
  const AttnRequest rq = attn_request<kPreRows, kPreTokens>(p, req);
  const int rows = rq.fresh * group;
  const int tile = rq.tiles - 1 - back;
  if (rows < p.split_rows || tile < 0 || tiles_max <= 0) return;  // (the whole CTA)
  const int row0 = tile * kPreRows;
  const int pos0 = rq.len - rq.fresh;
  const int last_row = min(row0 + kPreRows, rows) - 1;
  const int end = min(max(pos0 + last_row / group + 1, 0), rq.len);
  const int n = (end + kPreTokens - 1) / kPreTokens;  // tiles of keys
  if (warp == kPreSoftWarps + 1) {
    tmem_alloc(smem_u32(&sm_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm_tmem;

  if (warp < kPreSoftWarps) {
    // =================================================================== softmax
    regs_inc<96>();
    const int t = warp >> 3, half = (warp >> 2) & 1;
    const int r = (warp & 3) * 32 + lane;  // row of the tile
    const int row = row0 + t * 128 + r;
    const bool real = row < rows;
    const int i = real ? row / group : 0;
    const int hq = head * group + (real ? row - i * group : 0);
    float rowfac;
    {
      // q's row: its power of two, then this thread's half in fp16 into the
      // swizzled tile
      const uint4* qp = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(rq.q0) + i) * p.ldq_token + hq * p.ldq_head);
      uint32_t amax = 0;
#pragma unroll 8
      for (int c = 0; c < D / 8; ++c) {
        const uint4 w = real ? __ldg(qp + c) : make_uint4(0u, 0u, 0u, 0u);
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
        const uint4 w = real ? __ldg(qp + c) : make_uint4(0u, 0u, 0u, 0u);
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
    const int limit = real ? min(max(pos0 + i + 1, 0), rq.len) : 0x7FFFFFFF;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t s_at = tmem + lanes + t * 128 + half * 64;  // this half's S
    const uint32_t p_at = tmem + lanes + t * 128 + half * 32;  // and P
    const uint32_t o_at = tmem + lanes + 256 + t * D + half * (D / 2);
    float R = -INFINITY, l = 0.0f;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      ok = ok && mbar_wait(smem_u32(&sc_full[j & 3]), (j >> 2) & 1, &abort_flag) &&
           mbar_wait(smem_u32(&s_full[t]), j & 1, &abort_flag);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) {  // given up: only keep the tile's barrier company
        named_bar_sync(1 + t, 256);
        continue;
      }
      tc_fence_after();
      const PrefillScales& z = sc[j & 3];
      const int seen = limit - j * kPreTokens - 64 * half;  // columns below this are seen
      const bool masked = __any_sync(0xFFFFFFFFu, seen < 64);
      uint32_t s[2][32];
      tmem_ld_32x32b_x32(s_at, s[0]);
      tmem_ld_32x32b_x32(s_at + 32, s[1]);
      tmem_wait_ld(s[0]);
      tmem_wait_ld(s[1]);
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
        alpha = R > -INFINITY ? ex2(R - top) : 0.0f;
        R = top;
        l *= alpha;
      }
      if (__any_sync(0xFFFFFFFFu, alpha != 1.0f) && j > 0) {
        // S of this tile was committed after the last product into O, so O is
        // complete; each thread rescales its half of the head dimensions
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
      const float ref = (R > -INFINITY ? R : 0.0f) - 6.0f;
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
          l = fmaf(s0 + s1, z.back[gr], l);
        }
        tmem_st_32x32b_x16(p_at + 16 * q, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_full[t]));
    }
    // ---- out: each thread its half of the head dimensions
    sm_sum[t][half][r] = l;
    named_bar_sync(1 + t, 256);
    l += sm_sum[t][half ^ 1][r];
    if (n > 0 && ok) ok = mbar_wait(smem_u32(&o_full), 0, &abort_flag);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.0f ? __fdiv_rn(ex2(sm_ref), l) : 0.0f;
      const int64_t token = static_cast<int64_t>(rq.q0) + i;
      uint16_t* to = p.out + token * p.ldo_token + hq * p.ldo_head + half * (D / 2);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[16];
        if (n > 0) {
          tmem_ld_32x32b_x16(o_at + 16 * q, o);
          tmem_wait_ld(o);
        }
        if (real) {
#pragma unroll
          for (int k = 0; k < 16; k += 8) {
            uint32_t y[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float lo = l > 0.0f ? __uint_as_float(o[k + 2 * m]) * inv : 0.0f;
              const float hi = l > 0.0f ? __uint_as_float(o[k + 2 * m + 1]) * inv : 0.0f;
              const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
              y[m] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(to + 16 * q + k) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      if (real && p.lse && half == 0)
        p.lse[token * p.q_heads + hq] =
            l > 0.0f ? (R - sm_ref - 6.0f + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    tc_fence_before();
  } else {
    regs_dec<48>();
    if (warp == kPreSoftWarps) {
      // ================================================================= copies
      const int32_t* table = p.table + req * p.ld_table;
      const int boxes = kPreTokens / p.box_rows;
      int item = 0;
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) {
        // scales, a lane a granule
        float sk = 0.0f, lv = -INFINITY;
        if (lane < kPreGranules) {
          const int tk = j * kPreTokens + 16 * lane;
          if (tk < end) {
            const int64_t blk = __ldg(table + tk / p.block);  // end lies within the table's width
            if (blk >= 0 && blk < p.blocks) {
              sk = __ldg(p.k_scale + blk * p.kv_heads + head);
              const float sv = __ldg(p.v_scale + blk * p.kv_heads + head);
              lv = sv > 0.0f ? log2f(sv) : -1000.0f;
            } else {
              atomicOr(&g_status, 1u << 7);
              sm_gaps = 1;
            }
          }
        }
        float ref = lv;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, o));
        ref = __shfl_sync(0xFFFFFFFFu, ref, 0);
        if (j == 0 && lane == 0) sm_ref = ref > -500.0f ? ref : 0.0f;
        __syncwarp();
        ref = sm_ref;
        if (lv == -1000.0f) lv = ref - 60.0f;  // a block of zeros: its weight does not matter
        PrefillScales& z = sc[j & 3];
        if (lane < kPreGranules) {
          z.k[lane] = sk;
          z.lv[lane] = lv;
          z.back[lane] = lv > -INFINITY ? ex2(ref - lv) : 0.0f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sc_full[j & 3]));
        // the codes, a lane a box
        const int tb = j * kPreTokens + lane * p.box_rows;
        int64_t blk = -1;
        int off = 0;
        if (lane < boxes && tb < end) {
          const int col = tb / p.block;
          off = tb - col * p.block;
          blk = __ldg(table + col);
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
                        static_cast<int>(blk) * p.kv_heads + head);
        }
      }
      if (!ok) {  // let the copies in flight land (bounded) before the CTA ends
        for (int back_i = 1; back_i <= kPreSlots && item - back_i >= 0; ++back_i) {
          const int at = item - back_i;
          mbar_wait_bounded(smem_u32(&raw_full[at % kPreSlots]), (at / kPreSlots) & 1, 1000000ull);
        }
      }
    } else if (warp == kPreSoftWarps + 1) {
      // ================================================================= products
      if (n > 0) {
        constexpr uint32_t kIdS = idesc_f16_f32(128, kPreTokens);
        constexpr uint32_t kIdO = idesc_f16_f32(128, D) | (1u << 16);  // B is N-major
        const uint32_t kv0 = base + Sm::KV;
        auto product_s = [&](int t, int slot) {
          const uint64_t a = smem_desc_sw128(base + Sm::Q + t * Sm::TILE);
          const uint64_t b = smem_desc_sw128(kv0 + slot * Sm::TILE);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
            mma_f16_ss_warp(tmem + t * 128, a + at, b + at, kIdS, k > 0);
          }
        };
        auto product_o = [&](int t, int slot, bool first) {
          const uint64_t b = smem_desc_sw128_n(kv0 + slot * Sm::TILE, 16384);
#pragma unroll
          for (int k = 0; k < kPreTokens / 16; ++k)
            mma_f16_ts_warp(tmem + 256 + t * D, tmem + t * 128 + 8 * k, b + k * (2048 >> 4), kIdO,
                            !(first && k == 0));
        };
        auto wait_kv = [&](int it) {
          return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&kv_full[it % kPreSlots]),
                                                   (it / kPreSlots) & 1, &abort_flag));
        };
        bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&q_full), 0, &abort_flag)) && wait_kv(0);
        if (ok) {
          tc_fence_after();
          for (int t = 0; t < 2; ++t) {
            product_s(t, 0);
            mma_commit_warp(smem_u32(&s_full[t]));
          }
          mma_commit_warp(smem_u32(&kv_empty[0]));
        }
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const int v_slot = (2 * j + 1) % kPreSlots, k_slot = (2 * j + 2) % kPreSlots;
          const bool more = j + 1 < n;
          ok = wait_kv(2 * j + 1) && (!more || wait_kv(2 * j + 2));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&p_full[t]), j & 1, &abort_flag));
            if (!ok) break;
            tc_fence_after();
            product_o(t, v_slot, j == 0);
            if (t == 1) mma_commit_warp(smem_u32(&kv_empty[v_slot]));
            if (more) {
              product_s(t, k_slot);
              mma_commit_warp(smem_u32(&s_full[t]));
            }
          }
          if (ok && more) mma_commit_warp(smem_u32(&kv_empty[k_slot]));
        }
        if (ok) {
          mma_commit_warp(smem_u32(&o_full));
        } else {  // the products in flight end (bounded) before TMEM is freed
          mma_commit_warp(smem_u32(&drained));
          mbar_wait_bounded(smem_u32(&drained), 0, 1000000000ull);
        }
      }
      __syncwarp();
    } else {
      // ================================================================= conversion
      const int cw = warp - kPreSoftWarps - 2;
      bool ok = true;
#pragma unroll 1
      for (int item = 0; item < 2 * n && ok; ++item) {
        const int slot = item % kPreSlots, round = item / kPreSlots;
        ok = mbar_wait(smem_u32(&raw_full[slot]), round & 1, &abort_flag) &&
             (round == 0 || mbar_wait(smem_u32(&kv_empty[slot]), (round - 1) & 1, &abort_flag));
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const uint32_t from = base + Sm::CODES + slot * Sm::RAW;
        const uint32_t to = base + Sm::KV + slot * Sm::TILE;
        // the last tile may end inside a box, and a missing block leaves what
        // was there before
        const bool strange = E4M3 && (item >= 2 * n - 2 || *static_cast<volatile int*>(&sm_gaps));
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
            if (strange)
              w = make_uint4(without_nan_codes(w.x), without_nan_codes(w.y), without_nan_codes(w.z),
                             without_nan_codes(w.w));
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
  pdl_trigger();
  if (warp == kPreSoftWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace i8
