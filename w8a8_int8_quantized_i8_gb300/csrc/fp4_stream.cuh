// fp4_stream.cuh -- the 4-bit product for few tokens: the weights stream through
// the tensor core, tokens are the narrow operand.
//
//   D[channel, token] = sum_k w[channel, k] * x[token, k]
//
// A CTA takes 128 channels (of both weights, gated), NT tokens and a share of K.
// The tensor core's M dimension is the channels', so NT can be as small as 16: one
// token costs 16 columns and not 128 rows.  (A tile of tokens begins where a tile
// of their scales does: NT < 128 takes all tokens at once.)  Warp 0 fetches tiles of 256 elements
// by TMA (codes, 128-byte swizzle) and bulk copies (scales) into a ring, warp 1
// copies scales to tensor memory and issues products, and all warps read D, 32
// lanes and all of the tokens or half of them each.
//
// Channels alone do not fill the GPU at few tokens (4096 are 32 CTAs), so K is
// split over the CTAs of a cluster.  They meet in distributed shared memory: each
// CTA writes its partial sums of every token to the CTA that finishes this token,
// four tokens of a channel in 16 bytes, which adds them in the order of the splits
// (the same bits every time).  No workspace, no second launch.
//
// The fewest tokens, still bf16 (FUSED), are quantized here by the two warps without
// another role, in turns at the stages, while the weights are on their way: no
// launch of its own, no rows in memory.  What a row's scale needs (NV16) is the row's
// largest magnitude, which each CTA finds by itself (2 K bytes a token from L2; by
// the cluster together, with a barrier of it, one token took 2.5 us more).
//
// Bound by HBM where the weights come from there, else by a chain of latencies: one
// token by 6144 x 4096 (NV16, 4 splits) 4.9 us from L2 behind a quantizer, of them 1
// to the first tile, 2 of products, 1 for the cluster's meeting, and 4.5 with the
// quantizing in it; one token by two weights of 11008 x 4096, from HBM, 10.2 us (50
// MB, 5.0 TB/s); 256 tokens by 4096 x 4096 8.2 us.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "fp4_mma.cuh"
#include "fp4_quant.cuh"

namespace i8 {

constexpr int kFp4MaxSplits = 8;
constexpr int kFp4Prefetch = 6;  // tiles of K

// The most tokens that a CTA quantizes for itself.  us measured, so and with the
// quantizer's launch, of 1, 2, 3, 4 tokens by 6144 x 4096 from HBM:
//   MX32  4.8 4.9 4.8 4.8 and 6.5 6.6 6.6 6.6; by 28672 x 8192 20.9 .. 22.6 and 22.6 .. 22.9
//   NV16  5.3 5.5 and 6.8 6.9; built for four, 5.7 6.3 6.8 7.6: the rows' largest
//         magnitudes are found before the first product, by two warps
constexpr int fp4_fused_tokens(bool mx) { return mx ? 4 : 2; }

// Tokens that one of `splits` CTAs finishes: fours.
__host__ __device__ constexpr int fp4_each(int tokens, int splits) { return ((tokens + splits - 1) / splits + 3) / 4 * 4; }

// The most sums of tokens that a CTA gets from up to `most` splits.
constexpr int fp4_red_tokens(int tokens, int most) {
  int n = 0;
  for (int s = 2; s <= most; ++s) n = s * fp4_each(tokens, s) > n ? s * fp4_each(tokens, s) : n;
  return n;
}

template <bool MX, int NT, bool GATED, bool FUSED = false>
struct Fp4StreamCfg {
  static constexpr int WEIGHTS = GATED ? 2 : 1;
  static constexpr int TOKENS = fp4_fused_tokens(MX);  // FUSED
  static constexpr int SCALES = fp4_tile_bytes(MX ? 32 : 16);
  static constexpr int PARTS = SCALES / 512;
  static constexpr int OFF_T = WEIGHTS * 16384;
  static constexpr int OFF_WS = OFF_T + NT * 128;
  static constexpr int OFF_TS = OFF_WS + WEIGHTS * SCALES;
  static constexpr int STAGE = OFF_TS + SCALES;
  static constexpr uint32_t TX = WEIGHTS * (16384 + SCALES) + (FUSED ? 0 : NT * 128 + SCALES);
  // the sums to be finished, 512 bytes for each split, weight and token: a region
  // of their own for the fewest tokens, which saves a barrier of the cluster, else
  // the ring
  static constexpr int MAX_SPLITS = GATED ? kFp4MaxSplits / 2 : kFp4MaxSplits;
  static constexpr int RED = fp4_red_tokens(NT, MAX_SPLITS) * WEIGHTS * 512;
  static constexpr int RED_OWN = NT == 16 ? RED : 0;
  // two CTAs an SM, so that one's fetches run while the other meets its cluster
  // (and the next kernel begins); 128 tokens of two weights want half the GPU's
  // tensor memory and more, and get an SM to themselves
  static constexpr int ROOM = GATED && NT == 128 ? 222 * 1024 : 112 * 1024;
  static constexpr int STAGES = (ROOM - RED_OWN - 1024) / STAGE > 8 ? 8 : (ROOM - RED_OWN - 1024) / STAGE;
  // two warps for each 32 channels where there are tokens for both
  static constexpr int GROUPS = NT >= 64 ? 2 : 1;
  static constexpr int THREADS = 128 * GROUPS;
  static constexpr int OFF_RED = RED_OWN ? STAGES * STAGE : 0;
  static constexpr int SMEM = STAGES * STAGE + RED_OWN + 1024;
  // tensor memory: D, the weights' scales, the tokens'
  static constexpr int COL_WS = WEIGHTS * NT;
  static constexpr int COL_TS = COL_WS + WEIGHTS * 4 * PARTS;
  static constexpr int COLS_USED = COL_TS + 4 * PARTS;
  static constexpr int COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
  static_assert(COLS_USED <= 512 && STAGE % 1024 == 0 && NT % 16 == 0 && NT <= 128);
  // co-resident CTAs never wait for one another's tensor memory
  static_assert(STAGES >= 2 && (COLS <= 256 || SMEM > 120 * 1024));
  static_assert(RED_OWN != 0 || RED <= STAGES * STAGE);
  static_assert(!FUSED || NT == 16);
};

// Codes and scales of 256 elements of a token, of which this lane holds 8 (the whole
// warp calls), where a stage's tile of tokens has them (128-byte swizzle) and its
// tile of scales.
template <bool MX>
__device__ __forceinline__ void fp4_smem256(uint32_t codes, uint32_t scales, int row, int lane, bool inside, const uint4& x,
                                            float s, float inverse) {
  const Fp4Held<false> held{x};
  float unused = 0.0f;
  const Fp4QuantArgs none{};
  uint32_t top = fp4_top<false>(none, 0, held, unused);
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  if constexpr (MX) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  float t[8];
  fp4_widen<false>(none, 0, held, t);
  if constexpr (!MX) fp4_row_scaled(t, top, s, inverse);
  uint32_t scale;
  const uint32_t c = fp4_codes8<MX>(t, top, s, inverse, &scale);
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(codes + row * 128u + (((lane >> 2) ^ (row & 7)) << 4) + (lane & 3) * 4u),
               "r"(inside ? c : 0u)
               : "memory");
  constexpr int LB = MX ? 4 : 2;  // lanes of a block
  scale = inside ? scale << (8 * (lane / LB % 4)) : 0u;
  scale |= __shfl_xor_sync(0xFFFFFFFFu, scale, LB);
  scale |= __shfl_xor_sync(0xFFFFFFFFu, scale, 2 * LB);
  if (lane % (4 * LB) == 0)
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(scales + lane / (4 * LB) * 512u + row * 16u), "r"(scale) : "memory");
}

template <bool MX, int NT, int ACT, bool FUSED>
__global__ void __launch_bounds__(NT >= 64 ? 256 : 128, 1)
    fp4_stream_kernel(const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
                      const __grid_constant__ CUtensorMap tm_t, const Fp4GemmArgs p) {
  constexpr bool GATED = ACT != kFp4Plain;
  using Cfg = Fp4StreamCfg<MX, NT, GATED, FUSED>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[Cfg::STAGES];
  __shared__ __align__(8) uint64_t empty[Cfg::STAGES];
  __shared__ __align__(8) uint64_t done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ float token_scale[NT];
  __shared__ uint32_t warp_max[2][FUSED ? Cfg::TOKENS : 1];
  volatile int* abort_flag = &abort_word;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % p.splits, n_tile = static_cast<int>(blockIdx.x) / p.splits;
  const int n0 = n_tile * 128, m0 = static_cast<int>(blockIdx.y) * NT;
  const int kb0 = rank * p.deep_per_split, kb1 = min(p.deep, kb0 + p.deep_per_split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), FUSED ? 2 : 1);  // the producer, and a quantizing warp
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(&done), 1);
    abort_word = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), Cfg::COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w0);
    if constexpr (GATED) tma_prefetch_desc(&tm_w1);
    if constexpr (!FUSED) tma_prefetch_desc(&tm_t);
    // this CTA's weights on their way into L2 while the kernel before drains, more of
    // them than the ring holds: HBM's latency is paid once
    const int64_t ws0 = (static_cast<int64_t>(n_tile) * p.deep + kb0) * Cfg::SCALES;
    for (int kb = kb0; kb < min(kb1, kb0 + kFp4Prefetch); ++kb) {
      tma_prefetch_l2_2d(&tm_w0, kb * 128, n0);
      if constexpr (GATED) tma_prefetch_l2_2d(&tm_w1, kb * 128, n0);
    }
    const uint32_t ahead = static_cast<uint32_t>(min(kb1 - kb0, kFp4Prefetch) * Cfg::SCALES);
    bulk_prefetch_l2(p.w[0].scales + ws0, ahead);
    if constexpr (GATED) bulk_prefetch_l2(p.w[1].scales + ws0, ahead);
  }
  tc_fence_before();
  __syncthreads();
  // (every CTA of the cluster is there before another writes to it)
  if (Cfg::RED_OWN && p.splits > 1) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_trigger();
  // this thread's channel and its half of the tokens
  const int channel = threadIdx.x & 127, group = threadIdx.x >> 7;
  const int n = n0 + channel;
  float sw[Cfg::WEIGHTS], b[Cfg::WEIGHTS];
#pragma unroll
  for (int w = 0; w < Cfg::WEIGHTS; ++w) {
    sw[w] = n < p.N && p.w[w].row_scales ? p.w[w].row_scales[n] : 1.0f;
    b[w] = n < p.N && p.w[w].bias ? __uint_as_float(static_cast<uint32_t>(p.w[w].bias[n]) << 16) : 0.0f;
  }

  if (warp == 0 && lane == 0) {
    bool ok = true;
    int s = 0, issued = 0;
    uint32_t ph = 0;
    const int64_t tile = Cfg::SCALES;
    const uint8_t* ws0 = p.w[0].scales + static_cast<int64_t>(n_tile) * p.deep * tile;
    const uint8_t* ws1 = GATED ? p.w[1].scales + static_cast<int64_t>(n_tile) * p.deep * tile : nullptr;
    const uint8_t* ts = FUSED ? nullptr : p.scales + static_cast<int64_t>(m0 >> 7) * p.deep * tile;
    for (int kb = kb0; kb < kb1; ++kb) {
      const uint32_t bar = smem_u32(&full[s]), st = ring + static_cast<uint32_t>(s * Cfg::STAGE);
      if (!(ok = mbar_wait(smem_u32(&empty[s]), ph ^ 1u, abort_flag))) break;
      mbar_arrive_expect_tx(bar, Cfg::TX);
      tma_load_2d(st, &tm_w0, bar, kb * 128, n0);
      if constexpr (GATED) tma_load_2d(st + 16384, &tm_w1, bar, kb * 128, n0);
      if constexpr (!FUSED) tma_load_2d(st + Cfg::OFF_T, &tm_t, bar, kb * 128, m0);
      bulk_load(st + Cfg::OFF_WS, ws0 + kb * tile, Cfg::SCALES, bar);
      if constexpr (GATED) bulk_load(st + Cfg::OFF_WS + Cfg::SCALES, ws1 + kb * tile, Cfg::SCALES, bar);
      if constexpr (!FUSED) bulk_load(st + Cfg::OFF_TS, ts + kb * tile, Cfg::SCALES, bar);
      ++issued;
      if (++s == Cfg::STAGES) s = 0, ph ^= 1u;
    }
    // a CTA that gives up ends after its own copies
    if (!ok)
      for (int i = max(0, issued - Cfg::STAGES); i < issued; ++i)
        mbar_wait_bounded(smem_u32(&full[i % Cfg::STAGES]), (i / Cfg::STAGES) & 1, 100000000ull);
  } else if (warp == 1) {
    const uint32_t leader = elect_one();
    int s = 0;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&full[s]), ph, abort_flag))) break;
      tc_fence_after();
      const uint32_t st = ring + static_cast<uint32_t>(s * Cfg::STAGE);
      const uint64_t bd = smem_desc_sw128(st + Cfg::OFF_T);
      auto scales = [&](int j) {  // those of a part
#pragma unroll
        for (int w = 0; w < Cfg::WEIGHTS; ++w)
          copy_scales<1>(leader, tmem + Cfg::COL_WS + (w * Cfg::PARTS + j) * 4,
                         smem_desc_scales(st + Cfg::OFF_WS + w * Cfg::SCALES + j * 512));
        copy_scales<1>(leader, tmem + Cfg::COL_TS + j * 4, smem_desc_scales(st + Cfg::OFF_TS + j * 512));
      };
      scales(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // 64 elements, 32 bytes along the swizzled row
        const int part = MX ? j / 2 : j;
        if (MX ? j == 0 : j < 3) scales(part + 1);  // while the product before runs
        const uint32_t idesc = MX && (j & 1) ? fp4_idesc<MX>(128, NT, 2) : fp4_idesc<MX>(128, NT, 0);
#pragma unroll
        for (int w = 0; w < Cfg::WEIGHTS; ++w)
          mma_fp4<MX, 1>(leader, tmem + w * NT, smem_desc_sw128(st + w * 16384) + 2u * j, bd + 2u * j, idesc,
                         tmem + Cfg::COL_WS + (w * Cfg::PARTS + part) * 4, tmem + Cfg::COL_TS + part * 4,
                         kb > kb0 || j > 0 ? 1u : 0u);
      }
      commit_elected(leader, smem_u32(&empty[s]));
      if (++s == Cfg::STAGES) s = 0, ph ^= 1u;
    }
    commit_elected(leader, smem_u32(&done));
    mbar_wait_bounded(smem_u32(&done), 0u, 100000000ull);
  } else if (FUSED && warp >= 2) {
    constexpr int TOKENS = Cfg::TOKENS;
    const int me = warp - 2;
    auto load = [&](int row, int kb, int end) {
      const int e = kb * kFp4TileK + lane * 8;
      return row < p.M && kb < end && e < p.K ? *reinterpret_cast<const uint4*>(p.x + row * p.ldx + e)
                                              : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 next[TOKENS];
#pragma unroll
    for (int row = 0; row < TOKENS; ++row) next[row] = load(row, kb0 + me, kb1);
    float s[TOKENS], inverse[TOKENS];
#pragma unroll
    for (int row = 0; row < TOKENS; ++row) s[row] = inverse[row] = 1.0f;
    if constexpr (!MX) {
      constexpr int BATCH = 8;  // loads of a row in flight
      uint32_t top[TOKENS] = {};  // pairs of magnitudes, the signs undefined
      for (int kb = me; kb < p.deep; kb += 2 * BATCH) {
        uint4 v[TOKENS][BATCH];
#pragma unroll
        for (int row = 0; row < TOKENS; ++row)
#pragma unroll
          for (int i = 0; i < BATCH; ++i) v[row][i] = load(row, kb + 2 * i, p.deep);
#pragma unroll
        for (int row = 0; row < TOKENS; ++row)
#pragma unroll
          for (int i = 0; i < BATCH; ++i)
            for (uint32_t x : {v[row][i].x, v[row][i].y, v[row][i].z, v[row][i].w})
              top[row] = absmax_nan_bf16x2(top[row], x);
      }
#pragma unroll
      for (int row = 0; row < TOKENS; ++row) {
        const uint32_t m = top[row] & 0x7FFF7FFFu, t = __reduce_max_sync(0xFFFFFFFFu, max(m << 16, m & 0xFFFF0000u));
        if (lane == 0) warp_max[me][row] = t;
      }
      named_bar_sync(1, 64);
#pragma unroll
      for (int row = 0; row < TOKENS; ++row) {
        const float scale = fp4_row_scale(max(warp_max[0][row], warp_max[1][row]), s[row], inverse[row]);
        if (me == 0 && lane == 0) token_scale[row] = scale;
      }
    }
    if (me == 1 && lane < NT && (MX || lane >= TOKENS)) token_scale[lane] = 1.0f;
    int stage = me;
    uint32_t ph = 0;
    for (int kb = kb0 + me; kb < kb1; kb += 2) {
      uint4 v[TOKENS];
#pragma unroll
      for (int row = 0; row < TOKENS; ++row) {
        v[row] = next[row];
        next[row] = load(row, kb + 2, kb1);
      }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&empty[stage]), ph ^ 1u, abort_flag))) break;
      const uint32_t st = ring + static_cast<uint32_t>(stage * Cfg::STAGE);
#pragma unroll
      for (int row = 0; row < TOKENS; ++row)
        if (row < p.M)
          fp4_smem256<MX>(st + Cfg::OFF_T, st + Cfg::OFF_TS, row, lane, kb * kFp4TileK + lane * 8 < p.K, v[row], s[row],
                          inverse[row]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&full[stage]));
      if ((stage += 2) >= Cfg::STAGES) stage -= Cfg::STAGES, ph ^= 1u;
    }
  } else if (warp >= 2) {
    for (int i = threadIdx.x - 64; i < NT; i += Cfg::THREADS - 64)
      token_scale[i] = m0 + i < p.M ? (p.row_scales ? p.row_scales[m0 + i] : 1.0f) : 0.0f;
  }
  __syncwarp();
  mbar_wait(smem_u32(&done), 0u, abort_flag);
  __syncthreads();  // token_scale; the abort flag's last word
  tc_fence_after();
  const bool ok = *abort_flag == 0;
  const int count = min(NT, p.M - m0);
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const int c0 = group * (NT / Cfg::GROUPS), c1 = min(count, c0 + NT / Cfg::GROUPS);  // the columns that it reads
  // Finishes tokens c .. c + 3 of the tile (those below `end`) from the sums of this
  // thread's channel; four lanes exchange them so that each stores four channels
  // of one token.
  auto finish = [&](int c, int end, const float (&acc)[Cfg::WEIGHTS][4]) {
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float sa = token_scale[min(c + k, NT - 1)];
      v[k] = fp4_dequant(acc[0][k], sa, sw[0], b[0]);
      if constexpr (GATED) v[k] = fp4_gate<ACT>(v[k], fp4_dequant(acc[1][k], sa, sw[1], b[1]));
    }
    const uint32_t p01 = pack_bf16x2_rn(v[0], v[1]), p23 = pack_bf16x2_rn(v[2], v[3]);
    // with the odd or even neighbour: two tokens, of a pair of channels each
    const bool odd = lane & 1, high = lane & 2;
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? p01 : p23, 1);
    const uint32_t lo = odd ? got : p01, hi = odd ? p23 : got;  // the even and the odd channel's tokens
    const uint32_t t0 = __byte_perm(lo, hi, 0x5410), t1 = __byte_perm(lo, hi, 0x7632);
    // with the other pair: one token of four channels
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, high ? t0 : t1, 2);
    const int at = c + (odd ? 2 : 0) + (high ? 1 : 0);
    if (at < end && n < p.N)
      *reinterpret_cast<uint2*>(p.y + static_cast<int64_t>(m0 + at) * p.ldy + (n & ~3)) =
          high ? make_uint2(other, t1) : make_uint2(t0, other);
  };
  if (p.splits == 1) {
    if (ok)
#pragma unroll 2
      for (int c = c0; c < c1; c += 16) {
        uint32_t r[Cfg::WEIGHTS][16];
#pragma unroll
        for (int w = 0; w < Cfg::WEIGHTS; ++w) tmem_ld_32x32b_x16(lanes + w * NT + c, r[w]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          float acc[Cfg::WEIGHTS][4];
#pragma unroll
          for (int w = 0; w < Cfg::WEIGHTS; ++w)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[w][k] = __uint_as_float(r[w][i + k]);
          finish(c + i, count, acc);
        }
      }
  } else {
    // token c of the tile is finished by CTA c / each; in its shared memory lie
    // [split][weight][each / 4][128 channels][4 tokens]
    const int each = fp4_each(count, p.splits);
    const uint32_t red = ring + Cfg::OFF_RED;
    if constexpr (Cfg::RED_OWN != 0) cluster_wait();
    else cluster_sync_all();  // the rings are free: every CTA's products have ended
    if (ok) {
      const uint32_t at = static_cast<uint32_t>(rank * Cfg::WEIGHTS * each) * 512u + channel * 16u;
      int owner = c0 / each, slot = c0 - owner * each;
      uint32_t to = mapa_shared(red, min(owner, p.splits - 1)) + at;
#pragma unroll 2
      for (int c = c0; c < c1; c += 16) {
        uint32_t r[Cfg::WEIGHTS][16];
#pragma unroll
        for (int w = 0; w < Cfg::WEIGHTS; ++w) tmem_ld_32x32b_x16(lanes + w * NT + c, r[w]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          if (c + i < c1) {
            if (slot == each) {
              slot = 0;
              to = mapa_shared(red, ++owner) + at;
            }
#pragma unroll
            for (int w = 0; w < Cfg::WEIGHTS; ++w)
              st_cluster_v4(to + static_cast<uint32_t>(w * each + slot) * 512u,
                            make_uint4(r[w][i], r[w][i + 1], r[w][i + 2], r[w][i + 3]));
            slot += 4;
          }
        }
      }
    }
    cluster_sync_all();
    if (ok) {
      const int first = rank * each, end = min(count, first + each);
#pragma unroll 4
      for (int c = first + 4 * group; c < end; c += 4 * Cfg::GROUPS) {
        float acc[Cfg::WEIGHTS][4];
#pragma unroll
        for (int w = 0; w < Cfg::WEIGHTS; ++w) {
          const uint32_t at = red + static_cast<uint32_t>(w * each + c - first) * 512u + channel * 16u;
          uint4 u = lds128(at);
          acc[w][0] = __uint_as_float(u.x), acc[w][1] = __uint_as_float(u.y);
          acc[w][2] = __uint_as_float(u.z), acc[w][3] = __uint_as_float(u.w);
          for (int q = 1; q < p.splits; ++q) {
            u = lds128(at + static_cast<uint32_t>(q * Cfg::WEIGHTS * each) * 512u);
            acc[w][0] = __fadd_rn(acc[w][0], __uint_as_float(u.x));
            acc[w][1] = __fadd_rn(acc[w][1], __uint_as_float(u.y));
            acc[w][2] = __fadd_rn(acc[w][2], __uint_as_float(u.z));
            acc[w][3] = __fadd_rn(acc[w][3], __uint_as_float(u.w));
          }
        }
        finish(c, end, acc);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::COLS);
  }
}

}  // namespace i8
