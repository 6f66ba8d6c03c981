// fp4_pair.cuh -- the 4-bit product for many tokens: CTA pairs, one tile of 256
// tokens by 256 weight rows a pair (gated: 128 rows of each weight).
//
//   D[token, row] = sum_k x[token, k] * w[row, k]
//
// Each CTA of a pair loads 128 tokens' codes and 128 weight rows' codes of a
// stage (256 elements, 128-byte swizzle), its tokens' block scales and those of
// all 256 weight rows, which both halves of the product need; everything counts
// on CTA 0's barrier.  One thread of CTA 0 copies the scales to both CTAs' tensor
// memory and issues four M = 256, N = 256 products a stage.  Eight epilogue warps
// a CTA drain its 128 x 256 sums into registers, hand the buffer back, scale, add
// the bias (or gate), and turn 32 rows by 64 columns at a time round in shared
// memory to store four rows of 128 bytes at once (TMA stores made them wait for
// the buffer, 32 bytes from each lane are 32 lines an instruction).
//
// Tensor memory: 512 columns hold two buffers of 256 only without the scales' 48
// (NV16).  The second buffer therefore begins at column 208: while the epilogue
// warps that hold the 48 shared columns read them, nothing is issued; the rest of
// a tile is read while the next one's products run.
//
// Gated: CTA 0 loads the gate's rows and CTA 1 the up projection's, so the two
// values of an output are 128 columns apart in the same lane.
//
// Persistent: tiles go round the pairs, the larger operand's blocks slowest.  (The
// products take 64 elements each: the instruction's form for 96 does not divide a
// stage, or a tile of block scales, of 256.)
//
// 8192 x 8192 x 4096: 87 us MX32 (6.3 PFLOP/s), 90 us NV16; gated, 4096 tokens by two
// weights of 12288 x 4096, 141 and 146 us.  The products' own time at the clock that
// the power limit leaves bounds it: without the weights' loads it takes 79 us, without
// the copies of scales 87, without the epilogue 81.  Up to K = 2048 a tile's epilogue
// (2 to 2.5 us: its reads of shared memory queue behind the products') is the longer
// part.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "fp4_mma.cuh"

namespace i8 {

template <bool MX, bool GATED>
struct Fp4PairCfg {
  static constexpr int SCALES = fp4_tile_bytes(MX ? 32 : 16);
  static constexpr int PARTS = SCALES / 512;
  static constexpr int OFF_B = 16384;
  static constexpr int OFF_AS = 32768;
  static constexpr int OFF_BS = OFF_AS + SCALES;
  static constexpr int STAGE = OFF_BS + 2 * SCALES;
  static constexpr int STAGES = 5;
  static constexpr uint32_t TX = 2 * STAGE;  // both CTAs' loads
  static constexpr int TILE_N = GATED ? 128 : 256;
  static constexpr int EPI_WARPS = 8, EPI_WARP0 = 4, THREADS = 384;
  static constexpr int REG_LO = 136, REG_HI = 176;
  static_assert(128 * REG_LO + 256 * REG_HI <= THREADS * ((65536 / THREADS) & ~7));
  static constexpr int OFF_EPI = STAGES * STAGE;  // 4 KB for each epilogue warp
  // the tile's channel scales (fp32) and biases (bf16), two tiles' worth
  static constexpr int OFF_SCL = OFF_EPI + EPI_WARPS * 4096;
  static constexpr int OFF_BIAS = OFF_SCL + 2 * 256 * 4;
  static constexpr int SMEM = OFF_BIAS + 2 * 256 * 2 + 1024;
  static constexpr int COL_D1 = 208;               // the second buffer
  static constexpr int COL_AS = 464;
  static constexpr int COL_BS = COL_AS + 4 * PARTS;
  static_assert(COL_D1 + 256 <= COL_AS && COL_BS + 8 * PARTS <= 512 && STAGE % 1024 == 0);
  static_assert(SMEM <= 232448 - 512, "shared memory, with the barriers");
};

// Eight sums of a row of scale sa (twice) times their channels' scales, plus the
// biases where there are some (shared memory); in pairs.  (With the next eight's
// scales on their way it took longer: the registers are full.)
__device__ __forceinline__ void fp4_dequant8(const uint32_t* acc, unsigned long long sa, uint32_t scl, uint32_t bias,
                                             bool biased, float (&v)[8]) {
  const uint4 s0 = lds128(scl), s1 = lds128(scl + 16);
  const uint32_t s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
  unsigned long long r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    r[k] = f2_mul(f2_mul(f2(__uint_as_float(acc[2 * k]), __uint_as_float(acc[2 * k + 1])), sa),
                  f2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])));
  if (biased) {
    const uint4 bb = lds128(bias);
    const uint32_t b[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = f2_add(r[k], f2(bf16_lo(b[k]), bf16_hi(b[k])));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) f2_split(r[k], v[2 * k], v[2 * k + 1]);
}

template <bool MX, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b0,
                    const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ CUtensorMap tm_as,
                    const __grid_constant__ CUtensorMap tm_bs0, const __grid_constant__ CUtensorMap tm_bs1,
                    const __grid_constant__ Fp4GemmArgs p) {
  constexpr bool GATED = ACT != kFp4Plain;
  using Cfg = Fp4PairCfg<MX, GATED>;
  static_assert(Cfg::THREADS == 384);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_[Cfg::STAGES];
  __shared__ __align__(8) uint64_t empty_[Cfg::STAGES];
  __shared__ __align__(8) uint64_t accfull_[2];
  __shared__ __align__(8) uint64_t accfree_, chfull_, done_;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const uint32_t raw = smem_u32(smem_raw), ring = (raw + 1023u) & ~1023u;
  auto full = [&](int s) { return smem_u32(&full_[s]); };
  auto empty = [&](int s) { return smem_u32(&empty_[s]); };
  auto accfull = [&](int b) { return smem_u32(&accfull_[b]); };
  const uint32_t accfree = smem_u32(&accfree_), chfull = smem_u32(&chfull_), done = smem_u32(&done_);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int num_m = (p.M + 255) / 256, num_n = (p.N + Cfg::TILE_N - 1) / Cfg::TILE_N, tiles = num_m * num_n;
  const bool n_fastest = p.M > p.N;
  auto tile_of = [&](int i, int& mb, int& nb) {
    if (n_fastest) nb = i % num_n, mb = i / num_n;
    else mb = i % num_m, nb = i / num_m;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(full(s), 1);   // CTA 0: its producer's arrival and both CTAs' bytes
      mbar_init(empty(s), 1);  // the issuer's commit
    }
    for (int b = 0; b < 2; ++b) mbar_init(accfull(b), 1);
    mbar_init(accfree, 2 * Cfg::EPI_WARPS);
    mbar_init(chfull, Cfg::EPI_WARPS);
    mbar_init(done, 1);
    abort_word = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b0);
    if (GATED) tma_prefetch_desc(&tm_b1);
    tma_prefetch_desc(&tm_as);
    tma_prefetch_desc(&tm_bs0);
    if (GATED) tma_prefetch_desc(&tm_bs1);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();

  if (warp == 0) {
    regs_dec<Cfg::REG_LO>();
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(full(0), 0);
      Ring r;
      bool ok = true;
      int issued = 0;
      for (int i = pair; ok && i < tiles; i += pairs) {
        int mb, nb;
        tile_of(i, mb, nb);
        const int m0 = mb * 256 + static_cast<int>(rank) * 128;
        // this CTA's 128 weight rows
        const CUtensorMap* tm_b = GATED && rank == 1 ? &tm_b1 : &tm_b0;
        const int n0 = GATED ? nb * 128 : nb * 256 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < p.deep; ++kb) {
          if (!(ok = mbar_wait(empty(r.s), r.ph ^ 1u, abort_flag))) break;
          if (rank == 0) mbar_arrive_expect_tx(full(r.s), Cfg::TX);
          const uint32_t fb = full0 + 8u * static_cast<uint32_t>(r.s);
          const uint32_t st = ring + static_cast<uint32_t>(r.s * Cfg::STAGE);
          tma_load_2d_pair(st, &tm_a, fb, kb * 128, m0);
          tma_load_2d_pair(st + Cfg::OFF_B, tm_b, fb, kb * 128, n0);
          tma_load_2d_pair(st + Cfg::OFF_AS, &tm_as, fb, 0, (m0 >> 7) * p.deep + kb);
          const int row = (GATED ? nb : 2 * nb) * p.deep + kb;
          tma_load_2d_pair(st + Cfg::OFF_BS, &tm_bs0, fb, 0, row);
          if constexpr (GATED) tma_load_2d_pair(st + Cfg::OFF_BS + Cfg::SCALES, &tm_bs1, fb, 0, row);
          else tma_load_2d_pair(st + Cfg::OFF_BS + Cfg::SCALES, &tm_bs0, fb, 0, row + p.deep);
          r.advance(Cfg::STAGES);
          ++issued;
        }
      }
      // a pair that gives up ends after its copies, which CTA 0's barriers count
      if (!ok && rank == 0)
        for (int k = max(0, issued - Cfg::STAGES); k < issued; ++k)
          mbar_wait_bounded(full(k % Cfg::STAGES), (k / Cfg::STAGES) & 1, 100000000ull);
    }
  } else if (warp == 1) {
    regs_dec<Cfg::REG_LO>();
    if (rank == 0) {
      const uint32_t leader = elect_one();
      Ring r;
      bool ok = true;
      int t = 0;
      for (int i = pair; ok && i < tiles; i += pairs, ++t) {
        // the columns that this buffer shares with the one before have been read
        if (t > 0 && !(ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(accfree, (t - 1) & 1, abort_flag)))) break;
        tc_fence_after();
        const uint32_t d = tmem + (t & 1 ? Cfg::COL_D1 : 0);
        for (int kb = 0; kb < p.deep; ++kb) {
          if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(full(r.s), r.ph, abort_flag)))) break;
          tc_fence_after();
          const uint32_t st = ring + static_cast<uint32_t>(r.s * Cfg::STAGE);
          const uint64_t ad = smem_desc_sw128(st), bd = smem_desc_sw128(st + Cfg::OFF_B);
          auto scales = [&](int j) {  // those of a part
            copy_scales<2>(leader, tmem + Cfg::COL_AS + j * 4, smem_desc_scales(st + Cfg::OFF_AS + j * 512));
            copy_scales<2>(leader, tmem + Cfg::COL_BS + j * 8, smem_desc_scales(st + Cfg::OFF_BS + j * 512));
            copy_scales<2>(leader, tmem + Cfg::COL_BS + j * 8 + 4,
                           smem_desc_scales(st + Cfg::OFF_BS + Cfg::SCALES + j * 512));
          };
          scales(0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // 64 elements, 32 bytes along the swizzled row
            const int part = MX ? j / 2 : j;
            if (MX ? j == 0 : j < 3) scales(part + 1);  // while the product before runs
            const uint32_t idesc = MX && (j & 1) ? fp4_idesc<MX>(256, 256, 2) : fp4_idesc<MX>(256, 256, 0);
            mma_fp4<MX, 2>(leader, d, ad + 2u * j, bd + 2u * j, idesc, tmem + Cfg::COL_AS + part * 4,
                           tmem + Cfg::COL_BS + part * 8, kb > 0 || j > 0 ? 1u : 0u);
          }
          commit_pair_elected(leader, empty(r.s), 0x3);
          r.advance(Cfg::STAGES);
        }
        if (ok) commit_pair_elected(leader, accfull(t & 1), 0x3);
      }
      commit_pair_elected(leader, done, 0x1);
      mbar_wait_bounded(done, 0u, 100000000ull);
    }
  } else if (warp < Cfg::EPI_WARP0) {
    regs_dec<Cfg::REG_LO>();
  } else {
    regs_inc<Cfg::REG_HI>();
    const int ew = warp - Cfg::EPI_WARP0, quarter = warp & 3, half = ew >> 2;
    const uint32_t staging = ring + Cfg::OFF_EPI + static_cast<uint32_t>(ew) * 4096u;
    const uint32_t free0 = mapa_shared(accfree, 0);
    bool ok = true;
    int t = 0;
    // the scales and bias of a tile that this lane fetches, a tile ahead: of its
    // token, and of column 32 * ew + lane of the tile's 256
    float sa, s;
    uint16_t bb;
    auto fetch = [&](int i) {
      int mb, nb;
      tile_of(min(i, tiles - 1), mb, nb);
      const int m = mb * 256 + static_cast<int>(rank) * 128 + quarter * 32 + lane, c = ew * 32 + lane;
      const Fp4Weight& w = GATED && c >= 128 ? p.w[1] : p.w[0];
      const int n = GATED ? nb * 128 + (c & 127) : nb * 256 + c;
      sa = m < p.M && p.row_scales ? p.row_scales[m] : 1.0f;
      s = n < p.N && w.row_scales ? w.row_scales[n] : 1.0f;
      bb = n < p.N && w.bias ? w.bias[n] : static_cast<uint16_t>(0);
    };
    fetch(pair);
    for (int i = pair; ok && i < tiles; i += pairs, ++t) {
      int mb, nb;
      tile_of(i, mb, nb);
      const int m_base = mb * 256 + static_cast<int>(rank) * 128 + quarter * 32;
      // the tile's channel scales and biases, where the tile before has not its own
      const uint32_t scl = ring + Cfg::OFF_SCL + (t & 1) * 1024u, bias = ring + Cfg::OFF_BIAS + (t & 1) * 512u;
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(scl + 4u * (ew * 32 + lane)), "f"(s) : "memory");
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(bias + 2u * (ew * 32 + lane)), "h"(bb) : "memory");
      const unsigned long long sa_now = f2(sa, sa);
      __syncwarp();
      if (lane == 0) mbar_arrive(chfull);
      fetch(i + pairs);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(chfull, t & 1, abort_flag)) &&
           __all_sync(0xFFFFFFFFu, mbar_wait(accfull(t & 1), (t >> 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (t & 1 ? Cfg::COL_D1 : 0);
      // 128 columns of this warp: gated, 64 of each weight.  Those that the next
      // tile's buffer shares first: the last 48 of the first buffer (in the second
      // half's last 64), the first 48 of the second (in the first half's first 64)
      uint32_t acc[128];
      auto load = [&](int q) {
        const int col = GATED ? (q >> 1) * 128 + half * 64 + (q & 1) * 32 : half * 128 + q * 32;
        uint32_t r[32];
        tmem_ld_32x32b_x32(lanes + col, r);
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[q * 32 + k] = r[k];
      };
      auto hand_back = [&] {
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(accfree);
          else mbar_arrive_cluster(free0);
        }
      };
      if (t & 1) {
        if (half == 0) load(0), load(1);
        hand_back();
        if (half != 0) load(0), load(1);
        load(2), load(3);
      } else {
        if (half != 0) load(2), load(3);
        hand_back();
        load(0), load(1);
        if (half == 0) load(2), load(3);
      }
      tmem_wait_ld();
      tc_fence_before();
      const uint32_t row = staging + static_cast<uint32_t>(lane) * 128u, x = static_cast<uint32_t>(lane & 7);
#pragma unroll
      for (int g = 0; g < (GATED ? 1 : 2); ++g) {  // 64 columns of y
        const int c0 = half * (GATED ? 64 : 128) + g * 64;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float v[8], u[8];
          fp4_dequant8(&acc[g * 64 + c * 8], sa_now, scl + 4u * (c0 + c * 8), bias + 2u * (c0 + c * 8),
                       p.w[0].bias != nullptr, v);
          if constexpr (GATED) {
            fp4_dequant8(&acc[64 + c * 8], sa_now, scl + 4u * (128 + c0 + c * 8), bias + 2u * (128 + c0 + c * 8),
                         p.w[1].bias != nullptr, u);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = fp4_gate<ACT>(v[k], u[k]);
          }
          sts128(row + ((static_cast<uint32_t>(c) ^ x) << 4),
                 make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                            pack_bf16x2_rn(v[6], v[7])));
        }
        __syncwarp();
        // four rows of 128 bytes at a time
        const int n = nb * Cfg::TILE_N + c0 + (lane & 7) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = k * 4 + (lane >> 3);
          const uint4 v = lds128(staging + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>((lane & 7) ^ (r & 7)) << 4));
          if (m_base + r < p.M && n < p.N) *reinterpret_cast<uint4*>(p.y + static_cast<int64_t>(m_base + r) * p.ldy + n) = v;
        }
        __syncwarp();
      }
    }
  }

  __syncwarp();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer's loads, products and remote arrivals have ended
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace i8
