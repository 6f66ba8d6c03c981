// fp4_mma.cuh -- the tensor core's block-scaled 4-bit products: PTX wrappers,
// descriptors, and the steps that the two product kernels share.
#pragma once
#include <cstdint>

#include "fp4_format.cuh"
#include "gelu.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

// Instruction descriptor of kind::mxf4 (MX32) and kind::mxf4nvf4 (NV16): E2M1
// operands (format 1 in bits 7-9 and 10-12), both K-major, N >> 3 (bits 17-22),
// the scales' format (bit 23: 1 for E8M0), M >> 4 (bits 24-28), K = 64.  The
// scales' byte in a column: bits 4-5 (B) and 29-30 (A).
template <bool MX>
__device__ constexpr uint32_t fp4_idesc(int M, int N, int byte) {
  return (static_cast<uint32_t>(byte) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (MX ? 1u << 23 : 0u) | (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(byte) << 29);
}

// One lane of a converged warp: 1 in it, 0 in the others.  The issuing warp stays
// converged and its operands are the same in all lanes, so they reach the tensor
// core's instructions without a detour; one lane's predicate issues them.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t q;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(q));
  return q;
}

// D (+)= A * B^T of 64 elements, the operands scaled by blocks of 16 or 32.
#define I8_MMA_FP4(form)                                                                                \
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"          \
               "@q tcgen05.mma." form " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                \
               "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(leader)                \
               : "memory")
template <bool MX, int CTAS>
__device__ __forceinline__ void mma_fp4(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (MX && CTAS == 1) I8_MMA_FP4("cta_group::1.kind::mxf4.block_scale.scale_vec::2X");
  else if constexpr (MX) I8_MMA_FP4("cta_group::2.kind::mxf4.block_scale.scale_vec::2X");
  else if constexpr (CTAS == 1) I8_MMA_FP4("cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X");
  else I8_MMA_FP4("cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X");
}
#undef I8_MMA_FP4

// mma_commit and mma_commit_pair by the elected lane.
__device__ __forceinline__ void commit_elected(uint32_t leader, uint32_t bar) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
               "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
               "r"(leader)
               : "memory");
}
__device__ __forceinline__ void commit_pair_elected(uint32_t leader, uint32_t bar, uint16_t cta_mask) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
               "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
                   "r"(bar), "h"(cta_mask), "r"(leader)
               : "memory");
}

// Matrix descriptor of a 512-byte part of block scales: 32 rows of 16 bytes, no
// swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128u >> 4) << 32) |
         (static_cast<uint64_t>(1u) << 46);
}

// A part of block scales into four columns of tensor memory, the same for each
// quarter of the lanes.  Ordered with this thread's products before and behind it.
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t leader, uint32_t tmem, uint64_t desc) {
  if constexpr (CTAS == 1)
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                 "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem), "l"(desc), "r"(leader)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                 "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem), "l"(desc), "r"(leader)
                 : "memory");
}

// Bulk copy of `bytes` (a multiple of 16) from global memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The halves of a cluster's barrier (whole warps call): the arrival orders no
// memory, it only says that the CTA is there.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 16 bytes into the shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_cluster_v4(uint32_t to, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// What a product's epilogue does: nothing more, or act(g) * u.
enum Fp4Epilogue : int { kFp4Plain = 0, kFp4Silu = 1, kFp4Gelu = 2 };

// act(g) * u in fp32.  silu(g) = g / (1 + exp(-g)): exp(-g) = infinity gives 0.  (Both
// sides of the quotient in quarters: the reciprocal of a divisor above 2^126 is 0.)
template <int ACT>
__device__ __forceinline__ float fp4_gate(float g, float u) {
  if constexpr (ACT == kFp4Silu) return 0.25f * g * rcp_approx(fmaf(0.25f, __expf(-g), 0.25f)) * u;
  else return gelu_erf(g) * u;
}

struct Fp4Weight {
  const uint8_t* scales;
  const float* row_scales;  // null: ones
  const uint16_t* bias;     // null: zeros
};

struct Fp4GemmArgs {
  Fp4Weight w[2];           // the second of a gated product only
  const uint8_t* scales;    // the tokens'
  const float* row_scales;  // null: ones
  const uint16_t* x;        // or the tokens themselves, bf16
  int64_t ldx;
  uint16_t* y;
  int64_t ldy;
  int M, N;                 // tokens, channels
  int K, deep;              // elements, tiles of 256 of them
  int splits, deep_per_split;
};

// acc * s_a * s_w + bias.
__device__ __forceinline__ float fp4_dequant(float acc, float sa, float sw, float b) {
  return __fadd_rn(__fmul_rn(__fmul_rn(acc, sa), sw), b);
}

}  // namespace i8
