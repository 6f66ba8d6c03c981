// kv_attention.cuh -- causal attention of a step's new tokens over a paged
// cache held in 8 bits, one scale for each block of tokens and head.
//
// For a request of n tokens of which the last `new` are the step's, query
// token i (0-based) sits at position n - new + i and sees positions up to its
// own.  With codes ck, cv and block scales sk, sv of a kv head,
//   S[j]  = (q . ck[j]) * sk[block(j)] * scale
//   o     = sum_j e^(S[j] - M) sv[block(j)] cv[j] / sum_j e^(S[j] - M).
// The G = q_heads / kv_heads query heads that share a kv head, times the
// request's new tokens, are the rows r = i * G + g that read the same keys.
//
// Arithmetic:
//   * the codes are exact in fp16 (int8: |c| <= 127; E4M3: 4 significant bits;
//     read with fp16's exponent bias they are 2^-8 times their value, which the
//     scale makes good).  A row of q, bf16, is multiplied by the power of two
//     that brings its largest element into [2^14, 2^15): exact in fp16 except
//     for elements below 2^-28 of the largest, which keep an absolute error of
//     2^-40 of it.  So q . ck is a sum of exact products in fp32;
//   * softmax statistics and sums are fp32;
//   * P is rounded to fp16 (11 bits) for the second product, as
//     2^10 e^(S - M) sv / s_ref with s_ref the largest sv met so far: at most
//     2^10, and what lies 2^-35 below the maximum vanishes;
//   * both running references, M and s_ref, only grow; the accumulator is
//     rescaled when one does.
//
// The products run transposed: S^T = K q^T and O^T = V^T P^T, so that the
// tokens and the head dimension fill the 16-row side of the warp MMA
// (m16n8k16) and the few query rows its 8-wide side.  A warp takes 32 tokens
// at a time straight from global memory into the MMA's register fragments:
// the order of the head dimension inside a product and of the output's rows
// is free, so lane (g, c) = (lane / 4, lane % 4) reads 16 contiguous codes of
// token g of K, and of tokens 2c, 2c + 1 of V, and no shared memory is used.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnTile = 32;  // tokens a warp takes at a time (two halves of 16)

struct AttnArgs {
  const uint16_t* q;          // [tokens, q_heads, D] bf16
  int64_t ldq_token, ldq_head;
  const uint8_t* k;           // [blocks, kv_heads, B, D] codes
  const uint8_t* v;
  const float* k_scale;       // [blocks, kv_heads]
  const float* v_scale;
  const int32_t* table;       // [requests, width]
  int64_t ld_table;
  const int32_t* seq_lens;    // [requests]
  const int32_t* cu_new;      // [requests + 1]
  uint16_t* out;              // [tokens, q_heads, D] bf16
  int64_t ldo_token, ldo_head;
  float* lse;                 // [tokens, q_heads] or NULL
  float scale_log2;           // scale * log2(e)
  int64_t tokens;
  int64_t blocks;
  int32_t requests, width, block;
  int32_t q_heads, kv_heads, max_new;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four codes of a word as two fp16 pairs, (0, 1) and (2, 3).
template <bool E4M3>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    // sign to bit 15, the seven other bits to 13..7: 2^-8 times the value
    const uint32_t a = __byte_perm(w, 0u, 0x1404);
    const uint32_t b = __byte_perm(w, 0u, 0x3424);
    lo = (a & 0x80008000u) | ((a >> 1) & 0x3F803F80u);
    hi = (b & 0x80008000u) | ((b >> 1) & 0x3F803F80u);
  } else {
    s8x4_to_f16x4(w, lo, hi);
  }
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 t = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// What one warp holds of a row tile of 8 * NT rows.
template <int D, int NT>
struct AttnState {
  float o[D / 16][NT][4];  // O^T: rows d, columns 8 * nt + 2c + {0, 1}
  float m[NT][2];          // running maximum of S (log2 units) of those columns
  float l[NT][2];          // this lane's share of the sum of 2^(10 + S - m)
  float s_ref;             // largest block scale of V so far
};

// A row tile of a request's rows against tokens [begin, end) of one kv head,
// in steps of kAttnTile * kAttnWarps; the warp takes every kAttnWarps-th tile.
template <int D, bool E4M3, int NT>
__device__ __forceinline__ void attend_tiles(const AttnArgs& p, const int32_t* table, int head,
                                             const uint32_t (&qf)[NT][D / 16][2],
                                             const float (&rowfac)[NT][2],
                                             const int (&limit)[NT][2], int all_seen, int begin,
                                             int end, int warp, int lane, AttnState<D, NT>& st) {
  constexpr int KW = D / 64;   // 16-byte chunks of a token's K row a lane holds
  constexpr int VW = D / 128 > 0 ? D / 128 : 1;  // the same of V (8 bytes at D = 64)
  constexpr int VB = D / 8 < 16 ? D / 8 : 16;    // contiguous bytes of V a lane reads
  const int g = lane >> 2, c = lane & 3;
  const int64_t head_stride = static_cast<int64_t>(p.block) * D;

  for (int t0 = begin + warp * kAttnTile; t0 < end; t0 += kAttnTile * kAttnWarps) {
    uint4 kr[2][2][KW];      // [half][token g, g + 8][chunk]
    uint32_t vr[2][4][VW * 4];
    float sk[2], sv[2];
    bool gone[2];            // no such block: its tokens are left out
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = t0 + 16 * h;
      const int b = t / p.block;
      int64_t blk = -1;
      if (t < end) {  // end lies within the table's width
        blk = table[b];
        if (blk < 0 || blk >= p.blocks) {
          if (lane == 0) atomicOr(&g_status, 1u << 7);
          blk = -1;
        }
      }
      gone[h] = blk < 0;
      sk[h] = sv[h] = 0.0f;
      if (blk >= 0) {
        const int64_t base = (blk * p.kv_heads + head) * head_stride + static_cast<int64_t>(t - b * p.block) * D;
        const uint8_t* kp = p.k + base;
        const uint8_t* vp = p.v + base;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < KW; ++j)
            kr[h][i][j] = ld_stream_v4(kp + (g + 8 * i) * D + j * 64 + c * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tk = 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            if constexpr (VB == 16) {
              const uint4 x = ld_stream_v4(vp + tk * D + j * 128 + g * 16);
              vr[h][i][4 * j] = x.x;
              vr[h][i][4 * j + 1] = x.y;
              vr[h][i][4 * j + 2] = x.z;
              vr[h][i][4 * j + 3] = x.w;
            } else {
              const uint2 x = __ldg(reinterpret_cast<const uint2*>(vp + tk * D + g * 8));
              vr[h][i][0] = x.x;
              vr[h][i][1] = x.y;
            }
          }
        }
        sk[h] = p.k_scale[blk * p.kv_heads + head];
        sv[h] = p.v_scale[blk * p.kv_heads + head];
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < KW; ++j) kr[h][i][j] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < VW * 4; ++j) vr[h][i][j] = 0u;
      }
    }
    // ---- S^T
    float s[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[h][n][i] = 0.0f;
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        const uint32_t w0[4] = {kr[h][0][j].x, kr[h][0][j].y, kr[h][0][j].z, kr[h][0][j].w};
        const uint32_t w1[4] = {kr[h][1][j].x, kr[h][1][j].y, kr[h][1][j].z, kr[h][1][j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          codes_to_f16<E4M3>(w0[i], a0, a2);
          codes_to_f16<E4M3>(w1[i], a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_16816(s[h][n], a0, a1, a2, a3, qf[n][4 * j + i][0], qf[n][4 * j + i][1]);
        }
      }
    }
    // ---- softmax
    const bool masked = t0 + kAttnTile > all_seen || gone[0] || gone[1];
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[h][n][i] *= sk[h] * rowfac[n][i & 1];
          if (masked && (gone[h] || t0 + 16 * h + g + 8 * (i >> 1) >= limit[n][i & 1]))
            s[h][n][i] = -INFINITY;
          top[n][i & 1] = fmaxf(top[n][i & 1], s[h][n][i]);
        }
    }
    const float s_ref = fmaxf(st.s_ref, fmaxf(sv[0], sv[1]));
    const float grow = s_ref > 0.0f ? __fdividef(st.s_ref, s_ref) : 0.0f;
    bool moved = s_ref != st.s_ref;
    float alpha[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = top[n][i];
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
        const float m = fmaxf(st.m[n][i], x);
        moved = moved || m != st.m[n][i];
        // a row that has seen nothing yet keeps m = -inf: its factor is 0
        alpha[n][i] = m > -INFINITY ? ex2(st.m[n][i] - m) : 0.0f;
        st.m[n][i] = m;
        st.l[n][i] *= alpha[n][i];
      }
    st.s_ref = s_ref;
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) st.o[j][n][i] *= alpha[n][i & 1] * grow;
    }
    // ---- P^T and O^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float vs = s_ref > 0.0f ? __fdividef(sv[h], s_ref) : 0.0f;
      uint32_t b[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = st.m[n][i & 1];
          e[i] = s[h][n][i] > -INFINITY ? ex2(s[h][n][i] - m + 10.0f) : 0.0f;
          st.l[n][i & 1] += e[i];
        }
        b[n][0] = transpose_8x8(pack_f16x2(e[0] * vs, e[1] * vs));
        b[n][1] = transpose_8x8(pack_f16x2(e[2] * vs, e[3] * vs));
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {  // word j of the V rows: 4 head dimensions, 2 MMAs
        uint32_t f[2][4];                 // [tokens 2c.., 8 + 2c..][head dimension]
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = vr[h][2 * i][j], y = vr[h][2 * i + 1][j];
          codes_to_f16<E4M3>(__byte_perm(x, y, 0x5140), f[i][0], f[i][1]);
          codes_to_f16<E4M3>(__byte_perm(x, y, 0x7362), f[i][2], f[i][3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_16816(st.o[2 * j + i][n], f[0][2 * i], f[0][2 * i + 1], f[1][2 * i],
                      f[1][2 * i + 1], b[n][0], b[n][1]);
      }
    }
  }
}

// Head dimension of O^T row `half` (0: row g, 1: row g + 8) of m-tile j.
// m-tile 2w + i takes bytes 2i, 2i + 1 of word w of the lane's V chunk.
template <int D>
__device__ __forceinline__ int attn_out_dim(int j, int half, int g) {
  constexpr int VB = D / 8 < 16 ? D / 8 : 16;
  const int byte = 2 * j + half;               // among the lane's D / 8 bytes
  return (byte / VB) * 128 + g * VB + byte % VB;
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kAttnThreads) kv_attention_kernel(const AttnArgs p) {
  constexpr int ROWS = 8 * NT;
  extern __shared__ float sm_o[];   // [warps][ROWS][D]
  __shared__ float sm_m[kAttnWarps][ROWS], sm_l[kAttnWarps][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int row_tiles = (p.max_new * (p.q_heads / p.kv_heads) + ROWS - 1) / ROWS;
  const int req = blockIdx.x / row_tiles, head = blockIdx.y;
  const int group = p.q_heads / p.kv_heads;

  pdl_wait();
  const int64_t q0 = p.cu_new[req];
  int fresh = p.cu_new[req + 1] - p.cu_new[req];
  const int len = p.seq_lens[req];
  if (q0 < 0 || q0 + fresh > p.tokens || fresh > p.max_new) {
    if (threadIdx.x == 0) atomicOr(&g_status, 1u << 7);
    return;
  }
  const int rows = fresh * group;
  const int row0 = (blockIdx.x % row_tiles) * ROWS;
  if (row0 >= rows) return;
  const int pos0 = len - fresh;  // position of the request's first new token

  // q fragments (column n of a tile is row g) and what the lane's two columns
  // of S^T need: their factor and the first position that they do not see
  uint32_t qf[NT][D / 16][2];
  float rowfac[NT][2];
  int limit[NT][2];
  int most = 0, least = 0x7FFFFFFF;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 8 * n + g;
    const bool real = r < rows;
    const int i = real ? r / group : 0;
    const uint16_t* qp = p.q + (q0 + i) * p.ldq_token + (head * group + (real ? r - i * group : 0)) * p.ldq_head;
    uint2 w[D / 16];
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      // step j = 4 * chunk + word: head dimensions chunk * 64 + c * 16 + 4 * word ..
      const int d = (j >> 2) * 64 + c * 16 + (j & 3) * 4;
      w[j] = real ? __ldg(reinterpret_cast<const uint2*>(qp + d)) : make_uint2(0u, 0u);
      const uint32_t a = (w[j].x & 0x7FFF7FFFu), b = (w[j].y & 0x7FFF7FFFu);
      amax = max(amax, max(max(a & 0xFFFFu, a >> 16), max(b & 0xFFFFu, b >> 16)));
    }
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    // 2^e with e = 14 - exponent(amax): amax * 2^e in [2^14, 2^15).  For rows
    // of zeros or below 2^-100 the largest factor kept in range is 2^114.
    const int e = 14 - max(static_cast<int>(amax >> 7) - 127, -100);
    const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      qf[n][j][0] = pack_f16x2(__uint_as_float(w[j].x << 16) * up, __uint_as_float(w[j].x & 0xFFFF0000u) * up);
      qf[n][j][1] = pack_f16x2(__uint_as_float(w[j].y << 16) * up, __uint_as_float(w[j].y & 0xFFFF0000u) * up);
    }
    // row g's exponent and limit go to the lanes whose columns 2c, 2c + 1 it is
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * (E4M3 ? 256.0f : 1.0f) * p.scale_log2;
    const int lim = real ? min(max(pos0 + i + 1, 0), len) : 0;
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
      rowfac[n][i2] = __shfl_sync(0xFFFFFFFFu, down, (2 * c + i2) * 4);
      limit[n][i2] = __shfl_sync(0xFFFFFFFFu, lim, (2 * c + i2) * 4);
    }
    most = max(most, lim);
    least = min(least, real ? lim : 0x7FFFFFFF);
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (most > p.width * p.block) {  // more tokens than the table has columns for
    if (threadIdx.x == 0) atomicOr(&g_status, 1u << 7);
    most = p.width * p.block;
  }
  least = __reduce_min_sync(0xFFFFFFFFu, least);

  AttnState<D, NT> st;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    st.m[n][0] = st.m[n][1] = -INFINITY;
    st.l[n][0] = st.l[n][1] = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[j][n][i] = 0.0f;
  }
  st.s_ref = 0.0f;
  attend_tiles<D, E4M3, NT>(p, p.table + req * p.ld_table, head, qf, rowfac, limit, least, 0, most,
                            warp, lane, st);

  // ---- the four warps' parts meet
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = st.l[n][i];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      const int col = 8 * n + 2 * c + i;
      if (g == 0) {
        sm_m[warp][col] = st.m[n][i];
        sm_l[warp][col] = l;
      }
    }
  const float unit = st.s_ref * (E4M3 ? 256.0f : 1.0f);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sm_o[(warp * ROWS + 8 * n + 2 * c + (i & 1)) * D + attn_out_dim<D>(j, i >> 1, g)] =
            st.o[j][n][i] * unit;
  __syncthreads();
  pdl_trigger();
  for (int e = threadIdx.x * 2; e < ROWS * D; e += kAttnThreads * 2) {
    const int row = e / D, d = e - row * D;
    const int r = row0 + row;
    if (r >= rows) break;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, sm_m[w][row]);
    float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float f = sm_m[w][row] > -INFINITY ? ex2(sm_m[w][row] - m) : 0.0f;
      const float2 o = *reinterpret_cast<const float2*>(sm_o + (w * ROWS + row) * D + d);
      l = fmaf(f, sm_l[w][row], l);
      o0 = fmaf(f, o.x, o0);
      o1 = fmaf(f, o.y, o1);
    }
    const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;  // a row that sees nothing gives 0
    const int i = r / group, hq = head * group + r - i * group;
    const __nv_bfloat162 y = __floats2bfloat162_rn(o0 * inv, o1 * inv);
    *reinterpret_cast<__nv_bfloat162*>(p.out + (q0 + i) * p.ldo_token + hq * p.ldo_head + d) = y;
    if (p.lse && d == 0)
      p.lse[(q0 + i) * p.q_heads + hq] =
          l > 0.0f ? (m + (log2f(l) - 10.0f)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace i8
