// fp4_quant.cuh -- rows to microscaled 4-bit floating point (fp4_format.cuh), as
// they are or behind the residual's addition and the root-mean-square norm.
//
// With the norm, h = x + r and t = h * w in fp32; the norm's factor
// rstd = 1 / sqrt(mean(h^2) + eps) is one number for the row and goes into the
// row's scale, so codes and block scales are those of t and do not depend on the
// order in which the squares are summed.
//
// Bound by HBM: 2 bytes read (4 with a residual) and 0.56 written an element (and
// 2 of h).  A row a CTA of G warps; a lane holds V vectors of 8 elements, 256
// elements apart, so every element is read once.  A block is two (NV16) or four
// (MX32) neighbouring lanes: its largest magnitude takes one or two exchanges.
// Rows that the registers cannot hold (V = 0) are read twice, the second time
// mostly from L2.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "fp4_format.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

struct Fp4QuantArgs {
  const uint16_t *x, *res, *weight;
  uint16_t* h;
  uint8_t *codes, *scales;
  float* row_scales;
  int64_t ldx, ldr, ldh;
  int K, deep, G;  // deep: tiles of 256 elements to a row
  float eps;
};

// Elements e .. e + 7 of the row: t, and with the norm h and its squares' sums (as
// they are, and of h * 2^-80 and h * 2^80 for rows whose squares leave fp32's
// range).  Ordinary loads, of pointers that promise nothing: h may lie where x or
// the residual does, and a kernel that this one overlaps may have written them.
template <bool NORM>
__device__ __forceinline__ void fp4_load8(const Fp4QuantArgs& a, int64_t row, int e, float (&t)[8], uint32_t (&o)[4],
                                          float (&ss)[3]) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u), u = v, g = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  if (e < a.K) {
    v = *reinterpret_cast<const uint4*>(a.x + row * a.ldx + e);
    if (NORM && a.res) u = *reinterpret_cast<const uint4*>(a.res + row * a.ldr + e);
    if (NORM && a.weight) g = *reinterpret_cast<const uint4*>(a.weight + e);
  }
  const uint32_t x[4] = {v.x, v.y, v.z, v.w}, r[4] = {u.x, u.y, u.z, u.w}, w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    t[2 * j] = bf16_lo(x[j]);
    t[2 * j + 1] = bf16_hi(x[j]);
    if constexpr (NORM) {
      const float h0 = __fadd_rn(t[2 * j], bf16_lo(r[j])), h1 = __fadd_rn(t[2 * j + 1], bf16_hi(r[j]));
      const float s0 = h0 * 0x1p-80f, s1 = h1 * 0x1p-80f, l0 = h0 * 0x1p80f, l1 = h1 * 0x1p80f;
      ss[0] = fmaf(h0, h0, fmaf(h1, h1, ss[0]));
      ss[1] = fmaf(s0, s0, fmaf(s1, s1, ss[1]));
      ss[2] = fmaf(l0, l0, fmaf(l1, l1, ss[2]));
      t[2 * j] = __fmul_rn(h0, bf16_lo(w[j]));
      t[2 * j + 1] = __fmul_rn(h1, bf16_hi(w[j]));
      o[j] = pack_bf16x2_rn(h0, h1);
    }
  }
}

// 1 / sqrt(mean(h^2) + eps) from the three sums.
__device__ __forceinline__ float fp4_rstd(const float (&ss)[3], int K, float eps) {
  const float n = static_cast<float>(K);
  if (ss[0] >= 0x1p-60f && ss[0] < INFINITY) return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss[0], n), eps)));
  // (eps beside squares of 2^64 and more is nothing)
  if (!(ss[0] < 1.0f)) return __fdiv_rn(0x1p-80f, __fsqrt_rn(__fdiv_rn(ss[1], n)));
  // where eps * 2^160 overflows, squares below 2^-60 are nothing beside eps
  const float e = __fmul_rn(__fmul_rn(eps, 0x1p80f), 0x1p80f);
  if (!(e < INFINITY)) return __fdiv_rn(1.0f, __fsqrt_rn(eps));
  return __fdiv_rn(0x1p80f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss[2], n), e)));
}

// The codes and scales of the warp's 256 elements from `first` on, of which this
// lane holds 8 (the whole warp calls).
template <bool MX>
__device__ __forceinline__ void fp4_store256(const Fp4QuantArgs& a, int64_t row, int first, int lane,
                                             const float (&t)[8], float inverse) {
  uint32_t top = 0;  // bit patterns of magnitudes order like them; a NaN wins
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(fabsf(t[i])));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  if constexpr (MX) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  uint32_t s;
  const uint32_t c = fp4_codes8<MX>(t, top, inverse, &s);
  const int e = first + lane * 8;
  if (e < a.K) *reinterpret_cast<uint32_t*>(a.codes + row * (a.K / 2) + e / 2) = c;
  // the scales of four blocks make a word
  constexpr int LB = MX ? 4 : 2;  // lanes of a block
  s = e < a.K ? s << (8 * (lane / LB % 4)) : 0u;
  s |= __shfl_xor_sync(0xFFFFFFFFu, s, LB);
  s |= __shfl_xor_sync(0xFFFFFFFFu, s, 2 * LB);
  if (lane % (4 * LB) == 0 && e < a.deep * kFp4TileK)
    *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_at(row, e / (8 * LB), a.deep, 8 * LB)) = s;
}

template <int V, bool MX, bool NORM>
__global__ void __launch_bounds__(V == 0 ? 512 : 1024) fp4_quant_kernel(const Fp4QuantArgs a) {
  __shared__ float red_s[3][32];
  __shared__ uint32_t red_m[32];
  constexpr int H = V > 0 ? V : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int span = H * 256;  // a warp's elements, and in a long row its next ones
  const int step = a.G * span, end = a.deep * kFp4TileK;

  pdl_wait();  // the rows may be the previous kernel's output
  float t[H][8];
  uint32_t o[4];
  float ss[3] = {0.0f, 0.0f, 0.0f};
  uint32_t amax = 0;
  if constexpr (V > 0) {
    uint32_t hold[NORM ? H : 1][4];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int e = warp * span + i * 256 + lane * 8;
      fp4_load8<NORM>(a, row, e, t[i], o, ss);
      if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < 4; ++j) hold[i][j] = o[j];
      }
    }
    pdl_trigger();
    // each thread has read the elements that it writes
    if constexpr (NORM) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const int e = warp * span + i * 256 + lane * 8;
        if (a.h && e < a.K)
          *reinterpret_cast<uint4*>(a.h + row * a.ldh + e) = make_uint4(hold[i][0], hold[i][1], hold[i][2], hold[i][3]);
      }
    }
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(fabsf(t[i][j])));
  } else {
    for (int first = warp * span; first < end; first += step) {
      fp4_load8<NORM>(a, row, first + lane * 8, t[0], o, ss);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(fabsf(t[0][j])));
    }
  }
  float inverse = 1.0f;
  if (!MX || NORM) {
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if constexpr (NORM) {
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) ss[k] += __shfl_xor_sync(0xFFFFFFFFu, ss[k], d);
    }
    if (a.G > 1) {
      if (lane == 0) {
        red_m[warp] = amax;
        if constexpr (NORM) {
#pragma unroll
          for (int k = 0; k < 3; ++k) red_s[k][warp] = ss[k];
        }
      }
      __syncthreads();
      amax = 0;
      ss[0] = ss[1] = ss[2] = 0.0f;
      for (int j = 0; j < a.G; ++j) {
        amax = max(amax, red_m[j]);
        if constexpr (NORM) {
#pragma unroll
          for (int k = 0; k < 3; ++k) ss[k] += red_s[k][j];
        }
      }
    }
    const int k = nv16_row_exponent(amax);
    if constexpr (!MX) inverse = pow2f(-k);
    if (threadIdx.x == 0) {
      float s = MX ? 1.0f : amax == 0 ? 0.0f : pow2f(min(k, 127));
      if (NORM && amax != 0) s = __fmul_rn(s, fp4_rstd(ss, a.K, a.eps));
      if (!MX && amax >= 0x7F800000u) s = __uint_as_float(0x7FC00000u);  // infinity or NaN in the row
      a.row_scales[row] = s;
    }
  }
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int first = warp * span + i * 256;
      if (first < end) fp4_store256<MX>(a, row, first, lane, t[i], inverse);
    }
  } else {
    for (int first = warp * span; first < end; first += step) {
      fp4_load8<NORM>(a, row, first + lane * 8, t[0], o, ss);
      const int e = first + lane * 8;
      if (NORM && a.h && e < a.K)
        *reinterpret_cast<uint4*>(a.h + row * a.ldh + e) = make_uint4(o[0], o[1], o[2], o[3]);
      fp4_store256<MX>(a, row, first, lane, t[0], inverse);
    }
    pdl_trigger();
  }
}

}  // namespace i8
