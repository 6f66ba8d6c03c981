// fp4_quant.cuh -- rows to microscaled 4-bit floating point (fp4_format.cuh), as
// they are or behind the residual's addition and the root-mean-square norm.
//
// With the norm, h = x + r and t = h * w in fp32; the norm's factor
// rstd = 1 / sqrt(mean(h^2) + eps) is one number for the row and goes into the
// row's scale, so codes and block scales are those of t and do not depend on the
// order in which the squares are summed.
//
// Bound by HBM: 2 bytes read (4 with a residual) and 0.56 written an element (and
// 2 of h).  A row is G warps, a CTA R rows (several where they are short); a lane holds V vectors of 8 elements, 256
// elements apart, so every element is read once.  A block is two (NV16) or four
// (MX32) neighbouring lanes: its largest magnitude takes one or two exchanges.
// Rows that the registers cannot hold (V = 0) are read twice, the second time
// mostly from L2.
//
// The fewer warps a row, the better (8192 x 8192 NV16: V = 2 51 us, 4 40, 8 37, 4.7
// TB/s; MX32 28 us, 6.1 TB/s; with the residual and the norm, V = 4, 79 us, 5.6 TB/s,
// MX32 75, 5.8).  NV16 alone is the farthest from HBM's rate: it may write nothing
// before the row's maximum is known, a CTA has one row in flight, and a third of the
// warps that an SM holds are there; with the norm the same wait is shared by nearly
// three times the bytes.  A few rows are latency: 2 us for one to 64 rows of 4096.
#pragma once
#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "fp4_format.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

// Lane-wise larger magnitude of bf16 pairs; a NaN wins; the signs are to be masked
// off.
__device__ __forceinline__ uint32_t absmax_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

struct Fp4QuantArgs {
  const uint16_t *x, *res, *weight;
  uint16_t* h;
  uint8_t *codes, *scales;
  float* row_scales;
  int64_t ldx, ldr, ldh;
  int64_t rows;
  int K, deep, G, R;  // deep: tiles of 256 elements to a row
  float eps;
};

// Eight elements of a row that a lane holds: as they are, or with the norm h, not
// rounded (its product with the gain is made again where it is wanted: a register
// is dearer than a load from L1).
template <bool NORM>
struct Fp4Held {
  uint4 x;
};
template <>
struct Fp4Held<true> {
  float h[8];
};

// The gains of elements e .. e + 7, bf16.
__device__ __forceinline__ uint4 fp4_gains(const Fp4QuantArgs& a, int e) {
  return a.weight && e < a.K ? *reinterpret_cast<const uint4*>(a.weight + e)
                             : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
}

// Elements e .. e + 7 of the row as they are held.  Ordinary loads, of pointers that
// promise nothing: h may lie where x or the residual does, and a kernel that this
// one overlaps may have written them.
template <bool NORM>
__device__ __forceinline__ void fp4_load8(const Fp4QuantArgs& a, int64_t row, int e, Fp4Held<NORM>& held) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (e < a.K) v = *reinterpret_cast<const uint4*>(a.x + row * a.ldx + e);
  if constexpr (!NORM) {
    held.x = v;
  } else {
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (a.res && e < a.K) u = *reinterpret_cast<const uint4*>(a.res + row * a.ldr + e);
    const uint32_t x[4] = {v.x, v.y, v.z, v.w}, r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      held.h[2 * j] = __fadd_rn(bf16_lo(x[j]), bf16_lo(r[j]));
      held.h[2 * j + 1] = __fadd_rn(bf16_hi(x[j]), bf16_hi(r[j]));
    }
  }
}

// What is quantized: the elements, or t = h * gain.
template <bool NORM>
__device__ __forceinline__ void fp4_widen(const Fp4QuantArgs& a, int e, const Fp4Held<NORM>& held, float (&t)[8]) {
  if constexpr (NORM) {
    const uint4 g = fp4_gains(a, e);
    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[2 * j] = __fmul_rn(held.h[2 * j], bf16_lo(w[j]));
      t[2 * j + 1] = __fmul_rn(held.h[2 * j + 1], bf16_hi(w[j]));
    }
  } else {
    const uint32_t w[4] = {held.x.x, held.x.y, held.x.z, held.x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) t[2 * j] = bf16_lo(w[j]), t[2 * j + 1] = bf16_hi(w[j]);
  }
}

// Bits of the largest magnitude of what is quantized, which order like the values
// (a NaN wins), and with the norm the squares' sum.
template <bool NORM>
__device__ __forceinline__ uint32_t fp4_top(const Fp4QuantArgs& a, int e, const Fp4Held<NORM>& held, float& ss) {
  if constexpr (NORM) {
    float t[8];
    fp4_widen<true>(a, e, held, t);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m = max(m, __float_as_uint(fabsf(t[j])));
      ss = fmaf(held.h[j], held.h[j], ss);
    }
    return m;
  } else {
    const uint4& x = held.x;
    const uint32_t m = absmax_nan_bf16x2(absmax_nan_bf16x2(x.x, x.y), absmax_nan_bf16x2(x.z, x.w)) & 0x7FFF7FFFu;
    return max(m << 16, m & 0xFFFF0000u);
  }
}

// Of rows whose squares, or whose t, leave fp32's range: the squares' sums of h * 2^-80
// and of h * 2^80, and the bits of the largest magnitude of t * 2^-126.
__device__ __forceinline__ void fp4_down(Fp4Held<true>& held) {
#pragma unroll
  for (int j = 0; j < 8; ++j) held.h[j] = __fmul_rn(held.h[j], 0x1p-126f);
}
__device__ __forceinline__ void fp4_far(const Fp4QuantArgs& a, int e, const Fp4Held<true>& held, float (&ss)[3],
                                        uint32_t& down) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = held.h[j] * 0x1p-80f, l = held.h[j] * 0x1p80f;
    ss[1] = fmaf(s, s, ss[1]);
    ss[2] = fmaf(l, l, ss[2]);
  }
  Fp4Held<true> low = held;
  float unused = 0.0f;
  fp4_down(low);
  down = max(down, fp4_top<true>(a, e, low, unused));
}

template <bool NORM>
__device__ __forceinline__ void fp4_store_h(const Fp4QuantArgs& a, int64_t row, int e, const Fp4Held<NORM>& held) {
  if constexpr (NORM)
    if (a.h && e < a.K)
      *reinterpret_cast<uint4*>(a.h + row * a.ldh + e) =
          make_uint4(pack_bf16x2_rn(held.h[0], held.h[1]), pack_bf16x2_rn(held.h[2], held.h[3]),
                     pack_bf16x2_rn(held.h[4], held.h[5]), pack_bf16x2_rn(held.h[6], held.h[7]));
}

__device__ __forceinline__ void warp_sum(float& v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
}

// Whether a sum of squares says all there is to say.
__device__ __forceinline__ bool fp4_in_range(float ss) { return ss >= 0x1p-60f && ss < INFINITY; }

// scale / sqrt(mean(h^2) + eps) from the sum of squares and, where that is out of
// range, the two others; times 2^126 where `over`, t having been taken times 2^-126
// (by steps that stay in range).  The factor of rows below 2^-128 is no fp32 number (eps = 0):
// its product with NV16's scale is one again, and MX32 gets the largest there is.
__device__ __forceinline__ float fp4_normed_scale(float scale, const float (&ss)[3], int K, float eps, bool over) {
  const float n = static_cast<float>(K);
  if (fp4_in_range(ss[0])) {
    const float r = __fmul_rn(scale, __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss[0], n), eps))));
    return over ? __fmul_rn(r, 0x1p126f) : r;
  }
  // (eps beside squares of 2^64 and more is nothing)
  if (!(ss[0] < 1.0f)) {
    const float m = over ? 0x1p23f : 0x1p-40f;  // squared, 2^-80 or 2^-80 * 2^126
    return __fmul_rn(__fmul_rn(__fmul_rn(scale, m), __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss[1], n)))), m);
  }
  // where eps * 2^160 overflows, squares below 2^-60 are nothing beside eps
  const float e = __fmul_rn(__fmul_rn(eps, 0x1p80f), 0x1p80f);
  if (!(e < INFINITY)) return __fmul_rn(scale, __fdiv_rn(1.0f, __fsqrt_rn(eps)));
  const float d = __fsqrt_rn(__fadd_rn(__fdiv_rn(ss[2], n), e));
  const float r = d < 1.0f ? __fmul_rn(__fdiv_rn(scale, d), 0x1p80f) : __fmul_rn(scale, __fdiv_rn(0x1p80f, d));
  return r == INFINITY ? FLT_MAX : r;
}

// NV16: a row's scale from the bits of its largest magnitude, and s and 1 / s for its
// codes; s = 0 where they want a power of two before (fp4_row_scaled).
__device__ __forceinline__ float fp4_row_scale(uint32_t amax, float& s, float& inverse) {
  const int k = nv16_row_exponent(amax);
  inverse = pow2f(-k);
  s = abs(k) <= 100 ? pow2f(k) : 0.0f;
  if (amax >= 0x7F800000u) return __uint_as_float(0x7FC00000u);  // infinity or NaN in the row
  return amax == 0 ? 0.0f : pow2f(k);
}
__device__ __forceinline__ void fp4_row_scaled(float (&t)[8], uint32_t& top, float& s, float& inverse) {
  if (s == 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __fmul_rn(t[i], inverse);
    top = __float_as_uint(__fmul_rn(__uint_as_float(top), inverse));
    s = inverse = 1.0f;
  }
}

// The codes and scales of the warp's 256 elements from `first` on, of which this
// lane holds 8 with the largest magnitude `top` (the whole warp calls).  codes and
// scales: the row's, the latter where its tiles' first part has it.
template <bool MX, bool NORM>
__device__ __forceinline__ void fp4_store256(const Fp4QuantArgs& a, uint8_t* codes, uint8_t* scales, int first, int lane,
                                             const Fp4Held<NORM>& held, uint32_t top, float s, float inverse) {
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  if constexpr (MX) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  float t[8];
  fp4_widen<NORM>(a, first + lane * 8, held, t);
  if constexpr (!MX) fp4_row_scaled(t, top, s, inverse);
  uint32_t scale;
  const uint32_t c = fp4_codes8<MX>(t, top, s, inverse, &scale);
  const int e = first + lane * 8;
  if (e < a.K) *reinterpret_cast<uint32_t*>(codes + e / 2) = c;
  // the scales of four blocks make a word; those past K are 0
  constexpr int LB = MX ? 4 : 2;  // lanes of a block
  scale = e < a.K ? scale << (8 * (lane / LB % 4)) : 0u;
  scale |= __shfl_xor_sync(0xFFFFFFFFu, scale, LB);
  scale |= __shfl_xor_sync(0xFFFFFFFFu, scale, 2 * LB);
  if (lane % (4 * LB) == 0)
    *reinterpret_cast<uint32_t*>(scales + (first >> 8) * fp4_tile_bytes(8 * LB) + lane / (4 * LB) * 512) = scale;
}

// Registers a thread, at most: what the usual row needs.  The rare rows' code would take
// more and cost CTAs (8192 x 8192 with the norm, NV16: 79 us, and 99 with 86 registers).
constexpr int fp4_quant_registers(int V, bool mx, bool norm) {
  return V <= 1 ? (norm && !mx ? 40 : 32) : norm && V == 2 ? 56 : norm && V == 4 ? 80 : V == 8 && mx && !norm ? 64 : 128;
}

template <int V, bool MX, bool NORM>
__global__ void __maxnreg__(fp4_quant_registers(V, MX, NORM)) fp4_quant_kernel(const Fp4QuantArgs a) {
  __shared__ float red_s[3][32];
  __shared__ uint32_t red_m[32];
  constexpr int H = V > 0 ? V : 1;
  // (block: lanes, a row's warps, rows)
  const int lane = threadIdx.x, warp = threadIdx.y, local = threadIdx.z;
  // (a row behind the last one is the last one, read but not written)
  const bool mine = static_cast<int64_t>(blockIdx.x) * a.R + local < a.rows;
  const int64_t row = min(static_cast<int64_t>(blockIdx.x) * a.R + local, a.rows - 1);
  const int span = H * 256;  // a warp's elements, and in a long row its next ones
  const int step = a.G * span, end = a.deep * kFp4TileK;

  pdl_wait();  // the rows may be the previous kernel's output
  pdl_trigger();
  Fp4Held<NORM> held[H];
  uint32_t top[H];
  float ss[3] = {0.0f, 0.0f, 0.0f};
  uint32_t amax = 0;
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < H; ++i) fp4_load8<NORM>(a, row, warp * span + i * 256 + lane * 8, held[i]);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      top[i] = fp4_top<NORM>(a, warp * span + i * 256 + lane * 8, held[i], ss[0]);
      amax = max(amax, top[i]);
    }
  } else {
    for (int first = warp * span; first < end; first += step) {
      fp4_load8<NORM>(a, row, first + lane * 8, held[0]);
      amax = max(amax, fp4_top<NORM>(a, first + lane * 8, held[0], ss[0]));
    }
  }
  float s = 1.0f, inverse = 1.0f;
  bool over = false;  // t leaves fp32's range, h does not
  if (!MX || NORM) {
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if constexpr (NORM) warp_sum(ss[0]);
    if (a.G > 1) {
      if (lane == 0) {
        red_m[local * a.G + warp] = amax;
        if constexpr (NORM) red_s[0][local * a.G + warp] = ss[0];
      }
      __syncthreads();
      amax = 0;
      ss[0] = 0.0f;
      for (int j = 0; j < a.G; ++j) {
        amax = max(amax, red_m[local * a.G + j]);
        if constexpr (NORM) ss[0] += red_s[0][local * a.G + j];
      }
    }
    if constexpr (NORM) {
      // squares or t out of fp32's range in a row of the CTA: the other sums as well
      if (__syncthreads_or(!fp4_in_range(ss[0]) || amax == 0x7F800000u)) {
        uint32_t down = 0;
        if constexpr (V > 0) {
#pragma unroll
          for (int i = 0; i < H; ++i) fp4_far(a, warp * span + i * 256 + lane * 8, held[i], ss, down);
        } else {
          for (int first = warp * span; first < end; first += step) {
            fp4_load8<NORM>(a, row, first + lane * 8, held[0]);  // (h is not stored yet)
            fp4_far(a, first + lane * 8, held[0], ss, down);
          }
        }
        warp_sum(ss[1]);
        warp_sum(ss[2]);
        down = __reduce_max_sync(0xFFFFFFFFu, down);
        if (a.G > 1) {
          if (lane == 0) {
            red_s[1][local * a.G + warp] = ss[1];
            red_s[2][local * a.G + warp] = ss[2];
            red_m[local * a.G + warp] = down;  // (the first ones have been read)
          }
          __syncthreads();
          ss[1] = ss[2] = 0.0f;
          for (int j = 0; j < a.G; ++j) {
            ss[1] += red_s[1][local * a.G + j];
            ss[2] += red_s[2][local * a.G + j];
            down = max(down, red_m[local * a.G + j]);
          }
        }
        over = amax == 0x7F800000u && ss[1] < INFINITY;
        if (over) amax = down;
      }
      // (each thread has read the elements that it writes)
      if constexpr (V > 0) {
#pragma unroll
        for (int i = 0; i < H; ++i)
          if (mine) fp4_store_h<NORM>(a, row, warp * span + i * 256 + lane * 8, held[i]);
        if (over) {
          float unused = 0.0f;
#pragma unroll
          for (int i = 0; i < H; ++i) {
            fp4_down(held[i]);
            top[i] = fp4_top<NORM>(a, warp * span + i * 256 + lane * 8, held[i], unused);
          }
        }
      }
    }
    float scale = MX ? 1.0f : fp4_row_scale(amax, s, inverse);
    if (NORM && amax != 0) scale = fp4_normed_scale(scale, ss, a.K, a.eps, over);
    if (mine && warp == 0 && lane == 0) a.row_scales[row] = scale;
  }
  uint8_t* codes = a.codes + row * (a.K / 2);
  uint8_t* scales = a.scales + fp4_scale_at(row, 0, a.deep, MX ? 32 : 16);
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int first = warp * span + i * 256;
      if (mine && first < end) fp4_store256<MX, NORM>(a, codes, scales, first, lane, held[i], top[i], s, inverse);
    }
  } else {
    for (int first = warp * span; first < end; first += step) {
      float sum = 0.0f;
      fp4_load8<NORM>(a, row, first + lane * 8, held[0]);
      fp4_store_h<NORM>(a, row, first + lane * 8, held[0]);
      if constexpr (NORM)
        if (over) fp4_down(held[0]);
      fp4_store256<MX, NORM>(a, codes, scales, first, lane, held[0], fp4_top<NORM>(a, first + lane * 8, held[0], sum), s,
                             inverse);
    }
  }
}

}  // namespace i8
