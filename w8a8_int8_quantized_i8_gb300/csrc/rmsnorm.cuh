// rmsnorm.cuh -- the residual's addition, the root-mean-square norm with a
// gain, and the per-token quantizer of its output, in one pass over a row.
//
// For a row of x, a residual r and a gain w, all bf16:
//   h = x + r                      (stored as the new residual, bf16)
//   y = h * rstd * w,  rstd = 1 / sqrt(mean(h^2) + eps)
//   scale = max|y| / L,  code = rne(y / scale),  L = 127 (int8) or 448 (E4M3)
// rstd is one number for the row, so it cancels in y / scale.  With t = h * w:
//   code = rne(t / s_t),  s_t = max|t| / L,  scale = s_t * rstd.
// The sum of squares and max|t| therefore come out of the same reduction, one
// barrier a row, and the codes do not depend on the order in which the squares
// are summed.  h and t are fp32 (h is rounded to bf16 only where it is stored;
// the norm uses the unrounded sum), and the row is never rounded to bf16
// between the norm and the quantizer: one rounding, to the 8-bit code.
//
// The squares of a row leave fp32's range long before the row or its norm does.
// A vector of 8 whose squares do not fit well is put aside: its h is stored
// later (it may lie where x or r does).  A row whose sum of squares is infinite
// or below 2^-60 is then read again and done times 2^-80 or 2^80, which its scale
// undoes; the vectors not put aside do not count beside the others.
//
// Bound by HBM: 2 + 2 bytes read and 2 + 1 written an element.  A row a CTA, as
// in the quantizer: small CTAs spread evenly, each element is read once and
// stays in registers.  16384 x 3072, E4M3: 60.1 us, 5.9 TB/s (88 % of the
// measured copy rate); one row of 3072: 2.7 us, a launch.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

// 8 fp32 -> 8 int8 codes, rne(fl(t / s)): t * fl(1/s) is within 2^-15 of
// fl(t / s), so only a value within 2^-14 of a tie needs the IEEE division
// (quant.cuh has the bound; it does not depend on t being a bf16 value).
__device__ __forceinline__ uint2 quant_f32x8(const float (&t)[8], float s, float r, bool fast) {
  uint32_t b[8];
  float dmax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = __fmul_rn(t[i], r);
    const float y = __fadd_rn(q, kRoundMagic);
    dmax = fmaxf(dmax, fabsf(__fsub_rn(q, __fsub_rn(y, kRoundMagic))));
    b[i] = __float_as_uint(y);
  }
  if (!fast || !(dmax <= kNearTie)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = quant_exact(t[i], s);
  }
  return make_uint2(low_bytes4(b[0], b[1], b[2], b[3]), low_bytes4(b[4], b[5], b[6], b[7]));
}

// 8 fp32 -> 8 E4M3 codes of fl(t / s).  q = t * fl(1/s) is within 3 units in
// the last place of fl(t / s).  E4M3 keeps 3 of the 23 mantissa bits, so both
// round alike unless the 20 dropped bits of q lie within 4 of one half; below
// 2^-6 (E4M3's subnormals, another spacing) the division decides as well.
__device__ __forceinline__ uint2 quant_f32x8_e4m3(const float (&t)[8], float s, float r,
                                                  bool fast) {
  float q[8];
  bool sure = fast;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = __fmul_rn(t[i], r);
    const uint32_t u = __float_as_uint(q[i]);
    const bool tie = ((u & 0xFFFFFu) - (0x80000u - 4u)) <= 8u;
    sure = sure && !tie && (fabsf(q[i]) >= 0x1p-6f || t[i] == 0.0f);
  }
  if (!sure) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(t[i], s);
  }
  return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16),
                    e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}

// A row by its CTA of G warps, as kept by add_rmsnorm_quant_kernel.
struct NormRow {
  const uint16_t *x, *res, *weight;
  uint16_t* h;
  int8_t* q;
  float* scale;
  float eps;
  int K, G, V, first;  // first: the lane's first element of V vectors 256 elements apart
  uint32_t aside;      // those whose h is not stored yet
  float* red_s;
  uint32_t* red_m;
};

// The unrounded h of the lane's vector i, times f, and the same times the gain.
__device__ __forceinline__ void norm_again(const NormRow& a, int i, float f, float (&h)[8], float (&t)[8]) {
  const int e = a.first + i * 256;
  const bool kept = a.h == nullptr || ((a.aside >> i) & 1u);  // x and r are still there
  const uint4 c = *reinterpret_cast<const uint4*>((kept ? a.x : a.h) + e);
  uint4 d = make_uint4(0u, 0u, 0u, 0u), g = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  if (kept && a.res) d = *reinterpret_cast<const uint4*>(a.res + e);
  if (a.weight) g = *reinterpret_cast<const uint4*>(a.weight + e);
  const uint32_t x[4] = {c.x, c.y, c.z, c.w}, r[4] = {d.x, d.y, d.z, d.w}, w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[2 * j] = __fmul_rn(__fadd_rn(bf16_lo(x[j]), bf16_lo(r[j])), f);
    h[2 * j + 1] = __fmul_rn(__fadd_rn(bf16_hi(x[j]), bf16_hi(r[j])), f);
    t[2 * j] = __fmul_rn(h[2 * j], bf16_lo(w[j]));
    t[2 * j + 1] = __fmul_rn(h[2 * j + 1], bf16_hi(w[j]));
  }
}
// Stores the h of the vectors put aside.
__device__ __forceinline__ void norm_store_aside(const NormRow& a) {
  float h[8], t[8];
#pragma unroll 1
  for (int i = 0; i < a.V; ++i)
    if ((a.aside >> i) & 1u) {
      norm_again(a, i, 1.0f, h, t);
      *reinterpret_cast<uint4*>(a.h + a.first + i * 256) =
          make_uint4(pack_bf16x2_rn(h[0], h[1]), pack_bf16x2_rn(h[2], h[3]), pack_bf16x2_rn(h[4], h[5]),
                     pack_bf16x2_rn(h[6], h[7]));
    }
}
// A row whose sum of squares is out of range (the whole CTA calls).
template <int FMT>
__device__ __forceinline__ void norm_far_row(const NormRow& a, bool large) {
  const float f = large ? 0x1p-80f : 0x1p80f;
  float h[8], t[8], ss = 0.0f;
  uint32_t amax = 0;
#pragma unroll 1
  for (int i = 0; i < a.V && a.first + i * 256 < a.K; ++i) {
    norm_again(a, i, f, h, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ss = fmaf(h[j], h[j], ss);
      amax = max(amax, __float_as_uint(fabsf(t[j])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if (a.G > 1) {
    __syncthreads();  // the first sums have been read
    if ((threadIdx.x & 31) == 0) {
      a.red_s[threadIdx.x >> 5] = ss;
      a.red_m[threadIdx.x >> 5] = amax;
    }
    __syncthreads();
    ss = 0.0f;
    amax = 0;
    for (int j = 0; j < a.G; ++j) {
      ss += a.red_s[j];
      amax = max(amax, a.red_m[j]);
    }
  }
  const float s = __fdiv_rn(__uint_as_float(amax), FMT == kQuantE4M3 ? 448.0f : 127.0f);
  if (threadIdx.x == 0) {
    // s / f over sqrt(mean / f^2 + eps); where eps * f^2 overflows the mean is
    // nothing beside eps
    const float mean = __fdiv_rn(ss, static_cast<float>(a.K)), e = __fmul_rn(__fmul_rn(a.eps, f), f);
    const float rstd = e < INFINITY ? __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(mean, e)))
                                    : __fdiv_rn(0x1p-80f, __fsqrt_rn(a.eps));
    *a.scale = s == 0.0f ? 0.0f : __fmul_rn(s, rstd);
  }
  const bool fast = s >= 0x1p-126f;
  const float r = __frcp_rn(s);
#pragma unroll 1
  for (int i = 0; i < a.V && a.first + i * 256 < a.K; ++i) {
    norm_again(a, i, f, h, t);
    uint2 c = make_uint2(0u, 0u);
    if (s != 0.0f) {
      if constexpr (FMT == kQuantE4M3) c = quant_f32x8_e4m3(t, s, r, fast);
      else c = quant_f32x8(t, s, r, fast);
    }
    store_codes8<FMT>(a.q, a.first + i * 256, c);
  }
}

// Registers a thread: what the usual row needs.  The far row's code would take
// more and cost CTAs (16384 x 3072, E4M3: 60 us, and 67 without the limit).
constexpr int norm_registers(int V) { return V <= 4 ? 64 : V == 6 ? 80 : 104; }

// One row per CTA of G warps, V 16-byte vectors a lane in registers.
template <int V, int FMT>
__global__ void __maxnreg__(norm_registers(V)) add_rmsnorm_quant_kernel(
    const uint16_t* x, int K, int64_t ldx, const uint16_t* res, int64_t ldr, const uint16_t* weight,
    float eps, int8_t* q, int64_t ldq, float* scale, uint16_t* h_out, int64_t ldh, int G) {
  __shared__ float red_s[16];
  __shared__ uint32_t red_m[16];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int slice0 = warp * (32 * 8 * V);
  const uint16_t* xr = x + row * ldx;
  const uint16_t* rr = res ? res + row * ldr : nullptr;

  pdl_wait();
  uint4 v[V], u[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = slice0 + (i * 32 + lane) * 8;
    v[i] = u[i] = make_uint4(0u, 0u, 0u, 0u);
    // h_out may be res or x, and the kernel before may have written any of them
    // while this one lived: ordinary loads, of pointers that promise nothing;
    // each thread reads the elements that it writes, before it writes any
    if (e < K) {
      v[i] = *reinterpret_cast<const uint4*>(xr + e);
      if (rr) u[i] = *reinterpret_cast<const uint4*>(rr + e);
    }
  }
  pdl_trigger();

  float t[V][8];
  float ss = 0.0f;
  uint32_t aside = 0;  // the vectors put aside
  uint32_t amax = 0;  // bit patterns of |t| order like the values; a NaN wins
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = slice0 + (i * 32 + lane) * 8;
    const uint32_t a[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    const uint32_t b[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
    uint4 g = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);  // ones
    // (the gains are a model's: no kernel that this one may overlap writes them)
    if (weight && e < K) g = __ldg(reinterpret_cast<const uint4*>(weight + e));
    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
    uint32_t o[4];
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float h0 = __fadd_rn(bf16_lo(a[j]), bf16_lo(b[j]));
      const float h1 = __fadd_rn(bf16_hi(a[j]), bf16_hi(b[j]));
      sq = fmaf(h0, h0, sq);
      sq = fmaf(h1, h1, sq);
      t[i][2 * j] = __fmul_rn(h0, bf16_lo(w[j]));
      t[i][2 * j + 1] = __fmul_rn(h1, bf16_hi(w[j]));
      amax = max(amax, max(__float_as_uint(fabsf(t[i][2 * j])), __float_as_uint(fabsf(t[i][2 * j + 1]))));
      o[j] = pack_bf16x2_rn(h0, h1);
    }
    ss += sq;
    const bool wanted = h_out && e < K, fits = sq >= 0x1p-40f && sq <= 0x1p64f;
    aside |= wanted && !fits ? 1u << i : 0u;
    if (wanted && fits)
      *reinterpret_cast<uint4*>(h_out + row * ldh + e) = make_uint4(o[0], o[1], o[2], o[3]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if (G > 1) {
    if (lane == 0) {
      red_s[warp] = ss;
      red_m[warp] = amax;
    }
    __syncthreads();
    ss = 0.0f;
    amax = 0;
    for (int j = 0; j < G; ++j) {
      ss += red_s[j];
      amax = max(amax, red_m[j]);
    }
  }
  const bool in_range = ss >= 0x1p-60f && ss < INFINITY;  // the same in the whole CTA
  if (__builtin_expect(in_range, 1)) {
    const float s = __fdiv_rn(__uint_as_float(amax), FMT == kQuantE4M3 ? 448.0f : 127.0f);
    if (threadIdx.x == 0) {
      const float mean = __fdiv_rn(ss, static_cast<float>(K));
      const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(mean, eps)));
      scale[row] = amax == 0 ? 0.0f : __fmul_rn(s, rstd);
    }
    int8_t* qr = q + row * ldq * (FMT == kQuantF16 ? 2 : 1);
    const bool fast = s >= 0x1p-126f;
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = slice0 + (i * 32 + lane) * 8;
      if (e < K) {
        uint2 c = make_uint2(0u, 0u);
        if (amax != 0) {
          if constexpr (FMT == kQuantE4M3) c = quant_f32x8_e4m3(t[i], s, r, fast);
          else c = quant_f32x8(t[i], s, r, fast);
        }
        store_codes8<FMT>(qr, e, c);
      }
    }
  }
  if (__builtin_expect(!in_range || aside != 0, 0)) {
    const NormRow far{xr, rr, weight, h_out ? h_out + row * ldh : nullptr, q + row * ldq * (FMT == kQuantF16 ? 2 : 1),
                      scale + row, eps, K, G, V, slice0 + lane * 8, aside, red_s, red_m};
    if (!in_range) norm_far_row<FMT>(far, !(ss < 1.0f));
    norm_store_aside(far);
  }
}

}  // namespace i8
