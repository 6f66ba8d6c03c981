// heads_rotate.cuh -- the root-mean-square norm of each query and key head with a
// gain, and the rotation of its pairs by the token's position, in one pass.
//
// For a head x of D elements, of which the first R are rotated:
//   y = x * w / sqrt(mean(x^2) + eps)                  (x alone without a gain)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
// for the pairs i = 0 .. R/2 - 1, (a, b) = (i, i + R/2) or, interleaved,
// (2i, 2i + 1), by the angle position * inv_freq[i].  With several axes the pairs
// are shared out among them, each with its own positions.  fp32 inside, one
// rounding to bf16.
//
// The angle: a far position times a frequency has more digits than fp32, and only
// its fraction of a turn counts.  inv_freq / 2 pi is held as the sum of two fp32
// numbers, the position is taken as two parts that are exact in fp32, and
// each product as its rounded value (whose whole turns are dropped, exactly) and
// its rounding error (one fma).  Up to 2^20 the error is below 2^-24 turns.
//
// Bound by HBM: 2 bytes read and 2 written an element.  A lane holds 8 pairs, that
// is two vectors of 16 bytes, in either pairing; a row is up to 32 lanes.  The
// sines and cosines of a CTA's tokens are made once, in shared memory, for all
// their heads, while the first rows are on their way.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "fp4_quant.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

constexpr int kRotateMaxAxes = 4, kRotateThreads = 256;

struct RotateHeads {
  const uint16_t* in;
  uint16_t* out;
  const uint16_t* weight;  // null: no norm
  int64_t in_token, in_head, out_token, out_head;
};

struct RotateArgs {
  RotateHeads q, k;
  const int32_t* positions;  // [axes, tokens]
  int64_t ld_pos;
  const float* inv_freq;
  int tokens, q_heads, heads;  // heads: of q and k
  int dim, rotary, interleaved;
  int per_cta;                 // tokens
  int lanes_log2;              // lanes of a row
  int step_tokens, step_heads; // from a thread's row to its next
  int section_end[kRotateMaxAxes];
  float eps, inv_dim;
};

// position * f in turns, without whole ones.
__device__ __forceinline__ float rotate_turns(int32_t position, float f) {
  constexpr float kInvHi = 0.15915494f, kInvLo = 6.4206382e-09f;  // 1 / (2 pi)
  const float hi = __fmul_rn(f, kInvHi);
  const float lo = __fmaf_rn(f, kInvLo, __fmaf_rn(f, kInvHi, -hi));
  const float far = static_cast<float>((position >> 12) * 4096.0f), near = static_cast<float>(position & 4095);
  const float a = __fmul_rn(far, hi), b = __fmul_rn(near, hi);
  const float rest = __fmaf_rn(far, lo, __fmaf_rn(far, hi, -a)) + __fmaf_rn(near, lo, __fmaf_rn(near, hi, -b));
  const float t = (a - rintf(a)) + (b - rintf(b));
  const float s = t + rest;
  // (what the last sum rounded away; t and rest are both small)
  return (s - rintf(s)) + (t - s + rest);
}

// A row's two vectors of this lane and where they lie.
struct RotateItem {
  uint4 a, b;
  const RotateHeads* h;
  int local, head;  // the CTA's token, the head among those of q and k
};

__device__ __forceinline__ void rotate_load(const RotateArgs& p, RotateItem& t, bool valid, int64_t first, int at_a, int at_b) {
  t.h = t.head < p.q_heads ? &p.q : &p.k;
  t.a = t.b = make_uint4(0u, 0u, 0u, 0u);
  if (valid) {
    const uint16_t* x = t.h->in + (first + t.local) * t.h->in_token + (t.head < p.q_heads ? t.head : t.head - p.q_heads) * t.h->in_head;
    t.a = *reinterpret_cast<const uint4*>(x + at_a);
    if (at_b < p.dim) t.b = *reinterpret_cast<const uint4*>(x + at_b);
  }
}

__device__ __forceinline__ void rotate_widen(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16_lo(w[j]);
    x[2 * j + 1] = bf16_hi(w[j]);
  }
}

// The norm's factor where some row of the warp has squares out of fp32's range: from
// the sums of others as well (the whole warp calls).
__device__ __forceinline__ float rotate_far_rstd(const RotateArgs& p, const float (&a)[8], const float (&b)[8], float sum) {
  float ss[3] = {sum, 0.0f, 0.0f};
  for (int j = 0; j < 8; ++j) {
    const float s0 = a[j] * 0x1p-80f, s1 = b[j] * 0x1p-80f, l0 = a[j] * 0x1p80f, l1 = b[j] * 0x1p80f;
    ss[1] = fmaf(s0, s0, fmaf(s1, s1, ss[1]));
    ss[2] = fmaf(l0, l0, fmaf(l1, l1, ss[2]));
  }
  for (int d = 1 << p.lanes_log2 >> 1; d > 0; d >>= 1) {
    ss[1] += __shfl_xor_sync(0xFFFFFFFFu, ss[1], d);
    ss[2] += __shfl_xor_sync(0xFFFFFFFFu, ss[2], d);
  }
  return fp4_rstd(ss, p.dim, p.eps);
}

__global__ void __launch_bounds__(kRotateThreads, 5) heads_rmsnorm_rotate_kernel(const __grid_constant__ RotateArgs p) {
  extern __shared__ __align__(16) float2 turn[];  // (cos, sin) [tokens of the CTA][rotary / 2]
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per_cta;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.per_cta), p.tokens - first));
  const int half = p.rotary / 2, rows = count * p.heads;
  const int lane = threadIdx.x & ((1 << p.lanes_log2) - 1), stride = kRotateThreads >> p.lanes_log2;
  // this lane's elements of every row it works on: pairs 8 lane .. 8 lane + 7, or,
  // behind the rotated part, two vectors that lie side by side
  const bool turns = lane < (p.rotary >> 4);
  const bool split = turns && !p.interleaved;
  const int at_a = split ? lane * 8 : lane * 16, at_b = split ? at_a + half : at_a + 8;
  const bool inside = at_a < p.dim;

  pdl_wait();
  int row = threadIdx.x >> p.lanes_log2;
  RotateItem t;
  t.local = row / p.heads;
  t.head = row - t.local * p.heads;
  rotate_load(p, t, inside && row < rows, first, at_a, at_b);
  for (int i = threadIdx.x; i < count * half; i += kRotateThreads) {
    const int local = i / half, pair = i - local * half;
    int axis = 0;
#pragma unroll
    for (int a = 0; a < kRotateMaxAxes - 1; ++a) axis += pair >= p.section_end[a] ? 1 : 0;
    float s, c;
    sincospif(2.0f * rotate_turns(p.positions[axis * p.ld_pos + first + local], p.inv_freq[pair]), &s, &c);
    turn[i] = make_float2(c, s);
  }
  pdl_trigger();
  __syncthreads();
  for (int base = 0; base < rows; base += stride, row += stride) {  // the same rounds for whole warps
    float a[8], b[8];
    rotate_widen(t.a, a);
    rotate_widen(t.b, b);
    const bool valid = inside && row < rows;
    const RotateHeads* const h = t.h;
    const int local = t.local, head = t.head;
    t.local += p.step_tokens;
    t.head += p.step_heads;
    if (t.head >= p.heads) t.head -= p.heads, ++t.local;
    rotate_load(p, t, inside && row + stride < rows, first, at_a, at_b);
    if (p.q.weight || p.k.weight) {  // (whole warps: rows of q and k share them)
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
      for (int d = 1 << p.lanes_log2 >> 1; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
      float r = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
      if (__any_sync(0xFFFFFFFFu, valid && !(ss >= 0x1p-60f && ss < INFINITY))) r = rotate_far_rstd(p, a, b, ss);
      if (valid && h->weight) {
        float w[8];
        rotate_widen(*reinterpret_cast<const uint4*>(h->weight + at_a), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = a[j] * r * w[j];
        if (at_b < p.dim) {
          rotate_widen(*reinterpret_cast<const uint4*>(h->weight + at_b), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] = b[j] * r * w[j];
        }
      }
    }
    if (!valid) continue;
    if (turns) {
      const float4* cs = reinterpret_cast<const float4*>(turn + local * half + lane * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 u = cs[j];  // pairs 2 j and 2 j + 1 of the lane's eight
        if (p.interleaved) {
          float (&z)[8] = j < 2 ? a : b;
          const int k = 4 * (j & 1);
          const float z0 = z[k], z2 = z[k + 2];
          z[k] = z0 * u.x - z[k + 1] * u.y;
          z[k + 1] = z[k + 1] * u.x + z0 * u.y;
          z[k + 2] = z2 * u.z - z[k + 3] * u.w;
          z[k + 3] = z[k + 3] * u.z + z2 * u.w;
        } else {
          const float a0 = a[2 * j], a1 = a[2 * j + 1];
          a[2 * j] = a0 * u.x - b[2 * j] * u.y;
          b[2 * j] = b[2 * j] * u.x + a0 * u.y;
          a[2 * j + 1] = a1 * u.z - b[2 * j + 1] * u.w;
          b[2 * j + 1] = b[2 * j + 1] * u.z + a1 * u.w;
        }
      }
    }
    uint16_t* y = h->out + (first + local) * h->out_token + (head < p.q_heads ? head : head - p.q_heads) * h->out_head;
    *reinterpret_cast<uint4*>(y + at_a) = make_uint4(pack_bf16x2_rn(a[0], a[1]), pack_bf16x2_rn(a[2], a[3]),
                                                     pack_bf16x2_rn(a[4], a[5]), pack_bf16x2_rn(a[6], a[7]));
    if (at_b < p.dim)
      *reinterpret_cast<uint4*>(y + at_b) = make_uint4(pack_bf16x2_rn(b[0], b[1]), pack_bf16x2_rn(b[2], b[3]),
                                                       pack_bf16x2_rn(b[4], b[5]), pack_bf16x2_rn(b[6], b[7]));
  }
}

}  // namespace i8
