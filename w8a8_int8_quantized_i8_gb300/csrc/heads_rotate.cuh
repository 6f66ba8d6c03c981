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
  int section_end[kRotateMaxAxes];
  float eps;
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
  int64_t token, head;
  int local, at_a, at_b;  // local: the CTA's token; at_b = dim where there is no second vector
  bool valid;
};

__device__ __forceinline__ RotateItem rotate_load(const RotateArgs& p, int item, int count, int64_t first) {
  RotateItem t;
  const int lane = item & ((1 << p.lanes_log2) - 1), row = item >> p.lanes_log2;
  t.local = row / p.heads;
  const int head = row - t.local * p.heads;
  const int turning = p.rotary >> 4;  // lanes that rotate
  if (lane >= turning || p.interleaved) {
    t.at_a = lane * 16;
    t.at_b = t.at_a + 8;
  } else {
    t.at_a = lane * 8;
    t.at_b = t.at_a + p.rotary / 2;
  }
  t.valid = t.local < count && t.at_a < p.dim;
  t.token = first + t.local;
  t.h = head < p.q_heads ? &p.q : &p.k;
  t.head = head < p.q_heads ? head : head - p.q_heads;
  t.a = t.b = make_uint4(0u, 0u, 0u, 0u);
  if (t.valid) {
    const uint16_t* x = t.h->in + t.token * t.h->in_token + t.head * t.h->in_head;
    t.a = *reinterpret_cast<const uint4*>(x + t.at_a);
    if (t.at_b < p.dim) t.b = *reinterpret_cast<const uint4*>(x + t.at_b);
  }
  return t;
}

__device__ __forceinline__ void rotate_widen(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16_lo(w[j]);
    x[2 * j + 1] = bf16_hi(w[j]);
  }
}

__global__ void __launch_bounds__(kRotateThreads) heads_rmsnorm_rotate_kernel(const __grid_constant__ RotateArgs p) {
  extern __shared__ float2 turn[];  // (cos, sin) [tokens of the CTA][rotary / 2]
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per_cta;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.per_cta), p.tokens - first));
  const int half = p.rotary / 2, items = (count * p.heads) << p.lanes_log2;
  pdl_wait();
  RotateItem t = rotate_load(p, threadIdx.x, count, first);
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
  for (int item = threadIdx.x; item - static_cast<int>(threadIdx.x) < items; item += kRotateThreads) {
    float a[8], b[8];
    rotate_widen(t.a, a);
    rotate_widen(t.b, b);
    const RotateItem now = t;
    if (item - static_cast<int>(threadIdx.x) + kRotateThreads < items) t = rotate_load(p, item + kRotateThreads, count, first);
    if (p.q.weight || p.k.weight) {  // (whole warps: rows of q and k share them)
      float ss[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] = fmaf(a[j], a[j], fmaf(b[j], b[j], ss[0]));
      for (int d = 1 << p.lanes_log2 >> 1; d > 0; d >>= 1) ss[0] += __shfl_xor_sync(0xFFFFFFFFu, ss[0], d);
      if (__any_sync(0xFFFFFFFFu, now.valid && !(ss[0] >= 0x1p-60f && ss[0] < INFINITY))) {
        // squares out of fp32's range in some row: the sums of others as well
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float s0 = a[j] * 0x1p-80f, s1 = b[j] * 0x1p-80f, l0 = a[j] * 0x1p80f, l1 = b[j] * 0x1p80f;
          ss[1] = fmaf(s0, s0, fmaf(s1, s1, ss[1]));
          ss[2] = fmaf(l0, l0, fmaf(l1, l1, ss[2]));
        }
        for (int d = 1 << p.lanes_log2 >> 1; d > 0; d >>= 1) {
          ss[1] += __shfl_xor_sync(0xFFFFFFFFu, ss[1], d);
          ss[2] += __shfl_xor_sync(0xFFFFFFFFu, ss[2], d);
        }
      }
      if (now.valid && now.h->weight) {
        const float r = fp4_rstd(ss, p.dim, p.eps);
        float w[8];
        rotate_widen(*reinterpret_cast<const uint4*>(now.h->weight + now.at_a), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = a[j] * r * w[j];
        if (now.at_b < p.dim) {
          rotate_widen(*reinterpret_cast<const uint4*>(now.h->weight + now.at_b), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] = b[j] * r * w[j];
        }
      }
    }
    if (!now.valid) continue;
    const int lane = item & ((1 << p.lanes_log2) - 1);
    if (lane < (p.rotary >> 4)) {
      const float2* cs = turn + now.local * half + lane * 8;
      if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = cs[j], v = cs[j + 4];
          const float a0 = a[2 * j], b0 = b[2 * j];
          a[2 * j] = a0 * u.x - a[2 * j + 1] * u.y;
          a[2 * j + 1] = a[2 * j + 1] * u.x + a0 * u.y;
          b[2 * j] = b0 * v.x - b[2 * j + 1] * v.y;
          b[2 * j + 1] = b[2 * j + 1] * v.x + b0 * v.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 u = cs[j];
          const float a0 = a[j];
          a[j] = a0 * u.x - b[j] * u.y;
          b[j] = b[j] * u.x + a0 * u.y;
        }
      }
    }
    uint16_t* y = now.h->out + now.token * now.h->out_token + now.head * now.h->out_head;
    *reinterpret_cast<uint4*>(y + now.at_a) = make_uint4(pack_bf16x2_rn(a[0], a[1]), pack_bf16x2_rn(a[2], a[3]),
                                                         pack_bf16x2_rn(a[4], a[5]), pack_bf16x2_rn(a[6], a[7]));
    if (now.at_b < p.dim)
      *reinterpret_cast<uint4*>(y + now.at_b) = make_uint4(pack_bf16x2_rn(b[0], b[1]), pack_bf16x2_rn(b[2], b[3]),
                                                           pack_bf16x2_rn(b[4], b[5]), pack_bf16x2_rn(b[6], b[7]));
  }
}

}  // namespace i8
