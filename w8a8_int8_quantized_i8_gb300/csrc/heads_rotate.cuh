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
// 2 bytes read and 2 written an element.  A lane holds 8 pairs, that is two vectors
// of 16 bytes, in either pairing; a row is up to 32 lanes.  What bounds it is how
// many instructions an element takes, so the gains go into the sines and cosines:
// a CTA makes the four products
//   y_a = x_a (w_a cos) + x_b (-w_b sin),  y_b = x_a (w_a sin) + x_b (w_b cos)
// of its tokens once, in shared memory, for all their heads, while the first rows
// are on their way; x is multiplied by the norm's factor before.  16384 tokens of 40 heads of
// 128: 61 us, 5.5 TB/s; 64 tokens 3.4 us, a launch.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "fp4_quant.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

constexpr int kRotateMaxAxes = 4, kRotateThreads = 256;
constexpr int kRotateTable = 32 * 1024;  // bytes of products a CTA makes, at most, where it takes several tokens

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
  int kinds;                   // tables a token: 2 where q and k have gains of their own
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

__device__ __forceinline__ unsigned long long f2_fma(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// A lane's 16 elements as the firsts and the seconds of 8 pairs, and back.
__device__ __forceinline__ void rotate_widen(const uint4& v, const uint4& u, bool interleaved, float (&a)[8], float (&b)[8]) {
  const uint32_t w[8] = {v.x, v.y, v.z, v.w, u.x, u.y, u.z, u.w};
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = bf16_lo(w[j]), b[j] = bf16_hi(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[2 * j] = bf16_lo(w[j]), a[2 * j + 1] = bf16_hi(w[j]);
      b[2 * j] = bf16_lo(w[j + 4]), b[2 * j + 1] = bf16_hi(w[j + 4]);
    }
  }
}
__device__ __forceinline__ void rotate_narrow(const float (&a)[8], const float (&b)[8], bool interleaved, uint4& v, uint4& u) {
  uint32_t w[8];
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2_rn(a[j], b[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = pack_bf16x2_rn(a[2 * j], a[2 * j + 1]);
      w[j + 4] = pack_bf16x2_rn(b[2 * j], b[2 * j + 1]);
    }
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
  u = make_uint4(w[4], w[5], w[6], w[7]);
}

// The norm's factor of the rows whose squares leave fp32's range (the whole warp
// calls).  Their elements are left times 2^80 or 2^-80, which is exact, so that
// neither their squares nor the factor leave the range.  What it returns for the
// warp's other rows, which stay as they are, is not used: a row's bits are its own.
__device__ __forceinline__ float rotate_far_rstd(const RotateArgs& p, float sum, float (&a)[8], float (&b)[8]) {
  const float n = static_cast<float>(p.dim);
  const bool small = sum < 0x1p-60f;
  // where eps * 2^160 overflows, squares below 2^-60 are nothing beside eps
  const float up = fp4_in_range(sum) ? 1.0f : small ? 0x1p80f : 0x1p-80f, e = __fmul_rn(__fmul_rn(p.eps, up), up);
  const float f = e < INFINITY ? up : 1.0f;
  float ss = 0.0f;
  for (int j = 0; j < 8; ++j) {
    a[j] *= f;
    b[j] *= f;
    ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
  }
  for (int d = 1 << p.lanes_log2 >> 1; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
  return __fdiv_rn(1.0f, __fsqrt_rn(e < INFINITY ? __fadd_rn(__fdiv_rn(ss, n), e) : p.eps));
}

__global__ void __launch_bounds__(kRotateThreads, 4) heads_rmsnorm_rotate_kernel(const __grid_constant__ RotateArgs p) {
  // [tokens of the CTA][kinds][w_a cos, w_a sin, -w_b sin, w_b cos][pairs 0-3 or 4-7 of
  // a lane][lanes][4]: a row's lanes read side by side.  Lanes behind the rotated part
  // have their gains there
  extern __shared__ __align__(16) float turn[];
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
  const int group = (p.dim + 15) >> 4, pairs = group * 8;
  for (int i = threadIdx.x; i < count * pairs; i += kRotateThreads) {
    const int local = i / pairs, pair = i - local * pairs;
    float s = 0.0f, c = 1.0f;
    // the elements of the pair
    int one = 2 * pair, two = one + 1;
    if (!p.interleaved) {
      one = pair < half ? pair : (pair >> 3) * 16 + (pair & 7);
      two = pair < half ? pair + half : one + 8;
    }
    if (pair < half) {
      int axis = 0;
#pragma unroll
      for (int a = 0; a < kRotateMaxAxes - 1; ++a) axis += pair >= p.section_end[a] ? 1 : 0;
      sincospif(2.0f * rotate_turns(p.positions[axis * p.ld_pos + first + local], p.inv_freq[pair]), &s, &c);
    }
    for (int kind = 0; kind < p.kinds; ++kind) {
      const uint16_t* w = kind == 0 ? p.q.weight : p.k.weight;
      const float wa = w && one < p.dim ? __uint_as_float(static_cast<uint32_t>(w[one]) << 16) : 1.0f;
      const float wb = w && two < p.dim ? __uint_as_float(static_cast<uint32_t>(w[two]) << 16) : 1.0f;
      float* at = turn + (local * p.kinds + kind) * 4 * pairs + ((((pair >> 2) & 1) * group + (pair >> 3)) << 2) + (pair & 3);
      at[0] = wa * c;
      at[pairs] = wa * s;
      at[2 * pairs] = -wb * s;
      at[3 * pairs] = wb * c;
    }
  }
  pdl_trigger();
  __syncthreads();
  const bool norms = p.q.weight || p.k.weight;
  for (int base = 0; base < rows; base += stride, row += stride) {  // the same rounds for whole warps
    float a[8], b[8];
    rotate_widen(t.a, t.b, p.interleaved, a, b);
    const bool valid = inside && row < rows;
    const RotateHeads* const h = t.h;
    const int local = t.local, head = t.head;
    t.local += p.step_tokens;
    t.head += p.step_heads;
    if (t.head >= p.heads) t.head -= p.heads, ++t.local;
    rotate_load(p, t, inside && row + stride < rows, first, at_a, at_b);
    float r = 1.0f;
    if (norms) {  // (whole warps: rows of q and k share them)
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
      for (int d = 1 << p.lanes_log2 >> 1; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
      r = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
      const bool far = h->weight && !fp4_in_range(ss);  // (a row without a norm stays as it is)
      if (__any_sync(0xFFFFFFFFu, valid && far)) {
        const float f = rotate_far_rstd(p, far ? ss : 1.0f, a, b);
        if (far) r = f;
      }
      if (!h->weight) r = 1.0f;
    }
    const bool key = head >= p.q_heads;
    // (lanes without a row's elements stay with the warp, at the first products)
    const float4* m = reinterpret_cast<const float4*>(turn);
    if (valid) m += (local * p.kinds + (key ? p.kinds - 1 : 0)) * 8 * group + lane;
    const unsigned long long rr = f2(r, r);
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // four pairs
      const float4 ca = m[j * group], sa = m[(2 + j) * group], sb = m[(4 + j) * group], cb = m[(6 + j) * group];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = 4 * j + 2 * e;
        // (the norm's factor first: an element times its gain may leave fp32's range)
        const unsigned long long x = f2_mul(f2(a[k], a[k + 1]), rr), z = f2_mul(f2(b[k], b[k + 1]), rr);
        unsigned long long u, v;
        if (turns) {
          u = f2_fma(x, e ? f2(ca.z, ca.w) : f2(ca.x, ca.y), f2_mul(z, e ? f2(sb.z, sb.w) : f2(sb.x, sb.y)));
          v = f2_fma(x, e ? f2(sa.z, sa.w) : f2(sa.x, sa.y), f2_mul(z, e ? f2(cb.z, cb.w) : f2(cb.x, cb.y)));
        } else {  // (0 times what is not finite is not 0)
          u = f2_mul(x, e ? f2(ca.z, ca.w) : f2(ca.x, ca.y));
          v = f2_mul(z, e ? f2(cb.z, cb.w) : f2(cb.x, cb.y));
        }
        f2_split(u, a[k], a[k + 1]);
        f2_split(v, b[k], b[k + 1]);
      }
    }
    if (!valid) continue;
    uint4 v, u;
    rotate_narrow(a, b, p.interleaved, v, u);
    uint16_t* y = h->out + (first + local) * h->out_token + (key ? head - p.q_heads : head) * h->out_head;
    *reinterpret_cast<uint4*>(y + at_a) = v;
    if (at_b < p.dim) *reinterpret_cast<uint4*>(y + at_b) = u;
  }
}

}  // namespace i8
