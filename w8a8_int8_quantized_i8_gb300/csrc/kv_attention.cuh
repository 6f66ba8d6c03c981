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
//   * the codes are exact in fp16 (int8: |c| <= 127; E4M3: 4 significant bits,
//     2^-9 to 448).  A row of q, bf16, is multiplied by the power of two that
//     brings its largest element into [2^14, 2^15): exact in fp16 except for
//     elements below 2^-28 of the largest, which keep an absolute error of
//     2^-40 of it.  So q . ck is a sum of exact products in fp32;
//   * softmax statistics and sums are fp32;
//   * P is rounded to fp16 (11 bits) for the second product, as 2^(10 + s - R)
//     with s = log2(e) S + log2 sv, the log of a term's weight in O, and R its
//     running maximum in the row: at most 2^10, and what lies 2^-35 below the
//     maximum vanishes;
//   * the sum of exponentials counts every token, however small its block's
//     values are next to others'.  While log2 sv stays within 40 of that of
//     the first block, Lr, it adds P / sv, as 2^(10 + log2(e) S + Lr - R).  From
//     the first block on that is further off, or all zeros, it has a maximum X
//     of its own, that of log2(e) S alone, and adds 2^(log2(e) S - X) instead.
//     Either is l * 2^X, with X = R - 10 - Lr in the first form, and where parts
//     meet it is its logarithm L = X + log2 l: O * 2^(R - 10 - L) is the result.
//   * a row depends on the tokens that it sees and on nothing else.  NaN in its q,
//     in a scale or in a key makes it NaN, a NaN code of a value its head
//     dimension; infinite scales count as NaN.  Tokens that it does not see are
//     left out by their place, whatever they hold.
//
// Blocks, scales and q are read by ordinary loads: the kernels that write them
// may still run when this one begins (it waits for them, but lives meanwhile).
//
// The products run transposed: S^T = K q^T and O^T = V^T P^T, so that the
// tokens and the head dimension fill the 16-row side of the warp MMA
// (m16n8k16) and the few query rows its 8-wide side.  The order of the head
// dimension inside a product and of the output's rows is free, so lane (g, c)
// = (lane / 4, lane % 4) takes 16 contiguous codes of token g of K, and of
// tokens 2c, 2c + 1 of V.
//
// Every warp has a ring of its own in shared memory, which its first lane
// fills by TMA (16 or 32 tokens of a block are one contiguous piece of the
// cache) and which needs no barrier between warps.  The 128-byte swizzle makes
// the lanes' 16-byte reads free of bank conflicts: rows 2c, 2c + 1 at chunk g
// for V, rows g at chunks 2c + j for K.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"
#include "quant.cuh"

namespace i8 {

// Bound by HBM: 64 requests up to 8192 tokens, 32 query and 8 kv heads of 128,
// int8: 96.7 us, 5.0 TB/s (75 % of the measured copy rate); 64 of 4096 each: 90.0
// us (89 %); one request of 131071 tokens, E4M3: 53.6 us (75 %).  About 8 us of
// each are the start and the join.  Two stages and three CTAs an SM beat three
// and two (95 against 108 us), TMA the lanes' own cp.async (95 against 122).
// The two forms of the sum cost 4 % against one that goes by V alone (92 us).
//
// How the work is split.  An item is a request's row tile (8 * NT rows) of one
// kv head; its tokens come in units of 4 warps' tiles.  The units of all items,
// request after request, are one line that the resident CTAs cut into equal
// shares, so ragged lengths balance and one long context fills the GPU.  Nobody but the
// device knows the lengths: every CTA adds up the requests' units by itself
// (two loads a request).  A CTA that covers an item whole writes its rows; the
// pieces of an item that is cut go to the workspace (two slots a CTA: an item
// begun before its share, an item that goes on after it), and a second, small
// kernel joins them in the order of the tokens, so results do not depend on
// timing.
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
static_assert(kAttnThreads == 128, "the epilogues' ownership of rows is written for 128 threads");

// Tokens a warp takes at a time, in halves of 16, and its ring's stages.
template <int D>
struct AttnTile {
  static constexpr int HALVES = D == 256 ? 1 : 2;
  static constexpr int TOKENS = 16 * HALVES;
  static constexpr int UNIT = TOKENS * kAttnWarps;
  static constexpr int STAGES = 2;
  static constexpr int SIDE = TOKENS * D;      // bytes of K, or of V, in a stage
  static constexpr int STAGE = 2 * SIDE;
  static constexpr int BOX = D < 128 ? D : 128;  // bytes of a row in one TMA box
};
constexpr unsigned long long kDrainLimitNs = 1000000000ull;  // of a wait on the way out
constexpr int kAttnMeet = 4;    // m-tiles of O^T a warp's parts meet by at a time
constexpr int kJoinGroups = 4;  // groups of kAttnThreads that share an item's pieces in the join

struct AttnArgs {
  const uint16_t* q;          // [tokens, q_heads, D] bf16
  int64_t ldq_token, ldq_head;
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
  int32_t unit_cols, unit_rest;  // unit / block, unit % block
  int32_t box_rows;           // tokens of a TMA box
  int32_t split_rows;         // requests of this many rows a kv head are kv_prefill.cuh's
  float* pieces;              // workspace: [2 * workers][8 * NT * (D + 2)]
  int4* cut;                  // [2 * workers]: the item begun, but not ended, by a worker
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A running maximum as a reference for exponents: where nothing has been seen
// it is -inf, and any finite number will do (2^(-inf - 0) = 0).
__device__ __forceinline__ float exp_ref(float m) { return m > -INFINITY ? m : 0.0f; }

// Four codes of a word as two fp16 pairs, (0, 1) and (2, 3).
template <bool E4M3>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    s8x4_to_f16x4(w, lo, hi);
  }
}

// The bytes of a word that are E4M3's NaN codes, as a mask.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}
// An infinite scale as NaN (an infinity less an infinity).
__device__ __forceinline__ float scale_value(float s) { return s + (s - s); }

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
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
  float m[NT][2];          // running maximum R of those columns
  float l[NT][2];          // this lane's share of the sum of 2^(log2(e) S - X)
  float x[NT][2];          // X: the second form's maximum of this lane's scores
  float ref;               // Lr
};

// A warp's feed: where its copies of a segment of keys stand.
template <int D>
struct AttnFeed {
  using Tile = AttnTile<D>;
  static constexpr int H = Tile::HALVES;
  static constexpr int S = Tile::STAGES;
  const int32_t* table;     // the request's blocks
  int head;
  int t_first, end;         // the warp's first token of the segment, the segment's end
  int t_look, col, off;     // the next tile to look up: token, column of the table, offset in the block
  int next_id[H], next_off[H];  // looked up, not yet copied
  float ksc[S][H], vsc[S][H];   // block scales of the tiles in the ring
  uint32_t have[S];             // a bit for each half whose block exists
};

// Adds the calls' values up over the CTA: returns the exclusive sum before
// this thread, and the total.
__device__ __forceinline__ int64_t attn_scan(int64_t v, int64_t& total, int64_t* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  total = 0;
  int64_t before = 0;
#pragma unroll
  for (int w = 0; w < kAttnWarps; ++w) {
    if (w < warp) before += sm[w];
    total += sm[w];
  }
  return before + x - v;
}

// What a CTA needs to know of a request.
struct AttnRequest {
  int q0, fresh;
  int pos0;        // position of its first new token
  int len;         // its tokens that the table has room for
  int tiles;       // row tiles
  int per_item;    // units of an item
  int64_t units;
};

template <int ROWS, int UNIT>
__device__ __forceinline__ AttnRequest attn_request(const AttnArgs& p, int r) {
  AttnRequest a;
  a.q0 = p.cu_new[r];
  const int64_t fresh = static_cast<int64_t>(p.cu_new[r + 1]) - a.q0;
  const int len = max(0, p.seq_lens[r]);
  const bool bad = a.q0 < 0 || fresh < 0 || a.q0 + fresh > p.tokens || fresh > p.max_new;
  a.fresh = bad ? 0 : static_cast<int>(fresh);
  // the tokens past the table are absent; the others, and the rows, stay where
  // they are
  a.pos0 = len - a.fresh;
  a.len = min(len, p.width * p.block);
  if (bad || a.len < len) atomicOr(&g_status, 1u << 7);
  a.tiles = static_cast<int>((static_cast<int64_t>(a.fresh) * (p.q_heads / p.kv_heads) + ROWS - 1) / ROWS);
  a.per_item = max(1, (a.len + UNIT - 1) / UNIT);  // one even where there is nothing to see
  a.units = static_cast<int64_t>(a.per_item) * a.tiles * p.kv_heads;
  if (static_cast<int64_t>(a.fresh) * (p.q_heads / p.kv_heads) >= p.split_rows) a.units = 0;
  return a;
}

// log2 of a sum l * 2^x; -inf where nothing was seen.
__device__ __forceinline__ float attn_log(float x, float l) {
  return l == 0.0f ? -INFINITY : x + __log2f(l);
}
// What O is multiplied by, twice, for the result: its exponent's range is more
// than fp32's.  A row that sees nothing gives 0.
__device__ __forceinline__ float attn_factor(float o_ref, float L) {
  return L == -INFINITY ? 0.0f : ex2(0.5f * (o_ref - L));
}

// D / 16 contiguous head dimensions of one row, times f * f, to bf16.
template <int D>
__device__ __forceinline__ void attn_store_row(uint16_t* out, const float (&o)[D / 16], float f) {
  uint32_t w[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * i] * f * f, o[2 * i + 1] * f * f);
    w[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  if constexpr (D == 64) {
    *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < D / 32; i += 4)
      *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// In the epilogues thread t of kAttnThreads owns, of each column tile n, row
// 8n + 2c + ((t >> 5) & 1) and the head dimensions of m-tiles (t >> 6) * D / 32
// on (D / 16 of them, contiguous), with (g, c) those of its lane.
template <int D>
__device__ __forceinline__ int attn_own_dim(int t) {
  constexpr int VB = D / 8 < 16 ? D / 8 : 16;
  const int byte = (t >> 6) * (D / 16);
  return (byte / VB) * 128 + ((t & 31) >> 2) * VB + byte % VB;
}
__device__ __forceinline__ int attn_own_row(int t) { return 2 * (t & 3) + ((t >> 5) & 1); }

template <int D>
__device__ __forceinline__ void attn_write(const AttnArgs& p, int q0, int r, int head, int t,
                                           const float (&o)[D / 16], float m, float L) {
  const int group = p.q_heads / p.kv_heads;
  const int i = r / group, hq = head * group + r - i * group;
  const int d = attn_own_dim<D>(t);
  const int64_t token = static_cast<int64_t>(q0) + i;
  attn_store_row<D>(p.out + token * p.ldo_token + hq * p.ldo_head + d, o,
                    attn_factor(exp_ref(m) - 10.0f, L));
  if (p.lse && d == 0) p.lse[token * p.q_heads + hq] = L * 0.69314718055994531f;
}

__device__ __forceinline__ uint4 lds_16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds_8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Where a place in a token's row lies in a half (16 tokens) of a stage's K or
// V: boxes of 16 rows, each row's 16-byte chunks xor-ed with the row number
// (128-byte rows: by row & 7, 64-byte rows: by row / 2 & 3).
template <int D>
__device__ __forceinline__ uint32_t attn_place(int row, int byte) {
  if constexpr (D == 64) return row * 64 + (byte ^ (((row >> 1) & 3) << 4));
  return (byte >> 7) * (AttnTile<D>::TOKENS * 128) + row * 128 + ((byte & 127) ^ ((row & 7) << 4));
}

// First head dimension of K chunk j of lane column c (16 codes).
template <int D>
__host__ __device__ constexpr int attn_k_dim(int j, int c) {
  return D == 64 ? c * 16 : (j >> 1) * 128 + (2 * c + (j & 1)) * 16;
}

template <int D>
__device__ __forceinline__ void feed_look_up(const AttnArgs& p, AttnFeed<D>& f) {
  using Tile = AttnTile<D>;
#pragma unroll
  for (int h = 0; h < Tile::HALVES; ++h) {
    const bool wraps = f.off + 16 * h >= p.block;
    f.next_off[h] = wraps ? f.off + 16 * h - p.block : f.off + 16 * h;
    f.next_id[h] = f.t_look + 16 * h < f.end ? f.table[wraps ? f.col + 1 : f.col] : -1;
  }
  f.t_look += Tile::UNIT;
  f.col += p.unit_cols;
  f.off += p.unit_rest;
  if (f.off >= p.block) {
    f.off -= p.block;
    ++f.col;
  }
}

// Starts the copies of the tile at t0, whose blocks have been looked up, into
// stage `slot`; its scales go to place `into` of the feed.
template <int D>
__device__ __forceinline__ void feed_issue(const AttnArgs& p, AttnFeed<D>& f, const void* k_map,
                                           const void* v_map, uint32_t ring, uint32_t bars,
                                           int lane, int t0, int slot, int into) {
  using Tile = AttnTile<D>;
  constexpr int H = Tile::HALVES;
  if (t0 >= f.end) return;
  const uint32_t k_to = ring + slot * Tile::STAGE, v_to = k_to + Tile::SIDE;
  const uint32_t bar = bars + 8 * slot;
  uint32_t bytes = 0;
  bool there[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    there[h] = f.next_id[h] >= 0 && f.next_id[h] < p.blocks;
    // end lies within the table's width
    if (!there[h] && t0 + 16 * h < f.end && lane == 0) atomicOr(&g_status, 1u << 7);
    bytes += there[h] ? 32u * D : 0u;
  }
  // a box of 32 tokens where blocks are a multiple of that: the halves' ids agree
  const bool whole = H == 2 && p.box_rows == 32;
  if (whole) bytes = there[0] ? 64u * D : 0u;
  if (lane == 0) {
    mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (there[h] && !(whole && h == 1)) {
        const int row = f.next_id[h] * p.kv_heads + f.head;
#pragma unroll
        for (int b = 0; b < D / Tile::BOX; ++b) {
          const uint32_t at = b * (Tile::TOKENS * 128) + h * 16 * Tile::BOX;
          tma_load_3d(k_to + at, k_map, bar, b * Tile::BOX, f.next_off[h], row);
          tma_load_3d(v_to + at, v_map, bar, b * Tile::BOX, f.next_off[h], row);
        }
      }
  }
  f.have[into] = 0;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t row = static_cast<int64_t>(f.next_id[h]) * p.kv_heads + f.head;
    f.ksc[into][h] = there[h] ? p.k_scale[row] : 0.0f;
    f.vsc[into][h] = there[h] ? p.v_scale[row] : 0.0f;
    f.have[into] |= there[h] ? 1u << h : 0u;
  }
}

// Begins a segment, tokens [begin, end) of one kv head: the warp takes every
// kAttnWarps-th tile; its ring is filled but for the stage that the first
// round of attend_tiles fills.
template <int D>
__device__ __forceinline__ void feed_begin(const AttnArgs& p, AttnFeed<D>& f, const void* k_map,
                                           const void* v_map, const int32_t* table, int head,
                                           int begin, int end, uint32_t ring, uint32_t bars,
                                           int warp, int lane) {
  using Tile = AttnTile<D>;
  f.table = table;
  f.head = head;
  f.t_first = f.t_look = begin + warp * Tile::TOKENS;
  f.end = end;
  if (f.t_first >= end) return;
  f.col = f.t_first / p.block;
  f.off = f.t_first - f.col * p.block;
  feed_look_up(p, f);
#pragma unroll
  for (int i = 0; i < Tile::STAGES - 1; ++i) {
    feed_issue(p, f, k_map, v_map, ring, bars, lane, f.t_first + i * Tile::UNIT, i, i);
    feed_look_up(p, f);
  }
}

// A row tile of a request's rows against the segment that the feed has begun,
// from its tile at t0 on, which is in stage `slot`, to the end, or, without
// FAR, to the first tile whose values are far from the first one's.
// `ring` and `bars`: the shared-memory addresses of the warp's stages and of
// the barriers on which their copies count; `parity`: a bit for each stage.
template <int D, bool E4M3, int NT, bool FAR>
__device__ __forceinline__ void attend_tiles(const AttnArgs& p, AttnFeed<D>& f, const void* k_map,
                                             const void* v_map,
                                             const uint32_t (&qf)[NT][D / 16][2],
                                             const float (&rowfac)[NT][2],
                                             const int (&limit)[NT][2], int all_seen,
                                             uint32_t ring, uint32_t bars, uint32_t& parity,
                                             volatile int* abort_flag, int lane,
                                             AttnState<D, NT>& st, int& t0, int& slot) {
  using Tile = AttnTile<D>;
  constexpr int H = Tile::HALVES;
  constexpr int S = Tile::STAGES;
  constexpr int KW = D / 64;   // 16-byte chunks of a token's K row a lane takes
  constexpr int VW = D / 128 > 0 ? D / 128 : 1;  // the same of V (8 bytes at D = 64)
  constexpr int VB = D / 8 < 16 ? D / 8 : 16;    // contiguous bytes of V a lane takes
  const int g = lane >> 2, c = lane & 3;
#pragma unroll 1
  for (; t0 < f.end; t0 += Tile::UNIT) {
    float sk[H], lv[H], back[H];  // lv: log2 sv, back: 2^(Lr - lv)
    bool gone[H];                 // no such block: its tokens are left out
    bool far = false;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      sk[h] = scale_value(f.ksc[0][h]);
      gone[h] = !((f.have[0] >> h) & 1u);
      lv[h] = gone[h] ? st.ref : __log2f(f.vsc[0][h]);  // -inf for a block of zeros
      if (!FAR && h == 0 && t0 == f.t_first && lv[0] > -INFINITY) st.ref = lv[0];
      far = far || !(fabsf(lv[h] - st.ref) <= 40.0f);
      back[h] = ex2(st.ref - lv[h]);
    }
    if (!FAR && __builtin_expect(__any_sync(0xFFFFFFFFu, far), 0)) break;
    if (!mbar_wait(bars + 8 * slot, (parity >> slot) & 1u, abort_flag)) {
      // given up: what is on its way lands (bounded) while the CTA is there
#pragma unroll 1
      for (int i = 0; i < S - 1; ++i, t0 += Tile::UNIT)
        if (t0 < f.end) {
          const int at = (slot + i) % S;
          mbar_wait_bounded(bars + 8 * at, (parity >> at) & 1u, kDrainLimitNs);
        }
      t0 = f.end;
      break;
    }
    parity ^= 1u << slot;
#pragma unroll
    for (int i = 0; i + 2 < S; ++i) {
      f.have[i] = f.have[i + 1];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        f.ksc[i][h] = f.ksc[i + 1][h];
        f.vsc[i][h] = f.vsc[i + 1][h];
      }
    }
    const uint32_t stage = ring + slot * Tile::STAGE;
    __syncwarp();  // the whole warp is done with the tile before, whose stage is filled next
    feed_issue(p, f, k_map, v_map, ring, bars, lane, t0 + (S - 1) * Tile::UNIT,
               slot == 0 ? S - 1 : slot - 1, S - 2);
    feed_look_up(p, f);
    slot = slot + 1 == S ? 0 : slot + 1;
    // ---- S^T: all reads first, the halves' products in turn (a warp has few
    // neighbours on its scheduler to hide its latencies)
    uint4 kr[H][2][KW];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < KW; ++j)
          kr[h][i][j] = lds_16(stage + h * 16 * Tile::BOX + attn_place<D>(g + 8 * i, attn_k_dim<D>(j, c)));
    float s[H][NT][4];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[h][n][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4 * KW; ++j)  // word j % 4 of chunk j / 4
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint4 k0 = kr[h][0][j >> 2], k1 = kr[h][1][j >> 2];
        const uint32_t w0 = (j & 3) == 0 ? k0.x : (j & 3) == 1 ? k0.y : (j & 3) == 2 ? k0.z : k0.w;
        const uint32_t w1 = (j & 3) == 0 ? k1.x : (j & 3) == 1 ? k1.y : (j & 3) == 2 ? k1.z : k1.w;
        uint32_t a0, a1, a2, a3;
        codes_to_f16<E4M3>(w0, a0, a2);
        codes_to_f16<E4M3>(w1, a1, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_16816(s[h][n], a0, a1, a2, a3, qf[n][j][0], qf[n][j][1]);
      }
    // ---- V's codes, read while the softmax runs
    uint32_t vr[H][4][D / 32];  // the words of tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tk = 2 * c + (i & 1) + 8 * (i >> 1);
        const uint32_t half = stage + Tile::SIDE + h * 16 * Tile::BOX;
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          if constexpr (VB == 16) {
            const uint4 x = lds_16(half + attn_place<D>(tk, j * 128 + g * 16));
            vr[h][i][4 * j] = x.x;
            vr[h][i][4 * j + 1] = x.y;
            vr[h][i][4 * j + 2] = x.z;
            vr[h][i][4 * j + 3] = x.w;
          } else {
            const uint2 x = lds_8(half + attn_place<D>(tk, g * 8));
            vr[h][i][0] = x.x;
            vr[h][i][1] = x.y;
          }
        }
      }
    // ---- softmax
    const bool masked = t0 + Tile::TOKENS > all_seen || gone[0] || gone[H - 1];
    bool moved = false;
    float alpha[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[h][n][i] = fmaf(s[h][n][i], sk[h] * rowfac[n][i & 1], FAR ? 0.0f : lv[h]);
          if (masked && (gone[h] || t0 + 16 * h + g + 8 * (i >> 1) >= limit[n][i & 1]))
            s[h][n][i] = -INFINITY;
          top[i & 1] = fmaxf(top[i & 1], s[h][n][i]);
        }
      if constexpr (FAR) {  // (s without lv)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = fmaxf(st.x[n][i], top[i]);
          st.l[n][i] *= ex2(st.x[n][i] - exp_ref(x));
          st.x[n][i] = x;
          top[i] = -INFINITY;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            st.l[n][i] += ex2(s[h][n][i] - exp_ref(x)) + ex2(s[h][n][i + 2] - exp_ref(x));
            // (left out is left out, whatever lv is)
            s[h][n][i] = s[h][n][i] == -INFINITY ? -INFINITY : s[h][n][i] + lv[h];
            s[h][n][i + 2] = s[h][n][i + 2] == -INFINITY ? -INFINITY : s[h][n][i + 2] + lv[h];
            top[i] = fmaxf(top[i], fmaxf(s[h][n][i], s[h][n][i + 2]));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = top[i];
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
        const float m = fmaxf(st.m[n][i], x);
        moved = moved || m != st.m[n][i];
        alpha[n][i] = ex2(st.m[n][i] - exp_ref(m));
        st.m[n][i] = m;
        if constexpr (!FAR) st.l[n][i] *= alpha[n][i];
      }
    }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) st.o[j][n][i] *= alpha[n][i & 1];
    }
    // ---- P^T and O^T
#pragma unroll
    for (int h = 0; h < H; ++h) {
      uint32_t b[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = ex2(s[h][n][i] + (10.0f - exp_ref(st.m[n][i & 1])));
          if constexpr (!FAR) st.l[n][i & 1] = fmaf(e[i], back[h], st.l[n][i & 1]);
        }
        b[n][0] = transpose_8x8(pack_f16x2(e[0], e[1]));
        b[n][1] = transpose_8x8(pack_f16x2(e[2], e[3]));
      }
      if (E4M3 && masked) {
        // 0 * NaN is NaN: the codes of tokens that not every row sees go in as
        // zeros, and a product of "is NaN" and "is seen" says where they show
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < D / 32; ++j) bad |= nan_codes(vr[h][i][j]);
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, bad != 0), 0)) {
          uint32_t one[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int tk = t0 + 16 * h + g + 8 * x;
              one[n][x] = transpose_8x8(pack_f16x2(!gone[h] && tk < limit[n][0] ? 1.0f : 0.0f,
                                                   !gone[h] && tk < limit[n][1] ? 1.0f : 0.0f));
            }
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t w[4], f[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = nan_codes(vr[h][i][j]);
              vr[h][i][j] &= ~w[i];
              w[i] &= 0x38383838u;  // 1.0
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              codes_to_f16<E4M3>(__byte_perm(w[2 * i], w[2 * i + 1], 0x5140), f[i][0], f[i][1]);
              codes_to_f16<E4M3>(__byte_perm(w[2 * i], w[2 * i + 1], 0x7362), f[i][2], f[i][3]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_16816(count, f[0][2 * i], f[0][2 * i + 1], f[1][2 * i], f[1][2 * i + 1], one[n][0], one[n][1]);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if (count[x] != 0.0f) st.o[2 * j + i][n][x] = NAN;
              }
          }
        }
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

// CTAs an SM that the registers are cut to: as many as the accumulators of the
// column tiles allow, so that as many rings are in flight.
template <int D, int NT>
constexpr int attn_ctas() { return D == 64 ? (NT == 1 ? 4 : 3) : D == 128 && NT == 1 ? 3 : 2; }

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kAttnThreads, (attn_ctas<D, NT>()))
    kv_attention_kernel(const AttnArgs p, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map) {
  constexpr int ROWS = 8 * NT;
  constexpr int PIECE = ROWS * (D + 2);
  constexpr int UNIT = AttnTile<D>::UNIT;
  constexpr int S = AttnTile<D>::STAGES;
  // the warps' rings, on a 1024-byte boundary
  extern __shared__ uint8_t sm_attn[];
  __shared__ float sm_o[kAttnWarps * kAttnMeet * NT * 4 * 32];  // where the warps' parts meet
  __shared__ __align__(8) uint64_t sm_bars[kAttnWarps][S];
  __shared__ int abort_flag;
  __shared__ float sm_m[kAttnWarps][ROWS], sm_l[kAttnWarps][ROWS];  // R and L
  __shared__ int64_t sm_scan[kAttnWarps];
  __shared__ int64_t sm_base;
  __shared__ int sm_req;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int group = p.q_heads / p.kv_heads;
  const uint32_t ring = ((smem_u32(sm_attn) + 1023u) & ~1023u) + warp * (S * AttnTile<D>::STAGE);
  const uint32_t bars = smem_u32(sm_bars[warp]);
  uint32_t parity = 0;
  if (lane < S) mbar_init(bars + 8 * lane, 1);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
  }
  fence_mbarrier_init();
  fence_proxy_async_smem();
  __syncwarp();

  pdl_wait();
  // ---- this CTA's share of the units
  const int chunk = (p.requests + kAttnThreads - 1) / kAttnThreads;
  const int r_lo = min(p.requests, static_cast<int>(threadIdx.x) * chunk);
  const int r_hi = min(p.requests, r_lo + chunk);
  int64_t mine = 0, total;
  for (int r = r_lo; r < r_hi; ++r) mine += attn_request<ROWS, UNIT>(p, r).units;
  int64_t before = attn_scan(mine, total, sm_scan);
  const int64_t workers = min(total, static_cast<int64_t>(gridDim.x));
  if (blockIdx.x >= workers) {
    if (threadIdx.x == 0) p.cut[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  int64_t u = blockIdx.x * total / workers;
  const int64_t u_end = (blockIdx.x + 1) * total / workers;
  if (before <= u && u < before + mine) {
    int r = r_lo;
    for (; r < r_hi - 1; ++r) {
      const int64_t n = attn_request<ROWS, UNIT>(p, r).units;
      if (u < before + n) break;
      before += n;
    }
    sm_req = r;
    sm_base = before;
  }
  __syncthreads();
  if (threadIdx.x == 0) p.cut[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);

  // A segment: the part of an item in this share.
  struct Segment {
    int q0, pos0, len, rows;   // of the request
    int head, row0;
    int first, last, per_item; // units of the item
    int64_t item_u;            // the item's first unit
  };
  int req = sm_req;
  int64_t base = sm_base;      // the request's first unit
  AttnRequest rq = attn_request<ROWS, UNIT>(p, req);
  AttnFeed<D> feed;
  // finds the segment at u, begins its copies and moves u past it
  auto begin_segment = [&](Segment& sg) {
    for (; u >= base + rq.units && req + 1 < p.requests;) {
      base += rq.units;
      rq = attn_request<ROWS, UNIT>(p, ++req);
    }
    const int64_t item = (u - base) / rq.per_item;
    sg.q0 = rq.q0;
    sg.pos0 = rq.pos0;
    sg.len = rq.len;
    sg.rows = rq.fresh * group;
    sg.per_item = rq.per_item;
    sg.item_u = base + item * rq.per_item;
    sg.first = static_cast<int>(u - sg.item_u);
    sg.last = static_cast<int>(min(static_cast<int64_t>(rq.per_item), u_end - sg.item_u));
    sg.head = static_cast<int>(item / rq.tiles);
    sg.row0 = static_cast<int>(item - static_cast<int64_t>(sg.head) * rq.tiles) * ROWS;
    const int newest = (min(sg.row0 + ROWS, sg.rows) - 1) / group;  // new token of the tile's last row
    const int most = min(max(sg.pos0 + newest + 1, 0), sg.len);
    feed_begin<D>(p, feed, &k_map, &v_map, p.table + req * p.ld_table, sg.head, sg.first * UNIT,
                  min(most, sg.last * UNIT), ring, bars, warp, lane);
    u = sg.item_u + sg.last;
  };
  // every round ends an item or the share, so there are at most u_end - u
  for (; u < u_end;) {
    Segment sg;
    begin_segment(sg);                   // its first keys come while q is read

    // q fragments (column n of a tile is row g) and what the lane's two columns
    // of S^T need: their factor and the first position that they do not see
    uint32_t qf[NT][D / 16][2];
    float rowfac[NT][2];
    int limit[NT][2];
    int least = 0x7FFFFFFF;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = sg.row0 + 8 * n + g;
      const bool real = r < sg.rows;
      const int i = real ? r / group : 0;
      const uint16_t* qp = p.q + (static_cast<int64_t>(sg.q0) + i) * p.ldq_token +
                           (sg.head * group + (real ? r - i * group : 0)) * p.ldq_head;
      uint2 w[D / 16];
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const int d = attn_k_dim<D>(j >> 2, c) + (j & 3) * 4;  // step j = 4 * chunk + word
        w[j] = real ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0u, 0u);
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
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * p.scale_log2;
      const int lim = real ? min(max(sg.pos0 + i + 1, 0), sg.len) : 0;
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        rowfac[n][i2] = __shfl_sync(0xFFFFFFFFu, down, (2 * c + i2) * 4);
        limit[n][i2] = __shfl_sync(0xFFFFFFFFu, lim, (2 * c + i2) * 4);
      }
      least = min(least, real ? lim : 0x7FFFFFFF);
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);

    AttnState<D, NT> st;
    st.ref = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      st.m[n][0] = st.m[n][1] = -INFINITY;
      st.l[n][0] = st.l[n][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[j][n][i] = 0.0f;
    }
    int t0 = feed.t_first, at = 0;  // (the ring begins each segment at its first stage)
    attend_tiles<D, E4M3, NT, false>(p, feed, &k_map, &v_map, qf, rowfac, limit, least, ring, bars,
                                     parity, &abort_flag, lane, st, t0, at);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) st.x[n][i] = st.m[n][i] - 10.0f - st.ref;
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, t0 < feed.end), 0)) {
      attend_tiles<D, E4M3, NT, true>(p, feed, &k_map, &v_map, qf, rowfac, limit, least, ring, bars,
                                      parity, &abort_flag, lane, st, t0, at);
      // the lanes' sums on one X, that of the row
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = st.x[n][i];
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
          st.l[n][i] *= ex2(st.x[n][i] - exp_ref(x));
          st.x[n][i] = x;
        }
    }
    // ---- the four warps' parts meet
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = st.l[n][i];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        if (g == 0) {
          sm_m[warp][8 * n + 2 * c + i] = st.m[n][i];
          sm_l[warp][8 * n + 2 * c + i] = attn_log(st.x[n][i], l);
        }
      }
    const bool whole = sg.first == 0 && sg.last == sg.per_item;
    // a piece of an item begun earlier goes to the first slot, of one that
    // goes on to the second
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (sg.first == 0 ? 1 : 0);
    float* piece = p.pieces + slot * PIECE;
    // through kAttnMeet m-tiles' worth of shared memory at a time: in turn, a
    // thread of either half of the CTA finds the m-tiles that it owns there
    float o[NT][D / 16];
#pragma unroll
    for (int part = 0; part < D / 16 / kAttnMeet; ++part) {
      // m-tiles 2 * part + {0, 1} of each half of the head dimension's m-tiles
#pragma unroll
      for (int x = 0; x < kAttnMeet; ++x) {
        const int j = (x / (kAttnMeet / 2)) * (D / 32) + part * (kAttnMeet / 2) + x % (kAttnMeet / 2);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sm_o[((warp * kAttnMeet + x) * NT * 4 + n * 4 + i) * 32 + lane] = st.o[j][n][i];
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = 8 * n + attn_own_row(threadIdx.x);
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, sm_m[w][row]);
#pragma unroll
        for (int k = 0; k < kAttnMeet; ++k) o[n][part * kAttnMeet + k] = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
          const float f = ex2(sm_m[w][row] - exp_ref(m));
#pragma unroll
          for (int k = 0; k < kAttnMeet; ++k) {
            const int x = static_cast<int>(threadIdx.x >> 6) * (kAttnMeet / 2) + (k >> 1);
            const int i = 2 * (k & 1) + ((threadIdx.x >> 5) & 1);
            o[n][part * kAttnMeet + k] = fmaf(
                f, sm_o[((w * kAttnMeet + x) * NT * 4 + n * 4 + i) * 32 + lane], o[n][part * kAttnMeet + k]);
          }
        }
      }
      if (part + 1 < D / 16 / kAttnMeet) __syncthreads();  // read, before the next part
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = 8 * n + attn_own_row(threadIdx.x);
      float m = -INFINITY, most = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        m = fmaxf(m, sm_m[w][row]);
        most = fmaxf(most, sm_l[w][row]);
      }
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) l += ex2(sm_l[w][row] - exp_ref(most));
      const float L = attn_log(most, l);
      if (whole) {
        if (sg.row0 + row < sg.rows) attn_write<D>(p, sg.q0, sg.row0 + row, sg.head, threadIdx.x, o[n], m, L);
      } else {
        float* to = piece + (n * kAttnThreads + threadIdx.x) * (D / 16);
#pragma unroll
        for (int k = 0; k < D / 16; k += 4)
          *reinterpret_cast<float4*>(to + k) = make_float4(o[n][k], o[n][k + 1], o[n][k + 2], o[n][k + 3]);
        if (attn_own_dim<D>(threadIdx.x) == 0) {
          piece[ROWS * D + 2 * row] = m;
          piece[ROWS * D + 2 * row + 1] = L;
        }
      }
    }
    if (!whole && sg.first == 0 && threadIdx.x == 0) {
      // the worker that holds the item's last unit
      const int64_t w_end = ((sg.item_u + sg.per_item) * workers - 1) / total;
      p.cut[2 * blockIdx.x] = make_int4(static_cast<int>(w_end), sg.head, sg.row0, sg.rows);
      p.cut[2 * blockIdx.x + 1] = make_int4(sg.q0, 0, 0, 0);
    }
    __syncthreads();  // the sums have been read
    if (abort_flag) break;
  }
  // (not earlier: CTAs of the join beside those still at work cost 20 %)
  pdl_trigger();
}

// Joins the pieces of the items that workers began and did not end: CTA (w, n)
// the column tile n of worker w's.  Its groups of kAttnThreads take every
// kJoinGroups-th piece; the groups' sums meet in a fixed order.
template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads* kJoinGroups) kv_attention_join_kernel(const AttnArgs p) {
  constexpr int ROWS = 8 * NT;
  constexpr int PIECE = ROWS * (D + 2);
  __shared__ float sm_m[kJoinGroups][8], sm_x[kJoinGroups][8], sm_l[kJoinGroups][8];
  __shared__ float sm_o[kJoinGroups - 1][D / 16][kAttnThreads];
  const int w0 = blockIdx.x, n = blockIdx.y;
  const int t = threadIdx.x % kAttnThreads, grp = threadIdx.x / kAttnThreads;
  pdl_wait();
  const int4 cut = p.cut[2 * w0];
  pdl_trigger();
  if (cut.x < 0) return;
  const int q0 = p.cut[2 * w0 + 1].x;
  const int pieces = cut.x - w0 + 1;
  const int row = attn_own_row(t);
  float m = -INFINITY, xm = -INFINITY, l = 0.0f, o[D / 16];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) o[k] = 0.0f;
#pragma unroll 2
  for (int i = grp; i < pieces; i += kJoinGroups) {
    const float* piece = p.pieces + (i == 0 ? 2 * static_cast<int64_t>(w0) + 1 : 2 * (static_cast<int64_t>(w0) + i)) * PIECE;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(piece + ROWS * D) + 8 * n + row);  // R, L
    float4 v[D / 64];
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      v[k] = __ldcg(reinterpret_cast<const float4*>(piece + (n * kAttnThreads + t) * (D / 16)) + k);
    const float top = fmaxf(m, ml.x), most = fmaxf(xm, ml.y);
    const float keep = ex2(m - exp_ref(top)), add = ex2(ml.x - exp_ref(top));
    l = l * ex2(xm - exp_ref(most)) + ex2(ml.y - exp_ref(most));
    m = top;
    xm = most;
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      o[4 * k] = o[4 * k] * keep + v[k].x * add;
      o[4 * k + 1] = o[4 * k + 1] * keep + v[k].y * add;
      o[4 * k + 2] = o[4 * k + 2] * keep + v[k].z * add;
      o[4 * k + 3] = o[4 * k + 3] * keep + v[k].w * add;
    }
  }
  if (attn_own_dim<D>(t) == 0) {
    sm_m[grp][row] = m;
    sm_x[grp][row] = xm;
    sm_l[grp][row] = l;
  }
  if (grp > 0) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) sm_o[grp - 1][k][t] = o[k];
  }
  __syncthreads();
  if (grp > 0) return;
  float top = -INFINITY, most = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinGroups; ++i) {
    top = fmaxf(top, sm_m[i][row]);
    most = fmaxf(most, sm_x[i][row]);
  }
#pragma unroll
  for (int i = 0; i < kJoinGroups; ++i) {
    const float f = ex2(sm_m[i][row] - exp_ref(top));
    sum = fmaf(ex2(sm_x[i][row] - exp_ref(most)), sm_l[i][row], sum);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) o[k] = i == 0 ? o[k] * f : fmaf(f, sm_o[i > 0 ? i - 1 : 0][k][t], o[k]);
  }
  const int r = cut.z + 8 * n + row;
  if (r < cut.w) attn_write<D>(p, q0, r, cut.y, t, o, top, attn_log(most, sum));
}

}  // namespace i8
