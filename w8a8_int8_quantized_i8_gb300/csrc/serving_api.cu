// serving_api.cu -- the C ABI of the serving operators (declared in
// include/i8.h): the norm with the residual's addition and an 8-bit output,
// block tables, the 8-bit paged cache's append and the attention over it.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "../../include/i8.h"
#include "block_tables.cuh"
#include "host.h"
#include "kv_append.cuh"
#include "kv_attention.cuh"
#include "kv_prefill.cuh"
#include "ptx.cuh"
#include "rmsnorm.cuh"

namespace i8 {

cudaError_t take_serving_status(unsigned int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(*word));
  if (e == cudaSuccess && *word != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  }
  return e;
}

namespace {

constexpr int kMaxDevices = 64;

i8_status device_sms(int* sms) {
  static int cached[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return I8_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  if (cached[dev] == 0 &&
      cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return I8_ERR_CUDA;
  *sms = cached[dev];
  return I8_OK;
}

// Shared memory beyond 48 KB, allowed once per kernel and device.
template <auto KERN>
i8_status allow_smem(size_t bytes) {
  static bool done[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return I8_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  if (done[dev]) return I8_OK;
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) != cudaSuccess)
    return I8_ERR_CUDA;
  done[dev] = true;
  return I8_OK;
}

// ----------------------------------------------------------------- norm
struct NormArgs {
  const uint16_t *x, *res, *weight;
  uint16_t* h;
  int8_t* q;
  float* scale;
  int64_t rows, ldx, ldr, ldq, ldh;
  int K, G;
  float eps;
};

template <int V>
cudaError_t launch_norm_v(const NormArgs& a, int fmt, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.rows)), block(32 * a.G);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, block, 0, st, a.x, a.K, a.ldx, a.res, a.ldr, a.weight, a.eps, a.q,
                      a.ldq, a.scale, a.h, a.ldh, a.G);
  };
  if (fmt == kQuantE4M3) return go(add_rmsnorm_quant_kernel<V, kQuantE4M3>);
  if (fmt == kQuantF16) return go(add_rmsnorm_quant_kernel<V, kQuantF16>);
  return go(add_rmsnorm_quant_kernel<V, kQuantInt8>);
}

// ----------------------------------------------------------------- overlap
// Memory of an operand: `rows` rows of `bytes`, `stride` bytes apart.
struct Extent {
  const void* base;
  int64_t bytes;
  int64_t rows = 1;
  int64_t stride = 0;
};

// Whether rows of `t` and the one row of `v` share a byte.
bool overlap(const Extent& t, const Extent& v) {
  if (!t.base || !v.base || t.bytes <= 0 || t.rows <= 0 || v.bytes <= 0) return false;
  const int64_t lo = static_cast<int64_t>(reinterpret_cast<uintptr_t>(v.base) - reinterpret_cast<uintptr_t>(t.base));
  const int64_t hi = lo + v.bytes;  // from t's base on
  if (hi <= 0) return false;
  // the first row that ends behind lo
  const int64_t row = lo < t.bytes ? 0 : t.rows == 1 ? 1 : (lo - t.bytes) / t.stride + 1;
  return row < t.rows && row * t.stride < hi;
}

// Whether a row of `a` shares a byte with another row of `b` (both of as many
// rows): a row may lie where the other's same row does.
bool rows_cross(const Extent& a, const Extent& b) {
  if (!a.base || !b.base || a.rows <= 1) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
  if (d >= (a.rows - 1) * a.stride + a.bytes || d + (b.rows - 1) * b.stride + b.bytes <= 0) return false;
  if (a.stride != b.stride) {
    for (int64_t i = 0; i < b.rows; ++i) {
      const Extent row{static_cast<const char*>(b.base) + i * b.stride, b.bytes};
      const Extent before{a.base, a.bytes, i, a.stride};
      const Extent after{static_cast<const char*>(a.base) + (i + 1) * a.stride, a.bytes, a.rows - i - 1, a.stride};
      if (overlap(before, row) || overlap(after, row)) return true;
    }
    return false;
  }
  // row i + k of a begins d - k * stride before row i of b
  const int64_t k = d >= 0 ? d / a.stride : -((-d + a.stride - 1) / a.stride), r = d - k * a.stride;
  return (k != 0 && std::abs(k) < a.rows && r < a.bytes) ||
         (k + 1 != 0 && std::abs(k + 1) < a.rows && a.stride - r < b.bytes);
}

// Whether rows [tokens, heads] of `dim` elements, these strides apart, share an
// element.
bool rows_overlap(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
  if ((tokens > 1 && token < dim) || (heads > 1 && head < dim)) return true;
  if (tokens <= 1 || heads <= 1) return false;
  if (token >= head * (heads - 1) + dim || head >= token * (tokens - 1) + dim) return false;
  // neither inside the other: the tokens nearest to each head's offset
  for (int64_t h = 1; h < heads; ++h)
    for (int64_t t = h * head / token; t <= h * head / token + 1 && t < tokens; ++t)
      if (std::abs(h * head - t * token) < dim) return true;
  return false;
}

// ----------------------------------------------------------------- cache checks
i8_status check_cache(const i8_kv_cache* c) {
  if (!c || c->blocks < 0 || c->block_size <= 0 || c->kv_heads <= 0 || c->head_dim <= 0)
    return I8_ERR_INVALID_ARG;
  if (c->fmt != I8_CODES_INT8 && c->fmt != I8_CODES_E4M3) return I8_ERR_INVALID_ARG;
  if (c->blocks > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return I8_ERR_INVALID_ARG;
  if (c->block_size % 16 != 0 || c->block_size > 1024 || c->blocks > INT32_MAX ||
      c->kv_heads > 32767 || c->blocks * c->kv_heads > INT32_MAX)
    return I8_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return I8_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_scale) || !aligned4(c->v_scale))
    return I8_ERR_ALIGNMENT;
  return I8_OK;
}

// ----------------------------------------------------------------- attention
// Column tiles of 8 rows a CTA takes at once.  A second one shares the decoded
// codes of the first, but at 256 head dimensions its accumulators do not fit
// the registers.
int attention_nt(int64_t rows, int64_t head_dim) { return head_dim == 256 || rows <= 8 ? 1 : 2; }

template <int D, bool E4M3, int NT>
size_t attention_smem() {
  return 1024 + static_cast<size_t>(kAttnWarps) * AttnTile<D>::STAGES * AttnTile<D>::STAGE;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The cache's codes [blocks * kv_heads, block, D] in boxes of `rows` tokens by
// at most 128 bytes, swizzled (the warps' fragments) or as they are.  A third
// dimension for the block keeps every coordinate below 2^31 however large the
// cache is.
i8_status encode_cache(CUtensorMap* map, const void* base, const i8_kv_cache& c, int rows,
                       bool swizzle) {
  static std::mutex mu;
  static EncodeTiledFn encode = nullptr;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                           &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn)
        return I8_ERR_CUDA;
      encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
  }
  // (a cache of no blocks is never read: any extent and address will do)
  const cuuint64_t D = c.head_dim, B = c.block_size;
  const cuuint64_t dims[3] = {D, B, std::max<cuuint64_t>(1, static_cast<cuuint64_t>(c.blocks) * c.kv_heads)};
  const cuuint64_t strides[2] = {D, D * B};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(std::min<cuuint64_t>(D, 128)),
                             static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
                elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                !swizzle  ? CU_TENSOR_MAP_SWIZZLE_NONE
                : D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? I8_OK
             : I8_ERR_CUDA;
}

// CTAs of a kernel that are resident at once.
template <int D, bool E4M3, int NT>
i8_status attention_workers(int* workers) {
  static int cached[kMaxDevices] = {};
  static std::mutex mu;
  constexpr auto kern = kv_attention_kernel<D, E4M3, NT>;
  const size_t smem = attention_smem<D, E4M3, NT>();
  if (i8_status e = allow_smem<kern>(smem)) return e;
  int sms, dev = 0, per_sm = 0;
  if (i8_status e = device_sms(&sms)) return e;
  if (cudaGetDevice(&dev) != cudaSuccess) return I8_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  if (cached[dev] == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kAttnThreads, smem) != cudaSuccess ||
        per_sm < 1)
      return I8_ERR_CUDA;
    cached[dev] = sms * per_sm;
  }
  *workers = cached[dev];
  return I8_OK;
}

template <int D, int NT>
size_t attention_ws(int workers) {
  return static_cast<size_t>(workers) * 2 * (sizeof(int4) + sizeof(float) * 8 * NT * (D + 2));
}

// Rows of a request and kv head from which the tcgen05 kernel takes it.  It
// always pays for 256 rows; the warp kernel reads and converts the keys again
// for every 16.  us by the warp kernel / by tcgen05, requests of one length:
//                                    32 rows   64 rows   96 rows   128 rows   256
//   8 of 4096, 8 kv heads of 128     37 / 67   60 / 67   88 / 69   110 / 70   207 / 82
//   8 of 4096, 8 kv heads of 64      27 / 53   42 / 53   58 / 54    76 / 55   140 / 60
//   1 of 32768, 8 kv heads of 128    34 / 58   58 / 61   80 / 62   103 / 63   192 / 69
//   64 of 1024, 2 kv heads of 128    26 / 51   41 / 52   56 / 54    71 / 56   128 / 66
constexpr int kPrefillRows = 96;

template <int D>
size_t prefill_ws(int sms) {
  return static_cast<size_t>(sms) * 2 * (sizeof(int4) + sizeof(float) * kPreRows * (D + 2));
}

template <int D, bool E4M3>
i8_status launch_prefill(AttnArgs a, const i8_kv_cache* cache, void* ws, int sms, cudaStream_t st) {
  constexpr size_t smem = 1024 + PrefillSmem<D>::BYTES;
  if (i8_status e = allow_smem<kv_prefill_kernel<D, E4M3>>(smem)) return e;
  // the largest box of tokens that ends neither inside a block nor inside a tile
  a.box_rows = 16;
  while (a.box_rows < kPreTokens && a.block % (2 * a.box_rows) == 0) a.box_rows *= 2;
  a.cut = static_cast<int4*>(ws);
  a.pieces = reinterpret_cast<float*>(a.cut + 2 * static_cast<size_t>(sms));
  CUtensorMap k_map, v_map;
  const bool any = cache->blocks > 0;
  if (i8_status e = encode_cache(&k_map, any ? cache->k : ws, *cache, a.box_rows, false)) return e;
  if (i8_status e = encode_cache(&v_map, any ? cache->v : ws, *cache, a.box_rows, false)) return e;
  const dim3 grid(static_cast<unsigned>(sms));
  if (cudaError_t e = launch_pdl(kv_prefill_kernel<D, E4M3>, grid, dim3(kPreThreads), smem, st, a,
                                 k_map, v_map))
    return cuda_status(e);
  return cuda_status(launch_pdl(kv_prefill_join_kernel<D>, dim3(grid.x, kPreRows / kPreJoinRows),
                                dim3(32 * kPreJoinRows), 0, st, a));
}

template <int D, bool E4M3, int NT>
i8_status launch_attention(AttnArgs& a, const i8_kv_cache* cache, void* ws, size_t ws_bytes,
                           size_t* need, cudaStream_t st) {
  int workers;
  if (i8_status e = attention_workers<D, E4M3, NT>(&workers)) return e;
  // both kernels' pieces: the calls that follow one another may overlap
  const size_t own = attention_ws<D, NT>(workers);
  size_t bytes = own;
  const bool many = D <= 128 && static_cast<int64_t>(a.max_new) * (a.q_heads / a.kv_heads) >= kPrefillRows;
  int sms = 0;
  if (many) {
    if (i8_status e = device_sms(&sms)) return e;
    if constexpr (D <= 128) bytes += prefill_ws<D>(sms);
  }
  if (need) {
    *need = bytes;
    return I8_OK;
  }
  if (!ws || ws_bytes < bytes) return I8_ERR_WORKSPACE;
  if (!aligned16(ws)) return I8_ERR_ALIGNMENT;
  a.cut = static_cast<int4*>(ws);
  a.pieces = reinterpret_cast<float*>(a.cut + 2 * static_cast<size_t>(workers));
  a.split_rows = INT32_MAX;
  if constexpr (D <= 128) {
    if (many) {
      a.split_rows = kPrefillRows;
      if (i8_status e = launch_prefill<D, E4M3>(a, cache, static_cast<char*>(ws) + own, sms, st)) return e;
    }
  }
  a.unit_cols = AttnTile<D>::UNIT / a.block;
  a.unit_rest = AttnTile<D>::UNIT % a.block;
  a.box_rows = AttnTile<D>::HALVES == 2 && a.block % 32 == 0 ? 32 : 16;
  CUtensorMap k_map, v_map;
  const bool any = cache->blocks > 0;
  if (i8_status e = encode_cache(&k_map, any ? cache->k : ws, *cache, a.box_rows, true)) return e;
  if (i8_status e = encode_cache(&v_map, any ? cache->v : ws, *cache, a.box_rows, true)) return e;
  const dim3 grid(static_cast<unsigned>(workers));
  if (cudaError_t e = launch_pdl(kv_attention_kernel<D, E4M3, NT>, grid, dim3(kAttnThreads),
                                 attention_smem<D, E4M3, NT>(), st, a, k_map, v_map))
    return cuda_status(e);
  return cuda_status(launch_pdl(kv_attention_join_kernel<D, NT>, dim3(grid.x, NT),
                                dim3(kAttnThreads * kJoinGroups), 0, st, a));
}

// Runs the attention, or with `need` only says how much workspace it wants.
template <int D, bool E4M3>
i8_status attention_nt_dispatch(AttnArgs& a, const i8_kv_cache* cache, void* ws, size_t ws_bytes,
                                size_t* need, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.max_new) * (a.q_heads / a.kv_heads);
  if (attention_nt(rows, D) == 1) return launch_attention<D, E4M3, 1>(a, cache, ws, ws_bytes, need, st);
  return launch_attention<D, E4M3, D == 256 ? 1 : 2>(a, cache, ws, ws_bytes, need, st);
}

i8_status attention_dispatch(AttnArgs& a, const i8_kv_cache* cache, int head_dim, bool e4m3,
                             void* ws, size_t ws_bytes, size_t* need, cudaStream_t st) {
  switch (head_dim) {
    case 64:
      return e4m3 ? attention_nt_dispatch<64, true>(a, cache, ws, ws_bytes, need, st)
                  : attention_nt_dispatch<64, false>(a, cache, ws, ws_bytes, need, st);
    case 128:
      return e4m3 ? attention_nt_dispatch<128, true>(a, cache, ws, ws_bytes, need, st)
                  : attention_nt_dispatch<128, false>(a, cache, ws, ws_bytes, need, st);
    case 256:
      return e4m3 ? attention_nt_dispatch<256, true>(a, cache, ws, ws_bytes, need, st)
                  : attention_nt_dispatch<256, false>(a, cache, ws, ws_bytes, need, st);
  }
  return I8_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace i8

using namespace i8;

extern "C" {

i8_status i8_add_rmsnorm_quant_act_pertoken(const void* x, int64_t M, int64_t K, int64_t ldx,
                                            const void* residual, int64_t ldr, const void* weight,
                                            float eps, int fmt, void* q, int64_t ldq, float* s_a,
                                            void* h, int64_t ldh, i8_stream_t stream) {
  I8_NVTX();
  if (M < 0 || K <= 0 || ldx < K || ldq < K || (residual && ldr < K) || (h && ldh < K))
    return I8_ERR_INVALID_ARG;
  if (fmt != kQuantInt8 && fmt != kQuantE4M3 && fmt != kQuantF16) return I8_ERR_INVALID_ARG;
  if (!(eps >= 0.0f && eps <= 3.0e38f)) return I8_ERR_INVALID_ARG;
  if (M > 0 && (!x || !q || !s_a)) return I8_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > 32768 || M > INT32_MAX) return I8_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(q) || !aligned4(s_a) || ldx % 8 != 0 ||
      ldq % (fmt == kQuantF16 ? 8 : 16) != 0 || !aligned16(residual) ||
      (residual && ldr % 8 != 0) || !aligned16(weight) || !aligned16(h) || (h && ldh % 8 != 0))
    return I8_ERR_ALIGNMENT;
  // a row's CTA writes its h when others have not read theirs
  const Extent to{h, K * 2, M, ldh * 2};
  if (rows_cross(to, {x, K * 2, M, ldx * 2}) || rows_cross(to, {residual, K * 2, M, ldr * 2}))
    return I8_ERR_INVALID_ARG;
  if (M == 0) return I8_OK;
  const int vecs = static_cast<int>(K / 8);
  int G = 1;
  while (G < 16 && (vecs + 32 * G - 1) / (32 * G) > 6) G *= 2;
  const int need = (vecs + 32 * G - 1) / (32 * G);
  const NormArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual),
                   static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(h),
                   static_cast<int8_t*>(q), s_a, M, ldx, ldr, ldq, ldh, static_cast<int>(K), G, eps};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (need <= 1) e = launch_norm_v<1>(a, fmt, st);
  else if (need <= 2) e = launch_norm_v<2>(a, fmt, st);
  else if (need <= 4) e = launch_norm_v<4>(a, fmt, st);
  else if (need <= 6) e = launch_norm_v<6>(a, fmt, st);
  else e = launch_norm_v<8>(a, fmt, st);
  return cuda_status(e);
}

i8_status i8_build_block_tables(const int32_t* context_lens, const int32_t* new_lens,
                                int64_t requests, int32_t* block_tables, int64_t width,
                                int64_t ld_table, const int32_t* free_blocks, int64_t n_free,
                                const int32_t* taken, int64_t block_size, int64_t max_tokens,
                                int32_t* cu_new, int32_t* seq_lens, int64_t* slots,
                                int32_t* positions, int32_t* counts, i8_stream_t stream) {
  I8_NVTX();
  if (requests < 0 || width < 0 || ld_table < width || n_free < 0 || block_size <= 0 ||
      max_tokens < 0)
    return I8_ERR_INVALID_ARG;
  if (!cu_new || !counts || (max_tokens > 0 && (!slots || !positions)) || (n_free > 0 && !free_blocks) ||
      (requests > 0 && (!context_lens || !new_lens || !seq_lens || (width > 0 && !block_tables))))
    return I8_ERR_INVALID_ARG;
  if (requests > kTableMaxRequests || block_size > 1024 || width > INT32_MAX ||
      n_free > INT32_MAX - width || max_tokens > INT32_MAX || width * block_size > INT32_MAX)
    return I8_ERR_UNSUPPORTED;
  if (!aligned4(context_lens) || !aligned4(new_lens) || !aligned4(block_tables) ||
      !aligned4(free_blocks) || !aligned4(taken) || !aligned4(cu_new) || !aligned4(seq_lens) ||
      !aligned8(slots) || !aligned4(positions) || !aligned4(counts))
    return I8_ERR_ALIGNMENT;
  // every CTA reads the inputs for itself while others write
  const int64_t word = sizeof(int32_t);
  const Extent table{block_tables, width * word, requests, ld_table * word};
  const Extent in[] = {{context_lens, requests * word}, {new_lens, requests * word}, {taken, word},
                       {free_blocks, n_free * word}};
  const Extent out[] = {{cu_new, (requests + 1) * word}, {seq_lens, requests * word}, {slots, max_tokens * 2 * word},
                        {positions, max_tokens * word}, {counts, 3 * word}};
  for (const Extent& v : in)
    if (overlap(table, v)) return I8_ERR_INVALID_ARG;
  for (const Extent& v : out) {
    if (overlap(table, v)) return I8_ERR_INVALID_ARG;
    for (const Extent& u : in)
      if (overlap(u, v)) return I8_ERR_INVALID_ARG;
    for (const Extent& u : out)
      if (&u != &v && overlap(u, v)) return I8_ERR_INVALID_ARG;
  }
  TableArgs a{context_lens, new_lens, block_tables, free_blocks, taken, cu_new, seq_lens, slots,
              positions, counts, ld_table, n_free, max_tokens, static_cast<int32_t>(requests),
              static_cast<int32_t>(width), static_cast<int32_t>(block_size), -1};
  if ((block_size & (block_size - 1)) == 0)
    for (a.shift = 0; (int64_t{1} << a.shift) < block_size;) ++a.shift;
  int sms;
  if (i8_status e = device_sms(&sms)) return e;
  const size_t smem = sizeof(int32_t) * (3 * static_cast<size_t>(requests) + 1);
  if (i8_status e = allow_smem<block_tables_kernel>(sizeof(int32_t) * (3 * kTableMaxRequests + 1)))
    return e;
  const int64_t grid = std::max<int64_t>(
      1, std::min<int64_t>(sms, std::max((max_tokens + kTableThreads - 1) / kTableThreads,
                                         requests / (kTableThreads / 32))));
  return cuda_status(launch_pdl(block_tables_kernel, dim3(static_cast<unsigned>(grid)),
                                dim3(kTableThreads), smem, reinterpret_cast<cudaStream_t>(stream), a));
}

i8_status i8_kv_cache_append(const void* k, int64_t ldk_token, int64_t ldk_head, const void* v,
                             int64_t ldv_token, int64_t ldv_head, const int64_t* slots,
                             int64_t tokens, const i8_kv_cache* cache, i8_stream_t stream) {
  I8_NVTX();
  if (i8_status e = check_cache(cache)) return e;
  if (tokens < 0 || (tokens > 0 && (!k || !v || !slots))) return I8_ERR_INVALID_ARG;
  if (ldk_token < 0 || ldk_head < 0 || ldv_token < 0 || ldv_head < 0) return I8_ERR_INVALID_ARG;
  if (tokens > INT32_MAX) return I8_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned8(slots) || ldk_token % 8 != 0 ||
      ldk_head % 8 != 0 || ldv_token % 8 != 0 || ldv_head % 8 != 0)
    return I8_ERR_ALIGNMENT;
  if (tokens == 0 || cache->blocks == 0) return I8_OK;
  int sms;
  if (i8_status e = device_sms(&sms)) return e;
  AppendArgs a;
  a.k = {static_cast<const uint16_t*>(k), ldk_token, ldk_head, static_cast<uint8_t*>(cache->k),
         cache->k_scale};
  a.v = {static_cast<const uint16_t*>(v), ldv_token, ldv_head, static_cast<uint8_t*>(cache->v),
         cache->v_scale};
  a.slots = slots;
  a.tokens = tokens;
  a.blocks = cache->blocks;
  a.heads = cache->kv_heads;
  a.block = cache->block_size;
  a.dim_shift = cache->head_dim == 64 ? 6 : cache->head_dim == 128 ? 7 : 8;
  const int64_t units = tokens * 2 * cache->kv_heads;
  a.window = static_cast<int32_t>(std::min<int64_t>(
      kAppendMaxWindow, std::max<int64_t>(kAppendThreads / 32, units / (static_cast<int64_t>(sms) * 16))));
  const dim3 grid(static_cast<unsigned>((tokens + a.window - 1) / a.window),
                  static_cast<unsigned>(2 * cache->kv_heads));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(cache->fmt == I8_CODES_E4M3
                         ? launch_pdl(kv_append_kernel<true>, grid, dim3(kAppendThreads), 0, st, a)
                         : launch_pdl(kv_append_kernel<false>, grid, dim3(kAppendThreads), 0, st, a));
}

size_t i8_paged_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                          int fmt, int64_t max_new) {
  I8_NVTX();
  if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || q_heads > 65535 || max_new < 0 ||
      max_new > INT32_MAX || (fmt != I8_CODES_INT8 && fmt != I8_CODES_E4M3))
    return 0;
  AttnArgs a{};
  a.q_heads = static_cast<int32_t>(q_heads);
  a.kv_heads = static_cast<int32_t>(kv_heads);
  a.max_new = static_cast<int32_t>(max_new);
  size_t need = 0;
  if (attention_dispatch(a, nullptr, static_cast<int>(head_dim), fmt == I8_CODES_E4M3, nullptr, 0, &need,
                         nullptr) != I8_OK)
    return 0;
  return need;
}

i8_status i8_paged_attention(const void* q, int64_t ldq_token, int64_t ldq_head, int64_t tokens,
                             int64_t q_heads, const i8_kv_cache* cache,
                             const int32_t* block_tables, int64_t width, int64_t ld_table,
                             const int32_t* seq_lens, const int32_t* cu_new, int64_t requests,
                             int64_t max_new, float scale, void* out, int64_t ldo_token,
                             int64_t ldo_head, float* lse, void* ws, size_t ws_bytes,
                             i8_stream_t stream) {
  I8_NVTX();
  if (i8_status e = check_cache(cache)) return e;
  if (tokens < 0 || requests < 0 || width < 0 || ld_table < width || max_new < 0 || q_heads <= 0 ||
      q_heads % cache->kv_heads != 0)
    return I8_ERR_INVALID_ARG;
  if (ldq_token < 0 || ldq_head < 0 || ldo_token < 0 || ldo_head < 0) return I8_ERR_INVALID_ARG;
  if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return I8_ERR_INVALID_ARG;
  if (tokens > 0 && requests > 0 &&
      (!q || !out || !seq_lens || !cu_new || (width > 0 && !block_tables)))
    return I8_ERR_INVALID_ARG;
  if (tokens > INT32_MAX || requests > INT32_MAX || q_heads > 65535 ||
      width * cache->block_size > INT32_MAX - 1024)
    return I8_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out) || ldq_token % 8 != 0 || ldq_head % 8 != 0 ||
      ldo_token % 8 != 0 || ldo_head % 8 != 0 || !aligned4(block_tables) || !aligned4(seq_lens) ||
      !aligned4(cu_new) || !aligned4(lse))
    return I8_ERR_ALIGNMENT;
  if (rows_overlap(tokens, ldo_token, q_heads, ldo_head, cache->head_dim)) return I8_ERR_INVALID_ARG;
  if (tokens == 0 || requests == 0 || max_new == 0) return I8_OK;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.ldq_token = ldq_token;
  a.ldq_head = ldq_head;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.table = block_tables;
  a.ld_table = ld_table;
  a.seq_lens = seq_lens;
  a.cu_new = cu_new;
  a.out = static_cast<uint16_t*>(out);
  a.ldo_token = ldo_token;
  a.ldo_head = ldo_head;
  a.lse = lse;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.tokens = tokens;
  a.blocks = cache->blocks;
  a.requests = static_cast<int32_t>(requests);
  a.width = static_cast<int32_t>(width);
  a.block = cache->block_size;
  a.q_heads = static_cast<int32_t>(q_heads);
  a.kv_heads = cache->kv_heads;
  a.max_new = static_cast<int32_t>(std::min(max_new, tokens));
  return attention_dispatch(a, cache, cache->head_dim, cache->fmt == I8_CODES_E4M3, ws, ws_bytes, nullptr,
                            reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
