// fp4_api.cu -- the C ABI of the 4-bit route and of the heads' rotation (declared
// in include/i8.h): rows to microscaled 4-bit floating point, as they are or
// behind the norm, the product with a bias, the gated product, and the norm and
// rotation of query and key heads.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "../../include/i8.h"
#include "fp4_pair.cuh"
#include "fp4_quant.cuh"
#include "fp4_stream.cuh"
#include "heads_rotate.cuh"
#include "host.h"
#include "overlap.h"
#include "ptx.cuh"

namespace i8 {

cudaError_t take_fp4_status(unsigned int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_status, sizeof(*word));
  if (e == cudaSuccess && *word != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
  }
  return e;
}

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kFp4MaxK = 131072;

i8_status current_device(int* dev) {
  return cudaGetDevice(dev) == cudaSuccess && *dev >= 0 && *dev < kMaxDevices ? I8_OK : I8_ERR_CUDA;
}

i8_status device_sms(int dev, int* sms) {
  static int cached[kMaxDevices] = {};
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (cached[dev] == 0 &&
      cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return I8_ERR_CUDA;
  *sms = cached[dev];
  return I8_OK;
}

// Shared memory beyond 48 KB, allowed once per kernel and device.
template <auto KERN>
i8_status allow_smem(int dev, size_t bytes) {
  static bool done[kMaxDevices] = {};
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (done[dev]) return I8_OK;
  // (and all of the SM's: two CTAs that fit are meant to share it)
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess ||
      cudaFuncSetAttribute(KERN, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
          cudaSuccess)
    return I8_ERR_CUDA;
  done[dev] = true;
  return I8_OK;
}

// ----------------------------------------------------------------- rows
bool fp4_format(int fmt) { return fmt == I8_FP4_NV16 || fmt == I8_FP4_MX32; }
int fp4_deep(int64_t K) { return static_cast<int>((K + kFp4TileK - 1) / kFp4TileK); }

i8_status fp4_sizes(int64_t rows, int64_t K, int fmt) {
  if (rows < 0 || K <= 0 || !fp4_format(fmt)) return I8_ERR_INVALID_ARG;
  if (rows > INT32_MAX || K % 32 != 0 || K > kFp4MaxK) return I8_ERR_UNSUPPORTED;
  return I8_OK;
}

i8_status check_quant(const void* x, int64_t rows, int64_t K, int64_t ldx, int fmt, const void* codes,
                      const void* block_scales, const float* row_scales) {
  if (i8_status e = fp4_sizes(rows, K, fmt)) return e;
  if (ldx < K) return I8_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !codes || !block_scales || (fmt == I8_FP4_NV16 && !row_scales))) return I8_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(block_scales) || !aligned4(row_scales) || ldx % 8 != 0)
    return I8_ERR_ALIGNMENT;
  const Extent in{x, K * 2, rows, ldx * 2};
  const Extent out[] = {{codes, rows * (K / 2)},
                        {block_scales, static_cast<int64_t>(i8_fp4_block_scale_bytes(rows, K, fmt))},
                        {row_scales, fmt == I8_FP4_NV16 ? rows * 4 : 0}};
  for (const Extent& u : out) {
    if (overlap(in, u)) return I8_ERR_INVALID_ARG;
    for (const Extent& v : out)
      if (&u != &v && overlap(u, v)) return I8_ERR_INVALID_ARG;
  }
  return I8_OK;
}

template <bool MX, bool NORM>
cudaError_t launch_quant(Fp4QuantArgs& a, int64_t rows, cudaStream_t st) {
  const int vecs = a.deep;  // runs of 256 elements
  a.rows = rows;
  auto go = [&](auto kern, int V) {
    a.G = V > 0 ? (vecs + V - 1) / V : 16;
    a.R = V > 0 ? std::max(1, 4 / a.G) : 1;  // (long rows: one)
    return launch_pdl(kern, dim3(static_cast<unsigned>((rows + a.R - 1) / a.R)), dim3(32, a.G, a.R), 0, st, a);
  };
  // few rows: a warp for each 256 elements; many: fewer warps, with more in hand, to
  // meet at the row's barrier
  const int V = rows <= 512 ? 1 : vecs < 8 ? 2 : vecs < (NORM ? 64 : 32) ? 4 : 8;
  if (vecs > 128) return go(fp4_quant_kernel<0, MX, NORM>, 0);
  if (V == 1 && vecs <= 16) return go(fp4_quant_kernel<1, MX, NORM>, 1);
  if (V <= 2 && vecs <= 32) return go(fp4_quant_kernel<2, MX, NORM>, 2);
  if (V <= 4 && vecs <= 64) return go(fp4_quant_kernel<4, MX, NORM>, 4);
  return go(fp4_quant_kernel<8, MX, NORM>, 8);
}

// ----------------------------------------------------------------- products
i8_status check_rows(const i8_fp4_rows* r) {
  if (!r) return I8_ERR_INVALID_ARG;
  if (i8_status e = fp4_sizes(r->rows, r->K, r->fmt)) return e;
  if (r->rows > 0 && (!r->codes || !r->block_scales)) return I8_ERR_INVALID_ARG;
  if (!aligned16(r->codes) || !aligned16(r->block_scales) || !aligned4(r->row_scales)) return I8_ERR_ALIGNMENT;
  return I8_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

i8_status encode(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  static std::mutex mu;
  static EncodeTiledFn fn = nullptr;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!fn) {
      void* p = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !p)
        return I8_ERR_CUDA;
      fn = reinterpret_cast<EncodeTiledFn>(p);
    }
  }
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(map, type, rank, const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? I8_OK
             : I8_ERR_CUDA;
}

// The codes [rows, K / 2 bytes] in boxes of `box` rows by 128 bytes, swizzled;
// zeros outside.
i8_status encode_codes(CUtensorMap* map, const i8_fp4_rows& r, int box) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(r.K / 2), static_cast<cuuint64_t>(r.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(r.K / 2)};
  const cuuint32_t size[2] = {128, static_cast<cuuint32_t>(box)};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, r.codes, dims, strides, size, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The block scales, a tile of 128 rows by 256 elements a row of 8-byte words.
i8_status encode_scales(CUtensorMap* map, const i8_fp4_rows& r) {
  const cuuint64_t words = fp4_tile_bytes(r.fmt == I8_FP4_MX32 ? 32 : 16) / 8;
  const cuuint64_t dims[2] = {words, static_cast<cuuint64_t>((r.rows + 127) / 128) * fp4_deep(r.K)};
  const cuuint64_t strides[1] = {words * 8};
  const cuuint32_t size[2] = {static_cast<cuuint32_t>(words), 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, r.block_scales, dims, strides, size, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Clusters of lo .. hi of a kernel's CTAs that are resident at once: out[size].
// (For kernels with tensor memory the runtime counts one CTA an SM.  Two run where
// their shared memory, registers and tensor memory, `cols` columns each, fit: counted
// here.)
template <auto KERN>
i8_status resident_clusters(int dev, int sms, int threads, size_t smem, int cols, int lo, int hi,
                            int (&out)[kFp4MaxSplits + 1]) {
  static int cached[kMaxDevices][kFp4MaxSplits + 1] = {};
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (cached[dev][lo] == 0) {
    cudaFuncAttributes f;
    int room = 0, reserved = 0, regs = 0;
    if (cudaFuncGetAttributes(&f, KERN) != cudaSuccess ||
        cudaDeviceGetAttribute(&room, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&regs, cudaDevAttrMaxRegistersPerMultiprocessor, dev) != cudaSuccess)
      return I8_ERR_CUDA;
    const size_t block = (smem + f.sharedSizeBytes + reserved + 1023) / 1024 * 1024;
    const int per_sm = 2 * block <= static_cast<size_t>(room) && 2 * cols <= 512 && 2 * threads * ((f.numRegs + 7) / 8 * 8) <= regs ? 2 : 1;
    for (int size = lo; size <= hi; ++size) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(size * sms));
      cfg.blockDim = dim3(static_cast<unsigned>(threads));
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = static_cast<unsigned>(size);
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, KERN, &cfg) != cudaSuccess) n = 0;
      cached[dev][size] = n;
    }
    // two an SM: twice as many clusters, or as many as of half the size
    if (per_sm == 2)
      for (int size = hi; size >= lo; --size) cached[dev][size] = std::max(2 * cached[dev][size], cached[dev][std::max(lo, (size + 1) / 2)]);
    cudaGetLastError();
    if (cached[dev][lo] < 1) return I8_ERR_CUDA;
  }
  std::copy(cached[dev], cached[dev] + kFp4MaxSplits + 1, out);
  return I8_OK;
}

// K splits of the streaming kernel, by a model in tiles of K (0.2 us each): a CTA
// costs 10 besides its own, two on an SM slow each other down by 0.3, and CTAs that
// meet pay 2 and 0.03 for each other one and each sum of a token that they exchange.
// us measured (NV16) at 1, 2, 4, 8 splits:
//   1 token by 4096 x 11008   13.8  9.1  6.3  5.5
//   1 by 6144 x 4096           6.7  5.4  4.9  7.5 (two waves)
//   32 by 4096 x 4096          7.0  6.5  5.5  5.7
//   61 by 2080 x 5120          8.2  7.3  6.0  6.9 (seven splits)
//   128 by 4096 x 4096         8.0  8.2  7.9  12.1 (two waves)
int stream_splits(int tiles, int sums, int deep, int most, int sms, const int (&clusters)[kFp4MaxSplits + 1]) {
  int best = 1;
  double least = 0;
  for (int s = 1; s <= most && s <= deep; ++s) {
    const int each = (deep + s - 1) / s;
    if (clusters[s] < 1 || (deep + each - 1) / each != s) continue;  // no room, or a CTA without work
    if (g_opt.force_splits > 0 && s == std::min({g_opt.force_splits, most, deep})) return s;
    const int waves = (tiles + clusters[s] - 1) / clusters[s];
    const double shared = static_cast<int64_t>(tiles) * s > sms ? 1.3 : 1.0;
    const double cost = waves * (each * shared + 10.0) + (s > 1 ? 2.0 + 0.03 * sums * s : 0.0);
    if (s == 1 || cost < least) best = s, least = cost;
  }
  return best;
}

template <bool MX, int ACT>
i8_status launch_pair(Fp4GemmArgs& p, const i8_fp4_rows& t, const i8_fp4_rows* const (&w)[2], int dev, int sms,
                      cudaStream_t st) {
  constexpr bool GATED = ACT != kFp4Plain;
  using Cfg = Fp4PairCfg<MX, GATED>;
  constexpr auto kern = fp4_pair_kernel<MX, ACT>;
  if (i8_status e = allow_smem<kern>(dev, Cfg::SMEM)) return e;
  int clusters[kFp4MaxSplits + 1];
  if (i8_status e = resident_clusters<kern>(dev, sms, Cfg::THREADS, Cfg::SMEM, 512, 2, 2, clusters)) return e;
  CUtensorMap a, as, b[2], bs[2];
  if (i8_status e = encode_codes(&a, t, 128)) return e;
  if (i8_status e = encode_scales(&as, t)) return e;
  for (int k = 0; k < (GATED ? 2 : 1); ++k) {
    if (i8_status e = encode_codes(&b[k], *w[k], 128)) return e;
    if (i8_status e = encode_scales(&bs[k], *w[k])) return e;
  }
  if (!GATED) b[1] = b[0], bs[1] = bs[0];
  const int64_t tiles = static_cast<int64_t>((p.M + 255) / 256) * ((p.N + Cfg::TILE_N - 1) / Cfg::TILE_N);
  const int pairs = g_opt.max_ctas > 0 ? std::max(1, std::min(clusters[2], g_opt.max_ctas / 2)) : clusters[2];
  const dim3 grid(static_cast<unsigned>(2 * std::min<int64_t>(tiles, pairs)));
  return cuda_status(launch_pdl(kern, grid, dim3(Cfg::THREADS), Cfg::SMEM, st, a, b[0], b[1], as, bs[0], bs[1], p));
}

template <bool MX, int NT, int ACT, bool FUSED = false>
i8_status launch_stream(Fp4GemmArgs& p, const i8_fp4_rows& t, const i8_fp4_rows* const (&w)[2], int dev, int sms,
                        cudaStream_t st) {
  constexpr bool GATED = ACT != kFp4Plain;
  using Cfg = Fp4StreamCfg<MX, NT, GATED, FUSED>;
  constexpr auto kern = fp4_stream_kernel<MX, NT, ACT, FUSED>;
  if (i8_status e = allow_smem<kern>(dev, Cfg::SMEM)) return e;
  CUtensorMap m0, m1, mt;
  if (i8_status e = encode_codes(&m0, *w[0], 128)) return e;
  if (GATED) {
    if (i8_status e = encode_codes(&m1, *w[1], 128)) return e;
  } else {
    m1 = m0;
  }
  if (FUSED) mt = m0;
  else if (i8_status e = encode_codes(&mt, t, NT)) return e;
  int clusters[kFp4MaxSplits + 1];
  if (i8_status e = resident_clusters<kern>(dev, sms, Cfg::THREADS, Cfg::SMEM, Cfg::COLS, 1, Cfg::MAX_SPLITS, clusters)) return e;
  const int tiles = (p.N + 127) / 128 * ((p.M + NT - 1) / NT);
  const int best = stream_splits(tiles, NT * Cfg::WEIGHTS, p.deep, Cfg::MAX_SPLITS, sms, clusters);
  p.splits = best;
  p.deep_per_split = (p.deep + best - 1) / best;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + 127) / 128 * best), static_cast<unsigned>((p.M + NT - 1) / NT));
  cfg.blockDim = dim3(Cfg::THREADS);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeClusterDimension;
  attr[n].val.clusterDim.x = static_cast<unsigned>(best);
  attr[n].val.clusterDim.y = 1;
  attr[n].val.clusterDim.z = 1;
  ++n;
  if (g_opt.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(n);
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, m0, m1, mt, p));
}

// Whether pairs beat the streaming kernel at 128 tokens, both in us by a model of
// their waves.  Measured, stream / pair (NV16):
//   512 tokens by 4096 x 4096     8.9 / 10.8      gated, 128 by 11008 x 4096   11.5 / 17.7
//   1024 by 4096 x 4096          11.6 / 11.3      256                          21.1 / 18.4
//   2048 by 4096 x 4096          21.5 / 18.1      512 by 5640 x 2048           15.4 / 13.9
bool pair_is_faster(int M, int N, int deep, bool gated, int sms) {
  const int64_t ctas = static_cast<int64_t>((M + 127) / 128) * ((N + 127) / 128);
  const int64_t tiles = static_cast<int64_t>((M + 255) / 256) * ((N + (gated ? 127 : 255)) / (gated ? 128 : 256));
  const int64_t room = gated ? sms : 2 * static_cast<int64_t>(sms);
  const double stream = ctas <= sms && !gated ? 4.4 + 0.28 * deep : 1.5 + (ctas + room - 1) / room * (3.4 + 0.42 * deep);
  const double pair = 4.9 + (tiles + sms / 2 - 1) / (sms / 2) * std::max(0.4 * deep, 2.0);
  return pair < stream;
}

template <bool MX, int ACT>
i8_status launch_product(Fp4GemmArgs& p, const i8_fp4_rows& t, const i8_fp4_rows* const (&w)[2], int dev, int sms,
                         cudaStream_t st) {
  constexpr bool GATED = ACT != kFp4Plain;
  if (p.x) return launch_stream<MX, 16, ACT, true>(p, t, w, dev, sms, st);
  if (p.M <= 16) return launch_stream<MX, 16, ACT>(p, t, w, dev, sms, st);
  if (p.M <= 32) return launch_stream<MX, 32, ACT>(p, t, w, dev, sms, st);
  if (p.M <= 64) return launch_stream<MX, 64, ACT>(p, t, w, dev, sms, st);
  const bool pairs = g_opt.cta_pair == 0 ? p.M > 128 && pair_is_faster(p.M, p.N, p.deep, GATED, sms)
                                         : g_opt.cta_pair == 2 && p.M >= 256 && p.N >= 256;
  if (pairs) return launch_pair<MX, ACT>(p, t, w, dev, sms, st);
  return launch_stream<MX, 128, ACT>(p, t, w, dev, sms, st);
}

template <int ACT>
i8_status launch_format(Fp4GemmArgs& p, const i8_fp4_rows& t, const i8_fp4_rows* const (&w)[2], int dev, int sms,
                        cudaStream_t st) {
  return t.fmt == I8_FP4_MX32 ? launch_product<true, ACT>(p, t, w, dev, sms, st)
                              : launch_product<false, ACT>(p, t, w, dev, sms, st);
}

int64_t scale_bytes(const i8_fp4_rows* r) {
  return static_cast<int64_t>(i8_fp4_block_scale_bytes(r->rows, r->K, r->fmt));
}

i8_status check_product(const i8_fp4_rows* a, const i8_fp4_rows* w0, const i8_fp4_rows* w1, const void* b0,
                        const void* b1, const void* y, int64_t ldy) {
  if (i8_status e = check_rows(a)) return e;
  if (i8_status e = check_rows(w0)) return e;
  if (w1) {
    if (i8_status e = check_rows(w1)) return e;
    if (w1->rows != w0->rows || w1->K != w0->K || w1->fmt != w0->fmt) return I8_ERR_INVALID_ARG;
  }
  if (a->K != w0->K || a->fmt != w0->fmt) return I8_ERR_INVALID_ARG;
  if (ldy < w0->rows || (a->rows > 0 && w0->rows > 0 && !y)) return I8_ERR_INVALID_ARG;
  if (!aligned16(y) || ldy % 8 != 0 || !aligned16(b0) || !aligned16(b1)) return I8_ERR_ALIGNMENT;
  if (w0->rows % 8 != 0 || (a->rows + 127) / 128 > 65535 || w0->rows > INT32_MAX - 256) return I8_ERR_UNSUPPORTED;
  // other CTAs read the tokens and the weights while one writes its rows of y
  const Extent out{y, w0->rows * 2, a->rows, ldy * 2};
  for (const i8_fp4_rows* r : {a, w0, w1})
    if (r && (overlap(out, {r->codes, r->rows * (r->K / 2)}) || overlap(out, {r->block_scales, scale_bytes(r)}) ||
              overlap(out, {r->row_scales, r->rows * 4})))
      return I8_ERR_INVALID_ARG;
  return overlap(out, {b0, w0->rows * 2}) || overlap(out, {b1, w0->rows * 2}) ? I8_ERR_INVALID_ARG : I8_OK;
}

// Of checked operands.  x: null, or the tokens themselves (bf16, ldx apart), read in
// place of a's codes.
i8_status product(const i8_fp4_rows& a, const uint16_t* x, int64_t ldx, const i8_fp4_rows* w0, const i8_fp4_rows* w1,
                  const void* b0, const void* b1, int activation, void* y, int64_t ldy, cudaStream_t st) {
  if (a.rows == 0 || w0->rows == 0) return I8_OK;
  Fp4GemmArgs p{};
  p.w[0] = {static_cast<const uint8_t*>(w0->block_scales), w0->row_scales, static_cast<const uint16_t*>(b0)};
  if (w1) p.w[1] = {static_cast<const uint8_t*>(w1->block_scales), w1->row_scales, static_cast<const uint16_t*>(b1)};
  p.x = x;
  p.ldx = ldx;
  p.scales = static_cast<const uint8_t*>(a.block_scales);
  p.row_scales = a.row_scales;
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  p.M = static_cast<int>(a.rows);
  p.N = static_cast<int>(w0->rows);
  p.K = static_cast<int>(a.K);
  p.deep = fp4_deep(a.K);
  int dev, sms;
  if (i8_status e = current_device(&dev)) return e;
  if (i8_status e = device_sms(dev, &sms)) return e;
  const i8_fp4_rows* const w[2] = {w0, w1};
  if (!w1) return launch_format<kFp4Plain>(p, a, w, dev, sms, st);
  return activation == I8_GATE_SILU ? launch_format<kFp4Silu>(p, a, w, dev, sms, st)
                                    : launch_format<kFp4Gelu>(p, a, w, dev, sms, st);
}

// The tokens' rows in a workspace: codes, block scales, row scales.
struct TokenRows {
  i8_fp4_rows rows;
  size_t bytes;
  TokenRows(void* ws, int64_t M, int64_t K, int fmt) {
    const size_t codes = static_cast<size_t>(M) * (K / 2), scales = i8_fp4_block_scale_bytes(M, K, fmt);
    char* at = static_cast<char*>(ws);
    rows = {at, at + codes, fmt == I8_FP4_NV16 ? reinterpret_cast<float*>(at + codes + scales) : nullptr, M, K, fmt};
    bytes = codes + scales + (fmt == I8_FP4_NV16 ? static_cast<size_t>(M) * 4 : 0);
  }
};

i8_status linear(const void* x, int64_t M, int64_t K, int64_t ldx, const i8_fp4_rows* w0, const i8_fp4_rows* w1,
                 const void* b0, const void* b1, int activation, void* y, int64_t ldy, void* ws, size_t ws_bytes,
                 i8_stream_t stream) {
  if (i8_status e = check_rows(w0)) return e;
  if (K != w0->K) return I8_ERR_INVALID_ARG;
  if (i8_status e = fp4_sizes(M, K, w0->fmt)) return e;
  const TokenRows t(ws, M, K, w0->fmt);
  if (t.bytes > 0 && (!ws || ws_bytes < t.bytes)) return I8_ERR_WORKSPACE;
  if (!aligned16(ws)) return I8_ERR_ALIGNMENT;
  // what the product would refuse is refused before the tokens are written
  if (i8_status e = check_product(&t.rows, w0, w1, b0, b1, y, ldy)) return e;
  for (const i8_fp4_rows* r : {w0, w1})
    if (r && (overlap({ws, static_cast<int64_t>(t.bytes)}, {r->codes, r->rows * (r->K / 2)}) ||
              overlap({ws, static_cast<int64_t>(t.bytes)}, {r->block_scales, scale_bytes(r)}) ||
              overlap({ws, static_cast<int64_t>(t.bytes)}, {r->row_scales, r->rows * 4})))
      return I8_ERR_INVALID_ARG;
  for (const void* b : {b0, b1})
    if (overlap({ws, static_cast<int64_t>(t.bytes)}, {b, w0->rows * 2})) return I8_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // the fewest tokens are quantized by the product itself, unless y lies where x does:
  // other CTAs read x while one writes its channels of y
  if (M <= fp4_fused_tokens(w0->fmt == I8_FP4_MX32) && !overlap({x, K * 2, M, ldx * 2}, {y, ((M - 1) * ldy + w0->rows) * 2})) {
    if (i8_status e = check_quant(x, M, K, ldx, w0->fmt, t.rows.codes, t.rows.block_scales, t.rows.row_scales)) return e;
    return product(t.rows, static_cast<const uint16_t*>(x), ldx, w0, w1, b0, b1, activation, y, ldy, st);
  }
  if (i8_status e = i8_quant_rows_fp4(x, M, K, ldx, w0->fmt, const_cast<void*>(t.rows.codes),
                                      const_cast<void*>(t.rows.block_scales), const_cast<float*>(t.rows.row_scales), stream))
    return e;
  return product(t.rows, nullptr, 0, w0, w1, b0, b1, activation, y, ldy, st);
}

// ----------------------------------------------------------------- heads
// Memory of [tokens, heads] rows of `dim` bf16 elements.
struct HeadRows {
  const void* base;
  int64_t tokens, token, heads, head, dim;
};

// Whether the rows of two operands may share memory: by their whole ranges, or,
// with one stride between tokens that holds a token's heads, by the places in it.
bool heads_meet(const HeadRows& a, const HeadRows& b) {
  if (!a.base || !b.base || a.tokens <= 0 || a.heads <= 0 || b.heads <= 0) return false;
  auto span = [](const HeadRows& r) { return 2 * ((r.heads - 1) * r.head + r.dim); };
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
  const int64_t reach = (a.tokens - 1) * 2;
  if (d >= reach * a.token + span(a) || -d >= reach * b.token + span(b)) return false;
  if (a.tokens > 1 && a.token != b.token) return true;
  const int64_t period = a.tokens > 1 ? 2 * a.token : 0;
  if (period == 0 || span(a) > period || span(b) > period) return true;
  int64_t at = d % period;
  if (at < 0) at += period;
  return at < span(a) || period - at < span(b);
}

}  // namespace
}  // namespace i8

using namespace i8;

extern "C" {

size_t i8_fp4_block_scale_bytes(int64_t rows, int64_t K, int fmt) {
  I8_NVTX();
  if (fp4_sizes(rows, K, fmt) != I8_OK) return 0;
  return static_cast<size_t>((rows + 127) / 128) * fp4_deep(K) * fp4_tile_bytes(fmt == I8_FP4_MX32 ? 32 : 16);
}

i8_status i8_quant_rows_fp4(const void* x, int64_t rows, int64_t K, int64_t ldx, int fmt, void* codes,
                            void* block_scales, float* row_scales, i8_stream_t stream) {
  I8_NVTX();
  if (i8_status e = check_quant(x, rows, K, ldx, fmt, codes, block_scales, row_scales)) return e;
  if (rows == 0) return I8_OK;
  Fp4QuantArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(block_scales);
  a.row_scales = row_scales;
  a.K = static_cast<int>(K);
  a.deep = fp4_deep(K);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(fmt == I8_FP4_MX32 ? launch_quant<true, false>(a, rows, st) : launch_quant<false, false>(a, rows, st));
}

i8_status i8_add_rmsnorm_quant_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr,
                                   const void* weight, float eps, int fmt, void* codes, void* block_scales,
                                   float* row_scales, void* h, int64_t ldh, i8_stream_t stream) {
  I8_NVTX();
  if (i8_status e = fp4_sizes(M, K, fmt)) return e;
  if (ldx < K || (residual && ldr < K) || (h && ldh < K) || !(eps >= 0.0f && eps <= 3.0e38f)) return I8_ERR_INVALID_ARG;
  if (M > 0 && (!x || !codes || !block_scales || !row_scales)) return I8_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(block_scales) || !aligned4(row_scales) || ldx % 8 != 0 ||
      !aligned16(residual) || (residual && ldr % 8 != 0) || !aligned16(weight) || !aligned16(h) || (h && ldh % 8 != 0))
    return I8_ERR_ALIGNMENT;
  if (M == 0) return I8_OK;
  // a row's CTA writes its h when others have not read theirs, and a thread the
  // elements that it has read when others of the row have not read theirs
  const Extent to{h, K * 2, M, ldh * 2}, in{x, K * 2, M, ldx * 2}, other{residual, K * 2, M, ldr * 2}, gain{weight, K * 2};
  for (const Extent& from : {in, other})
    if (rows_cross(to, from) || rows_shifted(to, from)) return I8_ERR_INVALID_ARG;
  if (overlap(to, gain)) return I8_ERR_INVALID_ARG;
  const Extent out[] = {{codes, M * (K / 2)},
                        {block_scales, static_cast<int64_t>(i8_fp4_block_scale_bytes(M, K, fmt))},
                        {row_scales, M * 4}};
  for (const Extent& u : out) {
    if (overlap(in, u) || overlap(other, u) || overlap(to, u) || overlap(u, gain)) return I8_ERR_INVALID_ARG;
    for (const Extent& v : out)
      if (&u != &v && overlap(u, v)) return I8_ERR_INVALID_ARG;
  }
  Fp4QuantArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.res = static_cast<const uint16_t*>(residual);
  a.ldr = ldr;
  a.weight = static_cast<const uint16_t*>(weight);
  a.h = static_cast<uint16_t*>(h);
  a.ldh = ldh;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(block_scales);
  a.row_scales = row_scales;
  a.K = static_cast<int>(K);
  a.deep = fp4_deep(K);
  a.eps = eps;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(fmt == I8_FP4_MX32 ? launch_quant<true, true>(a, M, st) : launch_quant<false, true>(a, M, st));
}

i8_status i8_gemm_fp4_bias_bf16(const i8_fp4_rows* a, const i8_fp4_rows* w, const void* bias, void* y, int64_t ldy,
                                i8_stream_t stream) {
  I8_NVTX();
  if (i8_status e = check_product(a, w, nullptr, bias, nullptr, y, ldy)) return e;
  return product(*a, nullptr, 0, w, nullptr, bias, nullptr, 0, y, ldy, reinterpret_cast<cudaStream_t>(stream));
}

i8_status i8_gemm_fp4_gated_bf16(const i8_fp4_rows* a, const i8_fp4_rows* gate, const i8_fp4_rows* up,
                                 const void* gate_bias, const void* up_bias, int activation, void* y, int64_t ldy,
                                 i8_stream_t stream) {
  I8_NVTX();
  if (!up || (activation != I8_GATE_SILU && activation != I8_GATE_GELU)) return I8_ERR_INVALID_ARG;
  if (i8_status e = check_product(a, gate, up, gate_bias, up_bias, y, ldy)) return e;
  return product(*a, nullptr, 0, gate, up, gate_bias, up_bias, activation, y, ldy, reinterpret_cast<cudaStream_t>(stream));
}

size_t i8_linear_fp4_workspace_bytes(int64_t M, int64_t K, int fmt) {
  I8_NVTX();
  return fp4_sizes(M, K, fmt) == I8_OK ? TokenRows(nullptr, M, K, fmt).bytes : 0;
}

i8_status i8_linear_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, const i8_fp4_rows* w, const void* bias, void* y,
                        int64_t ldy, void* ws, size_t ws_bytes, i8_stream_t stream) {
  I8_NVTX();
  return linear(x, M, K, ldx, w, nullptr, bias, nullptr, 0, y, ldy, ws, ws_bytes, stream);
}

i8_status i8_gated_linear_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, const i8_fp4_rows* gate,
                              const i8_fp4_rows* up, const void* gate_bias, const void* up_bias, int activation, void* y,
                              int64_t ldy, void* ws, size_t ws_bytes, i8_stream_t stream) {
  I8_NVTX();
  if (!up || (activation != I8_GATE_SILU && activation != I8_GATE_GELU)) return I8_ERR_INVALID_ARG;
  return linear(x, M, K, ldx, gate, up, gate_bias, up_bias, activation, y, ldy, ws, ws_bytes, stream);
}

i8_status i8_heads_rmsnorm_rotate(const void* q, int64_t ldq_token, int64_t ldq_head, int64_t q_heads, const void* k,
                                  int64_t ldk_token, int64_t ldk_head, int64_t kv_heads, int64_t tokens,
                                  int64_t head_dim, const void* q_weight, const void* k_weight, float eps,
                                  const int32_t* positions, int64_t ld_positions, int64_t axes, const int32_t* sections,
                                  const float* inv_freq, int64_t rotary_dim, int interleaved, void* q_out,
                                  int64_t ldqo_token, int64_t ldqo_head, void* k_out, int64_t ldko_token,
                                  int64_t ldko_head, i8_stream_t stream) {
  I8_NVTX();
  if (tokens < 0 || head_dim <= 0 || q_heads < 0 || kv_heads < 0 || rotary_dim < 0 || rotary_dim > head_dim || axes < 1 ||
      axes > kRotateMaxAxes || !sections || !(eps >= 0.0f && eps <= 3.0e38f))
    return I8_ERR_INVALID_ARG;
  if (ldq_token < 0 || ldq_head < 0 || ldk_token < 0 || ldk_head < 0 || ldqo_token < 0 || ldqo_head < 0 ||
      ldko_token < 0 || ldko_head < 0 || (axes > 1 && ld_positions < tokens))
    return I8_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim > 512 || rotary_dim % 16 != 0 || tokens > INT32_MAX || q_heads + kv_heads > 32767)
    return I8_ERR_UNSUPPORTED;
  int64_t pairs = 0;
  for (int a = 0; a < axes; ++a) {
    if (sections[a] < 0 || sections[a] > rotary_dim / 2) return I8_ERR_INVALID_ARG;
    pairs += sections[a];
  }
  if (pairs != rotary_dim / 2) return I8_ERR_INVALID_ARG;
  if (tokens > 0 && ((q_heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)) ||
                     (rotary_dim > 0 && (!positions || !inv_freq))))
    return I8_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) ||
      !aligned16(k_weight) || !aligned4(positions) || !aligned4(inv_freq))
    return I8_ERR_ALIGNMENT;
  for (int64_t ld : {ldq_token, ldq_head, ldk_token, ldk_head, ldqo_token, ldqo_head, ldko_token, ldko_head})
    if (ld % 8 != 0) return I8_ERR_ALIGNMENT;
  if (tokens == 0 || q_heads + kv_heads == 0) return I8_OK;
  const HeadRows qi{q_heads ? q : nullptr, tokens, ldq_token, q_heads, ldq_head, head_dim};
  const HeadRows ki{kv_heads ? k : nullptr, tokens, ldk_token, kv_heads, ldk_head, head_dim};
  const HeadRows qo{q_heads ? q_out : nullptr, tokens, ldqo_token, q_heads, ldqo_head, head_dim};
  const HeadRows ko{kv_heads ? k_out : nullptr, tokens, ldko_token, kv_heads, ldko_head, head_dim};
  auto same = [](const HeadRows& a, const HeadRows& b) {
    return a.base == b.base && (a.tokens <= 1 || a.token == b.token) && (a.heads <= 1 || a.head == b.head);
  };
  // in place, or apart from everything that another CTA may still read
  if ((q_heads > 0 && rows_overlap(tokens, ldqo_token, q_heads, ldqo_head, head_dim)) ||
      (kv_heads > 0 && rows_overlap(tokens, ldko_token, kv_heads, ldko_head, head_dim)) || heads_meet(qo, ko) || heads_meet(qo, ki) ||
      heads_meet(ko, qi) || (heads_meet(qo, qi) && !same(qo, qi)) || (heads_meet(ko, ki) && !same(ko, ki)))
    return I8_ERR_INVALID_ARG;
  for (const HeadRows& r : {qo, ko})
    for (const Extent& v : {Extent{q_weight, head_dim * 2}, Extent{k_weight, head_dim * 2},
                            Extent{inv_freq, rotary_dim * 2}, Extent{positions, ((axes - 1) * ld_positions + tokens) * 4}}) {
      if (!r.base || !v.base || v.bytes <= 0) continue;
      const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(v.base) - reinterpret_cast<uintptr_t>(r.base));
      if (d < 2 * ((r.tokens - 1) * r.token + (r.heads - 1) * r.head + r.dim) && d + v.bytes > 0) return I8_ERR_INVALID_ARG;
    }
  RotateArgs p{};
  p.q = {static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), static_cast<const uint16_t*>(q_weight), ldq_token,
         ldq_head, ldqo_token, ldqo_head};
  p.k = {static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), static_cast<const uint16_t*>(k_weight), ldk_token,
         ldk_head, ldko_token, ldko_head};
  p.positions = positions;
  p.ld_pos = ld_positions;
  p.inv_freq = inv_freq;
  p.tokens = static_cast<int>(tokens);
  p.q_heads = static_cast<int>(q_heads);
  p.heads = static_cast<int>(q_heads + kv_heads);
  p.dim = static_cast<int>(head_dim);
  p.rotary = static_cast<int>(rotary_dim);
  p.interleaved = interleaved != 0;
  p.eps = eps;
  p.inv_dim = 1.0f / static_cast<float>(head_dim);
  int end = 0;
  for (int a = 0; a < kRotateMaxAxes; ++a) {
    if (a < axes) end += sections[a];
    p.section_end[a] = a < axes - 1 ? end : INT32_MAX;
  }
  while ((16 << p.lanes_log2) < head_dim) ++p.lanes_log2;
  p.step_tokens = (kRotateThreads >> p.lanes_log2) / p.heads;
  p.step_heads = (kRotateThreads >> p.lanes_log2) % p.heads;
  int dev, sms;
  if (i8_status e = current_device(&dev)) return e;
  if (i8_status e = device_sms(dev, &sms)) return e;
  p.kinds = q_weight || k_weight ? 2 : 1;
  // tokens a CTA: several rounds of its threads, but CTAs for every SM first
  const int64_t lanes = static_cast<int64_t>(p.heads) << p.lanes_log2;
  const size_t table = static_cast<size_t>(p.kinds) * ((p.dim + 15) / 16 * 8) * 4 * sizeof(float);
  p.per_cta = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({8 * kRotateThreads / lanes, tokens / (4 * static_cast<int64_t>(sms)), 8,
                            kRotateTable / static_cast<int64_t>(table)})));
  const size_t smem = p.per_cta * table;
  return cuda_status(launch_pdl(heads_rmsnorm_rotate_kernel, dim3(static_cast<unsigned>((tokens + p.per_cta - 1) / p.per_cta)),
                                dim3(kRotateThreads), smem, reinterpret_cast<cudaStream_t>(stream), p));
}

}  // extern "C"
