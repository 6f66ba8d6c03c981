// host.h -- what the library's two translation units share on the host: the
// process-wide options, the NVTX scope of an ABI call, small argument checks
// and the dependent launch.
#pragma once
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>

#include "../../include/i8.h"

namespace i8 {

// Process-wide tuning knobs (i8_set_option).
struct Options {
  int chunk_k = 1024;      // K per exact fp32 chunk (multiple of 64, <= 1024)
  int force_splits = 0;    // 0 = table
  int max_ctas = 0;        // 0 = all SMs
  int force_bn = 0;        // 0 = table, else 128 or 256
  int quant_vpl = 6;       // max 16-byte vectors per lane in the quantizer
  int cta_pair = 0;        // 0 = table, 1 = never, 2 = whenever the shape allows
  int skinny_max_m = 16;   // token counts up to this use the weight-streaming kernel (0 = off)
  int pdl = 1;             // launch with programmatic stream serialization
  int quant_rows = 0;      // quantizer rows per CTA (0 = by shape)
  int stream_k = 1;        // CTA-pair stream-K: 0 never, 1 by the table, 2 whenever pairs idle
  int nvtx = 0;            // NVTX range around every ABI call
  int pair_stage_k = 0;    // K per fp16 stage of the int8-code pair kernel: 0 (table) / 64 / 128
  int raster = 0;          // tile order: 0 table, 1 M blocks fastest, 2 N blocks fastest
};
extern Options g_opt;      // defined in i8_api.cu

// NVTX range for the lifetime of one ABI call (when I8_OPT_NVTX is on).
struct NvtxScope {
  bool on;
  explicit NvtxScope(const char* name) : on(g_opt.nvtx != 0) {
    if (on) nvtxRangePushA(name);
  }
  ~NvtxScope() {
    if (on) nvtxRangePop();
  }
};
#define I8_NVTX() NvtxScope i8_nvtx_scope_(__func__)

inline i8_status cuda_status(cudaError_t e) { return e == cudaSuccess ? I8_OK : I8_ERR_CUDA; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Launch with programmatic stream serialization (unless switched off): the
// kernel may be scheduled while the previous kernel of the stream drains.
// Every kernel launched this way calls pdl_wait() before it touches global
// memory, so the stream order of memory effects is unchanged.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g_opt.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Reads and clears the status word of the current device that the serving
// operators' kernels record into (each translation unit has a word of its
// own; serving_api.cu defines this).
cudaError_t take_serving_status(unsigned int* word);

}  // namespace i8
