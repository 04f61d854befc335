// fa_host.h - what the library's translation units share on the host: the
// checked per-device state, the tensor-map encoder and the launch helper.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/fa_b200.h"
#include "fa_fwd.cuh"

namespace fa {

// Status of the current device (FA_OK, FA_ERR_DEVICE or FA_ERR_BUILD), its
// number of SMs and the device address of the library's error flag.
int host_device(int* num_sms, int** dev_error);

// cuTensorMapEncodeTiled, or nullptr where the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 encoder();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every kernel is launched with programmatic stream serialisation: it may be
// scheduled while the previous kernel in the stream drains, runs its set-up
// (barriers, TMEM, descriptor prefetch), and waits in grid_dep_wait() before
// it touches global memory.
constexpr int kProgrammaticLaunch = 1;

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                   Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline int check_common(int B, int H, int N, int d, int causal, float scale) {
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B < 1 || H < 1 || N < 1) return FA_ERR_SHAPE;
  const long long total = (long long)B * H * N * d;
  if (total >= (1ll << 31)) return FA_ERR_SHAPE;
  if (causal != 0 && causal != 1) return FA_ERR_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_ARG;
  return FA_OK;
}

// H query heads share Hkv key/value heads (H == Hkv: ordinary attention).
inline int check_heads(int H, int Hkv) { return (Hkv >= 1 && Hkv <= H && H % Hkv == 0) ? FA_OK : FA_ERR_SHAPE; }

// A [BH, N, D] bf16 tensor seen as 3-D (d, n, bh); boxes of 64 x box_rows x 1
// (128 for the loads the tcgen05 descriptors read, 32 for the forward's O
// stores, one per warp) with the 128-byte swizzle.  Loads read 0 past N; stores
// drop rows past N.
inline bool make_map(CUtensorMap* map, const void* base, int BH, int N, int D,
              CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, unsigned box_rows = 128) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(N), cuuint64_t(BH)};
  cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(N) * D * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The FP32 dQ accumulator [BH, N, D] as 3-D (d, n, bh) with 32 x 32 boxes and
// the 128-byte swizzle, for TMA reduce-add.
inline bool make_map_dq(CUtensorMap* map, const void* base, int BH, int N, int D) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(N), cuuint64_t(BH)};
  cuuint64_t strides[2] = {cuuint64_t(D) * 4, cuuint64_t(N) * D * 4};
  cuuint32_t box[3] = {32, 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename E>
constexpr CUtensorMapDataType map_type() {
  return E::kMmaFmt == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Shift added to m on repeated-max rows (base-2 units): maps a maximum to 1 - 2^-8.
const double kDeltaLog2 = -std::log2(1.0 - 1.0 / 256.0);
// The same for fp16 P_bar: maps a maximum to 1 - 2^-11.
const double kDeltaLog2F16 = -std::log2(1.0 - 1.0 / 2048.0);

// The parameters of a fix_mode.
inline void set_fix(FwdParams& p, int fix_mode, bool f16) {
  // shift on repeated-max rows per fix_mode, in base-2 units: 1 and 5 map the
  // maxima to the largest value below 1 of the P_bar format (1 - 2^-8 in bf16,
  // 1 - 2^-11 in fp16), 2 to 0.5, 3 to exp(-1/16); 0 and 4 keep the plain shift
  const double delta = (fix_mode == 1 || fix_mode == 5) ? (f16 ? kDeltaLog2F16 : kDeltaLog2)
                       : fix_mode == 2                  ? 1.0
                       : fix_mode == 3                  ? 1.4426950408889634 / 16.0
                                                        : 0.0;
  p.delta_log2 = float(delta);
  p.fix_factor = float(std::exp2(-delta));
  p.fix = (fix_mode == 1 || fix_mode == 2 || fix_mode == 3 || fix_mode == 5) ? 1 : 0;
  p.self_norm = (fix_mode == 4) ? 1 : 0;
  p.near = (fix_mode == 5) ? 1 : 0;
}

}  // namespace fa
