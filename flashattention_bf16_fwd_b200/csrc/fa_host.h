// fa_host.h - what the library's translation units share on the host: the
// checked per-device state, the tensor-map encoder and the launch helper.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <utility>

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

}  // namespace fa
