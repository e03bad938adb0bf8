// fl_host.h — host helpers shared by the library's translation units: the thread-local
// error text, launch checks, tensor maps and the programmatic-dependent-launch wrapper.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/fused_linear.h"

namespace fl {
namespace host {

// Record a message for fl_last_error and return `st`.
fl_status fail(fl_status st, const char* fmt, ...);
// Forget the last failure's message (first statement of every entry point).
void clear_error();
// cudaGetLastError after a launch; with FL_SYNC_EACH_LAUNCH=1 also a synchronise.
fl_status after_launch(cudaStream_t s, const char* what);
// 2-D row-major tensor map: `inner` contiguous elements per row, `outer` rows, row pitch in
// bytes; a 128-byte (box of 128 bytes a row) or 64-byte swizzle.
fl_status make_map(CUtensorMap* m, const void* base, int dt, uint64_t inner, uint64_t outer, uint64_t pitch_bytes,
                   uint32_t box_inner, uint32_t box_outer, bool swizzle64 = false);

inline int esize(int dt) { return dt == FL_F32 ? 4 : 2; }
inline bool is_dtype(int dt) { return dt == FL_F16 || dt == FL_BF16 || dt == FL_F32; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// Launch with programmatic dependent launch allowed, with `smem` bytes of dynamic shared memory.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_smem(void (*kern)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                                   Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_b(void (*kern)(KArgs...), dim3 grid, unsigned block, cudaStream_t s, Args... args) {
  return launch_pdl_smem(kern, grid, block, 0, s, args...);
}

}  // namespace host
}  // namespace fl

#define FL_CUDA(call)                                                                                          \
  do {                                                                                                         \
    cudaError_t e_ = (call);                                                                                   \
    if (e_ != cudaSuccess) return fl::host::fail(FL_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_));         \
  } while (0)
