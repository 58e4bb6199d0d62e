// Host helpers of the calls that take no workspace: pointer checks and the launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gtr.h"

namespace gtr {

inline bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes from the first to behind the last element of `rows` rows of `width` elements, `ld` apart.
inline size_t span_bytes(long long rows, long long ld, long long width, int es) {
  return rows <= 0 ? 0 : (size_t)((rows - 1) * ld + width) * (size_t)es;
}

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// A runtime call that failed.  The runtime also keeps the error for whoever asks for the last one:
// it is taken out, or the next call that asks would report it as its own.
inline gtr_status_t cuda_failed() {
  (void)cudaGetLastError();
  return GTR_ERR_CUDA;
}

// Launch with programmatic stream serialisation: the kernel may start while its predecessor
// in the stream drains, and waits for it (griddepcontrol.wait) before its first access to
// global memory.  These kernels do not let their own successors start early
// (griddepcontrol.launch_dependents): blocks that wait on the SMs take the places of blocks that
// would run, and are packed on the SMs that have room first (one token's convolution 3.3 us with
// it, 2.3 us without; a norm of 1600 rows 3.6 and 3.0 us).  Every thread of such a kernel executes that wait, also those that then
// have nothing to do: a kernel that ended without it could end before its predecessor, and
// its successor would wait for the wrong one.
template <typename... KArgs, typename... Args>
gtr_status_t launch_serial(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...) == cudaSuccess ? GTR_OK
                                                                                         : cuda_failed();
}

}  // namespace gtr
