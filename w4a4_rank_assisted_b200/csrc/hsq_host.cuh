// hsq_host.cuh -- host helpers that the library's translation units share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "hsq_device.cuh"

#ifndef HSQ_PDL
#define HSQ_PDL 1  // launch with programmatic stream serialization (see grid_dep_wait)
#endif

namespace {

// Launch `kernel` so that it may start while the preceding kernel in the stream
// is still running; the kernel itself waits (grid_dep_wait) before touching
// memory that kernel may write.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(bool allow, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = (HSQ_PDL && allow) ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether the byte ranges [a, a + na) and [b, b + nb) meet.
inline bool ranges_meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline int device_sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  static int cache[64] = {0};
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

// Reads and clears this translation unit's status word on the current device.
inline cudaError_t take_status(unsigned* v) {
  cudaError_t e = cudaMemcpyFromSymbol(v, hsq::g_status, sizeof(*v));
  const unsigned zero = 0;
  if (e == cudaSuccess && *v) e = cudaMemcpyToSymbol(hsq::g_status, &zero, sizeof(zero));
  return e;
}

}  // namespace

namespace hsq {
// hsq_heads.cu's status word, read and cleared.
cudaError_t take_heads_status(unsigned* v);
}  // namespace hsq
