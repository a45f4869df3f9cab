// Host-side helpers shared by the entry points' translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe_fp4 {

// Record e for moe_fp4_last_cuda_error and return MOE_FP4_ECUDA (capi.cu).
int report_cuda_error(cudaError_t e);

// 2-D tensor map over a byte matrix [rows][inner] with `stride` bytes between
// rows, boxes of box_rows x 128 bytes, 128-byte swizzle, zero-filled outside
// (prefill.cu).  Encoded anew on every call.
CUresult encode_u8_map_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t stride,
                          uint32_t box_rows);

// SM count of the current device.
inline cudaError_t current_device_sms(int* sms) {
  static int cache[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && cache[dev] > 0) {
    *sms = cache[dev];
    return cudaSuccess;
  }
  int v = 0;
  e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64) cache[dev] = v;
  *sms = v;
  return cudaSuccess;
}

// Allow `kern` `bytes` of dynamic shared memory on the current device (once
// per kernel and device).
template <class Kern>
cudaError_t allow_smem(Kern kern, size_t bytes, bool (&seen)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && seen[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) seen[dev] = true;
  return e;
}

// A launch in plain stream order, or (`dependent`) with programmatic dependent
// launch: the kernel may become resident while its predecessor on the stream
// finishes; it waits for that one's completion (griddepcontrol.wait) before it
// touches global memory, and lets its own successor in only after that wait,
// so that no kernel ever runs beside one two launches before it.  The status
// is the launch's own: cudaGetLastError would also report, and clear, an
// error that an earlier call has reported already.
template <class Kern, class... Args>
cudaError_t launch_smem(Kern kern, unsigned grid, unsigned threads, size_t smem, bool dependent, cudaStream_t st,
                        const Args&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = at;
  c.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, args...);
}

template <class Kern, class... Args>
cudaError_t launch_dependent_smem(Kern kern, unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                                  const Args&... args) {
  return launch_smem(kern, grid, threads, smem, true, st, args...);
}

template <class Kern, class... Args>
cudaError_t launch_dependent(Kern kern, unsigned grid, unsigned threads, cudaStream_t st, const Args&... args) {
  return launch_dependent_smem(kern, grid, threads, 0, st, args...);
}

}  // namespace moe_fp4
