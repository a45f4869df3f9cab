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

}  // namespace moe_fp4
