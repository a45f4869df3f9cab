// The rounded steps of fp8_quant.cuh against the IEEE operations, counted on
// the GPU for test_rounding_gpu.py.
#include "fp8_quant.cuh"

using namespace moe_fp4;

namespace {

__device__ float value(int exponent, uint32_t significand) {  // 2^exponent <= v < 2^(exponent + 1)
  return __uint_as_float(((uint32_t)(127 + exponent) << 23) | significand);
}

__device__ uint32_t mixed(uint32_t x) {  // a fixed scramble of 32 bits
  x = (x ^ (x >> 16)) * 0x7feb352du;
  x = (x ^ (x >> 15)) * 0x846ca68bu;
  return x ^ (x >> 16);
}

__device__ bool same(float a, float b) { return __float_as_uint(a) == __float_as_uint(b); }

__global__ void reciprocals_of_all(int exponent, unsigned long long* bad) {
  unsigned long long n = 0;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < 1u << 23; i += gridDim.x * blockDim.x) {
    const float s = value(exponent, i), want = __frcp_rn(s);
    const float2 pair = reciprocals(both(-s));
    n += !same(recip_rn(s), want) || !same(pair.x, want) || !same(pair.y, want);
  }
  if (n) atomicAdd(bad, n);
}

__global__ void scales_of_all(int exponent, unsigned long long* bad) {
  unsigned long long n = 0;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < 1u << 23; i += gridDim.x * blockDim.x) {
    const float a = value(exponent, i);
    n += !same(block_scale(a), __fdiv_rn(a, 448.f));
  }
  if (n) atomicAdd(bad, n);
}

// v / s for s of every significand from `first`, and `each` v beside it:
// scrambled ones (kind 0), BF16 ones (kind 1), or those next to s, up to it
// (kind 2).
__global__ void quotients_of(int kind, uint32_t first, uint32_t each, int ev, int es, unsigned long long* bad) {
  unsigned long long n = 0;
  const uint32_t many = (1u << 23) - first;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < many; i += gridDim.x * blockDim.x) {
    const uint32_t k = first + i;
    const float s = value(es, k);
    const float2 y = both(reciprocals(both(-s)).x);
    for (uint32_t j = 0; j < each; ++j) {
      const uint32_t sv = kind == 0   ? mixed(k * each + j) & 0x7fffffu
                          : kind == 1 ? (j & 127u) << 16
                                      : (k >= j ? k - j : k);
      const float v = value(ev, sv);
      const float2 q = quotients(make_float2(v, -v), both(-s), y);
      const float want = __fdiv_rn(v, s);
      n += !same(q.x, want) || !same(q.y, -want);
    }
  }
  if (n) atomicAdd(bad, n);
}

// Runs one count to its end; (unsigned long long)-1 on a CUDA error.
template <class Launch>
unsigned long long count(Launch launch) {
  unsigned long long *bad = nullptr, n = ~0ull;
  if (cudaMalloc(&bad, sizeof(n)) != cudaSuccess) return n;
  cudaMemset(bad, 0, sizeof(n));
  launch(bad);
  if (cudaGetLastError() != cudaSuccess || cudaMemcpy(&n, bad, sizeof(n), cudaMemcpyDeviceToHost) != cudaSuccess) n = ~0ull;
  cudaFree(bad);
  return n;
}

}  // namespace

extern "C" unsigned long long count_reciprocals(int exponent) {
  return count([&](unsigned long long* bad) { reciprocals_of_all<<<1024, 256>>>(exponent, bad); });
}
extern "C" unsigned long long count_scales(int exponent) {
  return count([&](unsigned long long* bad) { scales_of_all<<<1024, 256>>>(exponent, bad); });
}
extern "C" unsigned long long count_quotients(int kind, unsigned first, unsigned each, int ev, int es) {
  return count([&](unsigned long long* bad) { quotients_of<<<1024, 256>>>(kind, first, each, ev, es, bad); });
}
