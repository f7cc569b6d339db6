// expert_internal.cuh - helpers shared by the local-expert kernels.
#pragma once

#include <stdio.h>

#include <atomic>

#include "gmm_experts.h"
#include "gmm_internal.cuh"

namespace gmm {

inline gmm_status launched() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return GMM_OK;
  fprintf(stderr, "libgmm: CUDA error %s\n", cudaGetErrorString(e));
  return GMM_ERR_CUDA;
}

// Lets `kernel` use `bytes` of dynamic shared memory on the current device;
// `done` (one for each kernel, static) holds the devices that have it already.
inline bool allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// Whether each address is a multiple of `bytes` (NULL is).
template <typename... P>
inline bool aligned(size_t bytes, const P*... p) {
  return ((... | (uintptr_t)p) & (bytes - 1)) == 0;
}

inline bool dtype_ok(int t) { return t >= GMM_F32 && t <= GMM_BF16; }
inline int dtype_size(int t) { return t == GMM_F32 ? 4 : 2; }

template <int XT> struct Elem;
template <> struct Elem<GMM_F32> { using T = float; };
template <> struct Elem<GMM_F16> { using T = __half; };
template <> struct Elem<GMM_BF16> { using T = __nv_bfloat16; };

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Exclusive prefix over a block of 1024 threads; wsum: 32 words.
__device__ __forceinline__ uint32_t block_exclusive_1024(uint32_t v, uint32_t* wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const uint32_t t = wsum[lane];
    uint32_t ti = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += u;
    }
    wsum[lane] = ti - t;
  }
  __syncthreads();
  return wsum[warp] + incl - v;
}

}  // namespace gmm
