// gate_internal.cuh - helpers shared by the learned gate's kernels.
#pragma once

#include "expert_internal.cuh"
#include "gmm_gate.h"

namespace gmm {
namespace gate {

constexpr int kMaxTop = 8;       // entries of a gate's row
constexpr int kMaxTeacher = 64;  // entries of a teacher's row

// Order of floats as unsigned numbers: -0 and 0 are one, every NaN is the largest.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kOrderedNegInf = 0x007fffffu;

struct MaxOp {
  template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct SumOp {
  template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

template <typename T, typename Op>
__device__ __forceinline__ T warp_reduce(T v, Op op) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Over the block, the same for every thread; `part`: 32 words of T.
template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, T none, Op op, T* part) {
  v = warp_reduce(v, op);
  __syncthreads();  // the last reduction's words are read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_reduce(lane < (int)(blockDim.x >> 5) ? part[lane] : none, op);
}

}  // namespace gate
}  // namespace gmm
