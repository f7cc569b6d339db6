// layer_norm.cu - layer norm of rows, and its gradients.
//
//   h = (x - mean) rstd,  y = w h + b
//   dx = (g - mean(g) - h mean(g h)) rstd,  g = w dy;  dw = sum dy h,  db = sum dy
//
// A block takes a row at a time; column d belongs to thread d mod 256 of every
// block, so a block's sums over its rows need no atomics.
#include "gate_internal.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 304;
constexpr int kMaxD = 32768;

template <typename T>
__device__ __forceinline__ void row_stats(const T* x, int D, float eps, float* part, float& mean,
                                          float& rstd) {
  float s = 0.f;
  for (int d = threadIdx.x; d < D; d += kThreads) s += to_f(x[d]);
  mean = block_reduce(s, 0.f, SumOp(), part) / D;
  float a = 0.f, b = 0.f;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    const float v = to_f(x[d]) - mean;
    a += v;
    b += v * v;
  }
  a = block_reduce(a, 0.f, SumOp(), part) / D;  // what rounding left of the mean
  b = block_reduce(b, 0.f, SumOp(), part) / D;
  mean += a;
  rstd = rsqrtf(fmaxf(b - a * a, 0.f) + eps);
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads)
norm_kernel(const T* __restrict__ X, int64_t N, int D, float eps, const W* __restrict__ weight,
            const W* __restrict__ bias, T* __restrict__ Y) {
  __shared__ float part[32];
  for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const T* x = X + n * D;
    float mean, rstd;
    row_stats(x, D, eps, part, mean, rstd);
    for (int d = threadIdx.x; d < D; d += kThreads) {
      const float w = weight ? to_f(weight[d]) : 1.f, b = bias ? to_f(bias[d]) : 0.f;
      Y[n * D + d] = from_f<T>(fmaf((to_f(x[d]) - mean) * rstd, w, b));
    }
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads)
norm_grad_kernel(const T* __restrict__ dY, const T* __restrict__ X, int64_t N, int D, float eps,
                 const W* __restrict__ weight, T* __restrict__ dX, float* __restrict__ sums) {
  __shared__ float part[32];
  float* dw = sums ? sums + (size_t)blockIdx.x * 2 * D : nullptr;
  if (sums)
    for (int d = threadIdx.x; d < 2 * D; d += kThreads) dw[d] = 0.f;
  __syncthreads();
  for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const T* x = X + n * D;
    const T* dy = dY + n * D;
    float mean, rstd;
    row_stats(x, D, eps, part, mean, rstd);
    float a = 0.f, b = 0.f;
    for (int d = threadIdx.x; d < D; d += kThreads) {
      const float h = (to_f(x[d]) - mean) * rstd, v = to_f(dy[d]);
      const float g = v * (weight ? to_f(weight[d]) : 1.f);
      a += g;
      b += g * h;
      if (sums) {
        dw[d] += v * h;
        dw[D + d] += v;
      }
    }
    a = block_reduce(a, 0.f, SumOp(), part) / D;
    b = block_reduce(b, 0.f, SumOp(), part) / D;
    if (dX)
      for (int d = threadIdx.x; d < D; d += kThreads) {
        const float h = (to_f(x[d]) - mean) * rstd;
        const float g = to_f(dy[d]) * (weight ? to_f(weight[d]) : 1.f);
        dX[n * D + d] = from_f<T>((g - a - h * b) * rstd);
      }
  }
}

template <typename W>
__global__ void __launch_bounds__(kThreads)
norm_finish_kernel(const float* __restrict__ sums, int blocks, int D, W* __restrict__ dweight,
                   W* __restrict__ dbias) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= 2 * D) return;
  double s = 0.0;
  for (int b = 0; b < blocks; ++b) s += sums[(size_t)b * 2 * D + i];
  if (i < D) dweight[i] = from_f<W>((float)s);
  else dbias[i - D] = from_f<W>((float)s);
}

bool norm_ok(int xdtype, int64_t N, int D, double eps, int wdtype) {
  return dtype_ok(xdtype) && (wdtype == xdtype || wdtype == GMM_F32) && N >= 0 && N <= INT32_MAX &&
         D >= 1 && eps >= 0.0 && eps < INFINITY;
}
int blocks_for(int64_t N) { return (int)(N < kMaxBlocks ? N : kMaxBlocks); }

}  // namespace
}  // namespace gmm

using namespace gmm;

#define BY_TYPES(CALL)                                              \
  if (xdtype == GMM_F32) CALL(float, float);                        \
  else if (xdtype == GMM_F16 && wdtype == GMM_F32) CALL(__half, float); \
  else if (xdtype == GMM_F16) CALL(__half, __half);                 \
  else if (wdtype == GMM_F32) CALL(__nv_bfloat16, float);           \
  else CALL(__nv_bfloat16, __nv_bfloat16);

extern "C" {

gmm_status gmm_layer_norm(const void* X, gmm_dtype xdtype, int64_t N, int D, double eps,
                          const void* weight, const void* bias, gmm_dtype wdtype, void* Y,
                          void* stream) {
  if (!norm_ok(xdtype, N, D, eps, wdtype)) return GMM_ERR_INVALID_ARG;
  if (D > kMaxD) return GMM_ERR_UNSUPPORTED;
  if (((uintptr_t)X | (uintptr_t)Y) % dtype_size(xdtype) ||
      ((uintptr_t)weight | (uintptr_t)bias) % dtype_size(wdtype))
    return GMM_ERR_INVALID_ARG;
  if (N == 0) return GMM_OK;
  if (!X || !Y) return GMM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope p("norm_kernel", s);
  const int b = (int)(N < 8 * 152 ? N : 8 * 152);
#define CALL(T, W) norm_kernel<T, W><<<b, kThreads, 0, s>>>((const T*)X, N, D, (float)eps, (const W*)weight, (const W*)bias, (T*)Y)
  BY_TYPES(CALL)
#undef CALL
  return launched();
}

size_t gmm_layer_norm_ws_bytes(int D) {
  return D >= 1 && D <= kMaxD ? align_up(sizeof(float) * 2 * (size_t)D * kMaxBlocks) : 0;
}

gmm_status gmm_layer_norm_grad(const void* dY, const void* X, gmm_dtype xdtype, int64_t N, int D,
                               double eps, const void* weight, gmm_dtype wdtype, void* dX,
                               void* dweight, void* dbias, void* ws, size_t ws_bytes, void* stream) {
  if (!norm_ok(xdtype, N, D, eps, wdtype)) return GMM_ERR_INVALID_ARG;
  if (D > kMaxD) return GMM_ERR_UNSUPPORTED;
  if (!dweight != !dbias) return GMM_ERR_INVALID_ARG;
  if (((uintptr_t)X | (uintptr_t)dY | (uintptr_t)dX) % dtype_size(xdtype) ||
      ((uintptr_t)weight | (uintptr_t)dweight | (uintptr_t)dbias) % dtype_size(wdtype))
    return GMM_ERR_INVALID_ARG;
  if (N > 0 && (!X || !dY)) return GMM_ERR_INVALID_ARG;
  if (dweight) {
    if (!ws || !aligned(256, (char*)ws)) return GMM_ERR_INVALID_ARG;
    if (ws_bytes < gmm_layer_norm_ws_bytes(D)) return GMM_ERR_WORKSPACE;
  }
  if ((N == 0 || !dX) && !dweight) return GMM_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const int b = blocks_for(N);
  if (N > 0) {
    ProfScope p("norm_grad_kernel", s);
#define CALL(T, W) norm_grad_kernel<T, W><<<b, kThreads, 0, s>>>((const T*)dY, (const T*)X, N, D, (float)eps, (const W*)weight, (T*)dX, dweight ? (float*)ws : nullptr)
    BY_TYPES(CALL)
#undef CALL
  }
  if (dweight) {
    ProfScope p("norm_finish_kernel", s);
#define CALL(T, W) norm_finish_kernel<W><<<(2 * D + kThreads - 1) / kThreads, kThreads, 0, s>>>((const float*)ws, b, D, (W*)dweight, (W*)dbias)
    BY_TYPES(CALL)
#undef CALL
  }
  return launched();
}

}  // extern "C"
