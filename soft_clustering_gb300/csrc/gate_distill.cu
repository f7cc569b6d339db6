// gate_distill.cu - distillation from a teacher's top entries.
//
//   row_n = w T^2 sum_t q_t (log q_t - log p[ids_t]),  loss = scale sum_n row_n
//   dL    = scale w T (p - q)
//
// A block takes a row at a time: the largest logit, the sum, the gradient; the
// few entries of the teacher are put right after the row is written.
#include "gate_internal.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 8 * 152;

template <typename T>
__global__ void __launch_bounds__(kThreads)
distill_kernel(const T* __restrict__ L, int64_t N, int K, int m, int gammas, int add, float temp,
               float scale, const int32_t* __restrict__ ids,
               const float* __restrict__ values, const float* __restrict__ weights,
               float* __restrict__ rows, double* __restrict__ part, T* __restrict__ dL) {
  __shared__ float partf[32];
  __shared__ float q_s[kMaxTeacher];
  __shared__ int id_s[kMaxTeacher];
  const float inv = 1.f / temp;
  double total = 0.0;
  for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const T* x = L + n * K;
    const float w = weights ? weights[n] : 1.f;
    // the teacher's entries, one a thread
    int id = -1;
    float u = -INFINITY;
    if (threadIdx.x < m) {
      id = ids[n * m + threadIdx.x];
      if (id < 0 || id >= K) id = -1;
      if (id >= 0) {
        const float v = values[n * m + threadIdx.x];
        u = (gammas ? logf(v) : v) * inv;
        if (u == -INFINITY) id = -1;
      }
    }
    const float umax = unordered(block_reduce(ordered(u), 0u, MaxOp(), (uint32_t*)partf));
    if (w == 0.f || umax == -INFINITY) {
      if (threadIdx.x == 0) rows[n] = 0.f;
      if (dL && !add)
        for (int k = threadIdx.x; k < K; k += kThreads) dL[n * K + k] = from_f<T>(0.f);
      continue;
    }
    float q = id >= 0 ? expf(u - umax) : 0.f;
    const float qsum = block_reduce(q, 0.f, SumOp(), partf);
    q /= qsum;
    float top = -INFINITY;
    for (int k = threadIdx.x; k < K; k += kThreads) {
      const float v = to_f(x[k]);
      top = v > top || isnan(v) ? v : top;
    }
    top = unordered(block_reduce(ordered(top), 0u, MaxOp(), (uint32_t*)partf));
    const bool none = top == -INFINITY;
    float sum = 0.f;
    if (!none)
      for (int k = threadIdx.x; k < K; k += kThreads) sum += expf((to_f(x[k]) - top) * inv);
    sum = block_reduce(sum, 0.f, SumOp(), partf);
    float term = 0.f;
    if (id >= 0 && q != 0.f) term = q * ((u - umax) - (to_f(x[id]) - top) * inv);
    term = block_reduce(term, 0.f, SumOp(), partf);
    float row = w * temp * temp * (term - logf(qsum) + logf(sum));
    if (none) row = w * INFINITY;
    if (threadIdx.x == 0) rows[n] = row;
    total += row;
    if (!dL) continue;
    if (threadIdx.x < m) q_s[threadIdx.x] = q, id_s[threadIdx.x] = id;
    T* d = dL + n * K;
    const float c = scale * w * temp;
    auto base = [&](int k) { return none ? 0.f : expf((to_f(x[k]) - top) * inv) / sum; };
    // every element is written by the thread that read it: the teacher's ones
    // with their share
    __syncthreads();
    for (int k = threadIdx.x; k < K; k += kThreads) {
      float v = base(k);
      for (int t = 0; t < m; ++t)
        if (id_s[t] == k) v -= q_s[t];
      v *= c;
      if (add) v += to_f(d[k]);
      d[k] = from_f<T>(v);
    }
  }
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

// The blocks' sums in order, in 64 bits.
__global__ void __launch_bounds__(kThreads)
distill_finish_kernel(const double* __restrict__ part, int blocks, double scale,
                      float* __restrict__ loss) {
  __shared__ double partd[32];
  double s = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kThreads) s += part[b];
  s = block_reduce(s, 0.0, SumOp(), partd);
  if (threadIdx.x == 0) *loss = (float)(s * scale);
}

}  // namespace
}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_distill_ws_bytes(void) { return align_up(sizeof(double) * kMaxBlocks); }

gmm_status gmm_distill(const void* L, gmm_dtype xdtype, int64_t N, int K, int m, int kind, int flags,
                       double temperature, double scale, const int32_t* ids, const float* values,
                       const float* weights, float* rows, float* loss, void* dL, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!dtype_ok(xdtype) || N < 0 || K < 1 || K > (1 << 18) || m < 1 || m > gate::kMaxTeacher ||
      N > INT32_MAX / m || (kind != GMM_TEACHER_LOGITS && kind != GMM_TEACHER_GAMMA) ||
      (flags & ~GMM_DISTILL_ADD) || !((float)temperature > 0.f) ||
      !((float)temperature < INFINITY) || !loss || !ws)
    return GMM_ERR_INVALID_ARG;
  if (N > 0 && (!L || !ids || !values || !rows)) return GMM_ERR_INVALID_ARG;
  if (((uintptr_t)L | (uintptr_t)dL) % dtype_size(xdtype) ||
      !aligned(4, ids, values, weights, rows, loss) || !aligned(256, (char*)ws))
    return GMM_ERR_INVALID_ARG;
  if (ws_bytes < gmm_distill_ws_bytes()) return GMM_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope p("distill_kernel", s, 2);
  const int b = (int)(N < 1 ? 1 : N < kMaxBlocks ? N : kMaxBlocks);
#define CALL(T) distill_kernel<T><<<b, kThreads, 0, s>>>((const T*)L, N, K, m, kind, flags & GMM_DISTILL_ADD, (float)temperature, (float)scale, ids, values, weights, rows, (double*)ws, (T*)dL)
  if (xdtype == GMM_F32) CALL(float);
  else if (xdtype == GMM_F16) CALL(__half);
  else CALL(__nv_bfloat16);
#undef CALL
  distill_finish_kernel<<<1, kThreads, 0, s>>>((const double*)ws, b, scale, loss);
  return launched();
}

}  // extern "C"
