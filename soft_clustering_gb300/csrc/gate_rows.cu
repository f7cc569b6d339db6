// gate_rows.cu - a learned gate: entry points, and what follows its kernels
// (gate_rows.cuh).
#include "gate_rows.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kThreads = 256;
constexpr int kFinishColumns = 32;
constexpr int kFinishThreads = 1024;

size_t ws_layout(int64_t N, int K, void* base, GateWs* w) {
  const int64_t b = N < 1 ? 1 : N < kGateGrid ? N : kGateGrid;
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o += align_up(n); return (char*)base + at; };
  GateWs t;
  t.ticket = (uint32_t*)take(4);
  t.part = (double*)take(sizeof(double) * ((K + kFinishColumns - 1) / kFinishColumns));
  t.rows = (int32_t*)take(sizeof(int32_t) * b);
  t.kept = (int32_t*)take(sizeof(int32_t) * b);
  t.mass = (float*)take(sizeof(float) * (size_t)b * K);
  t.counts = (int32_t*)take(sizeof(int32_t) * (size_t)b * K);
  t.scale = (float2*)take(sizeof(float2) * (size_t)(K > 16 * kGateBlockThreads ? N : 0));
  if (w) *w = t;
  return o;
}

// The blocks' sums in order, 32 columns a block, in 64 bits; the last block to
// end adds up the loss.
__global__ void __launch_bounds__(kFinishThreads)
gate_finish_kernel(GateWs ws, int blocks, int K, int64_t* __restrict__ counts, float* __restrict__ mass,
                   float* __restrict__ share, float* __restrict__ loss) {
  constexpr int R = kFinishThreads / kFinishColumns;
  __shared__ double part[32], sums[R][kFinishColumns + 1];
  __shared__ long long parti[32];
  __shared__ int numbers[R][kFinishColumns + 1];
  __shared__ bool last;
  long long rows = 0, all = 0;
  for (int b = threadIdx.x; b < blocks; b += kFinishThreads) rows += ws.rows[b], all += ws.kept[b];
  rows = block_reduce(rows, 0ll, SumOp(), parti);
  all = block_reduce(all, 0ll, SumOp(), parti);
  const int c = threadIdx.x % kFinishColumns, r = threadIdx.x / kFinishColumns;
  const int k = blockIdx.x * kFinishColumns + c;
  double s = 0.0;
  int n = 0;
  if (k < K)
    for (int b = r; b < blocks; b += R) {
      s += ws.mass[(size_t)b * K + k];
      n += ws.counts[(size_t)b * K + k];
    }
  sums[r][c] = s;
  numbers[r][c] = n;
  __syncthreads();
  double term = 0.0;
  if (r == 0 && k < K) {
    long long count = 0;
    s = 0.0;
#pragma unroll
    for (int i = 0; i < R; ++i) s += sums[i][c], count += numbers[i][c];
    const double f = rows > 0 && all > 0 ? (double)K * count / ((double)all * rows) : 0.0;
    counts[k] = count;
    mass[k] = (float)s;
    share[k] = (float)f;
    term = f * s;
  }
  term = block_reduce(term, 0.0, SumOp(), part);
  if (threadIdx.x == 0) {
    ws.part[blockIdx.x] = term;
    __threadfence();
    last = atomicAdd(ws.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  s = 0.0;
  for (int b = threadIdx.x; b < gridDim.x; b += kFinishThreads) s += __ldcg(ws.part + b);
  s = block_reduce(s, 0.0, SumOp(), part);
  if (threadIdx.x == 0) *loss = (float)s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
gate_grad_kernel(const T* __restrict__ L, int64_t N, int K, int m, int normalised,
                 const uint8_t* __restrict__ live, const int32_t* __restrict__ ids,
                 const float* __restrict__ gamma, const float* __restrict__ dgamma,
                 const float* __restrict__ share, float coef, T* __restrict__ dL) {
  __shared__ float partf[32];
  for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const T* x = L + n * K;
    T* d = dL + n * K;
    const bool on = !live || live[n];
    float top = -INFINITY;
    if (on)
      for (int k = threadIdx.x; k < K; k += kThreads) {
        const float v = to_f(x[k]);
        top = v > top || isnan(v) ? v : top;
      }
    // NaN is the largest
    top = unordered(block_reduce(ordered(top), 0u, MaxOp(), (uint32_t*)partf));
    if (!on || top == -INFINITY) {
      for (int k = threadIdx.x; k < K; k += kThreads) d[k] = from_f<T>(0.f);
      continue;
    }
    float v[kMaxTop], S = 0.f;
    int id[kMaxTop];
#pragma unroll
    for (int t = 0; t < kMaxTop; ++t) {
      id[t] = -1, v[t] = 0.f;
      if (dgamma && t < m) {
        id[t] = ids[n * m + t];
        if (id[t] >= K) id[t] = -1;
        if (id[t] >= 0) v[t] = gamma[n * m + t] * dgamma[n * m + t];
      }
      S += v[t];
    }
    if (normalised) {
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t)
        if (id[t] >= 0) v[t] -= gamma[n * m + t] * S;
      S = 0.f;
    }
    float sum = 0.f, dot = 0.f;
    for (int k = threadIdx.x; k < K; k += kThreads) {
      const float e = expf(to_f(x[k]) - top);
      sum += e;
      if (share) dot += e * share[k];
    }
    sum = block_reduce(sum, 0.f, SumOp(), partf);
    dot = block_reduce(dot, 0.f, SumOp(), partf) / sum;
    auto base = [&](int k) {
      const float p = expf(to_f(x[k]) - top) / sum;
      return p * ((share ? coef * (share[k] - dot) : 0.f) - S);
    };
    for (int k = threadIdx.x; k < K; k += kThreads) d[k] = from_f<T>(base(k));
    __syncthreads();
    if (threadIdx.x < m) {
      // the entries of a component together, by the first of them
      int k = -1;
      float w = 0.f;
      bool first = true;
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t)
        if (t == (int)threadIdx.x) k = id[t];
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t)
        if (id[t] == k) {
          if (t < (int)threadIdx.x) first = false;
          w += v[t];
        }
      if (k >= 0 && first) d[k] = from_f<T>(base(k) + w);
    }
  }
}

}  // namespace
}  // namespace gmm

using namespace gmm;

extern "C" {

static bool gate_ok(int xdtype, int64_t N, int K, int m, int flags) {
  return dtype_ok(xdtype) && K >= 1 && K <= kMaxK && m >= 1 && m <= gate::kMaxTop && N >= 0 &&
         N <= INT32_MAX / m && (flags & ~GMM_GATE_NORMALISED) == 0;
}

size_t gmm_gate_ws_bytes(int64_t N, int K, int m) {
  return gate_ok(GMM_F32, N, K, m, 0) ? ws_layout(N, K, nullptr, nullptr) : 0;
}

gmm_status gmm_gate(const void* L, gmm_dtype xdtype, int64_t N, int K, int m, int flags,
                    const uint8_t* live, int32_t* ids, float* gamma, float* lse, int64_t* counts,
                    float* mass, float* share, float* loss, void* ws, size_t ws_bytes,
                    void* stream) {
  if (!gate_ok(xdtype, N, K, m, flags)) return GMM_ERR_INVALID_ARG;
  const int outs = !!counts + !!mass + !!share + !!loss;
  if (outs != 0 && outs != 4) return GMM_ERR_INVALID_ARG;
  if (N > 0 && (!L || !ids || !gamma)) return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)L % dtype_size(xdtype) || !aligned(4, ids, gamma, lse, mass, share, loss) ||
      !aligned(8, counts))
    return GMM_ERR_INVALID_ARG;
  GateWs w{};
  if (outs) {
    if (!ws || !aligned(256, (char*)ws)) return GMM_ERR_INVALID_ARG;
    if (ws_bytes < ws_layout(N, K, ws, &w)) return GMM_ERR_WORKSPACE;
  }
  if (N == 0 && !outs) return GMM_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const GateArgs a{L, live, ids, gamma, lse, N, K, m, flags & GMM_GATE_NORMALISED, outs != 0, w};
  int64_t blocks;
  {
    ProfScope p("gate_kernel", s);
    blocks = xdtype == GMM_F32   ? launch_gate_f32(a, s)
             : xdtype == GMM_F16 ? launch_gate_f16(a, s)
                                 : launch_gate_bf16(a, s);
  }
  if (!blocks) return GMM_ERR_CUDA;
  if (outs) {
    ProfScope p("gate_finish_kernel", s);
    gate_finish_kernel<<<(K + kFinishColumns - 1) / kFinishColumns, kFinishThreads, 0, s>>>(
        w, (int)blocks, K, counts, mass, share, loss);
  }
  return launched();
}

gmm_status gmm_gate_grad(const void* L, gmm_dtype xdtype, int64_t N, int K, int m, int flags,
                         const uint8_t* live, const int32_t* ids, const float* gamma,
                         const float* dgamma, const float* share, double coef, void* dL,
                         void* stream) {
  if (!gate_ok(xdtype, N, K, m, flags)) return GMM_ERR_INVALID_ARG;
  if (N == 0) return GMM_OK;
  if (!L || !dL || (dgamma && (!ids || !gamma))) return GMM_ERR_INVALID_ARG;
  if (((uintptr_t)L | (uintptr_t)dL) % dtype_size(xdtype) || !aligned(4, ids, gamma, dgamma, share))
    return GMM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope p("gate_grad_kernel", s);
  const int b = (int)(N < 8 * 152 ? N : 8 * 152);
#define CALL(T) gate_grad_kernel<T><<<b, kThreads, 0, s>>>((const T*)L, N, K, m, flags, live, ids, gamma, dgamma, share, (float)coef, (T*)dL)
  if (xdtype == GMM_F32) CALL(float);
  else if (xdtype == GMM_F16) CALL(__half);
  else CALL(__nv_bfloat16);
#undef CALL
  return launched();
}

}  // extern "C"
