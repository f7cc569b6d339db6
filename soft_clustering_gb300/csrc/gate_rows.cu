// gate_rows.cu - a learned gate: the m largest logits of a row, their softmax,
// the balance loss, and the gradient of the logits.
//
//   gmm_gate       ids, gamma, lse; counts, mass, share, loss
//   gmm_gate_grad  dL = p (coef (share - <share, p>) - S) + v at ids
//
// A block takes a row at a time and passes over it once for each of the m
// entries, for the sum and for the mass.  Column k of a row belongs to thread
// k mod 256 of every block, so a block's sums over its rows need no atomics.
#include "gate_internal.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 304;

// A block's sums of the balance outputs: rows that count, then mass [K] and
// counts [K]; the head holds the finish's partial losses and its ticket.
struct Ws {
  float* mass;      // blocks * K
  int32_t* counts;  // blocks * K
  int32_t* rows;    // blocks
  double* part;     // finish blocks
  uint32_t* ticket;
};
constexpr int kFinishColumns = 256;

int blocks_for(int64_t N) { return (int)(N < 1 ? 1 : N < kMaxBlocks ? N : kMaxBlocks); }

size_t ws_layout(int64_t N, int K, void* base, Ws* w) {
  const int b = blocks_for(N), f = (K + kFinishColumns - 1) / kFinishColumns;
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o += align_up(n); return (char*)base + at; };
  Ws t;
  t.ticket = (uint32_t*)take(4);
  t.part = (double*)take(sizeof(double) * f);
  t.rows = (int32_t*)take(sizeof(int32_t) * b);
  t.mass = (float*)take(sizeof(float) * (size_t)b * K);
  t.counts = (int32_t*)take(sizeof(int32_t) * (size_t)b * K);
  if (w) *w = t;
  return o;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
gate_kernel(const T* __restrict__ L, int64_t N, int K, int m, int normalised,
            const uint8_t* __restrict__ live, int32_t* __restrict__ ids, float* __restrict__ gamma,
            float* __restrict__ lse, Ws ws, int balance) {
  __shared__ uint64_t part64[32];
  __shared__ float partf[32];
  float* mass = ws.mass + (size_t)blockIdx.x * K;
  int32_t* counts = ws.counts + (size_t)blockIdx.x * K;
  int rows = 0;
  if (balance) {
    for (int k = threadIdx.x; k < K; k += kThreads) mass[k] = 0.f, counts[k] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *ws.ticket = 0;
  }
  for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const T* x = L + n * K;
    uint64_t key[kMaxTop];
#pragma unroll
    for (int t = 0; t < kMaxTop; ++t) key[t] = 0;
    const bool on = !live || live[n];
    if (on) {
      uint64_t below = ~0ull;
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t) {
        if (t >= m) break;
        uint64_t best = 0;
        for (int k = threadIdx.x; k < K; k += kThreads) {
          const uint64_t v = (uint64_t)ordered(to_f(x[k])) << 32 | (0xfffffffeu - (uint32_t)k);  // never ~0
          if (v < below && v > best) best = v;
        }
        key[t] = below = block_reduce(best, (uint64_t)0, MaxOp(), part64);
      }
    }
    const float top = unordered((uint32_t)(key[0] >> 32));
    const bool some = (uint32_t)(key[0] >> 32) > kOrderedNegInf;
    float sum = 0.f;
    if (some)
      for (int k = threadIdx.x; k < K; k += kThreads) sum += expf(to_f(x[k]) - top);
    sum = block_reduce(sum, 0.f, SumOp(), partf);
    float g[kMaxTop], kept = 0.f;
    int id[kMaxTop];
#pragma unroll
    for (int t = 0; t < kMaxTop; ++t) {
      const uint32_t u = (uint32_t)(key[t] >> 32);
      id[t] = u > kOrderedNegInf ? (int)(0xfffffffeu - (uint32_t)key[t]) : -1;
      g[t] = id[t] >= 0 ? expf(unordered(u) - top) : 0.f;
      kept += g[t];
    }
    if (threadIdx.x == 0) {
      const float per = normalised ? kept : sum;
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t)
        if (t < m) {
          ids[n * m + t] = id[t];
          // a NaN or infinity in the row shows in the normalised shares too
          gamma[n * m + t] = id[t] >= 0 ? (isnan(sum) ? sum : g[t] / per) : 0.f;
          if (balance && id[t] >= 0) ++counts[id[t]];
        }
      if (lse) lse[n] = some ? top + logf(sum) : -INFINITY;
    }
    if (balance && some) {
      ++rows;
      for (int k = threadIdx.x; k < K; k += kThreads) mass[k] += expf(to_f(x[k]) - top) / sum;
    }
  }
  if (balance && threadIdx.x == 0) ws.rows[blockIdx.x] = rows;
}

// Columns of all blocks in order, in 64 bits; the last block to end adds up the loss.
__global__ void __launch_bounds__(kFinishColumns)
gate_finish_kernel(Ws ws, int blocks, int K, int64_t* __restrict__ counts, float* __restrict__ mass,
                   float* __restrict__ share, float* __restrict__ loss) {
  __shared__ double part[32];
  __shared__ long long parti[32];
  __shared__ bool last;
  long long rows = 0, all = 0;
  for (int b = threadIdx.x; b < blocks; b += kFinishColumns) rows += ws.rows[b];
  rows = block_reduce(rows, 0ll, SumOp(), parti);
  for (int64_t i = threadIdx.x; i < (int64_t)blocks * K; i += kFinishColumns) all += ws.counts[i];
  all = block_reduce(all, 0ll, SumOp(), parti);
  const int k = blockIdx.x * kFinishColumns + threadIdx.x;
  double term = 0.0;
  if (k < K) {
    double s = 0.0;
    long long c = 0;
    for (int b = 0; b < blocks; ++b) {
      s += ws.mass[(size_t)b * K + k];
      c += ws.counts[(size_t)b * K + k];
    }
    const double f = rows > 0 && all > 0 ? (double)K * c / ((double)all * rows) : 0.0;
    counts[k] = c;
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
  double s = 0.0;
  for (int b = threadIdx.x; b < gridDim.x; b += kFinishColumns) s += __ldcg(ws.part + b);
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
  Ws w{};
  if (outs) {
    if (!ws || !aligned(256, (char*)ws)) return GMM_ERR_INVALID_ARG;
    if (ws_bytes < ws_layout(N, K, ws, &w)) return GMM_ERR_WORKSPACE;
  }
  if (N == 0 && !outs) return GMM_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const int b = blocks_for(N);
  {
    ProfScope p("gate_kernel", s);
#define CALL(T) gate_kernel<T><<<b, kThreads, 0, s>>>((const T*)L, N, K, m, flags, live, ids, gamma, lse, w, outs != 0)
    if (xdtype == GMM_F32) CALL(float);
    else if (xdtype == GMM_F16) CALL(__half);
    else CALL(__nv_bfloat16);
#undef CALL
  }
  if (outs) {
    ProfScope p("gate_finish_kernel", s);
    gate_finish_kernel<<<(K + kFinishColumns - 1) / kFinishColumns, kFinishColumns, 0, s>>>(
        w, b, K, counts, mass, share, loss);
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
