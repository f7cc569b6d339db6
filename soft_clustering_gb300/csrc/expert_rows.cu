// expert_rows.cu - rows to their components' places and back.
//
//   gmm_spread    Y[slot[n,t]] = gamma[n,t] X[n];  dgamma[n,t] = <X[n], Z[slot[n,t]]>
//   gmm_collect   out[n] = sum_t gamma[n,t] Z[slot[n,t]]
//
// Each is the other's adjoint.  Both go by points: spread reads a point's row
// once for its m places, collect adds the m rows in registers in fp32 and
// rounds once, in the order of t.  Bound by HBM traffic: N D + R D elements,
// 2 R D + N D with dgamma.  A block is TX lanes along a row (vectors of up to
// 16 bytes) by 256 / TX points; with dgamma TX is at most a warp, so the dot
// products end in shuffles.  Kernels by the number of entries hold as many
// points in flight as registers allow, and the next turn's slots are fetched
// before this turn's rows are moved.
// Measured (of the 6.78 TB/s a copy reaches): collect of 65536 points, 2 x
// 2048 bf16, 134 us (6.0 TB/s); spread of 2000003 points, 4 x 128 f16, 404 us
// (6.3); spread with dgamma of 1000003 points, 4 x 128 f16, 359 us (6.1).
#include "expert_internal.cuh"

namespace gmm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxM = 8;

template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T v[V]; };

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& x) {
  *reinterpret_cast<Vec<T, V>*>(p) = x;
}

// Zeros in the rows from offsets[K] (at least 0) to R-1.
template <typename T, int V>
__device__ __forceinline__ void zero_tail(T* Y, int64_t R, int D, const int64_t* offsets, int K) {
  const int64_t r0 = max((int64_t)0, offsets[K]);
  if (r0 >= R) return;
  Vec<T, V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) z.v[i] = from_f<T>(0.f);
  const int64_t total = (R - r0) * (D / V);
  T* base = Y + r0 * D;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x)
    store_vec<T, V>(base + i * V, z);
}

// Points a thread has in flight: M rows of up to 16 bytes each for every one.
__host__ __device__ constexpr int points_in_flight(int M) { return M >= 4 ? 1 : M == 2 ? 2 : 4; }
// Blocks a multiprocessor holds (what the registers of those points leave).
__host__ __device__ constexpr int resident(int M) { return M >= 8 ? 2 : 4; }

// The M slots (and weights) of point n; -1 past m, past N and outside [0, R).
template <int M>
struct Slots {
  int32_t at[M];
  float w[M];
  __device__ __forceinline__ void load(const int32_t* __restrict__ slot,
                                       const float* __restrict__ gamma, int64_t n, int64_t N, int m) {
#pragma unroll
    for (int t = 0; t < M; ++t) {
      at[t] = -1;
      w[t] = 1.f;
      if (t < m && n < N) {
        at[t] = slot[n * m + t];
        if (gamma) w[t] = gamma[n * m + t];
      }
    }
  }
  __device__ __forceinline__ void check(int64_t R) {
#pragma unroll
    for (int t = 0; t < M; ++t)
      if (at[t] >= R) at[t] = -1;
  }
};

// Both kernels fetch the next turn's slots before they move this turn's rows:
// a row's address waits on its slot, and the two latencies in a row halve the
// bandwidth.
template <typename T, int V, int M, bool DG>
__global__ void __launch_bounds__(kThreads, resident(M))
spread_kernel(const T* __restrict__ X, int64_t N, int D, int m, int K, int64_t R,
              const int32_t* __restrict__ slot, const int64_t* __restrict__ offsets,
              const float* __restrict__ gamma, const T* __restrict__ Z, T* __restrict__ Y,
              float* __restrict__ dgamma, int tx_log2) {
  constexpr int P = points_in_flight(M);
  const int TX = 1 << tx_log2;
  const int tx = threadIdx.x & (TX - 1), ty = threadIdx.x >> tx_log2;
  const int rows = kThreads >> tx_log2;
  const int nv = D / V;
  const int64_t stride = (int64_t)gridDim.x * rows * P;
  int64_t n0 = (int64_t)blockIdx.x * rows * P;
  Slots<M> next[P];
#pragma unroll
  for (int u = 0; u < P; ++u) next[u].load(slot, gamma, n0 + u * rows + ty, N, m);
  // every lane of a warp takes the same number of turns (shuffles below)
  for (; n0 < N; n0 += stride) {
    Slots<M> s[P];
    float dot[P][M];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      s[u] = next[u];
      s[u].check(R);
      next[u].load(slot, gamma, n0 + stride + u * rows + ty, N, m);
#pragma unroll
      for (int t = 0; t < M; ++t) dot[u][t] = 0.f;
    }
    for (int c = tx; c < nv; c += TX) {
      Vec<T, V> x[P], z[P][M];
#pragma unroll
      for (int u = 0; u < P; ++u) {
        const int64_t n = n0 + u * rows + ty;
        if (n < N) x[u] = load_vec<T, V>(X + n * D + (int64_t)c * V);
        if (DG) {
#pragma unroll
          for (int t = 0; t < M; ++t)
            if (s[u].at[t] >= 0) z[u][t] = load_vec<T, V>(Z + (int64_t)s[u].at[t] * D + (int64_t)c * V);
        }
      }
#pragma unroll
      for (int u = 0; u < P; ++u) {
#pragma unroll
        for (int t = 0; t < M; ++t) {
          if (s[u].at[t] < 0) continue;
          T* y = Y + (int64_t)s[u].at[t] * D + (int64_t)c * V;
          if (DG) {
#pragma unroll
            for (int i = 0; i < V; ++i)
              dot[u][t] = fmaf(to_f(x[u].v[i]), to_f(z[u][t].v[i]), dot[u][t]);
          }
          if (gamma) {
            Vec<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(to_f(x[u].v[i]) * s[u].w[t]);
            store_vec<T, V>(y, o);
          } else {
            store_vec<T, V>(y, x[u]);
          }
        }
      }
    }
    if (DG) {
#pragma unroll
      for (int u = 0; u < P; ++u) {
        const int64_t n = n0 + u * rows + ty;
#pragma unroll
        for (int t = 0; t < M; ++t) {
          for (int o = TX >> 1; o > 0; o >>= 1)
            dot[u][t] += __shfl_xor_sync(0xffffffffu, dot[u][t], o);
          if (t < m && n < N && tx == 0) dgamma[n * m + t] = s[u].at[t] >= 0 ? dot[u][t] : 0.f;
        }
      }
    }
  }
  zero_tail<T, V>(Y, R, D, offsets, K);
}

template <typename T, int V, int M>
__global__ void __launch_bounds__(kThreads, resident(M))
collect_kernel(const T* __restrict__ Z, int64_t N, int D, int m, int64_t R,
               const int32_t* __restrict__ slot, const float* __restrict__ gamma,
               T* __restrict__ out, int tx_log2) {
  constexpr int P = points_in_flight(M);
  const int TX = 1 << tx_log2;
  const int tx = threadIdx.x & (TX - 1), ty = threadIdx.x >> tx_log2;
  const int rows = kThreads >> tx_log2;
  const int nv = D / V;
  const int64_t stride = (int64_t)gridDim.x * rows * P;
  int64_t n0 = (int64_t)blockIdx.x * rows * P;
  Slots<M> next[P];
#pragma unroll
  for (int u = 0; u < P; ++u) next[u].load(slot, gamma, n0 + u * rows + ty, N, m);
  for (; n0 < N; n0 += stride) {
    Slots<M> s[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      s[u] = next[u];
      s[u].check(R);
      next[u].load(slot, gamma, n0 + stride + u * rows + ty, N, m);
    }
    for (int c = tx; c < nv; c += TX) {
      Vec<T, V> z[P][M];
#pragma unroll
      for (int u = 0; u < P; ++u)
#pragma unroll
        for (int t = 0; t < M; ++t)
          if (s[u].at[t] >= 0) z[u][t] = load_vec<T, V>(Z + (int64_t)s[u].at[t] * D + (int64_t)c * V);
#pragma unroll
      for (int u = 0; u < P; ++u) {
        const int64_t n = n0 + u * rows + ty;
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
        for (int t = 0; t < M; ++t)
          if (s[u].at[t] >= 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(s[u].w[t], to_f(z[u][t].v[i]), acc[i]);
          }
        Vec<T, V> y;
#pragma unroll
        for (int i = 0; i < V; ++i) y.v[i] = from_f<T>(acc[i]);
        if (n < N) store_vec<T, V>(out + n * D + (int64_t)c * V, y);
      }
    }
  }
}

// Widest vector (in elements) that divides D and the addresses.
int vec_width(int D, int es, const void* a, const void* b, const void* c) {
  const uintptr_t bits = (uintptr_t)a | (uintptr_t)b | (uintptr_t)c;
  for (int v = 16 / es; v > 1; v >>= 1)
    if (D % v == 0 && bits % (uintptr_t)(v * es) == 0) return v;
  return 1;
}

int tx_log2_for(int nv, int most) {
  int l = 0;
  while ((1 << l) < nv && l < most) ++l;
  return l;
}

// Blocks: one for every `rows * P` points, up to those that are resident at
// once, which then take turns.
int64_t grid_for(int64_t N, int rows, int P, int most) {
  const int64_t g = (N + (int64_t)rows * P - 1) / ((int64_t)rows * P);
  return g > 152 * most ? 152 * most : g;
}

template <typename T, int V, int M>
void spread_launch_m(const void* X, int64_t N, int D, int m, int K, int64_t R, const int32_t* slot,
                     const int64_t* offsets, const float* gamma, const void* Z, void* Y,
                     float* dgamma, cudaStream_t s) {
  const int l = tx_log2_for(D / V, dgamma ? 5 : 8);
  int64_t grid = grid_for(N, kThreads >> l, points_in_flight(M), resident(M));
  const int64_t tail = (R * (D / V) + kThreads * 8 - 1) / (kThreads * 8);  // if every row were zero
  if (grid < tail) grid = tail < 152 * resident(M) ? tail : 152 * resident(M);
  if (grid < 1) grid = 1;
  if (dgamma)
    spread_kernel<T, V, M, true><<<(unsigned)grid, kThreads, 0, s>>>(
        (const T*)X, N, D, m, K, R, slot, offsets, gamma, (const T*)Z, (T*)Y, dgamma, l);
  else
    spread_kernel<T, V, M, false><<<(unsigned)grid, kThreads, 0, s>>>(
        (const T*)X, N, D, m, K, R, slot, offsets, gamma, (const T*)Z, (T*)Y, dgamma, l);
}

template <typename T, int V, int M>
void collect_launch_m(const void* Z, int64_t N, int D, int m, int64_t R, const int32_t* slot,
                      const float* gamma, void* out, cudaStream_t s) {
  const int l = tx_log2_for(D / V, 8);
  const int64_t grid = grid_for(N, kThreads >> l, points_in_flight(M), resident(M));
  collect_kernel<T, V, M><<<(unsigned)grid, kThreads, 0, s>>>((const T*)Z, N, D, m, R, slot, gamma,
                                                              (T*)out, l);
}

#define GMM_BY_M(m, CALL, ...)          \
  if ((m) == 1) CALL<T, V, 1>(__VA_ARGS__);      \
  else if ((m) == 2) CALL<T, V, 2>(__VA_ARGS__); \
  else if ((m) <= 4) CALL<T, V, 4>(__VA_ARGS__); \
  else CALL<T, V, 8>(__VA_ARGS__);

template <typename T, int V>
void spread_launch(const void* X, int64_t N, int D, int m, int K, int64_t R, const int32_t* slot,
                   const int64_t* offsets, const float* gamma, const void* Z, void* Y,
                   float* dgamma, cudaStream_t s) {
  GMM_BY_M(m, spread_launch_m, X, N, D, m, K, R, slot, offsets, gamma, Z, Y, dgamma, s)
}
template <typename T, int V>
void collect_launch(const void* Z, int64_t N, int D, int m, int64_t R, const int32_t* slot,
                    const float* gamma, void* out, cudaStream_t s) {
  GMM_BY_M(m, collect_launch_m, Z, N, D, m, R, slot, gamma, out, s)
}

#define GMM_BY_VEC(T, v, CALL)                      \
  switch (v) {                                      \
    case 8: if constexpr (sizeof(T) == 2) { CALL(T, 8); } break; \
    case 4: CALL(T, 4); break;                      \
    case 2: CALL(T, 2); break;                      \
    default: CALL(T, 1); break;                     \
  }
#define GMM_BY_TYPE(x, v, CALL)                             \
  if ((x) == GMM_F32) { GMM_BY_VEC(float, v, CALL) }        \
  else if ((x) == GMM_F16) { GMM_BY_VEC(__half, v, CALL) }  \
  else { GMM_BY_VEC(__nv_bfloat16, v, CALL) }

bool rows_ok(int xdtype, int64_t N, int D, int m, int64_t R) {
  return dtype_ok(xdtype) && N >= 0 && D >= 1 && m >= 1 && m <= kMaxM && R >= 0 &&
         R <= INT32_MAX && N <= INT32_MAX / m;
}

}  // namespace
}  // namespace gmm

using namespace gmm;

extern "C" {

gmm_status gmm_spread(const void* X, gmm_dtype xdtype, int64_t N, int D, int m, int K, int64_t R,
                      const int32_t* slot, const int64_t* offsets, const float* gamma,
                      const void* Z, void* Y, float* dgamma, void* stream) {
  if (!rows_ok(xdtype, N, D, m, R) || K < 1 || K > kMaxK || !offsets) return GMM_ERR_INVALID_ARG;
  if (N > 0 && (!X || !slot)) return GMM_ERR_INVALID_ARG;
  if (R > 0 && !Y) return GMM_ERR_INVALID_ARG;
  if ((N > 0 && R > 0) && (!Z != !dgamma)) return GMM_ERR_INVALID_ARG;
  const uintptr_t bits = (uintptr_t)X | (uintptr_t)Y | (uintptr_t)Z;
  if (bits % dtype_size(xdtype)) return GMM_ERR_INVALID_ARG;
  if (!aligned(4, slot, gamma, dgamma) || !aligned(8, offsets)) return GMM_ERR_INVALID_ARG;
  if (N == 0 && R == 0) return GMM_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const int v = vec_width(D, dtype_size(xdtype), X, Y, Z);
  ProfScope p("spread_kernel", s);
#define CALL(T, V) spread_launch<T, V>(X, N, D, m, K, R, slot, offsets, gamma, Z, Y, dgamma, s)
  GMM_BY_TYPE(xdtype, v, CALL)
#undef CALL
  return launched();
}

gmm_status gmm_collect(const void* Z, gmm_dtype xdtype, int64_t N, int D, int m, int64_t R,
                       const int32_t* slot, const float* gamma, void* out, void* stream) {
  if (!rows_ok(xdtype, N, D, m, R)) return GMM_ERR_INVALID_ARG;
  if (N == 0) return GMM_OK;
  if (!slot || !out || (R > 0 && !Z)) return GMM_ERR_INVALID_ARG;
  if (((uintptr_t)Z | (uintptr_t)out) % dtype_size(xdtype)) return GMM_ERR_INVALID_ARG;
  if (!aligned(4, slot, gamma)) return GMM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const int v = vec_width(D, dtype_size(xdtype), Z, out, nullptr);
  ProfScope p("collect_kernel", s);
#define CALL(T, V) collect_launch<T, V>(Z, N, D, m, R, slot, gamma, out, s)
  GMM_BY_TYPE(xdtype, v, CALL)
#undef CALL
  return launched();
}

}  // extern "C"
