// expert_few.cu - gmm_expert_product for few rows (single queries and small
// batches): every weight of the components that have a row is read once, so
// the time is that of streaming those weights, and of one launch.
//
// Block (x, r): row r's component is found by counting the offsets at or
// before it; the component's first row does the work of all its rows, up to
// kRows at a time, for 32 output features: a warp takes four of them, its
// lanes 8 input features of each at a time.  The 4 x kRows sums of a warp are
// added across its lanes by halving: 31 shuffles for 16 sums.
// 16 rows, 14 of 64 components of 1024 x 2048 in bf16: 14.2 us a call (4.2
// TB/s; the weights alone 8.7 us at the copy rate), of which the search, the
// first fetch and the last blocks take about five.  Three blocks a
// multiprocessor; with two, or with 64 features a block, 15 to 16.
#include "expert_product.cuh"

namespace gmm {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;
constexpr int kFeats = 4;                        // output features of a warp
constexpr int kBlockFeats = kFeats * kThreads / 32;

template <typename T> __device__ __forceinline__ void widen8(const uint4& q, float* x);
template <> __device__ __forceinline__ void widen8<__nv_bfloat16>(const uint4& q, float* x) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
template <> __device__ __forceinline__ void widen8<__half>(const uint4& q, float* x) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}

// N sums of each lane -> the sum over all lanes of number lane * N / 32 (N a
// power of two up to 32).
template <int N>
__device__ __forceinline__ float lane_sums(float* v) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = up ? v[i] : v[i + n / 2];
      const float keep = up ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <typename T, int NR>
__device__ __forceinline__ void few_rows(const T* __restrict__ A, const T* __restrict__ W,
                                         T* __restrict__ Y, int d_in, int d_out, int f0, int rows) {
  const int lane = threadIdx.x & 31;
  float acc[kFeats * NR];
#pragma unroll
  for (int i = 0; i < kFeats * NR; ++i) acc[i] = 0.f;
  const T* w[kFeats];
#pragma unroll
  for (int f = 0; f < kFeats; ++f) w[f] = W + (int64_t)min(f0 + f, d_out - 1) * d_in;
  // one row: 16 loads a lane in flight; more rows take the registers
#pragma unroll (NR == 1 ? 4 : NR == 2 ? 2 : 1)
  for (int c = lane * 8; c < d_in; c += 256) {
    uint4 q[kFeats];
#pragma unroll
    for (int f = 0; f < kFeats; ++f) q[f] = __ldcs(reinterpret_cast<const uint4*>(w[f] + c));
    float x[NR][8];
#pragma unroll
    for (int r = 0; r < NR; ++r)
      widen8<T>(__ldg(reinterpret_cast<const uint4*>(A + (int64_t)min(r, rows - 1) * d_in + c)), x[r]);
#pragma unroll
    for (int f = 0; f < kFeats; ++f) {
      float u[8];
      widen8<T>(q[f], u);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[f * NR + r] = fmaf(u[j], x[r][j], acc[f * NR + r]);
    }
  }
  constexpr int N = kFeats * NR, each = 32 / N;
  const float s = lane_sums<N>(acc);
  const int i = lane / each, f = f0 + i / NR, r = i % NR;
  if (lane % each == 0 && f < d_out && r < rows) Y[(int64_t)r * d_out + f] = from_f<T>(s);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3)
few_rows_kernel(const T* __restrict__ A, int64_t R, int d_in, int d_out, int K,
                const int64_t* __restrict__ offsets, const T* __restrict__ W, T* __restrict__ Y) {
  __shared__ int found[3][kThreads / 32];
  const int64_t row = blockIdx.y;
  const int warp = threadIdx.x >> 5;
  // the offsets at or before the row: how many, and the last; the first after
  int count = 0, last = (int)clamp_row(offsets[0], R), next = (int)R;
  for (int k = threadIdx.x; k < K; k += kThreads) {
    const int v = (int)clamp_row(offsets[k + 1], R);
    const bool before = v <= row;
    count += before;
    if (before) last = max(last, v);
    else next = min(next, v);
  }
  count = __reduce_add_sync(0xffffffffu, count);
  last = __reduce_max_sync(0xffffffffu, last);
  next = __reduce_min_sync(0xffffffffu, next);
  if ((threadIdx.x & 31) == 0) {
    found[0][warp] = count;
    found[1][warp] = last;
    found[2][warp] = next;
  }
  __syncthreads();
  int k = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    k += found[0][i];
    last = max(last, found[1][i]);
    next = min(next, found[2][i]);
  }
  if (k == K) {  // a row of nobody
    const int f = blockIdx.x * kBlockFeats + threadIdx.x;
    if (threadIdx.x < kBlockFeats && f < d_out) Y[row * d_out + f] = from_f<T>(0.f);
    return;
  }
  const int f0 = blockIdx.x * kBlockFeats + warp * kFeats;
  if (last != row || f0 >= d_out) return;
  const int n = next - (int)row;
  const T* w = W + (int64_t)k * d_in * d_out;
  for (int g = 0; g < n; g += kRows) {
    const T* a = A + (row + g) * d_in;
    T* y = Y + (row + g) * d_out;
    const int rows = min(kRows, n - g);
    if (rows == 1) few_rows<T, 1>(a, w, y, d_in, d_out, f0, rows);
    else if (rows == 2) few_rows<T, 2>(a, w, y, d_in, d_out, f0, rows);
    else few_rows<T, 4>(a, w, y, d_in, d_out, f0, rows);
  }
}

}  // namespace

gmm_status few_rows_product(const void* A, int xdtype, const void* W, void* Y, int64_t R, int d_in,
                            int d_out, int K, const int64_t* offsets, cudaStream_t s) {
  const dim3 grid((d_out + kBlockFeats - 1) / kBlockFeats, (unsigned)R);
  ProfScope p("few_rows_kernel", s);
  if (xdtype == GMM_BF16)
    few_rows_kernel<<<grid, kThreads, 0, s>>>((const __nv_bfloat16*)A, R, d_in, d_out, K, offsets,
                                              (const __nv_bfloat16*)W, (__nv_bfloat16*)Y);
  else
    few_rows_kernel<<<grid, kThreads, 0, s>>>((const __half*)A, R, d_in, d_out, K, offsets,
                                              (const __half*)W, (__half*)Y);
  return launched();
}

}  // namespace gmm
