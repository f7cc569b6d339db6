// expert_product.cu - the experts' products: argument checks, the list of row
// tiles, and the CUDA-core kernel that serves every size and type.
//
//   product     Y[r]  = W_k A[r]          rows r of component k
//   product_dx  dA[r] = W_k^T dY[r]
//   product_dw  dW_k  = sum_r dY[r] A[r]^T
//
// One fp32 kernel computes all three as C[i][j] = sum_l P[i][l] Q[j][l] with
// the strides of the case: 64 x 64 tiles, 16 steps of l staged in shared
// memory, 4 x 4 outputs a thread.  Bound by shared memory (two 16-byte reads
// for 16 products a thread): 8192 rows through 32 experts of 512 x 512 in
// fp32 take 172 us forward (25 TFLOP/s), 467 us for both gradients.  The
// 16-bit types take expert_product_tc.cu wherever their rows are aligned.
#include "expert_product.cuh"

namespace gmm {
namespace {

constexpr int kT = 64;        // tile rows and columns of the CUDA-core kernel
constexpr int kStep = 16;
constexpr int kListThreads = 1024;
constexpr int kListSmem = 4096;   // components whose first tiles fit in shared memory

// Row tiles of T rows for every component, in order, then those of the rows
// past offsets[K] (component -1: zeros).  Offsets are held within [0, R],
// and the list within its `room`, which ascending offsets cannot exceed.
// The kernel after it may start at once (its set-up overlaps this one) and
// waits for this one's end itself.
__global__ void __launch_bounds__(kListThreads)
tile_list_kernel(const int64_t* __restrict__ offsets, int K, int64_t R, int T, uint32_t room,
                 int32_t* __restrict__ count, uint32_t* __restrict__ first, int4* __restrict__ tiles) {
  __shared__ uint32_t wsum[32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t before[kListSmem + 1];
  const int G = K + 1;
  const int per = (G + kListThreads - 1) / kListThreads;
  const int k0 = min(G, (int)threadIdx.x * per), k1 = min(G, k0 + per);
  uint32_t mine = 0;
  for (int k = k0; k < k1; ++k) {
    const int64_t a = clamp_row(offsets[k], R), b = k < K ? clamp_row(offsets[k + 1], R) : R;
    if (b > a) mine += (uint32_t)((b - a + T - 1) / T);
  }
  uint32_t at = block_exclusive_1024(mine, wsum);
  if (G <= kListSmem) {
    // every thread writes tiles: the component of tile t is the last one that
    // starts at or before it
    for (int k = k0; k < k1; ++k) {
      const int64_t a = clamp_row(offsets[k], R), b = k < K ? clamp_row(offsets[k + 1], R) : R;
      before[k] = at;
      first[k] = min(at, room);
      if (b > a) at += (uint32_t)((b - a + T - 1) / T);
    }
    if (k1 == G && k0 < k1) {
      before[G] = at;
      *count = (int32_t)min(at, room);
    }
    __syncthreads();
    const uint32_t total = min(before[G], room);
    for (uint32_t t = threadIdx.x; t < total; t += kListThreads) {
      int lo = 0, hi = G - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int64_t a = clamp_row(offsets[lo], R), b = lo < K ? clamp_row(offsets[lo + 1], R) : R;
      const int64_t r = a + (int64_t)(t - before[lo]) * T;
      tiles[t] = make_int4(lo < K ? lo : -1, (int)r, (int)min((int64_t)T, b - r), 0);
    }
    return;
  }
  for (int k = k0; k < k1; ++k) {
    const int64_t a = clamp_row(offsets[k], R), b = k < K ? clamp_row(offsets[k + 1], R) : R;
    first[k] = min(at, room);
    for (int64_t r = a; r < b; r += T, ++at)
      if (at < room) tiles[at] = make_int4(k < K ? k : -1, (int)r, (int)min((int64_t)T, b - r), 0);
  }
  if (k1 == G && k0 < k1) *count = (int32_t)min(at, room);
}

// P[i][l] at p + i*pi + l*pl, likewise Q; C row-major with stride ldc.
template <typename T, typename TO>
__device__ __forceinline__ void tile_product(const T* __restrict__ p, int64_t pi, int64_t pl,
                                             const T* __restrict__ q, int64_t qj, int64_t ql,
                                             int rows, int cols, int64_t len, TO* __restrict__ c,
                                             int64_t ldc) {
  __shared__ float sp[kStep][kT + 4], sq[kStep][kT + 4];
  const int tid = threadIdx.x;
  const int ti = (tid >> 4) * 4, tj = (tid & 15) * 4;
  float acc[4][4] = {};
  for (int64_t l0 = 0; l0 < len; l0 += kStep) {
#pragma unroll
    for (int x = tid; x < kT * kStep; x += 256) {
      // neighbouring threads along whichever index is contiguous in memory
      const int ip = pl == 1 ? x / kStep : x % kT, lp = pl == 1 ? x % kStep : x / kT;
      sp[lp][ip] = (ip < rows && l0 + lp < len) ? to_f(p[ip * pi + (l0 + lp) * pl]) : 0.f;
      const int jq = ql == 1 ? x / kStep : x % kT, lq = ql == 1 ? x % kStep : x / kT;
      sq[lq][jq] = (jq < cols && l0 + lq < len) ? to_f(q[jq * qj + (l0 + lq) * ql]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int l = 0; l < kStep; ++l) {
      const float4 a = *reinterpret_cast<const float4*>(&sp[l][ti]);
      const float4 b = *reinterpret_cast<const float4*>(&sq[l][tj]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (ti + i < rows && tj + j < cols) c[(ti + i) * ldc + tj + j] = from_f<TO>(acc[i][j]);
}

// Rows (A or dY, width d_from) through W_k to width d_to.  DX: through W_k^T.
template <typename T, bool DX>
__global__ void __launch_bounds__(256)
rows_simt_kernel(const T* __restrict__ A, const T* __restrict__ W, T* __restrict__ Y, int d_from,
                 int d_to, const int32_t* __restrict__ count, const int4* __restrict__ tiles) {
  if ((int)blockIdx.x >= *count) return;
  const int4 t = tiles[blockIdx.x];
  const int j0 = blockIdx.y * kT;
  const int cols = min(kT, d_to - j0);
  const int64_t r0 = t.y;
  T* y = Y + r0 * d_to + j0;
  if (t.x < 0) {
    for (int x = threadIdx.x; x < t.z * cols; x += 256)
      y[(int64_t)(x / cols) * d_to + x % cols] = from_f<T>(0.f);
    return;
  }
  const T* w = W + (int64_t)t.x * d_from * d_to + (DX ? (int64_t)j0 : (int64_t)j0 * d_from);
  tile_product<T, T>(A + r0 * d_from, d_from, 1, w, DX ? 1 : d_from, DX ? d_to : 1, t.z, cols,
                     d_from, y, d_to);
}

template <typename T, typename TO>
__global__ void __launch_bounds__(256)
weights_simt_kernel(const T* __restrict__ dY, const T* __restrict__ A, TO* __restrict__ dW,
                    int d_in, int d_out, int K, const int64_t* __restrict__ offsets, int64_t R) {
  const int o0 = blockIdx.x * kT, i0 = blockIdx.y * kT;
  for (int k = blockIdx.z; k < K; k += gridDim.z) {
    const int64_t a = clamp_row(offsets[k], R), b = clamp_row(offsets[k + 1], R);
    tile_product<T, TO>(dY + a * d_out + o0, 1, d_out, A + a * d_in + i0, 1, d_in,
                        min(kT, d_out - o0), min(kT, d_in - i0), b > a ? b - a : 0,
                        dW + ((int64_t)k * d_out + o0) * d_in + i0, d_in);
  }
}

bool sizes_ok(int xdtype, int64_t R, int d_in, int d_out, int K) {
  return dtype_ok(xdtype) && R >= 0 && R <= INT32_MAX && K >= 1 && K <= kMaxK && d_in >= 1 &&
         d_out >= 1 && (int64_t)d_in * d_out <= INT32_MAX;
}

gmm_status check(int xdtype, int64_t R, int d_in, int d_out, int K, const int64_t* offsets,
                 const void* rows1, const void* rows2, const void* w, void* ws, size_t ws_bytes) {
  if (!sizes_ok(xdtype, R, d_in, d_out, K) || !offsets || !w || !ws) return GMM_ERR_INVALID_ARG;
  if (R > 0 && (!rows1 || !rows2)) return GMM_ERR_INVALID_ARG;
  if (((uintptr_t)rows1 | (uintptr_t)rows2 | (uintptr_t)w) % dtype_size(xdtype))
    return GMM_ERR_INVALID_ARG;
  if (!aligned(kAlign, ws) || !aligned(8, offsets)) return GMM_ERR_INVALID_ARG;
  if (ws_bytes < ProductLayout::make(R, d_in, d_out, K, xdtype).bytes) return GMM_ERR_WORKSPACE;
  return GMM_OK;
}

template <typename T>
gmm_status rows_simt(const void* A, int xdtype, const void* W, void* Y, int64_t R, int d_from,
                     int d_to, int K, bool dx, const int64_t* offsets, void* ws, cudaStream_t s) {
  const ProductLayout L = ProductLayout::make(R, d_from, d_to, K, xdtype);
  gmm_status r = list_tiles(offsets, K, R, kT, ws, L, s);
  if (r != GMM_OK || R == 0) return r;
  const dim3 grid((unsigned)ProductLayout::most_tiles(R, K, kT), (d_to + kT - 1) / kT);
  ProfScope p(dx ? "rows_simt_kernel(dx)" : "rows_simt_kernel", s);
  const int32_t* count = at<int32_t>(ws, L.off_count);
  const int4* tiles = at<int4>(ws, L.off_tiles);
  if (dx) rows_simt_kernel<T, true><<<grid, 256, 0, s>>>((const T*)A, (const T*)W, (T*)Y, d_from, d_to, count, tiles);
  else rows_simt_kernel<T, false><<<grid, 256, 0, s>>>((const T*)A, (const T*)W, (T*)Y, d_from, d_to, count, tiles);
  return launched();
}

template <typename T, typename TO>
gmm_status weights_simt(const void* dY, const void* A, void* dW, int64_t R, int d_in, int d_out,
                        int K, const int64_t* offsets, cudaStream_t s) {
  const dim3 grid((d_out + kT - 1) / kT, (d_in + kT - 1) / kT, K < 65535 ? K : 65535);
  ProfScope p("weights_simt_kernel", s);
  weights_simt_kernel<T, TO><<<grid, 256, 0, s>>>((const T*)dY, (const T*)A, (TO*)dW, d_in, d_out,
                                                  K, offsets, R);
  return launched();
}

gmm_status rows_product(const void* A, int xdtype, const void* W, void* Y, int64_t R, int d_from,
                        int d_to, int K, bool dx, const int64_t* offsets, void* ws,
                        cudaStream_t s) {
  const bool tc = tc_product_ok(xdtype, R, d_from, d_to, A, W, Y);
  if (tc && !dx && few_rows(R, K))
    return few_rows_product(A, xdtype, W, Y, R, d_from, d_to, K, offsets, s);
  if (tc)
    return tc_rows(A, xdtype, W, Y, R, d_from, d_to, K, dx, offsets, ws, s);
  if ((d_to + kT - 1) / kT > 65535) return GMM_ERR_UNSUPPORTED;
  switch (xdtype) {
    case GMM_F32: return rows_simt<float>(A, xdtype, W, Y, R, d_from, d_to, K, dx, offsets, ws, s);
    case GMM_F16: return rows_simt<__half>(A, xdtype, W, Y, R, d_from, d_to, K, dx, offsets, ws, s);
    default: return rows_simt<__nv_bfloat16>(A, xdtype, W, Y, R, d_from, d_to, K, dx, offsets, ws, s);
  }
}

}  // namespace

gmm_status list_tiles(const int64_t* offsets, int K, int64_t R, int T, void* ws,
                      const ProductLayout& L, cudaStream_t s) {
  ProfScope p("tile_list_kernel", s);
  tile_list_kernel<<<1, kListThreads, 0, s>>>(
      offsets, K, R, T, (uint32_t)ProductLayout::most_tiles(R, K, T), at<int32_t>(ws, L.off_count),
      at<uint32_t>(ws, L.off_first), at<int4>(ws, L.off_tiles));
  return launched();
}


}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_expert_ws_bytes(int64_t R, int d_in, int d_out, int K, gmm_dtype xdtype) {
  if (!sizes_ok(xdtype, R, d_in, d_out, K)) return 0;
  return ProductLayout::make(R, d_in, d_out, K, xdtype).bytes;
}

gmm_status gmm_expert_product(const void* A, gmm_dtype xdtype, int64_t R, int d_in, int d_out,
                              int K, const int64_t* offsets, const void* W, void* Y, void* ws,
                              size_t ws_bytes, void* stream) {
  const gmm_status r = check(xdtype, R, d_in, d_out, K, offsets, A, Y, W, ws, ws_bytes);
  if (r != GMM_OK) return r;
  return rows_product(A, xdtype, W, Y, R, d_in, d_out, K, false, offsets, ws, (cudaStream_t)stream);
}

gmm_status gmm_expert_product_dx(const void* dY, gmm_dtype xdtype, int64_t R, int d_in, int d_out,
                                 int K, const int64_t* offsets, const void* W, void* dA, void* ws,
                                 size_t ws_bytes, void* stream) {
  const gmm_status r = check(xdtype, R, d_in, d_out, K, offsets, dY, dA, W, ws, ws_bytes);
  if (r != GMM_OK) return r;
  return rows_product(dY, xdtype, W, dA, R, d_out, d_in, K, true, offsets, ws, (cudaStream_t)stream);
}

gmm_status gmm_expert_product_dw(const void* dY, const void* A, gmm_dtype xdtype, int64_t R,
                                 int d_in, int d_out, int K, const int64_t* offsets, void* dW,
                                 gmm_dtype wdtype, void* ws, size_t ws_bytes, void* stream) {
  gmm_status r = check(xdtype, R, d_in, d_out, K, offsets, dY, A, dW, ws, ws_bytes);
  if (r != GMM_OK) return r;
  if ((wdtype != xdtype && wdtype != GMM_F32) || (uintptr_t)dW % dtype_size(wdtype))
    return GMM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (R > 0 && tc_product_ok(xdtype, R, d_in, d_out, dY, A, dW))
    return tc_weights(dY, A, xdtype, R, d_in, d_out, K, offsets, dW, wdtype, ws, s);
  if ((d_in + kT - 1) / kT > 65535) return GMM_ERR_UNSUPPORTED;
  if (xdtype == GMM_F32) return weights_simt<float, float>(dY, A, dW, R, d_in, d_out, K, offsets, s);
  if (xdtype == GMM_F16) {
    if (wdtype == GMM_F32) return weights_simt<__half, float>(dY, A, dW, R, d_in, d_out, K, offsets, s);
    return weights_simt<__half, __half>(dY, A, dW, R, d_in, d_out, K, offsets, s);
  }
  if (wdtype == GMM_F32) return weights_simt<__nv_bfloat16, float>(dY, A, dW, R, d_in, d_out, K, offsets, s);
  return weights_simt<__nv_bfloat16, __nv_bfloat16>(dY, A, dW, R, d_in, d_out, K, offsets, s);
}

}  // extern "C"
