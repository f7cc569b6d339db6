// gate_rows.cu - a learned gate: entry points, and what follows its kernels
// (gate_rows.cuh, gate_grad.cuh).
#include "gate_grad.cuh"
#include "gate_rows.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kFinishThreads = 1024;
inline int finish_columns(int blocks, int K) { return blocks > 64 || K < 4096 ? 8 : 64; }

size_t ws_layout(int64_t N, int K, void* base, GateWs* w) {
  const int most = gate_blocks(K);
  const int64_t b = N < 1 ? 1 : N < most ? N : most;
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o += align_up(n); return (char*)base + at; };
  GateWs t;
  t.ticket = (uint32_t*)take(4);
  t.part = (double*)take(sizeof(double) * ((K + 7) / 8));
  const int64_t heads = b > kGateStreamGrid ? b : kGateStreamGrid;  // streamed rows have more blocks than sums
  t.rows = (int32_t*)take(sizeof(int32_t) * heads);
  t.kept = (int32_t*)take(sizeof(int32_t) * heads);
  t.mass = (float*)take(sizeof(float) * (size_t)b * K);
  t.counts = (int32_t*)take(sizeof(int32_t) * (size_t)b * K);
  t.scale = (float2*)take(sizeof(float2) * (size_t)(K > 16 * kGateBlockThreads ? N : 0));
  if (w) *w = t;
  return o;
}

// The blocks' sums in a fixed order, 8 columns a block (a sector), of few blocks
// 64: the threads of a column over the blocks, then a warp for each.  The last
// block to end adds up the loss.
template <int kFinishColumns>
__global__ void __launch_bounds__(kFinishThreads)
gate_finish_kernel(GateWs ws, GateBlocks blocks, int K, int64_t* __restrict__ counts, float* __restrict__ mass,
                   float* __restrict__ share, float* __restrict__ loss) {
  constexpr int kFinishRows = kFinishThreads / kFinishColumns;
  __shared__ Sum2 sums[kFinishRows][kFinishColumns + 1];
  __shared__ double terms[64];
  __shared__ int numbers[kFinishRows][kFinishColumns + 1], heads[2][32];
  __shared__ bool last;
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int column = threadIdx.x % kFinishColumns, row = threadIdx.x / kFinishColumns;
  const int k = blockIdx.x * kFinishColumns + column;
  Sum2 sum;
  int n = 0, rows = 0, all = 0;
  wait_for_last();
  for (int b = threadIdx.x; b < blocks.heads; b += kFinishThreads) rows += ws.rows[b], all += ws.kept[b];
  if (k < K) {
#pragma unroll 4
    for (int b = row; b < blocks.mass; b += kFinishRows) sum.add(ws.mass[(size_t)b * K + k]);
#pragma unroll 4
    for (int b = row; b < blocks.counts; b += kFinishRows) n += ws.counts[(size_t)b * K + k];
  }
  sums[row][column] = sum;
  numbers[row][column] = n;
  rows = __reduce_add_sync(0xffffffffu, rows);
  all = __reduce_add_sync(0xffffffffu, all);
  if (l == 0) heads[0][w] = rows, heads[1][w] = all;
  __syncthreads();
  for (int v = w; v < kFinishColumns; v += 32) {
    rows = __reduce_add_sync(0xffffffffu, heads[0][l]);
    all = __reduce_add_sync(0xffffffffu, heads[1][l]);
    double s = 0.0;
    n = 0;
#pragma unroll
    for (int i = l; i < kFinishRows; i += 32) s += sums[i][v].value(), n += numbers[i][v];
    s = warp_reduce(s, SumOp());
    n = __reduce_add_sync(0xffffffffu, n);
    const int c = blockIdx.x * kFinishColumns + v;
    if (l == 0) {
      double f = 0.0;
      if (c < K) {
        f = rows > 0 && all > 0 ? (double)K * n / ((double)all * rows) : 0.0;
        counts[c] = n;
        mass[c] = (float)s;
        share[c] = (float)f;
        f *= s;
      }
      terms[v] = f;
    }
  }
  __syncthreads();
  if (w != 0) return;
  double s = warp_reduce((l < kFinishColumns ? terms[l] : 0.0) + (l + 32 < kFinishColumns ? terms[l + 32] : 0.0), SumOp());
  if (gridDim.x == 1) {
    if (l == 0) *loss = (float)s;
    return;
  }
  if (l == 0) {
    ws.part[blockIdx.x] = s;
    __threadfence();
    last = atomicAdd(ws.ticket, 1u) == gridDim.x - 1;
  }
  __syncwarp();
  if (!last) return;
  __threadfence();
  s = 0.0;
  for (int b = l; b < gridDim.x; b += 32) s += __ldcg(ws.part + b);
  s = warp_reduce(s, SumOp());
  if (l == 0) *loss = (float)s;
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
  GateBlocks blocks;
  {
    ProfScope p("gate_kernel", s);
    blocks = xdtype == GMM_F32   ? launch_gate_f32(a, s)
             : xdtype == GMM_F16 ? launch_gate_f16(a, s)
                                 : launch_gate_bf16(a, s);
  }
  if (!blocks.heads) return GMM_ERR_CUDA;
  if (outs) {
    ProfScope p("gate_finish_kernel", s);
    const int columns = finish_columns(blocks.mass, K), g = (K + columns - 1) / columns;
    if (columns == 8)
      launch_behind(gate_finish_kernel<8>, g, kFinishThreads, s, w, blocks, K, counts, mass, share, loss);
    else
      launch_behind(gate_finish_kernel<64>, g, kFinishThreads, s, w, blocks, K, counts, mass, share, loss);
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
  const GradArgs a{L, live, ids, gamma, dgamma, share, dL, N, K, m, flags & GMM_GATE_NORMALISED, (float)coef};
  const bool ok = xdtype == GMM_F32   ? launch_grad_f32(a, s)
                  : xdtype == GMM_F16 ? launch_grad_f16(a, s)
                                      : launch_grad_bf16(a, s);
  return ok ? launched() : GMM_ERR_CUDA;
}

}  // extern "C"
