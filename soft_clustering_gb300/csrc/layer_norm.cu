// layer_norm.cu - layer norm of rows, and its gradients.
//
//   h = (x - mean) rstd,  y = w h + b
//   dx = (g - mean(g) - h mean(g h)) rstd,  g = w dy;  dw = sum dy h,  db = sum dy
//
// A row stays in the registers of its team from the load to the store, and the
// team's next row is fetched before this one is worked on.  Rows of up to 16
// elements a lane belong to a warp or a part of it, longer ones to a block of up
// to 512 threads, those beyond 8192 to a cluster of 2 or 4 blocks (rather than
// 1024 threads, whose 64 registers do not hold 16 elements, their weights and
// sums).  A lane has the same columns of every row: it keeps their weights, and in the gradient their sums over rows; the
// blocks' sums are joined in order by a second launch.
//
// The variance is taken about the mean, and what rounding left of the mean goes
// out with the same sums (sum d, sum d^2 over d = x - mean', and in the gradient
// sum g, sum g d): two rounds over the team a row.
//
// Bound by HBM: 2000003 rows of 128 f16 166 to 189 us from run to run (6.2 to 5.4
// TB/s), gradients of 65536 rows of 4096 bf16 277 us (5.8 TB/s; 8 elements a
// thread, twice the threads: 358).  Beyond 8192 the clusters' barriers are the
// bound: gradients of 8192 rows of 16384 bf16 335 us (2.4 TB/s).
#include "gate_internal.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kMaxD = 32768;
constexpr int kWarpThreads = 256;
constexpr int kWarpD = 512;        // longest row of a warp
constexpr int kBlockThreads = 512;
constexpr int kBlockD = 16 * kBlockThreads;
constexpr int kFinishColumns = 32;
constexpr int kFinishThreads = 1024;

struct Args {
  const void *X, *dY, *weight, *bias;
  void* Y;      // or dX
  float* sums;  // blocks * 2 * D
  int64_t N;
  int D;
  float eps;
};

// Takes a row's deviations from the mean into x, and its 1 / sigma; of the
// gradient also sum g and sum g h over the row's means.
template <bool GRAD, typename Team, int V, int P>
__device__ __forceinline__ void statistics(Team& team, float2 (&x)[P], const float2 (&y)[P],
                                           const float2 (&w)[P], float inv, int nv, bool full, float eps, float& rstd, float& mg,
                                           float& mgh) {
  float2 t = x[0];
#pragma unroll
  for (int i = 1; i < P; ++i) t = add2(t, x[i]);
  float s[1] = {t.x + t.y};
  team.sum(s);
  const float2 mean = both(s[0] * inv);
  if (!full) {  // columns past the row's: no deviation
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!inside<V>(2 * i, team.lane, team.size, nv)) x[i].x = mean.x;
      if (!inside<V>(2 * i + 1, team.lane, team.size, nv)) x[i].y = mean.y;
    }
  }
  float2 q0 = both(0.f), q1 = q0, q2 = q0, q3 = q0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    x[i] = sub2(x[i], mean);
    q0 = add2(q0, x[i]);
    q1 = fma2(x[i], x[i], q1);
    if (GRAD) {
      const float2 g = mul2(y[i], w[i]);
      q2 = add2(q2, g);
      q3 = fma2(g, x[i], q3);
    }
  }
  float left;
  if constexpr (GRAD) {
    float q[4] = {q0.x + q0.y, q1.x + q1.y, q2.x + q2.y, q3.x + q3.y};
    team.sum(q);
    left = q[0] * inv;
    const float var = q[1] * inv - left * left;
    rstd = rsqrtf((var < 0.f ? 0.f : var) + eps);  // not fmaxf: a NaN stays one
    mg = q[2] * inv;
    mgh = (q[3] * inv - left * mg) * rstd;
  } else {
    float q[2] = {q0.x + q0.y, q1.x + q1.y};
    team.sum(q);
    left = q[0] * inv;
    const float var = q[1] * inv - left * left;
    rstd = rsqrtf((var < 0.f ? 0.f : var) + eps);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = sub2(x[i], both(left));
}

// Rows n, n + stride, ... of the team; `end`: the first of its warp's, so that
// all lanes of a warp take the same number of turns.
template <typename T, typename W, int V, int NV, typename Team>
__device__ __forceinline__ void norm_rows(const Args& a, char* smem, Team team, int64_t n, int64_t stride,
                                          int64_t end) {
  constexpr int P = V * NV / 2;
  const int D = a.D, nv = D / V;
  const bool full = nv == NV * team.size;
  const float inv = 1.f / D;
  const T zero = from_f<T>(0.f);
  const int64_t step = (int64_t)stride * D;
  T* Y = (T*)a.Y + (int64_t)n * D;
  float2 w[P], b[P];
  load_columns<V, NV>(w, (const W*)a.weight, team.lane, team.size, nv, 1.f);
  load_columns<V, NV>(b, (const W*)a.bias, team.lane, team.size, nv, 0.f);
  Feed<T, V, NV, 1> feed;
  feed.start(smem, {(const T*)a.X}, n, stride, a.N, D, team.lane, team.size, nv, zero);
  for (; end < a.N; n += stride, end += stride) {
    Row<T, V, NV> row[1];
    feed.next(row);
    float2 x[P];
    row[0].get(x);
    float rstd, mg, mgh;
    statistics<false, Team, V>(team, x, x, x, inv, nv, full, a.eps, rstd, mg, mgh);
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = fma2(mul2(x[i], both(rstd)), w[i], b[i]);
    row[0].set(x);
    if (n < a.N) row[0].store(Y, team.lane, team.size, nv);
    Y += step;
  }
}

// Lanes of a warp: 32 / size rows at a time.
template <typename T, typename W, int V, int NV>
__global__ void __launch_bounds__(kWarpThreads) norm_warp_kernel(Args a, int size) {
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31, per = 32 / size;
  const uint32_t warp = (blockIdx.x * kWarpThreads + threadIdx.x) >> 5;
  const uint32_t warps = gridDim.x * (kWarpThreads / 32);
  norm_rows<T, W, V, NV>(a, smem, WarpTeam<0>(lane & (size - 1), size), warp * per + lane / size, warps * per,
                         warp * per);
}

template <typename T, typename W, int V, int NV, bool CLUSTER>
__global__ void __launch_bounds__(kBlockThreads) norm_block_kernel(Args a, int blocks) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[BlockTeam<CLUSTER>::kWords];
  const uint32_t c = blockIdx.x / blocks;
  if (CLUSTER) cluster_barrier();  // every block of the cluster runs
  norm_rows<T, W, V, NV>(a, smem, BlockTeam<CLUSTER>(part, blockDim.x), c, gridDim.x / blocks, c);
  if (CLUSTER) cluster_barrier();  // nothing is on its way to a block that has ended
}

template <typename T, typename W, int V, int NV, typename Team>
__device__ __forceinline__ void grad_rows(const Args& a, char* smem, Team team, int64_t n, int64_t stride,
                                          int64_t end, float2 (&dw)[V * NV / 2], float2 (&db)[V * NV / 2]) {
  constexpr int P = V * NV / 2;
  const int D = a.D, nv = D / V;
  const bool full = nv == NV * team.size;
  const float inv = 1.f / D;
  const T zero = from_f<T>(0.f);
  const int64_t step = (int64_t)stride * D;
  T* dX = a.Y ? (T*)a.Y + (int64_t)n * D : nullptr;
  float2 w[P];
  load_columns<V, NV>(w, (const W*)a.weight, team.lane, team.size, nv, 1.f);
#pragma unroll
  for (int i = 0; i < P; ++i) dw[i] = db[i] = both(0.f);
  Feed<T, V, NV, 2> feed;
  feed.start(smem, {(const T*)a.X, (const T*)a.dY}, n, stride, a.N, D, team.lane, team.size, nv, zero);
  for (; end < a.N; n += stride, end += stride) {
    Row<T, V, NV> row[2];
    feed.next(row);
    float2 x[P], y[P];
    row[0].get(x);
    row[1].get(y);
    float rstd, mg, mgh;
    statistics<true, Team, V>(team, x, y, w, inv, nv, full, a.eps, rstd, mg, mgh);
    if (n < a.N) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 h = mul2(x[i], both(rstd));
        dw[i] = fma2(y[i], h, dw[i]);
        db[i] = add2(db[i], y[i]);
        x[i] = mul2(fma2(h, both(-mgh), fma2(y[i], w[i], both(-mg))), both(rstd));
      }
      if (dX) {
        row[0].set(x);
        row[0].store(dX, team.lane, team.size, nv);
      }
    }
    if (dX) dX += step;
  }
}

template <typename T, typename W, int V, int NV>
__global__ void __launch_bounds__(kWarpThreads) norm_grad_warp_kernel(Args a, int size) {
  extern __shared__ __align__(16) char smem[];
  constexpr int E = V * NV;
  __shared__ float cols[2 * kWarpD];
  const int lane = threadIdx.x & 31, per = 32 / size;
  const uint32_t warp = (blockIdx.x * kWarpThreads + threadIdx.x) >> 5;
  const uint32_t warps = gridDim.x * (kWarpThreads / 32);
  float2 dw[E / 2], db[E / 2];
  grad_rows<T, W, V, NV>(a, smem, WarpTeam<0>(lane & (size - 1), size), warp * per + lane / size, warps * per,
                         warp * per, dw, db);
  if (!a.sums) return;
  let_next_start();
  // the warp's groups, then the warps in order
#pragma unroll
  for (int i = 0; i < E / 2; ++i)
    for (int o = size; o < 32; o <<= 1) {
      dw[i].x += __shfl_xor_sync(0xffffffffu, dw[i].x, o);
      dw[i].y += __shfl_xor_sync(0xffffffffu, dw[i].y, o);
      db[i].x += __shfl_xor_sync(0xffffffffu, db[i].x, o);
      db[i].y += __shfl_xor_sync(0xffffffffu, db[i].y, o);
    }
  for (int turn = 0; turn < kWarpThreads / 32; ++turn) {
    if ((int)(threadIdx.x >> 5) == turn && lane < size) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = column<V>(i, lane, size);
        if (c < a.D) {
          cols[c] = (turn ? cols[c] : 0.f) + (i & 1 ? dw[i / 2].y : dw[i / 2].x);
          cols[kWarpD + c] = (turn ? cols[kWarpD + c] : 0.f) + (i & 1 ? db[i / 2].y : db[i / 2].x);
        }
      }
    }
    __syncthreads();
  }
  float* out = a.sums + (size_t)blockIdx.x * 2 * a.D;
  for (int c = threadIdx.x; c < a.D; c += kWarpThreads) {
    out[c] = cols[c];
    out[a.D + c] = cols[kWarpD + c];
  }
}

template <typename T, typename W, int V, int NV, bool CLUSTER>
__global__ void __launch_bounds__(kBlockThreads) norm_grad_block_kernel(Args a, int blocks) {
  extern __shared__ __align__(16) char smem[];
  constexpr int E = V * NV;
  __shared__ float part[BlockTeam<CLUSTER>::kWords];
  float2 dw[E / 2], db[E / 2];
  const uint32_t at = blockIdx.x / blocks;
  const BlockTeam<CLUSTER> team(part, blockDim.x);
  if (CLUSTER) cluster_barrier();  // every block of the cluster runs
  grad_rows<T, W, V, NV>(a, smem, team, at, gridDim.x / blocks, at, dw, db);
  if (a.sums) {
    let_next_start();
    float* out = a.sums + (size_t)at * 2 * a.D;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = column<V>(i, team.lane, team.size);
      if (c < a.D) {
        out[c] = i & 1 ? dw[i / 2].y : dw[i / 2].x;
        out[a.D + c] = i & 1 ? db[i / 2].y : db[i / 2].x;
      }
    }
  }
  if (CLUSTER) cluster_barrier();  // nothing is on its way to a block that has ended
}

// The blocks' sums in a fixed order, 32 columns a block: a warp reads 32 columns
// of every 32nd block, then each column has a warp of its own.
template <typename W>
__global__ void __launch_bounds__(kFinishThreads)
norm_finish_kernel(const float* __restrict__ sums, int blocks, int D, W* __restrict__ dweight,
                   W* __restrict__ dbias) {
  static_assert(kFinishThreads == 32 * kFinishColumns, "a warp a column");
  __shared__ Sum2 part[32][kFinishColumns + 1];
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * kFinishColumns + l;
  Sum2 s;
  wait_for_last();
  if (i < 2 * D)
#pragma unroll 4
    for (int b = w; b < blocks; b += 32) s.add(sums[(size_t)b * 2 * D + i]);
  part[w][l] = s;
  __syncthreads();
  const float sum = warp_reduce(part[l][w].s, SumOp()), left = warp_reduce(part[l][w].left, SumOp());
  const float all = isfinite(sum) ? sum + left : sum;
  const int c = blockIdx.x * kFinishColumns + w;
  if (l == 0 && c < 2 * D) {
    if (c < D) dweight[c] = from_f<W>(all);
    else dbias[c - D] = from_f<W>(all);
  }
}

bool norm_ok(int xdtype, int64_t N, int D, double eps, int wdtype) {
  return dtype_ok(xdtype) && (wdtype == xdtype || wdtype == GMM_F32) && N >= 0 && N <= INT32_MAX &&
         D >= 1 && eps >= 0.0 && eps < INFINITY;
}

// Blocks for N rows: at most what the device holds at once, so that a block's
// sums run over as many rows as they can.
int64_t grid_for(int64_t rows_in_blocks, int resident) {
  const int64_t most = (int64_t)kSms * resident;
  return rows_in_blocks < 1 ? 1 : rows_in_blocks < most ? rows_in_blocks : most;
}

struct Plan {
  int size;      // lanes of a row; 0: a block or a cluster
  int per;       // elements a lane: 8 or 16
  int threads;
  int blocks;    // of a row
  int64_t grid;  // rows at a time for the latter, blocks of warps
};
Plan plan(int64_t N, int D, int V) {
  Plan p;
  p.blocks = 1;
  if (D <= kWarpD) {
    p.per = D <= (V == 1 ? 256 : 8) ? 8 : 16;
    p.size = 1;
    // as few lanes as hold the row; single elements are read as many at a time
    // as the row has
    while (p.size < 32 && p.size * (V == 1 ? 1 : p.per) < D) p.size <<= 1;
    p.threads = kWarpThreads;
    const int64_t rows = kWarpThreads / p.size;
    p.grid = grid_for((N + rows - 1) / rows, 4);
    return p;
  }
  p.size = 0;
  p.per = 16;
  while (D > p.blocks * kBlockD) p.blocks *= 2;
  p.threads = ((D + p.per * p.blocks - 1) / (p.per * p.blocks) + 31) / 32 * 32;
  const int resident = 1024 / p.threads;
  p.grid = grid_for(N, resident > 8 ? 8 : resident);
  if (p.blocks > 1 && p.grid > kSms * 2 / p.blocks) p.grid = kSms * 2 / p.blocks;
  return p;
}

template <typename T, typename W, int V, int NV, bool GRAD>
bool launch_rows(const Args& a, Plan& p, cudaStream_t s) {
  static std::atomic<uint64_t> done[3];
  static ResidentCache cache[3];
  const size_t smem = Feed<T, V, NV, GRAD ? 2 : 1>::bytes(p.threads);
  const int form = p.size ? 0 : p.blocks == 1 ? 1 : 2;
  void (*kernel)(Args, int);
  if constexpr (V * NV < 16)  // short rows alone
    {
    if constexpr (GRAD) kernel = norm_grad_warp_kernel<T, W, V, NV>;
    else kernel = norm_warp_kernel<T, W, V, NV>;
  }
  else if constexpr (GRAD)
    kernel = form == 0   ? norm_grad_warp_kernel<T, W, V, NV>
             : form == 1 ? norm_grad_block_kernel<T, W, V, NV, false>
                         : norm_grad_block_kernel<T, W, V, NV, true>;
  else
    kernel = form == 0   ? norm_warp_kernel<T, W, V, NV>
             : form == 1 ? norm_block_kernel<T, W, V, NV, false>
                         : norm_block_kernel<T, W, V, NV, true>;
  if (smem > 48 * 1024 - 8192 &&
      !allow_smem((const void*)kernel, Feed<T, V, NV, GRAD ? 2 : 1>::bytes(kBlockThreads), done[form]))
    return false;
  const int64_t most = resident(kernel, p.threads, smem, cache[form]) / p.blocks;
  if (p.grid > most) p.grid = most;
  if (form == 2) launch_clusters(kernel, (unsigned)p.grid * p.blocks, p.threads, smem, p.blocks, s, a, p.blocks);
  else kernel<<<(unsigned)p.grid, p.threads, smem, s>>>(a, form ? 1 : p.size);
  return true;
}

template <typename T, typename W, int V, bool GRAD>
bool launch(const Args& a, Plan& p, cudaStream_t s) {
  return p.per == 8 ? launch_rows<T, W, V, 8 / V, GRAD>(a, p, s) : launch_rows<T, W, V, 16 / V, GRAD>(a, p, s);
}

template <typename T, typename W, bool GRAD>
bool launch_typed(const Args& a, cudaStream_t s, int64_t& blocks) {
  const bool vectors = wide<T>(a.D, (const char*)a.X, (const char*)a.dY, (const char*)a.Y);
  Plan p = plan(a.N, a.D, vectors ? kWide<T> : 1);
  const bool ok = vectors ? launch<T, W, kWide<T>, GRAD>(a, p, s) : launch<T, W, 1, GRAD>(a, p, s);
  blocks = p.grid;
  return ok;
}

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
  const Args a{X, nullptr, weight, bias, Y, nullptr, N, D, (float)eps};
  int64_t blocks;
  bool ok;
  ProfScope p("norm_kernel", s);
#define CALL(T, W) ok = launch_typed<T, W, false>(a, s, blocks)
  BY_TYPES(CALL)
#undef CALL
  return ok ? launched() : GMM_ERR_CUDA;
}

size_t gmm_layer_norm_ws_bytes(int D) {
  if (D < 1 || D > kMaxD) return 0;
  const int64_t most = INT32_MAX;  // rows that fill the device
  const int64_t b1 = plan(most, D, 1).grid, b8 = plan(most, D, 8).grid, b4 = plan(most, D, 4).grid;
  const int64_t b = b1 > b8 ? (b1 > b4 ? b1 : b4) : (b8 > b4 ? b8 : b4);
  return align_up(sizeof(float) * 2 * (size_t)D * b);
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
  const Args a{X, dY, weight, nullptr, dX, dweight ? (float*)ws : nullptr, N, D, (float)eps};
  int64_t blocks = 0;
  if (N > 0) {
    ProfScope p("norm_grad_kernel", s);
    bool ok;
#define CALL(T, W) ok = launch_typed<T, W, true>(a, s, blocks)
    BY_TYPES(CALL)
#undef CALL
    if (!ok) return GMM_ERR_CUDA;
  }
  if (dweight) {
    ProfScope p("norm_finish_kernel", s);
    const unsigned g = (unsigned)((2 * (int64_t)D + kFinishColumns - 1) / kFinishColumns);
#define CALL(T, W) launch_behind(norm_finish_kernel<W>, g, kFinishThreads, s, (const float*)ws, (int)blocks, D, (W*)dweight, (W*)dbias)
    BY_TYPES(CALL)
#undef CALL
  }
  return launched();
}

}  // extern "C"
