// gate_distill.cu - distillation from a teacher's top entries.
//
//   row_n = w T^2 sum_t q_t (log q_t - log p[ids_t]),  loss = scale sum_n row_n
//   dL    = scale w T (p - q)
//
// One pass over the logits: a row stays in registers from its load to the
// gradient's store.  Rows of up to 512 logits belong to lanes of a warp, of up
// to 8192 to a block, 16 logits a thread; longer ones are streamed by a block
// twice, the second time out of L2.  The gradient is stored as p alone first;
// the lane that holds a teacher's entry puts that element right afterwards,
// from the logit that it read with the entry.  All exponents are of base 2.
#include "gate_internal.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kWarpThreads = 256;
constexpr int kWarpK = 512;
constexpr int kBlockThreads = 512;
constexpr int kBlockK = 16 * kBlockThreads;
constexpr int kMaxGrid = 8 * kSms;
constexpr int kStudent = 1 << 18;

struct Args {
  const void* L;
  const int32_t* ids;
  const float *values, *weights;
  float* rows;
  void* dL;
  double* part;  // a sum for each block
  int64_t N;
  int K, m, gammas, add;
  float T, inv, scale;
};

// A teacher's entries of one row, MT a lane of the `size` (a power of two) that
// share them, entry i * size + lane in place i.
template <int MT>
struct Entries {
  int id[MT];     // -1: none
  float b[MT];    // log2 q, but for a constant
  float x[MT];    // the student's logit
  float old[MT];  // what the gradient is added to
  float q[MT];

  template <typename T>
  __device__ __forceinline__ void load(const Args& a, int64_t n, bool on, int lane, int size) {
    const T* L = (const T*)a.L + n * a.K;
    const T* dL = (const T*)a.dL + n * a.K;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int t = i * size + lane;
      id[i] = -1;
      float v = 0.f;
      if (on && t < a.m) {
        id[i] = a.ids[n * a.m + t];
        v = a.values[n * a.m + t];
      }
      if ((uint32_t)id[i] >= (uint32_t)a.K) id[i] = -1;
      b[i] = (a.gammas ? log2f(v) : v * kLog2E) * a.inv;
      if (id[i] < 0 || b[i] == -INFINITY) id[i] = -1, b[i] = -INFINITY;
      x[i] = old[i] = 0.f;
      if (id[i] >= 0) {
        x[i] = to_f(L[id[i]]);
        if (a.add) old[i] = to_f(dL[id[i]]);
      }
    }
  }
  // q, and whether there is an entry.
  __device__ __forceinline__ bool normalise(WarpTeam team, float& logsum) {
    float top = b[0];
#pragma unroll
    for (int i = 1; i < MT; ++i) top = max_nan(top, b[i]);
    top = team.top(top);
    const bool some = top != -INFINITY;
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      b[i] -= some ? top : 0.f;
      q[i] = ex2(b[i]);
      s[0] += q[i];
    }
    team.sum(s);
    logsum = log2f(s[0]);
#pragma unroll
    for (int i = 0; i < MT; ++i) q[i] = some ? q[i] / s[0] : 0.f;
    return some;
  }
  // sum_t q_t (b_t - (x_t - top) k)
  __device__ __forceinline__ float divergence(WarpTeam team, float top, float k) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0 && q[i] != 0.f) s[0] += q[i] * (b[i] - (x[i] - top) * k);
    team.sum(s);
    return s[0];
  }
  // The gradient's elements at the entries, c (p - q) with the q of every entry
  // of that element, into q; the id stays with the first of them alone.
  __device__ __forceinline__ void gradient(WarpTeam team, int m, float c, float top, float k, float sum) {
    const int l = threadIdx.x & 31, base = l & ~(team.size - 1);
    float w[MT];
    bool first[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) w[i] = q[i], first[i] = true;
    bool twice = MT > 1;
    if (MT == 1) {
      const unsigned same = __match_any_sync(0xffffffffu, id[0] >= 0 ? id[0] << 5 | base : -1 - l);
      twice = __any_sync(0xffffffffu, (same & (same - 1)) != 0);
    }
    if (twice) {
#pragma unroll
      for (int i = 0; i < MT; ++i) w[i] = 0.f;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (j * team.size >= m) break;
        for (int o = 0; o < team.size; ++o) {
          const int id_o = __shfl_sync(0xffffffffu, id[j], base + o);
          const float q_o = __shfl_sync(0xffffffffu, q[j], base + o);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            if (id_o == id[i]) {
              w[i] += q_o;
              if (j < i || (j == i && o < team.lane)) first[i] = false;
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const float p = sum == 0.f ? 0.f : ex2((x[i] - top) * k) / sum;
      q[i] = fmaf(c, p - w[i], old[i]);
      if (!first[i]) id[i] = -1;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* d) const {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) d[id[i]] = from_f<T>(q[i]);
  }
};

// Sums of the threads' row losses, in the order of the threads.
__device__ __forceinline__ void store_total(const Args& a, double total) {
  __shared__ double part[32];
  total = block_reduce(total, 0.0, SumOp(), part);
  if (threadIdx.x == 0) a.part[blockIdx.x] = total;
}

__device__ __forceinline__ float row_loss(const Args& a, float w, float divergence, float logsum, float sum) {
  // a row with no student at all is infinitely far
  if (sum == 0.f) return w * INFINITY;
  return w * a.T * a.T * kLn2 * (divergence - logsum + log2f(sum));
}

template <typename T, int V, int NV, int MT>
__global__ void __launch_bounds__(kWarpThreads) distill_warp_kernel(Args a, int size) {
  extern __shared__ __align__(16) char smem[];
  constexpr int P = V * NV / 2;
  const int l = threadIdx.x & 31, per = 32 / size, K = a.K, nv = K / V;
  const int64_t warp = ((int64_t)blockIdx.x * kWarpThreads + threadIdx.x) >> 5;
  const int64_t stride = (int64_t)gridDim.x * (kWarpThreads / 32) * per;
  WarpTeam team{l & (size - 1), size};
  const float k = kLog2E * a.inv;
  const T none = from_f<T>(-INFINITY);
  int64_t n = warp * per + l / size;
  Feed<T, V, NV, 1, WeightedRows> feed;
  feed.start(smem, {(const T*)a.L}, n, stride, a.N, K, team.lane, size, nv, none, WeightedRows{a.weights});
  double total = 0.0;
  for (int64_t end = warp * per; end < a.N; n += stride, end += stride) {
    Row<T, V, NV> row[1], old;
    const bool on = feed.next(row);
    const float w = on ? (a.weights ? a.weights[n] : 1.f) : 0.f;
    Entries<MT> e;
    e.template load<T>(a, n, on, team.lane, size);
    T* d = (T*)a.dL + n * K;
    if (a.add && n < a.N) old.read(d, team.lane, size, nv);
    float logsum;
    const bool some = e.normalise(team, logsum);
    float top = team.top(lane_max(row[0]));
    if (top == -INFINITY) top = 0.f;
    float2 x[P];
    row[0].get(x);
    exponentials(x, top, k);
    float2 t = x[0];
#pragma unroll
    for (int i = 1; i < P; ++i) t = add2(t, x[i]);
    float s[1] = {t.x + t.y};
    team.sum(s);
    const float divergence = e.divergence(team, top, k);
    if (team.lane == 0 && n < a.N) {
      const float r = on && some ? row_loss(a, w, divergence, logsum, s[0]) : 0.f;
      a.rows[n] = r;
      total += r;
    }
    if (!a.dL) continue;
    const float c = a.scale * w * a.T;
    e.gradient(team, a.m, c, top, k, s[0]);
    const float f = s[0] == 0.f ? 0.f : c / s[0];
    if (n < a.N && (!a.add || (on && some))) {
      if (a.add) {
        float2 o[P];
        old.get(o);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = fma2(x[i], both(f), o[i]);
      } else if (on && some) {
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = mul2(x[i], both(f));
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = both(0.f);
      }
      row[0].set(x);
      row[0].store(d, team.lane, size, nv);
    }
    __syncwarp();
    e.store(d);
  }
  store_total(a, total);
}

// The first warp has the entries.
template <typename T, int V, int NV, int MT>
__global__ void __launch_bounds__(kBlockThreads) distill_block_kernel(Args a, int) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[BlockTeam<false>::kWords];
  __shared__ int some_s[2];
  constexpr int P = V * NV / 2;
  const int K = a.K, nv = K / V;
  const bool teacher = threadIdx.x < 32;
  BlockTeam<false> team(part);
  const WarpTeam first{(int)threadIdx.x & 31, 32};
  const float k = kLog2E * a.inv;
  const T none = from_f<T>(-INFINITY);
  Feed<T, V, NV, 1, WeightedRows> feed;
  feed.start(smem, {(const T*)a.L}, blockIdx.x, gridDim.x, a.N, K, team.lane, team.size, nv, none,
             WeightedRows{a.weights});
  double total = 0.0;
  Entries<MT> late;  // elements to be put right once the row before is stored
#pragma unroll
  for (int i = 0; i < MT; ++i) late.id[i] = -1, late.q[i] = 0.f;
  uint32_t turn = 0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, turn ^= 1) {
    Row<T, V, NV> row[1], old;
    const bool on = feed.next(row);
    const float w = on ? (a.weights ? a.weights[n] : 1.f) : 0.f;
    T* d = (T*)a.dL + n * K;
    Entries<MT> e;
    float logsum = 0.f;
    if (teacher) e.template load<T>(a, n, on, first.lane, 32);
    if (a.add) old.read(d, team.lane, team.size, nv);
    float top = team.top(lane_max(row[0]));
    const float low = top == -INFINITY ? 0.f : top;
    float2 x[P];
    row[0].get(x);
    exponentials(x, low, k);
    float2 t = x[0];
#pragma unroll
    for (int i = 1; i < P; ++i) t = add2(t, x[i]);
    float s[1] = {t.x + t.y};
    if (teacher) {
      const bool some = e.normalise(first, logsum);
      if (threadIdx.x == 0) some_s[turn] = some;
    }
    const float own = team.join(s, top, k);
    if (top == -INFINITY) top = 0.f;
    const bool some = on && some_s[turn];
    const float c = a.scale * w * a.T;
    if (teacher) {
      if (a.dL) late.store(d - (int64_t)gridDim.x * K);  // that row was stored before the barrier
      const float divergence = e.divergence(first, top, k);
      if (threadIdx.x == 0) {
        const float r = some ? row_loss(a, w, divergence, logsum, s[0]) : 0.f;
        a.rows[n] = r;
        total += r;
      }
      if (a.dL) {
        e.gradient(first, a.m, c, top, k, s[0]);
        late = e;
      }
    }
    if (!a.dL || (a.add && !some)) continue;
    const float f = s[0] == 0.f ? 0.f : c * own / s[0];
    if (a.add) {
      float2 o[P];
      old.get(o);
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = fma2(x[i], both(f), o[i]);
    } else if (some) {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = mul2(x[i], both(f));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = both(0.f);
    }
    row[0].set(x);
    row[0].store(d, team.lane, team.size, nv);
  }
  __syncthreads();
  if (teacher && a.dL && blockIdx.x < a.N) {
    const int64_t last = blockIdx.x + (a.N - 1 - blockIdx.x) / gridDim.x * gridDim.x;
    late.store((T*)a.dL + last * K);
  }
  store_total(a, total);
}

// Rows that no block holds, at any address: 16-byte vectors between the row's
// first and last boundary, single elements before and behind.
template <typename T>
struct Cover {
  static constexpr int V = kWide<T>;
  const T* row;
  int shift, K, nv;  // elements before the row in its first vector; vectors
  __device__ __forceinline__ Cover(const T* p, int K_) : row(p), K(K_) {
    shift = (int)((uintptr_t)p / sizeof(T) % V);
    nv = (shift + K + V - 1) / V;
  }
  __device__ __forceinline__ bool whole(int v) const { return v * V >= shift && (v + 1) * V <= shift + K; }
  // Vector v of `p`, a row as this one but for its address.
  __device__ __forceinline__ void load(Vec<T, V>& x, const T* p, int v, T none, bool same = true) const {
    if (same && whole(v)) {
      x = *reinterpret_cast<const Vec<T, V>*>(p + v * V - shift);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = v * V + e - shift;
        x.v[e] = c >= 0 && c < K ? p[c] : none;
      }
    }
  }
  __device__ __forceinline__ void store(const Vec<T, V>& x, T* p, int v, bool same) const {
    if (same && whole(v)) {
      *reinterpret_cast<Vec<T, V>*>(p + v * V - shift) = x;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = v * V + e - shift;
        if (c >= 0 && c < K) p[c] = x.v[e];
      }
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kBlockThreads) distill_stream_kernel(Args a, int) {
  __shared__ float part[BlockTeam<false>::kWords];
  __shared__ int some_s;
  constexpr int V = kWide<T>, U = 4, MT = 2;
  const int K = a.K;
  const bool teacher = threadIdx.x < 32;
  BlockTeam<false> team(part);
  const WarpTeam first{(int)threadIdx.x & 31, 32};
  const float k = kLog2E * a.inv;
  const T none = from_f<T>(-INFINITY);
  double total = 0.0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    const float w = a.weights ? a.weights[n] : 1.f;
    const bool on = w != 0.f;
    const T* L = (const T*)a.L + n * K;
    T* d = (T*)a.dL + n * K;
    Entries<MT> e;
    float logsum = 0.f;
    if (teacher) {
      e.template load<T>(a, n, on, first.lane, 32);
      const bool some = e.normalise(first, logsum);
      if (threadIdx.x == 0) some_s = some;
    }
    const Cover<T> row(L, K);
    float top = -INFINITY;
    float2 sum = both(0.f);
    if (on)
      for (int v0 = threadIdx.x; v0 < row.nv; v0 += U * kBlockThreads) {
        Row<T, V, U> x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = v0 + u * kBlockThreads;
          if (v < row.nv) {
            row.load(x.r[u], L, v, none);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x.r[u].v[i] = none;
          }
        }
        const float m = max_nan(top, lane_max(x));
        if (m == -INFINITY) continue;
        sum = mul2(sum, both(ex2((top - m) * k)));
        top = m;
        float2 f[U * V / 2];
        x.get(f);
        exponentials(f, top, k);
#pragma unroll
        for (int i = 0; i < U * V / 2; ++i) sum = add2(sum, f[i]);
      }
    // the warp's, then the block's
    float s[1] = {sum.x + sum.y};
    const float lane_top = top;
    top = warp_max(top);
    if (lane_top != -INFINITY) s[0] *= ex2((lane_top - top) * k);
    team.join(s, top, k);
    if (top == -INFINITY) top = 0.f;
    const bool some = on && some_s;
    const float c = a.scale * w * a.T;
    if (teacher) {
      const float divergence = e.divergence(first, top, k);
      if (threadIdx.x == 0) {
        const float r = some ? row_loss(a, w, divergence, logsum, s[0]) : 0.f;
        a.rows[n] = r;
        total += r;
      }
      if (a.dL) e.gradient(first, a.m, c, top, k, s[0]);
    }
    if (a.dL && (!a.add || some)) {
      const float f = s[0] == 0.f ? 0.f : c / s[0];
      const bool same = (((uintptr_t)L ^ (uintptr_t)d) & 15) == 0;
      // backwards: what was read last is nearest
      const int turns = (row.nv + U * kBlockThreads - 1) / (U * kBlockThreads);
      for (int i = turns - 1; i >= 0; --i) {
        const int v0 = i * U * kBlockThreads + threadIdx.x;
        Row<T, V, U> x, o;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = v0 + u * kBlockThreads;
          if (v < row.nv) {
            if (some) row.load(x.r[u], L, v, none);
            if (a.add) row.load(o.r[u], d, v, none, same);
          }
        }
        float2 y[U * V / 2];
        if (some) {
          x.get(y);
          exponentials(y, top, k);
          float2 z[U * V / 2];
          o.get(z);
#pragma unroll
          for (int j = 0; j < U * V / 2; ++j) y[j] = a.add ? fma2(y[j], both(f), z[j]) : mul2(y[j], both(f));
        } else {
#pragma unroll
          for (int j = 0; j < U * V / 2; ++j) y[j] = both(0.f);
        }
        x.set(y);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = v0 + u * kBlockThreads;
          if (v < row.nv) row.store(x.r[u], d, v, same);
        }
      }
    }
    __syncthreads();
    if (teacher && a.dL) e.store(d);
  }
  store_total(a, total);
}

// The blocks' sums in order, in 64 bits.
__global__ void __launch_bounds__(kWarpThreads)
distill_finish_kernel(const double* __restrict__ part, int blocks, double scale,
                      float* __restrict__ loss) {
  __shared__ double partd[32];
  double s = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kWarpThreads) s += part[b];
  s = block_reduce(s, 0.0, SumOp(), partd);
  if (threadIdx.x == 0) *loss = (float)(s * scale);
}

template <typename T, int V, int NV, int MT>
bool launch_block(const Args& a, int threads, int64_t grid, cudaStream_t s) {
  static std::atomic<uint64_t> done;
  using F = Feed<T, V, NV, 1, WeightedRows>;
  if (F::bytes(threads) > 48 * 1024 - 4096 &&
      !allow_smem((const void*)distill_block_kernel<T, V, NV, MT>, F::bytes(kBlockThreads), done))
    return false;
  distill_block_kernel<T, V, NV, MT><<<(unsigned)grid, threads, F::bytes(threads), s>>>(a, 0);
  return true;
}
template <typename T, int V, int NV, int MT>
bool launch_warp(const Args& a, int size, int64_t grid, cudaStream_t s) {
  static std::atomic<uint64_t> done;
  using F = Feed<T, V, NV, 1, WeightedRows>;
  if (F::bytes(kWarpThreads) > 48 * 1024 - 4096 &&
      !allow_smem((const void*)distill_warp_kernel<T, V, NV, MT>, F::bytes(kWarpThreads), done))
    return false;
  distill_warp_kernel<T, V, NV, MT><<<(unsigned)grid, kWarpThreads, F::bytes(kWarpThreads), s>>>(a, size);
  return true;
}

// Returns the blocks launched; 0: none.
template <typename T, int V>
int64_t launch(const Args& a, cudaStream_t s) {
  const int K = a.K, m = a.m;
  if (K <= kWarpK) {
    const int per = K <= (V == 1 ? 256 : 8) ? 8 : 16;
    int size = 1;
    while (size < 32 && size * (V == 1 ? 1 : per) < K) size <<= 1;
    while (size * 8 < m) size <<= 1;  // at most eight entries a lane
    const int64_t rows = kWarpThreads / size, need = (a.N + rows - 1) / rows;
    const int64_t grid = need < 1 ? 1 : need < 4 * kSms ? need : 4 * kSms;
    const bool ok = per == 8 ? (m <= size ? launch_warp<T, V, 8 / V, 1>(a, size, grid, s)
                                          : launch_warp<T, V, 8 / V, 8>(a, size, grid, s))
                             : (m <= size ? launch_warp<T, V, 16 / V, 1>(a, size, grid, s)
                                          : launch_warp<T, V, 16 / V, 8>(a, size, grid, s));
    return ok ? grid : 0;
  }
  const int threads = ((K + 15) / 16 + 31) / 32 * 32;
  const int resident = 1024 / threads < 8 ? 1024 / threads : 8;
  const int64_t grid = a.N < 1 ? 1 : a.N < (int64_t)resident * kSms ? a.N : (int64_t)resident * kSms;
  const bool ok = m <= 32 ? launch_block<T, V, 16 / V, 1>(a, threads, grid, s)
                          : launch_block<T, V, 16 / V, 2>(a, threads, grid, s);
  return ok ? grid : 0;
}

template <typename T>
int64_t launch_typed(const Args& a, cudaStream_t s) {
  if (a.K > kBlockK) {
    const int64_t grid = a.N < 1 ? 1 : a.N < 2 * kSms ? a.N : 2 * kSms;
    distill_stream_kernel<T><<<(unsigned)grid, kBlockThreads, 0, s>>>(a, 0);
    return grid;
  }
  return wide<T>(a.K, (const char*)a.L, (const char*)a.dL) ? launch<T, kWide<T>>(a, s) : launch<T, 1>(a, s);
}

}  // namespace
}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_distill_ws_bytes(void) { return align_up(sizeof(double) * kMaxGrid); }

gmm_status gmm_distill(const void* L, gmm_dtype xdtype, int64_t N, int K, int m, int kind, int flags,
                       double temperature, double scale, const int32_t* ids, const float* values,
                       const float* weights, float* rows, float* loss, void* dL, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!dtype_ok(xdtype) || N < 0 || K < 1 || K > kStudent || m < 1 || m > gate::kMaxTeacher ||
      N > INT32_MAX / m || (kind != GMM_TEACHER_LOGITS && kind != GMM_TEACHER_GAMMA) ||
      (flags & ~GMM_DISTILL_ADD) || !((float)temperature > 0.f) ||
      !((float)temperature < INFINITY) || !loss || !ws)
    return GMM_ERR_INVALID_ARG;
  if (N > 0 && (!L || !ids || !values || !rows)) return GMM_ERR_INVALID_ARG;
  if (((uintptr_t)L | (uintptr_t)dL) % dtype_size(xdtype) ||
      !aligned(4, ids, values, weights, rows, loss) || !aligned(256, (char*)ws))
    return GMM_ERR_INVALID_ARG;
  if (ws_bytes < gmm_distill_ws_bytes()) return GMM_ERR_WORKSPACE;
  const Args a{L, ids, values, weights, rows, dL, (double*)ws, N, K, m, kind == GMM_TEACHER_GAMMA,
               (flags & GMM_DISTILL_ADD) != 0 && dL, (float)temperature, (float)(1.0 / temperature),
               (float)scale};
  cudaStream_t s = (cudaStream_t)stream;
  int64_t blocks;
  {
    ProfScope p("distill_kernel", s);
    blocks = xdtype == GMM_F32   ? launch_typed<float>(a, s)
             : xdtype == GMM_F16 ? launch_typed<__half>(a, s)
                                 : launch_typed<__nv_bfloat16>(a, s);
  }
  if (!blocks) return GMM_ERR_CUDA;
  ProfScope p("distill_finish_kernel", s);
  distill_finish_kernel<<<1, kWarpThreads, 0, s>>>((const double*)ws, (int)blocks, scale, loss);
  return launched();
}

}  // extern "C"
