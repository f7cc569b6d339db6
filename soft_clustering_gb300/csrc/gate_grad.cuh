// gate_grad.cuh - the gradient of a learned gate's logits.
//
//   dL = p (coef (share - <share, p>) - S) + v at ids
//
// with v = gamma dgamma, S their sum over a row (normalised: v -= gamma S, S = 0).
// One pass: a row stays in registers from its load to its store (shapes as in
// the distillation's kernels: lanes of a warp up to 1024 logits, a block up to
// 16384, two readings beyond).  A lane has the same columns of every row and
// keeps their share of the balance loss in registers.  The entries' elements are
// put right where the row waits in shared memory (warps), or by a warp of their
// own after the next row's barrier (blocks).
//
// Bound by HBM where rows are long (65536 of 4096 bf16: 173 us, 6.2 TB/s).  With
// the balance loss (262144 of 1024 bf16, a tenth of them padding: 202 us, 5.1 TB/s)
// 120 registers leave 16 warps a multiprocessor, HBM at 61 % and the issue slots at
// 58 %.  Streamed, 2048 of 65536 bf16: 117 us, with the balance loss 300 (79), with
// half the rows padding 230.
//
// A normalised gate without the balance loss has a gradient at its entries alone:
// zeros are written and the logits not read (65536 of 4096 bf16: 86 us, 6.2 TB/s;
// 1000003 of 256 f16: 115, 4.9 TB/s).
#pragma once

#include "gate_internal.cuh"

namespace gmm {
namespace gate {

struct GradArgs {
  const void* L;
  const uint8_t* live;
  const int32_t* ids;
  const float *gamma, *dgamma, *share;
  void* dL;
  int64_t N;
  int K, m, normalised;
  float coef;
};

// Returns false where the device refuses.
bool launch_grad_f32(const GradArgs& a, cudaStream_t s);
bool launch_grad_f16(const GradArgs& a, cudaStream_t s);
bool launch_grad_bf16(const GradArgs& a, cudaStream_t s);

namespace grad_impl {

constexpr int kWarpThreads = 256;
constexpr int kBlockThreads = 512;

// A row's entries, MT a lane of those that share them: entry i * size + lane.
template <int MT>
struct Entries {
  int id[MT];     // -1: none
  float g[MT];    // gamma
  float v[MT];    // dgamma, then v, then the element
  float x[MT];    // the logit
  float c[MT];    // share

  __device__ __forceinline__ void fetch(const GradArgs& a, int64_t n, int lane, int size) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int t = i * size + lane;
      id[i] = -1;
      g[i] = v[i] = 0.f;
      if (a.dgamma && n < a.N && t < a.m) {
        id[i] = a.ids[n * a.m + t];
        g[i] = a.gamma[n * a.m + t];
        v[i] = a.dgamma[n * a.m + t];
      }
    }
  }
  // v and S; what is no entry of a row that counts has none.
  template <typename Team>
  __device__ __forceinline__ float check(const GradArgs& a, Team team, bool on) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (!on || (uint32_t)id[i] >= (uint32_t)a.K) id[i] = -1;
      v[i] = id[i] >= 0 ? g[i] * v[i] : 0.f;
      x[i] = c[i] = 0.f;
      if (id[i] >= 0 && a.share) c[i] = a.share[id[i]];
      s[0] += v[i];
    }
    team.sum(s);
    if (!a.normalised) return s[0];
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) v[i] -= g[i] * s[0];
    return 0.f;
  }
  template <typename At>
  __device__ __forceinline__ void gather(At at) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) x[i] = to_f(*at(id[i]));
  }
  // The elements at the entries, rsum 2^(..) (scale c + shift) and the v of every
  // entry of the element; the id stays with the first of them alone.
  template <typename Team>
  __device__ __forceinline__ void gradient(const GradArgs& a, Team team, const Base& base, float scale, float shift) {
    const int l = threadIdx.x & 31, group = l & ~(team.size - 1);
    float w[MT];
    bool first[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) w[i] = 0.f, first[i] = true;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if (j * team.size >= a.m) break;
      for (int o = 0; o < team.size && j * team.size + o < a.m; ++o) {
        const int id_o = __shfl_sync(0xffffffffu, id[j], group + o);
        const float v_o = __shfl_sync(0xffffffffu, v[j], group + o);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          if (id_o == id[i]) {
            w[i] += v_o;
            if (j < i || (j == i && o < team.lane)) first[i] = false;
          }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      v[i] = fmaf(ex2(base(x[i], kLog2E)), fmaf(scale, c[i], shift), w[i]);
      if (!first[i]) id[i] = -1;
    }
  }
  template <typename T, typename At>
  __device__ __forceinline__ void store(At at) const {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) *at(id[i]) = from_f<T>(v[i]);
  }
};

// Exponentials' sum and their product with `share`.
template <bool SHARE, int P>
__device__ __forceinline__ void sums_of(const float2 (&x)[P], const float2 (&c)[SHARE ? P : 1], float (&s)[SHARE ? 2 : 1]) {
  s[0] = total(x);
  if constexpr (SHARE) {
    float2 d = both(0.f);
#pragma unroll
    for (int i = 0; i < P; ++i) d = fma2(x[i], c[i], d);
    s[1] = d.x + d.y;
  }
}
// x (scale c + shift)
template <bool SHARE, int P>
__device__ __forceinline__ void apply(float2 (&x)[P], const float2 (&c)[SHARE ? P : 1], float scale, float shift) {
#pragma unroll
  for (int i = 0; i < P; ++i)
    x[i] = mul2(x[i], SHARE ? fma2(c[SHARE ? i : 0], both(scale), both(shift)) : both(shift));
}
// scale and shift of a row: p (coef (share - dot) - S) = e (scale share + shift)
template <bool SHARE>
__device__ __forceinline__ void factors(const GradArgs& a, const float (&s)[SHARE ? 2 : 1], float S, float own,
                                        float& scale, float& shift) {
  const float r = s[0] == 0.f ? 0.f : rcp(s[0]);
  scale = SHARE ? a.coef * r : 0.f;
  shift = -r * (SHARE ? fmaf(a.coef, s[SHARE ? 1 : 0] * r, S) : S);
  scale *= own;
  shift *= own;
}

template <typename T, int V, int NV, int MT, int S, bool SHARE>
__global__ void __launch_bounds__(kWarpThreads) grad_warp_kernel(GradArgs a) {
  extern __shared__ __align__(16) char smem[];
  constexpr int P = V * NV / 2, per = 32 / S;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const int l = threadIdx.x & 31, K = a.K, nv = K / V;
  const int64_t warp = ((int64_t)blockIdx.x * kWarpThreads + threadIdx.x) >> 5;
  const int64_t stride = (int64_t)gridDim.x * (kWarpThreads / 32) * per;
  WarpTeam<S> team(l & (S - 1), S);
  const T none = from_f<T>(-INFINITY);
  int64_t n = warp * per + l / S;
  float2 c[SHARE ? P : 1];
  if constexpr (SHARE) load_columns<V, NV>(c, a.share, team.lane, S, nv, 0.f);
  // the entries come with the row (eight a lane, or beside rows that wait in
  // registers: a row ahead)
  constexpr bool kWords = MT == 1 && F::kAsync;
  Words<3, F::kStages> words;
  words.start(smem + F::bytes(kWarpThreads), team.lane, a.m, stride);
  words.array(0, kWords && a.dgamma ? a.ids : nullptr, n, team.lane, a.m);
  words.array(1, kWords && a.dgamma ? a.gamma : nullptr, n, team.lane, a.m);
  words.array(2, kWords ? a.dgamma : nullptr, n, team.lane, a.m);
  F feed;
  feed.start(smem, {(const T*)a.L}, n, stride, a.N, K, team.lane, S, nv, none, LiveRows{a.live}, words);
  Entries<MT> ahead;
  if (!kWords) ahead.fetch(a, n, team.lane, S);
  const T* L = (const T*)a.L + n * K;
  T* d = (T*)a.dL + n * K;
  for (int64_t end = warp * per; end < a.N; n += stride, end += stride, L += stride * K, d += stride * K) {
    Row<T, V, NV> row[1];
    const bool on = feed.next(row, words);
    Entries<MT> e;
    if constexpr (kWords) {
      const bool is = a.dgamma && words.mine;
      e.id[0] = is ? words.template word<int>(feed.taken(), 0) : -1;
      e.g[0] = is ? words.template word<float>(feed.taken(), 1) : 0.f;
      e.v[0] = is ? words.template word<float>(feed.taken(), 2) : 0.f;
    } else {
      e = ahead;
      ahead.fetch(a, n + stride, team.lane, S);
    }
    const float sum_v = e.check(a, team, on);
    if constexpr (F::kAsync) {
      __syncwarp();
      e.gather([&](int i) { return feed.peer(i); });
      __syncwarp();
    } else {
      e.gather([&](int i) { return L + i; });
    }
    const Base base(team.top(lane_max(row[0])), kLog2E);
    float2 x[P];
    row[0].get(x);
    exponentials(x, base, kLog2E);
    float s[SHARE ? 2 : 1], scale, shift;
    sums_of<SHARE>(x, c, s);
    team.sum(s);
    factors<SHARE>(a, s, sum_v, 1.f, scale, shift);
    e.gradient(a, team, base, scale, shift);
    apply<SHARE>(x, c, scale, shift);
    row[0].set(x);
    if (!on) row[0].fill(from_f<T>(0.f));
    if constexpr (F::kAsync) {
      feed.put(row[0]);
      __syncwarp();
      e.template store<T>([&](int i) { return feed.peer(i); });
      __syncwarp();
      feed.again(row[0]);
      if (n < a.N) row[0].store(d, team.lane, S, nv);
      if (nv < NV * S) {  // what is no part of the row is no logit
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (j * S + team.lane >= nv)
#pragma unroll
            for (int i = 0; i < V; ++i) row[0].r[j].v[i] = none;
        feed.put(row[0]);
      }
    } else {
      if (n < a.N) row[0].store(d, team.lane, S, nv);
      __syncwarp();
      e.template store<T>([&](int i) { return d + i; });
    }
  }
}

// The entries' warp of a block, the last one: tells S before a row's barrier,
// hears the row's sums after it, and puts the row's elements right after the
// next barrier, before which the others have stored it.  Entries come two rows
// and their logits one row ahead.
template <typename T, bool SHARE>
__device__ __forceinline__ void entries_warp(const GradArgs& a, BlockTeam<false>& team, float* sum_v) {
  const WarpTeam<32> warp((int)threadIdx.x & 31, 32);
  const int64_t step = (int64_t)gridDim.x * a.K;
  const T* L = (const T*)a.L + (int64_t)blockIdx.x * a.K;
  T* d = (T*)a.dL + (int64_t)blockIdx.x * a.K;
  const LiveRows live{a.live};
  Entries<1> next, ahead, late;
  float S = 0.f;
  auto take = [&](int64_t n, const T* row) {  // of row n, whose words have come
    next = ahead;
    S = next.check(a, warp, n < a.N && live(n));
    next.gather([&](int i) { return row + i; });
  };
  ahead.fetch(a, blockIdx.x, warp.lane, 32);
  take(blockIdx.x, L);
  ahead.fetch(a, (int64_t)blockIdx.x + gridDim.x, warp.lane, 32);
  late.id[0] = -1;
  uint32_t turn = 0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, L += step, d += step, turn ^= 1) {
    Entries<1> e = next;
    const float mine = S;
    if (warp.lane == 0) sum_v[turn] = mine;
    take(n + gridDim.x, L + step);
    ahead.fetch(a, n + 2 * (int64_t)gridDim.x, warp.lane, 32);
    __syncthreads();
    late.template store<T>([&](int i) { return d - step + i; });
    float s[SHARE ? 2 : 1], top, scale, shift;
    team.hear(s, top, 0.f, kLog2E);
    factors<SHARE>(a, s, mine, 1.f, scale, shift);
    e.gradient(a, warp, Base(top, kLog2E), scale, shift);
    late = e;
  }
  __syncthreads();
  late.template store<T>([&](int i) { return d - step + i; });
}

template <typename T, int V, int NV, bool SHARE>
__global__ void __launch_bounds__(kBlockThreads + 32, 1) grad_block_kernel(GradArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[BlockTeam<false>::kWords];
  __shared__ float sum_v[2];
  constexpr int P = V * NV / 2;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const int K = a.K, nv = K / V;
  BlockTeam<false> team(part, blockDim.x - 32);
  if ((int)threadIdx.x >= team.size) {
    entries_warp<T, SHARE>(a, team, sum_v);
    return;
  }
  const T none = from_f<T>(-INFINITY);
  float2 c[SHARE ? P : 1];
  if constexpr (SHARE) load_columns<V, NV>(c, a.share, team.lane, team.size, nv, 0.f);
  F feed;
  feed.start(smem, {(const T*)a.L}, blockIdx.x, gridDim.x, a.N, K, team.lane, team.size, nv, none, LiveRows{a.live});
  T* d = (T*)a.dL + (int64_t)blockIdx.x * K;
  uint32_t turn = 0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, d += (int64_t)gridDim.x * K, turn ^= 1) {
    Row<T, V, NV> row[1];
    const bool on = feed.next(row);
    const float mine = team.top(lane_max(row[0]));
    float2 x[P];
    row[0].get(x);
    exponentials(x, Base(mine, kLog2E), kLog2E);
    float s[SHARE ? 2 : 1], top, scale, shift;
    sums_of<SHARE>(x, c, s);
    team.tell(s, mine);
    __syncthreads();
    const float own = team.hear(s, top, mine, kLog2E);
    factors<SHARE>(a, s, sum_v[turn], own, scale, shift);
    apply<SHARE>(x, c, scale, shift);
    row[0].set(x);
    if (!on) row[0].fill(from_f<T>(0.f));
    row[0].store(d, team.lane, team.size, nv);
  }
  __syncthreads();
}

// Rows that no block holds, read twice.
template <typename T, bool SHARE>
__global__ void __launch_bounds__(kBlockThreads + 32, 1) grad_stream_kernel(GradArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[BlockTeam<false>::kWords];
  __shared__ float sum_v[2];
  using F = Stream<T, LiveRows>;
  constexpr int V = kWide<T>, U = F::U, P = U * V / 2;
  const int K = a.K, t = threadIdx.x;
  BlockTeam<false> team(part, kBlockThreads);
  if (t >= kBlockThreads) {
    entries_warp<T, SHARE>(a, team, sum_v);
    return;
  }
  const T none = from_f<T>(-INFINITY);
  const int64_t step = (int64_t)gridDim.x * K;
  const T* L = (const T*)a.L + (int64_t)blockIdx.x * K;
  T* d = (T*)a.dL + (int64_t)blockIdx.x * K;
  const LiveRows live{a.live};
  F feed;
  feed.start(smem, (const T*)a.L, blockIdx.x, gridDim.x, a.N, K, 2, t, kBlockThreads, kBlockThreads, live);
  uint32_t turn = 0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, L += step, d += step, turn ^= 1) {
    const bool on = live(n);
    const int head = F::head_of(L, K), nv = (K - head) / V, tail = head + nv * V;
    const int turns = (nv + U * kBlockThreads - 1) / (U * kBlockThreads);
    const int edge = t < head ? t : t - head < K - tail ? tail + t - head : -1;  // an element outside the vectors
    const float xe = on && edge >= 0 ? to_f(L[edge]) : -INFINITY;
    const float ce = SHARE && edge >= 0 ? a.share[edge] : 0.f;
    float top = xe, sum = xe == -INFINITY ? 0.f : ex2(Base(xe, kLog2E)(xe, kLog2E)), dot = sum * ce;
    for (int i = 0; on && i < turns; ++i) {
      Row<T, V, U> x;
      feed.next(x);
      const int v0 = i * U * kBlockThreads + t;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * kBlockThreads >= nv)
#pragma unroll
          for (int e = 0; e < V; ++e) x.r[u].v[e] = none;
      const float m = max_nan(top, lane_max(x));
      if (m != top) {
        const float f = BlockTeam<false>::between(top, m, kLog2E);
        sum *= f;
        dot *= f;
        top = m;
      }
      float2 f[P];
      x.get(f);
      exponentials(f, Base(top, kLog2E), kLog2E);
      sum += total(f);
      if constexpr (SHARE) {
        float2 c[P];
        load_columns<V, U>(c, a.share + head + (int64_t)(v0 - t) * V, t, kBlockThreads, nv - (v0 - t), 0.f);
        float2 q = both(0.f);
#pragma unroll
        for (int j = 0; j < P; ++j) q = fma2(f[j], c[j], q);
        dot += q.x + q.y;
      }
    }
    const float mine = warp_max(top);
    const float f = BlockTeam<false>::between(top, mine == -INFINITY ? 0.f : mine, kLog2E);
    float s[SHARE ? 2 : 1], scale, shift;
    s[0] = sum * f;
    if constexpr (SHARE) s[1] = dot * f;
    team.tell(s, mine);
    __syncthreads();
    team.hear(s, top, mine, kLog2E);
    const Base base(top, kLog2E);
    factors<SHARE>(a, s, sum_v[turn], 1.f, scale, shift);
    if (edge >= 0) d[edge] = from_f<T>(on ? ex2(base(xe, kLog2E)) * fmaf(scale, ce, shift) : 0.f);
    const bool same = (((uintptr_t)L ^ (uintptr_t)d) & 15) == 0;
    T* out = d + head + (int64_t)t * V;
    for (int i = 0; i < turns; ++i, out += U * kBlockThreads * V) {
      Row<T, V, U> x;
      const int v0 = i * U * kBlockThreads + t;
      if (on) {
        feed.next(x);
        float2 y[P], c[SHARE ? P : 1];
        x.get(y);
        exponentials(y, base, kLog2E);
        if constexpr (SHARE)
          load_columns<V, U>(c, a.share + head + (int64_t)(v0 - t) * V, t, kBlockThreads, nv - (v0 - t), 0.f);
        apply<SHARE>(y, c, scale, shift);
        x.set(y);
      } else {
        x.fill(from_f<T>(0.f));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * kBlockThreads < nv) {
          if (same) *reinterpret_cast<Vec<T, V>*>(out + u * kBlockThreads * V) = x.r[u];
          else
#pragma unroll
            for (int e = 0; e < V; ++e) out[u * kBlockThreads * V + e] = x.r[u].v[e];
        }
    }
  }
  __syncthreads();
}

// Zeros, and v at the entries: a block a stretch of rows.
template <typename T>
__global__ void __launch_bounds__(kWarpThreads) grad_entries_kernel(GradArgs a, int64_t stretch) {
  const int64_t begin = blockIdx.x * stretch, end = begin + stretch < a.N ? begin + stretch : a.N;
  if (begin >= end) return;
  T* d = (T*)a.dL + begin * a.K;
  const int64_t count = (end - begin) * a.K;
  const int64_t h0 = ((16 - ((uintptr_t)d & 15)) & 15) / sizeof(T), head = h0 < count ? h0 : count;
  const int64_t nv = (count - head) / kWide<T>, tail = head + nv * kWide<T>;
  const T zero = from_f<T>(0.f);
  uint4* v = reinterpret_cast<uint4*>(d + head);
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < nv; i += kWarpThreads) v[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < head) d[threadIdx.x] = zero;
  if (threadIdx.x < count - tail) d[tail + threadIdx.x] = zero;
  if (!a.dgamma) return;
  __syncthreads();
  const LiveRows live{a.live};
  for (int64_t i = threadIdx.x; i < (end - begin) * a.m; i += kWarpThreads) {
    const int64_t r = i / a.m, n = begin + r;
    const int t = (int)(i - r * a.m);
    const int id = a.ids[n * a.m + t];
    if ((uint32_t)id >= (uint32_t)a.K || !live(n)) continue;
    float S = 0.f, w = 0.f;
    bool first = true;
    for (int o = 0; o < a.m; ++o) {
      const int id_o = a.ids[n * a.m + o];
      if ((uint32_t)id_o < (uint32_t)a.K) S += a.gamma[n * a.m + o] * a.dgamma[n * a.m + o];
    }
    for (int o = 0; o < a.m; ++o)
      if (a.ids[n * a.m + o] == id) {
        const float g = a.gamma[n * a.m + o];
        w += g * a.dgamma[n * a.m + o] - g * S;
        if (o < t) first = false;
      }
    if (first) d[r * a.K + id] = from_f<T>(w);
  }
}

template <typename T, int V, int E, int MT, int S>
bool launch_lanes(const GradArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done[2];
  static ResidentCache cache[2];
  constexpr int NV = E / V;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const size_t smem = F::bytes(kWarpThreads) + Words<3, F::kStages>::bytes(kWarpThreads);
  const int64_t rows = kWarpThreads / S, need = (a.N + rows - 1) / rows;
  int64_t grid;
  if (a.share) {
    if (!allow_smem((const void*)grad_warp_kernel<T, V, NV, MT, S, true>, smem, done[1])) return false;
    grid = resident(grad_warp_kernel<T, V, NV, MT, S, true>, kWarpThreads, smem, cache[1]);
    if (grid > need) grid = need;
    grad_warp_kernel<T, V, NV, MT, S, true><<<(unsigned)grid, kWarpThreads, smem, s>>>(a);
  } else {
    if (!allow_smem((const void*)grad_warp_kernel<T, V, NV, MT, S, false>, smem, done[0])) return false;
    grid = resident(grad_warp_kernel<T, V, NV, MT, S, false>, kWarpThreads, smem, cache[0]);
    if (grid > need) grid = need;
    grad_warp_kernel<T, V, NV, MT, S, false><<<(unsigned)grid, kWarpThreads, smem, s>>>(a);
  }
  return true;
}

template <typename T, int V, int E>
bool launch_block(const GradArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done[2];
  static ResidentCache cache[2];
  constexpr int NV = E / V;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const int threads = ((a.K + E - 1) / E + 31) / 32 * 32 + 32;
  int64_t grid;
  const size_t smem = F::bytes(threads), most = F::bytes(kBlockThreads + 32);
  if (a.share) {
    if (!allow_smem((const void*)grad_block_kernel<T, V, NV, true>, most, done[1])) return false;
    grid = resident(grad_block_kernel<T, V, NV, true>, threads, smem, cache[1]);
    if (grid > a.N) grid = a.N;
    grad_block_kernel<T, V, NV, true><<<(unsigned)grid, threads, smem, s>>>(a);
  } else {
    if (!allow_smem((const void*)grad_block_kernel<T, V, NV, false>, most, done[0])) return false;
    grid = resident(grad_block_kernel<T, V, NV, false>, threads, smem, cache[0]);
    if (grid > a.N) grid = a.N;
    grad_block_kernel<T, V, NV, false><<<(unsigned)grid, threads, smem, s>>>(a);
  }
  return true;
}

template <typename T>
bool launch_grad(const GradArgs& a, cudaStream_t s) {
  constexpr int V = kWide<T>;
  const int K = a.K;
  if (a.normalised && !a.share) {
    // stretches of about 64 KB
    const int64_t want = 65536 / ((int64_t)K * (int)sizeof(T)) + 1, least = (a.N + INT32_MAX - 1) / INT32_MAX;
    const int64_t stretch = want > least ? want : least;
    grad_entries_kernel<T><<<(unsigned)((a.N + stretch - 1) / stretch), kWarpThreads, 0, s>>>(a, stretch);
    return true;
  }
  if (wide<T>(K, (const char*)a.L, (const char*)a.dL)) {
    if (K <= 8) return launch_lanes<T, V, 8, kMaxTop, 1>(a, s);
    if (K <= 64) return launch_lanes<T, V, 8, 1, 8>(a, s);
    if (K <= 128) return launch_lanes<T, V, 16, 1, 8>(a, s);
    if (K <= 256) return launch_lanes<T, V, 32, 1, 8>(a, s);
    if (K <= 512) return launch_lanes<T, V, 32, 1, 16>(a, s);
    if (K <= 1024) return launch_lanes<T, V, 32, 1, 32>(a, s);
    if (K <= 32 * kBlockThreads) return launch_block<T, V, 32>(a, s);
  } else {
    if (K <= 64) return launch_lanes<T, 1, 8, 1, 8>(a, s);
    if (K <= 128) return launch_lanes<T, 1, 8, 1, 16>(a, s);
    if (K <= 256) return launch_lanes<T, 1, 8, 1, 32>(a, s);
    if (K <= 512) return launch_lanes<T, 1, 16, 1, 32>(a, s);
    if (K <= 16 * kBlockThreads) return launch_block<T, 1, 16>(a, s);
  }
  static std::atomic<uint64_t> done[2];
  const size_t smem = Stream<T, LiveRows>::bytes(kBlockThreads);
  const int64_t grid = a.N < 2 * kSms ? a.N : 2 * kSms;
  if (a.share) {
    if (!allow_smem((const void*)grad_stream_kernel<T, true>, smem, done[1])) return false;
    grad_stream_kernel<T, true><<<(unsigned)grid, kBlockThreads + 32, smem, s>>>(a);
  } else {
    if (!allow_smem((const void*)grad_stream_kernel<T, false>, smem, done[0])) return false;
    grad_stream_kernel<T, false><<<(unsigned)grid, kBlockThreads + 32, smem, s>>>(a);
  }
  return true;
}

}  // namespace grad_impl
}  // namespace gate
}  // namespace gmm
