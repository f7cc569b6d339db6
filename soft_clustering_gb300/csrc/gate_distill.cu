// gate_distill.cu - distillation from a teacher's top entries.
//
//   row_n = w T^2 sum_t q_t (log q_t - log p[ids_t]),  loss = scale sum_n row_n
//   dL    = scale w T (p - q)
//
// One pass over the logits: a row stays in registers from its load to the
// gradient's store, 32 logits a thread.  Rows of up to 1024 logits belong to
// lanes of a warp, of up to 16384 to a block; longer ones are streamed by a block
// twice, the second time out of L2.  Rows that do not start on 16 bytes are read
// by single elements, 8 or 16 a thread, up to 8192.  The gradient is p alone
// first; the lane that holds a teacher's entry puts that element right.  All
// exponents are of base 2.
//
// 1000003 rows of 256 f16 and 4 entries take 212 us with the gradient (149 at the
// copy rate; 16 logits a lane: 488): 125 registers leave 16 warps a multiprocessor,
// which wait on latency (issue slots at 51 %, HBM at 59 %).  8191 of 50257 bf16 and
// 32 entries, 355 us (243), are near their issue slots (74 %), 300 us with half the
// rows padding; the loss alone of 65536 of 4096 bf16 takes 123 us (79).
#include "gate_internal.cuh"

namespace gmm {
namespace {

using namespace gate;

constexpr int kWarpThreads = 256;
constexpr int kBlockThreads = 512;
constexpr int kStreamThreads = 512;
constexpr int kMaxGrid = 32 * kSms;  // blocks that a device can hold
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

// log of a teacher's share.  One below 2^-126, which lg2 takes for 0, is as good as
// any other: a temperature, or a row of nothing larger, makes it count.
__device__ __forceinline__ float log_of(float g) {
  const bool tiny = g < 1.17549435e-38f;
  return kLn2 * (lg2(tiny ? g * 0x1p64f : g) - (tiny ? 64.f : 0.f));
}

// A teacher's entries of one row, MT a lane of the `size` (a power of two) that
// share them, entry i * size + lane in place i.
template <int MT>
struct Entries {
  int id[MT];     // -1: none
  float b[MT];    // the value, of a gamma its log: T log q, but for a constant
  float x[MT];    // the student's logit
  float old[MT];  // what the gradient is added to
  float q[MT];

  // Row n's ids and values as they are, for `take` a row later.
  __device__ __forceinline__ void fetch(const Args& a, int64_t n, int lane, int size) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int t = i * size + lane;
      id[i] = -1;
      b[i] = 0.f;
      if (n < a.N && t < a.m) {
        id[i] = a.ids[n * a.m + t];
        b[i] = a.values[n * a.m + t];
      }
    }
  }
  __device__ __forceinline__ void check(const Args& a, bool on) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (!on || (uint32_t)id[i] >= (uint32_t)a.K) id[i] = -1;
      if (a.gammas) b[i] = log_of(b[i]);
      if (id[i] < 0) b[i] = -INFINITY;
      if (b[i] == -INFINITY) id[i] = -1;
      x[i] = old[i] = 0.f;
    }
  }
  // The student's logits at the entries, from `at(id)`.
  template <typename At>
  __device__ __forceinline__ void gather(At at) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) x[i] = to_f(*at(id[i]));
  }
  template <typename T>
  __device__ __forceinline__ void gather_old(const Args& a, const T* dL) {
    if (a.add) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (id[i] >= 0) old[i] = to_f(dL[id[i]]);
    }
  }
  // q, and whether there is an entry.  The largest is taken off the values as they
  // are: a product's rounding goes by its size, and the lowest number times log2 e
  // is no number.
  template <typename Team>
  __device__ __forceinline__ bool normalise(Team team, float k, float& logsum) {
    float top = b[0];
#pragma unroll
    for (int i = 1; i < MT; ++i) top = max_nan(top, b[i]);
    top = team.top(top);
    const bool some = top != -INFINITY;
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      b[i] -= some ? top : 0.f;
      q[i] = ex2(b[i] * k);
      s[0] += q[i];
    }
    team.sum(s);
    logsum = lg2(s[0]);
    const float r = some ? rcp(s[0]) : 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i) q[i] *= r;
    return some;
  }
  // sum_t q_t (b_t - (x_t - top)): in the logits' own units, which hold what a
  // temperature or log2 e times it does not
  template <typename Team>
  __device__ __forceinline__ float divergence(Team team, const Base& base) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0 && q[i] != 0.f) s[0] += q[i] * (b[i] - (x[i] - base.top));
    team.sum(s);
    return s[0];
  }
  // Whether two entries of some row in the warp are of one element.
  template <typename Team>
  __device__ __forceinline__ bool twice(Team team) const {
    if (MT > 1) return true;
    const int l = threadIdx.x & 31, group = l & ~(team.size - 1);
    const unsigned same = __match_any_sync(0xffffffffu, id[0] >= 0 ? id[0] << 5 | group : -1 - l);
    return __any_sync(0xffffffffu, (same & (same - 1)) != 0);
  }
  // The same by the elements' own words, which hold nothing of use any more:
  // of two lanes that write one, the one whose number is not there sees it.
  template <typename At>
  __device__ __forceinline__ bool twice_at(At at) const {
    using W = unsigned short;
    bool other = false;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) *reinterpret_cast<W*>(at(id[i])) = (W)(i * 32 + (threadIdx.x & 31));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) other |= *reinterpret_cast<const W*>(at(id[i])) != (W)(i * 32 + (threadIdx.x & 31));
    return __any_sync(0xffffffffu, other);
  }
  // The gradient's elements at the entries, c (p - q) with the q of every entry
  // of that element, into q; the id stays with the first of them alone.
  template <typename Team>
  __device__ __forceinline__ void gradient(Team team, int m, float c, const Base& base, float k, float rsum,
                                           bool twice) {
    const int l = threadIdx.x & 31, group = l & ~(team.size - 1);
    float w[MT];
    bool first[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) w[i] = q[i], first[i] = true;
    if (twice) {
#pragma unroll
      for (int i = 0; i < MT; ++i) w[i] = 0.f;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (j * team.size >= m) break;
        for (int o = 0; o < team.size; ++o) {
          const int id_o = __shfl_sync(0xffffffffu, id[j], group + o);
          const float q_o = __shfl_sync(0xffffffffu, q[j], group + o);
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
      q[i] = fmaf(c, ex2(base(x[i], k)) * rsum - w[i], old[i]);
      if (!first[i]) id[i] = -1;
    }
  }
  template <typename T, typename At>
  __device__ __forceinline__ void store(At at) const {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] >= 0) *at(id[i]) = from_f<T>(q[i]);
  }
};

// Sums of the threads' row losses, in the order of the threads.
__device__ __forceinline__ void store_total(const Args& a, double total) {
  __shared__ double part[32];
  let_next_start();
  total = block_reduce(total, 0.0, SumOp(), part);
  if (threadIdx.x == 0) a.part[blockIdx.x] = total;
}

__device__ __forceinline__ float row_loss(const Args& a, float w, float divergence, float logsum, float sum,
                                          const Base& base, float k) {
  // a row with no student at all is infinitely far
  if (sum == 0.f) return w * INFINITY;
  // T twice and not T^2, which may be past fp32 where the row's loss is not
  return w * a.T * (divergence + a.T * kLn2 * (lg2(sum) - base.over(k) - logsum));
}

// 1 / the sum; no student: p = 0
__device__ __forceinline__ float rsum_of(float sum) { return sum == 0.f ? 0.f : rcp(sum); }

// The gradient's elements at the entries are put into the row while it is in
// shared memory (read from there too): in device memory a scattered store and a
// scattered load for each took 127 of 296 us on 1000003 rows of 256 f16.
template <typename T, int V, int NV, int MT, int S>
__global__ void __launch_bounds__(kWarpThreads) distill_warp_kernel(Args a, int size_) {
  extern __shared__ __align__(16) char smem[];
  constexpr int P = V * NV / 2;
  using F = Feed<T, V, NV, 1, WeightedRows>;
  const int size = S ? S : size_;
  const int l = threadIdx.x & 31, per = 32 / size, K = a.K, nv = K / V;
  const int64_t warp = ((int64_t)blockIdx.x * kWarpThreads + threadIdx.x) >> 5;
  const int64_t stride = (int64_t)gridDim.x * (kWarpThreads / 32) * per;
  WarpTeam<S> team(l & (size - 1), size);
  const float k = kLog2E * a.inv;
  const T none = from_f<T>(-INFINITY);
  int64_t n = warp * per + l / size;
  F feed;
  feed.start(smem, {(const T*)a.L}, n, stride, a.N, K, team.lane, size, nv, none, WeightedRows{a.weights});
  Entries<MT> ahead;
  ahead.fetch(a, n, team.lane, size);
  const T* L = (const T*)a.L + n * K;
  T* d = (T*)a.dL + n * K;
  float wn = a.weights && n < a.N ? a.weights[n] : 1.f;
  Sum2 losses;
  for (int64_t end = warp * per; end < a.N; n += stride, end += stride, L += stride * K, d += stride * K) {
    Row<T, V, NV> row[1];
    const bool on = feed.next(row);
    Entries<MT> e = ahead;
    e.check(a, on);
    ahead.fetch(a, n + stride, team.lane, size);
    const float w = wn;
    if (a.weights && n + stride < a.N) wn = a.weights[n + stride];
    bool twice;
    if constexpr (F::kAsync) {
      __syncwarp();
      e.gather([&](int i) { return feed.peer(i); });
      __syncwarp();
      twice = a.dL && e.twice_at([&](int i) { return feed.peer(i); });
    } else {
      e.gather([&](int i) { return L + i; });
      twice = a.dL && e.twice(team);
    }
    e.gather_old(a, d);
    const Base base(team.top(lane_max(row[0])), k);
    float2 x[P];
    row[0].get(x);
    exponentials(x, base, k);
    float s[1] = {total(x)};
    team.sum(s);
    float logsum;
    const bool some = e.normalise(team, k, logsum) && on;
    const float divergence = e.divergence(team, base);
    if (team.lane == 0 && n < a.N) {
      const float r = some ? row_loss(a, w, divergence, logsum, s[0], base, k) : 0.f;
      a.rows[n] = r;
      losses.add(r);
    }
    if (!a.dL) continue;
    const float c = a.scale * w * a.T, rsum = rsum_of(s[0]);
    e.gradient(team, a.m, c, base, k, rsum, twice);
    const bool write = n < a.N && (!a.add || some);
    const float2 f = both(c * rsum);
    if (a.add) {
      Row<T, V, NV> old;
      old.fill(none);
      if (write) old.read(d, team.lane, team.size, nv);
      float2 o[P];
      old.get(o);
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = fma2(x[i], f, o[i]);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = mul2(x[i], f);
    }
    row[0].set(x);
    if (!some) row[0].fill(from_f<T>(0.f));
    if constexpr (F::kAsync) {
      feed.put(row[0]);
      __syncwarp();
      e.template store<T>([&](int i) { return feed.peer(i); });
      __syncwarp();
      feed.again(row[0]);
      if (write) row[0].store(d, team.lane, size, nv);
      // what is no part of the row is no logit
      if (nv < NV * size) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (j * size + team.lane >= nv)
#pragma unroll
            for (int i = 0; i < V; ++i) row[0].r[j].v[i] = none;
        feed.put(row[0]);
      }
    } else {
      if (write) row[0].store(d, team.lane, size, nv);
      __syncwarp();
      e.template store<T>([&](int i) { return d + i; });
    }
  }
  store_total(a, losses.value());
}

// The entries' warp of a block, the last one, which has no part of the row: what
// it waits for and works out goes beside the others' work.  Entries come two rows
// and the student's logits at them one row ahead.  It puts a row's elements right
// after the next row's barrier, before which the others have stored the row.
// `first` and `stride`: the rows of the block (the cluster, whose first block has
// them).
template <typename T, int MT, bool CLUSTER>
__device__ __forceinline__ Sum2 entries_warp(const Args& a, BlockTeam<CLUSTER>& team, float* some_s, int64_t first_row,
                                             int64_t stride) {
  const WarpTeam<32> warp((int)threadIdx.x & 31, 32);
  const int64_t step = stride * a.K;
  const T* L = (const T*)a.L + first_row * a.K;
  T* d = (T*)a.dL + first_row * a.K;
  const float k = kLog2E * a.inv;
  auto weight = [&](int64_t n) { return n >= a.N ? 0.f : a.weights ? a.weights[n] : 1.f; };
  Entries<MT> next, ahead, late;
  float w = weight(first_row), w_next = weight(first_row + stride);
  ahead.fetch(a, first_row, warp.lane, 32);
  next = ahead;
  next.check(a, w != 0.f);
  next.gather([&](int i) { return L + i; });
  ahead.fetch(a, first_row + stride, warp.lane, 32);
#pragma unroll
  for (int i = 0; i < MT; ++i) late.id[i] = -1;
  Sum2 losses;
  uint32_t turn = 0;
  for (int64_t n = first_row; n < a.N; n += stride, L += step, d += step, turn ^= 1) {
    Entries<MT> e = next;
    float logsum, top, s[1];
    const bool some = e.normalise(warp, k, logsum);
    if (CLUSTER) {
      if (warp.lane < (int)cluster_blocks()) team.to_block(some_s + turn, warp.lane, some ? 1.f : 0.f);
    } else if (warp.lane == 0) {
      some_s[turn] = some ? 1.f : 0.f;
    }
    next = ahead;
    next.check(a, w_next != 0.f);
    next.gather([&](int i) { return L + step + i; });
    ahead.fetch(a, n + 2 * stride, warp.lane, 32);
    const float w_after = weight(n + 2 * stride);
    e.gather_old(a, d);
    team.barrier();
    if (a.dL) late.template store<T>([&](int i) { return d - step + i; });
    team.hear(s, top, 0.f, k);
    const Base base(top, k);
    const float divergence = e.divergence(warp, base);
    if (warp.lane == 0) {
      const float r = some ? row_loss(a, w, divergence, logsum, s[0], base, k) : 0.f;
      a.rows[n] = r;
      losses.add(r);
    }
    if (a.dL) {
      e.gradient(warp, a.m, a.scale * w * a.T, base, k, rsum_of(s[0]), e.twice(warp));
      late = e;
    }
    w = w_next;
    w_next = w_after;
  }
  team.barrier();
  if (a.dL) late.template store<T>([&](int i) { return d - step + i; });
  return losses;
}

template <typename T, int V, int NV, int MT>
__global__ void __launch_bounds__(kBlockThreads + 32) distill_block_kernel(Args a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[BlockTeam<false>::kWords];
  __shared__ float some_s[2];
  constexpr int P = V * NV / 2;
  const int K = a.K, nv = K / V;
  BlockTeam<false> team(part, blockDim.x - 32);
  const float k = kLog2E * a.inv;
  const T none = from_f<T>(-INFINITY);
  uint32_t turn = 0;
  Sum2 losses;
  const int64_t step = (int64_t)gridDim.x * K;
  T* d = (T*)a.dL + (int64_t)blockIdx.x * K;
  if ((int)threadIdx.x >= team.size) {
    losses = entries_warp<T, MT, false>(a, team, some_s, blockIdx.x, gridDim.x);
  } else {
    Feed<T, V, NV, 1, WeightedRows> feed;
    feed.start(smem, {(const T*)a.L}, blockIdx.x, gridDim.x, a.N, K, team.lane, team.size, nv, none,
               WeightedRows{a.weights});
    float wn = a.weights && blockIdx.x < a.N ? a.weights[blockIdx.x] : 1.f;
    for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, d += step, turn ^= 1) {
      Row<T, V, NV> row[1];
      const bool on = feed.next(row);
      const float w = wn;
      if (a.weights && n + gridDim.x < a.N) wn = a.weights[n + gridDim.x];
      const float mine = team.top(lane_max(row[0]));
      float2 x[P];
      row[0].get(x);
      exponentials(x, Base(mine, k), k);
      float s[1] = {total(x)}, top;
      team.tell(s, mine);
      __syncthreads();
      if (!a.dL) {
        team.turn ^= 1;
        continue;
      }
      const bool some = on && some_s[turn] != 0.f;
      const float own = team.hear(s, top, mine, k);
      if (a.add && !some) continue;
      const float2 f = both(a.scale * w * a.T * own * rsum_of(s[0]));
      if (a.add) {
        Row<T, V, NV> old;
        old.read(d, team.lane, team.size, nv);
        float2 o[P];
        old.get(o);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = fma2(x[i], f, o[i]);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = mul2(x[i], f);
      }
      row[0].set(x);
      if (!some) row[0].fill(from_f<T>(0.f));
      row[0].store(d, team.lane, team.size, nv);
    }
    __syncthreads();
  }
  store_total(a, losses.value());
}

// A row to a block, two blocks a multiprocessor (U = 2) or one, or few rows to
// clusters of `blocks` each.
template <typename T, bool CLUSTER, int U>
__global__ void __launch_bounds__(kStreamThreads + 32, U == 2 ? 2 : 1) distill_stream_kernel(Args a, int blocks) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[BlockTeam<CLUSTER>::kWords];
  __shared__ float some_s[2];
  using F = Stream<T, WeightedRows, U>;
  constexpr int V = kWide<T>, P = U * V / 2, MT = 2;
  const int K = a.K;
  BlockTeam<CLUSTER> team(part, kStreamThreads);
  const float k = kLog2E * a.inv;
  const T none = from_f<T>(-INFINITY);
  const int64_t first = CLUSTER ? blockIdx.x / blocks : blockIdx.x, stride = CLUSTER ? gridDim.x / blocks : gridDim.x;
  const int64_t step = stride * K;
  const T* L = (const T*)a.L + first * K;
  T* d = (T*)a.dL + first * K;
  if (CLUSTER) cluster_barrier();  // every block of the cluster runs
  uint32_t turn = 0;
  Sum2 losses;
  if ((int)threadIdx.x >= kStreamThreads) {
    if (!CLUSTER || cluster_rank() == 0) {
      losses = entries_warp<T, MT, CLUSTER>(a, team, some_s, first, stride);
    } else {
      for (int64_t n = first; n < a.N; n += stride) team.barrier();
      team.barrier();
    }
  } else {
    const int t = team.lane, size = CLUSTER ? team.size : kStreamThreads;
    F feed;
    feed.start(smem, (const T*)a.L, first, stride, a.N, K, a.dL ? 2 : 1, t, size, kStreamThreads,
               WeightedRows{a.weights});
    for (int64_t n = first; n < a.N; n += stride, L += step, d += step, turn ^= 1) {
      const float w = a.weights ? a.weights[n] : 1.f;
      const bool on = w != 0.f;
      const int head = F::head_of(L, K), nv = (K - head) / V, tail = head + nv * V;
      const int turns = (nv + U * size - 1) / (U * size);
      // the elements outside the vectors, one a thread
      const int edge = t < head ? t : t - head < K - tail ? tail + t - head : -1;
      const float xe = on && edge >= 0 ? to_f(L[edge]) : -INFINITY;
      float top = xe;
      float2 sum = make_float2(xe == -INFINITY ? 0.f : ex2(Base(xe, k)(xe, k)), 0.f);
      for (int i = 0; on && i < turns; ++i) {
        Row<T, V, U> x;
        feed.next(x);
        if (i == turns - 1) {
          const int v0 = i * U * size + t;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (v0 + u * size >= nv)
#pragma unroll
              for (int e = 0; e < V; ++e) x.r[u].v[e] = none;
        }
        const float m = max_nan(top, lane_max(x));
        if (m != top) {
          sum = mul2(sum, both(BlockTeam<false>::between(top, m, k)));
          top = m;
        }
        float2 f[P];
        x.get(f);
        exponentials(f, Base(top, k), k);
#pragma unroll
        for (int j = 0; j < P; ++j) sum = add2(sum, f[j]);
      }
      // the warp's, then the block's
      const float mine = warp_max(top);
      float s[1] = {(sum.x + sum.y) * BlockTeam<false>::between(top, mine == -INFINITY ? 0.f : mine, k)};
      team.tell(s, mine);
      team.barrier();
      if (!a.dL) {
        team.turn ^= 1;
        continue;
      }
      const bool some = on && some_s[turn] != 0.f;
      team.hear(s, top, mine, k);
      const Base base(top, k);
      const float c = some ? a.scale * w * a.T * rsum_of(s[0]) : 0.f;
      const float2 f = both(c);
      const bool same = (((uintptr_t)L ^ (uintptr_t)d) & 15) == 0;
      if (edge >= 0 && (some || !a.add)) {
        float y = some ? ex2(base(xe, k)) * c : 0.f;
        if (a.add) y += to_f(d[edge]);
        d[edge] = from_f<T>(y);
      }
      T* out = d + head + (int64_t)t * V;
      for (int i = 0; i < turns; ++i, out += U * size * V) {
        Row<T, V, U> x;
        if (on) feed.next(x);
        else x.fill(from_f<T>(0.f));
        if (a.add && !some) continue;
        float2 y[P];
        x.get(y);
        exponentials(y, base, k);
        if (a.add) {
          Row<T, V, U> o;
          o.fill(none);
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (i * U * size + t + u * size < nv) {
              if (same) o.r[u] = *reinterpret_cast<const Vec<T, V>*>(out + u * size * V);
              else
#pragma unroll
                for (int e = 0; e < V; ++e) o.r[u].v[e] = out[u * size * V + e];
            }
          float2 z[P];
          o.get(z);
#pragma unroll
          for (int j = 0; j < P; ++j) y[j] = fma2(y[j], f, z[j]);
        } else {
#pragma unroll
          for (int j = 0; j < P; ++j) y[j] = mul2(y[j], f);
        }
        x.set(y);
        if (!some) x.fill(from_f<T>(0.f));
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i * U * size + t + u * size < nv) {
            if (same) *reinterpret_cast<Vec<T, V>*>(out + u * size * V) = x.r[u];
            else
#pragma unroll
              for (int e = 0; e < V; ++e) out[u * size * V + e] = x.r[u].v[e];
          }
      }
    }
    team.barrier();
  }
  store_total(a, losses.value());
}

// The blocks' sums in order, in 64 bits.
__global__ void __launch_bounds__(kWarpThreads)
distill_finish_kernel(const double* __restrict__ part, int blocks, double scale,
                      float* __restrict__ loss) {
  __shared__ double partd[32];
  wait_for_last();
  double s = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kWarpThreads) s += part[b];
  s = block_reduce(s, 0.0, SumOp(), partd);
  if (threadIdx.x == 0) *loss = (float)(s * scale);
}

template <typename T, int V, int NV, int MT>
int64_t launch_block(const Args& a, int threads, cudaStream_t s) {
  static std::atomic<uint64_t> done;
  static ResidentCache cache;
  using F = Feed<T, V, NV, 1, WeightedRows>;
  if (!allow_smem((const void*)distill_block_kernel<T, V, NV, MT>, F::bytes(kBlockThreads + 32), done)) return 0;
  const int64_t most = resident(distill_block_kernel<T, V, NV, MT>, threads, F::bytes(threads), cache);
  const int64_t grid = a.N < 1 ? 1 : a.N < most ? a.N : most;
  distill_block_kernel<T, V, NV, MT><<<(unsigned)grid, threads, F::bytes(threads), s>>>(a);
  return grid;
}
template <typename T, int V, int E, int MT, int S>
int64_t launch_warp(const Args& a, int size, cudaStream_t s) {
  static std::atomic<uint64_t> done;
  static ResidentCache cache;
  using F = Feed<T, V, E / V, 1, WeightedRows>;
  const size_t smem = F::bytes(kWarpThreads);
  if (!allow_smem((const void*)distill_warp_kernel<T, V, E / V, MT, S>, smem, done)) return 0;
  const int64_t rows = kWarpThreads / size, need = (a.N + rows - 1) / rows;
  const int64_t most = resident(distill_warp_kernel<T, V, E / V, MT, S>, kWarpThreads, smem, cache);
  const int64_t grid = need < 1 ? 1 : need < most ? need : most;
  distill_warp_kernel<T, V, E / V, MT, S><<<(unsigned)grid, kWarpThreads, smem, s>>>(a, size);
  return grid;
}
// With as many lanes as hold the row, but for entries: at most eight a lane.
template <typename T, int V, int E, int S>
int64_t launch_lanes(const Args& a, int size, cudaStream_t s) {
  return a.m <= size ? launch_warp<T, V, E, 1, S>(a, size, s) : launch_warp<T, V, E, 8, S>(a, size, s);
}

// Returns the blocks launched; 0: none.
template <typename T, int V>
int64_t launch(const Args& a, cudaStream_t s) {
  const int K = a.K, m = a.m;
  if constexpr (V == 1) {
    // single elements: read 32 at a time where the row has as many
    if (K <= 512) {
      int size = 1;
      while (size < 32 && (size < K || size * 8 < m)) size <<= 1;
      return K <= 256 ? launch_lanes<T, 1, 8, 0>(a, size, s) : launch_lanes<T, 1, 16, 0>(a, size, s);
    }
  } else {
    if (K <= 8 && m <= 8) return launch_lanes<T, V, 8, 1>(a, 1, s);
    if (K <= 64 && m <= 32) return launch_lanes<T, V, 16, 4>(a, 4, s);
    if (K <= 128 && m <= 32) return launch_lanes<T, V, 32, 4>(a, 4, s);
    if (K <= 256) return launch_lanes<T, V, 32, 8>(a, 8, s);
    if (K <= 512) return launch_lanes<T, V, 32, 16>(a, 16, s);
    if (K <= 1024) return launch_lanes<T, V, 32, 32>(a, 32, s);
  }
  constexpr int E = V > 1 ? 32 : 16;
  const int threads = ((K + E - 1) / E + 31) / 32 * 32 + 32;
  return m <= 32 ? launch_block<T, V, E / V, 1>(a, threads, s) : launch_block<T, V, E / V, 2>(a, threads, s);
}

template <typename T, bool CLUSTER, int U>
int64_t launch_stream(const Args& a, int64_t grid, int blocks, cudaStream_t s) {
  static std::atomic<uint64_t> done;
  const size_t smem = Stream<T, WeightedRows, U>::bytes(kStreamThreads);
  if (!allow_smem((const void*)distill_stream_kernel<T, CLUSTER, U>, smem, done)) return 0;
  if (CLUSTER)
    launch_clusters(distill_stream_kernel<T, CLUSTER, U>, (unsigned)grid, kStreamThreads + 32, smem, blocks, s, a, blocks);
  else
    distill_stream_kernel<T, CLUSTER, U><<<(unsigned)grid, kStreamThreads + 32, smem, s>>>(a, 1);
  return grid;
}

template <typename T>
int64_t launch_typed(const Args& a, cudaStream_t s) {
  const bool vectors = wide<T>(a.K, (const char*)a.L, (const char*)a.dL);
  if (a.K > (vectors ? 32 : 16) * kBlockThreads) {
    // few rows: as many blocks each as leave none without, a cluster's barrier
    // being some microseconds of a row's time
    int blocks = 1;
    while (blocks < 8 && a.N * blocks * 2 <= kSms) blocks *= 2;
    if (blocks > 1) return launch_stream<T, true, 4>(a, (a.N < 1 ? 1 : a.N) * blocks, blocks, s);
    // two rows a multiprocessor while L2 keeps them for their second reading
    // (50257 bf16: 354 us against 396 of one; 131072: 269 against 222)
    if ((int64_t)a.K * (int)sizeof(T) <= 160 * 1024)
      return launch_stream<T, false, 2>(a, a.N < 2 * kSms ? a.N : 2 * kSms, 1, s);
    return launch_stream<T, false, 4>(a, a.N < kSms ? a.N : kSms, 1, s);
  }
  return vectors ? launch<T, kWide<T>>(a, s) : launch<T, 1>(a, s);
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
      !((float)temperature < INFINITY) || !((float)(1.0 / temperature) * kLog2E < INFINITY) || !loss || !ws)
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
  launch_behind(distill_finish_kernel, 1, kWarpThreads, s, (const double*)ws, (int)blocks, scale, loss);
  return launched();
}

}  // extern "C"
