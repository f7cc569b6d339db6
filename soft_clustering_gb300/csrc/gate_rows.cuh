// gate_rows.cuh - a learned gate's answer: the m largest logits of a row, their
// shares of its softmax, and the balance loss's sums.
//
//   ids, gamma, lse; mass_k = sum_n p[n,k], counts_k
//
// One pass over the logits: a row stays in registers from its load on.  Rows of
// up to 1024 logits belong to lanes of a warp (8 at least, so that each of the
// m entries has one; a row of up to 8 logits has one lane to itself), of up to
// 16384 (fp32: 8192) to a block, 32 (16) logits a thread; longer ones are streamed by a block, and
// their mass is summed by columns in a second reading.  Rows that do not start
// on 16 bytes are read by single elements, up to 16 a thread.
//
// The m largest are found one at a time.  A lane keeps the largest of each of
// its vectors; its best and second best (of more than four entries its third too)
// are found beforehand, by all lanes at once.  A round takes the team's best (by
// value, then the lower column), and the lane that had it goes on to its next:
// only one that is taken from more often looks on, in the vector that its last
// came from, which waits in shared memory.  With sorting keys for all elements
// instead a round of all lanes would read every one again.
//
// A lane has the same columns of every row, so it sums their mass in registers;
// a block's sums are joined in order, by the finish over the blocks with what
// their roundings left.
//
// Bound by latency: 1000003 rows of 256 f16, m = 4, with the balance loss take 216
// us (of which the finish 13), where reading them takes 81: 166 instructions a warp
// for a row use 66 % of the issue slots, HBM is at 33 %, and 120 registers leave 15
// warps a multiprocessor.  65536 of 1024 fp32, m = 4: 71 us (40), of 4096 bf16 294
// (79).  Of streamed rows 2048 of 65536 bf16 take 607 us (319 without the balance
// loss; 40): the search 319 at 16 warps, the mass, read by single elements, 118,
// and the finish of 65536 columns in fp64 167.
#pragma once

#include "gate_internal.cuh"

namespace gmm {
namespace gate {

constexpr int kGateWarpThreads = 256;
constexpr int kGateBlockThreads = 512;
constexpr int kGateStreamGrid = 2 * kSms;
constexpr int kGateMassBlocks = 16;  // stretches of rows that are streamed
// Blocks that keep sums, at most: grids are as many as the device holds at once or
// these, and the workspace has room for these, which it has to know without asking
// the device.  8 bytes a column each: 20 MB at 8192 columns, 80 MB at 65536.
inline int gate_blocks(int K) { return (K <= 512 ? 4 : K <= 1100 ? 8 : K <= 4096 ? 4 : K <= 8192 ? 2 : 1) * kSms; }

// How many blocks left rows and entries, mass, and counts; none: a failure.
struct GateBlocks {
  int heads, mass, counts;
};

// A block's sums of the balance outputs, and of rows that are streamed what
// their second reading takes.
struct GateWs {
  float* mass;       // blocks * K
  int32_t* counts;   // blocks * K (of streamed rows: K)
  int32_t* rows;     // blocks: rows that count
  int32_t* kept;     // blocks: entries
  double* part;      // of the finish's blocks
  uint32_t* ticket;
  float2* scale;     // N: base (or top), 1 / sum
};

struct GateArgs {
  const void* L;
  const uint8_t* live;
  int32_t* ids;
  float *gamma, *lse;
  int64_t N;
  int K, m, normalised, balance;
  GateWs ws;
};

GateBlocks launch_gate_f32(const GateArgs& a, cudaStream_t s);
GateBlocks launch_gate_f16(const GateArgs& a, cudaStream_t s);
GateBlocks launch_gate_bf16(const GateArgs& a, cudaStream_t s);

namespace rows_impl {

constexpr uint32_t kNone = 0u;  // below every number's order

// A number's order; a logit that is not there (-inf) has none.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t o = ordered(x);
  return o > kOrderedNegInf ? o : kNone;
}

template <int V> __device__ __forceinline__ float vector_max(const Vec<float, V>& x) {
  float m = x.v[0];
#pragma unroll
  for (int e = 1; e < V; ++e) m = max_nan(m, x.v[e]);
  return m;
}
template <int V> __device__ __forceinline__ float vector_max(const Vec<__half, V>& x) {
  __half2 m = pair_at(x, 0);
#pragma unroll
  for (int e = 2; e < V; e += 2) m = __hmax2_nan(m, pair_at(x, e));
  return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}
template <int V> __device__ __forceinline__ float vector_max(const Vec<__nv_bfloat16, V>& x) {
  __nv_bfloat162 m = pair_at(x, 0);
#pragma unroll
  for (int e = 2; e < V; e += 2) m = __hmax2_nan(m, pair_at(x, e));
  return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
}

// The place of the first element equal to the vector's largest, `m` (a NaN: of
// the first NaN; there is none where m is a number).
template <typename T, int V> __device__ __forceinline__ int first_of_any(const Vec<T, V>& x, float m) {
  int at = V - 1;
#pragma unroll
  for (int e = V - 2; e >= 0; --e) {
    const float f = to_f(x.v[e]);
    if (f == m || f != f) at = e;
  }
  return at;
}
template <int V> __device__ __forceinline__ int first_of(const Vec<float, V>& x, float m) { return first_of_any(x, m); }
// Pairs compared at once: a bit for each element, those of the high halves above.
__device__ __forceinline__ int first_bit(uint32_t bits) { return __ffs((int)((bits | bits >> 16) & 0xffffu)) - 1; }
template <int V> __device__ __forceinline__ int first_of(const Vec<__half, V>& x, float m) {
  if (m != m) return first_of_any(x, m);
  const __half2 t = __float2half2_rn(m);
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    bits |= __heq2_mask(pair_at(x, e), t) & (1u << e | 1u << (16 + e + 1));
  return first_bit(bits);
}
template <int V> __device__ __forceinline__ int first_of(const Vec<__nv_bfloat16, V>& x, float m) {
  if (m != m) return first_of_any(x, m);
  const __nv_bfloat162 t = __float2bfloat162_rn(m);
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    bits |= __heq2_mask(pair_at(x, e), t) & (1u << e | 1u << (16 + e + 1));
  return first_bit(bits);
}

// A candidate of a warp's team: a number's order and its place among the team's
// up to 1024 (in the columns' order).  Larger is better: by value, then the lower
// place.  In one word for 16-bit types, whose orders as floats have 19 bits.
template <typename T> struct Key {
  uint32_t k;
  static __device__ __forceinline__ Key none() { return {0}; }
  static __device__ __forceinline__ Key make(uint32_t order, uint32_t place) {
    return {(order & 0xffffe000u) | (8191u - place)};
  }
  __device__ __forceinline__ bool is() const { return k != 0; }
  __device__ __forceinline__ bool same(const Key& o) const { return k == o.k; }
  // the low bits of an order: ones of a negative number, none of a positive one
  __device__ __forceinline__ uint32_t order() const { return (k & 0xffffe000u) | (k >> 31 ? 0u : 0x1fffu); }
  __device__ __forceinline__ uint32_t place() const { return 8191u - (k & 8191u); }
  template <int S> __device__ __forceinline__ Key best() const {
    if constexpr (S == 32) return {__reduce_max_sync(0xffffffffu, k)};
    uint32_t b = k;
#pragma unroll
    for (int s = S / 2; s; s >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, s));
    return {b};
  }
};
template <> struct Key<float> {
  uint32_t o, c;
  static __device__ __forceinline__ Key none() { return {kNone, 0}; }
  static __device__ __forceinline__ Key make(uint32_t order, uint32_t place) { return {order, ~place}; }
  __device__ __forceinline__ bool is() const { return o != kNone; }
  __device__ __forceinline__ bool same(const Key& k) const { return o == k.o && c == k.c; }
  __device__ __forceinline__ uint32_t order() const { return o; }
  __device__ __forceinline__ uint32_t place() const { return ~c; }
  template <int S> __device__ __forceinline__ Key best() const {
    Key b;
    if constexpr (S == 32) {
      b.o = __reduce_max_sync(0xffffffffu, o);
      b.c = __reduce_max_sync(0xffffffffu, o == b.o ? c : 0u);
    } else {
      b.o = o;
#pragma unroll
      for (int s = S / 2; s; s >>= 1) b.o = max(b.o, __shfl_xor_sync(0xffffffffu, b.o, s));
      b.c = o == b.o ? c : 0u;
#pragma unroll
      for (int s = S / 2; s; s >>= 1) b.c = max(b.c, __shfl_xor_sync(0xffffffffu, b.c, s));
    }
    return b;
  }
};

// A lane's best element not yet taken.  The second best (of more than four
// entries the third too) is found beforehand, by all lanes at once: a lane that
// is taken from more often looks on by itself, while the others wait.
template <typename T, int V, int NV, int S, typename F>
struct Best {
  static constexpr bool kWideRows = V > 1;
  static constexpr int N = kWideRows ? NV : V * NV;
  Key<T> key, next, third;
  uint32_t o[N];  // of each vector's (element's) largest left
  int j, e;       // where the last one picked is
  int known;      // how many of `next` and `third` are left

  __device__ __forceinline__ void start(const Row<T, V, NV>& r, const F& feed, int m) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (kWideRows) o[i] = order_of(vector_max(r.r[i]));
      else o[i] = order_of(to_f(r.at(i)));
    }
    key = pick(feed);
    known = m > 4 ? 2 : m > 1;
    next = third = Key<T>::none();
    if (m > 1) {
      drop(feed);
      next = pick(feed);
    }
    if (m > 4) {
      drop(feed);
      third = pick(feed);
    }
  }
  __device__ __forceinline__ Key<T> pick(const F& feed) {
    uint32_t order = o[0];
    j = 0, e = 0;
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (o[i] > order) order = o[i], j = i;
    if (order == kNone) return Key<T>::none();
    if constexpr (kWideRows) e = first_of(feed.vector(j), unordered(order));
    return Key<T>::make(order, (uint32_t)((j * S + (feed.lane & (S - 1))) * V + e));
  }
  // Takes the one last picked away.
  __device__ __forceinline__ void drop(const F& feed) {
    uint32_t left = kNone;
    if constexpr (kWideRows) {
      reinterpret_cast<T*>(feed.word(j))[e] = from_f<T>(-INFINITY);
      left = order_of(vector_max(feed.vector(j)));
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i == j) o[i] = left;
  }
  // Takes the best away from the lane that `won` (all of the warp call it).
  __device__ __forceinline__ void pop(const F& feed, bool won) {
    const bool look = won && known == 0;
    if (won) key = next, next = third, --known;
    if (__any_sync(0xffffffffu, look)) {
      if (look) {
        drop(feed);
        key = pick(feed);
        known = 0;
      }
    }
  }
};

// log of a row's sum of exponentials, taken with `base`.
__device__ __forceinline__ float log_sum(const Base& b, float k, float sum) {
  return b.top + kLn2 * (lg2(sum) - b.over(k));
}

// Adds a block's sums to the workspace: `rows` and `kept` of its threads.
__device__ __forceinline__ void store_counts(const GateArgs& a, int rows, int kept) {
  __shared__ int part[32];
  rows = block_reduce(rows, 0, SumOp(), part);
  kept = block_reduce(kept, 0, SumOp(), part);
  if (threadIdx.x == 0) {
    a.ws.rows[blockIdx.x] = rows;
    a.ws.kept[blockIdx.x] = kept;
    if (blockIdx.x == 0) *a.ws.ticket = 0;
  }
}

template <typename T, int V, int NV, int S, bool BALANCE>
__global__ void __launch_bounds__(kGateWarpThreads) gate_warp_kernel(GateArgs a) {
  extern __shared__ __align__(16) char smem[];
  constexpr int P = V * NV / 2, per = 32 / S;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const int l = threadIdx.x & 31, K = a.K, nv = K / V, m = a.m;
  const int64_t warp = ((int64_t)blockIdx.x * kGateWarpThreads + threadIdx.x) >> 5;
  const int64_t stride = (int64_t)gridDim.x * (kGateWarpThreads / 32) * per;
  WarpTeam<S> team(l & (S - 1), S);
  const T none = from_f<T>(-INFINITY);
  float* cols = reinterpret_cast<float*>(smem + F::bytes(kGateWarpThreads));  // K, at the end
  int32_t* counts = reinterpret_cast<int32_t*>(cols + K);
  if (BALANCE) {
    for (int k = threadIdx.x; k < K; k += kGateWarpThreads) counts[k] = 0;
    __syncthreads();
  }
  int64_t n = warp * per + l / S;
  F feed;
  feed.start(smem, {(const T*)a.L}, n, stride, a.N, K, team.lane, S, nv, none, LiveRows{a.live});
  float2 mass[BALANCE ? P : 1];
#pragma unroll
  for (int i = 0; i < (BALANCE ? P : 1); ++i) mass[i] = both(0.f);
  int rows = 0, kept = 0;
  int64_t at = n * m;
  for (int64_t end = warp * per; end < a.N; n += stride, end += stride, at += stride * m) {
    Row<T, V, NV> row[1];
    if (!feed.next(row)) row[0].fill(none);
    Best<T, V, NV, S, F> best;
    best.start(row[0], feed, m);
    // lane t takes the t-th; one lane alone writes them as they come
    Key<T> mine = Key<T>::none(), first = Key<T>::none();
    float other[S == 1 ? kMaxTop : 1];
    if constexpr (S == 1) {
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t) {
        if (t >= m) break;
        const Key<T> k = best.key;
        if (t == 0) first = k;
        other[t] = k.is() ? unordered(k.order()) : -INFINITY;
        if (n < a.N) a.ids[at + t] = k.is() ? (int)k.place() : -1;
        if (BALANCE && k.is()) {
          atomicAdd(counts + k.place(), 1);
          ++kept;
        }
        if (t + 1 < m) best.pop(feed, k.is());
      }
    } else {
#pragma unroll 1
      for (int t = 0; t < m; ++t) {
        const Key<T> k = best.key.template best<S>();
        if (t == 0) first = k;
        if (team.lane == t) mine = k;
        if (t + 1 < m) best.pop(feed, k.is() && k.same(best.key));  // places are one lane's
      }
    }
    const bool some = first.is();
    const Base base(some ? unordered(first.order()) : -INFINITY, kLog2E);
    float2 x[P];
    row[0].get(x);
    exponentials(x, base, kLog2E);
    float s[1] = {total(x)};
    team.sum(s);
    const float rsum = some ? rcp(s[0]) : 0.f;
    if (BALANCE) {
#pragma unroll
      for (int i = 0; i < P; ++i) mass[i] = fma2(x[i], both(rsum), mass[i]);
    }
    if (S == 1) {
      float all = 0.f;
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t)
        if (t < m) {
          float& e = other[S == 1 ? t : 0];
          e = e == -INFINITY ? 0.f : ex2(base(e, kLog2E));
          all += e;
        }
      const float r = !some ? 0.f : a.normalised ? rcp(s[0] == s[0] ? all : s[0]) : rsum;
#pragma unroll
      for (int t = 0; t < kMaxTop; ++t)
        if (t < m && n < a.N) a.gamma[at + t] = other[S == 1 ? t : 0] * r;
    } else {
      const float e = mine.is() ? ex2(base(unordered(mine.order()), kLog2E)) : 0.f;
      float r = rsum;
      if (a.normalised) {
        float all[1] = {e};
        team.sum(all);
        r = some ? rcp(s[0] == s[0] ? all[0] : s[0]) : 0.f;
      }
      if (team.lane < m && n < a.N) {
        a.ids[at + team.lane] = mine.is() ? (int)mine.place() : -1;
        a.gamma[at + team.lane] = mine.is() ? e * r : 0.f;
        if (BALANCE && mine.is()) {
          atomicAdd(counts + mine.place(), 1);
          ++kept;
        }
      }
    }
    if (team.lane == 0 && n < a.N) {
      if (a.lse) a.lse[n] = some ? log_sum(base, kLog2E, s[0]) : -INFINITY;
      rows += some;
    }
  }
  if (!BALANCE) return;
  let_next_start();
  // the warp's groups, then the warps in order
#pragma unroll
  for (int i = 0; i < (BALANCE ? P : 1); ++i)
#pragma unroll
    for (int o = 16; o >= S; o >>= 1) {
      mass[i].x += __shfl_xor_sync(0xffffffffu, mass[i].x, o);
      mass[i].y += __shfl_xor_sync(0xffffffffu, mass[i].y, o);
    }
  for (int turn = 0; turn < kGateWarpThreads / 32; ++turn) {
    if ((int)(threadIdx.x >> 5) == turn && l < S) {
#pragma unroll
      for (int i = 0; i < V * NV; ++i) {
        const int c = column<V>(i, l, S);
        const float2 f = mass[BALANCE ? i / 2 : 0];
        if (c < K) cols[c] = (turn ? cols[c] : 0.f) + (i & 1 ? f.y : f.x);
      }
    }
    __syncthreads();
  }
  for (int k = threadIdx.x; k < K; k += kGateWarpThreads) {
    a.ws.mass[(size_t)blockIdx.x * K + k] = cols[k];
    a.ws.counts[(size_t)blockIdx.x * K + k] = counts[k];
  }
  store_counts(a, rows, kept);
}

// One warp joins the block's lists: lane i has words i, i + 32, ... of `all` * 8.
// Lane t ends with the t-th, as its order and column.
__device__ __forceinline__ void join_lists(const uint64_t* keys, int all, int m, uint32_t& mine, uint32_t& id) {
  const int l = threadIdx.x & 31;
  uint64_t k[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) k[i] = l + 32 * i < all * kMaxTop && (l & 7) < m ? keys[l + 32 * i] : 0;
  mine = kNone, id = 0;
  for (int t = 0; t < m; ++t) {
    uint64_t b = k[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) b = k[i] > b ? k[i] : b;
    const uint32_t o = __reduce_max_sync(0xffffffffu, (uint32_t)(b >> 32));
    const uint32_t c = __reduce_max_sync(0xffffffffu, (uint32_t)(b >> 32) == o ? (uint32_t)b : 0u);
    const uint64_t won = (uint64_t)o << 32 | c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k[i] == won) k[i] = 0;
    if (l == t) mine = o, id = ~c;
  }
}

// A row's outputs from its list, by one warp.
__device__ __forceinline__ int store_row(const GateArgs& a, int64_t n, uint32_t mine, uint32_t id, bool some,
                                         const Base& base, float sum) {
  const int l = threadIdx.x & 31;
  const float e = mine == kNone ? 0.f : ex2(base(unordered(mine), kLog2E));
  float r = some ? rcp(sum) : 0.f;
  if (a.normalised) {
    const float all = warp_reduce(e, SumOp());
    r = some ? rcp(sum == sum ? all : sum) : 0.f;
  }
  if (l < a.m) {
    a.ids[n * a.m + l] = mine == kNone ? -1 : (int)id;
    a.gamma[n * a.m + l] = mine == kNone ? 0.f : e * r;
  }
  if (l == 0 && a.lse) a.lse[n] = some ? log_sum(base, kLog2E, sum) : -INFINITY;
  return l < a.m && mine != kNone;
}

template <typename T, int V, int NV, bool BALANCE>
__global__ void __launch_bounds__(kGateBlockThreads) gate_block_kernel(GateArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[BlockTeam<false>::kWords];
  __shared__ uint64_t lists[2][16 * kMaxTop];
  constexpr int P = V * NV / 2;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5, K = a.K, nv = K / V, m = a.m;
  BlockTeam<false> team(part, blockDim.x);
  const T none = from_f<T>(-INFINITY);
  int32_t* counts = reinterpret_cast<int32_t*>(smem + F::bytes(blockDim.x));
  if (BALANCE) {
    for (int k = threadIdx.x; k < K; k += blockDim.x) counts[k] = 0;
    __syncthreads();
  }
  F feed;
  feed.start(smem, {(const T*)a.L}, blockIdx.x, gridDim.x, a.N, K, team.lane, team.size, nv, none, LiveRows{a.live});
  float2 mass[BALANCE ? P : 1];
#pragma unroll
  for (int i = 0; i < (BALANCE ? P : 1); ++i) mass[i] = both(0.f);
  int rows = 0, kept = 0, duty = 0;
  uint32_t turn = 0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, turn ^= 1, duty = duty + 1 == team.all ? 0 : duty + 1) {
    Row<T, V, NV> row[1];
    if (!feed.next(row)) row[0].fill(none);
    Best<T, V, NV, 32, F> best;
    best.start(row[0], feed, m);
    Key<T> first = Key<T>::none(), tth = Key<T>::none();
#pragma unroll 1
    for (int t = 0; t < m; ++t) {
      const Key<T> k = best.key.template best<32>();
      if (t == 0) first = k;
      if (l == t) tth = k;
      if (t + 1 < m) best.pop(feed, k.is() && k.same(best.key));
    }
    if (l < m) {
      const int v = (int)tth.place() / V, c = ((v / 32) * team.size + w * 32 + v % 32) * V + (int)tth.place() % V;
      lists[turn][w * kMaxTop + l] = tth.is() ? (uint64_t)tth.order() << 32 | (uint32_t)~c : 0;
    }
    const float mine = first.is() ? unordered(first.order()) : -INFINITY;
    float2 x[P];
    row[0].get(x);
    exponentials(x, Base(mine, kLog2E), kLog2E);
    float s[1] = {total(x)}, top;
    team.tell(s, mine);
    __syncthreads();
    const float own = team.hear(s, top, mine, kLog2E);
    const bool some = top != -INFINITY;
    if (BALANCE) {
      const float2 f = both(some ? own * rcp(s[0]) : 0.f);
#pragma unroll
      for (int i = 0; i < P; ++i) mass[i] = fma2(x[i], f, mass[i]);
    }
    if (w == duty) {
      uint32_t order, id;
      join_lists(lists[turn], team.all, m, order, id);
      const int is = store_row(a, n, order, id, some, Base(top, kLog2E), s[0]);
      if (BALANCE && is) atomicAdd(counts + id, 1);
      kept += is;
      rows += some && l == 0;
    }
  }
  if (!BALANCE) return;
  let_next_start();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V * NV; ++i) {
    const int c = column<V>(i, team.lane, team.size);
    const float2 f = mass[BALANCE ? i / 2 : 0];
    if (c < K) a.ws.mass[(size_t)blockIdx.x * K + c] = i & 1 ? f.y : f.x;
  }
  for (int k = threadIdx.x; k < K; k += blockDim.x) a.ws.counts[(size_t)blockIdx.x * K + k] = counts[k];
  store_counts(a, rows, kept);
}

// Rows that no block holds.  A warp keeps the m largest so far, lane t the t-th;
// a batch is looked through only where its largest logits pass the last of them.
template <typename T>
__global__ void __launch_bounds__(kGateBlockThreads, 1) gate_stream_kernel(GateArgs a) {
  __shared__ float part[BlockTeam<false>::kWords];
  __shared__ uint64_t lists[2][16 * kMaxTop];
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5, K = a.K, m = a.m;
  BlockTeam<false> team(part, kGateBlockThreads);
  int32_t* counts = a.ws.counts;  // one for all blocks; sums of whole numbers have no order
  int rows = 0, kept = 0;
  uint32_t turn = 0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, turn ^= 1) {
    const T* L = (const T*)a.L + n * K;
    const bool on = !a.live || a.live[n];
    uint64_t list = 0, last = 0;  // lane t's, and the m-th
    float top = -INFINITY, sum = 0.f;
    // Takes what passes into the warp's list: `best(bound)` is a lane's largest
    // key up to `bound`.
    auto take = [&](auto best) {
      uint64_t bound = ~0ull;
      while (true) {
        const uint64_t b = best(bound);
        const uint32_t o = __reduce_max_sync(0xffffffffu, (uint32_t)(b >> 32));
        const uint32_t c = __reduce_max_sync(0xffffffffu, (uint32_t)(b >> 32) == o ? (uint32_t)b : 0u);
        const uint64_t won = (uint64_t)o << 32 | c;
        if (o == kNone || won <= last) break;
        const int at = __popc(__ballot_sync(0xffffffffu, l < m && list > won));
        const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
        list = l == at ? won : l > at ? up : list;
        if (l >= m) list = 0;
        last = __shfl_sync(0xffffffffu, list, m - 1);
        bound = won - 1;
      }
    };
    if (on) {
      constexpr int V = kWide<T>, U = 4;
      const int h0 = (int)((16 - ((uintptr_t)L & 15)) & 15) / (int)sizeof(T), head = h0 < K ? h0 : K;
      const int nv = (K - head) / V, tail = head + nv * V;
      const int t = threadIdx.x;
      const int edge = t < head ? t : t - head < K - tail ? tail + t - head : -1;
      const float xe = edge >= 0 ? to_f(L[edge]) : -INFINITY;
      take([&](uint64_t bound) {
        const uint64_t key = (uint64_t)order_of(xe) << 32 | (uint32_t)~edge;
        return key <= bound && order_of(xe) != kNone ? key : 0ull;
      });
      top = xe;
      if (xe != -INFINITY) sum = ex2(Base(xe, kLog2E)(xe, kLog2E));
      const int turns = (nv + U * kGateBlockThreads - 1) / (U * kGateBlockThreads);
      for (int i = 0; i < turns; ++i) {
        const int v0 = i * U * kGateBlockThreads + t;
        Row<T, V, U> x;
        x.fill(from_f<T>(-INFINITY));
        x.read(L + head + (int64_t)(v0 - t) * V, t, kGateBlockThreads, nv - (v0 - t));
        const float high = lane_max(x), to = max_nan(top, high);
        if (to != top) {
          sum *= BlockTeam<false>::between(top, to, kLog2E);
          top = to;
        }
        if (__any_sync(0xffffffffu, order_of(high) != kNone && order_of(high) >= (uint32_t)(last >> 32)))
          take([&](uint64_t bound) {
            uint64_t best = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int e = 0; e < V; ++e) {
                const uint32_t o = order_of(to_f(x.r[u].v[e]));
                const uint64_t key = (uint64_t)o << 32 | (uint32_t)~(head + (v0 + u * kGateBlockThreads) * V + e);
                if (o != kNone && key <= bound && key > best) best = key;
              }
            return best;
          });
        float2 f[U * V / 2];
        x.get(f);
        exponentials(f, Base(top, kLog2E), kLog2E);
        sum += total(f);
      }
    }
    if (l < m) lists[turn][w * kMaxTop + l] = list;
    const float mine = warp_max(top);
    float s[1] = {sum * BlockTeam<false>::between(top, mine == -INFINITY ? 0.f : mine, kLog2E)};
    team.tell(s, mine);
    __syncthreads();
    team.hear(s, top, mine, kLog2E);
    const bool some = top != -INFINITY;
    if (w == 0) {
      uint32_t order, id;
      join_lists(lists[turn], team.all, m, order, id);
      const Base base(top, kLog2E);
      const int is = store_row(a, n, order, id, some, base, s[0]);
      if (a.balance) {
        if (is) atomicAdd(counts + id, 1);
        if (l == 0) a.ws.scale[n] = make_float2(some ? top : 0.f, some ? rcp(s[0]) : 0.f);
      }
      kept += is;
      rows += some && l == 0;
    }
  }
  if (a.balance) store_counts(a, rows, kept);
}

// The mass of streamed rows, a thread a column, blockIdx.y a stretch of rows: N / 16
// additions one after another, so with what their roundings leave.
constexpr int kMassThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kMassThreads) gate_mass_kernel(GateArgs a, int64_t stretch) {
  const int k = blockIdx.x * kMassThreads + threadIdx.x;
  if (k >= a.K) return;
  const int64_t begin = blockIdx.y * stretch, end = begin + stretch < a.N ? begin + stretch : a.N;
  Sum2 sum;
#pragma unroll 8
  for (int64_t n = begin; n < end; ++n) {
    const float2 c = a.ws.scale[n];
    if (a.live && !a.live[n]) continue;
    const float x = to_f(((const T*)a.L)[n * a.K + k]);
    sum.add(c.y == 0.f ? 0.f : ex2(Base(c.x, kLog2E)(x, kLog2E)) * c.y);
  }
  a.ws.mass[(size_t)blockIdx.y * a.K + k] = (float)sum.value();
}

template <typename T, int V, int E, int S>
GateBlocks launch_lanes(const GateArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done[2];
  constexpr int NV = E / V;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const size_t feed = F::bytes(kGateWarpThreads);
  const int64_t rows = kGateWarpThreads / S, need = (a.N + rows - 1) / rows;
  static ResidentCache cache[2];
  int64_t grid = need < 1 ? 1 : need;
  auto at_most = [&](int64_t n) { grid = grid < n ? grid : n; };
  if (a.balance) {
    if (!allow_smem((const void*)gate_warp_kernel<T, V, NV, S, true>, feed + 8 * E * S, done[1])) return {};
    const size_t smem = feed + 8 * E * S;
    at_most(gate_blocks(a.K));
    at_most(resident(gate_warp_kernel<T, V, NV, S, true>, kGateWarpThreads, smem, cache[1]));
    gate_warp_kernel<T, V, NV, S, true><<<(unsigned)grid, kGateWarpThreads, feed + 8 * a.K, s>>>(a);
  } else {
    if (!allow_smem((const void*)gate_warp_kernel<T, V, NV, S, false>, feed, done[0])) return {};
    at_most(resident(gate_warp_kernel<T, V, NV, S, false>, kGateWarpThreads, feed, cache[0]));
    gate_warp_kernel<T, V, NV, S, false><<<(unsigned)grid, kGateWarpThreads, feed, s>>>(a);
  }
  return {(int)grid, (int)grid, (int)grid};
}

template <typename T, int V, int E>
GateBlocks launch_block(const GateArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done[2];
  constexpr int NV = E / V;
  using F = Feed<T, V, NV, 1, LiveRows>;
  const int threads = ((a.K + E - 1) / E + 31) / 32 * 32;
  static ResidentCache cache[2];
  int64_t grid = a.N < 1 ? 1 : a.N;
  auto at_most = [&](int64_t n) { grid = grid < n ? grid : n; };
  const size_t feed = F::bytes(threads);
  if (a.balance) {
    if (!allow_smem((const void*)gate_block_kernel<T, V, NV, true>, F::bytes(kGateBlockThreads) + 4 * E * kGateBlockThreads, done[1])) return {};
    at_most(gate_blocks(a.K));
    at_most(resident(gate_block_kernel<T, V, NV, true>, threads, feed + 4 * (size_t)E * threads, cache[1]));
    gate_block_kernel<T, V, NV, true><<<(unsigned)grid, threads, feed + 4 * (size_t)a.K, s>>>(a);
  } else {
    if (!allow_smem((const void*)gate_block_kernel<T, V, NV, false>, F::bytes(kGateBlockThreads), done[0])) return {};
    at_most(resident(gate_block_kernel<T, V, NV, false>, threads, feed, cache[0]));
    gate_block_kernel<T, V, NV, false><<<(unsigned)grid, threads, feed, s>>>(a);
  }
  return {(int)grid, (int)grid, (int)grid};
}

template <typename T>
GateBlocks launch_gate(const GateArgs& a, cudaStream_t s) {
  constexpr int V = kWide<T>;
  const int K = a.K;
  if (wide<T>(K, (const char*)a.L)) {
    if (K <= 8) return launch_lanes<T, V, 8, 1>(a, s);
    if (K <= 64) return launch_lanes<T, V, 8, 8>(a, s);
    if (K <= 128) return launch_lanes<T, V, 16, 8>(a, s);
    if (K <= 256) return launch_lanes<T, V, 32, 8>(a, s);
    if (K <= 512) return launch_lanes<T, V, 32, 16>(a, s);
    if (K <= 1024) return launch_lanes<T, V, 32, 32>(a, s);
    constexpr int E = sizeof(T) == 2 ? 32 : 16;  // rows ahead and counts fit in shared memory
    if (K <= E * kGateBlockThreads) return launch_block<T, V, E>(a, s);
  } else {
    if (K <= 64) return launch_lanes<T, 1, 8, 8>(a, s);
    if (K <= 128) return launch_lanes<T, 1, 8, 16>(a, s);
    if (K <= 256) return launch_lanes<T, 1, 8, 32>(a, s);
    if (K <= 512) return launch_lanes<T, 1, 16, 32>(a, s);
    if (K <= 16 * kGateBlockThreads) return launch_block<T, 1, 16>(a, s);
  }
  const int64_t grid = a.N < 1 ? 1 : a.N < kGateStreamGrid ? a.N : kGateStreamGrid;
  if (a.balance && cudaMemsetAsync(a.ws.counts, 0, sizeof(int32_t) * (size_t)K, s) != cudaSuccess) return {};
  gate_stream_kernel<T><<<(unsigned)grid, kGateBlockThreads, 0, s>>>(a);
  const int64_t blocks = grid < kGateMassBlocks ? grid : kGateMassBlocks;
  if (a.balance) {
    const dim3 g((K + kMassThreads - 1) / kMassThreads, (unsigned)blocks);
    gate_mass_kernel<T><<<g, kMassThreads, 0, s>>>(a, (a.N + blocks - 1) / blocks);
  }
  return {(int)grid, (int)blocks, 1};
}

}  // namespace rows_impl
}  // namespace gate
}  // namespace gmm
