// gate_internal.cuh - helpers shared by the learned gate's kernels.
//
// A row is held in registers by a team of threads: 1 to 32 lanes of a warp for
// short rows, a block, or a cluster of blocks for long ones.  Vector j of lane i
// of a team of `size` is number j * size + i of the row, V elements each: 16
// bytes where every row starts on such a boundary, else one element.
#pragma once

#include "expert_internal.cuh"
#include "gmm_gate.h"

namespace gmm {
namespace gate {

constexpr int kMaxTop = 8;       // entries of a gate's row
constexpr int kMaxTeacher = 64;  // entries of a teacher's row
constexpr int kSms = 152;

template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T v[V]; };

// Elements of one vector of a row: 16 bytes where the row length and all
// addresses allow it.
template <typename T> constexpr int kWide = 16 / (int)sizeof(T);
template <typename T, typename... P>
inline bool wide(int64_t width, const P*... p) {
  return width % kWide<T> == 0 && aligned(16, (const char*)p...);
}

// Two neighbouring elements as one word, in fp32, and back.
template <typename T> struct PairOf { using type = float2; };
template <> struct PairOf<__half> { using type = __half2; };
template <> struct PairOf<__nv_bfloat16> { using type = __nv_bfloat162; };
template <typename T> using Pair = typename PairOf<T>::type;

__device__ __forceinline__ float2 pair_of(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ __half2 pair_of(__half a, __half b) { return __halves2half2(a, b); }
__device__ __forceinline__ __nv_bfloat162 pair_of(__nv_bfloat16 a, __nv_bfloat16 b) { return __halves2bfloat162(a, b); }
__device__ __forceinline__ float2 to_f2(float2 a) { return a; }
__device__ __forceinline__ float2 to_f2(__half2 a) { return __half22float2(a); }
__device__ __forceinline__ float2 to_f2(__nv_bfloat162 a) { return __bfloat1622float2(a); }
template <typename T> __device__ __forceinline__ Pair<T> from_f2(float2 f);
template <> __device__ __forceinline__ float2 from_f2<float>(float2 f) { return f; }
template <> __device__ __forceinline__ __half2 from_f2<__half>(float2 f) { return __float22half2_rn(f); }
template <> __device__ __forceinline__ __nv_bfloat162 from_f2<__nv_bfloat16>(float2 f) { return __float22bfloat162_rn(f); }
// Elements e and e + 1 of a vector (e even).
template <typename T, int V> __device__ __forceinline__ Pair<T> pair_at(const Vec<T, V>& x, int e) {
  static_assert(V % 2 == 0, "pairs");
  return *reinterpret_cast<const Pair<T>*>(&x.v[e]);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// What a lane has of a row, as it is stored; its elements in order are pairs
// of fp32 numbers to the arithmetic.
template <typename T, int V, int NV>
struct Row {
  static constexpr int E = V * NV;
  static_assert(E % 2 == 0, "pairs");
  Vec<T, V> r[NV];
  __device__ __forceinline__ void fill(T none) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) r[j].v[e] = none;
  }
  __device__ __forceinline__ void store(T* __restrict__ p, int lane, int size, int nv) const {
    p += (int64_t)lane * V;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * size + lane < nv) *reinterpret_cast<Vec<T, V>*>(p + j * size * V) = r[j];
  }
  // What is inside the row; the rest is not written.
  __device__ __forceinline__ void read(const T* __restrict__ p, int lane, int size, int nv) {
    p += (int64_t)lane * V;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * size + lane < nv) r[j] = *reinterpret_cast<const Vec<T, V>*>(p + j * size * V);
  }
  __device__ __forceinline__ T& at(int i) { return r[i / V].v[i % V]; }
  __device__ __forceinline__ const T& at(int i) const { return r[i / V].v[i % V]; }
  __device__ __forceinline__ Pair<T> pair(int i) const {  // elements 2 i and 2 i + 1
    if constexpr (V == 1) return pair_of(at(2 * i), at(2 * i + 1));
    else return pair_at(r[2 * i / V], 2 * i % V);
  }
  __device__ __forceinline__ void get(float2 (&f)[E / 2]) const {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) f[i] = to_f2(pair(i));
  }
  __device__ __forceinline__ void set(const float2 (&f)[E / 2]) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const Pair<T> p = from_f2<T>(f[i]);
      if constexpr (V == 1) at(2 * i) = reinterpret_cast<const T*>(&p)[0], at(2 * i + 1) = reinterpret_cast<const T*>(&p)[1];
      else *reinterpret_cast<Pair<T>*>(&r[2 * i / V].v[2 * i % V]) = p;
    }
  }
};

// Which rows are fetched at all.
struct EveryRow {
  static constexpr bool kMasked = false;
  __device__ __forceinline__ bool operator()(int64_t) const { return true; }
};
struct LiveRows {  // bytes, or NULL
  static constexpr bool kMasked = true;
  const uint8_t* live;
  __device__ __forceinline__ bool operator()(int64_t n) const { return !live || live[n] != 0; }
};
struct WeightedRows {  // weights, or NULL
  static constexpr bool kMasked = true;
  const float* weights;
  __device__ __forceinline__ bool operator()(int64_t n) const { return !weights || weights[n] != 0.f; }
};

// Nothing beside the rows.
struct NoWords {
  __device__ __forceinline__ void fetch(uint32_t, bool) {}
};
// NW words of 4 bytes a lane that come with each row: entry `lane` of the m that
// a row has in each array.
template <int NW, int STAGES>
struct Words {
  static constexpr size_t bytes(int threads) { return (size_t)STAGES * NW * threads * 4; }
  const char* from[NW];  // NULL: none; this lane's of the next row
  int64_t step;
  char* slot;
  bool mine;  // whether this lane has an entry
  __device__ __forceinline__ void start(char* smem, int lane, int m, int64_t stride) {
    slot = smem + threadIdx.x * 4;
    mine = lane < m;
    step = stride * m * 4;
  }
  template <typename T>
  __device__ __forceinline__ void array(int w, const T* p, int64_t row, int lane, int m) {
    static_assert(sizeof(T) == 4, "words");
    from[w] = p ? reinterpret_cast<const char*>(p + row * m + lane) : nullptr;
  }
  __device__ __forceinline__ void fetch(uint32_t into, bool there) {
#pragma unroll
    for (int w = 0; w < NW; ++w)
      if (from[w]) {
        if (there && mine)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(
                           slot + (size_t)(into * NW + w) * blockDim.x * 4)),
                       "l"(from[w])
                       : "memory");
        from[w] += step;
      }
  }
  template <typename T> __device__ __forceinline__ T word(uint32_t stage, int w) const {
    return *reinterpret_cast<const T*>(slot + (size_t)(stage * NW + w) * blockDim.x * 4);
  }
};

// A lane's own vectors of the rows ahead, of NA arrays of one shape.  They wait in
// shared memory, put there by asynchronous copies kStages - 1 rows before they are
// used: the bytes in flight that HBM needs, without registers for them.  A lane
// reads what it copied itself, so there is nothing to synchronise.  Single 16-bit
// elements, for which there is no such copy, wait in registers, one row ahead.
template <typename T, int V, int NV, int NA, typename Rows = EveryRow>
struct Feed {
  static constexpr int kBytes = sizeof(T) * V;  // of a vector
  static constexpr bool kAsync = kBytes >= 4;
  // 512 threads' rows fit a multiprocessor's shared memory
  static constexpr int kStages = NA * NV * kBytes >= 128 ? 3 : 4;
  static constexpr size_t bytes(int threads) { return kAsync ? (size_t)kStages * NA * NV * threads * kBytes : 0; }
  const T* from[NA];  // the next row to be fetched, at this lane's first vector
  int64_t step;       // elements from a row to the next
  int left, size, lane, nv;
  char* slot;         // this thread's, [stage][array][vector][thread]
  uint32_t stage;
  Rows rows;
  int64_t row, stride;  // two behind the next one to be fetched (of masked rows alone)
  bool on, later;       // whether the next one is, and the one after it: known two rows ahead
  uint32_t were;        // whether the last ones were, a bit each
  Row<T, V, NV> ahead[kAsync ? 1 : NA];

  // Rows `row`, row + stride, ... below N of arrays of `width`-element rows; nv:
  // vectors of a row, those that a lane has past them are `none`.
  __device__ __forceinline__ void start(char* smem, const T* const (&array)[NA], int64_t row_, int64_t stride_, int64_t N,
                                        int64_t width, int lane_, int size_, int nv_, T none, Rows rows_ = Rows()) {
    NoWords no;
    start(smem, array, row_, stride_, N, width, lane_, size_, nv_, none, rows_, no);
  }
  template <typename W>
  __device__ __forceinline__ void start(char* smem, const T* const (&array)[NA], int64_t row_, int64_t stride_, int64_t N,
                                        int64_t width, int lane_, int size_, int nv_, T none, Rows rows_, W& words) {
    lane = lane_, size = size_, nv = nv_, stage = 0, step = stride_ * width;
    rows = rows_, row = row_, stride = stride_, were = 0;
    left = row < N ? (int)((N - row + stride - 1) / stride) : 0;
    if (Rows::kMasked) {
      on = left > 0 && rows(row);
      later = left > 1 && rows(row + stride);
      row += 2 * stride;
    }
#pragma unroll
    for (int a = 0; a < NA; ++a) from[a] = array[a] + row_ * width + (int64_t)lane * V;
#pragma unroll
    for (int a = 0; a < (kAsync ? 1 : NA); ++a) ahead[a].fill(none);
    if constexpr (kAsync) {
      slot = smem + threadIdx.x * kBytes;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j * size + lane >= nv)
          for (int s = 0; s < kStages * NA; ++s)
            *reinterpret_cast<Vec<T, V>*>(slot + (size_t)(s * NV + j) * blockDim.x * kBytes) = ahead[0].r[j];
#pragma unroll
      for (int s = 0; s < kStages - 1; ++s) fetch(s, words);
    } else {
      fetch(0, words);
    }
  }
  template <typename W>
  __device__ __forceinline__ void fetch(uint32_t into, W& words) {
    words.fetch(into, left > 0);
    const bool there = Rows::kMasked ? on : left > 0;
    were = were << 1 | (uint32_t)there;
    if (there) {
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (j * size + lane < nv) {
            if constexpr (kAsync) {
              const uint32_t to = (uint32_t)__cvta_generic_to_shared(
                  slot + (size_t)((into * NA + a) * NV + j) * blockDim.x * kBytes);
              if constexpr (kBytes == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from[a] + j * size * V) : "memory");
              else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from[a] + j * size * V), "n"(kBytes)
                             : "memory");
            }
            else
              ahead[a].r[j] = *reinterpret_cast<const Vec<T, V>*>(from[a] + j * size * V);
          }
    }
    if (kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
    --left;
    if (Rows::kMasked) {
      on = later;
      later = left > 1 && rows(row);
      row += stride;
    }
#pragma unroll
    for (int a = 0; a < NA; ++a) from[a] += step;
  }
  // In shared memory until the next call: this thread's vector j of the row that
  // `next` gave last, element `at` of that row whoever of the team holds it (which
  // takes a __syncwarp between lanes), and all of this thread's vectors.
  __device__ __forceinline__ uint32_t taken() const { return stage == 0 ? kStages - 1 : stage - 1; }
  __device__ __forceinline__ char* word(int j) const {
    static_assert(kAsync, "in shared memory");
    const uint32_t s = taken();
    return slot + (size_t)(s * NA * NV + j) * blockDim.x * kBytes;
  }
  __device__ __forceinline__ Vec<T, V> vector(int j) const { return *reinterpret_cast<const Vec<T, V>*>(word(j)); }
  __device__ __forceinline__ T* peer(int at) const {
    const int v = at / V, j = v / size;
    return reinterpret_cast<T*>(word(j) + (v - j * size - lane) * kBytes) + at % V;
  }
  __device__ __forceinline__ void put(const Row<T, V, NV>& r) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) *reinterpret_cast<Vec<T, V>*>(word(j)) = r.r[j];
  }
  __device__ __forceinline__ void again(Row<T, V, NV>& r) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) r.r[j] = vector(j);
  }
  // The next row and true; what was there before and false past the last one and
  // for a row that is not fetched.
  __device__ __forceinline__ bool next(Row<T, V, NV> (&out)[NA]) {
    NoWords no;
    return next(out, no);
  }
  template <typename W>
  __device__ __forceinline__ bool next(Row<T, V, NV> (&out)[NA], W& words) {
    if constexpr (kAsync) {
      fetch(stage == 0 ? kStages - 1 : stage - 1, words);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          out[a].r[j] = *reinterpret_cast<const Vec<T, V>*>(slot + (size_t)((stage * NA + a) * NV + j) * blockDim.x * kBytes);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int a = 0; a < NA; ++a) out[a] = ahead[a];
      fetch(0, words);
    }
    return were >> (kAsync ? kStages - 1 : 1) & 1u;
  }
};

// Whether a lane's element i (of the pairs above) is one of the row's.
template <int V>
__device__ __forceinline__ bool inside(int i, int lane, int size, int nv) {
  return (i / V) * size + lane < nv;
}
// The column of a lane's element i.
template <int V>
__device__ __forceinline__ int column(int i, int lane, int size) {
  return ((i / V) * size + lane) * V + i % V;
}

// A lane's columns of a vector of numbers; `none` where there is none.
template <int V, int NV, typename W>
__device__ __forceinline__ void load_columns(float2 (&c)[V * NV / 2], const W* __restrict__ p, int lane,
                                             int size, int nv, float none) {
  float f[V * NV];
#pragma unroll
  for (int i = 0; i < V * NV; ++i)
    f[i] = p && inside<V>(i, lane, size, nv) ? to_f(p[column<V>(i, lane, size)]) : none;
#pragma unroll
  for (int i = 0; i < V * NV / 2; ++i) c[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

// 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / x for x of 0.97 to 2^20 (or NaN) to an ulp, and log2 x to 2^-21.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The larger; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float warp_max(float v) {
  float y;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
  return y;
}
// A lane's largest element, in the row's own type.
template <int V, int NV>
__device__ __forceinline__ float lane_max(const Row<float, V, NV>& r) {
  float m = r.at(0);
#pragma unroll
  for (int i = 1; i < V * NV; ++i) m = max_nan(m, r.at(i));
  return m;
}
template <int V, int NV>
__device__ __forceinline__ float lane_max(const Row<__half, V, NV>& r) {
  __half2 m = r.pair(0);
#pragma unroll
  for (int i = 1; i < V * NV / 2; ++i) m = __hmax2_nan(m, r.pair(i));
  return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}
template <int V, int NV>
__device__ __forceinline__ float lane_max(const Row<__nv_bfloat16, V, NV>& r) {
  __nv_bfloat162 m = r.pair(0);
#pragma unroll
  for (int i = 1; i < V * NV / 2; ++i) m = __hmax2_nan(m, r.pair(i));
  return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
}
// x -> 2^(x k - base) with base = top k rounded: its rounding is a factor that
// all of a row have in common, so shares do not see it, and a logarithm of their
// sum takes base itself.  That factor is a number near 1 (2^-2^-5 to 2^2^-5) while
// |base| is below 2^20; from there on (masks of -1e9, small temperatures, bases
// that are infinite) the top is taken off first, which costs one more instruction.
struct Base {
  float top, base;
  __device__ __forceinline__ Base(float t, float k) : top(t == -INFINITY ? 0.f : t), base(top * k) {}
  __device__ __forceinline__ bool near() const { return fabsf(base) < 1048576.f; }  // not if NaN
  __device__ __forceinline__ float operator()(float x, float k) const {
    return near() ? fmaf(x, k, -base) : (x - top) * k;
  }
  // log2 of what the exponentials are too large by
  __device__ __forceinline__ float over(float k) const { return near() ? fmaf(top, k, -base) : 0.f; }
};
template <int P>
__device__ __forceinline__ void exponentials(float2 (&x)[P], const Base& b, float k) {
  if (!b.near()) {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = mul2(sub2(x[i], both(b.top)), both(k));
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = fma2(x[i], both(k), both(-b.base));
  }
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = make_float2(ex2(x[i].x), ex2(x[i].y));
}
template <int P>
__device__ __forceinline__ float total(const float2 (&x)[P]) {
  float2 t = x[0], u = x[1];
#pragma unroll
  for (int i = 2; i + 1 < P; i += 2) t = add2(t, x[i]), u = add2(u, x[i + 1]);
  t = add2(t, u);
  return t.x + t.y;
}

// Order of floats as unsigned numbers: -0 and 0 are one, every NaN is the largest.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kOrderedNegInf = 0x007fffffu;

// A long sum in fp32 with what its roundings left, near 48 bits: fp64 additions
// are some sixty times slower on this device.
struct Sum2 {
  float s = 0.f, left = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, z = t - s;
    left += (s - (t - z)) + (v - z);
    s = t;
  }
  // an infinite sum leaves NaN, which is not its value
  __device__ __forceinline__ double value() const { return isfinite(s) ? (double)s + left : (double)s; }
};

struct SumOp {
  template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

template <typename T, typename Op>
__device__ __forceinline__ T warp_reduce(T v, Op op) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Over the block, the same for every thread; `part`: 32 words of T.
template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, T none, Op op, T* part) {
  v = warp_reduce(v, op);
  __syncthreads();  // the last reduction's words are read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_reduce(lane < (int)(blockDim.x >> 5) ? part[lane] : none, op);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A part of a warp (or all of it): `size` lanes, a power of two; S: that, where
// it is known at compile time (else 0).
template <int S>
struct WarpTeam {
  int lane, size;
  __device__ __forceinline__ WarpTeam(int lane_, int size_) : lane(lane_), size(S ? S : size_) {}
  // The largest of the team's.
  __device__ __forceinline__ float top(float m) {
    if constexpr (S == 32) return warp_max(m);
    if (S == 0 && size == 32) return warp_max(m);
#pragma unroll
    for (int o = S ? S / 2 : 8; o; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, m, o);
      m = S || size > o ? max_nan(m, y) : m;
    }
    return m;
  }
  template <int Q> __device__ __forceinline__ void sum(float (&v)[Q]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      if (S && o >= S) continue;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        // selected rather than branched to: two instructions a step
        const float y = __shfl_xor_sync(0xffffffffu, v[q], o);
        v[q] = S || size > o ? v[q] + y : v[q];
      }
    }
  }
};

// A block, or a cluster of up to 8.  Each warp's sums of Q numbers go to shared
// memory (of every block of the cluster), where every warp adds them up.  A
// lane ends with one of the Q, so that 4 take 6 shuffles and not 20.  The words
// are in one of two halves in turn: who writes a half again has passed the
// barrier before which the others had read it.
template <bool CLUSTER>
struct BlockTeam {
  static constexpr int kWarps = CLUSTER ? 128 : 16;  // of the team
  static constexpr int kWords = 2 * 4 * kWarps;
  int lane, size;
  int all;  // warps
  float* part;
  uint32_t turn;

  // `threads` of each block, from the first on; the others may listen.
  __device__ __forceinline__ BlockTeam(float* p, int threads) : part(p), turn(0) {
    if (CLUSTER) {
      lane = (int)cluster_rank() * threads + (int)threadIdx.x;
      size = (int)cluster_blocks() * threads;
    } else {
      lane = (int)threadIdx.x;
      size = threads;
    }
    all = size >> 5;
  }
  __device__ __forceinline__ float top(float m) { return warp_max(m); }
  // As WarpTeam's, where `top` was the warp's: what a warp tells, and what every
  // warp, of the team or not, makes of it after the block's barrier.
  template <int Q> __device__ __forceinline__ void tell(const float (&v)[Q], float top) {
    static_assert(Q == 1 || Q == 2, "one or two sums, and the maxima");
    constexpr int G = 32 / Q;
    const int l = threadIdx.x & 31, q = l / G, c = l % G;
    float x = v[0];
    if (Q == 2) {
      const bool hi = l & 16;
      x = hi ? v[Q - 1] : v[0];
      x += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[Q - 1], 16);
    }
#pragma unroll
    for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    float* p = part + 4 * kWarps * turn;
    if (CLUSTER) {
      if (c < (int)cluster_blocks()) {
        to_block(p + q * kWarps + (lane >> 5), c, x);
        if (q == 0) to_block(p + 2 * kWarps + (lane >> 5), c, top);
      }
    } else if (c == 0) {
      p[q * kWarps + (threadIdx.x >> 5)] = x;
      if (q == 0) p[2 * kWarps + (threadIdx.x >> 5)] = top;
    }
  }
  // Between what is told and heard.
  static __device__ __forceinline__ void barrier() {
    if (CLUSTER) cluster_barrier();
    else __syncthreads();
  }
  // x at `p` of the cluster's block c.
  static __device__ __forceinline__ void to_block(void* p, int c, float x) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(there)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(c));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(x) : "memory");
  }
  // The team's top and sums with it; what takes a warp of top `mine` there.
  // Exponents between tops are roundings apart from those of Base, no more.
  template <int Q> __device__ __forceinline__ float hear(float (&v)[Q], float& top, float mine, float k) {
    constexpr int G = 32 / Q;
    const int l = threadIdx.x & 31, q = l / G, c = l % G;
    const float* p = part + 4 * kWarps * turn;
    turn ^= 1;
    float there = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWarps; i += G)
      if (c + i < all) there = max_nan(there, p[2 * kWarps + c + i]);
    top = warp_max(there);
    const float low = top == -INFINITY ? 0.f : top;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; i += G)
      if (c + i < all) x += p[q * kWarps + c + i] * between(p[2 * kWarps + c + i], low, k);
#pragma unroll
    for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
#pragma unroll
    for (int i = 0; i < Q; ++i) v[i] = Q == 1 ? x : __shfl_sync(0xffffffffu, x, i * G);
    return between(mine, low, k);
  }
  // What takes exponentials of Base(a) to those of Base(b); where one of the two
  // takes its top off and the other does not, from the one's base to the other's.
  static __device__ __forceinline__ float between(float a, float b, float k) {
    const Base p(a, k), q(b, k);
    if (a == -INFINITY) return 0.f;
    if (q.near()) return ex2(p.near() ? p.base - q.base : fmaf(a, k, -q.base));
    return ex2(p.near() ? -fmaf(b, k, -p.base) : (a - b) * k);
  }
  template <int Q> __device__ __forceinline__ void sum(float (&v)[Q]) {
    static_assert(Q == 1 || Q == 2 || Q == 4, "a power of two");
    constexpr int G = 32 / Q;  // lanes that end with the same one
    const int l = threadIdx.x & 31, q = l / G, c = l % G;
    float x;
    if (Q == 4) {
      const bool hi = l & 16, odd = l & 8;
      float a = hi ? v[Q - 2] : v[0], b = hi ? v[Q - 1] : v[Q / 4];
      const float sa = hi ? v[0] : v[Q - 2], sb = hi ? v[Q / 4] : v[Q - 1];
      a += __shfl_xor_sync(0xffffffffu, sa, 16);
      b += __shfl_xor_sync(0xffffffffu, sb, 16);
      x = odd ? b : a;
      x += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
    } else if (Q == 2) {
      const bool hi = l & 16;
      x = hi ? v[Q - 1] : v[0];
      x += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[Q - 1], 16);
    } else {
      x = v[0];
    }
#pragma unroll
    for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    float* p = part + 4 * kWarps * turn + q * kWarps;
    turn ^= 1;
    if (CLUSTER) {
      if (c < (int)cluster_blocks()) to_block(p + (lane >> 5), c, x);
      cluster_barrier();
    } else {
      if (c == 0) p[threadIdx.x >> 5] = x;
      __syncthreads();
    }
    x = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; i += G)
      if (c + i < all) x += p[c + i];
#pragma unroll
    for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
#pragma unroll
    for (int k = 0; k < Q; ++k) v[k] = Q == 1 ? x : __shfl_sync(0xffffffffu, x, k * G);
  }
};

// Rows that no block holds, at any address.  The 16-byte vectors between a row's
// first and last boundary go through shared memory as a Feed's do, kDepth copies
// a thread ahead, and without a break from the first reading of a row to the
// second (out of L2) and on to the next row; the elements before and behind,
// fewer than a vector, belong to one thread each.  Rows that do not count are
// passed over: who reads does not ask for theirs.
// U: vectors of a copy
template <typename T, typename Rows, int U_ = 4>
struct Stream {
  static constexpr int V = kWide<T>, U = U_, kDepth = U >= 4 ? 3 : 4;
  static constexpr size_t bytes(int threads) { return (size_t)kDepth * U * threads * 16; }
  const T* L;
  int64_t n, N, stride, row_step;
  int K, passes;
  Rows rows;
  // the copy to be asked for next
  const T* body;
  int nv, at, pass;
  uint32_t slot_in, slot_out;
  char* slot;
  int lane, size, threads;  // of those that share a row; of a block

  // Elements of a row before its first vector.
  static __device__ __forceinline__ int head_of(const T* p, int K) {
    const int h = (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T);
    return h < K ? h : K;
  }
  // To the next row that counts.
  __device__ __forceinline__ void row() {
    for (; n < N && !rows(n); n += stride) L += row_step;
    const int h = head_of(L, K);
    body = L + h;
    nv = (K - h) / V;
  }
  __device__ __forceinline__ void start(char* smem, const T* L_, int64_t n_, int64_t stride_, int64_t N_, int K_, int passes_,
                                        int lane_, int size_, int threads_, Rows rows_) {
    L = L_ + n_ * K_, n = n_, N = N_, stride = stride_, row_step = stride_ * K_, K = K_, passes = passes_;
    lane = lane_, size = size_, threads = threads_, rows = rows_;
    at = lane, pass = 0, slot_in = slot_out = 0;
    slot = smem + threadIdx.x * 16;
    row();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) ask();
  }
  __device__ __forceinline__ void ask() {
    if (n < N) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at + u * size < nv)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(
                           slot + (size_t)(slot_in * U + u) * threads * 16)),
                       "l"(body + (int64_t)(at + u * size) * V)
                       : "memory");
      at += U * size;
      if (at - lane >= nv) {
        at = lane;
        if (++pass == passes) {
          pass = 0;
          n += stride;
          L += row_step;
          row();
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    slot_in = slot_in == kDepth - 1 ? 0 : slot_in + 1;
  }
  __device__ __forceinline__ void next(Row<T, V, U>& x) {
    ask();
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
#pragma unroll
    for (int u = 0; u < U; ++u)
      x.r[u] = *reinterpret_cast<const Vec<T, V>*>(slot + (size_t)(slot_out * U + u) * threads * 16);
    slot_out = slot_out == kDepth - 1 ? 0 : slot_out + 1;
  }
};

// Blocks of `kernel` that the device holds at once, so that a grid of persistent
// blocks is one wave: `cache` (static, one for each kernel) keeps the answer for
// each number of warps (the devices of a process are alike).
struct ResidentCache {
  std::atomic<int> per_sm[33];
};
template <typename K>
inline int64_t resident(K kernel, int threads, size_t smem, ResidentCache& cache) {
  std::atomic<int>& c = cache.per_sm[threads / 32];
  int n = c.load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, (const void*)kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
    c.store(n, std::memory_order_relaxed);
  }
  return (int64_t)n * kSms;
}

// The kernel that joins the blocks' sums is launched while they still run: they
// say when it may be (at their end), it waits for all they have written.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
inline void launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = threads;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, kernel, args...);
}

// Launches `kernel` as clusters of `cluster` blocks (1: without any).
template <typename... P, typename... A>
inline void launch_clusters(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                            cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = threads;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace gate
}  // namespace gmm
