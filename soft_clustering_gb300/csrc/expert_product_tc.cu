// expert_product_tc.cu - the experts' products on the tensor cores (16-bit
// types, rows of a multiple of 16 bytes at 16-byte aligned addresses).
//
// All three are C[i][j] = sum_l P[i][l] Q[j][l] per component k, P the
// 128-row operand of tcgen05.mma and Q the operand of up to 256 columns:
//
//   product     i = output feature, j = row, l = input feature: P = W_k, Q = A
//   product_dx  i = input feature,  j = row, l = output feature: P = W_k^T, Q = dY
//   product_dw  i = output feature, j = input feature, l = row:  P = dY^T, Q = A^T
//
// With the rows as the columns of the product a component's last tile takes
// as many columns as it has rows (to the next 16): ragged components cost
// their own rows, not whole tiles.  Operands whose l is contiguous in memory
// are staged K-major, the others (W_k^T, dY^T, A^T) MN-major; either way a
// stage is boxes of 64 x 64 elements in 128-byte swizzled rows, fetched by
// TMA, so no operand is ever transposed by a copy.  Boxes that run past a
// component's rows fetch its neighbour's: as columns they are not stored, as
// terms of a sum (product_dw) they are zeroed in shared memory first, in both
// operands, so no infinity or NaN passes from one component to another.
//
// A persistent block per multiprocessor: two warps fetch (192 KB of stages in
// flight), one issues the products into one of two 256-column accumulators,
// eight read the other one back and store it, and for product_dw one zeroes
// the rows of the next component ahead of the products.  Sums are fp32 in
// tensor memory, rounded once.
//
// Where the output features fill tiles of 256, two blocks work as a pair
// (cta_group::2): each fetches half of the columns, so a stage is 32 KB in
// place of 48 for the same products.  65536 rows through 32 experts of 2048 x
// 2048 in bf16: 297 us (1.85 PFLOP/s, 95 % of the measured burst rate; 355 us
// with single blocks, bound by shared memory, which has to take 192 bytes a
// cycle).  Runs that last are bound by the power limit (about 350 us).
// What the rest is bound by: 1000001 rows through 256 experts of 128 x 128 in
// f16, HBM traffic (87 us a call, 6.0 TB/s); dX of 16385 rows x 64 experts of
// 1024 x 2048, the weights' traffic (70 us a call, 54 at the measured copy
// rate); dW of them (88 us, 54) the stages' latency, four or five a tile before
// it is stored, and at a component's end the hand-over of mended rows.
#include <cuda.h>

#include <type_traits>

#include "expert_product.cuh"
#include "tc_ptx.cuh"

namespace gmm {
namespace {

constexpr int kBox = 8192;                 // 64 rows x 128 bytes
constexpr int kTileM = 128, kTileN = 256, kTileK = 64;   // kTileM: of one block
constexpr int kRing = 192 * 1024;          // stages: 4 of 48 KB, or 6 of 32 KB in a pair
template <int CG> constexpr int kStageBytes = (kTileM + kTileN / CG) * kTileK * 2;
template <int CG> constexpr int kStages = kRing / kStageBytes<CG>;
constexpr int kBackWarps = 8;              // two for each quarter of the accumulator's lanes
constexpr int kThreads = 64 + 32 * kBackWarps + 64;  // fetch P, issue, read back, mend, fetch Q
constexpr int kMendWarp = 2 + kBackWarps;  // dw: zeroes rows of the next component
constexpr int kFetchQWarp = kMendWarp + 1;
constexpr int kOutBytes = 4096;            // what a read-back warp has on its way out
constexpr int kOutPitch = 80;              // bytes of a staged row of 32 outputs: no bank conflicts
constexpr int kOutAt = kRing;
constexpr int kBarsAt = kOutAt + kBackWarps * kOutBytes;
constexpr int kRowOut = 32 * kOutPitch;    // product, dx: the staged rows of a warp
constexpr int kFirstAt = kOutAt + kBackWarps * kRowOut;  // ... and behind them, each component's first tile
constexpr int kMostCounted = 1000;         // components (more than these fit)
static_assert(kFirstAt + 4 * (kMostCounted + 2) <= kBarsAt, "first tiles");
constexpr int kSmem = kBarsAt + 256 + 1024;
constexpr uint32_t kWait = 2000000;        // polls of up to a microsecond
constexpr uint64_t kWaitNs = 2000000000;   // of a pair

enum { kProduct = 0, kDx = 1, kDw = 2 };

struct TcArgs {
  const int64_t* offsets;
  const int32_t* count;  // the list of row tiles; NULL: every block counts
  const int4* tiles;     // the components' tiles itself
  DeviceStatus* st;
  int64_t R;
  int K, d_from, d_to;  // rows' width and the output's (dw: d_in, d_out)
};

// One tile: `n` columns, the contraction's `len` terms.
struct Tile {
  int k, i0, j0, n, len;
  int64_t row0;
};

// The tiles of one block (or pair), every `step`-th from `first`: row tiles
// (dw: components, or stretches of their rows) k, feature tiles i, and for dw column tiles j, the last
// one running fastest.  What of a tile comes from memory is fetched a tile
// ahead, and no division is done per tile: every role walks for itself, and
// the time between a tile's last product and the next one's first is idle.
template <int MODE, int CG>
struct Walk {
  const uint32_t* before;  // product, dx: tiles before each component (shared memory)
  int mt, nt, limit, k, i, j, dk, di, dj, g;
  int4 q;
  int64_t b, e;
  __device__ __forceinline__ Walk(const TcArgs& a, const uint32_t* first_tiles, int first, int step)
      : before(first_tiles) {
    mt = (a.d_to + CG * kTileM - 1) / (CG * kTileM);
    nt = MODE == kDw ? (a.d_from + kTileN - 1) / kTileN : 1;
    limit = a.tiles ? *a.count : MODE == kDw ? a.K : (int)before[a.K + 1];
    j = first % nt;
    i = first / nt % mt;
    k = first / nt / mt;
    dj = step % nt;
    di = step / nt % mt;
    dk = step / nt / mt;
    g = 0;
    q = make_int4(-1, 0, 0, 0);
    b = e = 0;
    fetch(a);
  }
  __device__ __forceinline__ void fetch(const TcArgs& a) {
    if (k >= limit) return;
    if (a.tiles) {
      q = a.tiles[k];
    } else if (MODE == kDw) {
      b = a.offsets[k];
      e = a.offsets[k + 1];
    } else {
      g = component_of((uint32_t)k, g, a.K);
      b = a.offsets[g];
      e = g < a.K ? a.offsets[g + 1] : a.R;
    }
  }
  // The component of row tile t, not before g: a few steps on, or a search.
  __device__ __forceinline__ int component_of(uint32_t t, int g, int K) const {
#pragma unroll
    for (int x = 0; x < 3; ++x, ++g)
      if (before[g + 1] > t) return g;
    int hi = K;  // before[K + 1] > t
    while (g < hi) {
      const int mid = (g + hi) >> 1;
      if (before[mid + 1] > t) hi = mid;
      else g = mid + 1;
    }
    return g;
  }
  __device__ __forceinline__ bool more() const { return k < limit; }
  __device__ __forceinline__ Tile take(const TcArgs& a) {
    Tile w;
    w.i0 = i * CG * kTileM;
    if (MODE == kDw) {
      w.k = k;
      w.j0 = j * kTileN;
      w.n = min(kTileN, a.d_from - w.j0);
      if (a.tiles) {  // a stretch of a component's rows
        w.row0 = q.y;
        w.len = q.x < 0 ? 0 : q.z;
      } else {
        const int64_t lo = clamp_row(b, a.R), hi = clamp_row(e, a.R);
        w.row0 = lo;
        w.len = hi > lo ? (int)(hi - lo) : 0;
      }
    } else {
      w.j0 = 0;
      if (a.tiles) {
        w.k = q.x;
        w.row0 = q.y;
        w.n = q.z;
      } else {
        w.k = g < a.K ? g : -1;
        w.row0 = clamp_row(b, a.R) + (int64_t)(k - (int)before[g]) * kTileN;
        w.n = (int)min((int64_t)kTileN, clamp_row(e, a.R) - w.row0);
      }
      w.len = w.k < 0 ? 0 : a.d_from;
    }
    if (MODE == kDw) {
      j += dj;
      if (j >= nt) { j -= nt; ++i; }
    }
    i += di;
    if (i >= mt) { i -= mt; ++k; }
    k += dk;
    fetch(a);
    return w;
  }
};

// before[g]: row tiles of the components before g (g = K: the rows past them),
// before[K + 1]: all of them.  By the whole block.
__device__ __forceinline__ void count_tiles(const TcArgs& a, uint32_t* before) {
  __shared__ uint32_t warp_sums[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.K + 1, per = (G + kThreads - 1) / kThreads;
  const int k0 = min(G, (int)threadIdx.x * per), k1 = min(G, k0 + per);
  uint32_t mine = 0;
  for (int k = k0; k < k1; ++k) {
    const int64_t b = clamp_row(a.offsets[k], a.R), e = k < a.K ? clamp_row(a.offsets[k + 1], a.R) : a.R;
    const uint32_t n = e > b ? (uint32_t)((e - b + kTileN - 1) / kTileN) : 0u;
    before[k] = n;
    mine += n;
  }
  uint32_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  uint32_t at = sum - mine;
  for (int w = 0; w < warp; ++w) at += warp_sums[w];
  for (int k = k0; k < k1; ++k) {
    const uint32_t n = before[k];
    before[k] = at;
    at += n;
  }
  if (k1 == G && k0 < k1) before[G] = at;
}

// TMA of one box.  `bar`: a shared::cluster address; with PAIR it may be the
// other block's of the pair.
template <bool PAIR>
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(tc::smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(tc::smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                       uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// One lane of a converged warp.  (Copies and products take their operands
// from uniform registers; behind a test of the lane number each of them costs
// 130 to 170 cycles to issue, more than a product of 128 x 256 x 16 takes.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---- pairs of blocks (cta_group::2)

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of this block's `p` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrival at a barrier of either block that passes on an accumulator read
// back.  (Not a release to the cluster, which waits about 1000 cycles for the
// thread's earlier stores to global memory: no write is handed over here.
// tcgen05.wait::ld has the values in registers before the arrival, so nothing
// of the accumulator is still to be read when the next products go there.)
__device__ __forceinline__ void arrive_read(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrival at a barrier of either block that passes on writes to this block's
// shared memory: the products that read them are issued by the other block, so
// the arrival is a release to the cluster (without a scope it would be one to
// this block alone), and wait_pair acquires there.  It takes about half a
// microsecond a ragged end: 82 us of the kernel's time for dW of 16385 rows x
// 64 experts of 1024 x 2048, where single blocks take as long and lose more
// elsewhere (65536 rows x 32 experts of 2048 x 2048: 325 us, single 366).
__device__ __forceinline__ void arrive_written(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits for the phase with this parity, acquiring what either block of the
// pair released; gives up after kWaitNs.
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity) {
  uint64_t end = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_addr(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 15) == 15) {
      uint64_t now;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      if (end == 0) end = now + kWaitNs;
      else if (now > end) return false;
    }
  }
}
template <int CG>
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity) {
  return CG == 2 ? wait_pair(bar, parity) : tc::mbar_wait(bar, parity, kWait);
}
template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t* dst) {
  if (CG == 1) {
    tc::tmem_alloc(dst, 512);
    tc::tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_addr(dst)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_give(uint32_t at) {
  if (CG == 1) tc::tmem_dealloc(at, 512);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(512u) : "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t p, uint64_t q, uint32_t id, uint32_t add) {
  if (CG == 1) {
    tc::mma_f16(d, p, q, id, add);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(p), "l"(q), "r"(id), "r"(add)
        : "memory");
  }
}
// Arrives on `bar` (in a pair: of both blocks) when the products issued so
// far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CG == 1) {
    tc::mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            tc::smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
  }
}

// Descriptor of an MN-major operand in 128-byte swizzled boxes of 64 (MN) x
// 64 (K): the next 64 along MN is a box (8192 bytes) away (leading byte
// offset), the next 8 along K 1024 bytes (stride byte offset).
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(kBox >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Instruction descriptor: fp32 accumulator, both operands f16 or bf16, P / Q
// MN-major where told (bits 15, 16).
__device__ __forceinline__ uint32_t idesc(bool bf16, bool p_mn, bool q_mn, int m, int n) {
  const uint32_t f = bf16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)p_mn << 15) | ((uint32_t)q_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <typename TO> struct Pair;
template <> struct Pair<__half> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __halves2half2(__float2half_rn(a), __float2half_rn(b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// Accumulator lanes `lanes` .. + 15 of 32 columns: register 4 c + 2 u + v is
// lane 8 u + t / 4, column 8 c + 2 (t % 4) + v of thread t.
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// 32 features x 32 columns of the accumulator (from `src`) as 32 rows of 32
// outputs: transposed on their way into the warp's piece of shared memory (8 x
// 8 at a time), then 64 bytes a row to memory.  `left` rows and `feats`
// features of them are wanted (feats a multiple of 8).
template <typename TO>
__device__ __forceinline__ void store_rows(uint32_t src, bool some, uint8_t* piece, TO* out, int64_t ld,
                                           int left, int feats) {
  const int lane = threadIdx.x & 31;
  if (some) {
    uint32_t r[2][16];
    tmem_ld16x32(src, r[0]);
    tmem_ld16x32(src + (16u << 16), r[1]);
    tmem_wait16(r[0]);
    tmem_wait16(r[1]);
    uint32_t at = tc::smem_addr(piece) + (lane & 7) * kOutPitch + (lane >> 3) * 16;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t h[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        h[x] = Pair<TO>::pack(__uint_as_float(r[x >> 1][4 * c + 2 * (x & 1)]),
                              __uint_as_float(r[x >> 1][4 * c + 2 * (x & 1) + 1]));
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                       at + c * 8 * kOutPitch),
                   "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                   : "memory");
    }
    __syncwarp();
  }
  const int row = lane >> 2, chunk = lane & 3;
  TO* p = out + row * ld + chunk * 8;
  const bool mine = chunk * 8 < feats;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (some) v = *reinterpret_cast<const uint4*>(piece + (8 * x + row) * kOutPitch + chunk * 16);
    if (mine && 8 * x + row < left) *reinterpret_cast<uint4*>(p + 8 * x * ld) = v;
  }
  __syncwarp();
}

// 128 bytes of this lane's row of dW (64 or 32 columns) into the warp's piece
// in shared memory, 128-byte swizzled as the store's tensor map has it: eight
// lanes fill all eight 16-byte places of a line.
__device__ __forceinline__ void stage_line(const uint32_t* w, uint8_t* piece) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(piece + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y,
                                             int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::
                   "l"(map),
               "r"(x), "r"(y), "r"(z), "r"(tc::smem_addr(src))
               : "memory");
}

// Rows left .. left + rows - 1 of `boxes` boxes from p: zeros (128 bytes each).
__device__ __forceinline__ void zero_rows(uint8_t* p, int boxes, int left, int rows) {
  const int lane = threadIdx.x & 31;
  for (int box = 0; box < boxes; ++box)
    for (int r = lane >> 3; r < rows; r += 4)
      *reinterpret_cast<uint4*>(p + box * kBox + (left + r) * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  __syncwarp();
}

// CG = 2: a pair of blocks (a cluster, on two multiprocessors) on tiles of 256
// rows; each block holds 128 of them, fetches half of the columns, and reads
// its 128 rows of the accumulator back.  The first block issues the products;
// the fetched bytes of both are counted on its barriers.
template <int MODE, typename T, typename TO, int CG>
__global__ void __launch_bounds__(kThreads, 1)
expert_tc_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                 const __grid_constant__ CUtensorMap map_out, TO* __restrict__ out, TcArgs a) {
  extern __shared__ uint8_t raw[];
  constexpr int S = kStages<CG>, B = kStageBytes<CG>;
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarsAt);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;         // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2]
  uint64_t* odd_full = acc_empty + 2;     // [S] there, but with rows to be zeroed first
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(odd_full + S);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kPmn = MODE != kProduct, kQmn = MODE == kDw;
  uint32_t* before = reinterpret_cast<uint32_t*>(smem + kFirstAt);
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int first = blockIdx.x / CG, step = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&full[i], CG);  // the fetching warp, or both blocks' mending warps
      tc::mbar_init(&empty[i], 1);
      tc::mbar_init(&odd_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&acc_full[i], 1);
      tc::mbar_init(&acc_empty[i], kBackWarps * CG);
    }
    tc::mbar_fence_init();
  }
  if (warp == 1) tmem_take<CG>(tmem_at);
  if (a.tiles) {
    // the list and everything before it is there
    asm volatile("griddepcontrol.wait;" ::: "memory");
  } else if (MODE != kDw) {
    count_tiles(a, before);
  }
  tc::tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (CG == 2) cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_at;
  if (warp == 0 || warp == kFetchQWarp) {
    // P by one warp, which also counts on the barrier what is to come, Q by
    // the other: a copy takes about 100 cycles to issue, and one warp's four
    // to six a stage were what short contractions waited for
    const bool fetch_p = warp == 0;
    uint32_t it = 0;
    uint32_t odd_fills = 0, last_odd = 0;  // a bit a stage: an odd number of odd fills; the last one is odd
    bool ok = true;
    for (Walk<MODE, CG> walk(a, before, first, step); ok && walk.more();) {
      const Tile w = walk.take(a);
      // this block's columns
      const int cols = CG == 2 ? ((w.n + 31) & ~31) / 2 : w.n;
      const int boxes = (cols + 63) / 64, at = (int)rank * cols;
      const int i0 = w.i0 + (int)rank * kTileM;
      for (int l = 0; l < w.len; l += kTileK, ++it) {
        const int s = it % S;
        if (it >= S && !wait_on<CG>(&empty[s], ((it / S) - 1) & 1)) {
          // the wait took far longer than the copies in flight can
          if (lane == 0) raise_status(a.st, GMM_ERR_TIMEOUT);
          ok = false;
          break;
        }
        // the end of a component, with rows of the next one up to the next
        // 16: to the mending warp first
        const bool odd = MODE == kDw && w.len - l < kTileK && (w.len - l) % 16 != 0;
        if (MODE == kDw) {
          last_odd = (last_odd & ~(1u << s)) | ((uint32_t)odd << s);
          odd_fills ^= (uint32_t)odd << s;
        }
        if (elect_one()) {
          uint8_t* p = smem + s * B;
          uint8_t* q = p + kTileM * kTileK * 2;
          const uint32_t bytes = (2 + boxes) * kBox;
          const uint32_t bar = odd                    ? tc::smem_addr(&odd_full[s])
                               : CG == 2 && rank != 0 ? in_block(&full[s], 0)
                                                      : tc::smem_addr(&full[s]);
          constexpr bool PAIR = CG == 2;
          if (fetch_p) {
            if (odd) {
              tc::mbar_arrive_expect_tx(&odd_full[s], bytes);
            } else if (rank == 0) {
              tc::mbar_arrive_expect_tx(&full[s], CG * bytes);
              if (CG == 2) tc::mbar_arrive(&full[s]);
            }
            if (MODE == kProduct) {
              tma_3d<PAIR>(p, &map_p, l, i0, w.k, bar);
              tma_3d<PAIR>(p + kBox, &map_p, l, i0 + 64, w.k, bar);
            } else if (MODE == kDx) {
              tma_3d<PAIR>(p, &map_p, i0, l, w.k, bar);
              tma_3d<PAIR>(p + kBox, &map_p, i0 + 64, l, w.k, bar);
            } else {
              tma_2d<PAIR>(p, &map_p, i0, (int)w.row0 + l, bar);
              tma_2d<PAIR>(p + kBox, &map_p, i0 + 64, (int)w.row0 + l, bar);
            }
          } else {
            for (int b = 0; b < boxes; ++b) {
              if (MODE == kDw) tma_2d<PAIR>(q + b * kBox, &map_q, w.j0 + at + 64 * b, (int)w.row0 + l, bar);
              else tma_2d<PAIR>(q + b * kBox, &map_q, l, (int)w.row0 + at + 64 * b, bar);
            }
          }
        }
        __syncwarp();
      }
    }
    // No copy is in flight when the blocks end, also where a wait gave up: the
    // last copies to each stage, of both warps, are on the barrier of its fill
    // (a pair's on the first block's, and neither block leaves before the other).
    if (fetch_p)
      for (uint32_t s = 0; s < S && s < it; ++s) {
        const bool odd = (last_odd >> s) & 1;
        if (!odd && rank != 0) continue;
        const uint32_t fill = (it - 1 - s) / S;  // of this stage
        if (!wait_on<CG>(odd ? &odd_full[s] : &full[s], odd ? ((odd_fills >> s) & 1) ^ 1 : fill & 1)) {
          if (lane == 0) raise_status(a.st, GMM_ERR_TIMEOUT);
          break;
        }
      }
  } else if (warp == 1 && rank == 0) {
    uint32_t it = 0, acc = 0;
    bool ok = true;
    for (Walk<MODE, CG> walk(a, before, first, step); ok && walk.more();) {
      const Tile w = walk.take(a);
      if (w.len == 0) continue;
      const int b = acc & 1;
      if (acc >= 2 && !wait_on<CG>(&acc_empty[b], ((acc >> 1) - 1) & 1)) ok = false;
      const uint32_t d = tmem + b * kTileN;
      const int n = CG == 2 ? (w.n + 31) & ~31 : (w.n + 15) & ~15;
      const uint32_t id = idesc(std::is_same<T, __nv_bfloat16>::value, kPmn, kQmn, CG * kTileM, n);
      for (int l = 0; ok && l < w.len; l += kTileK, ++it) {
        const int s = it % S;
        if (!wait_on<CG>(&full[s], (it / S) & 1)) {
          ok = false;
          break;
        }
        uint8_t* p = smem + s * B;
        const int left = min(kTileK, w.len - l);
        const int steps = (left + 15) / 16;
        __syncwarp();
        tc::tc_fence_after();
        const uint32_t ps = tc::smem_addr(p), qs = ps + kTileM * kTileK * 2;
        const uint64_t dp = kPmn ? sdesc_mn128(ps) : tc::sdesc_k128(ps);
        const uint64_t dq = kQmn ? sdesc_mn128(qs) : tc::sdesc_k128(qs);
        // a descriptor's address counts 16 bytes: 16 terms on
        constexpr int kP = (kPmn ? 2048 : 32) / 16, kQ = (kQmn ? 2048 : 32) / 16;
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < kTileK / 16; ++x)
            if (x < steps) mma<CG>(d, dp + x * kP, dq + x * kQ, id, (l > 0 || x > 0) ? 1u : 0u);
          commit<CG>(&empty[s]);
          if (l + kTileK >= w.len) commit<CG>(&acc_full[b]);
        }
        __syncwarp();
      }
      ++acc;
    }
    if (!ok) {
      if (lane == 0) raise_status(a.st, GMM_ERR_TIMEOUT);
      // the products issued so far end before their memory is given back
      if (it > 0) wait_on<CG>(&empty[(it - 1) % S], ((it - 1) / S) & 1);
    }
  } else if (warp == kMendWarp) {
    // ahead of the products: zeroes this block's rows of the next component
    // in a component's last stage and passes the stage on
    if (MODE == kDw) {
      uint32_t it = 0, phases = 0;  // a bit for each stage's barrier
      for (Walk<MODE, CG> walk(a, before, first, step); walk.more();) {
        const Tile w = walk.take(a);
        const int blocks = (w.len + kTileK - 1) / kTileK;
        it += blocks;
        const int left = w.len - (blocks - 1) * kTileK;
        if (blocks == 0 || left % 16 == 0) continue;
        const int s = (it - 1) % S;
        if (!wait_on<CG>(&odd_full[s], (phases >> s) & 1)) {
          if (lane == 0) raise_status(a.st, GMM_ERR_TIMEOUT);
          break;
        }
        phases ^= 1u << s;
        const int cols = CG == 2 ? ((w.n + 31) & ~31) / 2 : w.n;
        zero_rows(smem + s * B, 2 + (cols + 63) / 64, left, (left + 15) / 16 * 16 - left);
        if (lane == 0) {
          if (CG == 2) arrive_written(in_block(&full[s], 0));
          else tc::mbar_arrive(&full[s]);
        }
        __syncwarp();
      }
    }
  } else if (warp >= 2) {
    const int quarter = warp & 3;       // the TMEM lanes this warp may read
    const int half = (warp - 2) >> 2;   // every other stretch of columns
    uint8_t* piece = smem + kOutAt + (warp - 2) * (MODE == kDw ? kOutBytes : kRowOut);
    uint32_t acc = 0;
    for (Walk<MODE, CG> walk(a, before, first, step); walk.more();) {
      const Tile w = walk.take(a);
      const int b = acc & 1;
      const int i0 = w.i0 + (int)rank * kTileM + quarter * 32;
      if (w.len > 0) {
        if (!wait_on<CG>(&acc_full[b], (acc >> 1) & 1)) {
          if (lane == 0) raise_status(a.st, GMM_ERR_TIMEOUT);
          break;
        }
        tc::tc_fence_after();
      }
      const uint32_t src = tmem + b * kTileN + ((uint32_t)(quarter * 32) << 16);
      if constexpr (MODE == kDw) {
        // 32 rows x 128 bytes at a time; the tensor map cuts off what is past
        // dW's edges
        constexpr int W = 128 / sizeof(TO);
        for (int c = half * W; c < w.n && i0 < a.d_to; c += 2 * W) {
          uint32_t r[2][32];
          if (w.len > 0) {
            tc::tmem_ld32_issue(src + c, r[0]);
            if (W == 64) tc::tmem_ld32_issue(src + c + 32, r[1]);
            tc::tmem_wait32(r[0]);
            if (W == 64) tc::tmem_wait32(r[1]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[0][j] = r[1][j] = 0u;
          }
          if constexpr (W == 64) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              r[0][j] = Pair<TO>::pack(__uint_as_float(r[0][2 * j]), __uint_as_float(r[0][2 * j + 1]));
#pragma unroll
            for (int j = 0; j < 16; ++j)
              r[0][16 + j] = Pair<TO>::pack(__uint_as_float(r[1][2 * j]), __uint_as_float(r[1][2 * j + 1]));
          }
          if (lane == 0)  // the last store has read the piece
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
          stage_line(r[0], piece);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&map_out, piece, w.j0 + c, i0, w.k);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      } else if (i0 < a.d_to) {
        for (int c = half * 32; c < w.n; c += 64)
          store_rows(src + c, w.len > 0, piece, out + (w.row0 + c) * (int64_t)a.d_to + i0, a.d_to,
                     w.n - c, a.d_to - i0);
      }
      if (w.len > 0) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) arrive_read(in_block(&acc_empty[b], 0));
          else tc::mbar_arrive(&acc_empty[b]);
        }
        ++acc;
      }
    }
    if (MODE == kDw && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  __syncwarp();
  if (CG == 2) cluster_sync();  // neither block leaves while the other may reach it
  if (warp == 1) {
    tc::tc_fence_after();
    tmem_give<CG>(tmem);
  }
}

// dW[k] = the sum of its stretches' partial sums, in order.
template <typename TO>
__global__ void __launch_bounds__(256)
join_kernel(const float* __restrict__ part, const uint32_t* __restrict__ first, int64_t quads,
            TO* __restrict__ dW) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  const int k = blockIdx.y;
  const uint32_t s0 = first[k], s1 = first[k + 1];
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* p = reinterpret_cast<const float4*>(part) + i;
#pragma unroll 8
  for (uint32_t s = s0; s < s1; ++s) {
    const float4 v = p[(int64_t)s * quads];
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  TO* o = dW + ((int64_t)k * quads + i) * 4;
  if constexpr (sizeof(TO) == 4)
    *reinterpret_cast<float4*>(o) = sum;
  else
    *reinterpret_cast<uint2*>(o) = make_uint2(Pair<TO>::pack(sum.x, sum.y), Pair<TO>::pack(sum.z, sum.w));
}

template <typename TO>
gmm_status join(const void* ws, const ProductLayout& L, int K, int d_in, int d_out, void* dW,
                cudaStream_t s) {
  const int64_t quads = (int64_t)d_in * d_out / 4;
  ProfScope p("join_kernel", s);
  join_kernel<TO><<<dim3((unsigned)((quads + 255) / 256), K), 256, 0, s>>>(
      at<float>(ws, L.off_part), at<uint32_t>(ws, L.off_first), quads, (TO*)dW);
  return launched();
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// Dense [d2][d1][d0] (d2 = 0: two dimensions), boxes of rows x 128 bytes.
bool encode(CUtensorMap* m, int type, const void* base, int64_t d0, int64_t d1, int64_t d2, int rows) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t es = (cuuint64_t)dtype_size(type);
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  const cuuint64_t strides[2] = {(cuuint64_t)d0 * es, (cuuint64_t)d0 * (cuuint64_t)d1 * es};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
  const CUtensorMapDataType dt = type == GMM_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : type == GMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  return fn(m, dt, d2 ? 3 : 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Of the current device; 0 where that cannot be told.
int multiprocessors() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int MODE, typename T, typename TO, int CG>
gmm_status go_as(const CUtensorMap& mp, const CUtensorMap& mq, const CUtensorMap& mo, void* out,
                 const TcArgs& a, int64_t most, cudaStream_t s) {
  const int sms = multiprocessors();
  static std::atomic<uint64_t> allowed;
  if (sms < CG || !allow_smem((const void*)expert_tc_kernel<MODE, T, TO, CG>, kSmem, allowed))
    return GMM_ERR_CUDA;
  const int64_t tiles = most * ((a.d_to + CG * kTileM - 1) / (CG * kTileM));
  const unsigned grid = (unsigned)(tiles < sms / CG ? tiles : sms / CG) * CG;
  ProfScope p(MODE == kProduct ? "expert_tc_kernel" : MODE == kDx ? "expert_tc_kernel(dx)" : "expert_tc_kernel(dw)", s);
  // may start while the kernel that makes its list runs
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = a.tiles != nullptr;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, expert_tc_kernel<MODE, T, TO, CG>, mp, mq, mo, (TO*)out, a);
  return launched();
}

// Pairs where the 256 rows of a tile are all there, or nearly so: what is
// missing costs as much as it would hold, and pairs win 16 % (above).
bool pairs(int d_to) {
  const int t = (d_to + 255) / 256 * 256;
  return (t - d_to) * 8 <= t;
}

// most: row tiles at most (dw: components x column tiles).
template <int MODE, typename T, typename TO>
gmm_status go(const CUtensorMap& mp, const CUtensorMap& mq, const CUtensorMap& mo, void* out,
              const TcArgs& a, int64_t most, cudaStream_t s) {
  return pairs(a.d_to) ? go_as<MODE, T, TO, 2>(mp, mq, mo, out, a, most, s)
                       : go_as<MODE, T, TO, 1>(mp, mq, mo, out, a, most, s);
}

}  // namespace

bool tc_product_ok(int xdtype, int64_t R, int d_in, int d_out, const void* a, const void* b, const void* c) {
  return tc_widths_ok(xdtype, d_in, d_out) && R <= INT32_MAX - 256 && aligned(16, a, b, c);
}

gmm_status tc_rows(const void* A, int xdtype, const void* W, void* Y, int64_t R, int d_from,
                   int d_to, int K, bool dx, const int64_t* offsets, void* ws, cudaStream_t s) {
  const ProductLayout L = ProductLayout::make(R, d_from, d_to, K, xdtype);
  // Up to kMostCounted components every block counts their tiles itself in
  // place of a kernel that lists them: experts of 128 x 128 in bf16, 30000
  // rows, a call: 12.8 us (listed 16.3) with 600 components, 17.6 (16.7) with
  // 1000, 27.1 (23.6) with 2000.  The crossing is somewhat below 1000, where the
  // room for their first tiles ends.
  const bool listed = K > kMostCounted || R == 0;
  if (listed) {
    const gmm_status r = list_tiles(offsets, K, R, kTileN, ws, L, s);
    if (r != GMM_OK || R == 0) return r;
  }
  CUtensorMap mp, mq;
  const int d_in = dx ? d_to : d_from, d_out = dx ? d_from : d_to;
  if (!encode(&mp, xdtype, W, d_in, d_out, K, 64) || !encode(&mq, xdtype, A, d_from, R, 0, 64))
    return GMM_ERR_CUDA;
  TcArgs a{offsets, at<int32_t>(ws, L.off_count), listed ? at<int4>(ws, L.off_tiles) : nullptr,
           at<DeviceStatus>(ws, 0), R, K, d_from, d_to};
  const int64_t most = ProductLayout::most_tiles(R, K, kTileN);
  if (most * ((d_to + kTileM - 1) / kTileM) > INT32_MAX) return GMM_ERR_UNSUPPORTED;
  if (xdtype == GMM_BF16) {
    using T = __nv_bfloat16;
    return dx ? go<kDx, T, T>(mp, mq, mq, Y, a, most, s) : go<kProduct, T, T>(mp, mq, mq, Y, a, most, s);
  }
  using T = __half;
  return dx ? go<kDx, T, T>(mp, mq, mq, Y, a, most, s) : go<kProduct, T, T>(mp, mq, mq, Y, a, most, s);
}

gmm_status tc_weights(const void* dY, const void* A, int xdtype, int64_t R, int d_in, int d_out,
                      int K, const int64_t* offsets, void* dW, int wdtype, void* ws,
                      cudaStream_t s) {
  CUtensorMap mp, mq, mo;
  if (!encode(&mp, xdtype, dY, d_out, R, 0, 64) || !encode(&mq, xdtype, A, d_in, R, 0, 64))
    return GMM_ERR_CUDA;
  const int64_t nt = (d_in + kTileN - 1) / kTileN;
  TcArgs a{offsets, nullptr, nullptr, at<DeviceStatus>(ws, 0), R, K, d_in, d_out};
  const int64_t stretch = dw_stretch_rows(R, d_in, d_out, K);
  if (stretch > 0) {
    // few tiles of long sums
    const ProductLayout L = ProductLayout::make(R, d_in, d_out, K, xdtype);
    const int64_t most = ProductLayout::most_tiles(R, K, (int)stretch);
    float* part = at<float>(ws, L.off_part);
    if (!encode(&mo, GMM_F32, part, d_in, d_out, most, 32)) return GMM_ERR_CUDA;
    gmm_status r = list_tiles(offsets, K, R, (int)stretch, ws, L, s);
    if (r != GMM_OK) return r;
    a.count = at<int32_t>(ws, L.off_count);
    a.tiles = at<int4>(ws, L.off_tiles);
    r = xdtype == GMM_BF16 ? go<kDw, __nv_bfloat16, float>(mp, mq, mo, part, a, most * nt, s)
                           : go<kDw, __half, float>(mp, mq, mo, part, a, most * nt, s);
    if (r != GMM_OK) return r;
    if (wdtype == GMM_F32) return join<float>(ws, L, K, d_in, d_out, dW, s);
    if (wdtype == GMM_BF16) return join<__nv_bfloat16>(ws, L, K, d_in, d_out, dW, s);
    return join<__half>(ws, L, K, d_in, d_out, dW, s);
  }
  if (!encode(&mo, wdtype, dW, d_in, d_out, K, 32)) return GMM_ERR_CUDA;
  const int64_t most = (int64_t)K * nt;
  if (most * ((d_out + kTileM - 1) / kTileM) > INT32_MAX) return GMM_ERR_UNSUPPORTED;
  if (xdtype == GMM_BF16) {
    using T = __nv_bfloat16;
    return wdtype == GMM_F32 ? go<kDw, T, float>(mp, mq, mo, dW, a, most, s) : go<kDw, T, T>(mp, mq, mo, dW, a, most, s);
  }
  using T = __half;
  return wdtype == GMM_F32 ? go<kDw, T, float>(mp, mq, mo, dW, a, most, s) : go<kDw, T, T>(mp, mq, mo, dW, a, most, s);
}

}  // namespace gmm
