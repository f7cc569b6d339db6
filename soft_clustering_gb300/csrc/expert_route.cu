// expert_route.cu - gmm_route: the entries of a top-m table in the order of
// their components (a stable counting sort), with the way back.
//
// slot[e] = offsets[k] + #{e' < e : ids[e'] = k}, k = ids[e]; entry[slot[e]]
// = e.  Entries left out form group K: their slot is -1 and their places past
// offsets[K] hold -1 in `entry`.
//
// Up to kTinyE entries one block does it alone (latency is all that counts):
// each thread ranks one entry against all others in shared memory, and
// offsets[k] is the number of sorted keys below k.
// Above that: per block of entries a histogram, a prefix over the blocks for
// each group, and a scatter whose warps take consecutive segments of the
// block's entries.  The scatter counts its segments again (shared-memory
// atomics, the order does not matter), turns the counts into each segment's
// first place, and then walks the segments in order, __match_any_sync ranking
// the equal keys of 32 entries: fixed places, so the result never varies.
// The walk waits on latencies more than on anything else: ids are fetched
// kBatch at a time a lane, a batch ahead, and a batch's ranks are taken before
// its places, which depend on one another.
// Floor: 4 bytes read and 8 written per entry.  8000012 entries to 4096
// components: 12 + 7 + 92 us; the scatter is bound by latency (16 warps a
// multiprocessor, as many as the counts' shared memory allows) and by its
// 4-byte writes to scattered places.  4 entries: 3.6 us.
#include "expert_internal.cuh"

namespace gmm {
namespace {

constexpr int kTinyE = 1024;
constexpr int kCountThreads = 1024;
constexpr int kSlice = 24576;          // groups per shared-memory histogram pass
constexpr int kBatch = 8;              // entries a lane fetches at once
constexpr int kMaxWarps = 8;           // scatter warps per block
constexpr size_t kScatterSmem = 192 * 1024;

// Group of an id: K for entries left out.
__device__ __forceinline__ int group_of(int32_t id, int K) {
  return (id >= 0 && id < K) ? id : K;
}

__global__ void __launch_bounds__(kTinyE)
route_tiny_kernel(const int32_t* __restrict__ ids, int E, int K, int64_t* __restrict__ offsets,
                  int32_t* __restrict__ entry, int32_t* __restrict__ slot) {
  __shared__ __align__(16) int key[kTinyE];
  __shared__ int sorted[kTinyE];
  const int e = threadIdx.x;
  const int padded = (E + 3) & ~3;
  const int mine = e < E ? group_of(ids[e], K) : INT32_MAX;
  if (e < padded) key[e] = mine;
  __syncthreads();
  int rank = 0;
  for (int i = 0; i < padded; i += 4) {
    const int4 q = *reinterpret_cast<const int4*>(key + i);
    rank += (q.x < mine) || (q.x == mine && i < e);
    rank += (q.y < mine) || (q.y == mine && i + 1 < e);
    rank += (q.z < mine) || (q.z == mine && i + 2 < e);
    rank += (q.w < mine) || (q.w == mine && i + 3 < e);
  }
  if (e < E) {
    sorted[rank] = mine;
    slot[e] = mine < K ? rank : -1;
    entry[rank] = mine < K ? e : -1;
  }
  __syncthreads();
  for (int k = e; k <= K; k += blockDim.x) {  // number of keys below k
    int lo = 0, hi = E;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sorted[mid] < k) lo = mid + 1;
      else hi = mid;
    }
    offsets[k] = lo;
  }
}

// counts[b][k]: entries of group k in block b's `tile` entries.
__global__ void __launch_bounds__(kCountThreads)
route_count_kernel(const int32_t* __restrict__ ids, int64_t E, int K, int tile,
                   uint32_t* __restrict__ counts) {
  extern __shared__ uint32_t bins[];
  const int64_t b = blockIdx.x;
  const int64_t e0 = b * tile, e1 = min(E, e0 + tile);
  const int G = K + 1;
  for (int k0 = 0; k0 < G; k0 += kSlice) {
    const int ks = min(kSlice, G - k0);
    for (int i = threadIdx.x; i < ks; i += kCountThreads) bins[i] = 0u;
    __syncthreads();
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kBatch * kCountThreads) {
      int k[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        k[j] = e + j * kCountThreads < e1 ? group_of(ids[e + j * kCountThreads], K) - k0 : -1;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (k[j] >= 0 && k[j] < ks) atomicAdd(&bins[k[j]], 1u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ks; i += kCountThreads) counts[(size_t)b * G + k0 + i] = bins[i];
    __syncthreads();
  }
}

// Block: 32 groups (lanes) x 32 stretches of blocks (warps).  counts[b][k]
// becomes the entries of k in blocks before b; tot[k] the entries of k.
__global__ void __launch_bounds__(1024)
route_scan_blocks_kernel(uint32_t* __restrict__ counts, int64_t nb, int G,
                         uint32_t* __restrict__ tot) {
  __shared__ uint32_t part[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;
  const int64_t per = (nb + 31) / 32;
  const int64_t b0 = min(nb, w * per), b1 = min(nb, b0 + per);
  uint32_t sum = 0;
  if (k < G)
#pragma unroll 8
    for (int64_t b = b0; b < b1; ++b) sum += counts[(size_t)b * G + k];
  part[w][lane] = sum;
  __syncthreads();
  if (w == 0) {
    uint32_t run = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t v = part[i][lane];
      part[i][lane] = run;
      run += v;
    }
    if (k < G) tot[k] = run;
  }
  __syncthreads();
  if (k < G) {
    uint32_t run = part[w][lane];
    for (int64_t b = b0; b < b1; b += kBatch) {
      uint32_t v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) v[j] = b + j < b1 ? counts[(size_t)(b + j) * G + k] : 0u;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (b + j < b1) counts[(size_t)(b + j) * G + k] = run;
        run += v[j];
      }
    }
  }
}

// One block: offsets[k] = entries of the groups before k, k = 0 .. K.
__global__ void __launch_bounds__(1024)
route_scan_groups_kernel(const uint32_t* __restrict__ tot, int K, int64_t* __restrict__ offsets) {
  __shared__ uint32_t wsum[32];
  const int per = (K + 1 + 1023) / 1024;
  const int k0 = min(K + 1, (int)threadIdx.x * per), k1 = min(K + 1, k0 + per);
  uint32_t mine = 0;
  for (int k = k0; k < k1; ++k) mine += tot[k];
  uint32_t run = block_exclusive_1024(mine, wsum);
  for (int k = k0; k < k1; ++k) {
    offsets[k] = run;
    run += tot[k];
  }
}

// hist[w][k]: entries of group k in the segments before warp w's, then with
// the warp's running count; two counts to a word (a block holds at most 65535
// entries).  base[k]: the block's first place of group k, in shared memory
// where it fits (`base_here`); every block then adds up the groups' totals
// itself and the first one writes offsets, which elsewhere are there already.
__global__ void __launch_bounds__(kMaxWarps * 32)
route_scatter_kernel(const int32_t* __restrict__ ids, int64_t E, int K, int seg, int base_here,
                     const uint32_t* __restrict__ counts, const uint32_t* __restrict__ tot,
                     int64_t* __restrict__ offsets, int32_t* __restrict__ entry,
                     int32_t* __restrict__ slot) {
  extern __shared__ uint32_t words[];
  __shared__ uint32_t sums[kMaxWarps];
  const int G = K + 1, H = (G + 1) / 2;  // words of one warp's counts
  const int warps = blockDim.x >> 5;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t b = blockIdx.x;
  const int64_t e0 = (b * warps + w) * (int64_t)seg;
  const int64_t e1 = min(E, e0 + seg);
  const uint32_t* before = counts + (size_t)b * G;
  uint32_t* base = words + (size_t)warps * H;
  for (int i = threadIdx.x; i < warps * H; i += blockDim.x) words[i] = 0u;
  if (base_here)
    for (int k = threadIdx.x; k < G; k += blockDim.x) base[k] = tot[k];
  __syncthreads();
  if (warps > 1)
    for (int64_t e = e0 + lane; e < e1; e += kBatch * 32) {
      int k[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) k[j] = e + j * 32 < e1 ? group_of(ids[e + j * 32], K) : -1;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (k[j] >= 0) atomicAdd(&words[(size_t)w * H + (k[j] >> 1)], (k[j] & 1) ? 0x10000u : 1u);
    }
  if (base_here) {
    // prefix over the groups, each thread a stretch
    const int per = (G + blockDim.x - 1) / blockDim.x;
    const int k0 = min(G, (int)threadIdx.x * per), k1 = min(G, k0 + per);
    uint32_t mine = 0;
    for (int k = k0; k < k1; ++k) mine += base[k];
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) sums[w] = incl;
    __syncthreads();
    uint32_t run = incl - mine;
    for (int i = 0; i < w; ++i) run += sums[i];
    for (int k = k0; k < k1; ++k) {
      const uint32_t v = base[k];
      base[k] = run;
      run += v;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < G; k += blockDim.x) {
      if (b == 0) offsets[k] = base[k];
      base[k] += before[k];
    }
  }
  if (warps > 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      uint32_t run = 0;  // both halves at once: neither sum reaches 65536
      for (int x = 0; x < warps; ++x) {
        const uint32_t v = words[(size_t)x * H + i];
        words[(size_t)x * H + i] = run;
        run += v;
      }
    }
  }
  __syncthreads();
  uint16_t* mine = reinterpret_cast<uint16_t*>(words + (size_t)w * H);
  int32_t next[kBatch];  // ids as they are: what is done with them would wait for them
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (e0 + lane + j * 32 < e1) next[j] = ids[e0 + lane + j * 32];
  for (int64_t e = e0 + lane; e - lane < e1; e += kBatch * 32) {
    int k[kBatch];
    unsigned same[kBatch];
    uint32_t first[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      k[j] = e + j * 32 < e1 ? group_of(next[j], K) : -1;
      const int64_t f = e + (kBatch + j) * 32;
      if (f < e1) next[j] = ids[f];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      same[j] = __match_any_sync(0xffffffffu, k[j]);
      first[j] = 0;
      if (k[j] >= 0)
        first[j] = (base_here ? base[k[j]] : (uint32_t)offsets[k[j]] + before[k[j]]) +
                   __popc(same[j] & ((1u << lane) - 1u));
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      uint32_t at = 0;
      if (k[j] >= 0) at = mine[k[j]];
      __syncwarp();
      if (k[j] >= 0 && lane == __ffs(same[j]) - 1) mine[k[j]] = (uint16_t)(at + __popc(same[j]));
      __syncwarp();
      first[j] += at;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (k[j] >= 0) {
        slot[e + j * 32] = k[j] < K ? (int32_t)first[j] : -1;
        entry[first[j]] = k[j] < K ? (int32_t)(e + j * 32) : -1;
      }
  }
}

struct RouteLayout {
  int warps, seg, tile, base_here;
  int64_t nb;
  size_t smem, off_counts, off_tot, bytes;
  static RouteLayout make(int64_t E, int K) {
    RouteLayout L;
    const size_t per_warp = sizeof(uint32_t) * (size_t)((K + 2) / 2);
    const size_t bases = sizeof(uint32_t) * (size_t)(K + 1);
    L.warps = kMaxWarps;
    while (L.warps > 1 && per_warp * L.warps + bases > kScatterSmem) L.warps >>= 1;
    L.base_here = per_warp * L.warps + bases <= kScatterSmem;
    L.smem = per_warp * L.warps + (L.base_here ? bases : 0);
    // one wave of two blocks a multiprocessor, as far as a block's 16-bit
    // counts reach (a block's K counters are written, scanned and read once
    // more: few long blocks)
    int64_t seg = (E + (int64_t)L.warps * 304 - 1) / ((int64_t)L.warps * 304);
    const int64_t most = 65535 / L.warps / 32 * 32;
    seg = seg < 256 ? 256 : seg > most ? most : (seg + 31) / 32 * 32;
    L.seg = (int)seg;
    L.tile = L.warps * L.seg;
    L.nb = (E + L.tile - 1) / L.tile;
    size_t o = 0;
    L.off_counts = o; o = align_up(o + sizeof(uint32_t) * (size_t)(K + 1) * (size_t)L.nb);
    L.off_tot = o;    o = align_up(o + sizeof(uint32_t) * (size_t)(K + 1));
    L.bytes = o;
    return L;
  }
};

bool route_sizes_ok(int64_t N, int m, int K) {
  return N >= 0 && m >= 1 && m <= 8 && K >= 1 && K <= kMaxK && N <= INT32_MAX / m;
}

}  // namespace
}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_route_ws_bytes(int64_t N, int m, int K) {
  if (!route_sizes_ok(N, m, K)) return 0;
  return RouteLayout::make(N * m, K).bytes;
}

gmm_status gmm_route(const int32_t* ids, int64_t N, int m, int K, int64_t* offsets,
                     int32_t* entry, int32_t* slot, void* ws, size_t ws_bytes, void* stream) {
  if (!route_sizes_ok(N, m, K) || !offsets || !ws) return GMM_ERR_INVALID_ARG;
  if (N > 0 && (!ids || !entry || !slot)) return GMM_ERR_INVALID_ARG;
  if (!aligned(4, ids, entry, slot, ws) || !aligned(8, offsets)) return GMM_ERR_INVALID_ARG;
  const int64_t E = N * m;
  const RouteLayout L = RouteLayout::make(E, K);
  if (ws_bytes < L.bytes) return GMM_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  if (E <= kTinyE) {
    ProfScope p("route_tiny_kernel", s);
    // one thread an entry, and enough of them for the K + 1 offsets
    int threads = (int)((E + 31) / 32 * 32);
    const int spread = (K + 1 + 31) / 32 * 32;
    if (threads < spread) threads = spread < kTinyE ? spread : kTinyE;
    route_tiny_kernel<<<1, threads, 0, s>>>(ids, (int)E, K, offsets, entry, slot);
    return launched();
  }
  uint32_t* counts = at<uint32_t>(ws, L.off_counts);
  uint32_t* tot = at<uint32_t>(ws, L.off_tot);
  const int G = K + 1;
  const size_t bins = sizeof(uint32_t) * (size_t)(G < kSlice ? G : kSlice);
  static std::atomic<uint64_t> scatter_allowed, count_allowed;
  if (!allow_smem((const void*)route_scatter_kernel, kScatterSmem, scatter_allowed) ||
      !allow_smem((const void*)route_count_kernel, sizeof(uint32_t) * kSlice, count_allowed))
    return GMM_ERR_CUDA;
  ProfScope p("route_kernels", s, L.base_here ? 3 : 4);
  gmm_status r;
  route_count_kernel<<<(unsigned)L.nb, kCountThreads, bins, s>>>(ids, E, K, L.tile, counts);
  if ((r = launched()) != GMM_OK) return r;
  route_scan_blocks_kernel<<<(K + 1 + 31) / 32, 1024, 0, s>>>(counts, L.nb, K + 1, tot);
  if ((r = launched()) != GMM_OK) return r;
  if (!L.base_here) {
    route_scan_groups_kernel<<<1, 1024, 0, s>>>(tot, K, offsets);
    if ((r = launched()) != GMM_OK) return r;
  }
  route_scatter_kernel<<<(unsigned)L.nb, L.warps * 32, L.smem, s>>>(
      ids, E, K, L.seg, L.base_here, counts, tot, offsets, entry, slot);
  return launched();
}

}  // extern "C"
