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
// A persistent block per multiprocessor: one warp fetches (four stages of 48
// KB), one issues the products into one of two 256-column accumulators, four
// read the other one back and store it.  Sums are fp32 in tensor memory,
// rounded once.
#include <cuda.h>

#include <type_traits>

#include "expert_product.cuh"
#include "tc_ptx.cuh"

namespace gmm {
namespace {

constexpr int kStages = 4;
constexpr int kBox = 8192;                 // 64 rows x 128 bytes
constexpr int kTileM = 128, kTileN = 256, kTileK = 64;
constexpr int kStageBytes = (kTileM + kTileN) * kTileK * 2;
constexpr int kThreads = 192;              // fetch, issue, four read back
constexpr int kOutBytes = 4096;            // 32 rows x 128 bytes of dW on their way out
constexpr int kOutAt = kStages * kStageBytes;            // two for each read-back warp
constexpr int kBarsAt = kOutAt + 4 * 2 * kOutBytes;
constexpr int kSmem = kBarsAt + 256 + 1024;
constexpr uint32_t kWait = 2000000;        // polls of up to a microsecond

enum { kProduct = 0, kDx = 1, kDw = 2 };

struct TcArgs {
  const int64_t* offsets;
  const int32_t* count;
  const int4* tiles;
  DeviceStatus* st;
  int64_t R;
  int K, d_from, d_to;  // rows' width and the output's (dw: d_in, d_out)
};

// One tile: `n` columns, the contraction's `len` terms.
struct Tile {
  int k, i0, j0, n, len;
  int64_t row0;
};

template <int MODE>
__device__ __forceinline__ int tile_total(const TcArgs& a) {
  if (MODE == kDw) return a.K * ((a.d_to + kTileM - 1) / kTileM) * ((a.d_from + kTileN - 1) / kTileN);
  return *a.count * ((a.d_to + kTileM - 1) / kTileM);
}

template <int MODE>
__device__ __forceinline__ Tile tile_at(const TcArgs& a, int t) {
  Tile w;
  const int mt = (a.d_to + kTileM - 1) / kTileM;
  if (MODE == kDw) {
    const int nt = (a.d_from + kTileN - 1) / kTileN;
    w.k = t / (mt * nt);
    const int r = t % (mt * nt);
    w.i0 = (r / nt) * kTileM;
    w.j0 = (r % nt) * kTileN;
    w.n = min(kTileN, a.d_from - w.j0);
    const int64_t b = clamp_row(a.offsets[w.k], a.R), e = clamp_row(a.offsets[w.k + 1], a.R);
    w.row0 = b;
    w.len = e > b ? (int)(e - b) : 0;
  } else {
    const int4 q = a.tiles[t / mt];
    w.k = q.x;
    w.row0 = q.y;
    w.n = q.z;
    w.i0 = (t % mt) * kTileM;
    w.j0 = 0;
    w.len = q.x < 0 ? 0 : a.d_from;
  }
  return w;
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(tc::smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(tc::smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_addr(bar))
      : "memory");
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
__device__ __forceinline__ uint32_t idesc(bool bf16, bool p_mn, bool q_mn, int n) {
  const uint32_t f = bf16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)p_mn << 15) | ((uint32_t)q_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTileM >> 4) << 24);
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

// 32 columns (rows of the output) of this lane's feature; lanes exchange so
// that each holds two neighbouring features of every other row.
template <typename TO>
__device__ __forceinline__ void store_rows(const float* v, TO* out, int64_t ld, int f, int d_to,
                                           int left) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1;
  const bool live = f < d_to;  // d_to is even
  TO* p = out + (f & ~1);
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
    const uint32_t w = odd ? Pair<TO>::pack(got, v[j + 1]) : Pair<TO>::pack(v[j], got);
    const int r = j + (odd ? 1 : 0);
    if (live && r < left) *reinterpret_cast<uint32_t*>(p + (int64_t)r * ld) = w;
  }
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

template <int MODE, typename T, typename TO>
__global__ void __launch_bounds__(kThreads, 1)
expert_tc_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                 const __grid_constant__ CUtensorMap map_out, TO* __restrict__ out, TcArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarsAt);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2]
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kPmn = MODE != kProduct, kQmn = MODE == kDw;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&acc_full[i], 1);
      tc::mbar_init(&acc_empty[i], 4);
    }
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_at, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_at;
  // the list (or the cleared status word) and everything before it is there
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = tile_total<MODE>(a);

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        const Tile w = tile_at<MODE>(a, t);
        const int boxes = (w.n + 63) / 64;
        for (int l = 0; l < w.len; l += kTileK, ++it) {
          const int s = it % kStages;
          if (it >= kStages && !tc::mbar_wait(&empty[s], ((it / kStages) - 1) & 1, kWait)) {
            raise_status(a.st, GMM_ERR_TIMEOUT);
            ok = false;
            break;
          }
          uint8_t* p = smem + s * kStageBytes;
          uint8_t* q = p + kTileM * kTileK * 2;
          tc::mbar_arrive_expect_tx(&full[s], (2 + boxes) * kBox);
          if (MODE == kProduct) {
            tma_3d(p, &map_p, l, w.i0, w.k, &full[s]);
            tma_3d(p + kBox, &map_p, l, w.i0 + 64, w.k, &full[s]);
          } else if (MODE == kDx) {
            tma_3d(p, &map_p, w.i0, l, w.k, &full[s]);
            tma_3d(p + kBox, &map_p, w.i0 + 64, l, w.k, &full[s]);
          } else {
            tma_2d(p, &map_p, w.i0, (int)w.row0 + l, &full[s]);
            tma_2d(p + kBox, &map_p, w.i0 + 64, (int)w.row0 + l, &full[s]);
          }
          for (int b = 0; b < boxes; ++b) {
            if (MODE == kDw) tma_2d(q + b * kBox, &map_q, w.j0 + 64 * b, (int)w.row0 + l, &full[s]);
            else tma_2d(q + b * kBox, &map_q, l, (int)w.row0 + 64 * b, &full[s]);
          }
        }
      }
      if (!ok)  // the copies in flight end before the block does
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
          tc::mbar_wait(&full[i % kStages], (i / kStages) & 1, kWait);
    }
  } else if (warp == 1) {
    uint32_t it = 0, acc = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile w = tile_at<MODE>(a, t);
      if (w.len == 0) continue;
      const int b = acc & 1;
      if (acc >= 2 && !tc::mbar_wait(&acc_empty[b], ((acc >> 1) - 1) & 1, kWait)) ok = false;
      const uint32_t d = tmem + b * kTileN;
      const int n = (w.n + 15) & ~15;
      const uint32_t id = idesc(std::is_same<T, __nv_bfloat16>::value, kPmn, kQmn, n);
      for (int l = 0; ok && l < w.len; l += kTileK, ++it) {
        const int s = it % kStages;
        if (!tc::mbar_wait(&full[s], (it / kStages) & 1, kWait)) {
          ok = false;
          break;
        }
        uint8_t* p = smem + s * kStageBytes;
        uint8_t* q = p + kTileM * kTileK * 2;
        const int left = min(kTileK, w.len - l);
        const int steps = (left + 15) / 16;
        if (MODE == kDw && left < 16 * steps) {
          // rows of the next component, up to the next 16: 128 bytes of each box
          const int rows = 16 * steps - left, boxes = 2 + (w.n + 63) / 64;
          for (int x = lane; x < boxes * rows * 8; x += 32) {
            const int box = x / (rows * 8), r = left + (x / 8) % rows, c = x & 7;
            *reinterpret_cast<uint4*>(p + box * kBox + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          tc::tc_fence_after();
          const uint32_t ps = tc::smem_addr(p), qs = tc::smem_addr(q);
          for (int x = 0; x < steps; ++x) {
            const uint64_t dp = kPmn ? sdesc_mn128(ps + x * 2048) : tc::sdesc_k128(ps + x * 32);
            const uint64_t dq = kQmn ? sdesc_mn128(qs + x * 2048) : tc::sdesc_k128(qs + x * 32);
            tc::mma_f16(d, dp, dq, id, (l > 0 || x > 0) ? 1u : 0u);
          }
          tc::mma_commit(&empty[s]);
          if (l + kTileK >= w.len) tc::mma_commit(&acc_full[b]);
        }
        __syncwarp();
      }
      ++acc;
    }
    if (!ok && lane == 0) raise_status(a.st, GMM_ERR_TIMEOUT);
  } else {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    uint32_t acc = 0, piece = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const Tile w = tile_at<MODE>(a, t);
      const int b = acc & 1;
      const int f = w.i0 + quarter * 32 + lane;
      if (w.len > 0) {
        if (!tc::mbar_wait(&acc_full[b], (acc >> 1) & 1, kWait)) {
          if (lane == 0) raise_status(a.st, GMM_ERR_TIMEOUT);
          break;
        }
        tc::tc_fence_after();
      }
      const uint32_t src = tmem + b * kTileN + ((uint32_t)(quarter * 32) << 16);
      if constexpr (MODE == kDw) {
        // pieces of 32 rows x 128 bytes, two in flight; the tensor map cuts
        // off what is past dW's edges
        constexpr int W = 128 / sizeof(TO);
        uint8_t* pieces = smem + kOutAt + quarter * 2 * kOutBytes;
        const int y = w.i0 + quarter * 32;
        for (int c = 0; c < w.n && y < a.d_to; c += W, ++piece) {
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
          uint8_t* at = pieces + (piece & 1) * kOutBytes;
          if (lane == 0)  // the store before the last one has read its piece
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
          stage_line(r[0], at);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&map_out, at, w.j0 + c, y, w.k);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      } else {
        for (int c = 0; c < w.n; c += 32) {
          float v[32];
          if (w.len > 0) {
            tc::tmem_ld32(src + c, v);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
          }
          store_rows(v, out + (w.row0 + c) * (int64_t)a.d_to, a.d_to, f, a.d_to, w.n - c);
        }
      }
      if (w.len > 0) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty[b]);
        ++acc;
      }
    }
    if (MODE == kDw && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
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

int multiprocessors() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

template <int MODE, typename T, typename TO>
gmm_status go(const CUtensorMap& mp, const CUtensorMap& mq, const CUtensorMap& mo, void* out,
              const TcArgs& a, int64_t most, cudaStream_t s) {
  const int sms = multiprocessors();
  if (sms < 1 || cudaFuncSetAttribute(expert_tc_kernel<MODE, T, TO>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return GMM_ERR_CUDA;
  const unsigned grid = (unsigned)(most < sms ? most : sms);
  ProfScope p(MODE == kProduct ? "expert_tc_kernel" : MODE == kDx ? "expert_tc_kernel(dx)" : "expert_tc_kernel(dw)", s);
  // may start while the kernel that makes its list runs
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, expert_tc_kernel<MODE, T, TO>, mp, mq, mo, (TO*)out, a);
  return launched();
}

}  // namespace

bool tc_product_ok(int xdtype, int64_t R, int d_in, int d_out, const void* a, const void* b, const void* c) {
  return xdtype != GMM_F32 && R <= INT32_MAX - 256 && d_in % 8 == 0 && d_out % 8 == 0 &&
         ((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) % 16 == 0;
}

gmm_status tc_rows(const void* A, int xdtype, const void* W, void* Y, int64_t R, int d_from,
                   int d_to, int K, bool dx, const int64_t* offsets, void* ws, cudaStream_t s) {
  const ProductLayout L = ProductLayout::make(R, d_from, d_to, K);
  const gmm_status r = list_tiles(offsets, K, R, kTileN, ws, L, s);
  if (r != GMM_OK || R == 0) return r;
  CUtensorMap mp, mq;
  const int d_in = dx ? d_to : d_from, d_out = dx ? d_from : d_to;
  if (!encode(&mp, xdtype, W, d_in, d_out, K, 64) || !encode(&mq, xdtype, A, d_from, R, 0, 64))
    return GMM_ERR_CUDA;
  TcArgs a{offsets, at<int32_t>(ws, L.off_count), at<int4>(ws, L.off_tiles), at<DeviceStatus>(ws, 0),
           R, K, d_from, d_to};
  const int64_t most = ProductLayout::most_tiles(R, K, kTileN) * ((d_to + kTileM - 1) / kTileM);
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
  if (!encode(&mp, xdtype, dY, d_out, R, 0, 64) || !encode(&mq, xdtype, A, d_in, R, 0, 64) ||
      !encode(&mo, wdtype, dW, d_in, d_out, K, 32))
    return GMM_ERR_CUDA;
  const gmm_status r = clear_status(ws, s);
  if (r != GMM_OK) return r;
  TcArgs a{offsets, nullptr, nullptr, at<DeviceStatus>(ws, 0), R, K, d_in, d_out};
  const int64_t most =
      (int64_t)K * ((d_out + kTileM - 1) / kTileM) * ((d_in + kTileN - 1) / kTileN);
  if (most > INT32_MAX) return GMM_ERR_UNSUPPORTED;
  if (xdtype == GMM_BF16) {
    using T = __nv_bfloat16;
    return wdtype == GMM_F32 ? go<kDw, T, float>(mp, mq, mo, dW, a, most, s) : go<kDw, T, T>(mp, mq, mo, dW, a, most, s);
  }
  using T = __half;
  return wdtype == GMM_F32 ? go<kDw, T, float>(mp, mq, mo, dW, a, most, s) : go<kDw, T, T>(mp, mq, mo, dW, a, most, s);
}

}  // namespace gmm
