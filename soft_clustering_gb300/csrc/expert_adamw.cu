// expert_adamw.cu - gmm_adamw_step: one AdamW step over many tensors.
//
// The table of tensors travels in the launch's parameters (up to kTable at a
// time), so nothing is kept between calls and one launch serves a whole
// model.  A warp takes 256 consecutive elements of a tensor at a time, eight
// to a lane: the block that shares one scale where the moments are held in 8
// bits, so its largest value is a shuffle away.  Every operation is the
// IEEE one in the documented order (no contraction), so the results are the
// formula's in fp32 to the bit; square roots and divisions included.
// Bound by HBM traffic: 28 bytes an element in fp32, 10 with 16-bit
// parameters and gradients and 8-bit moments.
#include <cmath>

#include "expert_internal.cuh"

namespace gmm {
namespace {

constexpr int kBlockElems = 256;   // elements of one scale, and of one warp's turn
constexpr int kWarps = 8;
constexpr int kChunk = kWarps * kBlockElems;  // elements of one block's turn
constexpr float kTiny = 1e-30f;    // blocks below it are held as zeros

struct AdamwEntry {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  int32_t first;     // the tensor's first chunk in this launch
  int8_t pt, gt;     // gmm_dtype
  int8_t wide;       // every array aligned for eight-element accesses
  int8_t pad;
};

struct AdamwConst {
  float gs, b1, c1, b2, c2, root, eps, decay, rate;
  int count, chunks;
  const int32_t* skip;
};

template <int COUNT>
struct AdamwTable {
  AdamwConst k;
  AdamwEntry e[COUNT];
};

__device__ __forceinline__ void load8(const void* base, int type, int64_t i, float* x) {
  if (type == GMM_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (type == GMM_F16) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[j]);
        x[2 * j] = __half2float(__low2half(h));
        x[2 * j + 1] = __half2float(__high2half(h));
      } else {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ void store8(void* base, int type, int64_t i, const float* x) {
  if (type == GMM_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (type == GMM_F16) {
        const __half2 h = __halves2half2(__float2half_rn(x[2 * j]), __float2half_rn(x[2 * j + 1]));
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ float load1(const void* base, int type, int64_t i) {
  if (type == GMM_F32) return static_cast<const float*>(base)[i];
  if (type == GMM_F16) return __half2float(static_cast<const __half*>(base)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}

__device__ __forceinline__ void store1(void* base, int type, int64_t i, float x) {
  if (type == GMM_F32) static_cast<float*>(base)[i] = x;
  else if (type == GMM_F16) static_cast<__half*>(base)[i] = __float2half_rn(x);
  else static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(x);
}

// `cnt` (0..8) elements from i; the rest read as zeros.
__device__ __forceinline__ void load_n(const void* base, int type, int64_t i, int cnt, bool wide,
                                       float* x) {
  if (wide && cnt == 8) return load8(base, type, i, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = j < cnt ? load1(base, type, i + j) : 0.f;
}
__device__ __forceinline__ void store_n(void* base, int type, int64_t i, int cnt, bool wide,
                                        const float* x) {
  if (wide && cnt == 8) return store8(base, type, i, x);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < cnt) store1(base, type, i + j, x[j]);
}

// Eight 8-bit codes as two words.
__device__ __forceinline__ uint2 load_codes(const void* base, int64_t i, int cnt, bool wide) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  if (wide && cnt == 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < cnt) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void* base, int64_t i, int cnt, bool wide, uint2 c) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  if (wide && cnt == 8) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < cnt) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// c|c| S
__device__ __forceinline__ void decode_m(uint2 c, float scale, float* x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = j < 4 ? c.x : c.y;
    const float f = (float)(int8_t)(w >> (8 * (j & 3)));
    x[j] = __fmul_rn(f * fabsf(f), scale);
  }
}
__device__ __forceinline__ void decode_root(uint2 c, float scale, float* x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = j < 4 ? c.x : c.y;
    const float f = (float)((w >> (8 * (j & 3))) & 0xffu);
    x[j] = __fmul_rn(f * f, scale);
  }
}

// Codes of eight values whose block's largest magnitude is `big`.
template <int TOP>
__device__ __forceinline__ uint2 encode(const float* x, float big, float* scale) {
  const bool zero = !(big >= kTiny);
  *scale = zero ? 0.f : __fmul_rn(big, (float)(1.0 / (TOP * TOP)));
  const float inv = zero ? 0.f : __fmul_rn(__fdiv_rn(1.f, big), (float)(TOP * TOP));
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float c = fminf(rintf(__fsqrt_rn(__fmul_rn(fabsf(x[j]), inv))), (float)TOP);
    if (TOP == 255) {
      if (x[j] > 0.f) c = fmaxf(c, 1.f);
    } else if (x[j] < 0.f) {
      c = -c;
    }
    w[j >> 2] |= ((uint32_t)(int)c & 0xffu) << (8 * (j & 3));
  }
  return make_uint2(w[0], w[1]);
}

// The tensor of a chunk: the last entry whose first chunk is not after it.
template <int COUNT>
__device__ __forceinline__ int tensor_of(const AdamwTable<COUNT>& t, int chunk) {
  int lo = 0, hi = t.k.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int BITS, int COUNT>
__global__ void __launch_bounds__(kWarps * 32)
adamw_kernel(const __grid_constant__ AdamwTable<COUNT> t) {
  const AdamwConst& k = t.k;
  if (k.skip && *k.skip != 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int chunk = blockIdx.x; chunk < k.chunks; chunk += gridDim.x) {
    const AdamwEntry& e = t.e[tensor_of(t, chunk)];
    const int64_t block = (int64_t)(chunk - e.first) * kWarps + warp;
    const int64_t i = block * kBlockElems + lane * 8;
    if (block * kBlockElems >= e.n) continue;  // the same for the whole warp
    const int cnt = (int)max((int64_t)0, min((int64_t)8, e.n - i));
    const bool wide = e.wide;
    float g[8], p[8], m[8], v[8], root[8];
    load_n(e.g, e.gt, i, cnt, wide, g);
    if (e.master) load_n(e.master, GMM_F32, i, cnt, wide, p);
    else load_n(e.p, e.pt, i, cnt, wide, p);
    if (BITS == 32) {
      load_n(e.m, GMM_F32, i, cnt, wide, m);
      load_n(e.v, GMM_F32, i, cnt, wide, v);
    } else {
      const uint2 mc = load_codes(e.m, i, cnt, wide), vc = load_codes(e.v, i, cnt, wide);
      decode_m(mc, e.ms[block], m);
      decode_root(vc, e.vs[block], root);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(root[j], root[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = __fmul_rn(g[j], k.gs);
      m[j] = __fadd_rn(__fmul_rn(m[j], k.b1), __fmul_rn(gj, k.c1));
      v[j] = __fadd_rn(__fmul_rn(v[j], k.b2), __fmul_rn(__fmul_rn(gj, gj), k.c2));
      root[j] = __fsqrt_rn(v[j]);
      const float den = __fadd_rn(__fmul_rn(root[j], k.root), k.eps);
      p[j] = __fsub_rn(__fmul_rn(p[j], k.decay), __fdiv_rn(__fmul_rn(m[j], k.rate), den));
    }
    if (e.master) store_n(e.master, GMM_F32, i, cnt, wide, p);
    store_n(e.p, e.pt, i, cnt, wide, p);
    if (BITS == 32) {
      store_n(e.m, GMM_F32, i, cnt, wide, m);
      store_n(e.v, GMM_F32, i, cnt, wide, v);
    } else {
      float mb = 0.f, rb = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= cnt) m[j] = root[j] = 0.f;  // past the end
        mb = fmaxf(mb, fabsf(m[j]));
        rb = fmaxf(rb, root[j]);
      }
      mb = warp_max(mb);
      rb = warp_max(rb);
      float ms, vs;
      const uint2 mc = encode<127>(m, mb, &ms);
      const uint2 vc = encode<255>(root, rb, &vs);
      store_codes(e.m, i, cnt, wide, mc);
      store_codes(e.v, i, cnt, wide, vc);
      if (lane == 0) {
        e.ms[block] = ms;
        e.vs[block] = vs;
      }
    }
  }
}

// Moments in fp32: entry.p and entry.master are the outputs here.
template <int BITS, int COUNT>
__global__ void __launch_bounds__(kWarps * 32)
adamw_moments_kernel(const __grid_constant__ AdamwTable<COUNT> t) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int chunk = blockIdx.x; chunk < t.k.chunks; chunk += gridDim.x) {
    const AdamwEntry& e = t.e[tensor_of(t, chunk)];
    const int64_t block = (int64_t)(chunk - e.first) * kWarps + warp;
    const int64_t i = block * kBlockElems + lane * 8;
    if (block * kBlockElems >= e.n) continue;
    const int cnt = (int)max((int64_t)0, min((int64_t)8, e.n - i));
    const bool wide = e.wide;
    float m[8], v[8];
    if (BITS == 32) {
      load_n(e.m, GMM_F32, i, cnt, wide, m);
      load_n(e.v, GMM_F32, i, cnt, wide, v);
    } else {
      decode_m(load_codes(e.m, i, cnt, wide), e.ms[block], m);
      decode_root(load_codes(e.v, i, cnt, wide), e.vs[block], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
    }
    store_n(e.p, GMM_F32, i, cnt, wide, m);
    store_n(e.master, GMM_F32, i, cnt, wide, v);
  }
}

bool tensors_ok(const gmm_adamw_tensor* ts, int count, int bits, bool step) {
  if (count < 0 || (count > 0 && !ts) || (bits != 32 && bits != 8)) return false;
  for (int i = 0; i < count; ++i) {
    const gmm_adamw_tensor& t = ts[i];
    if (t.n < 0 || t.n > ((int64_t)1 << 40)) return false;
    if (step && (!dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype))) return false;
    if (t.n == 0) continue;
    if (!t.m || !t.v) return false;
    if (bits == 8 && (!t.m_scale || !t.v_scale)) return false;
    if (((uintptr_t)t.m_scale | (uintptr_t)t.v_scale) % 4) return false;
    if (bits == 32 && ((uintptr_t)t.m | (uintptr_t)t.v) % 4) return false;
    if (step) {
      if (!t.param || !t.grad) return false;
      if ((uintptr_t)t.param % dtype_size(t.param_dtype) ||
          (uintptr_t)t.grad % dtype_size(t.grad_dtype) || (uintptr_t)t.master % 4)
        return false;
    }
  }
  return true;
}

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// Launches `kernel-by-table-size` over the non-empty tensors, as many at a
// time as a table holds (and as 2^30 chunks).
template <int COUNT, typename Fill, typename Go>
gmm_status over_tables(const gmm_adamw_tensor* ts, int count, const AdamwConst& k, Fill fill, Go go) {
  AdamwTable<COUNT> t;
  t.k = k;
  t.k.count = 0;
  int64_t chunks = 0;
  for (int i = 0; i <= count; ++i) {
    const bool end = i == count;
    const int64_t c = end ? 0 : chunks_of(ts[i].n);
    if (t.k.count > 0 && (end || t.k.count == COUNT || chunks + c > (1 << 30))) {
      t.k.chunks = (int)chunks;
      go(t);
      const gmm_status r = launched();
      if (r != GMM_OK) return r;
      t.k.count = 0;
      chunks = 0;
    }
    if (end || c == 0) continue;
    AdamwEntry& e = t.e[t.k.count++];
    e = AdamwEntry{};
    fill(i, e);
    e.n = ts[i].n;
    e.first = (int32_t)chunks;
    chunks += c;
  }
  return GMM_OK;
}

constexpr int kSmallTable = 16, kTable = 400;
unsigned grid_for(int chunks) { return (unsigned)(chunks < 152 * 8 ? chunks : 152 * 8); }

}  // namespace
}  // namespace gmm

using namespace gmm;

extern "C" {

gmm_status gmm_adamw_step(const gmm_adamw_tensor* ts, int count, const gmm_adamw_opts* o,
                          void* stream) {
  if (!o || !tensors_ok(ts, count, o->state_bits, true)) return GMM_ERR_INVALID_ARG;
  if (o->step < 1 || !(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) ||
      !(o->eps >= 0) || !std::isfinite(o->lr) || !std::isfinite(o->weight_decay) ||
      !std::isfinite(o->grad_scale) || !std::isfinite(o->eps))
    return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)o->skip % 4) return GMM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  AdamwConst k{};
  k.gs = (float)o->grad_scale;
  k.b1 = (float)o->beta1;
  k.c1 = (float)(1.0 - o->beta1);
  k.b2 = (float)o->beta2;
  k.c2 = (float)(1.0 - o->beta2);
  k.root = (float)std::pow(1.0 - std::pow(o->beta2, (double)o->step), -0.5);
  k.eps = (float)o->eps;
  k.decay = (float)(1.0 - o->lr * o->weight_decay);
  k.rate = (float)(o->lr / (1.0 - std::pow(o->beta1, (double)o->step)));
  k.skip = o->skip;
  const int bits = o->state_bits;
  auto fill = [&](int i, AdamwEntry& e) {
    const gmm_adamw_tensor& t = ts[i];
    e.p = t.param; e.g = t.grad; e.master = t.master; e.m = t.m; e.v = t.v;
    e.ms = t.m_scale; e.vs = t.v_scale;
    e.pt = (int8_t)t.param_dtype; e.gt = (int8_t)t.grad_dtype;
    const uintptr_t mv = (uintptr_t)t.m | (uintptr_t)t.v;
    const uintptr_t rest = (uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.master;
    e.wide = rest % 16 == 0 && mv % (bits == 8 ? 8 : 16) == 0;
  };
  ProfScope p("adamw_kernel", s);
  auto go = [&](const auto& t) {
    constexpr int C = sizeof(t.e) / sizeof(t.e[0]);
    if (bits == 32) adamw_kernel<32, C><<<grid_for(t.k.chunks), kWarps * 32, 0, s>>>(t);
    else adamw_kernel<8, C><<<grid_for(t.k.chunks), kWarps * 32, 0, s>>>(t);
  };
  return count <= kSmallTable ? over_tables<kSmallTable>(ts, count, k, fill, go)
                              : over_tables<kTable>(ts, count, k, fill, go);
}

gmm_status gmm_adamw_moments(const gmm_adamw_tensor* ts, int count, int state_bits,
                             float* const* m_out, float* const* v_out, void* stream) {
  if (!tensors_ok(ts, count, state_bits, false) || (count > 0 && (!m_out || !v_out)))
    return GMM_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (ts[i].n > 0 && (!m_out[i] || !v_out[i] || ((uintptr_t)m_out[i] | (uintptr_t)v_out[i]) % 4))
      return GMM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  auto fill = [&](int i, AdamwEntry& e) {
    const gmm_adamw_tensor& t = ts[i];
    e.p = m_out[i]; e.master = v_out[i]; e.m = t.m; e.v = t.v;
    e.ms = t.m_scale; e.vs = t.v_scale;
    const uintptr_t mv = (uintptr_t)t.m | (uintptr_t)t.v;
    e.wide = ((uintptr_t)m_out[i] | (uintptr_t)v_out[i]) % 16 == 0 &&
             mv % (state_bits == 8 ? 8 : 16) == 0;
  };
  ProfScope p("adamw_moments_kernel", s);
  auto go = [&](const auto& t) {
    constexpr int C = sizeof(t.e) / sizeof(t.e[0]);
    if (state_bits == 32) adamw_moments_kernel<32, C><<<grid_for(t.k.chunks), kWarps * 32, 0, s>>>(t);
    else adamw_moments_kernel<8, C><<<grid_for(t.k.chunks), kWarps * 32, 0, s>>>(t);
  };
  return count <= kSmallTable ? over_tables<kSmallTable>(ts, count, AdamwConst{}, fill, go)
                              : over_tables<kTable>(ts, count, AdamwConst{}, fill, go);
}

}  // extern "C"
