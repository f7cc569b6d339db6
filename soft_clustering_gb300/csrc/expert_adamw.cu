// expert_adamw.cu - gmm_adamw_step: one AdamW step over many tensors.
//
// The table of tensors travels in the launch's parameters (up to kTable at a
// time), so nothing is kept between calls and one launch serves a whole
// model.  A warp takes 256 consecutive elements of a tensor at a time, eight
// to a lane: the block that shares one scale where the moments are held in 8
// bits, so its largest value is a warp reduction away.  Blocks take
// contiguous stretches of the list (one search of the table each) and fetch
// the next turn's operands before they work on the present ones.
//
// Bound by HBM traffic: 28 bytes an element in fp32, 10 with 16-bit
// parameters and gradients and 8-bit moments.  With fp32 moments every
// operation is the IEEE one in the documented order.  With 8-bit moments the
// arithmetic competes with the traffic (10 bytes leave about 50 instructions
// an element), so there
//   - bytes become floats and floats codes by adding 2^23 (or 1.5 2^23), on
//     the FP32 pipe instead of the conversion unit;
//   - square roots are approximate (2 units in the last place) wherever the
//     rounding to a code cannot depend on it: a root within kNear of halfway
//     between two codes, about one in 2500, is taken again exactly, so the
//     codes and scales are those of the exact roots;
//   - the parameter's update uses the approximate root and reciprocal: a
//     relative error of the update below 2^-21, under the rounding of the
//     parameter.
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

// Byte j of two words as a float (unsigned, or two's complement).
template <bool SIGNED>
__device__ __forceinline__ float code_float(uint2 c, int j) {
  const uint32_t w = (j < 4 ? c.x : c.y) ^ (SIGNED ? 0x80808080u : 0u);
  // bits 0x4B0000cc are 2^23 + cc
  const float f = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | (j & 3)));
  return f - (SIGNED ? 8388736.f : 8388608.f);
}

// c|c| S
__device__ __forceinline__ void decode_m(uint2 c, float scale, float* x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = code_float<true>(c, j);
    x[j] = __fmul_rn(f * fabsf(f), scale);
  }
}
__device__ __forceinline__ void decode_root(uint2 c, float scale, float* x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = code_float<false>(c, j);
    x[j] = __fmul_rn(f * f, scale);
  }
}

__device__ __forceinline__ float sqrt_near(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_near(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 255 x (2^-22 for each root and the product between them) is 2e-4 at most.
constexpr float kNear = 0.5f - 2e-4f;
constexpr float kMagic = 12582912.f;  // 1.5 2^23: x + kMagic holds rint(x) in its low bits

// Scale of a block whose largest magnitude is `big`, and its inverse.
template <int TOP>
__device__ __forceinline__ float2 scale_of(float big) {
  if (!(big >= kTiny)) return make_float2(0.f, 0.f);
  return make_float2(__fmul_rn(big, (float)(1.0 / (TOP * TOP))),
                     __fmul_rn(__fdiv_rn(1.f, big), (float)(TOP * TOP)));
}

// Codes of eight m.
__device__ __forceinline__ uint2 encode_m(const float* m, float inv) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = __fmul_rn(fabsf(m[j]), inv);
    float s = sqrt_near(x);
    t[j] = s + kMagic;
    if (fabsf(s - (t[j] - kMagic)) > kNear) t[j] = __fsqrt_rn(x) + kMagic;
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = __float_as_uint(t[4 * h + j]);
      b[j] = m[4 * h + j] < 0.f ? 0u - u : u;  // the low byte of -c
    }
    w[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

// Codes of eight sqrt(v); root is near, v exact.
__device__ __forceinline__ uint2 encode_root(const float* v, const float* root, float inv) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float s = sqrt_near(root[j] * inv);
    t[j] = s + kMagic;
    const bool tiny = v[j] < 1e-36f && v[j] > 0.f;  // the near root of a subnormal is 0
    if (fabsf(s - (t[j] - kMagic)) > kNear || tiny)
      t[j] = __fsqrt_rn(__fmul_rn(__fsqrt_rn(v[j]), inv)) + kMagic;
    if (v[j] > 0.f) t[j] = fmaxf(t[j], 1.f + kMagic);
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = __byte_perm(__byte_perm(__float_as_uint(t[4 * h]), __float_as_uint(t[4 * h + 1]), 0x0040),
                       __byte_perm(__float_as_uint(t[4 * h + 2]), __float_as_uint(t[4 * h + 3]), 0x0040),
                       0x5410);
  return make_uint2(w[0], w[1]);
}

// Largest of the warp's non-negative values (their bits order them).
__device__ __forceinline__ float warp_max_pos(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
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

// Eight elements as they lie in memory: 4 words of 16-bit ones, 8 of floats.
template <bool HALF> struct Raw { uint32_t w[HALF ? 4 : 8]; };

template <bool HALF>
__device__ __forceinline__ void fetch(Raw<HALF>& r, const void* base, int64_t i, int cnt, bool wide) {
  if (wide && cnt == 8) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * (HALF ? 2 : 4));
    const uint4 a = p[0];
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    if constexpr (!HALF) {
      const uint4 b = p[1];
      r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < (HALF ? 4 : 8); ++j) r.w[j] = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < cnt) {
      if (HALF) r.w[j / 2] |= (uint32_t)static_cast<const uint16_t*>(base)[i + j] << (16 * (j & 1));
      else r.w[j] = static_cast<const uint32_t*>(base)[i + j];
    }
}
template <bool HALF>
__device__ __forceinline__ void widen(const Raw<HALF>& r, int type, float* x) {
  if constexpr (!HALF) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r.w[j]);
  } else if (type == GMM_F16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[j]));
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(r.w[j] << 16);
      x[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
    }
  }
}

// Where a warp is in the list: its tensor, and its eight elements there.
struct Place {
  int e;
  int64_t block, i;
  int cnt;   // 0: nothing for this lane; < 0: nothing for this warp
};

template <int COUNT>
__device__ __forceinline__ Place place_of(const AdamwTable<COUNT>& t, int e, int chunk) {
  while (e + 1 < t.k.count && t.e[e + 1].first <= chunk) ++e;
  Place p;
  p.e = e;
  p.block = (int64_t)(chunk - t.e[e].first) * kWarps + (threadIdx.x >> 5);
  p.i = p.block * kBlockElems + (threadIdx.x & 31) * 8;
  const int64_t n = t.e[e].n;
  p.cnt = p.block * kBlockElems >= n ? -1 : (int)max((int64_t)0, min((int64_t)8, n - p.i));
  return p;
}

template <int BITS, bool PH, bool GH> struct Operands {
  Raw<PH> p;
  Raw<GH> g;
  uint32_t m[BITS == 32 ? 8 : 2], v[BITS == 32 ? 8 : 2];
  float ms, vs;
};

template <int BITS, bool PH, bool GH>
__device__ __forceinline__ void fetch_all(Operands<BITS, PH, GH>& o, const AdamwEntry& e, const Place& q) {
  if (q.cnt < 0) return;
  const bool wide = e.wide;
  fetch<GH>(o.g, e.g, q.i, q.cnt, wide);
  fetch<PH>(o.p, e.master ? (const void*)e.master : e.p, q.i, q.cnt, wide);
  if constexpr (BITS == 32) {
    Raw<false> r;
    fetch<false>(r, e.m, q.i, q.cnt, wide);
#pragma unroll
    for (int j = 0; j < 8; ++j) o.m[j] = r.w[j];
    fetch<false>(r, e.v, q.i, q.cnt, wide);
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = r.w[j];
  } else {
    const uint2 mc = load_codes(e.m, q.i, q.cnt, wide), vc = load_codes(e.v, q.i, q.cnt, wide);
    o.m[0] = mc.x; o.m[1] = mc.y;
    o.v[0] = vc.x; o.v[1] = vc.y;
    o.ms = e.ms[q.block];
    o.vs = e.vs[q.block];
  }
}

template <int BITS, bool PH, bool GH>
__device__ __forceinline__ void step_block(const AdamwConst& k, const AdamwEntry& e, const Place& q,
                                           const Operands<BITS, PH, GH>& o) {
  const bool wide = e.wide;
  float g[8], p[8], m[8], v[8], root[8];
  widen<GH>(o.g, e.gt, g);
  widen<PH>(o.p, e.pt, p);
  if constexpr (BITS == 32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = __uint_as_float(o.m[j]);
      v[j] = __uint_as_float(o.v[j]);
    }
  } else {
    decode_m(make_uint2(o.m[0], o.m[1]), o.ms, m);
    decode_root(make_uint2(o.v[0], o.v[1]), o.vs, root);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(root[j], root[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = __fmul_rn(g[j], k.gs);
    m[j] = __fadd_rn(__fmul_rn(m[j], k.b1), __fmul_rn(gj, k.c1));
    v[j] = __fadd_rn(__fmul_rn(v[j], k.b2), __fmul_rn(__fmul_rn(gj, gj), k.c2));
    if constexpr (BITS == 32) {
      root[j] = __fsqrt_rn(v[j]);
      const float den = __fadd_rn(__fmul_rn(root[j], k.root), k.eps);
      p[j] = __fsub_rn(__fmul_rn(p[j], k.decay), __fdiv_rn(__fmul_rn(m[j], k.rate), den));
    } else {
      root[j] = sqrt_near(v[j]);
      const float den = fmaf(root[j], k.root, k.eps);
      float r = rcp_near(den);
      // outside the reciprocal's range, or the near root's: the exact form
      if (!(den > 1e-18f && den < 1e37f))
        r = __fdiv_rn(1.f, __fadd_rn(__fmul_rn(__fsqrt_rn(v[j]), k.root), k.eps));
      p[j] = __fsub_rn(__fmul_rn(p[j], k.decay), __fmul_rn(__fmul_rn(m[j], k.rate), r));
    }
  }
  if (e.master) store_n(e.master, GMM_F32, q.i, q.cnt, wide, p);
  store_n(e.p, e.pt, q.i, q.cnt, wide, p);
  if constexpr (BITS == 32) {
    store_n(e.m, GMM_F32, q.i, q.cnt, wide, m);
    store_n(e.v, GMM_F32, q.i, q.cnt, wide, v);
  } else {
    if (q.cnt < 8) {  // past the end
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= q.cnt) m[j] = v[j] = root[j] = 0.f;
    }
    float mb = 0.f, vb = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mb = fmaxf(mb, fabsf(m[j]));
      vb = fmaxf(vb, v[j]);
    }
    const float2 ms = scale_of<127>(warp_max_pos(mb));
    const float2 vs = scale_of<255>(__fsqrt_rn(warp_max_pos(vb)));
    store_codes(e.m, q.i, q.cnt, wide, encode_m(m, ms.y));
    store_codes(e.v, q.i, q.cnt, wide, encode_root(v, root, vs.y));
    if ((threadIdx.x & 31) == 0) {
      e.ms[q.block] = ms.x;
      e.vs[q.block] = vs.x;
    }
  }
}

// PH, GH: 16-bit parameters (no master) and gradients.
template <int BITS, bool PH, bool GH, int COUNT>
__global__ void __launch_bounds__(kWarps * 32)
adamw_kernel(const __grid_constant__ AdamwTable<COUNT> t) {
  const AdamwConst& k = t.k;
  if (k.skip && *k.skip != 0) return;
  const int c0 = (int)((int64_t)k.chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)k.chunks * (blockIdx.x + 1) / gridDim.x);
  if (c0 >= c1) return;
  Place here = place_of(t, tensor_of(t, c0), c0);
  Operands<BITS, PH, GH> o;
  fetch_all(o, t.e[here.e], here);
  for (int c = c0; c < c1; ++c) {
    Operands<BITS, PH, GH> next;
    Place there = here;
    if (c + 1 < c1) {
      there = place_of(t, here.e, c + 1);
      fetch_all(next, t.e[there.e], there);
    }
    if (here.cnt >= 0) step_block<BITS, PH, GH>(k, t.e[here.e], here, o);
    o = next;
    here = there;
  }
}

// Moments in fp32: entry.p and entry.master are the outputs here.
template <int BITS, int COUNT>
__global__ void __launch_bounds__(kWarps * 32)
adamw_moments_kernel(const __grid_constant__ AdamwTable<COUNT> t) {
  const int c0 = (int)((int64_t)t.k.chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)t.k.chunks * (blockIdx.x + 1) / gridDim.x);
  if (c0 >= c1) return;
  int at = tensor_of(t, c0);
  for (int c = c0; c < c1; ++c) {
    const Place q = place_of(t, at, c);
    at = q.e;
    if (q.cnt < 0) continue;
    const AdamwEntry& e = t.e[q.e];
    const bool wide = e.wide;
    float m[8], v[8];
    if (BITS == 32) {
      load_n(e.m, GMM_F32, q.i, q.cnt, wide, m);
      load_n(e.v, GMM_F32, q.i, q.cnt, wide, v);
    } else {
      decode_m(load_codes(e.m, q.i, q.cnt, wide), e.ms[q.block], m);
      decode_root(load_codes(e.v, q.i, q.cnt, wide), e.vs[q.block], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
    }
    store_n(e.p, GMM_F32, q.i, q.cnt, wide, m);
    store_n(e.master, GMM_F32, q.i, q.cnt, wide, v);
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

// Launches over the non-empty tensors that `take` wants, as many at a time as
// a table holds (and as 2^30 chunks).
template <int COUNT, typename Take, typename Fill, typename Go>
gmm_status over_tables(const gmm_adamw_tensor* ts, int count, const AdamwConst& k, Take take,
                       Fill fill, Go go) {
  AdamwTable<COUNT> t;
  t.k = k;
  t.k.count = 0;
  int64_t chunks = 0;
  for (int i = 0; i <= count; ++i) {
    const bool end = i == count;
    const int64_t c = end || !take(i) ? 0 : chunks_of(ts[i].n);
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
  // one launch for each kind of operands that is there: 16-bit or fp32
  // parameters (with a master: fp32) and gradients
  for (int kind = 0; kind < 4; ++kind) {
    const bool ph = kind & 1, gh = kind & 2;
    auto take = [&](int i) {
      return (ts[i].param_dtype != GMM_F32 && !ts[i].master) == ph && (ts[i].grad_dtype != GMM_F32) == gh;
    };
    auto go = [&](const auto& t) {
      constexpr int C = sizeof(t.e) / sizeof(t.e[0]);
      const unsigned grid = grid_for(t.k.chunks);
#define GMM_GO(B)                                                                        \
  if (ph && gh) adamw_kernel<B, true, true, C><<<grid, kWarps * 32, 0, s>>>(t);           \
  else if (ph) adamw_kernel<B, true, false, C><<<grid, kWarps * 32, 0, s>>>(t);           \
  else if (gh) adamw_kernel<B, false, true, C><<<grid, kWarps * 32, 0, s>>>(t);           \
  else adamw_kernel<B, false, false, C><<<grid, kWarps * 32, 0, s>>>(t);
      if (bits == 32) { GMM_GO(32) } else { GMM_GO(8) }
#undef GMM_GO
    };
    const gmm_status r = count <= kSmallTable ? over_tables<kSmallTable>(ts, count, k, take, fill, go)
                                              : over_tables<kTable>(ts, count, k, take, fill, go);
    if (r != GMM_OK) return r;
  }
  return GMM_OK;
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
  auto all = [](int) { return true; };
  return count <= kSmallTable ? over_tables<kSmallTable>(ts, count, AdamwConst{}, all, fill, go)
                              : over_tables<kTable>(ts, count, AdamwConst{}, all, fill, go);
}

}  // extern "C"
