// expert_adamw.cu - gmm_adamw_step: one AdamW step over many tensors.
//
// The table of tensors travels in the launch's parameters (up to kTable at a
// time), so nothing is kept between calls and one launch serves a whole
// model.  A warp takes 256 consecutive elements of a tensor at a time, eight
// to a lane: the block that shares one scale where the moments are held in 8
// bits, so its largest value is a warp reduction away.  Blocks take
// contiguous stretches of the list (one search of the table each), up to 16
// turns a warp in one tensor, and fetch ahead: three turns through shared
// memory where the moments are bytes (a lane has 24 bytes a turn, too little
// in flight otherwise), one turn in registers where they are floats.
//
// Bound by HBM traffic in fp32, 28 bytes an element, where every operation is
// the IEEE one in the documented order.  With 16-bit parameters and gradients
// and 8-bit moments an element is 10 bytes, which leave time for about 40
// instructions, so there the arithmetic is the bound, and
//   - bytes become floats and floats codes by adding 2^23 (or 1.5 2^23), on
//     the FP32 pipe instead of the conversion unit;
//   - square roots are approximate (2 units in the last place) wherever the
//     rounding to a code cannot depend on it: a root within kNear of halfway
//     between two codes, about one in 2500, is taken again exactly, so the
//     codes and scales are those of the exact roots;
//   - the parameter's update uses the approximate root and reciprocal, which
//     add 2^-21 of the update: under the rounding of a 16-bit parameter, not
//     under that of an fp32 one (or master) near zero;
//   - products and sums go by pairs of elements (packed fp32 operations).
// Rounding codes to the nearest loses every change below half a code; seeded
// rounding does not, and takes random bits for both moments of every element.
// Measured: 1e8 elements in fp32 419 us (6.68 TB/s, 98 % of the copy rate),
// counted on the device 446.  2e8 bf16 elements with 8-bit moments, nearest,
// 473 us (4.2 TB/s): 66 instructions an element, issue slots 75 % busy, four
// blocks a multiprocessor; seeded 802 us: 108 instructions, 72 %, three blocks.
// With a master copy and fp32 gradients 1008 and 1164 us.  Their moments in
// fp32 317 us (6.3 TB/s).
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "expert_internal.cuh"

namespace gmm {
namespace {

constexpr int kBlockElems = 256;   // elements of one scale, and of one warp's turn
constexpr int kWarps = 8;
constexpr int kMaxTurns = 16;       // consecutive turns of a warp in one tensor
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
  int32_t first;     // the tensor's first chunk in this launch (kWarps x turns of 256 elements)
  int32_t index;     // the tensor's place in the caller's list
  int8_t pt, gt;     // gmm_dtype
  int8_t wide;       // every array aligned for eight-element accesses
  int8_t pad;
};

struct AdamwConst {
  float gs, b1, c1, b2, c2, root, eps, decay, rate;
  int count, chunks, turns;
  int eps_covers;    // eps is far above the root of a subnormal
  int seeded;        // 8 bits: codes by random numbers of (step, tensor, element)
  const int32_t* skip;
  // a step counted on the device: taken so far (NULL: root and rate are there)
  const int64_t* steps;
  int64_t number;    // of this step
  double lr, beta1, beta2;
};

template <int COUNT>
struct AdamwTable {
  AdamwConst k;
  AdamwEntry e[COUNT];
};

// The eight elements a lane has of its warp's 256: consecutive ones where the
// moments are bytes, two fours where they are floats, so that a warp's
// accesses are whole lines either way.
template <int BITS>
__device__ __forceinline__ int lane_elem(int j) {
  const int lane = threadIdx.x & 31;
  return BITS == 8 ? lane * 8 + j : (j >> 2) * 128 + lane * 4 + (j & 3);
}

// Eight elements as they lie in memory: 4 words of 16-bit ones, 8 of floats.
template <bool HALF> struct Raw { uint32_t w[HALF ? 4 : 8]; };

// `i`: first element of the warp's 256; `left` of them are the tensor's, and
// where all are (`full`, which asks for aligned arrays) the accesses are wide.
template <int BITS, bool HALF>
__device__ __forceinline__ void fetch(Raw<HALF>& r, const void* base, int64_t i, int left, bool full) {
  const int lane = threadIdx.x & 31;
  if (full) {
    if constexpr (HALF && BITS == 8) {
      const uint4 a = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i)[lane];
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    } else if constexpr (HALF) {
      const uint2* p = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
      const uint2 a = p[lane], b = p[lane + 32];
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = b.x; r.w[3] = b.y;
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
      const uint4 a = p[BITS == 8 ? 2 * lane : lane], b = p[BITS == 8 ? 2 * lane + 1 : lane + 32];
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
      r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < (HALF ? 4 : 8); ++j) r.w[j] = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int x = lane_elem<BITS>(j);
    if (x < left) {
      if (HALF) r.w[j / 2] |= (uint32_t)static_cast<const uint16_t*>(base)[i + x] << (16 * (j & 1));
      else r.w[j] = static_cast<const uint32_t*>(base)[i + x];
    }
  }
}

template <int BITS, bool HALF>
__device__ __forceinline__ void put(const Raw<HALF>& r, void* base, int64_t i, int left, bool full) {
  const int lane = threadIdx.x & 31;
  if (full) {
    if constexpr (HALF && BITS == 8) {
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i)[lane] =
          make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else if constexpr (HALF) {
      uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i);
      p[lane] = make_uint2(r.w[0], r.w[1]);
      p[lane + 32] = make_uint2(r.w[2], r.w[3]);
    } else {
      uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(base) + i);
      p[BITS == 8 ? 2 * lane : lane] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
      p[BITS == 8 ? 2 * lane + 1 : lane + 32] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int x = lane_elem<BITS>(j);
    if (x < left) {
      if (HALF) static_cast<uint16_t*>(base)[i + x] = (uint16_t)(r.w[j / 2] >> (16 * (j & 1)));
      else static_cast<uint32_t*>(base)[i + x] = r.w[j];
    }
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

template <int BITS>
__device__ __forceinline__ void put_float(const float* x, float* base, int64_t i, int left, bool full) {
  Raw<false> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.w[j] = __float_as_uint(x[j]);
  put<BITS, false>(r, base, i, left, full);
}
template <int BITS>
__device__ __forceinline__ void put_param(const float* x, int type, void* base, int64_t i, int left,
                                          bool full) {
  if (type == GMM_F32) return put_float<BITS>(x, static_cast<float*>(base), i, left, full);
  Raw<true> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (type == GMM_F16) {
      const __half2 h = __halves2half2(__float2half_rn(x[2 * j]), __float2half_rn(x[2 * j + 1]));
      r.w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
      r.w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  put<BITS, true>(r, base, i, left, full);
}

// Eight 8-bit codes as two words.
__device__ __forceinline__ uint2 fetch_codes(const void* base, int64_t i, int left, bool full) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  const int x = lane_elem<8>(0);
  if (full) return reinterpret_cast<const uint2*>(p)[threadIdx.x & 31];
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (x + j < left) w[j >> 2] |= (uint32_t)p[x + j] << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(void* base, int64_t i, int left, bool full, uint2 c) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  const int x = lane_elem<8>(0);
  if (full) {
    reinterpret_cast<uint2*>(p)[threadIdx.x & 31] = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (x + j < left) p[x + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// The sum of two products, each rounded by itself: packed products and packed
// sums end up as one fused operation, scalar sums do not.
__device__ __forceinline__ float2 sum_rn(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
__device__ __forceinline__ float with_sign(float x, float of) {  // x >= 0
  return __uint_as_float(__float_as_uint(x) | (__float_as_uint(of) & 0x80000000u));
}

// Byte J of a word as the float 2^23 + byte.
template <int J>
__device__ __forceinline__ float code_bits(uint32_t w) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | J));
}
// Four codes as floats (unsigned, or two's complement).
template <bool SIGNED>
__device__ __forceinline__ void code_floats(uint32_t w, float2* f) {
  if (SIGNED) w ^= 0x80808080u;
  const float2 off = both(SIGNED ? -8388736.f : -8388608.f);
  f[0] = add2(make_float2(code_bits<0>(w), code_bits<1>(w)), off);
  f[1] = add2(make_float2(code_bits<2>(w), code_bits<3>(w)), off);
}

// c|c| S
__device__ __forceinline__ void decode_m(uint2 c, float scale, float2* x) {
  code_floats<true>(c.x, x);
  code_floats<true>(c.y, x + 2);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = mul2(make_float2(x[j].x * fabsf(x[j].x), x[j].y * fabsf(x[j].y)), both(scale));
}
// c^2 S
__device__ __forceinline__ void decode_root(uint2 c, float scale, float2* x) {
  code_floats<false>(c.x, x);
  code_floats<false>(c.y, x + 2);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(x[j], x[j]), both(scale));
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

// A near root of value / S is off by less than 2^-22 of itself (twice 2^-23
// for the two roots, half of each product's 2^-24): 6.1e-5 at 255.
constexpr float kNear = 0.5f - 1.5e-4f;
constexpr float kMagic = 12582912.f;  // 1.5 2^23: x + kMagic holds rint(x) in its low bits

// Scale of a block whose largest magnitude is `big`, and its inverse.  A value
// that is not finite has no code: the scale is NaN then, and so is every value
// of the block from there on.
template <int TOP>
__device__ __forceinline__ float2 scale_of(float big) {
  if (big < kTiny) return make_float2(0.f, 0.f);
  if (!(big <= FLT_MAX)) return make_float2(NAN, NAN);
  return make_float2(__fmul_rn(big, (float)(1.0 / (TOP * TOP))),
                     __fmul_rn(__frcp_rn(big), (float)(TOP * TOP)));
}

__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b) {
  const uint32_t x = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
  const uint32_t y = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
  return __byte_perm(x, y, 0x5410);
}
// Codes to be: t + kMagic of eight values; how far the farthest is from its
// whole number.
__device__ __forceinline__ float round_all(float2* t) {
  float far = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 s = t[j];
    t[j] = add2(s, both(kMagic));
    const float2 d = sub2(s, add2(t[j], both(-kMagic)));
    far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
  }
  return far;
}

// Codes of eight m.
__device__ __forceinline__ uint2 encode_m(const float2* m, float inv) {
  float2 t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = mul2(m[j], both(inv));
    t[j].x = with_sign(sqrt_near(fabsf(x.x)), m[j].x);
    t[j].y = with_sign(sqrt_near(fabsf(x.y)), m[j].y);
  }
  if (round_all(t) > kNear) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = mul2(m[j], both(inv));
      t[j].x = with_sign(__fsqrt_rn(fabsf(x.x)), m[j].x) + kMagic;
      t[j].y = with_sign(__fsqrt_rn(fabsf(x.y)), m[j].y) + kMagic;
    }
  }
  return make_uint2(low_bytes(t[0], t[1]), low_bytes(t[2], t[3]));
}

// Whether a byte of w is zero.
__device__ __forceinline__ bool zero_byte(uint32_t w) {
  return ((w - 0x01010101u) & ~w & 0x80808080u) != 0u;
}
// Byte j of w, where it is zero and v is not, becomes 1.
__device__ __forceinline__ uint32_t above_zero(uint32_t w, float2 a, float2 b) {
  const float v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (v[j] > 0.f && !((w >> (8 * j)) & 0xffu)) w |= 1u << (8 * j);
  return w;
}

// Codes of eight sqrt(v); root is near, v exact.  The near root of a
// subnormal is 0, and so is its code unless S is as small; there, and near
// halfway, the root is taken again.
__device__ __forceinline__ uint2 encode_root(const float2* v, const float2* root, float inv) {
  float2 t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = mul2(root[j], both(inv));
    t[j].x = sqrt_near(x.x);
    t[j].y = sqrt_near(x.y);
  }
  if (round_all(t) > kNear || inv > 1e18f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[j].x = __fsqrt_rn(__fmul_rn(__fsqrt_rn(v[j].x), inv)) + kMagic;
      t[j].y = __fsqrt_rn(__fmul_rn(__fsqrt_rn(v[j].y), inv)) + kMagic;
    }
  }
  uint32_t a = low_bytes(t[0], t[1]), b = low_bytes(t[2], t[3]);
  if (zero_byte(a)) a = above_zero(a, v[0], v[1]);
  if (zero_byte(b)) b = above_zero(b, v[2], v[3]);
  return make_uint2(a, b);
}

// The larger of two values, NaN where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Sixteen random bits for each of eight values: Philox4x32 with ten rounds
// (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011), a function of the counter and the key alone.
__device__ __forceinline__ uint4 philox(uint4 c, uint2 key) {
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint32_t h0 = __umulhi(0xD2511F53u, c.x), l0 = 0xD2511F53u * c.x;
    const uint32_t h1 = __umulhi(0xCD9E8D57u, c.z), l1 = 0xCD9E8D57u * c.z;
    c = make_uint4(h1 ^ c.y ^ key.x, l1, h0 ^ c.w ^ key.y, l0);
    key.x += 0x9E3779B9u;
    key.y += 0xBB67AE85u;
  }
  return c;
}

// Seeded codes of eight values: the next code up with the probability that
// makes the held value's expectation the value itself, so that an average that
// moves by less than a code a step still moves at its own rate.  x = value / S
// lies between c^2 and (c + 1)^2; the value held is linear in c^2 for m, and
// for v, whose root is held, v is linear in c^4.  `which` 0: m, 1: v.
template <int TOP, bool SQUARE>
__device__ __forceinline__ void seeded_codes(const float* x, const AdamwConst& k, const AdamwEntry& e,
                                             int64_t block, float* code) {
  const uint64_t unit = (uint64_t)block * 32 + (threadIdx.x & 31);
  const uint4 r = philox(make_uint4((uint32_t)unit, (uint32_t)(unit >> 32), (uint32_t)e.index, SQUARE),
                         make_uint2((uint32_t)k.number, (uint32_t)((uint64_t)k.number >> 32)));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = ((float)((w[j >> 1] >> (16 * (j & 1))) & 0xffffu) + 0.5f) * (1.f / 65536.f);
    const float c = floorf(sqrt_near(x[j])), c2 = c * c, step = 2.f * c + 1.f;
    const bool up = SQUARE ? u * step * (2.f * c2 + step) < (x[j] - c2) * (x[j] + c2) : u * step < x[j] - c2;
    code[j] = fminf(up ? c + 1.f : c, (float)TOP);
  }
}
__device__ __forceinline__ uint2 seeded_m(const float2* m, float inv, const AdamwConst& k,
                                          const AdamwEntry& e, int64_t block) {
  float x[8], c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(fabsf(j & 1 ? m[j >> 1].y : m[j >> 1].x), inv);
  seeded_codes<127, false>(x, k, e, block, c);
  float2 t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    t[j] = make_float2(with_sign(c[2 * j], m[j].x) + kMagic, with_sign(c[2 * j + 1], m[j].y) + kMagic);
  return make_uint2(low_bytes(t[0], t[1]), low_bytes(t[2], t[3]));
}
// v > 0 keeps a code above zero, as in encode_root; where S is as small as the
// root of a subnormal the roots are taken again.
__device__ __forceinline__ uint2 seeded_root(const float2* v, const float2* root, float inv,
                                             const AdamwConst& k, const AdamwEntry& e, int64_t block) {
  float x[8], c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float r = j & 1 ? root[j >> 1].y : root[j >> 1].x;
    if (inv > 1e18f) r = __fsqrt_rn(j & 1 ? v[j >> 1].y : v[j >> 1].x);
    x[j] = __fmul_rn(r, inv);
  }
  seeded_codes<255, true>(x, k, e, block, c);
  float2 t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    t[j].x = (v[j].x > 0.f ? fmaxf(c[2 * j], 1.f) : c[2 * j]) + kMagic;
    t[j].y = (v[j].y > 0.f ? fmaxf(c[2 * j + 1], 1.f) : c[2 * j + 1]) + kMagic;
  }
  return make_uint2(low_bytes(t[0], t[1]), low_bytes(t[2], t[3]));
}

// Largest of the warp's non-negative values (their bits order them, NaN last).
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

// Where a warp is in a tensor: 256 elements, `left` of them the tensor's.
struct Place {
  int left;
  bool full;
  int64_t block;
};
__device__ __forceinline__ Place place_of(const AdamwEntry& e, int64_t block) {
  Place p;
  p.block = block;
  const int64_t left = e.n - block * kBlockElems;
  p.left = left > kBlockElems ? kBlockElems : left < 0 ? 0 : (int)left;
  p.full = e.wide && p.left == kBlockElems;
  return p;
}

template <int BITS, bool PH, bool GH> struct Operands {
  Raw<PH> p;
  Raw<GH> g;
  Raw<false> m, v;   // 8 bits: two words of codes each
  float ms, vs;
};

template <int BITS, bool PH, bool GH>
__device__ __forceinline__ void fetch_all(Operands<BITS, PH, GH>& o, const AdamwEntry& e, const Place& q) {
  const int64_t i = q.block * kBlockElems;
  fetch<BITS, GH>(o.g, e.g, i, q.left, q.full);
  fetch<BITS, PH>(o.p, e.master ? (const void*)e.master : e.p, i, q.left, q.full);
  if constexpr (BITS == 32) {
    fetch<BITS, false>(o.m, e.m, i, q.left, q.full);
    fetch<BITS, false>(o.v, e.v, i, q.left, q.full);
  } else {
    const uint2 mc = fetch_codes(e.m, i, q.left, q.full), vc = fetch_codes(e.v, i, q.left, q.full);
    o.m.w[0] = mc.x; o.m.w[1] = mc.y;
    o.v.w[0] = vc.x; o.v.w[1] = vc.y;
    o.ms = e.ms[q.block];
    o.vs = e.vs[q.block];
  }
}

// fp32 moments: the documented operations, one by one.
template <bool MORE, bool PH, bool GH>
__device__ __forceinline__ void step_block(const AdamwConst& k, const AdamwEntry& e, const Place& q,
                                           const Operands<32, PH, GH>& o) {
  float g[8], p[8], m[8], v[8];
  widen<GH>(o.g, e.gt, g);
  widen<PH>(o.p, e.pt, p);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = __fmul_rn(g[j], k.gs);
    m[j] = __fadd_rn(__fmul_rn(__uint_as_float(o.m.w[j]), k.b1), __fmul_rn(gj, k.c1));
    v[j] = __fadd_rn(__fmul_rn(__uint_as_float(o.v.w[j]), k.b2), __fmul_rn(__fmul_rn(gj, gj), k.c2));
    const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v[j]), k.root), k.eps);
    p[j] = __fsub_rn(__fmul_rn(p[j], k.decay), __fdiv_rn(__fmul_rn(m[j], k.rate), den));
  }
  const int64_t i = q.block * kBlockElems;
  if (e.master) put_float<32>(p, e.master, i, q.left, q.full);
  put_param<32>(p, e.pt, e.p, i, q.left, q.full);
  put_float<32>(m, static_cast<float*>(e.m), i, q.left, q.full);
  put_float<32>(v, static_cast<float*>(e.v), i, q.left, q.full);
}

// 8-bit moments: pairs of elements, each half rounded as one by one.
template <bool MORE, bool PH, bool GH>
__device__ __forceinline__ void step_block(const AdamwConst& k, const AdamwEntry& e, const Place& q,
                                           const Operands<8, PH, GH>& o) {
  float g[8], p[8];
  widen<GH>(o.g, e.gt, g);
  widen<PH>(o.p, e.pt, p);
  float2 m[4], v[4], root[4];
  decode_m(make_uint2(o.m.w[0], o.m.w[1]), o.ms, m);
  decode_root(make_uint2(o.v.w[0], o.v.w[1]), o.vs, root);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 gj = mul2(make_float2(g[2 * j], g[2 * j + 1]), both(k.gs));
    m[j] = sum_rn(mul2(m[j], both(k.b1)), mul2(gj, both(k.c1)));
    v[j] = sum_rn(mul2(mul2(root[j], root[j]), both(k.b2)), mul2(mul2(gj, gj), both(k.c2)));
    root[j] = make_float2(sqrt_near(v[j].x), sqrt_near(v[j].y));
    const float2 den = fma2(root[j], both(k.root), both(k.eps));
    float2 r = make_float2(rcp_near(den.x), rcp_near(den.y));
    if (!k.eps_covers) {  // a subnormal v's root, flushed to 0 above, may count
      r.x = __fdiv_rn(1.f, fmaf(__fsqrt_rn(v[j].x), k.root, k.eps));
      r.y = __fdiv_rn(1.f, fmaf(__fsqrt_rn(v[j].y), k.root, k.eps));
    }
    const float2 pj = mul2(make_float2(p[2 * j], p[2 * j + 1]), both(k.decay));
    const float2 up = mul2(mul2(m[j], both(k.rate)), r);
    p[2 * j] = __fsub_rn(pj.x, up.x);
    p[2 * j + 1] = __fsub_rn(pj.y, up.y);
  }
  const int64_t i = q.block * kBlockElems;
  if (e.master) put_float<8>(p, e.master, i, q.left, q.full);
  put_param<8>(p, e.pt, e.p, i, q.left, q.full);
  if (!q.full) {  // nothing past the end
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (lane_elem<8>(2 * j) >= q.left) m[j].x = v[j].x = root[j].x = 0.f;
      if (lane_elem<8>(2 * j + 1) >= q.left) m[j].y = v[j].y = root[j].y = 0.f;
    }
  }
  float mb = 0.f, vb = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    mb = max_nan(mb, max_nan(fabsf(m[j].x), fabsf(m[j].y)));
    vb = max_nan(vb, max_nan(v[j].x, v[j].y));
  }
  const float2 ms = scale_of<127>(warp_max_pos(mb));
  const float2 vs = scale_of<255>(__fsqrt_rn(warp_max_pos(vb)));
  if (MORE && k.seeded) {
    put_codes(e.m, i, q.left, q.full, seeded_m(m, ms.y, k, e, q.block));
    put_codes(e.v, i, q.left, q.full, seeded_root(v, root, vs.y, k, e, q.block));
  } else {
    put_codes(e.m, i, q.left, q.full, encode_m(m, ms.y));
    put_codes(e.v, i, q.left, q.full, encode_root(v, root, vs.y));
  }
  if ((threadIdx.x & 31) == 0) {
    e.ms[q.block] = ms.x;
    e.vs[q.block] = vs.x;
  }
}

// The odd blocks: a tensor's end, or arrays that are not aligned.
template <int BITS, bool PH, bool GH, bool MORE>
__device__ __noinline__ void odd_block(const AdamwConst& k, const AdamwEntry& e, int64_t block) {
  const Place q = place_of(e, block);
  if (q.left == 0) return;
  Operands<BITS, PH, GH> o;
  fetch_all(o, e, q);
  step_block<MORE>(k, e, q, o);
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A lane's operands of a full block in 8 bits, on their way through shared
// memory: kAhead turns are in flight without holding registers.  A lane reads
// back only what it copied, so no barrier is needed.
constexpr int kAhead = 3;
template <bool PH, bool GH>
__host__ __device__ constexpr int stage_bytes() { return (GH ? 512 : 1024) + (PH ? 512 : 1024) + 512; }
template <bool PH, bool GH>
constexpr size_t ring_bytes() { return (size_t)kWarps * (kAhead + 1) * stage_bytes<PH, GH>(); }

template <bool PH, bool GH>
__device__ __forceinline__ void stage_copy(uint8_t* st, const AdamwEntry& e, int64_t i) {
  const int lane = threadIdx.x & 31;
  const char* g = static_cast<const char*>(e.g) + i * (GH ? 2 : 4);
  const char* p = (e.master ? reinterpret_cast<const char*>(e.master) : static_cast<const char*>(e.p)) + i * (PH ? 2 : 4);
#pragma unroll
  for (int x = 0; x < (GH ? 1 : 2); ++x)
    copy_async16(st + x * 512 + lane * 16, g + (GH ? lane * 16 : lane * 32 + x * 16));
  st += GH ? 512 : 1024;
#pragma unroll
  for (int x = 0; x < (PH ? 1 : 2); ++x)
    copy_async16(st + x * 512 + lane * 16, p + (PH ? lane * 16 : lane * 32 + x * 16));
  st += PH ? 512 : 1024;
  copy_async8(st + lane * 8, static_cast<const uint8_t*>(e.m) + i + lane * 8);
  copy_async8(st + 256 + lane * 8, static_cast<const uint8_t*>(e.v) + i + lane * 8);
}

template <bool PH, bool GH>
__device__ __forceinline__ void stage_read(Operands<8, PH, GH>& o, const uint8_t* st) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 0; x < (GH ? 1 : 2); ++x) {
    const uint4 a = *reinterpret_cast<const uint4*>(st + x * 512 + lane * 16);
    o.g.w[4 * x] = a.x; o.g.w[4 * x + 1] = a.y; o.g.w[4 * x + 2] = a.z; o.g.w[4 * x + 3] = a.w;
  }
  st += GH ? 512 : 1024;
#pragma unroll
  for (int x = 0; x < (PH ? 1 : 2); ++x) {
    const uint4 a = *reinterpret_cast<const uint4*>(st + x * 512 + lane * 16);
    o.p.w[4 * x] = a.x; o.p.w[4 * x + 1] = a.y; o.p.w[4 * x + 2] = a.z; o.p.w[4 * x + 3] = a.w;
  }
  st += PH ? 512 : 1024;
  const uint2 m = *reinterpret_cast<const uint2*>(st + lane * 8);
  const uint2 v = *reinterpret_cast<const uint2*>(st + 256 + lane * 8);
  o.m.w[0] = m.x; o.m.w[1] = m.y;
  o.v.w[0] = v.x; o.v.w[1] = v.y;
}

// The full blocks of a warp's turns in one chunk; returns how many it did.
template <bool MORE, bool PH, bool GH>
__device__ __forceinline__ int full_turns(const AdamwConst& k, const AdamwEntry& e, int64_t block,
                                          uint8_t* ring, std::integral_constant<int, 8>) {
  constexpr int B = stage_bytes<PH, GH>();
  const int64_t fulls = e.wide ? e.n / kBlockElems : 0;  // full blocks of the tensor
  const int64_t room = (fulls - block + kWarps - 1) / kWarps;
  const int turns = room < 0 ? 0 : (int)min((int64_t)k.turns, room);
  if (turns == 0) return 0;
#pragma unroll
  for (int x = 0; x < kAhead; ++x) {
    if (x < turns) stage_copy<PH, GH>(ring + x * B, e, (block + x * kWarps) * kBlockElems);
    copy_commit();
  }
  float ms = e.ms[block], vs = e.vs[block];
  int slot = 0, ahead = kAhead;
  for (int turn = 0; turn < turns; ++turn, block += kWarps) {
    if (turn + kAhead < turns)
      stage_copy<PH, GH>(ring + ahead * B, e, (block + kAhead * kWarps) * kBlockElems);
    copy_commit();
    Operands<8, PH, GH> o;
    o.ms = ms;
    o.vs = vs;
    if (turn + 1 < turns) {
      ms = e.ms[block + kWarps];
      vs = e.vs[block + kWarps];
    }
    copy_wait<kAhead>();
    stage_read(o, ring + slot * B);
    step_block<MORE>(k, e, Place{kBlockElems, true, block}, o);
    slot = slot == kAhead ? 0 : slot + 1;
    ahead = ahead == kAhead ? 0 : ahead + 1;
  }
  return turns;
}

// fp32 moments: a turn's operands are fetched into registers a turn ahead.
template <bool MORE, bool PH, bool GH>
__device__ __forceinline__ int full_turns(const AdamwConst& k, const AdamwEntry& e, int64_t block,
                                          uint8_t*, std::integral_constant<int, 32>) {
  const int64_t fulls = e.wide ? e.n / kBlockElems : 0;
  const int64_t room = (fulls - block + kWarps - 1) / kWarps;
  const int turns = room < 0 ? 0 : (int)min((int64_t)k.turns, room);
  if (turns == 0) return 0;
  Operands<32, PH, GH> o;
  fetch_all(o, e, Place{kBlockElems, true, block});
  for (int turn = 0; turn < turns; ++turn, block += kWarps) {
    Operands<32, PH, GH> next;
    if (turn + 1 < turns) fetch_all(next, e, Place{kBlockElems, true, block + kWarps});
    step_block<MORE>(k, e, Place{kBlockElems, true, block}, o);
    o = next;
  }
  return turns;
}

// The number of a step that is counted on the device, and both bias
// corrections by one thread.
__device__ __forceinline__ void correct_by_count(AdamwConst& k) {
  __shared__ float at[2];
  const int64_t taken = *k.steps;
  k.number = (taken < 0 ? 0 : taken) + 1;
  if (threadIdx.x == 0) {
    const double n = (double)k.number;
    at[0] = (float)pow(1.0 - pow(k.beta2, n), -0.5);
    at[1] = (float)(k.lr / (1.0 - pow(k.beta1, n)));
  }
  __syncthreads();
  k.root = at[0];
  k.rate = at[1];
}

// PH, GH: 16-bit parameters (no master) and gradients.  MORE: the step may be
// counted on the device, and codes may be seeded.  That is a kernel of its own,
// since what it computes takes registers that the 8-bit step lacks.
template <bool MORE> using ConstOf = std::conditional_t<MORE, AdamwConst, const AdamwConst&>;
template <int BITS, bool PH, bool GH, bool MORE, int COUNT>
__global__ void __launch_bounds__(kWarps * 32, BITS == 8 ? (MORE ? 3 : 4) : 2)
adamw_kernel(const __grid_constant__ AdamwTable<COUNT> t) {
  extern __shared__ __align__(16) uint8_t rings[];
  ConstOf<MORE> k = t.k;
  if (k.skip && *k.skip != 0) return;
  if constexpr (MORE) {
    if (k.steps) correct_by_count(k);
  }
  const int warp = threadIdx.x >> 5;
  uint8_t* ring = rings + warp * (kAhead + 1) * stage_bytes<PH, GH>();
  const int c0 = (int)((int64_t)k.chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)k.chunks * (blockIdx.x + 1) / gridDim.x);
  if (c0 >= c1) return;
  int at = tensor_of(t, c0);
  for (int c = c0; c < c1; ++c) {
    while (at + 1 < k.count && t.e[at + 1].first <= c) ++at;
    const AdamwEntry e = t.e[at];
    const int64_t block = (int64_t)(c - e.first) * kWarps * k.turns + warp;
    for (int turn = full_turns<MORE, PH, GH>(k, e, block, ring, std::integral_constant<int, BITS>());
         turn < k.turns; ++turn)
      odd_block<BITS, PH, GH, MORE>(k, t.e[at], block + turn * kWarps);
  }
}

// Moments in fp32: entry.p and entry.master are the outputs here.  Bytes are
// read a word at a time, so that the floats are written as whole lines.
template <int BITS>
__device__ __forceinline__ void moments_block(const AdamwEntry& e, const Place& q) {
  const int lane = threadIdx.x & 31;
  const int64_t i = q.block * kBlockElems;
  float x[8], y[8];
  if (BITS == 32) {
    Raw<false> r;
    fetch<32, false>(r, e.m, i, q.left, q.full);
    widen<false>(r, GMM_F32, x);
    fetch<32, false>(r, e.v, i, q.left, q.full);
    widen<false>(r, GMM_F32, y);
  } else {
    uint2 mc, vc;
    if (q.full) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.m) + i);
      mc = make_uint2(p[lane], p[lane + 32]);
      p = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.v) + i);
      vc = make_uint2(p[lane], p[lane + 32]);
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int z = lane_elem<32>(j);
        if (z < q.left) {
          w[j >> 2] |= (uint32_t)static_cast<const uint8_t*>(e.m)[i + z] << (8 * (j & 3));
          w[2 + (j >> 2)] |= (uint32_t)static_cast<const uint8_t*>(e.v)[i + z] << (8 * (j & 3));
        }
      }
      mc = make_uint2(w[0], w[1]);
      vc = make_uint2(w[2], w[3]);
    }
    float2 m[4], v[4];
    decode_m(mc, e.ms[q.block], m);
    decode_root(vc, e.vs[q.block], v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 s = mul2(v[j], v[j]);
      x[2 * j] = m[j].x; x[2 * j + 1] = m[j].y;
      y[2 * j] = s.x; y[2 * j + 1] = s.y;
    }
  }
  put_float<32>(x, static_cast<float*>(e.p), i, q.left, q.full);
  put_float<32>(y, e.master, i, q.left, q.full);
}

template <int BITS, int COUNT>
__global__ void __launch_bounds__(kWarps * 32)
adamw_moments_kernel(const __grid_constant__ AdamwTable<COUNT> t) {
  const AdamwConst& k = t.k;
  const int c0 = (int)((int64_t)k.chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)k.chunks * (blockIdx.x + 1) / gridDim.x);
  if (c0 >= c1) return;
  int at = tensor_of(t, c0);
  for (int c = c0; c < c1; ++c) {
    while (at + 1 < k.count && t.e[at + 1].first <= c) ++at;
    const AdamwEntry e = t.e[at];
    const int64_t block = (int64_t)(c - e.first) * kWarps * k.turns + (threadIdx.x >> 5);
    const Place last = place_of(e, block + (k.turns - 1) * kWarps);
    if (last.full) {
#pragma unroll 4
      for (int turn = 0; turn < k.turns; ++turn) {
        Place q{kBlockElems, true, block + turn * kWarps};
        moments_block<BITS>(e, q);
      }
    } else {
      for (int turn = 0; turn < k.turns; ++turn) {
        const Place q = place_of(e, block + turn * kWarps);
        if (q.left > 0) moments_block<BITS>(e, q);
      }
    }
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

// Turns of a warp in one chunk: enough chunks for every warp of two blocks a
// multiprocessor, then up to kMaxTurns (the table is read once a chunk).
int turns_for(const gmm_adamw_tensor* ts, int count) {
  int64_t n = 0;
  for (int i = 0; i < count; ++i) n += ts[i].n;
  const int64_t t = n / ((int64_t)kBlockElems * kWarps * 304);
  return t < 1 ? 1 : t > kMaxTurns ? kMaxTurns : (int)t;
}

// Launches over the non-empty tensors that `take` wants, as many at a time as
// a table holds (and as 2^30 chunks).
template <int COUNT, typename Take, typename Fill, typename Go>
gmm_status over_tables(const gmm_adamw_tensor* ts, int count, const AdamwConst& k, Take take,
                       Fill fill, Go go) {
  AdamwTable<COUNT> t;
  t.k = k;
  t.k.turns = turns_for(ts, count);
  t.k.count = 0;
  int64_t chunks = 0;
  for (int i = 0; i <= count; ++i) {
    const bool end = i == count;
    const int64_t chunk = (int64_t)kBlockElems * kWarps * t.k.turns;
    const int64_t c = end || !take(i) ? 0 : (ts[i].n + chunk - 1) / chunk;
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
// Blocks: one a chunk, up to `most` a multiprocessor, each a contiguous
// stretch of the list.  The step in 8 bits, which computes as much as it
// waits, has the four that are resident (2e8 elements: 467 us; with 8 488 us);
// what waits for memory alone several waves of smaller stretches (the step in
// fp32, 1e8 elements: 422 us with 16, 441 with 2; moments from 8 bits, 2e8:
// 317 us with 24, 340 with 4 or 12).
unsigned grid_for(int chunks, int most) { return (unsigned)(chunks < 152 * most ? chunks : 152 * most); }

template <int BITS, bool PH, bool GH, bool MORE, int COUNT>
void launch_step(const AdamwTable<COUNT>& t, cudaStream_t s) {
  const size_t smem = BITS == 8 ? ring_bytes<PH, GH>() : 0;
  static std::atomic<uint64_t> allowed;
  const auto kernel = adamw_kernel<BITS, PH, GH, MORE, COUNT>;
  // what the kernel has of its own counts too: 48 KB of rings may be too much
  if (smem > 0 && !allow_smem((const void*)kernel, smem, allowed)) return;
  kernel<<<grid_for(t.k.chunks, BITS == 8 ? (MORE ? 3 : 4) : 16), kWarps * 32, smem, s>>>(t);
}

__global__ void count_step_kernel(int64_t* steps) { *steps = (*steps < 0 ? 0 : *steps) + 1; }

// steps: of a step that is counted on the device, or NULL.
gmm_status adamw_step(const gmm_adamw_tensor* ts, int count, const gmm_adamw_opts* o, int64_t* steps,
                      void* stream) {
  if (!o || !tensors_ok(ts, count, o->state_bits, true)) return GMM_ERR_INVALID_ARG;
  if (o->rounding != 0 && o->rounding != 1) return GMM_ERR_INVALID_ARG;
  if ((!steps && o->step < 1) || !(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) ||
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
  if (steps) {
    k.steps = steps;
    k.lr = o->lr;
    k.beta1 = o->beta1;
    k.beta2 = o->beta2;
  } else {
    k.root = (float)std::pow(1.0 - std::pow(o->beta2, (double)o->step), -0.5);
    k.rate = (float)(o->lr / (1.0 - std::pow(o->beta1, (double)o->step)));
  }
  k.eps = (float)o->eps;
  k.decay = (float)(1.0 - o->lr * o->weight_decay);
  k.skip = o->skip;
  k.eps_covers = o->eps >= 1e-10;
  const int bits = o->state_bits;
  k.number = o->step;
  k.seeded = bits == 8 && o->rounding == 1;
  const bool more = steps != nullptr || k.seeded;
  auto fill = [&](int i, AdamwEntry& e) {
    const gmm_adamw_tensor& t = ts[i];
    e.p = t.param; e.g = t.grad; e.master = t.master; e.m = t.m; e.v = t.v;
    e.ms = t.m_scale; e.vs = t.v_scale;
    e.index = i;
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
#define GMM_GO(B, M)                                  \
  if (ph && gh) launch_step<B, true, true, M>(t, s);   \
  else if (ph) launch_step<B, true, false, M>(t, s);   \
  else if (gh) launch_step<B, false, true, M>(t, s);   \
  else launch_step<B, false, false, M>(t, s);
      if (more) {
        if (bits == 32) { GMM_GO(32, true) } else { GMM_GO(8, true) }
      } else {
        if (bits == 32) { GMM_GO(32, false) } else { GMM_GO(8, false) }
      }
#undef GMM_GO
    };
    const gmm_status r = count <= kSmallTable ? over_tables<kSmallTable>(ts, count, k, take, fill, go)
                                              : over_tables<kTable>(ts, count, k, take, fill, go);
    if (r != GMM_OK) return r;
  }
  if (!steps) return GMM_OK;
  count_step_kernel<<<1, 1, 0, s>>>(steps);
  return launched();
}

}  // namespace
}  // namespace gmm

using namespace gmm;

extern "C" {

gmm_status gmm_adamw_step(const gmm_adamw_tensor* ts, int count, const gmm_adamw_opts* o,
                          void* stream) {
  return adamw_step(ts, count, o, nullptr, stream);
}

gmm_status gmm_adamw_step_counted(const gmm_adamw_tensor* ts, int count, const gmm_adamw_opts* o,
                                  int64_t* steps, void* stream) {
  if (!steps || (uintptr_t)steps % 8) return GMM_ERR_INVALID_ARG;
  return adamw_step(ts, count, o, steps, stream);
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
    if (state_bits == 32) adamw_moments_kernel<32, C><<<grid_for(t.k.chunks, 24), kWarps * 32, 0, s>>>(t);
    else adamw_moments_kernel<8, C><<<grid_for(t.k.chunks, 24), kWarps * 32, 0, s>>>(t);
  };
  auto all = [](int) { return true; };
  return count <= kSmallTable ? over_tables<kSmallTable>(ts, count, AdamwConst{}, all, fill, go)
                              : over_tables<kTable>(ts, count, AdamwConst{}, all, fill, go);
}

}  // extern "C"
