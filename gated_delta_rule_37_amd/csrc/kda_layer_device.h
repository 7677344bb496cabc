// Device helpers of the operators around the recurrence: typed loads and
// stores of a few neighbouring elements as FP32, sums over lane groups.
#ifndef KDA_LAYER_DEVICE_H_
#define KDA_LAYER_DEVICE_H_

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_device.h"

namespace kda {

// Element storage: FP32 or the raw bits of a bf16.
typedef float fp32_t;
typedef uint16_t bf16_t;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Vectors at any address that suits their elements (the hardware reads and
// writes them whole; aligned ones cost nothing extra).
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// One aligned vector; STREAM: past the caches, which pays where a call's
// tensors are larger than the 256 MB last-level cache (kStreamBytes) and costs
// where the next launch finds them there.
template <bool STREAM, typename V>
__device__ __forceinline__ V fetch(const V* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  return *p;
}
template <bool STREAM, typename V>
__device__ __forceinline__ void put(V* p, V v) {
  if constexpr (STREAM) {
    __builtin_nontemporal_store(v, p);
  } else {
    *p = v;
  }
}
// The same at any address; with STREAM it is an aligned one.
template <bool STREAM>
__device__ __forceinline__ u32x2 fetch4(const bf16_t* p) {
  if constexpr (STREAM) return fetch<true>(reinterpret_cast<const u32x2*>(p));
  return *reinterpret_cast<const u32x2_any*>(p);
}
template <bool STREAM>
__device__ __forceinline__ f32x4 fetch4(const fp32_t* p) {
  if constexpr (STREAM) return fetch<true>(reinterpret_cast<const f32x4*>(p));
  return *reinterpret_cast<const f32x4_any*>(p);
}
template <bool STREAM>
__device__ __forceinline__ void put4(bf16_t* p, u32x2 v) {
  if constexpr (STREAM) {
    put<true>(reinterpret_cast<u32x2*>(p), v);
  } else {
    *reinterpret_cast<u32x2_any*>(p) = v;
  }
}
template <bool STREAM>
__device__ __forceinline__ void put4(fp32_t* p, f32x4 v) {
  if constexpr (STREAM) {
    put<true>(reinterpret_cast<f32x4*>(p), v);
  } else {
    *reinterpret_cast<f32x4_any*>(p) = v;
  }
}

// VEC (1, 4 or 8) neighbouring elements at p as FP32.  With VEC = 8, p is
// aligned to 16 bytes; with VEC = 4 to the element.
template <int VEC, bool STREAM = false>
__device__ __forceinline__ void load(const bf16_t* p, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    const u32x4 w = fetch<STREAM>(reinterpret_cast<const u32x4*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else if constexpr (VEC == 4) {
    const u32x2 w = fetch4<STREAM>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    static_assert(VEC == 1, "");
    x[0] = bf2f(*p);
  }
}
template <int VEC, bool STREAM = false>
__device__ __forceinline__ void load(const fp32_t* p, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    const f32x4 a = fetch<STREAM>(reinterpret_cast<const f32x4*>(p)), b = fetch<STREAM>(reinterpret_cast<const f32x4*>(p + 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  } else if constexpr (VEC == 4) {
    const f32x4 a = fetch4<STREAM>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i];
  } else {
    static_assert(VEC == 1, "");
    x[0] = *p;
  }
}

// Eight elements at any address.
__device__ __forceinline__ void load8_any(const bf16_t* p, float (&x)[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8_any(const fp32_t* p, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = a[i];
    x[4 + i] = b[i];
  }
}
__device__ __forceinline__ void store8_any(bf16_t* p, const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<u32x4_any*>(p) = w;
}
__device__ __forceinline__ void store8_any(fp32_t* p, const float (&x)[8]) {
  const f32x4 a = {x[0], x[1], x[2], x[3]}, b = {x[4], x[5], x[6], x[7]};
  *reinterpret_cast<f32x4_any*>(p) = a;
  *reinterpret_cast<f32x4_any*>(p + 4) = b;
}

// The same, rounded to nearest even for bf16.
template <int VEC, bool STREAM = false>
__device__ __forceinline__ void store(bf16_t* p, const float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    put<STREAM>(reinterpret_cast<u32x4*>(p), w);
  } else if constexpr (VEC == 4) {
    u32x2 w;
    w[0] = pack_bf16(x[0], x[1]);
    w[1] = pack_bf16(x[2], x[3]);
    put4<STREAM>(p, w);
  } else {
    *p = static_cast<uint16_t>(pack_bf16(x[0], 0.f));
  }
}
template <int VEC, bool STREAM = false>
__device__ __forceinline__ void store(fp32_t* p, const float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    f32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = x[i];
      b[i] = x[4 + i];
    }
    put<STREAM>(reinterpret_cast<f32x4*>(p), a);
    put<STREAM>(reinterpret_cast<f32x4*>(p + 4), b);
  } else if constexpr (VEC == 4) {
    f32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = x[i];
    put4<STREAM>(p, a);
  } else {
    *p = x[0];
  }
}

// Sum over the 16 lanes of a DPP row, the same bits in each lane (rotations
// by 8, 4, 2 and 1 add the same pairs everywhere).
template <int N>
__device__ __forceinline__ float row_rotate(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float x) {
  x += row_rotate<8>(x);
  x += row_rotate<4>(x);
  x += row_rotate<2>(x);
  x += row_rotate<1>(x);
  return x;
}
__device__ __forceinline__ float sum32(float x) {
  x = sum16(x);
  return x + __shfl_xor(x, 16);
}
__device__ __forceinline__ float sum64(float x) {
  x = sum32(x);
  return x + __shfl_xor(x, 32);
}

// Sum of the rows first, first + 16, ... below `rows` of one column of a
// row-major matrix (p: the column's first element), eight loads in flight.
__device__ __forceinline__ float column_sum(const float* p, int64_t row, int32_t first, int32_t rows) {
  float part[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) part[i] = 0.f;
  int32_t r = first;
  for (; r + 7 * 16 < rows; r += 8 * 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) part[i] += p[(r + i * 16) * row];
  }
  for (; r < rows; r += 16) part[0] += p[r * row];
  return ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.92596299e-08f;   // log2(e) - kLog2e
constexpr float kLn2 = 0.6931471805599453f;

// Raw storage of VEC elements, so that a load can stay in flight unconverted.
template <typename E, int VEC>
struct RawVec {
  E e[VEC];
};
template <>
struct RawVec<bf16_t, 4> {
  u32x2 w;
};
template <>
struct RawVec<fp32_t, 4> {
  f32x4 a;
};
// Makes what follows compute from the raw registers again, instead of keeping
// the values that were computed from them before alive.
__device__ __forceinline__ void forget(RawVec<bf16_t, 1>& r) {
  uint32_t w = r.e[0];
  asm volatile("" : "+v"(w));
  r.e[0] = static_cast<bf16_t>(w);
}
__device__ __forceinline__ void forget(RawVec<fp32_t, 1>& r) { asm volatile("" : "+v"(r.e[0])); }
__device__ __forceinline__ void forget(RawVec<bf16_t, 4>& r) { asm volatile("" : "+v"(r.w)); }
__device__ __forceinline__ void forget(RawVec<fp32_t, 4>& r) { asm volatile("" : "+v"(r.a)); }

template <bool STREAM, typename E>
__device__ __forceinline__ void load_raw(const E* p, RawVec<E, 1>& r) { r.e[0] = fetch<STREAM>(p); }
template <bool STREAM>
__device__ __forceinline__ void load_raw(const bf16_t* p, RawVec<bf16_t, 4>& r) {
  r.w = fetch4<STREAM>(p);
}
template <bool STREAM>
__device__ __forceinline__ void load_raw(const fp32_t* p, RawVec<fp32_t, 4>& r) {
  r.a = fetch4<STREAM>(p);
}
__device__ __forceinline__ float element(const RawVec<bf16_t, 1>& r, int) { return bf2f(r.e[0]); }
__device__ __forceinline__ float element(const RawVec<fp32_t, 1>& r, int) { return r.e[0]; }
__device__ __forceinline__ float element(const RawVec<bf16_t, 4>& r, int i) {
  return __uint_as_float(i % 2 == 0 ? r.w[i / 2] << 16 : r.w[i / 2] & 0xffff0000u);
}
__device__ __forceinline__ float element(const RawVec<fp32_t, 4>& r, int i) { return r.a[i]; }

// 1 - e^g, given a = e^g.  The difference cancels near 0; for |g| < 1/4 the
// Taylor sum to g^6 / 6! replaces it, exact to 2^-24 relative.
__device__ __forceinline__ float one_minus_exp(float g, float a) {
  float s = 1.f / 720.f;
  s = s * g + 1.f / 120.f;
  s = s * g + 1.f / 24.f;
  s = s * g + 1.f / 6.f;
  s = s * g + 0.5f;
  s = s * g + 1.f;
  float near = -g * s;
  asm("" : "+v"(near));   // both sides and a select: cheaper than branching around the sum
  return fabsf(g) < 0.25f ? near : 1.f - a;
}

// e^x by the hardware's 2^p, p = x log2(e); results below 2^-126 are 0.  p is
// rounded, to half a unit of up to 2^7, so the relative error is about 1 + |x|
// units of 2^-24: for results that are stored in bf16.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
// The same for fp32 results, to at most 4 units (2^p itself 2): what p lost, and
// log2(e) itself, is worked in to first order.  Where 2^p is 0, infinite or NaN
// there is nothing to correct.
__device__ __forceinline__ float exact_exp(float x) {
  const float p = x * kLog2e, e = __builtin_amdgcn_exp2f(p);
  const float lost = __fmaf_rn(x, kLog2e, -p) + x * kLog2eLow;
  return fabsf(p) < 128.f ? __fmaf_rn(e, lost * kLn2, e) : e;
}

// sigmoid(z) and sigmoid(-z) = 1 - sigmoid(z), from e^-|z|: each to a few units
// of its own value however small it is, so that a gradient of a saturated gate,
// up * down, is not the 0 that 1 - up rounds to from z = 17 on.
struct Sigmoids {
  float up, down;
};
__device__ __forceinline__ Sigmoids sigmoids(float z) {
  const float t = exact_exp(-fabsf(z)), large = __builtin_amdgcn_rcpf(1.f + t), small = t * large;
  return z < 0.f ? Sigmoids{small, large} : Sigmoids{large, small};
}
__device__ __forceinline__ float sigmoidf(float z) { return __builtin_amdgcn_rcpf(1.f + exact_exp(-z)); }

}  // namespace kda

#endif  // KDA_LAYER_DEVICE_H_
