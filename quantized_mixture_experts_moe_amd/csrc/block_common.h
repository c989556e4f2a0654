// Building blocks of the operators around the experts (fp8 quantizer and
// products, balance loss, norms): loads of eight values, wave and group
// reductions, and the symmetric quantization recipe (not installed).
#pragma once
#include <math.h>

#include "block_internal.h"
#include "quant_common.h"

namespace qmoe {
namespace bk {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Element types of activations: bf16 bits or fp32.
template <bool F32>
struct El {
  typedef uint16_t T;
};
template <>
struct El<true> {
  typedef float T;
};

__device__ inline float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ inline uint16_t f32_bf16(float v) {  // round to nearest even, NaN kept
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ inline uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)f32_bf16(lo) | ((uint32_t)f32_bf16(hi) << 16);
}

template <bool F32>
__device__ inline float load1(const void* p, size_t i) {
  if constexpr (F32)
    return reinterpret_cast<const float*>(p)[i];
  else
    return bf16_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <bool F32>
__device__ inline void store1(void* p, size_t i, float v) {
  if constexpr (F32)
    reinterpret_cast<float*>(p)[i] = v;
  else
    reinterpret_cast<uint16_t*>(p)[i] = f32_bf16(v);
}

// Eight consecutive values at element i (the byte address a multiple of 16).
template <bool F32>
__device__ inline void load8(const void* p, size_t i, float v[8]) {
  if constexpr (F32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[2 * j] = __uint_as_float(a[j] << 16);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  }
}
template <bool F32>
__device__ inline void store8(void* p, size_t i, const float v[8]) {
  if constexpr (F32) {
    f32x4* q = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + i) =
        u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
              pack_bf16(v[6], v[7])};
  }
}

// Four consecutive values (the byte address a multiple of their size).
template <bool F32>
__device__ inline void store4(void* p, size_t i, const float v[4]) {
  if constexpr (F32)
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i) = f32x4{v[0], v[1], v[2], v[3]};
  else
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p) + i) =
        u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// x of the lane that DPP control CTRL names.
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, false);
}

// Maximum of |x|'s bit pattern over each 16-lane row, in every lane of it:
// for finite values the order of the patterns is that of the magnitudes,
// and an infinity or NaN is above every finite one.
__device__ inline uint32_t row16_max(uint32_t x) {
  x = max(x, dpp<0xB1>(x));   // quad_perm [1,0,3,2]
  x = max(x, dpp<0x4E>(x));   // quad_perm [2,3,0,1]
  x = max(x, dpp<0x141>(x));  // row_half_mirror
  x = max(x, dpp<0x140>(x));  // row_mirror
  return x;
}
__device__ inline uint32_t wave_max(uint32_t x) {
  x = row16_max(x);
  uint32_t r = (uint32_t)__builtin_amdgcn_readlane((int)x, 0);
#pragma unroll
  for (int row = 1; row < 4; row++)
    r = max(r, (uint32_t)__builtin_amdgcn_readlane((int)x, 16 * row));
  return r;
}
__device__ inline float readlane(float x, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}
// Sum over the 64 lanes, the same in every lane (a fixed order).
__device__ inline float wave_sum(float x) {
  x += __uint_as_float(dpp<0xB1>(__float_as_uint(x)));
  x += __uint_as_float(dpp<0x4E>(__float_as_uint(x)));
  x += __uint_as_float(dpp<0x141>(__float_as_uint(x)));
  x += __uint_as_float(dpp<0x140>(__float_as_uint(x)));
  return (readlane(x, 0) + readlane(x, 16)) + (readlane(x, 32) + readlane(x, 48));
}

// Maximum over the 64 lanes (NaN lanes are passed over), in every lane.
__device__ inline float wave_fmax(float x) {
  x = fmaxf(x, __uint_as_float(dpp<0xB1>(__float_as_uint(x))));
  x = fmaxf(x, __uint_as_float(dpp<0x4E>(__float_as_uint(x))));
  x = fmaxf(x, __uint_as_float(dpp<0x141>(__float_as_uint(x))));
  x = fmaxf(x, __uint_as_float(dpp<0x140>(__float_as_uint(x))));
  return fmaxf(fmaxf(readlane(x, 0), readlane(x, 16)), fmaxf(readlane(x, 32), readlane(x, 48)));
}
// Sum of doubles over the 64 lanes, the same in every lane (a fixed order).
template <int CTRL>
__device__ inline double dpp64(double x) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, x);
  const unsigned long long lo = dpp<CTRL>((uint32_t)b), hi = dpp<CTRL>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}
__device__ inline double readlane64(double x, int lane) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, x);
  const unsigned long long lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const unsigned long long hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, hi << 32 | lo);
}
__device__ inline double wave_sum64(double x) {
  x += dpp64<0xB1>(x);
  x += dpp64<0x4E>(x);
  x += dpp64<0x141>(x);
  x += dpp64<0x140>(x);
  return (readlane64(x, 0) + readlane64(x, 16)) + (readlane64(x, 32) + readlane64(x, 48));
}

__device__ inline uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale of a group from its largest magnitude pattern: absmax / qmax, at
// least the smallest normal number (so that the quotients below stay
// finite), 1 for a group of zeros, NaN for a group that holds an infinity or
// a NaN (its codes are 0, and every product with the scale is NaN).
__device__ inline float group_scale(uint32_t amax, float qmax) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (amax == 0u) return 1.0f;
  return fmaxf(__uint_as_float(amax) / qmax, 0x1p-126f);
}

// Quantizer of one group: the scale and what the correctly rounded
// quotients need (quant_common.h).
struct Quant {
  float s, r;
  bool refine, bad;
  __device__ inline Quant(uint32_t amax, float qmax) {
    s = group_scale(amax, qmax);
    refine = s >= 0x1p-60f;
    r = 1.0f / s;
    bad = amax >= 0x7f800000u;
  }
  // No clamp: a quotient is at most 448 (1 + 2^-24) in size, which rounds to
  // 448 (the next step up would begin at 464).
  __device__ inline uint32_t e4m3x4(float a, float b, float c, float d) const {
    if (bad) return 0u;
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(rq::quotient(a, s, r, refine),
                                            rq::quotient(b, s, r, refine), 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(rq::quotient(c, s, r, refine),
                                        rq::quotient(d, s, r, refine), v, true);
    return (uint32_t)v;
  }
  __device__ inline uint32_t i8x4(float a, float b, float c, float d) const {
    return bad ? 0u : rq::quant4<false>(a, b, c, d, s, r, refine);
  }
};

// SiLU(g) * u = g / (1 + 2^(-g log2 e)) * u, a few units in the last place
// off: the exponent's argument in two parts (the product with log2 e rounded,
// and what the rounding and the constant's own tail leave, which enters as a
// factor 1 + tail ln 2), the hardware's power of two, and its reciprocal
// improved by one Newton step.  (The library's exponential and an IEEE
// division cost twice the instructions, and the quantizer's time is these.)
__device__ inline float silu_mul(float g, float u) {
  // Outside [-1000, 128] SiLU(g) is 0 or g; the product below stays finite.
  const float c = __builtin_amdgcn_fmed3f(g, -1000.0f, 128.0f);
  const float hi = c * -1.44269502162933349609375f;
  const float lo = __builtin_fmaf(c, -1.44269502162933349609375f, -hi) - c * 1.925963033500e-8f;
  if (hi >= 100.0f) {
    // 1 does not count beside the power, which is near the end of fp32's range
    // or beyond: g 2^-hi u with the whole part of hi applied last, u made
    // smaller before, so that no step but the last leaves the range.
    if (!(g > -INFINITY)) return __uint_as_float(0x7fc00000u);  // -inf or NaN
    const float n = rintf(hi);
    float e = __builtin_amdgcn_exp2f(n - hi);
    e = __builtin_fmaf(e, lo * -0.693147180559945f, e);
    return ldexpf(c * e * (u * 0x1p-32f), 32 - (int)n);
  }
  float e = __builtin_amdgcn_exp2f(hi);
  e = __builtin_fmaf(e, lo * 0.693147180559945f, e);
  const float d = 1.0f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  return g * r * u;
}

}  // namespace bk
}  // namespace qmoe
