// hs_values.cuh -- element types of the norm kernels: single values and 16-byte
// chunks to and from fp32, E4M3 codes, and the inverse of a norm.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/hisparse.h"
#include "hs_device.cuh"

namespace hs {

template <int kDtype>
struct Elem;
template <>
struct Elem<HS_DT_F32> {
  static constexpr int kBytes = 4, kChunk = 4;
  __device__ static float load(const unsigned char* p) { return *reinterpret_cast<const float*>(p); }
  __device__ static void store(unsigned char* p, float x) { *reinterpret_cast<float*>(p) = x; }
};
template <>
struct Elem<HS_DT_F16> {
  static constexpr int kBytes = 2, kChunk = 8;
  __device__ static float load(const unsigned char* p) {
    return __half2float(*reinterpret_cast<const __half*>(p));
  }
  __device__ static void store(unsigned char* p, float x) {
    *reinterpret_cast<__half*>(p) = __float2half_rn(x);
  }
};
template <>
struct Elem<HS_DT_BF16> {
  static constexpr int kBytes = 2, kChunk = 8;
  __device__ static float load(const unsigned char* p) {
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
  }
  __device__ static void store(unsigned char* p, float x) {
    *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
  }
};

// Round to nearest even; finite overflow and infinities go to +-448, NaN stays.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

template <int kDtype>
__device__ __forceinline__ void unpack(uint4 raw, float* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == HS_DT_F32) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (kDtype == HS_DT_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <int kDtype>
__device__ __forceinline__ uint4 pack(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == HS_DT_F32) {
      w[i] = __float_as_uint(x[i]);
    } else if constexpr (kDtype == HS_DT_F16) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 / sqrt(mean square + eps) as two factors, for values are multiplied by one after the
// other: the inverse of a subnormal root is past fp32's range.  0 where both are zero, so
// that zeros stay zero without eps too (0 times infinity would be NaN).  Where the squares
// leave fp32's range, or all but do, sum_of(f) is asked for the sum of squares of the
// values times the power of two f: 2^96 takes the least of them (2^-149) to 2^-53, and
// those of a mean square below 2^-100 to 2^54 at most.
struct InverseRms {
  float pre, inv;
};
template <typename Sum>
__device__ __forceinline__ InverseRms inverse_rms(float sum_sq, float inv_dim, float eps, Sum sum_of) {
  float ms = sum_sq * inv_dim + eps;
  InverseRms r{1.f, 1.f};
  if (ms < 0x1p-100f) {
    r.pre = 0x1p96f;
    ms = sum_of(r.pre) * inv_dim + eps * r.pre * r.pre;
  } else if (ms > 0x1p127f && eps < 0x1p126f) {
    r = InverseRms{0x1p-40f, 0x1p-40f};  // (what that makes subnormal ends below 2^-149)
    ms = sum_of(0x1p-80f) * inv_dim + eps * 0x1p-80f * 0x1p-80f;
  }
  r.inv = ms == 0.f ? 0.f : rsqrtf(ms) * r.inv;
  return r;
}

// The larger of `top` and the magnitude of x, as bits: they order like the values, and
// a NaN is above them all and stays.
__device__ __forceinline__ uint32_t larger_bits(uint32_t top, float x) {
  return max(top, __float_as_uint(x) & 0x7FFFFFFFu);
}
// The scale of codes whose largest value has these bits: 1/448 of it, or the power of two
// not below that; 0 below the smallest normal number.
__device__ __forceinline__ float code_scale(uint32_t top, bool pow2) {
  const float s = __uint_as_float(top) * (1.0f / 448.0f);
  uint32_t b = __float_as_uint(s);
  if (b < 0x00800000u) return 0.f;
  // (an infinity, whose mantissa is 0, and a NaN stay what they are)
  if (pow2 && b < 0x7F800000u) b = (b + 0x007FFFFFu) & 0xFF800000u;
  return __uint_as_float(b);
}
// What values are multiplied by on their way to codes.
__device__ __forceinline__ float code_factor(float scale) { return scale == 0.f ? 0.f : 1.0f / scale; }

// One chunk of 8 or 4 values times f to E4M3 codes.
template <int kE>
__device__ __forceinline__ void store_codes(unsigned char* d, const float (&x)[kE], float f) {
  uint32_t w[kE / 4];
#pragma unroll
  for (int i = 0; i < kE / 4; ++i)
    w[i] = e4m3_pair(x[4 * i] * f, x[4 * i + 1] * f) | e4m3_pair(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16;
  if constexpr (kE == 8)
    *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(d) = w[0];
}

// 16 bytes that this kernel may write again (the read-only path is not for those).
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

}  // namespace hs
