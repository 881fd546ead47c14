// sv_kv.hpp -- device side of the 4-bit cache: its format (specverify_pass.h)
// and its page table.
#pragma once

#include "sv_device.hpp"
#include "sv_pass.h"

namespace sv {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 8 neighbouring values of 16 or 32 bits as fp32.
template <int DT>
struct Eight {
  u32x4 w[DT == SV_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const char* at) {
    const u32x4* v = reinterpret_cast<const u32x4*>(at);
#pragma unroll
    for (int i = 0; i < (DT == SV_F32 ? 2 : 1); ++i) w[i] = __builtin_nontemporal_load(v + i);
  }
  __device__ __forceinline__ void store(char* at) const {
    u32x4* v = reinterpret_cast<u32x4*>(at);
#pragma unroll
    for (int i = 0; i < (DT == SV_F32 ? 2 : 1); ++i) __builtin_nontemporal_store(w[i], v + i);
  }
  __device__ __forceinline__ void get(float* x) const {
    if constexpr (DT == SV_F16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[0][i] & 0xffffu));
        x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[0][i] >> 16));
      }
    } else {
      unpack<DT>(w[0], x);
      if constexpr (DT == SV_F32) unpack<DT>(w[1], x + 4);
    }
  }
  __device__ __forceinline__ void set(const float* x) {
    if constexpr (DT == SV_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == SV_F16) {
          const uint16_t lo = __builtin_bit_cast(uint16_t, (_Float16)x[2 * i]);
          const uint16_t hi = __builtin_bit_cast(uint16_t, (_Float16)x[2 * i + 1]);
          w[0][i] = lo | (uint32_t)hi << 16;
        } else {
          const f32x2 y = {x[2 * i], x[2 * i + 1]};
          w[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
        }
      }
    }
  }
};

// The byte of the scale of a block whose largest magnitude has these bits (of
// an fp32): 2^(e-2) for a magnitude in [2^e, 2^(e+1)), 2^(e-1) from 1.75 * 2^e on.
// Adding a quarter of the mantissa's range carries into the exponent there.
// The smallest scale is 2^-126 (also for zeros), the largest 2^125, whose 6 is
// still finite; 255 stands for NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t magnitude) {
  if (magnitude >= 0x7f800000u) return 255;
  const int e = (int)((magnitude + 0x200000u) >> 23) - 2;
  return (uint32_t)min(max(e, 1), 252);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 values as 8 codes, the first in the lowest 4 bits: the nearest that the
// format gives, ties to even, 6 beyond it.
__device__ __forceinline__ uint32_t encode8(const float* x, float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
  return w;
}
__device__ __forceinline__ void decode8(uint32_t w, float scale, float* x) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
  x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}

// Where 8 values (d8 = d / 8) of a token's row stand within a head's part of a
// page.  Of the values' rows a sixteenth is D/32 bytes, so the 4 bytes of 8
// values are two sixteenths at D = 64, one at 128 and half of one at 256.
template <int D>
__device__ __forceinline__ int64_t key_at(int64_t slot, int d8) { return slot * (D / 2) + d8 * 4; }
template <int D>
__device__ __forceinline__ int64_t value_at(int64_t slot, int d8) {
  const int byte = d8 * 4;
  return ((slot / 4 * 16 + byte / (D / 32)) * 4 + slot % 4) * (D / 32) + byte % (D / 32);
}
template <int D>
__device__ __forceinline__ int64_t key_scale_at(int64_t slot, int block) { return slot * (D / 32) + block; }
template <int D>
__device__ __forceinline__ int64_t value_scale_at(int64_t slot, int block) {
  return (slot / 4 * (D / 32) + block) * 4 + slot % 4;
}

__device__ __forceinline__ void flag(int32_t* err, int32_t bit) { atomicOr(err, bit); }

}  // namespace sv
