// sv_distill.hpp -- pieces that the distillation kernels share: a row's
// teacher in LDS, its normaliser, and the gradient of a vector of logits.
#pragma once

#include "sv_draft.h"
#include "sv_topmass.hpp"

namespace sv {

// A 64-bit constant, formed in scalar registers where it stands: left alone
// the compiler lifts such constants out of the loop over rows into vector
// registers, which there hold a row.
__device__ __forceinline__ double here(double c) {
  asm volatile("" : "+s"(c));
  return c;
}
// e^x for x <= 0 in 64 bits to about 1e-11: x = n log 2 + r with |r| <= log(2) / 2
// (log 2 in two parts, the first short enough that n times it is exact), and
// the series of e^r to r^9 / 9!; 0 below the range.
__device__ __forceinline__ double exp_d(double x) {
  x = fmax(x, here(-800.0));
  const double n = rint(x * here(1.4426950408889634));
  double r = fma(n, here(-0.693147180369123816490), x);
  r = fma(n, here(-1.90821492927058770002e-10), r);
  double p = fma(here(1.0 / 362880.0), r, here(1.0 / 40320.0));
  p = fma(p, r, here(1.0 / 5040.0));
  p = fma(p, r, here(1.0 / 720.0));
  p = fma(p, r, here(1.0 / 120.0));
  p = fma(p, r, here(1.0 / 24.0));
  p = fma(p, r, here(1.0 / 6.0));
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)n);
}
// log x of an x in the range of fp32 by one step of Newton's method on
// e^y = x from a 32-bit logarithm (1e-7 before, 1e-13 after); -inf of 0.
__device__ __forceinline__ double log_d(double x) {
  if (!(x > 0.0)) return -__builtin_huge_val();
  const double y = (double)__builtin_amdgcn_logf((float)x) * here(0.6931471805599453);
  // e^-y with a non-positive argument
  return y >= 0.0 ? y + (x * exp_d(-y) - 1.0) : y + (x - exp_d(y)) / x;
}

// A row's teacher tokens in LDS: id (-1: absent), value, the drafter's logit.
struct alignas(16) Teacher {
  int32_t id[SV_MAX_TEACHER];
  float t[SV_MAX_TEACHER];
  float z[SV_MAX_TEACHER];
  int live;
};

// Whether token i's id stands among those before it (ids in LDS).  Every token
// compares with all k, four to a load, none waiting for another.
__device__ __forceinline__ bool repeated(const int32_t* ids, int i, int32_t id, int k) {
  const int4* v = reinterpret_cast<const int4*>(ids);
  bool twice = false;
#pragma unroll 4
  for (int j = 0; j < k; j += 4) {
    const int4 w = v[j >> 2];
    twice |= ((w.x == id) & (j < i)) | ((w.y == id) & (j + 1 < i)) | ((w.z == id) & (j + 2 < i)) |
             ((w.w == id) & (j + 3 < i));
  }
  return twice && id >= 0;
}

// The teacher's normaliser: its largest exponent m and Z relative to it.
struct Norm {
  double m, z;
};
__device__ __forceinline__ Norm wave_teacher_norm(const Teacher& s, int k, double rest, double invT, int lane) {
  float tm = kNegInf;
  for (int i = lane; i < k; i += kWave) tm = fmaxf(tm, s.t[i]);
  tm = wave_fmax(tm);
  Norm n;
  n.m = fmax((double)tm * invT, rest);
  double z = 0.0;
#pragma unroll 1
  for (int i = lane; i < k; i += kWave)
    if (s.t[i] > kNegInf) z += exp_d((double)s.t[i] * invT - n.m);
  n.z = wave_sum(z) + exp_d(rest - n.m);
  return n;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// E values as one vector of the row's type (bf16: round to nearest even).
template <int DT>
__device__ __forceinline__ u32x4 pack(const float* x) {
  u32x4 d;
  if constexpr (DT == SV_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * i], x[2 * i + 1]}, bf16x2));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = __float_as_uint(x[i]);
  }
  return d;
}
template <int DT>
__device__ __forceinline__ void store_elem(void* row, int64_t i, float x) {
  if constexpr (DT == SV_BF16)
    reinterpret_cast<__bf16*>(row)[i] = (__bf16)x;
  else
    reinterpret_cast<float*>(row)[i] = x;
}

// What the gradient of a row needs outside I: dz_v = each * 2^((z_v - m) c).
struct GradRow {
  float m, each;
};
// Of a row whose largest logit is m, inv = 1 / sum exp((z - m) / T).
__device__ __forceinline__ GradRow grad_row(float m, double p0, double q0, double scale, double inv) {
  const double other = p0 > 0.0 ? (q0 > 0.0 ? 1.0 - p0 / q0 : 0.0) : 1.0;
  return GradRow{m, (float)(other * scale * inv)};
}

__device__ __forceinline__ float grad_elem(float z, const GradRow& g, float c) {
  return g.each * fast_exp2((z - g.m) * c);
}
template <int DT>
__device__ __forceinline__ u32x4 grad_vec(const u32x4 d, const GradRow& g, float c) {
  constexpr int E = Fmt<DT>::kPerVec;
  float x[E];
  unpack<DT>(d, x);
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = grad_elem(x[e], g, c);
  return pack<DT>(x);
}

// One 16-byte non-temporal store at byte offset `off` of a range (nothing past
// its end).  The gradient is not read again here; plain stores keep lines in
// the caches and reach 4.3 TB/s of reads and writes where these reach 4.8-5.1
// (gradients of 2048 x 152064 and 4096 x 128256 bf16 rows).
__device__ __forceinline__ void store_range(__amdgpu_buffer_rsrc_t r, uint32_t off, const u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, 2);
}

}  // namespace sv
