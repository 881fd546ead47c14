// sv_distill.hpp -- pieces that the distillation kernels share: a row's
// teacher in LDS, its normaliser, and the gradient of a vector of logits.
#pragma once

#include "sv_draft.h"
#include "sv_topmass.hpp"

namespace sv {

// A row's teacher in LDS.  Token i belongs to the i-th of the block's token
// threads (whole waves): each wave sums its own tokens' exponentials, against
// its own largest value, and one wave then joins the waves' sums (lane by
// lane, so that no step takes longer for more tokens than one pass over them).
constexpr int kTW = SV_MAX_TEACHER / kWave;  // token waves
struct alignas(16) Teacher {
  int32_t id[SV_MAX_TEACHER];  // -1: absent
  float t[SV_MAX_TEACHER];     // value (-inf: no mass)
  double p[SV_MAX_TEACHER];    // exp((t - tm) / T), then the probability
  double ts[kTW];              // its wave's sum
  float tm[kTW];               // its wave's largest value
  int live;                    // the row has teacher mass
  int dup;                     // an id comes twice
};
// The drafter's logits at these tokens.
struct Drafter {
  float z[SV_MAX_TEACHER];
  double e[SV_MAX_TEACHER];  // exp((z - zm) / T)
  float g[SV_MAX_TEACHER];   // the loss's gradient there
  double zs[kTW];
  float zm[kTW];
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

// Token i's exponential and its wave's sum (every token wave whole).
__device__ __forceinline__ double wave_exponentials(float x, double invT, float* m, double* e) {
  *m = wave_fmax(x);
  *e = x > kNegInf ? exp_d(((double)x - (double)*m) * invT) : 0.0;
  return wave_sum(*e);
}
__device__ __forceinline__ void token_teacher(Teacher& s, int i, float t, int k, double invT) {
  const int w = i / kWave;
  float m = kNegInf;
  double e = 0.0, sum = 0.0;
  if (w * kWave < k) sum = wave_exponentials(t, invT, &m, &e);
  s.t[i] = t;
  s.p[i] = e;
  if (i % kWave == 0) {
    s.tm[w] = m;
    s.ts[w] = sum;
  }
}
__device__ __forceinline__ void token_drafter(Drafter& s, int i, float z, int k, double invT) {
  const int w = i / kWave;
  float m = kNegInf;
  double e = 0.0, sum = 0.0;
  if (w * kWave < k) sum = wave_exponentials(z, invT, &m, &e);
  s.z[i] = z;
  s.e[i] = e;
  if (i % kWave == 0) {
    s.zm[w] = m;
    s.zs[w] = sum;
  }
}

// One wave: the teacher's probabilities in s.p; p_0 and the normaliser
// Z = zs e^zm.
struct Norm {
  double zm, zs, p0;
};
__device__ __forceinline__ Norm wave_teacher(Teacher& s, int k, double rest, double invT, int lane) {
  double a = -__builtin_huge_val(), w = 0.0;
  if (lane < kTW && s.tm[lane] > kNegInf) {
    a = (double)s.tm[lane] * invT;
    w = s.ts[lane];
  }
  if (lane == kTW && rest > -__builtin_huge_val()) {
    a = rest;
    w = 1.0;
  }
  Norm n;
  n.zm = readlane_d(a, 0);
#pragma unroll
  for (int l = 1; l <= kTW; ++l) n.zm = fmax(n.zm, readlane_d(a, l));
  const double f = w > 0.0 ? exp_d(a - n.zm) : 0.0;
  w *= f;
  n.zs = readlane_d(w, 0);
#pragma unroll
  for (int l = 1; l <= kTW; ++l) n.zs += readlane_d(w, l);
  const double inv = 1.0 / n.zs;
  n.p0 = readlane_d(w, kTW) * inv;
#pragma unroll 1
  for (int i = lane; i < k; i += kWave) s.p[i] *= readlane_d(f, i / kWave) * inv;
  return n;
}

// One wave: the row's sums from the partial sums outside I, a lane each
// (lanes below kPL: pm, ps), and the tokens'.  m is the row's largest logit
// (-inf: it has none), sum = sum_v exp((z_v - m) / T); m0, s0 the same outside
// I; fac: the factor that brings token wave w's exponentials to m (lane kPL + w)
// and that of s0 (lane kPL + kTW).
constexpr int kPL = kWave - kTW - 1;
struct RowSums {
  float m, m0;
  double sum, s0, fac;
};
__device__ __forceinline__ RowSums wave_row_sums(const Drafter& s, float pm, double ps, double invT, int lane) {
  RowSums r;
  if (lane >= kPL) {
    pm = lane < kPL + kTW ? s.zm[lane - kPL] : kNegInf;
    ps = lane < kPL + kTW ? s.zs[lane - kPL] : 0.0;
  }
  r.m0 = wave_fmax(lane < kPL ? pm : kNegInf);
  r.m = wave_fmax(pm);
  // lane by lane: a partial sum outside I to m0, a token wave's to m, m0 to m
  const float x = lane == kPL + kTW ? r.m0 : pm;
  r.fac = x > kNegInf ? exp_d(((double)x - (double)(lane < kPL ? r.m0 : r.m)) * invT) : 0.0;
  ps *= r.fac;
  r.s0 = wave_sum(lane < kPL ? ps : 0.0);
  r.sum = r.s0 * readlane_d(r.fac, kPL + kTW);
#pragma unroll
  for (int w = 0; w < kTW; ++w) r.sum += readlane_d(ps, kPL + w);
  return r;
}

// One wave: the loss from the joined sums.  log p_i - log q_i is
// (t_i - z_i) / T less the difference of the normalisers' logarithms.
__device__ __forceinline__ double wave_loss(const Teacher& s, const Drafter& q, int k, double rest, const Norm& n,
                                            const RowSums& r, double invT, int lane) {
  const double ln = log_d(lane == 0 ? n.zs : lane == 1 ? r.sum : r.s0);
  const double lt = n.zm + readlane_d(ln, 0), lq = (double)r.m * invT + readlane_d(ln, 1);
  double loss = 0.0;
#pragma unroll 1
  for (int i = lane; i < k; i += kWave) {
    const double p = s.p[i];
    if (p > 0.0) loss += p * (((double)s.t[i] * invT - (double)q.z[i] * invT) - (lt - lq));
  }
  loss = wave_sum(loss);
  if (n.p0 > 0.0) loss += n.p0 * ((rest - lt) - ((double)r.m0 * invT + readlane_d(ln, 2) - lq));
  return loss;
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

// What the gradient of a row needs outside I: dz_v = each * 2^((z_v - m) c), m
// the largest logit outside I.  There it is
//   (g / T) (q_v - p_0 q_v / q_0) = (g / T) e^((z_v - m_0) / T) (e^((m_0 - m) / T) / s - p_0 / s_0),
// of which nothing overflows however little of q is outside I.
struct GradRow {
  float m, each;
};
// m0, s0 of the row; ratio = e^((m_0 - m) / T) / s; scale = g / T.
__device__ __forceinline__ GradRow grad_row(float m0, double s0, double p0, double ratio, double scale) {
  if (!(s0 > 0.0)) return GradRow{0.f, 0.f};  // every logit outside I is -inf
  return GradRow{m0, (float)(scale * (ratio - p0 / s0))};
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
