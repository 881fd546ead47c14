// sv_distill_held.hip -- loss and gradient of distillation in one read of the
// logits: a block holds a row in registers between the two (gfx950).
//
// The formulas and their arithmetic are those of sv_distill.hip.  A row's
// gradient needs the row's sums, so two passes read every logit twice; a
// compute unit's registers (512 KB) hold a row of up to about 190 thousand
// bf16 logits, so here each is read once and its gradient written once.
//
// Blocks are persistent and walk rows r, r + grid, ...; while a row's gradient
// is stored, the next row's vectors are loaded into the registers that fall
// free, so that the memory stays busy between rows.  What the next row's
// teacher needs (validity, repeats, whether it has a target at all) is
// prepared a row ahead for the same reason.
//
// A byte of LDS per vector marks the tokens of I; bits past V stay set for
// good.  The gradients at the tokens of I are stored, after the row's vectors,
// by the thread that stored the vector they lie in: a thread's stores to one
// place stay in order, and no wait for the next row's loads comes between.
#include "sv_distill.hpp"
#include "sv_internal.h"

namespace sv {

namespace {

// Stores that may touch the same bytes in two types.
typedef u32x4 u32x4_alias __attribute__((may_alias));
typedef __bf16 bf16_alias __attribute__((may_alias));
typedef float f32_alias __attribute__((may_alias));

template <int DT>
__device__ __forceinline__ void store_elem_alias(void* row, int64_t i, float x) {
  if constexpr (DT == SV_BF16)
    reinterpret_cast<bf16_alias*>(row)[i] = (__bf16)x;
  else
    reinterpret_cast<f32_alias*>(row)[i] = x;
}

// A row's teacher on its way into LDS: thread i holds token i.
struct Fetched {
  int32_t id;
  float t, rest;
};
__device__ __forceinline__ Fetched fetch_teacher(const DistillParams& a, int r) {
  Fetched f{-1, kNegInf, kNegInf};
  if ((int)threadIdx.x < a.k) {
    f.id = a.ids[(int64_t)r * a.k + threadIdx.x];
    f.t = a.vals[(int64_t)r * a.k + threadIdx.x];
  }
  if (a.rest) f.rest = a.rest[r];
  return f;
}
// First half: the ids in range.  A barrier, then the second half: repeats
// out, liveness.  (Visible after the next barrier.)
__device__ __forceinline__ void teacher_ids(const DistillParams& a, Fetched& f, Teacher& s) {
  if (f.id < -1 || f.id >= a.V) {
    set_error(a.err, SV_DERR_TOKEN);
    f.id = -1;
  }
  if (threadIdx.x < SV_MAX_TEACHER) s.id[threadIdx.x] = f.id;
  if (threadIdx.x == 0) s.live = f.rest > kNegInf;
}
// The repeats are found here and taken out of s.id by the caller after another barrier (drop_repeats).
__device__ __forceinline__ bool teacher_live(const DistillParams& a, Fetched& f, Teacher& s) {
  bool twice = false;
  if (f.id >= 0)
    for (int j = 0; j < (int)threadIdx.x; ++j) twice |= s.id[j] == f.id;
  if (twice) {
    set_error(a.err, SV_DERR_TOKEN);
    f.id = -1;
  }
  if (threadIdx.x < SV_MAX_TEACHER) s.t[threadIdx.x] = f.id >= 0 ? f.t : kNegInf;
  if (f.id >= 0 && f.t > kNegInf) s.live = 1;
  return twice;
}

// -inf in place of vector d's marked elements (a bit each).
template <int DT>
__device__ __forceinline__ void mask_vec(u32x4& d, uint32_t mk) {
  if constexpr (DT == SV_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = ((mk >> (2 * i)) & 1u ? 0xffffu : 0u) | ((mk >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
      d[i] = (d[i] & ~m) | (0xff80ff80u & m);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = (mk >> i) & 1u ? 0xff800000u : d[i];
  }
}

}  // namespace

template <int DT, int NT, int NV>
__global__ __launch_bounds__(NT) void distill_held_kernel(DistillParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  constexpr int NW = NT / kWave;
  constexpr int FU = 2;  // vectors folded at a time
  static_assert(NV % FU == 0 && NT >= SV_MAX_TEACHER && NW <= kWave, "shape");
  __shared__ uint32_t s_mark[NV * NT / 4];
  __shared__ Teacher s_t[2];
  __shared__ double s_p[SV_MAX_TEACHER];  // the teacher's probabilities
  __shared__ float s_max[NW];
  __shared__ double s_sum[NW];
  __shared__ GradRow s_g;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = tid / kWave;
  const int nvec = (int)a.nvec;
  const int nfull = a.V / E;
  const int tail = a.V - nfull * E;  // elements of the last, shorter vector
  const uint8_t* mark = reinterpret_cast<const uint8_t*>(s_mark);
  // marks: none, but for what lies past V
  for (int i = tid; i < NV * NT / 4; i += NT) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = i * 4 + j;
      const uint32_t b = v < nfull ? 0u : v == nfull && tail ? (0xffu << tail) & 0xffu : 0xffu;
      m |= b << (8 * j);
    }
    s_mark[i] = m;
  }
  int r = blockIdx.x;
  if (r >= a.R) return;
  u32x4 d[NV];
  auto row_of = [&](int row) { return row_ptr(a.z, row, a.sb); };
  // a row that is not read is a range of no bytes, whose loads give zeros
  auto row_range = [&](int row, bool read) { return range_rsrc(row_of(row), read ? (uint32_t)nvec * 16u : 0u); };
  const uint32_t off0 = (uint32_t)tid * 16u;
  // the first row's teacher
  int b = 0;
  float z = kNegInf, ztail = 0.f;
  {
    Fetched f = fetch_teacher(a, r);
    teacher_ids(a, f, s_t[0]);
    lds_sync();
    const bool twice = teacher_live(a, f, s_t[0]);
    lds_sync();
    if (twice) s_t[0].id[tid] = -1;
    lds_sync();
    const bool live = s_t[0].live != 0;
    const __amdgpu_buffer_rsrc_t rs = row_range(r, live);
    if (live && f.id >= 0) z = load_elem<DT>(row_of(r), f.id);
    if (live && tid < tail) ztail = load_elem<DT>(row_of(r), (int64_t)nfull * E + tid);
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = load_range(rs, off0 + (uint32_t)(i * NT * 16));
  }
  for (;;) {
    Teacher& s = s_t[b];
    Teacher& sn = s_t[b ^ 1];
    const bool live = s.live != 0;  // block-uniform
    const int rn = r + (int)gridDim.x;
    const bool next = rn < a.R;
    Fetched f{-1, kNegInf, kNegInf};
    if (next) f = fetch_teacher(a, rn);
    const int32_t id = tid < SV_MAX_TEACHER ? s.id[tid] : -1;
    if (live && id >= 0) atomicOr(&s_mark[id / E / 4], 1u << ((id / E % 4) * 8 + id % E));
    lds_sync();  // A: the marks
    // the teacher's normaliser and probabilities (wave 0), while the row arrives
    Norm n{0.0, 1.0};
    const double rest = a.rest ? (double)a.rest[r] : -__builtin_huge_val();
    if (live && wave == 0) {
      n = wave_teacher_norm(s, a.k, rest, a.invT, lane);
#pragma unroll 1
      for (int i = lane; i < a.k; i += kWave)
        s_p[i] = s.t[i] > kNegInf ? exp_d((double)s.t[i] * a.invT - n.m) / n.z : 0.0;
    }
    Mass acc;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; i += FU) {
        // the marked tokens leave the row for good: their gradients are stored apart
        uint32_t mk[FU], any = 0;
        float x[FU * E];
#pragma unroll
        for (int u = 0; u < FU; ++u) any |= mk[u] = mark[(i + u) * NT + tid];
        if (any) {
#pragma unroll
          for (int u = 0; u < FU; ++u) mask_vec<DT>(d[i + u], mk[u]);
        }
#pragma unroll
        for (int u = 0; u < FU; ++u) unpack<DT>(d[i + u], x + u * E);
        fold_values<FU * E, true>(x, a.c, acc);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (tid < SV_MAX_TEACHER) s.z[tid] = id >= 0 ? z : kNegInf;
      const float wm = wave_fmax(acc.m);
      const double ws = wave_sum(acc.m == kNegInf ? 0.0 : (double)acc.s * (double)fast_exp2((acc.m - wm) * a.c));
      if (lane == 0) {
        s_max[wave] = wm;
        s_sum[wave] = ws;
      }
    }
    if (next) teacher_ids(a, f, sn);
    lds_sync();  // B: every wave's mass, the drafter's logits of I, the next row's ids
    bool twice = false;
    if (next) twice = teacher_live(a, f, sn);
    if (live && id >= 0) atomicAnd(&s_mark[id / E / 4], ~(1u << ((id / E % 4) * 8 + id % E)));
    float st_m = 0.f, st_s = 0.f, st_m0 = 0.f, st_s0 = 0.f, loss = 0.f;
    if (live && wave == 0) {
      // the mass outside I, the whole row's, and the gradient's factors
      const float wm = lane < NW ? s_max[lane] : kNegInf;
      const double ws = lane < NW ? s_sum[lane] : 0.0;
      const float m0 = wave_fmax(wm);
      const double s0 = wave_sum(ws * rescale(wm, m0, a.c));
      float m = kNegInf;
#pragma unroll 1
      for (int i = lane; i < a.k; i += kWave) m = fmaxf(m, s.z[i]);
      m = fmaxf(wave_fmax(m), m0);
      GradRow g{0.f, 0.f};
      if (m > kNegInf) {
        double sum = 0.0;
  #pragma unroll 1
      for (int i = lane; i < a.k; i += kWave)
          if (s.z[i] > kNegInf) sum += exp_d(((double)s.z[i] - (double)m) * a.invT);
        sum = wave_sum(sum);
        const double out = s0 > 0.0 ? s0 * exp_d(((double)m0 - (double)m) * a.invT) : 0.0;
        sum += out;
        const double inv = 1.0 / sum;
        const double p0 = exp_d(rest - n.m) / n.z;
        const double scale = (a.g ? (double)a.g[r] : 1.0) * a.invT;
        g = grad_row(m, p0, out * inv, scale, inv);
        // the loss, and the gradient at the tokens of I in place of their logits
        const double ln = log_d(lane == 0 ? n.z : lane == 1 ? sum : s0);
        const double lt = n.m + readlane_d(ln, 0), lq = (double)m * a.invT + readlane_d(ln, 1);
        double l = 0.0;
  #pragma unroll 1
      for (int i = lane; i < a.k; i += kWave) {
          const double p = s_p[i], zi = (double)s.z[i] * a.invT;
          if (p > 0.0) l += p * (((double)s.t[i] * a.invT - lt) - (zi - lq));
          const double q = s.z[i] > kNegInf ? exp_d(zi - (double)m * a.invT) * inv : 0.0;
          s.z[i] = (float)((q - p) * scale);
        }
        l = wave_sum(l);
        if (p0 > 0.0) l += p0 * ((rest - lt) - ((double)m0 * a.invT + readlane_d(ln, 2) - lq));
        loss = (float)l;
        st_m = m;
        st_s = (float)sum;
        st_m0 = m0;
        st_s0 = (float)s0;
      } else {
        if (lane == 0) set_error(a.err, SV_DERR_ROW);
  #pragma unroll 1
      for (int i = lane; i < a.k; i += kWave) s.z[i] = 0.f;
      }
      if (lane == 0) s_g = g;
    } else if (wave == 0) {
      if (lane == 0) s_g = GradRow{0.f, 0.f};
#pragma unroll 1
      for (int i = lane; i < a.k; i += kWave) s.z[i] = 0.f;
    }
    lds_sync();  // C: the factors, the gradients of I, the next row's liveness
    if (twice) sn.id[tid] = -1;
    const bool nlive = next && sn.live != 0;
    const __amdgpu_buffer_rsrc_t rs = row_range(nlive ? rn : r, nlive);
    char* out = static_cast<char*>(a.grad) + (int64_t)r * a.gb;
    const __amdgpu_buffer_rsrc_t ro = range_rsrc(out, (uint32_t)nfull * 16u);
    float zt = 0.f;
    if (nlive) {
      if (f.id >= 0) z = load_elem<DT>(row_of(rn), f.id);
      if (tid < tail) zt = load_elem<DT>(row_of(rn), (int64_t)nfull * E + tid);
    }
    const GradRow g = s_g;
    {
      uint32_t off = off0;
      asm volatile("" : "+v"(off));  // the NV offsets are formed as they are used, not kept
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        // the row stays packed: without this the compiler keeps the fold's
        // unpacked values alive beside it, twice the registers there are
        asm volatile("" : "+v"(d[i]));
        store_range(ro, off, grad_vec<DT>(d[i], g, a.c));
        d[i] = load_range(rs, off);
        off += NT * 16;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (tid < tail) store_elem_alias<DT>(out, (int64_t)nfull * E + tid, grad_elem(ztail, g, a.c));
    // the tokens of I whose vectors this wave's threads stored
    for (int i0 = 0; i0 < a.k; i0 += kWave) {
      const int i = i0 + lane;
      const int32_t ti = i < a.k ? s.id[i] : -1;
      const float tv = i < a.k ? s.z[i] : 0.f;
      // in the shorter last vector thread e stored element e
      const int owner = ti / E < nfull ? ti / E % NT : ti - nfull * E;
      uint64_t mine = __ballot(ti >= 0 && owner / kWave == wave);
      while (mine) {
        const int q = __builtin_ctzll(mine);
        mine &= mine - 1;
        const int oid = __builtin_amdgcn_readlane(ti, q);
        const float ov = readlane_f(tv, q);
        const int ol = __builtin_amdgcn_readlane(owner, q) & (kWave - 1);
        if (lane == ol) store_elem_alias<DT>(out, oid, ov);
      }
    }
    if (tid == 0) {
      a.out_loss[r] = loss;
      reinterpret_cast<float4*>(a.out_stat)[r] = make_float4(st_m, st_s, st_m0, st_s0);
    }
    if (!next) return;
    ztail = zt;
    r = rn;
    b ^= 1;
    lds_sync();  // the next row's ids are final; this row's teacher may be overwritten
  }
}

namespace {

template <int DT, int NT, int NV>
hipError_t launch_held(const DistillParams& p, hipStream_t s) {
  static int cache[64];
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  int cap = dev >= 0 && dev < 64 ? cache[dev] : 0;
  if (cap == 0) {
    cap = device_capacity(reinterpret_cast<const void*>(&distill_held_kernel<DT, NT, NV>), NT, dev);
    if (cap <= 0) return hipErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) cache[dev] = cap;
  }
  const unsigned grid = (unsigned)(p.R < cap ? p.R : cap);
  distill_held_kernel<DT, NT, NV><<<dim3(grid), dim3(NT), 0, s>>>(p);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_held_dt(const DistillParams& p, hipStream_t s) {
  const int64_t n = p.nvec;
  if (n <= 256 * 4) return launch_held<DT, 256, 4>(p, s);
  if (n <= 256 * 8) return launch_held<DT, 256, 8>(p, s);
  if (n <= 512 * 8) return launch_held<DT, 512, 8>(p, s);
  if (n <= 512 * 16) return launch_held<DT, 512, 16>(p, s);
  if (n <= 1024 * 12) return launch_held<DT, 1024, 12>(p, s);
  if (n <= 1024 * 16) return launch_held<DT, 1024, 16>(p, s);
  if (n <= 1024 * 20) return launch_held<DT, 1024, 20>(p, s);
  return launch_held<DT, 1024, 24>(p, s);
}

}  // namespace

hipError_t launch_distill_held(const DistillParams& p, sv_dtype dt, hipStream_t s) {
  return dt == SV_BF16 ? launch_held_dt<SV_BF16>(p, s) : launch_held_dt<SV_F32>(p, s);
}

}  // namespace sv
