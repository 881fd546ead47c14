// sv_distill.hip -- distillation from a teacher's top logits on gfx950: the
// loss KL(p || q) over the teacher's k tokens I and one class for all others,
// and its gradient.
//
//   p_i = exp(t_i / T) / Z, p_0 = exp(rest) / Z, Z = sum_i exp(t_i / T) + exp(rest)
//   q = softmax(z / T), q_0 = sum_{v not in I} q_v
//   loss = sum_i p_i log(p_i / q_i) + p_0 log(p_0 / q_0)
//   dz_v = (g / T) (q_v - p_v) in I, (g / T) q_v (1 - p_0 / q_0) elsewhere
//
// Both passes stream V logits a row and are bound by memory; an exponential
// a logit (a quarter-rate instruction) and the conversion of bf16 pairs are
// most of the arithmetic.
//
// Everything of size k is computed in 64 bits: the loss is a difference of
// logarithms near 10 that may be 1e-2 itself.  The row's sums are 32-bit per
// thread and 64-bit across threads.  The sum outside I is formed without the
// tokens of I (a byte of LDS per 16-byte vector marks them), so q_0 keeps its
// digits where I holds nearly everything, and the error that the sum's
// elements share (that of log2(e) / T in 32 bits) enters the loss only times
// q_0 - p_0.
#include "sv_distill.hpp"

namespace sv {

constexpr int kDNT = 256;
constexpr int kDU = 4;     // vectors in flight per thread
static_assert(SV_MAX_TEACHER == kDNT, "a thread a teacher token");

// A row's teacher on its way: thread i holds token i, its value, the rest.
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

// Into LDS (a block of at least SV_MAX_TEACHER threads).  Out-of-range and
// repeated ids are flagged and become absent.  Returns whether the row has
// teacher mass, in every thread; the drafter's logits are loaded if so.
template <int DT>
__device__ __forceinline__ bool place_teacher(const DistillParams& a, Fetched f, const void* row, Teacher& s,
                                              bool report) {
  const int i = threadIdx.x;
  const bool bad = f.id < -1 || f.id >= a.V;
  if (bad) f.id = -1;
  s.id[i] = f.id;
  if (i == 0) s.live = f.rest > kNegInf;
  lds_sync();
  bool twice = false;
  if (i < ((a.k + kWave - 1) & ~(kWave - 1))) twice = repeated(s.id, i, f.id, a.k);
  if (report && (bad || twice)) set_error(a.err, SV_DERR_TOKEN);
  if (twice) f.id = -1;
  s.t[i] = f.id >= 0 ? f.t : kNegInf;
  if (f.id >= 0 && f.t > kNegInf) s.live = 1;
  lds_sync();
  const bool live = s.live != 0;
  s.id[i] = f.id;
  s.z[i] = live && f.id >= 0 ? load_elem<DT>(row, f.id) : kNegInf;
  return live;
}

// The loss and the statistics of one row from the sum outside I, by one wave.
__device__ __forceinline__ void finish_loss(const DistillParams& a, int r, const Teacher& s, const Partial& out,
                                            int lane) {
  const double rest = a.rest ? (double)a.rest[r] : -__builtin_huge_val();
  const Norm n = wave_teacher_norm(s, a.k, rest, a.invT, lane);
  float m = kNegInf;
  for (int i = lane; i < a.k; i += kWave) m = fmaxf(m, s.z[i]);
  m = fmaxf(wave_fmax(m), out.m);
  if (m == kNegInf) {
    if (lane == 0) {
      set_error(a.err, SV_DERR_ROW);
      a.out_loss[r] = 0.f;
      reinterpret_cast<float4*>(a.out_stat)[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  double sum = 0.0;
  for (int i = lane; i < a.k; i += kWave)
    if (s.z[i] > kNegInf) sum += exp_d(((double)s.z[i] - (double)m) * a.invT);
  sum = wave_sum(sum);
  if (out.s > 0.0) sum += out.s * exp_d(((double)out.m - (double)m) * a.invT);
  const double lt = n.m + log_d(n.z);
  const double lq = (double)m * a.invT + log_d(sum);
  double loss = 0.0;
  for (int i = lane; i < a.k; i += kWave) {
    const double lp = (double)s.t[i] * a.invT - lt;
    const double p = s.t[i] > kNegInf ? exp_d(lp) : 0.0;
    if (p > 0.0) loss += p * (lp - ((double)s.z[i] * a.invT - lq));
  }
  loss = wave_sum(loss);
  const double p0 = exp_d(rest - lt);
  if (p0 > 0.0) loss += p0 * ((rest - lt) - ((double)out.m * a.invT + log_d(out.s) - lq));
  if (lane == 0) {
    a.out_loss[r] = (float)loss;
    reinterpret_cast<float4*>(a.out_stat)[r] = make_float4(m, (float)sum, out.m, (float)out.s);
  }
}

// kDU vectors of a row; tokens of I and elements past V become -inf.
template <int DT, bool LAST>
__device__ __forceinline__ void fold_group(const u32x4 (&d)[kDU], const uint8_t* mark, int64_t first, int64_t nv,
                                           int64_t v0, int V, float c, Mass& acc) {
  constexpr int E = Fmt<DT>::kPerVec;
  float x[kDU * E];
#pragma unroll
  for (int u = 0; u < kDU; ++u) unpack<DT>(d[u], x + u * E);
  uint32_t mk[kDU];
#pragma unroll
  for (int u = 0; u < kDU; ++u) {
    const int64_t i = first + (int64_t)u * kDNT;
    mk[u] = !LAST || i < nv ? mark[i] : 0xffu;
    if (LAST && i < nv && (v0 + i + 1) * E > V) mk[u] |= 0xffu << (V - (v0 + i) * E);
  }
  if (mk[0] | mk[1] | mk[2] | mk[3]) {
#pragma unroll
    for (int u = 0; u < kDU; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((mk[u] >> e) & 1u) x[u * E + e] = kNegInf;
  }
  fold_values<kDU * E>(x, c, acc);
}

template <int DT>
__global__ __launch_bounds__(kDNT) void distill_loss_kernel(DistillParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  extern __shared__ uint32_t s_mark[];  // a byte per vector of the part: its tokens in I
  __shared__ Teacher s;
  const int r = blockIdx.x / a.nch;
  const int ch = blockIdx.x - r * a.nch;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const void* row = row_ptr(a.z, r, a.sb);
  const int64_t v0 = (int64_t)ch * a.vpc;
  const int64_t nv = (v0 + a.vpc < a.nvec ? v0 + a.vpc : a.nvec) - v0;
  // the row's first vectors are on their way while its teacher is prepared
  const Fetched f = fetch_teacher(a, r);
  const __amdgpu_buffer_rsrc_t rs = range_rsrc(static_cast<const u32x4*>(row) + v0, (uint32_t)(nv * 16));
  uint32_t off = threadIdx.x * 16u;
  u32x4 cur[kDU];
#pragma unroll
  for (int u = 0; u < kDU; ++u) cur[u] = load_range(rs, off + (uint32_t)(u * kDNT * 16));
  for (int i = threadIdx.x; i < (int)(nv + 3) / 4; i += kDNT) s_mark[i] = 0u;
  if (!place_teacher<DT>(a, f, row, s, ch == 0)) {  // block-uniform, the same for all of the row's blocks
    if (ch == 0 && threadIdx.x == 0) {
      a.out_loss[r] = 0.f;
      reinterpret_cast<float4*>(a.out_stat)[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  if (threadIdx.x < a.k) {
    const int32_t id = s.id[threadIdx.x];
    const int64_t i = (int64_t)id / E - v0;
    if (id >= 0 && i >= 0 && i < nv) atomicOr(&s_mark[i >> 2], 1u << ((i & 3) * 8 + id % E));
  }
  lds_sync();
  const uint8_t* mark = reinterpret_cast<const uint8_t*>(s_mark);
  Mass acc;
  {
    // groups of kDU * kDNT vectors; the last one is masked (and may hold the row's end)
    const int64_t full = (nv - 1) / (kDU * kDNT);
    for (int64_t k = 0; k < full; ++k) {
      off += kDU * kDNT * 16;
      u32x4 nxt[kDU];
#pragma unroll
      for (int u = 0; u < kDU; ++u) nxt[u] = load_range(rs, off + (uint32_t)(u * kDNT * 16));
      fold_group<DT, false>(cur, mark, k * (kDU * kDNT) + threadIdx.x, nv, v0, a.V, a.c, acc);
#pragma unroll
      for (int u = 0; u < kDU; ++u) cur[u] = nxt[u];
    }
    fold_group<DT, true>(cur, mark, full * (kDU * kDNT) + threadIdx.x, nv, v0, a.V, a.c, acc);
  }
  Partial out = block_mass<kDNT>(acc, a.c);
  if (a.nch > 1) {
    Partial* parts = static_cast<Partial*>(a.parts) + (int64_t)r * a.nch;
    if (threadIdx.x == 0) put_partial(parts + ch, out);
    if (!arrive_last<kDNT>(&a.cnt[r], (uint32_t)a.nch)) return;
    if (wave == 0) {
      float m = kNegInf;
      for (int i = lane; i < a.nch; i += kWave) m = fmaxf(m, get_partial(parts + i).m);
      out.m = wave_fmax(m);
      double t = 0.0;
      for (int i = lane; i < a.nch; i += kWave) {
        const Partial p = get_partial(parts + i);
        t += p.s * rescale(p.m, out.m, a.c);
      }
      out.s = wave_sum(t);
      if (lane == 0) __hip_atomic_store(&a.cnt[r], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (wave == 0) finish_loss(a, r, s, out, lane);
}

// ---------------------------------------------------------------------------
// Gradient.
// ---------------------------------------------------------------------------
// One wave: the row's factors, and (q_i - p_i) g / T in place of s.z.
__device__ __forceinline__ GradRow wave_grad_row(const DistillParams& a, int r, Teacher& s, const float4 st, int lane) {
  const double rest = a.rest ? (double)a.rest[r] : -__builtin_huge_val();
  const Norm n = wave_teacher_norm(s, a.k, rest, a.invT, lane);
  const double scale = (a.g ? (double)a.g[r] : 1.0) * a.invT;
  const double inv = 1.0 / (double)st.y;
  for (int i = lane; i < a.k; i += kWave) {
    const double p = s.t[i] > kNegInf ? exp_d((double)s.t[i] * a.invT - n.m) / n.z : 0.0;
    const double q = s.z[i] > kNegInf ? exp_d(((double)s.z[i] - (double)st.x) * a.invT) * inv : 0.0;
    s.z[i] = (float)((q - p) * scale);
  }
  const double p0 = exp_d(rest - n.m) / n.z;
  const double q0 = st.w > 0.f ? (double)st.w * exp_d(((double)st.z - (double)st.x) * a.invT) * inv : 0.0;
  return grad_row(st.x, p0, q0, scale, inv);
}

// A block per (row part): the gradient outside I streams through, then the
// part's tokens of I are written over it.  In place this holds: the block
// reads its tokens' logits before it writes, and no other block's.
template <int DT>
__global__ __launch_bounds__(kDNT) void distill_grad_kernel(DistillParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  __shared__ Teacher s;
  __shared__ GradRow s_g;
  const int r = blockIdx.x / a.nch2;
  const int ch = blockIdx.x - r * a.nch2;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const u32x4* row = static_cast<const u32x4*>(row_ptr(a.z, r, a.sb));
  char* out = static_cast<char*>(a.grad) + (int64_t)r * a.gb;
  u32x4* outv = reinterpret_cast<u32x4*>(out);
  const int64_t v0 = (int64_t)ch * a.vpc2;
  const int64_t v1 = v0 + a.vpc2 < a.nvec ? v0 + a.vpc2 : a.nvec;
  const int64_t nfull = a.V / E;
  const int64_t vf = v1 < nfull ? v1 : nfull;  // whole vectors; the row's last one may be shorter
  // the part's first vectors are on their way while the row's factors are formed
  const Fetched f = fetch_teacher(a, r);
  u32x4 d[kDU];
#pragma unroll
  for (int u = 0; u < kDU; ++u) {
    const int64_t v = v0 + threadIdx.x + u * kDNT;
    if (v < vf) d[u] = load_vec(row, v);
  }
  const float4 st = reinterpret_cast<const float4*>(a.stat)[r];
  if (!(st.y > 0.f)) {  // no teacher mass, or no finite logit
    for (int64_t v = v0 + threadIdx.x; v < vf; v += kDNT)
      __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, outv + v);
    if (v1 > nfull && threadIdx.x < a.V - nfull * E) store_elem<DT>(out, nfull * E + threadIdx.x, 0.f);
    return;
  }
  place_teacher<DT>(a, f, row, s, ch == 0);
  lds_sync();
  if (wave == 0) {
    const GradRow g = wave_grad_row(a, r, s, st, lane);
    if (lane == 0) s_g = g;
  }
  lds_sync();
  const GradRow g = s_g;
  for (int64_t v = v0 + threadIdx.x; v < vf; v += kDU * kDNT) {
#pragma unroll
    for (int u = 0; u < kDU; ++u)
      if (v + u * kDNT < vf) __builtin_nontemporal_store(grad_vec<DT>(d[u], g, a.c), outv + v + u * kDNT);
#pragma unroll
    for (int u = 0; u < kDU; ++u)
      if (v + (kDU + u) * kDNT < vf) d[u] = load_vec(row, v + (kDU + u) * kDNT);
  }
  if (v1 > nfull && threadIdx.x < a.V - nfull * E) {
    const int e = threadIdx.x;
    const float z = load_elem<DT>(row, nfull * E + e);
    store_elem<DT>(out, nfull * E + e, grad_elem(z, g, a.c));
  }
  __builtin_amdgcn_s_waitcnt(0);  // the stream's stores are done before any token's
  __syncthreads();
  if (threadIdx.x < a.k) {
    const int32_t id = s.id[threadIdx.x];
    if (id >= 0 && id / E >= v0 && id / E < v1) store_elem<DT>(out, id, s.z[threadIdx.x]);
  }
}

hipError_t launch_distill_loss(const DistillParams& p, sv_dtype dt, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.R * p.nch));
  const size_t lds = (size_t)((p.vpc + 3) / 4 * 4);
  if (dt == SV_BF16)
    distill_loss_kernel<SV_BF16><<<grid, dim3(kDNT), lds, s>>>(p);
  else
    distill_loss_kernel<SV_F32><<<grid, dim3(kDNT), lds, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_distill_grad(const DistillParams& p, sv_dtype dt, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.R * p.nch2));
  if (dt == SV_BF16)
    distill_grad_kernel<SV_BF16><<<grid, dim3(kDNT), 0, s>>>(p);
  else
    distill_grad_kernel<SV_F32><<<grid, dim3(kDNT), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace sv
