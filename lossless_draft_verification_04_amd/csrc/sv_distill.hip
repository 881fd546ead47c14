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
// most of the arithmetic.  4096 x 128256 bf16 rows: loss 159 us, 6.6 TB/s (a
// plain read reaches 7.1).  2048 x 152064, a tenth of them empty: gradient 234
// us, 5.05 TB/s of reads and writes (a copy 4.9).  Short calls are latencies:
// 333 x 20011 fp32 loss 8.9 us, 40 x 32000 bf16 gradient 5.7 us.  Short rows in
// great numbers feel a block's start and end, which no other row's work covers:
// loss of 2048 x 32000 bf16 rows 33 us, 3.9 TB/s; 2048 x 64000 48 us, 5.5 TB/s.
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

// Into LDS: thread i has token i.  Out-of-range and repeated ids are flagged
// and become absent.  Returns whether the row has teacher mass, in every
// thread; if so *z is on its way, the drafter's logit of the thread's token.
template <int DT>
__device__ __forceinline__ bool place_teacher(const DistillParams& a, Fetched& f, const void* row, Teacher& s,
                                              bool report, float* z) {
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
  if (f.id >= 0 && f.t > kNegInf) s.live = 1;
  lds_sync();
  const bool live = s.live != 0;
  *z = kNegInf;
  if (live && f.id >= 0) *z = load_elem<DT>(row, f.id);
  s.id[i] = f.id;
  token_teacher(s, i, f.id >= 0 ? f.t : kNegInf, a.k, a.invT);
  return live;
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
  __shared__ Drafter q;
  __shared__ float s_max[kDNT / kWave];
  __shared__ double s_sum[kDNT / kWave];
  const int r = blockIdx.x / a.nch;
  const int ch = blockIdx.x - r * a.nch;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const void* row = row_ptr(a.z, r, a.sb);
  const int64_t v0 = (int64_t)ch * a.vpc;
  const int64_t nv = (v0 + a.vpc < a.nvec ? v0 + a.vpc : a.nvec) - v0;
  // the row's first vectors are on their way while its teacher is prepared
  Fetched f = fetch_teacher(a, r);
  const __amdgpu_buffer_rsrc_t rs = range_rsrc(static_cast<const u32x4*>(row) + v0, (uint32_t)(nv * 16));
  uint32_t off = threadIdx.x * 16u;
  u32x4 cur[kDU];
#pragma unroll
  for (int u = 0; u < kDU; ++u) cur[u] = load_range(rs, off + (uint32_t)(u * kDNT * 16));
  for (int i = threadIdx.x; i < (int)(nv + 3) / 4; i += kDNT) s_mark[i] = 0u;
  float z;
  if (!place_teacher<DT>(a, f, row, s, ch == 0, &z)) {  // block-uniform, the same for all of the row's blocks
    if (ch == 0 && threadIdx.x == 0) {
      a.out_loss[r] = 0.f;
      reinterpret_cast<float4*>(a.out_stat)[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  if (f.id >= 0) {
    const int64_t i = (int64_t)f.id / E - v0;
    if (i >= 0 && i < nv) atomicOr(&s_mark[i >> 2], 1u << ((i & 3) * 8 + f.id % E));
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
  token_drafter(q, threadIdx.x, z, a.k, a.invT);
  const float wm = wave_fmax(acc.m);
  const double ws = wave_sum(acc.m == kNegInf ? 0.0 : (double)acc.s * (double)fast_exp2((acc.m - wm) * a.c));
  if (lane == 0) {
    s_max[wave] = wm;
    s_sum[wave] = ws;
  }
  lds_sync();
  // wave 0: its lanes' partial sums outside I, then the row's
  float pm = kNegInf;
  double ps = 0.0;
  if (wave == 0 && lane < kDNT / kWave) {
    pm = s_max[lane];
    ps = s_sum[lane];
  }
  if (a.nch > 1) {
    Partial* parts = static_cast<Partial*>(a.parts) + (int64_t)r * a.nch;
    if (wave == 0) {
      Partial out;
      out.pad = 0.f;
      out.m = wave_fmax(pm);
      out.s = wave_sum(ps * rescale(pm, out.m, a.c));
      if (lane == 0) put_partial(parts + ch, out);
    }
    if (!arrive_last<kDNT>(&a.cnt[r], (uint32_t)a.nch)) return;
    if (wave == 0) {
      pm = kNegInf;
      ps = 0.0;
      if (lane < kPL)
        for (int i = lane; i < a.nch; i += kPL) {
          const Partial p = get_partial(parts + i);
          const float m = fmaxf(pm, p.m);
          ps = ps * rescale(pm, m, a.c) + p.s * rescale(p.m, m, a.c);
          pm = m;
        }
      if (lane == 0) __hip_atomic_store(&a.cnt[r], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (wave != 0) return;
  const double rest = (double)f.rest;
  const Norm n = wave_teacher(s, a.k, rest, a.invT, lane);
  const RowSums w = wave_row_sums(q, pm, ps, a.invT, lane);
  if (w.m == kNegInf) {
    if (lane == 0) {
      set_error(a.err, SV_DERR_ROW);
      a.out_loss[r] = 0.f;
      reinterpret_cast<float4*>(a.out_stat)[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const double loss = wave_loss(s, q, a.k, rest, n, w, a.invT, lane);
  if (lane == 0) {
    a.out_loss[r] = (float)loss;
    reinterpret_cast<float4*>(a.out_stat)[r] = make_float4(w.m, (float)w.sum, w.m0, (float)w.s0);
  }
}

// ---------------------------------------------------------------------------
// Gradient.
// ---------------------------------------------------------------------------
// A block per (row part): the gradient outside I streams through, then the
// part's tokens of I are written over it.  In place this holds: the block
// reads its tokens' logits before it writes, and no other block's.
template <int DT>
__global__ __launch_bounds__(kDNT) void distill_grad_kernel(DistillParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  __shared__ Teacher s;
  __shared__ GradRow s_g;
  __shared__ double s_scale;
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
  Fetched f = fetch_teacher(a, r);
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
  float z;
  place_teacher<DT>(a, f, row, s, ch == 0, &z);
  // q at the thread's token, before any thread stores over it
  const double inv = 1.0 / (double)st.y;
  double q = z > kNegInf ? exp_d(((double)z - (double)st.x) * a.invT) * inv : 0.0;
  asm volatile("" : "+v"(q));  // read before the barrier: the barrier orders LDS only
  lds_sync();
  if (wave == 0) {
    const Norm n = wave_teacher(s, a.k, (double)f.rest, a.invT, lane);
    const double scale = (a.g ? (double)a.g[r] : 1.0) * a.invT;
    const double ratio = st.w > 0.f ? exp_d(((double)st.z - (double)st.x) * a.invT) * inv : 0.0;
    if (lane == 0) {
      s_g = grad_row(st.z, (double)st.w, n.p0, ratio, scale);
      s_scale = scale;
    }
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
  if (f.id >= 0 && f.id / E >= v0 && f.id / E < v1)
    store_elem<DT>(out, f.id, (float)((q - s.p[threadIdx.x]) * s_scale));
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
