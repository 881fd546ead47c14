// sv_distill_held.hip -- loss and gradient of distillation in one read of the
// logits: a block holds a row in registers between the two (gfx950).
//
// The formulas and their arithmetic are those of sv_distill.hip.  A row's
// gradient needs the row's sums, so two passes read every logit twice; a
// compute unit's registers (512 KB) hold a row of up to about 130 thousand
// bf16 logits beside what the work takes, so here each is read once and its
// gradient written once: 4096 x 128256 bf16 rows, a tenth of them empty, 407 us
// at 4.9 TB/s (a copy's rate); 2000 rows 210 us, 278 in two launches.  96 x
// 32000 fp32 rows: 12.6 us, the latencies of one row's turn.
//
// Longer rows spill some registers to memory: 12, 40, 68 and 160 bytes a thread
// at 18, 20, 22 and 24 vectors (rows of up to 147456, 163840, 180224 and 196608
// bf16 logits; 12, 36, 76 and 112 in fp32).  Counted, 2000 rows of 152064 read
// 584 MiB of 580 and write 595, in 252 us; of 196608, 779 of 750 and 814, in
// 341 us.  Two launches take 330 and 423.
//
// Blocks are persistent and walk rows r, r + grid, ...; while a row's gradient
// is stored, the next row's vectors are loaded into the registers that fall
// free, so that the memory stays busy between rows.  What the next row's
// teacher needs (validity, repeats, whether it has a target at all) is
// prepared a row ahead for the same reason.
//
// A byte of LDS per vector marks the tokens of I; bits past V stay set for
// good.  The gradients at the tokens of I are stored, after the row's vectors,
// by the wave that stored the vector they lie in: a wave's stores to one place
// stay in order, and no wait for the next row's loads comes between.
#include <atomic>

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

// A row's teacher on its way into LDS.  Token i is held by the i-th thread
// from the block's last SV_MAX_TEACHER on (wave 0 has the scalar work).
struct Fetched {
  int32_t id;
  float t, rest;
};
__device__ __forceinline__ Fetched fetch_teacher(const DistillParams& a, int r, int i) {
  Fetched f{-1, kNegInf, kNegInf};
  if (i >= 0 && i < a.k) {
    f.id = a.ids[(int64_t)r * a.k + i];
    f.t = a.vals[(int64_t)r * a.k + i];
  }
  if (a.rest) f.rest = a.rest[r];
  return f;
}
// The ids in range.  After a barrier, teacher_tokens.
__device__ __forceinline__ void teacher_ids(const DistillParams& a, Fetched& f, Teacher& s, int i) {
  if (f.id < -1 || f.id >= a.V) {
    set_error(a.err, SV_DERR_TOKEN);
    f.id = -1;
  }
  if (i >= 0) s.id[i] = f.id;
  if (i == 0) {
    s.live = f.rest > kNegInf;
    s.dup = 0;
  }
}
// The marks and exponentials in, whether there is mass at all; final after a
// barrier, behind which teacher_repeats looks after an id that comes twice (its
// mark was set already).
template <int E>
__device__ __forceinline__ void teacher_tokens(const DistillParams& a, const Fetched& f, Teacher& s, uint32_t* mark,
                                               int i) {
  if (i < 0) return;  // whole waves
  if (f.id >= 0) {
    const uint32_t bit = 1u << ((f.id / E % 4) * 8 + f.id % E);
    if (atomicOr(&mark[f.id / E / 4], bit) & bit) s.dup = 1;
    if (f.t > kNegInf) s.live = 1;
  }
  token_teacher(s, i, f.id >= 0 ? f.t : kNegInf, a.k, a.invT);
}
// The block's threads, for a row with repeats (s.dup): they become absent.
__device__ __forceinline__ void teacher_repeats(const DistillParams& a, Fetched& f, Teacher& s, int i) {
  const bool twice = i >= 0 && repeated(s.id, i, f.id, a.k);
  lds_sync();
  if (twice) {
    set_error(a.err, SV_DERR_TOKEN);
    f.id = -1;
    s.id[i] = -1;
  }
  if (i == 0) s.live = f.rest > kNegInf;
  lds_sync();
  if (i >= 0) {
    if (f.id >= 0 && f.t > kNegInf) s.live = 1;
    token_teacher(s, i, f.id >= 0 ? f.t : kNegInf, a.k, a.invT);
  }
  lds_sync();
}

}  // namespace

// 128 registers a thread at most, so that two blocks of 512 threads share a
// compute unit: one stores while the other waits for its row's sums (2000 x
// 34480 bf16 rows 94 us in one block of 138 registers, 81 in two; 600 rows 38
// and 30).
template <int DT, int NT, int NV>
__global__ __launch_bounds__(NT, 4) void distill_held_kernel(DistillParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  constexpr int NW = NT / kWave;
  constexpr int FU = 2;                   // vectors folded at a time
  constexpr int LAG = NV < 4 ? NV : 4;    // loads ahead of the fold
  constexpr int kMarks = NV * NT / 4;     // words of marks
  constexpr int kLossWave = NW > 2 ? 1 : 0, kNextWave = NW > 2 ? 2 : 0;
  static_assert(NV % FU == 0 && LAG % FU == 0 && NT >= SV_MAX_TEACHER && NW <= kPL, "shape");
  __shared__ uint32_t s_mark[2][kMarks];
  __shared__ Teacher s_t[2];
  __shared__ Drafter s_q;
  __shared__ float s_max[NW];
  __shared__ double s_sum[NW];
  __shared__ Norm s_n[2];       // of the teachers in s_t
  __shared__ double s_scale[2];  // g / T of those rows
  __shared__ RowSums s_r;
  __shared__ GradRow s_g;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = tid / kWave;
  const int ti = tid - (NT - SV_MAX_TEACHER);  // this thread's teacher token (negative: none)
  const int nvec = (int)a.nvec;
  const int nfull = a.V / E;
  const int tail = a.V - nfull * E;  // elements of the last, shorter vector
  int r = blockIdx.x;
  if (r >= a.R) return;
  u32x4 d[NV];
  auto row_of = [&](int row) { return row_ptr(a.z, row, a.sb); };
  // a row that is not read is a range of no bytes, whose loads give zeros
  auto row_range = [&](int row, bool read) { return range_rsrc(row_of(row), read ? (uint32_t)nvec * 16u : 0u); };
  const uint32_t off0 = (uint32_t)tid * 16u;
  Mass acc;
  // FU vectors from i on: the marked tokens leave the row for good (their
  // gradients are stored apart), the others go into the mass
  auto fold = [&](int i, const uint8_t* mark) {
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
  };
  auto clear_mark = [&](int b, int32_t id) { atomicAnd(&s_mark[b][id / E / 4], ~(1u << ((id / E % 4) * 8 + id % E))); };
  // one wave: a row's teacher as probabilities
  auto teacher_probs = [&](int row, int b) {
    const double scale = (a.g ? (double)a.g[row] : 1.0) * a.invT;
    const Norm n = wave_teacher(s_t[b], a.k, a.rest ? (double)a.rest[row] : -__builtin_huge_val(), a.invT, lane);
    if (lane == 0) {
      s_n[b] = n;
      s_scale[b] = scale;
    }
  };
  // the first row: its teacher, its vectors, its mass
  int b = 0;
  Fetched cur = fetch_teacher(a, r, ti);
  {
    // its vectors are asked for once rest is here, ahead of the rest of its
    // teacher's preparation; the row number counts as divergent here, so that
    // each load stands in a loop over lanes (later rows' do not)
    const __amdgpu_buffer_rsrc_t rs = row_range(r, true);
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = load_range(rs, off0 + (uint32_t)(i * NT * 16));
  }
  // marks: none, but for what lies past V
  for (int i = tid; i < kMarks; i += NT) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = i * 4 + j;
      const uint32_t w = v < nfull ? 0u : v == nfull && tail ? (0xffu << tail) & 0xffu : 0xffu;
      m |= w << (8 * j);
    }
    s_mark[0][i] = s_mark[1][i] = m;
  }
  float z = kNegInf, ztail = 0.f;
  {
    teacher_ids(a, cur, s_t[0], ti);
    lds_sync();
    teacher_tokens<E>(a, cur, s_t[0], s_mark[0], ti);
    lds_sync();
    if (s_t[0].dup) teacher_repeats(a, cur, s_t[0], ti);
    const bool live = s_t[0].live != 0;
    if (live && cur.id >= 0) z = load_elem<DT>(row_of(r), cur.id);
    if (live && tid < tail) ztail = load_elem<DT>(row_of(r), (int64_t)nfull * E + tid);
    if (!live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] = u32x4{0u, 0u, 0u, 0u};
    } else {
      if (wave == kNextWave) teacher_probs(r, 0);
#pragma unroll
      for (int i = 0; i < NV; i += FU) {
        fold(i, reinterpret_cast<const uint8_t*>(s_mark[0]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // a row a turn: its vectors are here and summed up thread by thread
  for (;;) {
    Teacher& s = s_t[b];
    Teacher& sn = s_t[b ^ 1];
    const bool live = s.live != 0;  // block-uniform
    const int rn = r + (int)gridDim.x;
    const bool next = rn < a.R;
    Fetched f{-1, kNegInf, kNegInf};
    if (next) f = fetch_teacher(a, rn, ti);
    const float wm = wave_fmax(acc.m);
    const double ws = wave_sum(acc.m == kNegInf ? 0.0 : (double)acc.s * (double)fast_exp2((acc.m - wm) * a.c));
    if (lane == 0) {
      s_max[wave] = wm;
      s_sum[wave] = ws;
    }
    if (ti >= 0) token_drafter(s_q, ti, live && cur.id >= 0 ? z : kNegInf, a.k, a.invT);
    if (next) teacher_ids(a, f, sn, ti);
    lds_sync();  // B: every wave's mass, the drafter's logits of I, the next row's ids
    if (wave == 0) {
      // the row's sums, the gradient's factors, and the gradient at the tokens of I
      GradRow g{0.f, 0.f};
      RowSums w{kNegInf, kNegInf, 0.0, 0.0, 0.0};
      if (live) {
        w = wave_row_sums(s_q, lane < NW ? s_max[lane] : kNegInf, lane < NW ? s_sum[lane] : 0.0, a.invT, lane);
        if (w.m == kNegInf && lane == 0) set_error(a.err, SV_DERR_ROW);
      }
      const bool some = w.m > kNegInf;
      const double inv = some ? 1.0 / w.sum : 0.0, scale = some ? s_scale[b] : 0.0;
      if (some) g = grad_row(w.m0, w.s0, s_n[b].p0, readlane_d(w.fac, kPL + kTW) * inv, scale);
#pragma unroll 1
      for (int i = lane; i < a.k; i += kWave)
        s_q.g[i] = some ? (float)((s_q.e[i] * readlane_d(w.fac, kPL + i / kWave) * inv - s.p[i]) * scale) : 0.f;
      if (lane == 0) {
        s_g = g;
        s_r = w;
      }
    }
    // meanwhile: this row's marks go, the next row's tokens and marks come
    if (cur.id >= 0) clear_mark(b, cur.id);
    if (next) teacher_tokens<E>(a, f, sn, s_mark[b ^ 1], ti);
    lds_sync();  // C: the factors, the gradients of I, the next row's teacher and marks
    if (next && sn.dup) teacher_repeats(a, f, sn, ti);  // block-uniform
    const bool nlive = next && sn.live != 0;
    const __amdgpu_buffer_rsrc_t rs = row_range(nlive ? rn : r, nlive);
    char* out = static_cast<char*>(a.grad) + (int64_t)r * a.gb;
    const __amdgpu_buffer_rsrc_t ro = range_rsrc(out, (uint32_t)nfull * 16u);
    const GradRow g = s_g;
    if (wave == kLossWave) {
      const RowSums w = s_r;
      const bool some = w.m > kNegInf;
      double loss = 0.0;
      if (some)
        loss = wave_loss(s, s_q, a.k, a.rest ? (double)a.rest[r] : -__builtin_huge_val(), s_n[b], w, a.invT, lane);
      if (lane == 0) {
        a.out_loss[r] = (float)loss;
        reinterpret_cast<float4*>(a.out_stat)[r] =
            some ? make_float4(w.m, (float)w.sum, w.m0, (float)w.s0) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    z = kNegInf;
    float zt = 0.f;
    if (nlive) {
      if (f.id >= 0) z = load_elem<DT>(row_of(rn), f.id);
      if (tid < tail) zt = load_elem<DT>(row_of(rn), (int64_t)nfull * E + tid);
    }
    if (nlive && wave == kNextWave) teacher_probs(rn, b ^ 1);
    acc = Mass{};
    // store this row's gradient, load the next row behind it, and fold that
    // LAG vectors behind the loads
    const uint8_t* mark = reinterpret_cast<const uint8_t*>(s_mark[b ^ 1]);
    uint32_t off = off0;
    asm volatile("" : "+v"(off));  // the NV offsets are formed as they are used, not kept
#pragma unroll
    for (int i = 0; i < NV + LAG; ++i) {
      if (i < NV) {
        // the row stays packed: without this the compiler keeps the fold's
        // unpacked values alive beside it, twice the registers there are
        asm volatile("" : "+v"(d[i]));
        store_range(ro, off, grad_vec<DT>(d[i], g, a.c));
        d[i] = load_range(rs, off);
        off += NT * 16;
        __builtin_amdgcn_sched_barrier(0);
      }
      if (i >= LAG && (i - LAG) % FU == FU - 1) {
        if (nlive) fold(i - LAG - (FU - 1), mark);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (tid < tail) store_elem_alias<DT>(out, (int64_t)nfull * E + tid, grad_elem(ztail, g, a.c));
    // the tokens of I whose vectors this wave stored: a wave's stores to one
    // place stay in order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    for (int i = lane; i < a.k; i += kWave) {
      const int32_t id = s.id[i];
      // in the shorter last vector thread e stored element e
      const int owner = id / E < nfull ? id / E % NT : id - nfull * E;
      if (id >= 0 && owner / kWave == wave) store_elem_alias<DT>(out, id, s_q.g[i]);
    }
    if (!next) return;
    ztail = zt;
    cur.id = f.id;
    r = rn;
    b ^= 1;
    lds_sync();  // the tokens of I are stored: their row in LDS may be written again
  }
}

namespace {

template <int DT, int NT, int NV>
hipError_t launch_held(const DistillParams& p, hipStream_t s) {
  static std::atomic<int> cache[64];  // of any host thread
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  int cap = dev >= 0 && dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (cap == 0) {
    cap = device_capacity(reinterpret_cast<const void*>(&distill_held_kernel<DT, NT, NV>), NT, dev);
    if (cap <= 0) return hipErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) cache[dev].store(cap, std::memory_order_relaxed);
  }
  const unsigned grid = (unsigned)(p.R < cap ? p.R : cap);
  distill_held_kernel<DT, NT, NV><<<dim3(grid), dim3(NT), 0, s>>>(p);
  return hipGetLastError();
}

// The fewest vectors a thread, in steps of two, that hold the row: a place that
// holds nothing costs nearly as much as one that does (2000 bf16 rows of 34480
// logits, 4310 vectors: 81 us in 512 threads of 16, 67 of 10; of 20000: 50 us
// of 8, 44 of 6; 600 of 140000: 91 us in 1024 threads of 20, 88 of 18).
template <int DT, int NT, int NV, int MOST>
hipError_t launch_held_nv(const DistillParams& p, hipStream_t s) {
  if constexpr (NV < MOST)
    if (p.nvec > NT * NV) return launch_held_nv<DT, NT, NV + 2, MOST>(p, s);
  return launch_held<DT, NT, NV>(p, s);
}

template <int DT>
hipError_t launch_held_dt(const DistillParams& p, hipStream_t s) {
  if (p.nvec <= 256 * 8) return launch_held_nv<DT, 256, 4, 8>(p, s);
  if (p.nvec <= 512 * 16) return launch_held_nv<DT, 512, 6, 16>(p, s);
  static_assert(kHeldVecs == 1024 * 24, "the longest row");
  return launch_held_nv<DT, 1024, 10, 24>(p, s);
}

}  // namespace

hipError_t launch_distill_held(const DistillParams& p, sv_dtype dt, hipStream_t s) {
  return dt == SV_BF16 ? launch_held_dt<SV_BF16>(p, s) : launch_held_dt<SV_F32>(p, s);
}

}  // namespace sv
