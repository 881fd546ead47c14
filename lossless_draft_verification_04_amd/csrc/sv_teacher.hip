// sv_teacher.hip -- the verifier's top logits and the mass outside them, a
// distillation target per row, on gfx950.
//
// Per row: the k largest logits (value descending, index ascending) and
// rest = log sum over the others of exp(z / T), natural logarithm.  A read of
// each row bounds it from below; the work beside it is one exponential (a
// quarter-rate instruction), its argument, a maximum and an addition a logit,
// more than half of the vector unit's time at the memory's rate.
//
// One launch: a block per (row part).  The block finds its part's list and
// the mass outside it (sv_topmass.hpp); a row in one part is written by its
// block, otherwise the row's last block merges the parts: what a part listed
// and the row does not is counted back into the mass.
//
// 2048 x 151936 bf16 rows, 64 values that no two stand in one thread's share:
// 106 us, 5.85 TB/s (a plain read reaches 7.1); what is missing is a block's
// start (a window whose loads wait for each other) and the selection at its
// end, which only the other blocks of a compute unit cover.  Unordered rows
// have some 7 threads with two of the 64, whose vectors are read again: 137 us.
// 17 x 32000 fp32 rows, 8 values: 10 us, a chain of latencies (four loads,
// bound, candidates, ranks, stores).
#include "sv_draft.h"
#include "sv_topmass.hpp"

namespace sv {

__device__ __forceinline__ void put_target(const TeacherParams& a, int r, int lane, float lv, int32_t li,
                                           const Partial& rest) {
  if (lane < a.k) {
    a.out_ids[(int64_t)r * a.k + lane] = li != kNoIdx ? li : -1;
    a.out_vals[(int64_t)r * a.k + lane] = li != kNoIdx ? lv : kNegInf;
  }
  if (lane == 0) a.out_rest[r] = rest.s > 0.0 ? (float)((double)rest.m * a.invT + log(rest.s)) : kNegInf;
}

template <int DT, int NT>
__global__ __launch_bounds__(NT, 4) void teacher_kernel(TeacherParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  const int r = blockIdx.x / a.nch;
  const int ch = blockIdx.x - r * a.nch;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int64_t v0 = (int64_t)ch * a.vpc;
  const int64_t v1 = v0 + a.vpc < a.nvec ? v0 + a.vpc : a.nvec;
  __shared__ alignas(16) double s_merge[kPartEntries];
  Partial rest;
  const TopPair t =
      block_topk_mass<NT, E>(MassRow<DT>{row_ptr(a.logits, r, a.sb), a.V}, v0, v1, a.V, a.k, a.c, &rest);
  if (a.nch == 1) {
    if (wave == 0) put_target(a, r, lane, t.v, t.i, rest);
    return;
  }
  TopEntry* lists = static_cast<TopEntry*>(a.lists) + (int64_t)r * a.nch * a.k;
  Partial* parts = static_cast<Partial*>(a.parts) + (int64_t)r * a.nch;
  if (wave == 0) {
    if (lane < a.k) put_entry(lists + (int64_t)ch * a.k + lane, t.v, t.i);
    if (lane == 0) put_partial(parts + ch, rest);
  }
  if (!arrive_last<NT>(&a.cnt[r], (uint32_t)a.nch)) return;
  if (wave == 0) {
    float lv;
    int32_t li;
    const Partial whole = wave_merge_parts(lists, parts, a.nch, a.k, a.c, lane, s_merge, lv, li);
    put_target(a, r, lane, lv, li, whole);
    if (lane == 0) __hip_atomic_store(&a.cnt[r], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

template <int DT>
static void launch_teacher_dt(const TeacherParams& p, hipStream_t s) {
  const int64_t grid = (int64_t)p.R * p.nch;
  if (grid > kTopWide)
    teacher_kernel<DT, 256><<<dim3((unsigned)grid), dim3(256), 0, s>>>(p);
  else
    teacher_kernel<DT, 512><<<dim3((unsigned)grid), dim3(512), 0, s>>>(p);
}

hipError_t launch_teacher(const TeacherParams& p, sv_dtype dt, hipStream_t s) {
  if (dt == SV_BF16)
    launch_teacher_dt<SV_BF16>(p, s);
  else
    launch_teacher_dt<SV_F32>(p, s);
  return hipGetLastError();
}

}  // namespace sv
