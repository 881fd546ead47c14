// sv_beam.hip -- beam search on gfx950: one step's selection over beams and
// vocabulary, and the reordering of the beams' states that follows it.
#include "sv_draft.h"
#include "sv_topmass.hpp"

namespace sv {

// ---------------------------------------------------------------------------
// Selection.  A continuation (w, v) scores s_w + z_{w,v} / T - lse_w with
// lse_w = log sum_u exp(z_{w,u} / T); within a beam the order is that of the
// logits, so the N best of a sequence are among the N best of each beam.
//
// One launch: a block per (row part) finds the part's N best and the mass
// outside them (sv_topmass.hpp), in one read of the row; dead and finished
// beams' blocks read nothing.  The sequence's last block joins: a wave a beam
// merges the beam's parts, scores its list and merges that into the wave's
// running list; the waves' lists then merge pairwise.  A merge of two sorted
// lists, a lane an entry, is one exchange with the other list reversed and
// log2(N) compare-exchange steps (a bitonic merge), so the join takes a few
// steps more where there are more beams, not more rounds of a selection.
// 64 x 8 beams of 128256 bf16 logits, a tenth dead, 16 kept: 30 us, 3.9 TB/s
// (17 us of it the read): 512 blocks start at once, two to a compute unit, so
// their starts (flags and scores, then the first window, load after load),
// selections and joins come at the same time and nothing covers them.
// 1 x 4 beams of 32000: 12.6 us, latencies of the start, the pass, the hand-off
// and the join.
// Scores are formed and compared in 64 bits.  Within a beam the order is that
// of the list, by logit and then token, and the comparison goes by the place
// there: a score of large magnitude (-1e30 for a beam that is to lose) rounds
// every logit away, and the merges need lists that are sorted as they compare.
// ---------------------------------------------------------------------------
constexpr double kNoScore = -__builtin_huge_val();

// A continuation: lane l of a sorted list holds the l-th best.
struct Cont {
  double s;    // score (kNoScore: none)
  int32_t at;  // beam * kWave + place in the beam's list
  int32_t tok;
};
__device__ __forceinline__ bool cont_better(const Cont& a, const Cont& b) {
  return (a.s > b.s) | ((a.s == b.s) & (a.at < b.at));
}
__device__ __forceinline__ Cont cont_from(const Cont& c, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(c.s);
  const int at = lane * 4;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)(uint32_t)b);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)(uint32_t)(b >> 32));
  Cont r;
  r.s = __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
  r.at = __builtin_amdgcn_ds_bpermute(at, c.at);
  r.tok = __builtin_amdgcn_ds_bpermute(at, c.tok);
  return r;
}
// The P best of two sorted lists of P (a power of two <= 64; empty entries
// last), sorted.  y comes reversed: lane l holds entry P - 1 - l.
__device__ __forceinline__ Cont cont_merge(Cont x, const Cont& y, int P, int lane) {
  if (cont_better(y, x)) x = y;  // the P best, falling then rising
  for (int h = P / 2; h > 0; h /= 2) {
    const Cont o = cont_from(x, lane ^ h);
    const bool low = (lane & h) == 0;  // keeps the better of the two
    if (cont_better(o, x) == low) x = o;
  }
  return x;
}

template <int NW>
struct BeamLds {
  Cont list[NW][kWave];
  alignas(16) double merge[NW][kPartEntries];
  float scores[SV_MAX_BEAMS];
  int32_t finished[SV_MAX_BEAMS];
};

template <int DT, int NT>
__global__ __launch_bounds__(NT, 4) void beam_select_kernel(BeamParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  constexpr int NW = NT / kWave;
  __shared__ BeamLds<NW> lds;
  const int r = blockIdx.x / a.nch;  // row (b, w)
  const int ch = blockIdx.x - r * a.nch;
  const int b = r / a.W;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int N = a.N;
  const bool done = a.finished && a.finished[r] != 0;
  const bool live = !done && a.scores[r] > kNegInf;  // block-uniform
  if (threadIdx.x < (unsigned)a.W) {  // for the join, if it falls to this block
    lds.scores[threadIdx.x] = a.scores[(int64_t)b * a.W + threadIdx.x];
    lds.finished[threadIdx.x] = a.finished ? a.finished[(int64_t)b * a.W + threadIdx.x] : 0;
  }
  TopEntry* lists = static_cast<TopEntry*>(a.lists);
  Partial* parts = static_cast<Partial*>(a.parts);
  if (live) {
    const int64_t v0 = (int64_t)ch * a.vpc;
    const int64_t v1 = v0 + a.vpc < a.nvec ? v0 + a.vpc : a.nvec;
    Partial rest;
    const TopPair t =
        block_topk_mass<NT, E>(MassRow<DT>{row_ptr(a.logits, r, a.sb), a.V}, v0, v1, a.V, N, a.c, &rest);
    if (wave == 0) {
      const int64_t part = (int64_t)r * a.nch + ch;
      if (lane < N) put_entry(lists + part * N + lane, t.v, t.i);
      if (lane == 0) put_partial(parts + part, rest);
    }
  }
  if (!arrive_last<NT>(&a.cnt[b], (uint32_t)(a.W * a.nch))) return;
  int P = 1;
  while (P < N) P *= 2;
  const Cont none{kNoScore, -1, -1};
  Cont best = none;
  for (int w = wave; w < a.W; w += NW) {
    const int64_t row = (int64_t)b * a.W + w;
    const float sc = lds.scores[w];
    Cont own = none;
    if (!(sc > kNegInf)) continue;  // wave-uniform
    if (lds.finished[w] != 0) {
      if (lane == 0) own = Cont{(double)sc, w * kWave, a.pad};
    } else {
      float lv;
      int32_t li;
      const Partial rest = wave_merge_parts(lists + row * a.nch * N, parts + row * a.nch, a.nch, N, a.c, lane,
                                            lds.merge[wave], lv, li);
      // all of the row's mass: what its list holds and the rest
      const float m = fmaxf(rest.m, readlane_f(lv, 0));
      if (m > kNegInf) {
        const double s = wave_sum(lane < N ? rescale(lv, m, a.c) : 0.0) + rest.s * rescale(rest.m, m, a.c);
        const double shift = (double)sc - ((double)m * a.invT + log_d(s));
        if (lane < N && lv > kNegInf) own = Cont{shift + (double)lv * a.invT, w * kWave + lane, li};
      } else if (lane == 0) {
        set_error(a.err, SV_DERR_ROW);
      }
    }
    best = w == wave ? own : cont_merge(best, cont_from(own, lane ^ (P - 1)), P, lane);
  }
  // the waves' lists, in pairs; a wave past the beams has an empty one
  for (int d = 1; d < NW && d < a.W; d *= 2) {
    if ((wave & (2 * d - 1)) == d) lds.list[wave][lane] = best;
    lds_sync();
    if ((wave & (2 * d - 1)) == 0 && wave + d < a.W)
      best = cont_merge(best, lds.list[wave + d][lane ^ (P - 1)], P, lane);
  }
  if (wave != 0) return;
  if (lane < N) {
    a.out_beam[(int64_t)b * N + lane] = best.s > kNoScore ? best.at / kWave : -1;
    a.out_tok[(int64_t)b * N + lane] = best.s > kNoScore ? best.tok : -1;
    a.out_score[(int64_t)b * N + lane] = (float)best.s;
  }
  if (lane == 0) __hip_atomic_store(&a.cnt[b], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int DT>
static void launch_beam_dt(const BeamParams& p, hipStream_t s) {
  const int64_t grid = (int64_t)p.B * p.W * p.nch;
  if (grid > kTopWide)
    beam_select_kernel<DT, 256><<<dim3((unsigned)grid), dim3(256), 0, s>>>(p);
  else
    beam_select_kernel<DT, 512><<<dim3((unsigned)grid), dim3(512), 0, s>>>(p);
}

hipError_t launch_beam(const BeamParams& p, sv_dtype dt, hipStream_t s) {
  if (dt == SV_BF16)
    launch_beam_dt<SV_BF16>(p, s);
  else
    launch_beam_dt<SV_F32>(p, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Reordering.  A thread owns one place of a segment for all N beams of a
// sequence: it loads the N pieces from their parents, then stores them.  No
// other thread touches that place, so the same kernel works in place (all
// loads of a thread come before its stores).  A source that several beams
// follow is loaded by the same thread, from the cache after the first time.
// Memory-bound: every source once, every moved beam once.  A thread looks its
// parents up again for each load and each store, which other threads' work
// hides in a large state; a small one (32 x 8 x 513 int32: 7.7 us) is that chain.
//
// Places are of U bytes, at any alignment (unaligned vector accesses are
// native; beams of a ragged cache rarely share one), and the last bytes of a
// segment are places of 4 bytes and of one, each a thread's.  U is 16 unless
// more than 16 beams in place would have to be held at once.
//
// A state larger than the last-level cache is stored past it (NTS: 2.1 GB in
// place 506 -> 484 us, 4.9 TB/s of reads and writes; 439 MB 99 -> 78 us; the
// time goes with how many beams follow themselves: 372 to 537 us); a
// smaller one stays there for its next reader (275 MB: 50 us, 55 past it).
// ---------------------------------------------------------------------------
template <int U>
struct Bytes;
template <>
struct Bytes<16> {
  typedef u32x4 T __attribute__((aligned(1), may_alias));
};
template <>
struct Bytes<8> {
  typedef uint64_t T __attribute__((aligned(1), may_alias));
};
template <>
struct Bytes<4> {
  typedef uint32_t T __attribute__((aligned(1), may_alias));
};
template <>
struct Bytes<1> {
  typedef uint8_t T __attribute__((may_alias));
};

constexpr int kRNT = kReorderThreads;

// One place of U bytes for all beams.
template <int U, int MAXN, bool NTS>
__device__ __forceinline__ void reorder_place(const ReorderParams& a, const char* src, char* dst, const int32_t* parent) {
  using T = typename Bytes<U>::T;
  for (int n0 = 0; n0 < a.N; n0 += MAXN) {  // in place: one round (N <= MAXN)
    T v[MAXN];
#pragma unroll
    for (int i = 0; i < MAXN; ++i) {
      const int n = n0 + i;
      const int32_t p = n < a.N ? parent[n] : -1;
      if (p >= 0 && p < a.W && !(a.inplace && p == n)) v[i] = *reinterpret_cast<const T*>(src + (int64_t)p * a.ss[2]);
    }
#pragma unroll
    for (int i = 0; i < MAXN; ++i) {
      const int n = n0 + i;
      const int32_t p = n < a.N ? parent[n] : -1;
      if (p >= 0 && p < a.W && !(a.inplace && p == n)) {
        T* to = reinterpret_cast<T*>(dst + (int64_t)n * a.ds[2]);
        if constexpr (NTS)
          __builtin_nontemporal_store(v[i], to);
        else
          *to = v[i];
      }
    }
  }
}

template <int U, int MAXN, bool NTS>
__global__ __launch_bounds__(kRNT) void reorder_kernel(ReorderParams a, int64_t nblk) {
  // block -> (layer, sequence, segment, chunk)
  int64_t q = blockIdx.x;
  const int64_t chunk = q % nblk;
  q /= nblk;
  const int h = (int)(q % a.H);
  q /= a.H;
  const int b = (int)(q % a.B);
  const int64_t l = q / a.B;
  int64_t len = a.lens ? (int64_t)a.lens[b] : a.S;
  const int32_t* parent = a.parent + (int64_t)b * a.N;
  if (chunk == 0 && h == 0 && l == 0) {
    if (threadIdx.x < a.N) {
      const int32_t p = parent[threadIdx.x];
      if (p < -1 || p >= a.W) set_error(a.err, SV_DERR_RANGE);
    }
    if (threadIdx.x == 0 && (len < 0 || len > a.S)) set_error(a.err, SV_DERR_RANGE);
  }
  if (len < 0 || len > a.S) return;
  const int64_t bytes = len * a.pos;
  const char* src = a.src + l * a.ss[0] + (int64_t)b * a.ss[1] + (int64_t)h * a.ss[3];
  char* dst = a.dst + l * a.ds[0] + (int64_t)b * a.ds[1] + (int64_t)h * a.ds[3];
  const int64_t j = chunk * kRNT + threadIdx.x;
  const int64_t nu = bytes / U;
  const int64_t n4 = bytes % U / 4;
  if (j < nu)
    reorder_place<U, MAXN, NTS>(a, src + j * U, dst + j * U, parent);
  else if (j < nu + n4)
    reorder_place<4, MAXN, false>(a, src + nu * U + (j - nu) * 4, dst + nu * U + (j - nu) * 4, parent);
  else if (j < nu + n4 + bytes % 4)
    reorder_place<1, MAXN, false>(a, src + bytes / 4 * 4 + (j - nu - n4), dst + bytes / 4 * 4 + (j - nu - n4), parent);
}

constexpr double kPastCache = 320.0 * (1 << 20);  // bytes of a state that the 256 MB cache no longer serves

template <int U, int MAXN>
static hipError_t launch_reorder_u(const ReorderParams& p, hipStream_t s) {
  const int64_t nblk = reorder_blocks(p.S * p.pos, U);
  const int64_t grid = nblk * p.L * p.B * p.H;
  if (grid > kReorderMostBlocks) return hipErrorInvalidValue;
  if ((double)p.L * p.B * p.N * p.H * p.S * p.pos > kPastCache)
    reorder_kernel<U, MAXN, true><<<dim3((unsigned)grid), dim3(kRNT), 0, s>>>(p, nblk);
  else
    reorder_kernel<U, MAXN, false><<<dim3((unsigned)grid), dim3(kRNT), 0, s>>>(p, nblk);
  return hipGetLastError();
}

hipError_t launch_reorder(const ReorderParams& p, hipStream_t s) {
  switch (reorder_unit(p.N, p.inplace)) {
    case 16: return p.N <= 8 ? launch_reorder_u<16, 8>(p, s) : launch_reorder_u<16, 16>(p, s);
    case 8: return launch_reorder_u<8, 32>(p, s);
    default: return launch_reorder_u<4, 64>(p, s);
  }
}

}  // namespace sv
