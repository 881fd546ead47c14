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
// beams' blocks read nothing.  The sequence's last block merges each beam's
// parts (a wave per beam) and then the beams: up to 512 candidates by a
// thread each, which counts the better ones; more by one wave that holds the
// head of every sorted list, a lane a beam, and takes the best head N times
// (64 beams of 64: 64 steps where counting would compare 4096 x 4096).  Scores are formed and compared in 64 bits: differences between
// beams near 1e-7 of a score decide as the inputs have it.
// ---------------------------------------------------------------------------
constexpr int kBNT = 512;

struct BeamLds {
  TopEntry list[SV_MAX_BEAMS * SV_MAX_FANOUT];
  double shift[SV_MAX_BEAMS];  // s_w - lse_w; -inf: no continuation
  uint64_t merge[kBNT / kWave][kPartEntries];
};

// The order of doubles as unsigned integers (larger = better; -inf lowest of
// the values, 0 below all).
__device__ __forceinline__ uint64_t double_key(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ uint64_t wave_key_max(uint64_t k) {
  key_max_step<kRowShr + 1, 0xF>(k);
  key_max_step<kRowShr + 2, 0xF>(k);
  key_max_step<kRowShr + 4, 0xF>(k);
  key_max_step<kRowShr + 8, 0xF>(k);
  key_max_step<kRowBcast15, 0xA>(k);
  key_max_step<kRowBcast31, 0xC>(k);
  return readlane_u64(k, kWave - 1);
}

template <int DT>
__global__ __launch_bounds__(kBNT, 4) void beam_select_kernel(BeamParams a) {
  constexpr int E = Fmt<DT>::kPerVec;
  __shared__ BeamLds lds;
  const int r = blockIdx.x / a.nch;  // row (b, w)
  const int ch = blockIdx.x - r * a.nch;
  const int b = r / a.W;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int N = a.N;
  const bool done = a.finished && a.finished[r] != 0;
  const bool live = !done && a.scores[r] > kNegInf;  // block-uniform
  TopEntry* lists = static_cast<TopEntry*>(a.lists);
  Partial* parts = static_cast<Partial*>(a.parts);
  if (live) {
    const int64_t v0 = (int64_t)ch * a.vpc;
    const int64_t v1 = v0 + a.vpc < a.nvec ? v0 + a.vpc : a.nvec;
    Partial rest;
    const TopPair t =
        block_topk_mass<kBNT, E>(MassRow<DT>{row_ptr(a.logits, r, a.sb), a.V}, v0, v1, a.V, N, a.c, &rest);
    if (wave == 0) {
      const int64_t part = (int64_t)r * a.nch + ch;
      if (lane < N) put_entry(lists + part * N + lane, t.v, t.i);
      if (lane == 0) put_partial(parts + part, rest);
    }
  }
  if (!arrive_last<kBNT>(&a.cnt[b], (uint32_t)(a.W * a.nch))) return;
  // every beam's list and normaliser, a wave a beam
  for (int w = wave; w < a.W; w += kBNT / kWave) {
    const int64_t row = (int64_t)b * a.W + w;
    const bool fin = a.finished && a.finished[row] != 0;
    const float sc = a.scores[row];
    float lv = kNegInf;
    int32_t li = kNoIdx;
    double shift = -__builtin_huge_val();
    if (sc > kNegInf) {
      if (fin) {
        if (lane == 0) {
          lv = 0.f;
          li = a.pad;
        }
        shift = (double)sc;
      } else {
        const Partial rest = wave_merge_parts(lists + row * a.nch * N, parts + row * a.nch, a.nch, N, a.c, lane,
                                              lds.merge[wave], lv, li);
        // all of the row's mass: what its list holds and the rest
        const float m = fmaxf(rest.m, readlane_f(lv, 0));
        if (m > kNegInf) {
          const double s = wave_sum(lane < N ? rescale(lv, m, a.c) : 0.0) + rest.s * rescale(rest.m, m, a.c);
          shift = (double)sc - ((double)m * a.invT + log_d(s));
        } else if (lane == 0) {
          set_error(a.err, SV_DERR_ROW);
        }
      }
    }
    if (lane < N) lds.list[w * SV_MAX_FANOUT + lane] = TopEntry{lv, li};
    if (lane == 0) lds.shift[w] = shift;
  }
  lds_sync();
  constexpr double kNone = -__builtin_huge_val();
  // score of beam w's p-th candidate (-inf: none)
  auto score_of = [&](int w, int p) -> double {
    const double shift = lds.shift[w];
    const TopEntry t = lds.list[w * SV_MAX_FANOUT + p];
    if (!(shift > kNone) || t.val == kNegInf) return kNone;
    return shift + (double)t.val * a.invT;
  };
  const int n = a.W * N;
  if (n <= kBNT) {
    // a thread a candidate: its place is the number of better ones, earlier
    // ones first where scores tie
    uint64_t* keys = lds.merge[0];
    int* slot = reinterpret_cast<int*>(lds.merge[kBNT / kPartEntries]);
    const int i = threadIdx.x;
    const int w = i / N;
    const double sc = i < n ? score_of(w, i - w * N) : kNone;
    const uint64_t k = sc > kNone ? double_key(sc) : 0ull;
    keys[i] = k;
    if (i < N) slot[i] = -1;
    lds_sync();
    int above = 0;
    if ((i & ~(kWave - 1)) < n)
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const uint64_t o = keys[j];
        above += (o > k) | ((o == k) & (j < i)) ? 1 : 0;
      }
    if (k != 0ull && above < N) {
      slot[above] = i;
      a.out_score[(int64_t)b * N + above] = (float)sc;
    }
    lds_sync();
    if (i < N) {
      const int at = slot[i];
      a.out_beam[(int64_t)b * N + i] = at >= 0 ? at / N : -1;
      a.out_tok[(int64_t)b * N + i] = at >= 0 ? lds.list[at / N * SV_MAX_FANOUT + at % N].idx : -1;
      if (at < 0) a.out_score[(int64_t)b * N + i] = kNegInf;
    }
  } else if (wave == 0) {
    // a lane a beam: the best head of the sorted lists, N times
    int pos = 0;
    double cur = lane < a.W ? score_of(lane, 0) : kNone;
    int32_t ob = -1, ot = -1;
    float os = kNegInf;
    for (int m = 0; m < N; ++m) {
      const uint64_t k = cur > kNone ? double_key(cur) : 0ull;
      const uint64_t best = wave_key_max(k);
      if (best == 0ull) break;
      const int win = __builtin_ctzll(__ballot(k == best));  // ties: the lowest beam
      const int p = __builtin_amdgcn_readlane(pos, win);
      const double sc = readlane_d(cur, win);
      if (lane == m) {
        ob = win;
        ot = lds.list[win * SV_MAX_FANOUT + p].idx;
        os = (float)sc;
      }
      if (lane == win) {
        ++pos;
        cur = pos < N ? score_of(lane, pos) : kNone;
      }
    }
    if (lane < N) {
      a.out_beam[(int64_t)b * N + lane] = ob;
      a.out_tok[(int64_t)b * N + lane] = ot;
      a.out_score[(int64_t)b * N + lane] = os;
    }
  }
  if (threadIdx.x == 0) __hip_atomic_store(&a.cnt[b], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

hipError_t launch_beam(const BeamParams& p, sv_dtype dt, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.B * p.W * p.nch));
  if (dt == SV_BF16)
    beam_select_kernel<SV_BF16><<<grid, dim3(kBNT), 0, s>>>(p);
  else
    beam_select_kernel<SV_F32><<<grid, dim3(kBNT), 0, s>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Reordering.  A thread owns one vector of U bytes at one place of a segment,
// for all N beams of a sequence: it loads the N vectors from their parents,
// then stores them.  No other thread touches that place, so the same kernel
// works in place (all loads of a thread come before its stores).  A source
// that several beams follow is loaded by the same thread, from the cache
// after the first time.  Memory-bound: every source once, every moved beam
// once.
// ---------------------------------------------------------------------------
template <int U>
struct Bytes;
template <>
struct Bytes<16> {
  using T = u32x4;
};
template <>
struct Bytes<8> {
  using T = uint64_t;
};
template <>
struct Bytes<4> {
  using T = uint32_t;
};
template <>
struct Bytes<2> {
  using T = uint16_t;
};
template <>
struct Bytes<1> {
  using T = uint8_t;
};

constexpr int kRNT = 256;

template <int U, int MAXN>
__global__ __launch_bounds__(kRNT) void reorder_kernel(ReorderParams a, int64_t nblk) {
  using T = typename Bytes<U>::T;
  // block -> (layer, sequence, segment, chunk)
  int64_t q = blockIdx.x;
  const int64_t chunk = q % nblk;
  q /= nblk;
  const int h = (int)(q % a.H);
  q /= a.H;
  const int b = (int)(q % a.B);
  const int64_t l = q / a.B;
  int64_t len = a.lens ? (int64_t)a.lens[b] : a.S;
  if (len < 0 || len > a.S) {
    if (threadIdx.x == 0 && chunk == 0 && h == 0 && l == 0) set_error(a.err, SV_DERR_RANGE);
    len = 0;
  }
  const int64_t bytes = len * a.pos;
  const int64_t off = (chunk * kRNT + threadIdx.x) * U;
  const char* src = a.src + l * a.ss[0] + (int64_t)b * a.ss[1] + (int64_t)h * a.ss[3] + off;
  char* dst = a.dst + l * a.ds[0] + (int64_t)b * a.ds[1] + (int64_t)h * a.ds[3] + off;
  const int32_t* parent = a.parent + (int64_t)b * a.N;
  if (chunk == 0 && h == 0 && l == 0 && threadIdx.x < a.N) {
    const int32_t p = parent[threadIdx.x];
    if (p < -1 || p >= a.W) set_error(a.err, SV_DERR_RANGE);
  }
  if (off >= bytes) return;
  const bool whole = off + U <= bytes;
  for (int n0 = 0; n0 < a.N; n0 += MAXN) {  // in place: one round (N <= MAXN)
    T v[MAXN];
#pragma unroll
    for (int i = 0; i < MAXN; ++i) {
      const int n = n0 + i;
      if (n < a.N) {
        const int32_t p = parent[n];
        if (p >= 0 && p < a.W && !(a.inplace && p == n) && whole)
          v[i] = *reinterpret_cast<const T*>(src + (int64_t)p * a.ss[2]);
      }
    }
#pragma unroll
    for (int i = 0; i < MAXN; ++i) {
      const int n = n0 + i;
      if (n < a.N) {
        const int32_t p = parent[n];
        if (p >= 0 && p < a.W && !(a.inplace && p == n) && whole)
          *reinterpret_cast<T*>(dst + (int64_t)n * a.ds[2]) = v[i];
      }
    }
  }
  if (!whole) {
    // the last bytes of a segment whose length is no multiple of U, a byte
    // of all beams at a time
    for (int64_t j = 0; off + j < bytes; ++j) {
      for (int n0 = 0; n0 < a.N; n0 += MAXN) {
        uint8_t v[MAXN];
#pragma unroll
        for (int i = 0; i < MAXN; ++i) {
          const int n = n0 + i;
          const int32_t p = n < a.N ? parent[n] : -1;
          if (p >= 0 && p < a.W) v[i] = *reinterpret_cast<const uint8_t*>(src + (int64_t)p * a.ss[2] + j);
        }
#pragma unroll
        for (int i = 0; i < MAXN; ++i) {
          const int n = n0 + i;
          const int32_t p = n < a.N ? parent[n] : -1;
          if (p >= 0 && p < a.W) *reinterpret_cast<uint8_t*>(dst + (int64_t)n * a.ds[2] + j) = v[i];
        }
      }
    }
  }
}

template <int U>
static hipError_t launch_reorder_u(const ReorderParams& p, hipStream_t s) {
  const int64_t bytes = p.S * p.pos;
  const int64_t nblk = (bytes + (int64_t)U * kRNT - 1) / ((int64_t)U * kRNT);
  const int64_t grid = nblk * p.L * p.B * p.H;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const dim3 g((unsigned)grid);
  // in place every beam's vector is held at once
  if (p.N <= 8)
    reorder_kernel<U, 8><<<g, dim3(kRNT), 0, s>>>(p, nblk);
  else if (p.N <= 16 || !p.inplace)
    reorder_kernel<U, 16><<<g, dim3(kRNT), 0, s>>>(p, nblk);
  else if constexpr (U <= 8) {
    if (p.N <= 32)
      reorder_kernel<U, 32><<<g, dim3(kRNT), 0, s>>>(p, nblk);
    else if constexpr (U <= 4)
      reorder_kernel<U, 64><<<g, dim3(kRNT), 0, s>>>(p, nblk);
    else
      return launch_reorder_u<4>(p, s);
  } else {
    return launch_reorder_u<8>(p, s);
  }
  return hipGetLastError();
}

hipError_t launch_reorder(const ReorderParams& p, int vec, hipStream_t s) {
  switch (vec) {
    case 16: return launch_reorder_u<16>(p, s);
    case 8: return launch_reorder_u<8>(p, s);
    case 4: return launch_reorder_u<4>(p, s);
    case 2: return launch_reorder_u<2>(p, s);
    default: return launch_reorder_u<1>(p, s);
  }
}

}  // namespace sv
