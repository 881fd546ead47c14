// sv_topmass.hpp -- a block's top-F values of a range of 16-byte vectors and
// the mass (sum of exponentials) outside them, in one pass over the range.
// Shared by the teacher's pass and beam search.
//
// The selection is that of sv_topk.hpp: each thread keeps its best vector, a
// bound from groups of threads, candidates in LDS.  The mass is summed beside
// it so that no listed value ever enters a sum: a thread folds every vector
// but its best one (a new best vector sends the old one into the sum), and
// once the F-th best key is known adds what its best vector holds below it.
// Only a thread that owns a listed value outside its best vector has its sum
// dropped and its vectors read again, spread over its wave.  So the mass
// keeps full relative precision however little of it there is, where a
// difference "all minus the top" would keep none.
#pragma once

#include "sv_device.hpp"
#include "sv_topk.hpp"

namespace sv {

// A sum of exponentials: sum of 2^(c (x - m)), m the largest x (-inf, 0: of
// nothing).
struct Mass {
  float m = kNegInf;
  float s = 0.f;
};

// a <- a + the E values x (-inf: nothing).  The shift is m, as fma(x, c, -c m);
// where c m is not finite (rows masked with the type's lowest value), as
// (x - m) c; SUB: always so (no branch, an operation more a value).
template <int E, bool SUB = false>
__device__ __forceinline__ void fold_values(const float (&x)[E], float c, Mass& a) {
  float fm = x[0];
#pragma unroll
  for (int e = 1; e < E; ++e) fm = fmaxf(fm, x[e]);
  const float mn = fmaxf(a.m, fm);
  const float ref = mn == kNegInf ? 0.f : mn;
  const float cm = c * ref;
  float t[E];
  if (!SUB && __builtin_expect(fabsf(cm) <= 3e38f, 1)) {
#pragma unroll
    for (int e = 0; e < E; ++e) t[e] = fast_exp2(__builtin_fmaf(x[e], c, -cm));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) t[e] = fast_exp2((x[e] - ref) * c);
  }
#pragma unroll
  for (int w = E / 2; w > 0; w >>= 1)
#pragma unroll
    for (int e = 0; e < w; ++e) t[e] += t[e + w];
  a.s = __builtin_fmaf(a.s, fast_exp2((a.m - ref) * c), t[0]);
  a.m = mn;
}

// 2^(c (a - b)) for a merge of sums, a <= b; 0 for a = -inf.
__device__ __forceinline__ double rescale(float a, float b, float c) {
  return a == kNegInf ? 0.0 : exp2_d((double)c * ((double)a - (double)b));
}

// The block's sum of its threads' masses, in every thread.
template <int NT>
__device__ Partial block_mass(const Mass& a, float c) {
  Partial p;
  p.pad = 0.f;
  p.m = block_fmax<NT>(a.m);
  p.s = block_sum<NT>(a.m == kNegInf ? 0.0 : (double)a.s * (double)fast_exp2((a.m - p.m) * c));
  return p;
}

// Values of vector v below the key kth, the others -inf.
template <int E, class Src>
__device__ __forceinline__ void values_below(const Src& src, const typename Src::Data& d, int64_t v, uint64_t kth,
                                             float (&x)[E]) {
  src.values(d, v, x);
  const int32_t i0 = (int32_t)(v * E);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (top_key(x[e], i0 + e) >= kth) x[e] = kNegInf;
}

// As block_topk (wave 0 returns the list of the range's F best), and mass =
// this thread's share of the sum over the range's other values.  F >= 1.
template <int NT, int E, class Src>
__device__ __forceinline__ TopPair block_topk_mass(const Src src, int64_t v0, int64_t v1, int V, int F, float c,
                                                   Mass* mass) {
  constexpr int kWin = 4;  // vectors in flight per thread
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int tid = threadIdx.x;
  __shared__ uint64_t s_cand[kCand];
  __shared__ uint32_t s_gm[NT];
  __shared__ uint64_t s_key[kCand];
  __shared__ uint64_t s_sel[kWave];
  __shared__ uint64_t s_tau;
  __shared__ int s_nc;
  float lv = kNegInf;
  int32_t li = kNoIdx;
  const int64_t span = v1 - v0;
  const int64_t nk = span > 0 ? (span + NT - 1) / NT : 0;  // vectors per thread at most
  const bool held = nk <= kWin;                            // block-uniform: every vector stays in registers
  float bm = kNegInf;    // the best vector's largest value, offset and data
  int32_t bo = kNoIdx;
  typename Src::Data bd{};
  bool more = false;     // the thread owns vectors besides its best one
  Mass rest;             // their mass; rest.m is their largest value
  typename Src::Data d[kWin];
#pragma unroll
  for (int u = 0; u < kWin; ++u) {
    const int64_t a = v0 + tid + (int64_t)u * NT;
    if (a < v1) d[u] = src.load(a);
  }
  if (held) {
#pragma unroll
    for (int u = 0; u < kWin; ++u) {
      const int64_t vu = v0 + tid + (int64_t)u * NT;
      if (vu < v1) {
        float x[E];
        src.values(d[u], vu, x);
        float vm = x[0];
#pragma unroll
        for (int e = 1; e < E; ++e) vm = fmaxf(vm, x[e]);
        const int32_t o = (int32_t)(vu - v0);
        const bool t = (bo == kNoIdx) | top_better(vm, o, bm, bo);
        bm = t ? vm : bm;
        bo = t ? o : bo;
      }
    }
  } else {
    for (int64_t v = v0 + tid; v < v1; v += (int64_t)kWin * NT) {
      typename Src::Data nx[kWin];
#pragma unroll
      for (int u = 0; u < kWin; ++u) {
        const int64_t a = v + (int64_t)(kWin + u) * NT;
        if (a < v1) nx[u] = src.load(a);
      }
#pragma unroll
      for (int u = 0; u < kWin; ++u) {
        const int64_t vu = v + (int64_t)u * NT;
        if (vu < v1) {
          float x[E];
          src.values(d[u], vu, x);
          float vm = x[0];
#pragma unroll
          for (int e = 1; e < E; ++e) vm = fmaxf(vm, x[e]);
          const int32_t o = (int32_t)(vu - v0);
          if (bo == kNoIdx) {
            bm = vm;
            bo = o;
            bd = d[u];
          } else {
            const bool t = top_better(vm, o, bm, bo);
            typename Src::Data f = d[u];
            int32_t fo = o;
            if (t) {
              f = bd;
              fo = bo;
              bm = vm;
              bo = o;
              bd = d[u];
            }
            src.values(f, v0 + fo, x);
            fold_values<E>(x, c, rest);
            more = true;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kWin; ++u) d[u] = nx[u];
    }
  }
  // the bound tau from below on the F-th best key (see block_topk)
  const uint64_t tkey = bo == kNoIdx ? 0ull : top_key(bm, (int32_t)((v0 + bo) * E));
  constexpr int kMaxH = NT / kWave;
  static_assert(kMaxH >= 1 && kMaxH <= 16 && kMaxH * kWave == NT, "whole waves, at most 16");
  int H = 1;
  while (H < kMaxH && 8 * F > kWave * H) H *= 2;  // block-uniform
  const int GS = NT / (kWave * H);
  {
    uint64_t k = tkey;
    if (GS >= 2) key_max_step<kRowShr + 1, 0xF>(k);
    if (GS >= 4) key_max_step<kRowShr + 2, 0xF>(k);
    if (GS >= 8) key_max_step<kRowShr + 4, 0xF>(k);
    if (GS >= 16) key_max_step<kRowShr + 8, 0xF>(k);
    if ((lane & (GS - 1)) == GS - 1) s_gm[tid / GS] = (uint32_t)(k >> 32);  // 0: the group holds nothing
  }
  if (tid == 0) s_nc = 0;
  lds_sync();
  if (wave == 0) {
    uint32_t p = 0;
    uint32_t gh[kMaxH];
#pragma unroll
    for (int h = 0; h < kMaxH; ++h) gh[h] = h < H ? s_gm[h * kWave + lane] : 0u;
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t q = p | (1u << bit);
      int cnt = 0;
#pragma unroll
      for (int h = 0; h < kMaxH; ++h) cnt += __builtin_popcountll(__ballot(gh[h] >= q));
      if (cnt >= F) p = q;
    }
    if (lane == 0) s_tau = (uint64_t)p << 32;
  }
  lds_sync();
  uint64_t tau = s_tau;
  // the thread's vectors besides its best may hold a key of at least t
  auto others_reach = [&](uint64_t t) { return more && top_key(rest.m, (int32_t)((v0 + tid) * E)) >= t; };
  // f(vs, d) for every vector of the wave's lanes with `pick`, one per lane at
  // a time (vs < 0: none); bo of its owner is passed on
  auto spread = [&](bool pick, auto&& f) {
    const uint64_t fm = __ballot(pick);
    if (!fm) return;  // wave-uniform
    const int nkk = (int)nk;
    const int items = __builtin_popcountll(fm) * nkk;
    for (int base = 0; base < items; base += kWave) {
      const int t = base + lane;
      const int j = t < items ? t / nkk : -1;
      int sl = 0;  // the j-th such lane of the wave
      uint64_t m = fm;
      for (int q = 0; m; ++q) {
        const int bl = __builtin_ctzll(m);
        m &= m - 1;
        sl = j == q ? bl : sl;
      }
      const int32_t sbo = __shfl(bo, sl, kWave);
      int64_t vs = -1;
      if (j >= 0) {
        const int64_t r = (int64_t)(wave * kWave + sl) + (int64_t)(t - j * nkk) * NT;
        if (r < span) vs = v0 + r;
      }
      typename Src::Data dd{};
      if (vs >= 0) dd = src.load(vs);
      f(vs, sbo, dd);
    }
  };
  int nc;
  for (;;) {  // block-uniform; tau rises on every repetition
    const bool sel = tkey != 0ull && tkey >= tau;
    if (held) {
#pragma unroll
      for (int u = 0; u < kWin; ++u) {
        const int64_t vu = v0 + tid + (int64_t)u * NT;
        flag_candidates<E>(src, d[u], sel && vu < v1 ? vu : -1, V, tau, s_cand, &s_nc);
      }
    } else {
      const bool full = sel && others_reach(tau);
      flag_candidates<E>(src, bd, sel && !full ? v0 + bo : -1, V, tau, s_cand, &s_nc);
      spread(full, [&](int64_t vs, int32_t, const typename Src::Data& dd) {
        flag_candidates<E>(src, dd, vs, V, tau, s_cand, &s_nc);
      });
    }
    lds_sync();
    nc = s_nc;
    if (nc <= kCand) break;
    tau = block_select<NT>(s_cand, s_key, s_sel, kCand, F, &s_tau);
    if (tid == 0) s_nc = 0;
    lds_sync();
  }
  if (nc <= kWave) {  // block-uniform
    if (wave == 0) {
      wave_rank(s_cand, nc, F, lane, lv, li);
      if (lane == F - 1) s_tau = li == kNoIdx ? 0ull : top_key(lv, li);
    }
    lds_sync();
  } else {
    block_select<NT>(s_cand, s_key, s_sel, nc, F, &s_tau);
    if (wave == 0 && lane < F) {
      lv = cand_value(s_sel[lane]);
      li = (int32_t)(s_sel[lane] >> 32);
    }
  }
  // the F-th best key; 0 where fewer are listed, which then are all there are
  const uint64_t kth = s_tau;
  float x[E];
  if (held) {
    Mass a;
#pragma unroll
    for (int u = 0; u < kWin; ++u) {
      const int64_t vu = v0 + tid + (int64_t)u * NT;
      if (vu < v1) {
        values_below<E>(src, d[u], vu, kth, x);
        fold_values<E>(x, c, a);
      }
    }
    *mass = a;
  } else {
    const bool redo = others_reach(kth);
    if (redo) rest = Mass{};
    if (bo != kNoIdx) {
      values_below<E>(src, bd, v0 + bo, kth, x);
      fold_values<E>(x, c, rest);
    }
    spread(redo, [&](int64_t vs, int32_t sbo, const typename Src::Data& dd) {
      if (vs < 0 || vs == v0 + sbo) return;
      float y[E];
      values_below<E>(src, dd, vs, kth, y);
      fold_values<E>(y, c, rest);
    });
    *mass = rest;
  }
  return TopPair{lv, li};
}

// The lists and masses of a row's nch parts as the row's: (lv, li) is the
// merged list (lane l = l-th best); the return value is the mass outside it,
// in every lane.  Called by one wave.
__device__ __forceinline__ Partial wave_merge_parts(const TopEntry* lists, const Partial* parts, int nch, int F,
                                                    float c, int lane, float& lv, int32_t& li) {
  lv = kNegInf;
  li = kNoIdx;
  wave_merge_entries(lists, nch * F, F, lv, li, lane);
  const float kv = readlane_f(lv, F - 1);
  const int32_t ki = __builtin_amdgcn_readlane(li, F - 1);
  const uint64_t kth = ki == kNoIdx ? 0ull : top_key(kv, ki);
  // the parts' masses and the listed values that did not make the row's list
  float m = kNegInf;
  for (int i = lane; i < nch; i += kWave) m = fmaxf(m, get_partial(parts + i).m);
  for (int i = lane; i < nch * F; i += kWave) {
    const TopEntry t = get_entry(lists + i);
    if (t.idx != kNoIdx && top_key(t.val, t.idx) < kth) m = fmaxf(m, t.val);
  }
  Partial r;
  r.pad = 0.f;
  r.m = wave_fmax(m);
  double s = 0.0;
  for (int i = lane; i < nch; i += kWave) {
    const Partial p = get_partial(parts + i);
    s += p.s * rescale(p.m, r.m, c);
  }
  for (int i = lane; i < nch * F; i += kWave) {
    const TopEntry t = get_entry(lists + i);
    if (t.idx != kNoIdx && top_key(t.val, t.idx) < kth) s += rescale(t.val, r.m, c);
  }
  r.s = wave_sum(s);
  return r;
}

}  // namespace sv
