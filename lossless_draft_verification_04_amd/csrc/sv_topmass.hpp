// sv_topmass.hpp -- a block's top-F values of a range of 16-byte vectors and
// the mass (sum of exponentials) outside them, in one pass over the range.
// Shared by the teacher's pass and beam search.
//
// The selection is that of sv_topk.hpp: each thread keeps its best vector, a
// bound from groups of threads, candidates in LDS.  The mass must keep its
// digits where the list holds nearly everything, so it is no difference of
// rounded sums: beside the selection each thread adds up, in 64 bits, the
// 32-bit sums of its vectors but its best one, against a reference that its
// wave takes from its first vectors.  Once the list is known the best vector's
// unlisted values are added; another vector that holds a listed value (found
// with the candidates, where a thread's second largest value reaches the
// bound) is taken out again whole -- the same instructions on the same bits
// give the same 32-bit sum, so it leaves nothing behind but roundings -- and
// its other values are put back.  A wave whose sum turns out useless (values
// 2^100 above the reference, a mass near underflow below it, or one that is
// small against a value taken out) reads its vectors once more and sums the
// unlisted values, in 64 bits again, against one near their largest.
#pragma once

#include "sv_device.hpp"
#include "sv_topk.hpp"

namespace sv {

// Up to this many blocks, one to a compute unit, have 512 threads each, more
// 256.  Teacher's pass, bf16, 64 values, 256 threads / 512: 2048 x 151936 rows
// 109 us / 122; 2000 x 4000 24.5 / 36.8; 1536 x 32000 33.6 / 47.0; 480 x 32000
// 16.6 / 18.3; 300 x 128256 27.9 / 28.1; 256 x 128256 25.5 / 21.5; 17 x 152064
// 25.4 / 20.9.  Beams, 16 kept: 64 x 8 of 128256 32.6 / 33.1; 72 x 8 38.4 / 44.4.
constexpr int64_t kTopWide = 256;

// A 64-bit constant, formed in scalar registers where it stands: left alone
// the compiler lifts such constants out of the loop over rows into vector
// registers, which there hold a row.
__device__ __forceinline__ double here(double c) {
  asm volatile("" : "+s"(c));
  return c;
}
// e^x for x <= 0 in 64 bits to about 1e-11: x = n log 2 + r with |r| <= log(2) / 2
// (log 2 as its first 40 bits, which n times are exact, and the next 53), and
// the series of e^r to r^9 / 9!; 0 below the range.
__device__ __forceinline__ double exp_d(double x) {
  x = fmax(x, here(-800.0));
  const double n = rint(x * here(1.4426950408889634));
  double r = fma(n, here(-0x1.62e42fefa2p-1), x);
  r = fma(n, here(-0x1.9ef35793c7673p-41), r);
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

// A sum of exponentials: sum of 2^(c (x - m)), m the largest x (-inf, 0: of
// nothing).
struct Mass {
  float m = kNegInf;
  float s = 0.f;
};

// a <- a + the E values x (-inf: nothing).  The shift is m, as fma(x, c, -c m),
// whose -c m carries a rounding of 2^-25 |c m| into every term; past 2^6 (values
// far from 0, a low temperature, rows masked with the type's lowest value) it
// is (x - m) c; SUB: always so (no branch, an operation more a value).
template <int E, bool SUB = false>
__device__ __forceinline__ void fold_values(const float (&x)[E], float c, Mass& a) {
  float fm = x[0];
#pragma unroll
  for (int e = 1; e < E; ++e) fm = fmaxf(fm, x[e]);
  const float mn = fmaxf(a.m, fm);
  const float ref = mn == kNegInf ? 0.f : mn;
  const float cm = c * ref;
  float t[E];
  if (!SUB && __builtin_expect(fabsf(cm) <= 64.f, 1)) {
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

// The same over any number of vectors (a row of 2^24 logits gives a thread
// thousands): added up in 64 bits, each vector's values in 32.  m is a value
// that the largest passes by 2^32 at most, so that it seldom moves: a factor
// for every new largest value would bring its own rounding thousands of times.
struct LongMass {
  float m = kNegInf;
  double s = 0.0;
};
template <int E>
__device__ __forceinline__ void fold_long(const float (&x)[E], float c, LongMass& a) {
  float fm = x[0];
#pragma unroll
  for (int e = 1; e < E; ++e) fm = fmaxf(fm, x[e]);
  if ((fm - a.m) * c > 32.f) {  // the first finite value too: a.m = -inf
    a.s *= (double)fast_exp2((a.m - fm) * c);
    a.m = fm;
  }
  const float ref = a.m == kNegInf ? 0.f : a.m;
  float t[E];
#pragma unroll
  for (int e = 0; e < E; ++e) t[e] = fast_exp2((x[e] - ref) * c);
#pragma unroll
  for (int w = E / 2; w > 0; w >>= 1)
#pragma unroll
    for (int e = 0; e < w; ++e) t[e] += t[e + w];
  a.s += (double)t[0];
}

// 2^(c (a - b)) for a merge of sums, a <= b; 0 for a = -inf.
__device__ __forceinline__ double rescale(float a, float b, float c) {
  return a == kNegInf ? 0.0 : exp2_d((double)c * ((double)a - (double)b));
}

// -inf in place of the elements of vector d that mk marks (a bit each).
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

// One logit row as a value source for block_topk_mass: what lies past V is
// masked as its vector is loaded, so no other step looks at V.
template <int DT>
struct MassRow {
  static constexpr int E = Fmt<DT>::kPerVec;
  const void* row;
  int V;
  __device__ __forceinline__ u32x4 load_whole(int64_t v) const { return load_vec(row, v); }  // not the row's last
  __device__ __forceinline__ u32x4 load(int64_t v) const {
    u32x4 d = load_vec(row, v);
    if ((int)v == V / E) mask_vec<DT>(d, 0xffu << (V % E));  // the row's last vector, if it is a shorter one
    return d;
  }
  using Data = u32x4;
  static constexpr bool kSkipNegInf = false;
  __device__ __forceinline__ void values(const u32x4& d, int64_t, float* x) const { unpack<DT>(d, x); }
  __device__ __forceinline__ static u32x4 none() {
    u32x4 d{0u, 0u, 0u, 0u};
    mask_vec<DT>(d, 0xffu);
    return d;
  }
};

// Keeps a vector packed across a phase: without it the compiler holds the
// unpacked values of one use for the next, twice the registers.
__device__ __forceinline__ void stay_packed(u32x4& d) { asm volatile("" : "+v"(d)); }

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

// An entry's order as a positive double (larger = better; 0: none): the value's
// order bits over 24 bits of complemented index, 56 bits in all, read as the
// bits of a double, whose comparison is one full-rate instruction.
__device__ __forceinline__ double order_of(float v, int32_t i) {
  const uint64_t k = top_key(v, i);
  return i == kNoIdx ? 0.0 : __longlong_as_double((long long)(((k >> 32) << 24) | (k & 0xffffffull)));
}

// The 32-bit sum of 2^(c x - r) over a vector's values: the same instructions
// wherever a vector is added or taken out.
template <int E>
__device__ __forceinline__ float vec_sum(const float (&x)[E], float c, float r) {
  float t[E];
#pragma unroll
  for (int e = 0; e < E; ++e) t[e] = fast_exp2(__builtin_fmaf(x[e], c, -r));
#pragma unroll
  for (int w = E / 2; w > 0; w >>= 1)
#pragma unroll
    for (int e = 0; e < w; ++e) t[e] += t[e + w];
  return t[0];
}

// As block_topk (wave 0 returns the list of the range's F best), and mass =
// the sum over the range's other values, in every thread.  F >= 1.
template <int NT, int E, class Src>
__device__ __forceinline__ TopPair block_topk_mass(const Src src, int64_t v0, int64_t v1, int V, int F, float c,
                                                   Partial* mass) {
  // vectors of a thread's window: the loop over whole windows has the next one
  // in flight; the first window (in fp32 the last ones too) waits for each load
  // in turn, as each stands under a condition and is masked where it is made
  constexpr int kWin = 4;
  constexpr int NW = NT / kWave;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int tid = threadIdx.x;
  __shared__ uint64_t s_cand[kCand];
  __shared__ uint64_t s_gk[NT];
  __shared__ alignas(16) uint64_t s_key[kCand];
  __shared__ uint64_t s_sel[kWave];
  __shared__ uint64_t s_tau;
  __shared__ int s_nc;
  __shared__ float s_wm[NW];
  __shared__ double s_ws[NW];
  __shared__ int32_t s_hit[NW][kWave];
  float lv = kNegInf;
  int32_t li = kNoIdx;
  const int span = (int)(v1 - v0);
  const int nk = span > 0 ? (span + NT - 1) / NT : 0;  // vectors per thread at most
  const bool held = nk <= kWin;                        // block-uniform: every vector stays in registers
  float bm = kNegInf;    // the best vector's largest value, offset and data
  int32_t bo = kNoIdx;
  typename Src::Data bd = Src::none();
  const bool more = tid + NT < span;  // the thread owns vectors besides its best one
  float om = kNegInf;                 // their largest value
  double sum = 0.0;                   // of all its vectors but the best one
  float bs = 0.f;                     // and of that one
  float ref = kNegInf, r = 0.f;       // the wave's reference and c times it
  typename Src::Data d[kWin];
#pragma unroll
  for (int u = 0; u < kWin; ++u)
    if (tid + u * NT < span) d[u] = src.load(v0 + tid + u * NT);
  auto largest = [&](const typename Src::Data& dd) {
    float x[E];
    src.values(dd, 0, x);
    float vm = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) vm = fmaxf(vm, x[e]);
    return vm;
  };
  if (held) {
#pragma unroll
    for (int u = 0; u < kWin; ++u) {
      const int32_t o = tid + u * NT;
      if (o < span) {
        const float vm = largest(d[u]);
        const bool t = top_better(vm, o, bm, bo);  // an empty best (-inf, kNoIdx) loses to any vector
        bm = t ? vm : bm;
        bo = t ? o : bo;
      }
      stay_packed(d[u]);
    }
  } else {
    // the wave's reference, near the largest values that are no outliers: the
    // largest over its threads of the smallest of the first window's vectors'
    // largest values (all kWin are there: nk > kWin); of masked ones 0
    {
      float m = __builtin_huge_valf(), top = kNegInf;
#pragma unroll
      for (int u = 0; u < kWin; ++u) {
        const float vm = largest(d[u]);
        m = fminf(m, vm);
        top = fmaxf(top, vm);
        stay_packed(d[u]);
      }
      ref = wave_fmax(m);
      if (ref == kNegInf) ref = wave_fmax(top);
      if (ref == kNegInf) ref = 0.f;
      r = c * ref;
    }
    auto take = [&](const typename Src::Data& dd, int32_t o) {
      float x[E];
      src.values(dd, 0, x);
      float vm = x[0];
#pragma unroll
      for (int e = 1; e < E; ++e) vm = fmaxf(vm, x[e]);
      const bool t = top_better(vm, o, bm, bo);
      om = __builtin_amdgcn_fmed3f(om, bm, vm);  // the second largest: om <= bm
#pragma unroll
      for (int i = 0; i < 4; ++i) bd[i] = t ? dd[i] : bd[i];
      bm = t ? vm : bm;
      bo = t ? o : bo;
      const float s = vec_sum<E>(x, c, r);
      sum += (double)(t ? bs : s);
      bs = t ? s : bs;
    };
    int32_t o = tid;
    for (; o + (2 * kWin - 1) * NT < span - 1; o += kWin * NT) {
      // this window and the next are whole, without the last vector
      typename Src::Data nx[kWin];
#pragma unroll
      for (int u = 0; u < kWin; ++u) nx[u] = src.load_whole(v0 + o + (kWin + u) * NT);
#pragma unroll
      for (int u = 0; u < kWin; ++u) take(d[u], o + u * NT);
#pragma unroll
      for (int u = 0; u < kWin; ++u) d[u] = nx[u];
    }
    for (; o < span; o += kWin * NT) {  // twice at most
      typename Src::Data nx[kWin];
#pragma unroll
      for (int u = 0; u < kWin; ++u)
        if (o + (kWin + u) * NT < span) nx[u] = src.load(v0 + o + (kWin + u) * NT);
#pragma unroll
      for (int u = 0; u < kWin; ++u)
        if (o + u * NT < span) take(d[u], o + u * NT);
#pragma unroll
      for (int u = 0; u < kWin; ++u) d[u] = nx[u];
    }
  }
  // the bound tau from below on the F-th best key (see block_topk)
  const uint64_t tkey = bo == kNoIdx ? 0ull : top_key(bm, (int32_t)((v0 + bo) * E));
  constexpr int kMaxH = NT / kWave;
  static_assert(kMaxH >= 1 && kMaxH <= 16 && kMaxH * kWave == NT, "whole waves, at most 16");
  // four times as many groups as listed values: more of them lengthen the
  // search, fewer loosen the bound, so that more threads' other vectors are
  // read again (2048 x 151936 bf16 rows, 64 values: 131 us at twice as many,
  // 108 at four and eight times; 128 x 32000, 16 values: 11.3, 11.4, 12.6 us)
  int H = 1;
  while (H < kMaxH && 4 * F > kWave * H) H *= 2;  // block-uniform
  const int GS = NT / (kWave * H);
  {
    uint64_t k = tkey;
    if (GS >= 2) key_max_step<kRowShr + 1, 0xF>(k);
    if (GS >= 4) key_max_step<kRowShr + 2, 0xF>(k);
    if (GS >= 8) key_max_step<kRowShr + 4, 0xF>(k);
    if (GS >= 16) key_max_step<kRowShr + 8, 0xF>(k);
    // as a key that the vector's best element has at least; 0: the group holds nothing
    if ((lane & (GS - 1)) == GS - 1) s_gk[tid / GS] = k ? k - (E - 1) : 0ull;
  }
  if (tid == 0) s_nc = 0;
  lds_sync();
  if (wave == 0) {
    uint64_t gk[kMaxH];
    uint32_t hi = 0;  // the bound's upper 32 bits, of which the upper 16 are sought
    int n = 0;
    if (H == 1) {  // one group per lane (F <= 16)
      gk[0] = s_gk[lane];
      const uint32_t gh = (uint32_t)(gk[0] >> 32);
#pragma unroll
      for (int bit = 31; bit >= 16; --bit) {
        const uint32_t q = hi | (1u << bit);
        if (__builtin_popcountll(__ballot(gh >= q)) >= F) hi = q;
      }
      n = __builtin_popcountll(__ballot(gh >= hi));
#pragma unroll
      for (int h = 1; h < kMaxH; ++h) gk[h] = 0ull;
    } else {
#pragma unroll
      for (int h = 0; h < kMaxH; ++h) gk[h] = h < H ? s_gk[h * kWave + lane] : 0ull;
      for (int bit = 31; bit >= 16; --bit) {
        const uint32_t q = hi | (1u << bit);
        int cnt = 0;
#pragma unroll
        for (int h = 0; h < kMaxH; ++h) cnt += __builtin_popcountll(__ballot((uint32_t)(gk[h] >> 32) >= q));
        if (cnt >= F) hi = q;
      }
#pragma unroll
      for (int h = 0; h < kMaxH; ++h) n += __builtin_popcountll(__ballot((uint32_t)(gk[h] >> 32) >= hi));
    }
    uint64_t p = (uint64_t)hi << 32;
    // many groups tie in the upper 16 bits of the value (bf16: all of it): the
    // bound goes on to the whole value and the index, without which rows of
    // few values list far too many (512 x 128256 bf16 zeros: 349 us, 28 so)
    if (hi != 0u && n > 2 * F + 16) {
      auto take = [&](int bit) {
        const uint64_t q = p | (1ull << bit);
        int cnt = 0;
#pragma unroll
        for (int h = 0; h < kMaxH; ++h) cnt += __builtin_popcountll(__ballot(gk[h] >= q));
        if (cnt >= F) p = q;
      };
      if constexpr (E == 4) {
#pragma unroll 1
        for (int bit = 47; bit >= 32; --bit) take(bit);
      } else {
        p |= (p >> 63) ? 0ull : 0xffffull << 32;  // of negative values these bits are set
      }
      p |= 0xffull << 24;  // as in every key: indices have 24 bits
#pragma unroll 1
      for (int bit = 23; bit >= 0; --bit) take(bit);
    }
    if (lane == 0) s_tau = p;
  }
  lds_sync();
  uint64_t tau = s_tau;
  // the thread's vectors besides its best may hold a key of at least t: they
  // come after it where they tie with it, and in any case not before the first
  const int32_t oo = om == bm ? bo + NT : bo == tid ? tid + NT : tid;
  const uint64_t okey = more ? top_key(om, (int32_t)((v0 + oo) * E)) : 0ull;
  auto others_reach = [&](uint64_t t) { return okey != 0ull && okey >= t; };
  // f(vs, o, d) for every vector of the wave's lanes with `pick`: two such
  // lanes' vectors at a time, one each per lane (vs < 0: none), o the owner's
  // best vector
  auto spread = [&](bool pick, auto&& f) {
    constexpr int kOwners = 2;
    uint64_t m = __ballot(pick);
    while (m) {  // wave-uniform
      int own[kOwners];
#pragma unroll
      for (int q = 0; q < kOwners; ++q) {
        own[q] = m ? __builtin_ctzll(m) : -1;
        m &= m - 1;
      }
      for (int k = lane; k - lane < nk; k += kWave) {
        typename Src::Data dd[kOwners];
        int64_t vs[kOwners];
#pragma unroll
        for (int q = 0; q < kOwners; ++q) {
          const int at = wave * kWave + own[q] + k * NT;
          vs[q] = own[q] >= 0 && at < span ? v0 + at : -1;
          if (vs[q] >= 0) dd[q] = src.load(vs[q]);
        }
#pragma unroll
        for (int q = 0; q < kOwners; ++q)
          f(vs[q], __builtin_amdgcn_readlane(bo, own[q] >= 0 ? own[q] : 0), dd[q]);
      }
    }
  };
  int nc;
  int hits = 0;  // the wave's vectors, none a thread's best one, that reach tau: their offsets in s_hit, the first kWave
  bool first = true;
  for (;;) {  // block-uniform; tau rises on every repetition
    hits = 0;
    const bool sel = tkey != 0ull && tkey >= tau;
    if (held) {
#pragma unroll
      for (int u = 0; u < kWin; ++u) {
        const int64_t vu = v0 + tid + (int64_t)u * NT;
        flag_candidates<E>(src, d[u], sel && vu < v1 ? vu : -1, V, tau, s_cand, &s_nc);
        stay_packed(d[u]);
      }
    } else {
      const bool full = sel && others_reach(tau);
      flag_candidates<E>(src, bd, sel && !full ? v0 + bo : -1, V, tau, s_cand, &s_nc);
      stay_packed(bd);
      spread(full, [&](int64_t vs, int32_t sbo, const typename Src::Data& dd) {
        const bool hit = vs >= 0 && top_key(largest(dd), (int32_t)(vs * E)) >= tau;
        if (__ballot(hit) == 0ull) return;
        flag_candidates<E>(src, dd, hit ? vs : -1, V, tau, s_cand, &s_nc);
        const uint64_t rest = __ballot(hit && vs != v0 + sbo);
        const int at = hits + __builtin_popcountll(rest & ((1ull << lane) - 1));
        if (((rest >> lane) & 1u) && at < kWave) s_hit[wave][at] = (int32_t)(vs - v0);
        hits += __builtin_popcountll(rest);
      });
    }
    lds_sync();
    nc = s_nc;
    if (nc <= kCand) break;
    tau = block_select<NT>(s_cand, s_key, s_sel, kCand, F, &s_tau);
    first = false;
    if (tid == 0) s_nc = 0;
    lds_sync();
  }
  // a candidate's place is the number of better ones, counted over LDS
  {
    double* keys = reinterpret_cast<double*>(s_key);
    const double2* pairs = reinterpret_cast<const double2*>(s_key);
    if (tid == 0) s_tau = 0ull;
    for (int i = tid; i < kCand; i += NT) {  // past the last one 0, above none
      const uint64_t cd = i < nc ? s_cand[i] : 0ull;
      keys[i] = i < nc ? order_of(cand_value(cd), (int32_t)(cd >> 32)) : 0.0;
    }
    lds_sync();
    for (int i = tid; i < nc; i += NT) {
      const double k = keys[i];
      int above = 0;
#pragma unroll 4
      for (int j = 0; j < nc; j += 2) {
        const double2 o = pairs[j >> 1];
        above += (o.x > k ? 1 : 0) + (o.y > k ? 1 : 0);
      }
      if (above < F) s_sel[above] = s_cand[i];
      if (above == F - 1) s_tau = cand_key(s_cand[i]);
    }
    lds_sync();
    if (wave == 0 && lane < F && lane < nc) {
      lv = cand_value(s_sel[lane]);
      li = (int32_t)(s_sel[lane] >> 32);
    }
  }
  // the F-th best key; 0 where fewer are listed, which then are all there are
  const uint64_t kth = s_tau;
  // the wave's mass outside the list: ws relative to wm
  double ws = 0.0;
  float wm = kNegInf;
  bool again = held;  // wave-uniform
  if (!held) {
    float gone = 0.f;
    // a vector with listed values: out whole, its other values back
    auto strip = [&](int64_t v, const typename Src::Data& dd) {
      float y[E];
      src.values(dd, v, y);
      const float s = vec_sum<E>(y, c, r);
      values_below<E>(src, dd, v, kth, y);
      gone += s;
      sum -= (double)s;
      sum += (double)vec_sum<E>(y, c, r);
    };
    if (tkey >= kth && bo != kNoIdx) {
      float y[E];
      values_below<E>(src, bd, v0 + bo, kth, y);
      bs = vec_sum<E>(y, c, r);
    }
    sum += (double)bs;
    auto strip_listed = [&](int64_t v, const typename Src::Data& dd) {
      if (top_key(largest(dd), (int32_t)(v * E)) >= kth) strip(v, dd);
    };
    // a bound from a repetition depends on the order of arrivals, and with it
    // which lane would take which of the noted vectors out
    if (first && hits <= kWave) {  // wave-uniform
      if (lane < hits) {
        const int64_t v = v0 + s_hit[wave][lane];
        strip_listed(v, src.load(v));
      }
    } else {
      spread(others_reach(kth), [&](int64_t vs, int32_t sbo, const typename Src::Data& dd) {
        if (vs >= 0 && vs != v0 + sbo) strip_listed(vs, dd);
      });
    }
    ws = wave_sum(sum);
    // what went leaves up to 2^-53 of itself behind at each of its lane's nk
    // additions: 2^-25 of what stays (2^-19 if all 64 lanes agreed in size and
    // sign).  Values 2^-126 of the reference are lost; a NaN fails every test.
    again = (wave_fmax(bm) > kNegInf) &
            (!(ws > 0x1p-70) | !(ws < 0x1p100) | !(ws > 0x1p-28 * nk * (double)wave_fmax(gone)) | !(fabsf(r) <= 0x1p30f));
    if (!again) {
      wm = ref;
      ws *= exp2_d((double)r - (double)c * (double)ref);  // r is not quite c ref: 2^-25 of it, 2^5 at most
    }
  }
  if (again) {
    float x[E];
    if (held) {
      Mass own;  // of kWin vectors at most
#pragma unroll
      for (int u = 0; u < kWin; ++u) {
        const int o = tid + u * NT;
        if (o < span) {
          values_below<E>(src, d[u], v0 + o, kth, x);
          fold_values<E>(x, c, own);
        }
      }
      wm = wave_fmax(own.m);
      ws = wave_sum(own.m == kNegInf ? 0.0 : (double)own.s * (double)fast_exp2((own.m - wm) * c));
    } else {
      LongMass own;
      for (int o = tid; o < span; o += kWin * NT) {
#pragma unroll
        for (int u = 0; u < kWin; ++u)
          if (o + u * NT < span) d[u] = src.load(v0 + o + u * NT);
#pragma unroll
        for (int u = 0; u < kWin; ++u)
          if (o + u * NT < span) {
            const int64_t v = v0 + o + u * NT;
            if (top_key(largest(d[u]), (int32_t)(v * E)) >= kth)
              values_below<E>(src, d[u], v, kth, x);
            else
              src.values(d[u], v, x);
            fold_long<E>(x, c, own);
          }
      }
      wm = wave_fmax(own.m);
      ws = wave_sum(own.s * rescale(own.m, wm, c));
    }
  }
  if (lane == 0) {
    s_wm[wave] = ws > 0.0 ? wm : kNegInf;
    s_ws[wave] = ws;
  }
  lds_sync();
  const float pm = lane < NW ? s_wm[lane] : kNegInf;
  mass->pad = 0.f;
  mass->m = wave_fmax(pm);
  mass->s = wave_sum(pm == kNegInf ? 0.0 : s_ws[lane] * rescale(pm, mass->m, c));
  return TopPair{lv, li};
}

// Entries of all parts of a row, at most (a row's parts times F), and parts.
constexpr int kPartEntries = 256;
constexpr int kMostParts = 16;
constexpr int kPerLane = kPartEntries / kWave;

// An order's value and index (a value of -0 comes back as 0).
__device__ __forceinline__ float order_value(double k) {
  const uint32_t o = (uint32_t)((uint64_t)__double_as_longlong(k) >> 24);
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int32_t order_index(double k) {
  return (int32_t)(~(uint32_t)(uint64_t)__double_as_longlong(k) & 0xffffffu);
}
__device__ __forceinline__ double order_from(double k, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(k);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(lane * 4, (int)(uint32_t)b);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(lane * 4, (int)(uint32_t)(b >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Runs of P lanes that fall and then rise, sorted: log2 P compare-exchange steps.
__device__ __forceinline__ double order_clean(double x, int P, int lane) {
  for (int h = P / 2; h > 0; h /= 2) {
    const double o = order_from(x, lane ^ h);
    x = (o > x) == ((lane & h) == 0) ? o : x;  // the lower lane keeps the larger
  }
  return x;
}

// The lists and masses of a row's nch parts (nch * F <= kPartEntries) as the
// row's: (lv, li) is the merged list (lane l = l-th best); the return value is
// the mass outside it, in every lane.  Called by one wave, with kPartEntries
// words of LDS of its own.  All is loaded in one round; the lists, a run of P
// lanes each (P the power of two from F on), merge as sorted ones do: the
// better of one and the other reversed, then order_clean.  Its steps grow with
// the logarithm of F and the lists, where counting every entry's place grows
// with their product (8 beams of 152064 in 4 parts, 64 kept: 24.1 and 31.4 us;
// 8 kept: 15.2 and 15.0).  The code is kept short: it runs once, from cold.
__device__ __forceinline__ Partial wave_merge_parts(const TopEntry* lists, const Partial* parts, int nch, int F,
                                                    float c, int lane, double* keys, float& lv, int32_t& li) {
  Partial r;
  r.pad = 0.f;
  if (nch == 1) {
    TopEntry t{kNegInf, kNoIdx};
    if (lane < F) t = get_entry(lists + lane);
    r = get_partial(parts);
    lv = t.val;
    li = t.idx;
    return r;
  }
  const int n = nch * F;
  TopEntry t[kPerLane];
  double key[kPerLane];
  Partial p{kNegInf, 0.f, 0.0};
#pragma unroll
  for (int q = 0; q < kPerLane; ++q) {
    t[q] = TopEntry{kNegInf, kNoIdx};
    if (q * kWave + lane < n) t[q] = get_entry(lists + q * kWave + lane);
  }
  if (lane < nch) p = get_partial(parts + lane);
#pragma unroll
  for (int q = 0; q < kPerLane; ++q) {
    key[q] = order_of(t[q].val, t[q].idx);
    keys[q * kWave + lane] = key[q];
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  int P = 1;
  while (P < F) P *= 2;
  const int e = lane & (P - 1), list = lane / P;
  auto entry = [&](int l, int at) { return l < nch && at < F ? keys[l * F + at] : 0.0; };
  double best = entry(list, e);
#pragma unroll 1
  for (int l = kWave / P; l < nch; l += kWave / P) {  // the runs of the next lists
    const double o = entry(l + list, P - 1 - e);
    best = order_clean(o > best ? o : best, P, lane);
  }
#pragma unroll 1
  for (int g = P; g < kWave && g < P * nch; g *= 2) {  // the runs among themselves
    const double o = order_from(best, lane ^ (g + P - 1));
    best = order_clean(o > best ? o : best, P, lane);
  }
  __builtin_amdgcn_wave_barrier();
  // what is listed no longer goes back into the mass
  const double kth = readlane_d(best, F - 1);  // 0: fewer than F entries, all of them listed
  float m = p.m;
#pragma unroll
  for (int q = 0; q < kPerLane; ++q)
    if (key[q] > 0.0 && key[q] < kth) m = fmaxf(m, t[q].val);
  r.m = wave_fmax(m);
  double s = p.s * rescale(p.m, r.m, c);
#pragma unroll
  for (int q = 0; q < kPerLane; ++q)
    if (key[q] > 0.0 && key[q] < kth && t[q].val > kNegInf) s += (double)fast_exp2((t[q].val - r.m) * c);
  r.s = wave_sum(s);
  const bool in = lane < F && best > 0.0;
  lv = in ? order_value(best) : kNegInf;
  li = in ? order_index(best) : kNoIdx;
  return r;
}

}  // namespace sv
