// sv_rope.hip -- rotary positions of a window's queries and keys.
//
// y = factor * R(t f_i) x on the pairs (x_i, y_i) of each head; the gradient is
// the transposed rotation.  A block takes some tokens: it forms their angles
// once, in 64 bits and reduced to a turn (t f_i has far more digits than 32
// bits hold at distant positions), puts sine and cosine into LDS, and turns
// all heads with them.  Reads and writes each value once: bound by memory for
// many tokens, by the launch for few.
#include "sv_kv.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 4096;  // of a block at most (32 KB of LDS)

template <int DT>
struct Elem;
template <>
struct Elem<SV_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float get(T v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ T set(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
template <>
struct Elem<SV_F16> {
  using T = uint16_t;
  static __device__ __forceinline__ float get(T v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ T set(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};
template <>
struct Elem<SV_F32> {
  using T = uint32_t;
  static __device__ __forceinline__ float get(T v) { return __uint_as_float(v); }
  static __device__ __forceinline__ T set(float x) { return __float_as_uint(x); }
};

// V elements of 2 or 4 bytes.
template <typename T, int V>
struct Pack {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> take(const char* at) {
  if constexpr (V == 1) {
    return {{*reinterpret_cast<const T*>(at)}};
  } else {
    static_assert(sizeof(T) * V == 16, "a vector");
    return __builtin_bit_cast(Pack<T, V>, *reinterpret_cast<const u32x4*>(at));
  }
}
template <typename T, int V>
__device__ __forceinline__ void put(char* at, const Pack<T, V>& x) {
  if constexpr (V == 1)
    *reinterpret_cast<T*>(at) = x.v[0];
  else
    *reinterpret_cast<u32x4*>(at) = __builtin_bit_cast(u32x4, x);
}

// Items of a head's row: V pairs each where pairs are (i, i + R/2), V / 2 (one
// where V is 1) where they are neighbours; then V values each that are copied.
struct Rows {
  int pairs;   // of an item
  int turned;  // items that turn
  int all;     // and those that copy
};
__host__ __device__ inline Rows rows_of(int D, int R, int V, bool interleaved, bool copy) {
  Rows r;
  r.pairs = interleaved && V > 1 ? V / 2 : V;
  r.turned = R / 2 / r.pairs;
  r.all = r.turned + (copy ? (D - R) / V : 0);
  return r;
}

template <int DT, int V>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeParams p, const int tokens, const bool copy) {
  using T = typename Elem<DT>::T;
  extern __shared__ float s_angle[];  // [tokens][R/2] cosines, then as many sines
  const int half = p.R / 2;
  const int64_t all = (int64_t)p.B * p.N;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int some = (int)min((int64_t)tokens, all - t0);
  float* const s_cos = s_angle;
  float* const s_sin = s_angle + tokens * half;
  for (int x = threadIdx.x; x < some * half; x += kThreads) {
    const int i = x % half;
    const int64_t t = t0 + x / half;
    int64_t pos;
    if (p.positions) {
      pos = p.positions[t];
    } else {
      const int64_t b = t / p.N;
      int n = (int)(t - b * p.N);
      pos = p.lens ? p.lens[b] : 0;
      if (p.parent) {
        const int32_t* parent = p.parent + b * p.N;
        while (n > 0) {  // at most N steps: a parent stands before its node
          const int up = parent[n];
          if (up < 0 || up >= n) {
            if (i == 0) flag(p.err, SV_DERR_TREE);
            break;
          }
          n = up;
          ++pos;
        }
      } else {
        pos += n;
      }
    }
    const double turns = (double)pos * (p.freq[i] * 0.15915494309189535);
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    s_cos[x] = c * p.factor;
    s_sin[x] = (p.inverse ? -s : s) * p.factor;
  }
  __syncthreads();
  const Rows rows = rows_of(p.D, p.R, V, p.interleaved, copy);
  const int heads = p.heads[0] + p.heads[1];
  const int items = some * heads * rows.all;
  constexpr int es = sizeof(T);
  for (int x = threadIdx.x; x < items; x += kThreads) {
    const int row = x / rows.all, item = x - row * rows.all;
    const int t = row / heads;
    int h = row - t * heads;
    const int which = h >= p.heads[0];
    h -= which ? p.heads[0] : 0;
    const int64_t b = (t0 + t) / p.N, n = t0 + t - b * p.N;
    const char* in = p.in[which] + b * p.is[which][0] + n * p.is[which][1] + h * p.is[which][2];
    char* out = p.out[which] + b * p.os[which][0] + n * p.os[which][1] + h * p.os[which][2];
    if (item >= rows.turned) {
      const int64_t at = (p.R + (int64_t)(item - rows.turned) * V) * es;
      put<T, V>(out + at, take<T, V>(in + at));
      continue;
    }
    const int i0 = item * rows.pairs;
    const float* c = s_cos + t * half + i0;
    const float* s = s_sin + t * half + i0;
    if (p.interleaved && V > 1) {
      const int64_t at = (int64_t)i0 * 2 * es;
      Pack<T, V> v = take<T, V>(in + at);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float a = Elem<DT>::get(v.v[2 * j]), d = Elem<DT>::get(v.v[2 * j + 1]);
        v.v[2 * j] = Elem<DT>::set(a * c[j] - d * s[j]);
        v.v[2 * j + 1] = Elem<DT>::set(d * c[j] + a * s[j]);
      }
      put<T, V>(out + at, v);
    } else {
      const int64_t ax = (int64_t)(p.interleaved ? 2 * i0 : i0) * es;
      const int64_t ay = (int64_t)(p.interleaved ? 2 * i0 + 1 : i0 + half) * es;
      Pack<T, V> v = take<T, V>(in + ax), w = take<T, V>(in + ay);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float a = Elem<DT>::get(v.v[j]), d = Elem<DT>::get(w.v[j]);
        v.v[j] = Elem<DT>::set(a * c[j] - d * s[j]);
        w.v[j] = Elem<DT>::set(d * c[j] + a * s[j]);
      }
      put<T, V>(out + ax, v);
      put<T, V>(out + ay, w);
    }
  }
}

// Whether rows are 16-byte aligned and every item a whole vector.
bool vectors(const RopeParams& p, int es) {
  const int V = 16 / es;
  if (p.R % (p.interleaved ? V : 2 * V) || p.D % V) return false;
  for (int w = 0; w < 2; ++w) {
    if (!p.heads[w]) continue;
    if (reinterpret_cast<uintptr_t>(p.in[w]) % 16 || reinterpret_cast<uintptr_t>(p.out[w]) % 16) return false;
    for (int i = 0; i < 3; ++i)
      if (p.is[w][i] % 16 || p.os[w][i] % 16) return false;
  }
  return true;
}

template <int DT>
hipError_t rope(const RopeParams& p, hipStream_t s) {
  constexpr int es = sizeof(typename Elem<DT>::T);
  const bool vec = vectors(p, es);
  bool copy = false;  // in place, what does not turn stays
  for (int w = 0; w < 2; ++w) copy = copy || (p.heads[w] && p.in[w] != p.out[w]);
  const Rows rows = rows_of(p.D, p.R, vec ? 16 / es : 1, p.interleaved, copy);
  // a block's tokens: enough for every thread to have an item or two, as far as their angles fit
  const int64_t per = (int64_t)(p.heads[0] + p.heads[1]) * rows.all;
  int tokens = (int)(1 + 2 * kThreads / (per + 1));
  const int most = kAngles / (p.R / 2) > 1 ? kAngles / (p.R / 2) : 1;
  if (tokens > most) tokens = most;
  const int64_t all = (int64_t)p.B * p.N;
  const dim3 grid((uint32_t)((all + tokens - 1) / tokens));
  const size_t lds = (size_t)tokens * (p.R / 2) * 2 * sizeof(float);
  if (vec)
    rope_kernel<DT, 16 / es><<<grid, kThreads, lds, s>>>(p, tokens, copy);
  else
    rope_kernel<DT, 1><<<grid, kThreads, lds, s>>>(p, tokens, copy);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeParams& p, sv_dtype dt, hipStream_t s) {
  return dt == SV_BF16 ? rope<SV_BF16>(p, s) : dt == SV_F16 ? rope<SV_F16>(p, s) : rope<SV_F32>(p, s);
}

}  // namespace sv
