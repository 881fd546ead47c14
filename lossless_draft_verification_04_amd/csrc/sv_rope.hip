// sv_rope.hip -- rotary positions of a window's queries and keys.
//
// y = factor * R(t f_i) x on the pairs (x_i, y_i) of each head; the gradient is
// the transposed rotation.  A thread takes 16 bytes of a head's row (twice,
// where a pair's halves lie R/2 apart) in up to 8 heads of a token one after
// another: it forms the angles of its pairs once for them, in 64 bits and
// reduced to a turn (t f_i has far more digits than 32 bits hold at distant
// positions).  Reads and writes each value once: bound by memory for many tokens
// (8 x 2048 nodes, 40 heads of 128 in fp32: 146 us, a copy of as many bytes 137;
// with a token's angles in LDS for all heads 170), by the launch for few (4 us).
#include "sv_kv.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;

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
    return __builtin_bit_cast(Pack<T, V>, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at)));
  }
}
template <typename T, int V>
__device__ __forceinline__ void put(char* at, const Pack<T, V>& x) {
  if constexpr (V == 1)
    *reinterpret_cast<T*>(at) = x.v[0];
  else
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, x), reinterpret_cast<u32x4*>(at));
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

// Threads stand (slot, item): `slots` of a block take `run` rows (token, head) one
// after another each, `wide` items of a row beside one another.
struct Shape {
  int32_t wide, slots, run, copy;
};

// SPLIT: a pair's halves lie R/2 apart.
template <int DT, int V, bool SPLIT>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeParams p, const Shape shape) {
  using T = typename Elem<DT>::T;
  constexpr int es = sizeof(T);
  constexpr int kPairs = SPLIT || V == 1 ? V : V / 2;  // of an item
  constexpr int kAhead = 4;                            // rows' loads at a time
  const int half = p.R / 2, heads = p.heads[0] + p.heads[1];
  const Rows rows = rows_of(p.D, p.R, V, !SPLIT, shape.copy);
  const int slot = threadIdx.x / shape.wide, lane = threadIdx.x - slot * shape.wide;
  // a tree's parents, of the block's first sequence
  __shared__ int32_t s_parent[SV_MAX_N];
  int64_t staged = -1;
  if (p.parent && !p.positions) {
    staged = (int64_t)blockIdx.x * shape.slots * shape.run / heads / p.N;
    for (int i = threadIdx.x; i < p.N; i += kThreads) s_parent[i] = p.parent[staged * p.N + i];
    __syncthreads();
  }
  if (slot >= shape.slots) return;
  const int64_t all = (int64_t)p.B * p.N * heads;
  const int64_t row0 = ((int64_t)blockIdx.x * shape.slots + slot) * shape.run;
  const int64_t row1 = min(row0 + shape.run, all);
  if (row0 >= row1) return;
  for (int item = blockIdx.y * shape.wide + lane; item < rows.all; item += gridDim.y * shape.wide) {
    const bool turned = item < rows.turned;
    const int64_t at0 = (turned ? (int64_t)item * (SPLIT ? V : 2 * kPairs) : p.R + (int64_t)(item - rows.turned) * V) * es;
    const int64_t at1 = at0 + (SPLIT ? half : 1) * es;  // the other half, where it is a vector of its own
    int64_t t = row0 / heads;
    int h = (int)(row0 - t * heads);
    int64_t b = t / p.N;
    int n = (int)(t - b * p.N);
    bool fresh = true;
    float c[kPairs], s[kPairs];
    for (int64_t row = row0; row < row1;) {
      Pack<T, V> v[kAhead], w[kAhead];
      char* out[kAhead];
      const int count = (int)min((int64_t)min(kAhead, heads - h), row1 - row);  // of the same token
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (a >= count) break;
        const int which = h + a >= p.heads[0];
        const int hh = h + a - (which ? p.heads[0] : 0);
        const char* in = p.in[which] + b * p.is[which][0] + n * p.is[which][1] + hh * p.is[which][2];
        out[a] = p.out[which] + b * p.os[which][0] + n * p.os[which][1] + hh * p.os[which][2];
        v[a] = take<T, V>(in + at0);
        if ((SPLIT || V == 1) && turned) w[a] = take<T, V>(in + at1);
      }
      if (fresh && turned) {  // while the first loads fly
        int64_t pos;
        if (p.positions) {
          pos = p.positions[b * p.N + n];
        } else {
          pos = p.lens ? p.lens[b] : 0;
          if (p.parent) {
            const int32_t* parent = p.parent + b * p.N;
            for (int i = n; i > 0; ++pos) {  // at most N steps: a parent stands before its node
              const int up = b == staged ? s_parent[i] : parent[i];
              if (up < 0 || up >= i) {
                if (item == 0) flag(p.err, SV_DERR_TREE);
                break;
              }
              i = up;
            }
          } else {
            pos += n;
          }
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const double turns = (double)pos * (p.freq[item * kPairs + j] * 0.15915494309189535);
          // the rest of a turn to 32 bits, off by 2^-26 turns at most: about what sine,
          // cosine and products of 32 bits are off by (5.1e-8 in all; 3.5e-8 with sine
          // and cosine in 64)
          sincospif(2.0f * (float)(turns - rint(turns)), &s[j], &c[j]);
          c[j] *= p.factor;
          s[j] *= p.inverse ? -p.factor : p.factor;
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (a >= count) break;
        if (turned) {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            T& first = v[a].v[SPLIT || V == 1 ? j : 2 * j];
            T& second = SPLIT || V == 1 ? w[a].v[j] : v[a].v[V == 1 ? 0 : 2 * j + 1];
            const float x = Elem<DT>::get(first), y = Elem<DT>::get(second);
            first = Elem<DT>::set(x * c[j] - y * s[j]);
            second = Elem<DT>::set(y * c[j] + x * s[j]);
          }
          if (SPLIT || V == 1) put<T, V>(out[a] + at1, w[a]);
        }
        put<T, V>(out[a] + at0, v[a]);
      }
      row += count;
      h += count;
      fresh = h == heads;
      if (fresh) {
        h = 0;
        if (++n == p.N) {
          n = 0;
          ++b;
        }
      }
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

template <int DT, int V>
void run(const RopeParams& p, const Shape& shape, dim3 grid, hipStream_t s) {
  if (p.interleaved)
    rope_kernel<DT, V, false><<<grid, kThreads, 0, s>>>(p, shape);
  else
    rope_kernel<DT, V, true><<<grid, kThreads, 0, s>>>(p, shape);
}

template <int DT>
hipError_t rope(const RopeParams& p, hipStream_t s) {
  constexpr int es = sizeof(typename Elem<DT>::T);
  const bool vec = vectors(p, es);
  Shape shape;
  shape.copy = 0;  // in place, what does not turn stays
  for (int w = 0; w < 2; ++w) shape.copy |= p.heads[w] && p.in[w] != p.out[w];
  const Rows rows = rows_of(p.D, p.R, vec ? 16 / es : 1, p.interleaved, shape.copy);
  shape.wide = rows.all < kThreads ? rows.all : kThreads;
  shape.slots = kThreads / shape.wide;
  const int64_t all = (int64_t)p.B * p.N * (p.heads[0] + p.heads[1]);
  // Rows of a slot: one where there are few, up to 8 for as many as fill the device.
  const int64_t fill = all / (2048 * (int64_t)shape.slots);
  shape.run = fill < 1 ? 1 : fill > 8 ? 8 : (int)fill;
  const int64_t blocks = (all + (int64_t)shape.slots * shape.run - 1) / ((int64_t)shape.slots * shape.run);
  if (blocks > UINT32_MAX / kThreads) return hipErrorInvalidValue;  // threads of a launch's dimension
  const dim3 grid((uint32_t)blocks, (uint32_t)((rows.all + shape.wide - 1) / shape.wide));
  if (vec)
    run<DT, 16 / es>(p, shape, grid, s);
  else
    run<DT, 1>(p, shape, grid, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeParams& p, sv_dtype dt, hipStream_t s) {
  return dt == SV_BF16 ? rope<SV_BF16>(p, s) : dt == SV_F16 ? rope<SV_F16>(p, s) : rope<SV_F32>(p, s);
}

}  // namespace sv
