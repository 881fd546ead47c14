// sv_kv_attention.hip -- attention of a window's nodes over the 4-bit cache.
#include "sv_kv.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 16;       // tokens of a tile, rows of a tile
constexpr int kWaveTokens = 32; // tokens of a wave's step: two tiles

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 y = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
}

// ---------------------------------------------------------------------------
// Which part of the work a block does: all steps (128 tokens of a sequence for
// one key head and group of rows) stand in one line, sequence by sequence,
// and block i of W takes steps [i T / W, (i + 1) T / W).
// ---------------------------------------------------------------------------
struct Span {
  int32_t len, news;  // news = 0: nothing to do
  int64_t u0, units;  // first step of the sequence's tokens, number of steps
};

__device__ __forceinline__ Span span_of(const AttentionParams& p, int64_t b) {
  Span s;
  s.len = p.lens[b];
  s.news = p.news ? p.news[b] : p.N;
  s.u0 = s.units = 0;
  if (s.len < 0 || s.news < 0 || s.news > p.N || (int64_t)s.len + s.news > p.c.room) {
    s.news = -1;
    return s;
  }
  if (s.news == 0) return s;
  const int64_t lo = p.reach > 0 ? max((int64_t)s.len - p.reach + 1, (int64_t)0) : 0;
  s.u0 = lo / kAttentionUnit;
  s.units = ((int64_t)s.len + s.news + kAttentionUnit - 1) / kAttentionUnit - s.u0;
  return s;
}

// First step of block i.
__device__ __forceinline__ int64_t start_of(int64_t i, int64_t total, int64_t blocks) {
  return (int64_t)((uint64_t)i * (uint64_t)total / (uint64_t)blocks);
}
// The block that has step x.
__device__ __forceinline__ int block_of(int64_t x, int64_t total, int64_t blocks) {
  return (int)((((uint64_t)x + 1) * (uint64_t)blocks - 1) / (uint64_t)total);
}

// ---------------------------------------------------------------------------
// Fragments.  A wave's lane is (l, g): l = lane % 16, g = lane / 16.
//
// Scores are made transposed, S^T = K Q^T, by 16x16x128 products of 4-bit keys
// (row l of a tile, values 32g .. 32g + 31: 16 neighbouring bytes of the cache,
// with the byte of their scale) and 8-bit queries (row l, values 16g .. + 15 and
// 64 + 16g .. + 15).  The result has the tile's tokens 4g .. 4g + 3 of row l in a
// lane, which is the layout that the second product, O^T = V^T P^T in bf16,
// wants its P in: no lane exchanges anything.  V^T's lane has D/16 neighbouring
// values (a sixteenth of a row) of tokens 4g .. 4g + 3, which is how the cache
// holds them.  O^T has values (D/4) g .. of row l in a lane.
// ---------------------------------------------------------------------------
template <int D>
struct Tokens {  // what a wave reads of 32 tokens
  static constexpr int kK = D == 64 ? 1 : D / 64;  // 16-byte loads of keys
  static constexpr int kV = D / 32;                // 8-byte pieces of values
  i32x4 k[kK];
  uint32_t ks[kK];  // their scales' bytes
  u32x4 v[kV / 2];  // tile 0's, then tile 1's
  uint32_t vs[2];   // scales of 4 tokens
};

// The sum of `parts` such products is Q's exactly: bf16 has 8 bits, an e4m3
// value 4, fp16 11.  A row has one scale, which takes its largest magnitude
// to [128, 256); part i holds what the parts before left, times 2^(5 i).
template <int D, int PARTS>
struct Query {
  static constexpr int kSteps = D == 64 ? 1 : D / 128;
  static constexpr int kWords = D == 64 ? 4 : 8;
  uint32_t w[PARTS][kSteps][kWords];
  uint32_t scale;  // the byte of part 0's
};

template <int D, int DT, int PARTS>
__device__ __forceinline__ void load_query(Query<D, PARTS>* out, const char* row, bool live, int g) {
  constexpr int kHalves = D / 64;  // pieces of 16 values: (64 h + 16 g)
  float x[kHalves][16];
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    if (live) {
      Eight<DT> e[2];
      e[0].load(row + (64 * h + 16 * g) * 2);
      e[1].load(row + (64 * h + 16 * g + 8) * 2);
      e[0].get(x[h]);
      e[1].get(x[h] + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[h][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[h][i]) & 0x7fffffffu);
  }
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
  // 2^(e - 7) of a magnitude in [2^e, 2^(e + 1)); parts behind go 2^-10 below it.
  // Rows that are not finite get the scale that stands for NaN.
  const int e = (int)(m >> 23) - 7;
  const int byte = m >= 0x7f800000u ? 255 : min(max(e, 16), 250);
  out->scale = (uint32_t)byte;
  const float up = __uint_as_float((uint32_t)(254 - (byte == 255 ? 127 : byte)) << 23);
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = byte == 255 ? 0.f : x[h][i + j] * up;
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
        out->w[q][h / 2][(h % 2) * 4 + i / 4] = (uint32_t)w;
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
        y[0] = (y[0] - a[0]) * 32.f;
        y[1] = (y[1] - a[1]) * 32.f;
        y[2] = (y[2] - b[0]) * 32.f;
        y[3] = (y[3] - b[1]) * 32.f;
      }
    }
}

// Scores of tile u's 16 tokens for a tile of rows.
template <int D, int PARTS>
__device__ __forceinline__ f32x4 scores(const Tokens<D>& t, int u, const Query<D, PARTS>& q, int g) {
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int kSteps = Query<D, PARTS>::kSteps;
#pragma unroll
  for (int part = PARTS - 1; part >= 0; --part) {  // the smallest first
    const int sb = q.scale == 255 ? 255 : (int)q.scale - 5 * part;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      // D = 64: one product's 128 values are two tiles' keys; the queries stand
      // in the half of this tile, with zeros in the other
      const int at = D == 64 ? 0 : u * kSteps + s;
      const i32x8 a = {t.k[at][0], t.k[at][1], t.k[at][2], t.k[at][3], 0, 0, 0, 0};
      const uint32_t* w = q.w[part][s];
      i32x8 b;
      int sa = (int)t.ks[at];
      if constexpr (D == 64) {
        if (g / 2 != u) sa = 127;  // the other tile's scales may be NaN, or too large for sums beside them
        const i32x8 b0 = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
        const i32x8 b1 = {0, 0, 0, 0, (int)w[0], (int)w[1], (int)w[2], (int)w[3]};
        b = u ? b1 : b0;
      } else {
        b = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], (int)w[4], (int)w[5], (int)w[6], (int)w[7]};
      }
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 0, 0, sa, 0, sb);
    }
  }
  return acc;
}

template <int SEL>
__device__ __forceinline__ uint32_t two_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}
__device__ __forceinline__ uint32_t byte_pair(uint32_t w, float scale, int sel) {
  switch (sel) {
    case 0: return two_bf16<0>(w, scale);
    case 1: return two_bf16<1>(w, scale);
    case 2: return two_bf16<2>(w, scale);
    default: return two_bf16<3>(w, scale);
  }
}

// Values 2j and 2j + 1 of the lane's sixteenth for its 8 tokens, as the A
// operands of two products.
template <int D>
__device__ __forceinline__ void value_pair(const Tokens<D>& t, const float* scale, int j, u32x4* even, u32x4* odd) {
  constexpr int kBytes = D / 32;  // of a token
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const int at0 = k * kBytes + j, at1 = at0 + kBytes;
      constexpr int kWordsOfTile = kBytes;  // 4 tokens x kBytes / 4
      const int w0 = u * kWordsOfTile + at0 / 4, w1 = u * kWordsOfTile + at1 / 4;
      const uint32_t a = byte_pair(t.v[w0 / 4][w0 % 4], scale[4 * u + k], at0 % 4);
      const uint32_t b = byte_pair(t.v[w1 / 4][w1 % 4], scale[4 * u + k + 1], at1 % 4);
      (*even)[2 * u + k / 2] = __builtin_amdgcn_perm(b, a, 0x05040100u);
      (*odd)[2 * u + k / 2] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    }
  }
}

// The state of a tile of rows in a wave.  m is the reference of the row's
// exponentials (-inf: none yet), `base` what is subtracted (m, or 0).
template <int D>
struct Rows16 {
  f32x4 o[D / 16];
  f32x4 l;  // sums of the probabilities, the same in all four
  float m, base;
};

// ---------------------------------------------------------------------------
// The tree: for each node of the group of rows its ancestors, as bits, and
// each node's depth.
// ---------------------------------------------------------------------------
struct TreeShared {
  int32_t parent[SV_MAX_N];
  int32_t depth[SV_MAX_N];
};

template <int D, int TILES, int DT>
__global__ __launch_bounds__(kThreads, TILES * D <= 256 ? 2 : 1) void attention_kernel(const AttentionParams p) {
  constexpr int kParts = DT == SV_F16 ? 3 : 2;
  constexpr int kProbs = DT == SV_F16 ? 2 : 1;
  constexpr int kRows = TILES * kTile;
  constexpr int kStride = D + 4;
  __shared__ __align__(16) float s_o[kWaves][kTile][kStride];
  __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];
  __shared__ TreeShared s_tree;
  __shared__ uint32_t s_bits[kRows][SV_MAX_N / 32];
  __shared__ int64_t s_scan[kWaves];
  __shared__ int64_t s_first[2];  // the block's first sequence, steps before it

  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l = lane % 16, g = lane / 16;
  const int64_t each = (int64_t)p.c.H * p.groups;  // items of a sequence
  AttentionItem* const desc = static_cast<AttentionItem*>(p.desc);

  // all sequences' steps, and the one this block begins in
  int64_t total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t before = 0;
    int64_t begin = 0, blocks = 0;
    if (pass) {
      blocks = min((int64_t)gridDim.x, total);
      if ((int64_t)blockIdx.x >= blocks) break;
      begin = start_of(blockIdx.x, total, blocks);
    }
    for (int64_t b0 = 0; b0 < p.B; b0 += kThreads) {
      const int64_t b = b0 + tid;
      int64_t mine = 0;
      if (b < p.B) {
        const Span s = span_of(p, b);
        mine = s.units * each;
        if (s.news < 0 && pass == 0 && blockIdx.x == 0) flag(p.err, SV_DERR_RANGE);
      }
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int64_t up = __shfl_up(incl, o, kWave);
        if (lane >= o) incl += up;
      }
      if (lane == kWave - 1) s_scan[wave] = incl;
      __syncthreads();
      for (int w = 0; w < wave; ++w) incl += s_scan[w];
      int64_t sum = 0;
      for (int w = 0; w < kWaves; ++w) sum += s_scan[w];
      if (pass && mine && before + incl - mine <= begin && begin < before + incl) {
        s_first[0] = b;
        s_first[1] = before + incl - mine;
      }
      before += sum;
      __syncthreads();
    }
    total = before;
  }
  const int64_t blocks = min((int64_t)gridDim.x, total);
  if ((int64_t)blockIdx.x >= blocks) {
    if (tid == 0) desc[blockIdx.x].b = -1;
    return;
  }
  const int64_t begin = start_of(blockIdx.x, total, blocks), end = start_of(blockIdx.x + 1, total, blocks);
  int64_t b = s_first[0], line = s_first[1];  // steps before sequence b
  int64_t at = begin;
  Span span = span_of(p, b);
  bool open = false;  // whether the last item goes on in the next block

  while (at < end) {
    while (at >= line + span.units * each) {
      line += span.units * each;
      span = span_of(p, ++b);
    }
    const int64_t item = (at - line) / span.units;
    const int64_t first = line + item * span.units;  // the item's first step
    const int64_t stop = min(first + span.units, end);
    const int h = (int)(item / p.groups), group = (int)(item % p.groups);
    const int64_t u0 = span.u0 + (at - first), u1 = span.u0 + (stop - first);
    const bool whole = at == first && stop == first + span.units;
    const int slot = 2 * (int)blockIdx.x + (at == begin ? 0 : 1);
    const int len = span.len, news = span.news;
    const int hi = len + news;  // tokens and nodes
    const int row0 = group * kRows;

    // ---- the rows
    __syncthreads();
    const int node0 = row0 / p.G;  // first node of the group
    const int nodes = min((row0 + kRows - 1) / p.G, p.N - 1) - node0 + 1;
    if (p.parent) {
      const int32_t* parent = p.parent + b * p.N;
      for (int i = tid; i < news; i += kThreads) s_tree.parent[i] = i ? parent[i] : -1;
      for (int i = tid; i < nodes * (SV_MAX_N / 32); i += kThreads) (&s_bits[0][0])[i] = 0;
      __syncthreads();
      for (int i = tid; i < news; i += kThreads) {
        int n = i, d = 0;
        bool bad = false;
        for (;;) {
          const int up = s_tree.parent[n];
          if (n == 0) break;
          if (up < 0 || up >= n) {
            bad = true;
            break;
          }
          n = up;
          ++d;
        }
        if (bad) flag(p.err, SV_DERR_TREE);
        s_tree.depth[i] = d;
        if (i >= node0 && i < node0 + nodes) {
          uint32_t* bits = s_bits[i - node0];
          int a = i;
          for (int k = 0; k <= d; ++k) {
            bits[a / 32] |= 1u << (a % 32);
            a = a ? s_tree.parent[a] : 0;
          }
        }
      }
      __syncthreads();
    }
    Query<D, kParts> q[TILES];
    Rows16<D> rows[TILES];
    int node[TILES], pos[TILES];
    float slope[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int row = row0 + t * kTile + l;
      const int n = row / p.G, head = h * p.G + row % p.G;
      const bool live = n < news;
      node[t] = live ? n : -1;
      pos[t] = len + (live ? (p.parent ? s_tree.depth[n] : n) : 0);
      slope[t] = live && p.slopes ? p.slopes[head] * kLog2e : 0.f;
      load_query<D, DT, kParts>(&q[t], p.q + b * p.qs[0] + n * p.qs[1] + head * p.qs[2], live, g);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) rows[t].o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      rows[t].l = f32x4{0.f, 0.f, 0.f, 0.f};
      rows[t].m = kNegInf;
      rows[t].base = 0.f;
    }

    // ---- the tokens
    const int32_t* pages = p.c.pages + b * p.c.max_pages;
    const int64_t in_page = ((int64_t)1 << p.c.pshift) - 1;
    const int last_tile = (hi - 1) / kTile * kTile;
    const auto page_at = [&](int64_t token) {
      return __builtin_amdgcn_readfirstlane(pages[token >> p.c.pshift]);
    };
    const auto tile_at = [&](int64_t u, int tile) {
      return (int)min(u * kAttentionUnit + wave * kWaveTokens + tile * kTile, (int64_t)last_tile);
    };
    const auto fetch = [&](int64_t u, Tokens<D>* t, int* bad) {
      *bad = 0;
      const char* base[2];
      int64_t s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tt = tile_at(u, i);
        int id = page_at(tt);
        if ((uint32_t)id >= (uint32_t)p.c.num_pages) {
          id = 0;
          *bad |= 1 << i;
        }
        base[i] = p.c.pool + id * p.c.page_stride + h * p.c.head;
        s[i] = tt & in_page;
      }
      if constexpr (D == 64) {
        const int i = g / 2;
        const char* kb = i ? base[1] : base[0];
        const int64_t row = (i ? s[1] : s[0]) + l;
        t->k[0] = *reinterpret_cast<const i32x4*>(kb + row * (D / 2) + (g % 2) * 16);
        t->ks[0] = (uint8_t)kb[p.c.ks + row * (D / 32) + g % 2];
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < D / 128; ++k) {
            t->k[i * (D / 128) + k] = *reinterpret_cast<const i32x4*>(base[i] + (s[i] + l) * (D / 2) + k * 64 + g * 16);
            t->ks[i * (D / 128) + k] = (uint8_t)base[i][p.c.ks + (s[i] + l) * (D / 32) + k * 4 + g];
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const char* vb = base[i] + p.c.vc + ((s[i] / 4 + g) * 16 + l) * (D / 8);
        if constexpr (D == 64) {
          const uint64_t w = *reinterpret_cast<const uint64_t*>(vb);
          t->v[0][2 * i] = (uint32_t)w;
          t->v[0][2 * i + 1] = (uint32_t)(w >> 32);
        } else {
#pragma unroll
          for (int k = 0; k < D / 128; ++k) t->v[i * (D / 128) + k] = reinterpret_cast<const u32x4*>(vb)[k];
        }
        t->vs[i] = *reinterpret_cast<const uint32_t*>(base[i] + p.c.vs +
                                                      ((s[i] / 4 + g) * (D / 32) + l * (D / 16) / 32) * 4);
      }
    };

    const auto step = [&](int64_t u, Tokens<D>& t, int bad) {
      const int t0 = (int)(u * kAttentionUnit) + wave * kWaveTokens;
      if (t0 >= hi) return;
      if (bad && lane == 0) flag(p.err, SV_DERR_RANGE);
      // some row does not see some of these tokens
      const bool partial = bad || t0 + kWaveTokens > len || (p.reach > 0 && t0 <= hi - 1 - p.reach);
      float scale[8];
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t s = (t.vs[i / 4] >> (8 * (i % 4))) & 255u;
        // beyond the largest scale there is only NaN, and bytes never written,
        // whose values may overflow: they are added where they are seen
        nan = nan || s > 252;
        if (partial && s > 252) s = 127;
        scale[i] = scale_of(s);
      }
      nan = partial && __any(nan);
      u32x4 pr[TILES][kProbs];
      uint32_t seen[TILES];  // bit i: row l sees token i of the lane's 8
#pragma unroll
      for (int r = 0; r < TILES; ++r) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x4 s = scores<D, kParts>(t, i, q[r], g);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[4 * i + k] = s[k] * p.scale;
        }
        if (p.cap > 0.f) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // cap tanh(s / cap) = cap (1 - 2 / (1 + e^(2 s / cap)))
            const float e = __builtin_amdgcn_exp2f(x[i] * (2.f * kLog2e / p.cap));
            x[i] = p.cap - 2.f * p.cap * __builtin_amdgcn_rcpf(1.f + e);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= kLog2e;
        seen[r] = 0xffu;
        if (partial || p.slopes) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int tok = t0 + (i / 4) * kTile + 4 * g + i % 4;
            const int j = tok - len;  // node of the window, if not before it
            int at_pos = tok;
            bool see = node[r] >= 0 && tok < hi && !(bad >> (i / 4) & 1);
            if (see && j >= 0) {
              if (p.parent) {
                see = s_bits[node[r] - node0][j / 32] >> (j % 32) & 1;
                at_pos = len + s_tree.depth[j];
              } else {
                see = j <= node[r];
              }
            }
            const int d = pos[r] - at_pos;
            if (p.reach > 0) see = see && d < p.reach;
            x[i] -= slope[r] * (float)d;
            if (!see) {
              x[i] = kNegInf;
              seen[r] &= ~(1u << i);
            }
          }
        }
        float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        // A new reference only where a row's scores pass the old one by 2^8:
        // probabilities up to that are as exact
        if (__any(top > rows[r].m + 8.f)) {
          top = fmaxf(top, __shfl_xor(top, 16, kWave));
          top = fmaxf(top, __shfl_xor(top, 32, kWave));
          const float m = fmaxf(rows[r].m, top);
          const float base = m > kNegInf ? m : 0.f;
          const float f = __builtin_amdgcn_exp2f(rows[r].m - base);
          rows[r].m = m;
          rows[r].base = base;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) rows[r].o[i] *= f;
          rows[r].l *= f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_exp2f(x[i] - rows[r].base);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pr[r][0][i] = pack_bf16(x[2 * i], x[2 * i + 1]);
          if constexpr (kProbs == 2) {
            const float lo = x[2 * i] - __uint_as_float(pr[r][0][i] << 16);
            const float up = x[2 * i + 1] - __uint_as_float(pr[r][0][i] & 0xffff0000u);
            pr[r][1][i] = pack_bf16(lo, up);
          }
        }
      }
      const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
      for (int r = 0; r < TILES; ++r)
#pragma unroll
        for (int c = kProbs - 1; c >= 0; --c)
          rows[r].l = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, ones),
                                                              __builtin_bit_cast(bf16x8, pr[r][c]), rows[r].l, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        u32x4 va, vb;
        value_pair<D>(t, scale, j, &va, &vb);
#pragma unroll
        for (int r = 0; r < TILES; ++r)
#pragma unroll
          for (int c = kProbs - 1; c >= 0; --c) {
            rows[r].o[2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, va), __builtin_bit_cast(bf16x8, pr[r][c]), rows[r].o[2 * j], 0, 0, 0);
            rows[r].o[2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, vb), __builtin_bit_cast(bf16x8, pr[r][c]), rows[r].o[2 * j + 1], 0, 0, 0);
          }
      }
      if (nan) {
        // the NaN blocks among tokens that not all rows see: a product of what
        // is NaN with what is seen says which sums they reach
        u32x4 va = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (((t.vs[i / 4] >> (8 * (i % 4))) & 255u) > 252) va[i / 2] |= 0x3f80u << (16 * (i % 2));
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
          u32x4 vb = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (seen[r] >> i & 1) vb[i / 2] |= 0x3f80u << (16 * (i % 2));
          const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
          const f32x4 hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, va),
                                                                    __builtin_bit_cast(bf16x8, vb), zero, 0, 0, 0);
          // a lane's sixteenth lies in one block: its sums all have it
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (hit[k] > 0.f) rows[r].o[i][k] = __builtin_nanf("");
        }
      }
    };

    {
      Tokens<D> now, next;
      int bad, bad_next = 0;
      fetch(u0, &now, &bad);
      for (int64_t u = u0; u < u1; ++u) {
        if (u + 1 < u1) fetch(u + 1, &next, &bad_next);
        step(u, now, bad);
        now = next;
        bad = bad_next;
      }
    }

    // ---- the waves' sums together, a tile of rows at a time
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      if (g == 0) {
        s_m[wave][t * kTile + l] = rows[t].m;
        s_l[wave][t * kTile + l] = rows[t].l[0];
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      float m = kNegInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) m = fmaxf(m, s_m[w][t * kTile + l]);
      const float f = rows[t].m > kNegInf ? __builtin_amdgcn_exp2f(rows[t].m - m) : (m > kNegInf ? 0.f : 1.f);
      // NaN scores leave m at -inf: their sums are NaN, times anything
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < D / 16; i += 4) {
          const f32x4 v = {rows[t].o[i][k] * f, rows[t].o[i + 1][k] * f, rows[t].o[i + 2][k] * f, rows[t].o[i + 3][k] * f};
          *reinterpret_cast<f32x4*>(&s_o[wave][l][(4 * g + k) * (D / 16) + i]) = v;
        }
      __syncthreads();
      // a row to 16 threads, D/16 neighbouring values each
      const int r = tid / 16, c = tid % 16;
      const int rr = t * kTile + r, row = row0 + rr;
      const int n = row / p.G, head = h * p.G + row % p.G;
      float mm = kNegInf, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][rr]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = s_m[w][rr];
        ll += s_l[w][rr] * (mw > kNegInf ? __builtin_amdgcn_exp2f(mw - mm) : (mm > kNegInf ? 0.f : 1.f));
      }
      float o[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; i += 4) {
        f32x4 v = *reinterpret_cast<const f32x4*>(&s_o[0][r][c * (D / 16) + i]);
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += *reinterpret_cast<const f32x4*>(&s_o[w][r][c * (D / 16) + i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i + k] = v[k];
      }
      if (whole) {
        if (n < news) {
          const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) o[i] = ll == 0.f ? 0.f : o[i] * inv;
          char* out = p.out + b * p.os[0] + n * p.os[1] + head * p.os[2] + c * (D / 16) * 2;
          if constexpr (D == 64) {
            uint64_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint16_t e = DT == SV_F16 ? __builtin_bit_cast(uint16_t, (_Float16)o[i])
                                              : __builtin_bit_cast(uint16_t, (__bf16)o[i]);
              w |= (uint64_t)e << (16 * i);
            }
            *reinterpret_cast<uint64_t*>(out) = w;
          } else {
#pragma unroll
            for (int i = 0; i < D / 16; i += 8) {
              Eight<DT> e;
              e.set(o + i);
              *reinterpret_cast<u32x4*>(out + i * 2) = e.w[0];
            }
          }
          if (p.lse && c == 0)
            p.lse[((int64_t)b * p.N + n) * p.Hq + head] =
                ll == 0.f ? kNegInf : (mm > kNegInf ? mm : 0.f) / kLog2e + __builtin_amdgcn_logf(ll) / kLog2e;
        }
      } else {
        float* po = p.part_o + ((int64_t)slot * kRows + rr) * D + c * (D / 16);
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)
          *reinterpret_cast<f32x4*>(po + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
        if (c == 0) {
          p.part_ml[((int64_t)slot * kRows + rr) * 2] = mm;
          p.part_ml[((int64_t)slot * kRows + rr) * 2 + 1] = ll;
        }
      }
      __syncthreads();
    }
    if (at == first && stop < first + span.units) {  // the item goes on: its first block describes it
      open = true;
      if (tid == 0) {
        AttentionItem d;
        d.b = (int)b;
        d.h = h;
        d.group = group;
        d.first = blockIdx.x;
        d.last = block_of(first + span.units - 1, total, blocks);
        d.slot = slot;
        d.pad[0] = d.pad[1] = 0;
        desc[blockIdx.x] = d;
      }
    }
    at = stop;
  }
  if (!open && tid == 0) desc[blockIdx.x].b = -1;
}

// ---------------------------------------------------------------------------
// Items that several blocks share: their parts together.
// ---------------------------------------------------------------------------
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void join_kernel(const AttentionParams p) {
  const AttentionItem it = static_cast<const AttentionItem*>(p.desc)[blockIdx.x];
  if (it.b < 0) return;
  const int rows = p.tiles * kTile;
  const int r = blockIdx.y * kTile + threadIdx.x / 16, c = threadIdx.x % 16;
  const int row = it.group * rows + r;
  const int n = row / p.G, head = it.h * p.G + row % p.G;
  const int news = p.news ? p.news[it.b] : p.N;
  if (n >= news) return;
  const auto slot_of = [&](int j) { return (int64_t)(j == it.first ? it.slot : 2 * j) * rows + r; };
  float m = kNegInf;
  for (int j = it.first; j <= it.last; ++j) m = fmaxf(m, p.part_ml[slot_of(j) * 2]);
  float o[D / 16], l = 0.f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i] = 0.f;
  for (int j = it.first; j <= it.last; ++j) {
    const int64_t s = slot_of(j);
    const float mj = p.part_ml[s * 2];
    const float f = mj > kNegInf ? __builtin_amdgcn_exp2f(mj - m) : (m > kNegInf ? 0.f : 1.f);
    l += p.part_ml[s * 2 + 1] * f;
    const float* po = p.part_o + s * D + c * (D / 16);
#pragma unroll
    for (int i = 0; i < D / 16; i += 4) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(po + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i + k] += v[k] * f;
    }
  }
  const float inv = 1.f / l;
  char* out = p.out + it.b * p.os[0] + n * p.os[1] + head * p.os[2] + c * (D / 16) * 2;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const float y = l == 0.f ? 0.f : o[i] * inv;
    reinterpret_cast<uint16_t*>(out)[i] =
        DT == SV_F16 ? __builtin_bit_cast(uint16_t, (_Float16)y) : __builtin_bit_cast(uint16_t, (__bf16)y);
  }
  if (p.lse && c == 0)
    p.lse[((int64_t)it.b * p.N + n) * p.Hq + head] =
        l == 0.f ? kNegInf : (m > kNegInf ? m : 0.f) / kLog2e + __builtin_amdgcn_logf(l) / kLog2e;
}

template <int D, int DT>
hipError_t attention(const AttentionParams& p, hipStream_t s) {
  const dim3 grid((uint32_t)p.blocks);
  switch (p.tiles) {
    case 1: attention_kernel<D, 1, DT><<<grid, kThreads, 0, s>>>(p); break;
    case 2: attention_kernel<D, 2, DT><<<grid, kThreads, 0, s>>>(p); break;
    default:
      if constexpr (D != 256) {
        if (p.tiles == 3)
          attention_kernel<D, 3, DT><<<grid, kThreads, 0, s>>>(p);
        else
          attention_kernel<D, 4, DT><<<grid, kThreads, 0, s>>>(p);
      }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  join_kernel<D, DT><<<dim3((uint32_t)p.blocks, (uint32_t)p.tiles), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_attention(const AttentionParams& p, sv_dtype dt, int D, hipStream_t s) {
  if (dt == SV_BF16)
    return D == 64 ? attention<64, SV_BF16>(p, s) : D == 128 ? attention<128, SV_BF16>(p, s) : attention<256, SV_BF16>(p, s);
  return D == 64 ? attention<64, SV_F16>(p, s) : D == 128 ? attention<128, SV_F16>(p, s) : attention<256, SV_F16>(p, s);
}

}  // namespace sv
