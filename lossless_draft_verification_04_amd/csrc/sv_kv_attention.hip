// sv_kv_attention.hip -- attention of a window's nodes over the 4-bit cache.
//
// One pass over the tokens with a running reference and sum of each row:
//   out_i = sum_j 2^(s_ij - m_i) v_j / sum_j 2^(s_ij - m_i),  s in exponents of 2.
// Rows are nodes x query heads of one key head, in tiles of 16; a step of a wave
// is 32 tokens.  A wave holds its rows' sums in registers; the waves' streams of
// tokens and the blocks' parts of a sequence are joined at the end, always in
// the same order.
//
// What bounds it (6.1 TB/s is what a read of HBM reaches, 1147 TFLOP/s what a large
// bf16 product does; busy: shares of the kernel's time by counters; the times of
// this file, one build against another in turn on one device, belong together):
//   few rows: memory.  64 sequences of one token, 8 x 128 heads: 428 MB in 96 us,
//     4.5 TB/s, about 5 once it runs; its start, the blocks' ends and the join are
//     some 15 us.  With heads of 64 (214 MB, 70 to 75 us with a bias) a step has half
//     the bytes for as many addresses, scores and exponentials: vector instructions
//     busy 58%, matrix 9%.
//   many rows: vector and matrix instructions, in part one after the other.  32
//     chains of 17 nodes x 32 heads of 128: 117 to 120 us, of which memory would need
//     37 and the products, at a large product's rate, 48; busy 45% and 26%.  The
//     conversions of keys and values are shared by a wave's tiles, the exponentials
//     are not.  Trees of heads of 256 in fp16, with a cap: 61% and 36%.
//   one window: 16.5 us of dependent loads (lengths, queries, pages, tokens, parts),
//     5 of them the second launch.
#include "sv_kv.hpp"

namespace sv {

namespace {

constexpr int kTile = 16;       // tokens of a tile, rows of a tile
constexpr int kWaveTokens = 32; // tokens of a wave's step: two tiles

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
// Blocks of the join, each of which looks through all items: 256, 512, 1024, 2048
// take 15.9, 16.5, 17.8, 19.8 us in all for one window, 124, 119, 121, 125 for 32
// chains of 17 nodes x 32 heads.
constexpr int kJoinBlocks = 512, kJoinThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 y = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
}

// ---------------------------------------------------------------------------
// Which part of the work a block does: all steps (32 tokens of a sequence for
// each of the block's streams, for one key head and group of rows) stand in one
// line, sequence by sequence, and block i of W takes steps [i T / W, (i + 1) T / W).
// ---------------------------------------------------------------------------
struct Span {
  int32_t len, news;  // news = 0: nothing to do
  int64_t u0, units;  // first step of the sequence's tokens, number of steps
};

// The first token that a row of the window may see: those of a root at place len.
__device__ __forceinline__ int64_t first_seen(int32_t len, int32_t reach) {
  return reach > 0 ? max((int64_t)len - reach + 1, (int64_t)0) : 0;
}

template <int UNIT>
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
  s.u0 = first_seen(s.len, p.reach) / UNIT;
  s.units = ((int64_t)s.len + s.news + UNIT - 1) / UNIT - s.u0;
  return s;
}

// First step of block i; the number of blocks is one or three times a power of
// two, and blocks take a step each where there are fewer steps.
__device__ __forceinline__ int64_t start_of(int64_t i, int64_t total, const AttentionParams& p) {
  if (total < p.blocks) return min(i, total);
  const uint64_t x = (uint64_t)i * (uint64_t)total >> p.log_blocks;
  return (int64_t)(p.blocks >> p.log_blocks == 3 ? x / 3 : x);
}
// The block that has step x.
__device__ __forceinline__ int block_of(int64_t x, int64_t total, const AttentionParams& p) {
  return total < p.blocks ? (int)x : (int)((((uint64_t)x + 1) * (uint64_t)p.blocks - 1) / (uint64_t)total);
}
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
  return (uint64_t)x >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}

// ---------------------------------------------------------------------------
// Fragments.  A wave's lane is (l, g): l = lane % 16, g = lane / 16.
//
// Scores are made transposed, S^T = K Q^T: the codes of the keys become bf16 as
// they are multiplied (which holds them exactly), 8 neighbouring values of row l
// in a lane, beside the same values of a query.  At D = 64 a lane has values
// 16g .. 16g + 15, else 32g .. 32g + 31 of each 128 (16 neighbouring bytes of the
// cache); products take them 8 at a time.  The result has the tile's tokens
// 4g .. 4g + 3 of row l in a lane, which is the layout that the second product,
// O^T = V^T P^T in bf16, wants its P in: no lane exchanges anything.  V^T's lane
// has D/16 neighbouring values (a sixteenth of a row) of tokens 4g .. 4g + 3,
// which is how the cache holds them.  O^T has values (D/4) g .. of row l in a lane.
//
// The product of 4 and 8 bits would take the codes as they are, but it is no sum
// in 32 bits: within a block of 32 it drops what lies some 2^-17 below the largest
// product (51200 sums of random codes were off by up to 2^-10.4 of it; 76800 of the
// bf16 product's by 2^-20.5), so that beside one large channel a score is a guess.
// What bf16 costs: conversions in each wave, and for fp16 two products of 16 bits
// for three of 8 -- 2 trees of 64 nodes x 16 heads of 256 in fp16 over 65536 tokens
// 265 us, 231 with 4 and 8 bits; 32 chains of 17 nodes 119 and 117; single tokens
// and windows the same.
// ---------------------------------------------------------------------------
template <int D>
struct Tokens {  // what a wave reads of 32 tokens
  static constexpr int kK = D / 64;    // 16 bytes of keys: tile 0's, then tile 1's
  static constexpr int kS = D == 64 ? 2 : kK;
  static constexpr int kV = D / 32;    // 8-byte pieces of values
  u32x4 k[kK];
  uint32_t ks[kS];  // their scales' bytes
  u32x4 v[kV / 2];  // tile 0's, then tile 1's
  uint32_t vs[2];   // scales of 4 tokens
};

// A query's values as operands: bf16 as it is, fp16 (11 bits of digits) as two
// parts of bf16 (8), the second what the first leaves: at most 3 bits, so the sum
// of their products is Q's.
template <int D, int PARTS>
struct Query {
  static constexpr int kSteps = D / 32;  // products of 32 values
  u32x4 w[PARTS][kSteps];
};

template <int D>
struct QueryRow {  // a lane's 8 values for each product
  u32x4 v[D / 32];
};
template <int D>
__device__ __forceinline__ void fetch_query(QueryRow<D>* out, const char* row, bool live, int g) {
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    const int at = D == 64 ? 16 * g + 8 * s : s / 4 * 128 + 32 * g + s % 4 * 8;
    out->v[s] = live ? *reinterpret_cast<const u32x4*>(row + at * 2) : u32x4{0, 0, 0, 0};
  }
}
template <int D, int DT, int PARTS>
__device__ __forceinline__ void split_query(Query<D, PARTS>* out, const QueryRow<D>& in, bool turn) {
  constexpr uint32_t kInf = DT == SV_F16 ? 0x7c00u : 0x7f80u;
  const uint32_t sign = turn ? 0x80008000u : 0u;
  bool bad = false;  // an infinity or NaN in the row
#pragma unroll
  for (int s = 0; s < D / 32; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = in.v[s][i];
      bad = bad || (w & kInf) == kInf || (w >> 16 & kInf) == kInf;
      if constexpr (DT == SV_F16) {
        const float x = (float)__builtin_bit_cast(_Float16, (uint16_t)(w & 0xffffu));
        const float y = (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
        const uint32_t hi = pack_bf16(x, y);
        out->w[0][s][i] = hi ^ sign;
        out->w[1][s][i] = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u)) ^ sign;
      } else {
        out->w[0][s][i] = w ^ sign;
      }
    }
  const uint64_t any = __ballot(bad);  // lanes l, l + 16, .. share a row
  if (any >> (threadIdx.x % 16) & 0x0001000100010001ull)
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
      for (int s = 0; s < D / 32; ++s) out->w[p][s] = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
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

// The lane's 8 values of tile u's keys for product s, as bf16.
template <int D>
__device__ __forceinline__ u32x4 key_step(const Tokens<D>& t, int u, int s) {
  const int at = D == 64 ? 0 : u * (D / 128) + s / 4;
  const uint32_t w = t.k[at][D == 64 ? 2 * u + s : s % 4];
  const float scale = scale_of(t.ks[D == 64 ? u : at]);
  return u32x4{two_bf16<0>(w, scale), two_bf16<1>(w, scale), two_bf16<2>(w, scale), two_bf16<3>(w, scale)};
}

// Scores of both tiles' tokens for TT tiles of rows.  `words(r, part, s)`: a
// query's values.  AHEAD: they are asked for a product ahead (where they lie in LDS
// and registers are left for them: trees of heads of 256 in fp16 274 to 265 us).
template <int D, int PARTS, int TT, bool AHEAD, typename W>
__device__ __forceinline__ void scores(const Tokens<D>& t, f32x4 (*acc)[2], const W& words) {
#pragma unroll
  for (int r = 0; r < TT; ++r) acc[r][0] = acc[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 q[2][TT][PARTS];
  const auto take = [&](int s) {
#pragma unroll
    for (int r = 0; r < TT; ++r)
#pragma unroll
      for (int part = 0; part < PARTS; ++part) q[s % 2][r][part] = words(r, part, s);
  };
  if constexpr (AHEAD) take(0);
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    if constexpr (AHEAD) {
      if (s + 1 < D / 32) take(s + 1);
    } else {
      take(s);
    }
    const u32x4 k[2] = {key_step<D>(t, 0, s), key_step<D>(t, 1, s)};
#pragma unroll
    for (int r = 0; r < TT; ++r)
#pragma unroll
      for (int part = PARTS - 1; part >= 0; --part)  // the smaller first
#pragma unroll
        for (int u = 0; u < 2; ++u)
          acc[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[u]),
                                                              __builtin_bit_cast(bf16x8, q[s % 2][r][part]), acc[r][u], 0, 0, 0);
    if constexpr (AHEAD) __builtin_amdgcn_sched_barrier(0);
  }
}

// The scale of token k of 4 from the word that holds their bytes, for a
// conversion: it takes the exponent's bits alone, so the bits of the
// neighbouring bytes may stand around them.
__device__ __forceinline__ float scale_in(uint32_t w, int k) {
  return __uint_as_float(k == 3 ? w >> 1 : w << (23 - 8 * k));
}

// Values 2j and 2j + 1 of the lane's sixteenth for its 8 tokens, as the A
// operands of two products.
template <int D>
__device__ __forceinline__ void value_pair(const Tokens<D>& t, const uint32_t* vs, int j, u32x4* even, u32x4* odd) {
  constexpr int kBytes = D / 32;  // of a token
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const int at0 = k * kBytes + j, at1 = at0 + kBytes;
      constexpr int kWordsOfTile = kBytes;  // 4 tokens x kBytes / 4
      const int w0 = u * kWordsOfTile + at0 / 4, w1 = u * kWordsOfTile + at1 / 4;
      const uint32_t a = byte_pair(t.v[w0 / 4][w0 % 4], scale_in(vs[u], k), at0 % 4);
      const uint32_t b = byte_pair(t.v[w1 / 4][w1 % 4], scale_in(vs[u], k + 1), at1 % 4);
      (*even)[2 * u + k / 2] = __builtin_amdgcn_perm(b, a, 0x05040100u);
      (*odd)[2 * u + k / 2] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    }
  }
}

// The state of a tile of rows in a wave: `base` is the reference of the row's
// exponentials, `limit` the score beyond which it moves (-inf: there is no
// reference yet, base is 0).
template <int D>
struct Rows16 {
  f32x4 o[D / 16];
  f32x4 l;  // sums of the probabilities, the same in all four
  float base, limit;
  __device__ __forceinline__ float reference() const { return limit > kNegInf ? base : kNegInf; }
};

// The kernel's arguments, read again from where they lie, and the thread's
// number as if it were new: what a phase does not use is not kept in registers
// through it, and nothing of one phase is formed ahead of another.
__device__ __forceinline__ const AttentionParams& arguments() {
  uint64_t u = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(u));
  return *(const AttentionParams*)(const __attribute__((address_space(4))) AttentionParams*)u;
}
__device__ __forceinline__ int thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

constexpr int kChunks = SV_MAX_N / 32 + 1;  // steps of 32 tokens that hold nodes

template <int N>
struct Number {
  static constexpr int value = N;
};

// A block's waves (attention_form() says which): `SPLIT` of them take rows, TILES tiles of 16 each, beside one
// another, and there are so many streams of tokens.  Waves of the same stream
// read the same tokens, the second one out of the cache beside it.
template <int TILES, int SPLIT>
struct Form {
  static constexpr int kStreams = SPLIT == 1 ? 4 : 8 / SPLIT;
  static constexpr int kWaves = SPLIT * kStreams, kThreads = kWaves * kWave;
  static constexpr int kUnit = kStreams * kWaveTokens;  // tokens of a step
  static constexpr int kRows = SPLIT * TILES * kTile;
  static constexpr int kPages = SPLIT == 1 ? 512 : 256;  // page numbers that a wave has at a time
};

// What the waves of a block share.  QUERY: words of queries kept here.
template <int D, typename FORM, int QUERY>
struct Shared : FORM {
  using FORM::kRows;
  using FORM::kWaves;
  static constexpr int ROWS = kRows;
  union {
    struct {  // while a segment is worked on
      u32x4 q[QUERY ? QUERY : 1];  // queries of many rows (the waves' are the same)
      int32_t page[kWaves][FORM::kPages];  // each wave's own; -1 for one that is none of the pool
      int32_t parent[SV_MAX_N];  // a tree's window
    };
    float o[kWaves][kTile][D + 4];  // as it ends
  };
  float m[kWaves][ROWS], l[kWaves][ROWS];
  // trees: the nodes' depths, and what the group's rows see of the last tokens
  // before the window and of its nodes: bit i of sees[r][k] stands for token
  // 32 (len / 32 + k) + i
  int32_t depth[SV_MAX_N];
  uint32_t sees[ROWS][kChunks];
  int32_t pos[ROWS];   // the rows' positions
  float slope[ROWS];   // and slopes, of exponents of 2
  // where the block stands: steps of all, its next one, its last + 1, those
  // before sequence b, and that sequence
  int64_t scan[kWaves];
  int64_t total, at, end, line, units;
  int32_t b, len, news, u0;
  int32_t open;  // whether the last item goes on in the next block
  // the segment at hand
  int32_t first, stop, h, group, slot, whole;
};

// All sequences' steps, and the place that the block begins in; false: none.
template <typename S>
__device__ __forceinline__ bool plan(const AttentionParams& p, S& sh) {
  constexpr int kThreads = S::kThreads, kWaves = S::kWaves;
  const int tid = thread(), lane = tid % kWave, wave = tid / kWave;
  const int64_t each = (int64_t)p.c.H * p.groups;  // items of a sequence
  int64_t total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t before = 0, begin = 0;
    if (pass) {
      begin = start_of(blockIdx.x, total, p);
      if (begin >= total) return false;
      if (tid == 0) {
        sh.total = total;
        sh.at = begin;
        sh.end = start_of(blockIdx.x + 1, total, p);
        sh.open = 0;
      }
    }
    for (int64_t b0 = 0; b0 < p.B; b0 += kThreads) {
      const int64_t b = b0 + tid;
      Span s;
      int64_t mine = 0;
      if (b < p.B) {
        s = span_of<S::kUnit>(p, b);
        mine = s.units * each;
        if (s.news < 0 && pass == 0 && blockIdx.x == 0) flag(p.err, SV_DERR_RANGE);
      }
      int64_t incl = mine;
      if (p.B > 1) {
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
          const int64_t up = __shfl_up(incl, o, kWave);
          if (lane >= o) incl += up;
        }
      }
      if (p.B > 1 ? lane == kWave - 1 : tid == 0) sh.scan[wave] = incl;
      __syncthreads();
      const int waves = min((int)((p.B - b0 + kWave - 1) / kWave), kWaves);
      int64_t sum = 0;
      for (int w = 0; w < waves; ++w) {
        if (w < wave) incl += sh.scan[w];
        sum += sh.scan[w];
      }
      if (p.B <= kThreads) {  // one look is enough
        total = sum;
        begin = start_of(blockIdx.x, total, p);
        if (begin >= total) return false;
        if (tid == 0) {
          sh.total = total;
          sh.at = begin;
          sh.end = start_of(blockIdx.x + 1, total, p);
          sh.open = 0;
        }
      }
      if ((pass || p.B <= kThreads) && mine && before + incl - mine <= begin && begin < before + incl) {
        sh.b = (int32_t)b;
        sh.line = before + incl - mine;
        sh.units = s.units;
        sh.len = s.len;
        sh.news = s.news;
        sh.u0 = (int32_t)s.u0;
      }
      before += sum;
      __syncthreads();
    }
    total = before;
    if (p.B <= kThreads) return total > 0;
  }
  return true;
}

// The next segment: the part of an item that the block does.
template <typename S>
__device__ __forceinline__ void segment(const AttentionParams& p, S& sh) {
  if (thread() == 0) {
    const int64_t each = (int64_t)p.c.H * p.groups;
    const int64_t at = sh.at;
    int64_t line = sh.line, units = sh.units;
    if (at >= line + units * each) {
      int b = sh.b;
      Span span;
      do {
        line += units * each;
        span = span_of<S::kUnit>(p, ++b);
        units = span.units;
      } while (at >= line + units * each);
      sh.b = b;
      sh.line = line;
      sh.units = units;
      sh.len = span.len;
      sh.news = span.news;
      sh.u0 = (int32_t)span.u0;
    }
    const int64_t item = divide(at - line, units), first = line + item * units;  // the item's first step
    const int64_t last = first + units, stop = min(last, sh.end);
    const int h = (int)((uint32_t)item / (uint32_t)p.groups), group = (int)item - h * p.groups;
    const int slot = 2 * (int)blockIdx.x + (at == start_of(blockIdx.x, sh.total, p) ? 0 : 1);
    sh.h = h;
    sh.group = group;
    sh.first = sh.u0 + (int)(at - first);
    sh.stop = sh.u0 + (int)(stop - first);
    sh.whole = at == first && stop == last;
    sh.slot = slot;
    sh.at = stop;
    if (at == first && stop < last) {  // the item goes on: its first block describes it
      AttentionItem d;
      d.b = sh.b;
      d.h = h;
      d.group = group;
      d.news = sh.news;
      d.slot = slot;
      d.last = block_of(last - 1, sh.total, p);
      static_cast<AttentionItem*>(p.desc)[blockIdx.x] = d;
      sh.open = 1;
    }
  }
  __syncthreads();
}

// What a tree's rows see, and the nodes' depths.
template <typename S>
__device__ __forceinline__ void tree(const AttentionParams& p, S& sh) {
  constexpr int ROWS = S::kRows, kThreads = S::kThreads;
  const int tid = thread(), len = sh.len, news = sh.news;
  const int32_t* parent = p.parent + (int64_t)sh.b * p.N;
  for (int i = tid; i < news; i += kThreads) {
    const int32_t a = i ? parent[i] : -1;
    const bool bad = i && (a < 0 || a >= i);
    sh.parent[i] = bad ? -1 : a;
    if (bad) flag(p.err, SV_DERR_TREE);
  }
  const int row0 = sh.group * ROWS, lead = len % 32;  // tokens of the first of these steps that stand before the window
  const int chunks = (lead + news + 31) / 32;
  for (int i = tid; i < ROWS * chunks; i += kThreads) {
    const int r = i / chunks, k = i - r * chunks;
    sh.sees[r][k] = k == 0 && (row0 + r) / p.G < news ? (1u << lead) - 1 : 0u;
  }
  __syncthreads();
  for (int i = tid; i < news; i += kThreads) {
    int d = 0;
    for (int n = sh.parent[i]; n >= 0; n = sh.parent[n]) ++d;
    sh.depth[i] = d;
  }
  for (int r = tid; r < ROWS; r += kThreads) {
    const int n = (row0 + r) / p.G;
    if (n < news) {
      int most = p.reach > 0 ? p.reach : SV_MAX_N + 1;
      for (int a = n; a >= 0 && most > 0; a = sh.parent[a], --most)
        sh.sees[r][(lead + a) / 32] |= 1u << ((lead + a) % 32);
    }
  }
  __syncthreads();
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// What a part's sums count beside others whose largest reference is m.  A part
// that saw nothing has zeros, or NaN, which stay NaN.
__device__ __forceinline__ float part_weight(float own, float m) {
  return own > kNegInf ? __builtin_amdgcn_exp2f(own - m) : (m > kNegInf ? 0.f : 1.f);
}

// The largest of three, NaN where one is: an instruction, where fmaxf first
// quiets each of its operands.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// COUNT (4, 8 or 16) of a row's sums from `col` on, and its statistics, as
// output: o / l, and the logarithm of the sum of e^s.  Biases are held relative
// to the root's distances.
template <int D, int DT, int COUNT>
__device__ __forceinline__ void finish(const AttentionParams& p, int b, int n, int head, int col, const float* o,
                                       float m, float l, int depth) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  char* out = p.out + b * p.os[0] + n * p.os[1] + head * p.os[2] + col * 2;
#pragma unroll
  for (int i = 0; i < COUNT; i += 4) {
    uint64_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float y = l == 0.f ? 0.f : o[i + k] * inv;
      const uint16_t e =
          DT == SV_F16 ? __builtin_bit_cast(uint16_t, (_Float16)y) : __builtin_bit_cast(uint16_t, (__bf16)y);
      w |= (uint64_t)e << (16 * k);
    }
    *reinterpret_cast<uint64_t*>(out + i * 2) = w;
  }
  if (p.lse && col == 0) {
    float x = l == 0.f ? kNegInf : ((m > kNegInf ? m : 0.f) + __builtin_amdgcn_logf(l)) / kLog2e;
    if (p.slopes) x -= p.slopes[head] * (float)depth;
    p.lse[((int64_t)b * p.N + n) * p.Hq + head] = x;
  }
}

// Waves of a SIMD that the registers leave room for: one tile of rows takes up
// to 128 registers at D = 64, 168 at 128 and 256 at 256, three at 128 take 256.
// Registers spilled, or one wave a SIMD, cost more than rows split over waves
// (32 windows of 5 nodes, D = 128, two tiles a wave: 65 us with 2 waves, 94 with 1).
constexpr int kernel_waves(int D, int tiles, int split) {
  return split > 1 || tiles > 1 ? 2 : D == 64 ? 4 : D == 128 ? 3 : 2;
}

template <int D, int TILES, int SPLIT, int DT>
__global__ __launch_bounds__((Form<TILES, SPLIT>::kThreads), (kernel_waves(D, TILES, SPLIT))) void attention_kernel(
    const AttentionParams) {
  using F = Form<TILES, SPLIT>;
  constexpr int kParts = DT == SV_F16 ? 2 : 1;
  constexpr int kProbs = DT == SV_F16 ? 2 : 1;
  constexpr int kRows = F::kRows, kWaves = F::kWaves, kStreams = F::kStreams, kThreads = F::kThreads, kUnit = F::kUnit;
  constexpr bool kQueryLds = TILES * D > 256 || TILES > 2 || (SPLIT > 1 && D == 128) || (D == 256 && (SPLIT > 1 || DT == SV_F16));
  constexpr int kSteps = Query<D, kParts>::kSteps;
  __shared__ __align__(16) Shared<D, F, kQueryLds ? SPLIT * TILES * kParts * kSteps * kWave : 0> sh;

  if (!plan(arguments(), sh)) {
    if (threadIdx.x == 0) static_cast<AttentionItem*>(arguments().desc)[blockIdx.x].b = -1;
    return;
  }
  bool more;
  do {
    segment(arguments(), sh);
    const int len = uniform(sh.len), news = uniform(sh.news);
    const int hi = len + news;  // tokens and nodes
    const int u0 = uniform(sh.first), u1 = uniform(sh.stop);

    // ---- the rows
    u32x4 q[kQueryLds ? 1 : TILES][kParts][kSteps];
    const int last_tile = (hi - 1) / kTile * kTile;
    {
      const AttentionParams& p = arguments();
      const int tid = thread(), lane = tid % kWave, wave = uniform(tid / kWave), l = lane % 16, g = lane / 16;
      const char* const q_at = p.q + sh.b * p.qs[0];
      const auto query = [&](int t, QueryRow<D>* out) {
        const int row = sh.group * kRows + t * kTile + l;
        const int n = row / p.G, head = sh.h * p.G + row - n * p.G;
        fetch_query<D>(out, q_at + n * p.qs[1] + head * p.qs[2], n < news, g);
      };
      constexpr int kAll = SPLIT * TILES;
      constexpr int kMine = kQueryLds ? (kAll + kWaves - 1) / kWaves : TILES;
      QueryRow<D> in[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = kQueryLds ? wave + i * kWaves : SPLIT > 1 ? wave / kStreams * TILES + i : i;
        if (t < kAll) query(t, &in[i]);
      }
      if (p.parent && (u1 * kUnit > len / 32 * 32 || p.reach > 0)) tree(p, sh);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = kQueryLds ? wave + i * kWaves : SPLIT > 1 ? wave / kStreams * TILES + i : i;
        if (t < kAll) {
          Query<D, kParts> mine;
          split_query<D, DT, kParts>(&mine, in[i], p.scale < 0.f);
#pragma unroll
          for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
              if constexpr (kQueryLds)
                sh.q[((t * kParts + part) * kSteps + s) * kWave + lane] = mine.w[part][s];
              else
                q[i][part][s] = mine.w[part][s];
            }
        }
      }
      if (tid < kRows) {
        const int row = sh.group * kRows + tid;
        const int n = row / p.G, head = sh.h * p.G + row - n * p.G;
        const bool live = n < news;
        sh.pos[tid] = len + (!live ? 0 : p.parent && p.reach > 0 ? sh.depth[n] : n);
        sh.slope[tid] = live && p.slopes ? p.slopes[head] * kLog2e : 0.f;
      }
    }
    __syncthreads();

    // ---- the tokens, for a wave of TT tiles of rows, from tile `tile0` of the group
    // on.  Waves go through this apart: no barriers in it.
    Rows16<D> rows[TILES];
    const auto body = [&](auto count) {
      constexpr int TT = decltype(count)::value;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) rows[t].o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        rows[t].l = f32x4{0.f, 0.f, 0.f, 0.f};
        rows[t].limit = kNegInf;
        rows[t].base = 0.f;
      }
      const AttentionParams& p = arguments();
      const int tid = thread(), lane = tid % kWave, wave = uniform(tid / kWave), l = lane % 16, g = lane / 16;
      const int stream = wave % kStreams, tile0 = wave / kStreams * TILES;
      // Scores are held as exponents of 2: s * unit, with s the product, or (bent)
      // already so where a cap, a bias or a scale of 0 comes first.  A negative
      // scale has turned the queries.
      const float c = fabsf(p.scale) * kLog2e;
      const bool bent = p.cap > 0.f || p.slopes || c == 0.f;
      const float unit = bent ? 1.f : c, per_unit = 1.f / unit;
      const bool is_tree = p.parent != nullptr;
      const int reach = p.reach;
      const char* const pool = p.c.pool + uniform(sh.h) * p.c.head;
      const int64_t page_stride = p.c.page_stride;
      const int pshift = p.c.pshift, in_page = (1 << pshift) - 1;
      const uint32_t off_ks = (uint32_t)p.c.ks, off_vc = (uint32_t)p.c.vc, off_vs = (uint32_t)p.c.vs;
      int page0 = 0;  // page that the wave's first number stands for
      int32_t* const page = sh.page[wave];
      // Offsets of a lane within a tile: 32 bits beside a wave's base address.
      const uint32_t lane_k = l * (D / 2) + (D == 64 ? g * 8 : g * 16);
      const uint32_t lane_ks = l * (D / 32) + (D == 64 ? g / 2 : g);
      const uint32_t lane_v = (g * 16 + l) * (D / 8), lane_vs = (g * (D / 32) + l * (D / 16) / 32) * 4;
      const auto fetch = [&](int u, Tokens<D>* t) {
        const char* base[2];
        uint32_t s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tt = min(u * kUnit + stream * kWaveTokens + i * kTile, last_tile);
          const int id = max(uniform(page[(tt >> pshift) - page0]), 0);
          base[i] = pool + id * page_stride;
          s[i] = (uint32_t)(tt & in_page);
        }
        const uint32_t at_k = opaque(lane_k), at_ks = opaque(lane_ks), at_v = opaque(lane_v), at_vs = opaque(lane_vs);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const char* kb = base[i] + s[i] * (D / 2);
          const char* sb = base[i] + off_ks + s[i] * (D / 32);
          if constexpr (D == 64) {
            const uint64_t w = *reinterpret_cast<const uint64_t*>(kb + at_k);
            t->k[0][2 * i] = (uint32_t)w;
            t->k[0][2 * i + 1] = (uint32_t)(w >> 32);
            t->ks[i] = (uint8_t)sb[at_ks];
          } else {
#pragma unroll
            for (int k = 0; k < D / 128; ++k) {
              t->k[i * (D / 128) + k] = *reinterpret_cast<const u32x4*>(kb + k * 64 + at_k);
              t->ks[i * (D / 128) + k] = (uint8_t)(sb + k * 4)[at_ks];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const char* vb = base[i] + off_vc + s[i] * (D / 2);
          if constexpr (D == 64) {
            const uint64_t w = *reinterpret_cast<const uint64_t*>(vb + at_v);
            t->v[0][2 * i] = (uint32_t)w;
            t->v[0][2 * i + 1] = (uint32_t)(w >> 32);
          } else {
#pragma unroll
            for (int k = 0; k < D / 128; ++k)
              t->v[i * (D / 128) + k] = *reinterpret_cast<const u32x4*>(vb + k * 16 + at_v);
          }
          t->vs[i] = *reinterpret_cast<const uint32_t*>(base[i] + off_vs + s[i] * (D / 32) + at_vs);
        }
      };

      // One step of a wave: 32 tokens.  `masked`: some row may not see some of them.
      const auto step = [&](int u, const Tokens<D>& t, bool masked) {
        const int t0 = u * kUnit + stream * kWaveTokens;
        if (t0 >= hi) return;
        if (kQueryLds) asm volatile("" ::: "memory");  // the queries are read where they are used
        masked = masked || t0 + kWaveTokens > len || (reach > 0 && t0 <= hi - 1 - reach);
        uint32_t vs[2] = {t.vs[0], t.vs[1]};
        uint32_t gone = 0;  // tokens without a page
        bool nan = false;
        if (masked) {
          // Beyond the largest scale there is only NaN, and bytes never written,
          // whose values may overflow: they are added where they are seen
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((vs[i / 4] >> (8 * (i % 4)) & 255u) > 252u) {
              nan = true;
              vs[i / 4] &= ~(255u << (8 * (i % 4)));
            }
          nan = __any(nan);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (page[(min(t0 + i * kTile, last_tile) >> pshift) - page0] < 0) gone |= 0xffffu << (16 * i);
        }
        // what row l of tile r sees of the lane's tokens: bits 0 .. 3 and 16 .. 19
        const auto seen = [&](int r) {
          uint32_t w = ~gone;
          const int pos = sh.pos[(tile0 + r) * kTile + l];
          if (t0 + kWaveTokens > len)
            w &= is_tree ? sh.sees[(tile0 + r) * kTile + l][t0 / 32 - len / 32] : bits_below(pos + 1 - t0);
          // (a node's place is no lower than its position: what this lets through of a tree is masked above)
          if (reach > 0) w &= ~bits_below(pos - t0 + 1 - reach);
          return w >> (4 * g);
        };
        float x[TT][8];
        {
          f32x4 sum[TT][2];
          scores<D, kParts, TT, kQueryLds && D == 256>(t, sum, [&](int r, int part, int at) {
            if constexpr (kQueryLds)
              return sh.q[(((tile0 + r) * kParts + part) * kSteps + at) * kWave + lane];
            else
              return q[r][part][at];
          });
#pragma unroll
          for (int r = 0; r < TT; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[r][i] = sum[r][i / 4][i % 4];
        }
        if (bent) {
          const AttentionParams& a = arguments();
          const float cap = a.cap * kLog2e, up = 2.f / a.cap;
          const auto bend = [&](float s) {  // cap tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap))
            return fmaf(-2.f * cap, __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(s * up)), cap);
          };
#pragma unroll
          for (int r = 0; r < TT; ++r) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[r][i] *= c;
          }
          if (a.cap > 128.f) {
            // that is off by 2^-21 of the cap: too much beside small scores under a
            // large cap, which take the series (its next term: 2^-29 of the score)
            const float part = 1.f / cap;
#pragma unroll
            for (int r = 0; r < TT; ++r) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float t = x[r][i] * part, t2 = t * t;
                const float low = fmaf(t2, fmaf(t2, fmaf(t2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
                x[r][i] = t2 < 1.f / 64.f ? x[r][i] * low : bend(x[r][i]);
              }
            }
          } else if (a.cap > 0.f) {
#pragma unroll
            for (int r = 0; r < TT; ++r)
#pragma unroll
              for (int i = 0; i < 8; ++i) x[r][i] = bend(x[r][i]);
          }
          if (a.slopes) {  // relative to the root's distances, which all of a row's scores share
            const int t1 = t0 + 4 * g - len;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = (float)(t1 + (i / 4) * kTile + i % 4);
            if (is_tree && t0 + kWaveTokens > len) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int at = t1 + (i / 4) * kTile + i % 4;
                if (at >= 0 && at < news) d[i] = (float)sh.depth[at];
              }
            }
#pragma unroll
            for (int r = 0; r < TT; ++r) {
              const float slope = sh.slope[(tile0 + r) * kTile + l];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[r][i] = fmaf(slope, d[i], x[r][i]);
            }
          }
        }
        if (masked) {
#pragma unroll
          for (int r = 0; r < TT; ++r) {
            const uint32_t w = seen(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[r][i] = w >> (16 * (i / 4) + i % 4) & 1 ? x[r][i] : kNegInf;
          }
        }
        // New references only where a row's scores pass the old one by 8: up to
        // 2^8 probabilities and their sums are as exact as up to 1, and what a row
        // moves at first is most of what it ever moves
        float top[TT];
        bool move = false;
#pragma unroll
        for (int r = 0; r < TT; ++r) {
          // (a row that sees NaN is NaN, whatever its reference)
          float m = __builtin_elementwise_maximum(x[r][0], x[r][1]);
#pragma unroll
          for (int i = 2; i < 8; i += 2) m = max3(m, x[r][i], x[r][i + 1]);
          top[r] = m;
          move = move || top[r] > rows[r].limit;
        }
        if (__any(move)) {
#pragma unroll
          for (int r = 0; r < TT; ++r) {
            if (!__any(top[r] > rows[r].limit)) continue;
            float m = fmaxf(top[r], __shfl_xor(top[r], 16, kWave));
            m = fmaxf(m, __shfl_xor(m, 32, kWave)) * unit;
            const float old = rows[r].reference();
            m = fmaxf(old, m);
            if (m > kNegInf) {
              const float f = __builtin_amdgcn_exp2f(old - m);
              rows[r].base = m;
              rows[r].limit = (m + 8.f) * per_unit;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) rows[r].o[i] *= f;
              rows[r].l *= f;
            }
          }
        }
        // Probabilities are rounded to what the second product takes, and summed as
        // rounded, so that a row whose tokens' values are alike loses nothing: to
        // the 8 bits of bf16, whose results are themselves rounded to 8 (off by
        // 0.0019 to 0.0023 of 64 bits' in all, the rounding of the results alone
        // 0.0017), in fp16 to two parts, 16 bits, beside results of 11.  Two parts
        // for bf16 too give 0.0017 and take 144 us instead of 119 for 32 chains of
        // 17 nodes x 32 heads, 377 instead of 313 for 1024 nodes, 77 instead of 73
        // for single tokens.
        u32x4 pr[TT][kProbs];
#pragma unroll
        for (int r = 0; r < TT; ++r) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[r][i] = __builtin_amdgcn_exp2f(fmaf(x[r][i], unit, -rows[r].base));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pr[r][0][i] = pack_bf16(x[r][2 * i], x[r][2 * i + 1]);
            if constexpr (kProbs == 2) {
              const float lo = x[r][2 * i] - __uint_as_float(pr[r][0][i] << 16);
              const float up = x[r][2 * i + 1] - __uint_as_float(pr[r][0][i] & 0xffff0000u);
              pr[r][1][i] = pack_bf16(lo, up);
            }
          }
        }
        // The second products ahead of the other wave's vector instructions, where
        // there are many rows: 2 trees of 64 nodes x 16 heads of 256 in fp16 over 65536
        // tokens 278 to 265 us, 1024 nodes x 32 heads 322 to 313; single tokens gain
        // nothing
        constexpr bool kAhead = SPLIT * TILES > 1;
        if constexpr (kAhead) __builtin_amdgcn_s_setprio(1);
        const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
        for (int r = 0; r < TT; ++r)
#pragma unroll
          for (int e = kProbs - 1; e >= 0; --e)
            rows[r].l = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, ones),
                                                                __builtin_bit_cast(bf16x8, pr[r][e]), rows[r].l, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          u32x4 va, vb;
          value_pair<D>(t, vs, j, &va, &vb);
#pragma unroll
          for (int r = 0; r < TT; ++r)
#pragma unroll
            for (int e = kProbs - 1; e >= 0; --e) {
              rows[r].o[2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, va), __builtin_bit_cast(bf16x8, pr[r][e]), rows[r].o[2 * j], 0, 0, 0);
              rows[r].o[2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, vb), __builtin_bit_cast(bf16x8, pr[r][e]), rows[r].o[2 * j + 1], 0, 0, 0);
            }
        }
        if constexpr (kAhead) __builtin_amdgcn_s_setprio(0);
        if (nan) {
          // the NaN blocks among tokens that not all rows see: a product of what
          // is NaN with what is seen says which sums they reach
          u32x4 va = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((t.vs[i / 4] >> (8 * (i % 4)) & 255u) > 252u) va[i / 2] |= 0x3f80u << (16 * (i % 2));
#pragma unroll
          for (int r = 0; r < TT; ++r) {
            const uint32_t w = seen(r);
            u32x4 vb = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (w >> (16 * (i / 4) + i % 4) & 1) vb[i / 2] |= 0x3f80u << (16 * (i % 2));
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

      // so many steps at a time (they may begin and end inside a page)
      const int at_once = ((F::kPages - 1) << pshift) / kUnit;
      for (int v0 = u0; v0 < u1; v0 += at_once) {
        const int v1 = min(v0 + at_once, u1);
        page0 = v0 * kUnit >> pshift;
        bool lost = false;
        {
          const AttentionParams& a = arguments();
          const int32_t* pages = a.c.pages + (int64_t)sh.b * a.c.max_pages + page0;
          const int staged = (min(v1 * kUnit - 1, last_tile) >> pshift) - page0 + 1;
          // pages behind the reach, in the step that it ends in, may be gone
          const int needed = (int)(first_seen(len, reach) >> pshift) - page0;
          for (int i = lane; i < staged; i += kWave) {
            const int32_t id = pages[i];
            const bool bad = (uint32_t)id >= (uint32_t)a.c.num_pages;
            lost = lost || (bad && i >= needed);
            page[i] = bad ? -1 : id;
          }
          if (lost) flag(a.err, SV_DERR_RANGE);
          lost = __any(lost);
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a lane reads what others have written
        }
        // The next step's loads fly while this one is worked on; behind the last
        // it is read again, so that the number of loads in flight is known.
        Tokens<D> even, odd;
        fetch(v0, &even);
        for (int u = v0;;) {
          fetch(min(u + 1, v1 - 1), &odd);
          step(u, even, lost);
          if (++u >= v1) break;
          fetch(min(u + 1, v1 - 1), &even);
          step(u, odd, lost);
          if (++u >= v1) break;
        }
      }
    };
    // The last rows' waves may have a tile less to do (5 tiles in 2 x 3: 119 us,
    // with three in both 131).
    const auto first_tile = [&](int wave) { return wave / kStreams * TILES; };
    const bool fewer = SPLIT > 1 && TILES > 1 &&
                       arguments().all_tiles - sh.group * SPLIT * TILES - first_tile(uniform(thread() / kWave)) < TILES;
    if (fewer)
      body(Number<(TILES > 1 ? TILES - 1 : 1)>{});
    else
      body(Number<TILES>{});

    // ---- the streams' sums together, a tile of rows at a time
    {
      const AttentionParams& a = arguments();
      const int id = thread(), l = id % 16, g = id % kWave / 16, wave = uniform(id / kWave);
      const int tile0 = first_tile(wave), w0 = wave / kStreams * kStreams;  // the wave of the first stream
      const int b = sh.b, row0 = sh.group * kRows + tile0 * kTile, slot = sh.slot;
      const bool whole = sh.whole;
      more = sh.at < sh.end;  // read ahead of the barriers behind which the next segment is planned
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        if (g == 0) {
          sh.m[wave][t * kTile + l] = rows[t].reference();
          sh.l[wave][t * kTile + l] = rows[t].l[0];
        }
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const bool here = t < TILES - 1 || !fewer;
        if (here) {
          const Rows16<D>& mine = rows[t];
          float m = kNegInf;
#pragma unroll
          for (int w = 0; w < kStreams; ++w) m = fmaxf(m, sh.m[w0 + w][t * kTile + l]);
          const float f = part_weight(mine.reference(), m);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < D / 16; i += 4) {
              const f32x4 v = {mine.o[i][k] * f, mine.o[i + 1][k] * f, mine.o[i + 2][k] * f, mine.o[i + 3][k] * f};
              *reinterpret_cast<f32x4*>(&sh.o[wave][l][(4 * g + k) * (D / 16) + i]) = v;
            }
        }
        __syncthreads();
        // a row to 4 threads of each stream, neighbouring values each
        constexpr int kCols = 4 * kStreams, kCount = D / kCols;
        const int in = id - w0 * kWave;
        const int r = in / kCols, col = in % kCols * kCount;
        const int rr = t * kTile + r, row = row0 + rr;
        const int n = row / a.G, head = sh.h * a.G + row - n * a.G;
        if (here && n < sh.news) {
          float mm = kNegInf, ll = 0.f;
#pragma unroll
          for (int w = 0; w < kStreams; ++w) mm = fmaxf(mm, sh.m[w0 + w][rr]);
#pragma unroll
          for (int w = 0; w < kStreams; ++w) ll += sh.l[w0 + w][rr] * part_weight(sh.m[w0 + w][rr], mm);
          float o[kCount];
#pragma unroll
          for (int i = 0; i < kCount; i += 4) {
            f32x4 v = *reinterpret_cast<const f32x4*>(&sh.o[w0][r][col + i]);
#pragma unroll
            for (int w = 1; w < kStreams; ++w) v += *reinterpret_cast<const f32x4*>(&sh.o[w0 + w][r][col + i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i + k] = v[k];
          }
          if (whole) {
            finish<D, DT, kCount>(a, b, n, head, col, o, mm, ll, a.parent ? sh.depth[n] : n);
          } else {
            const int64_t part = (int64_t)slot * kRows + tile0 * kTile + rr;
            float* po = a.part_o + part * D + col;
#pragma unroll
            for (int i = 0; i < kCount; i += 4)
              *reinterpret_cast<f32x4*>(po + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
            if (col == 0) {
              a.part_ml[part * 2] = mm;
              a.part_ml[part * 2 + 1] = ll;
            }
          }
        }
        __syncthreads();
      }
    }
  } while (more);
  if (threadIdx.x == 0 && !sh.open) static_cast<AttentionItem*>(arguments().desc)[blockIdx.x].b = -1;
}

// ---------------------------------------------------------------------------
// Items that several blocks share: their parts together.
// ---------------------------------------------------------------------------
// Blocks take some rows of an item in turn.  D/4 threads stand beside one
// another for a row's values, so a block has kSlices of them: where the item has
// few parts each takes a row and adds them up by itself; where it has many they
// take a row together, a slice of the parts each, whose sums are added up in LDS
// in a fixed order.
template <int D, int DT>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const AttentionParams p) {
  constexpr int kThreads = kJoinThreads, kWaves = kThreads / kWave;
  constexpr int kCols = D / 4, kSlices = kThreads / kCols, kFew = 8;
  constexpr int kItems = kAttentionBlocks / kThreads;  // of a thread
  __shared__ f32x4 s_sum[kSlices][kCols];
  __shared__ float s_l[kSlices], s_m[kSlices];
  __shared__ int32_t s_scan[kWaves];
  __shared__ int32_t s_first, s_piece;
  const AttentionItem* const items = static_cast<const AttentionItem*>(p.desc);
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, rows = p.split * p.tiles * kTile;
  // every block's item, if one begins there and goes on, and the pieces it makes
  const int each = p.blocks / kThreads, i0 = tid * each;
  int32_t parts[kItems], some[kItems];  // parts behind the first, rows of nodes
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int i = i0 + min(k, each - 1);
    const AttentionItem& it = items[i];
    parts[k] = it.b < 0 ? 0 : it.last - i;
    some[k] = max(min(rows, it.news * p.G - it.group * rows), 0);
  }
  int32_t end[kItems], count = 0;  // end of the pieces up to an item, from the thread's first on
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (k < each && parts[k] > 0) count += parts[k] < kFew ? (some[k] + kSlices - 1) / kSlices : some[k];
    end[k] = count;
  }
  int32_t incl = count;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(incl, o, kWave);
    if (lane >= o) incl += up;
  }
  if (lane == kWave - 1) s_scan[wave] = incl;
  __syncthreads();
  int32_t pieces = 0, before = incl - count;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += s_scan[w];
    pieces += s_scan[w];
  }
  const int col = tid % kCols, slice = tid / kCols;
  for (int x = blockIdx.x; x < pieces; x += gridDim.x) {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int32_t from = k ? end[k - 1] : 0;
      if (x - before >= from && x - before < end[k]) {
        s_first = i0 + k;
        s_piece = x - before - from;
      }
    }
    __syncthreads();
    const int first = uniform(s_first), piece = uniform(s_piece);
    const AttentionItem it = items[first];
    const int last = it.last;
    const bool few = last - first < kFew;
    const int r = few ? piece * kSlices + slice : piece;
    const int row = it.group * rows + r;
    const int n = row / p.G, head = it.h * p.G + row - n * p.G;
    const bool live = r < rows && n < it.news;
    const auto slot_of = [&](int j) { return (int64_t)(j == first ? it.slot : 2 * j) * rows + r; };
    const int from = few ? first : first + slice, by = few ? 1 : kSlices;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f, m = kNegInf;
    for (int j0 = from; j0 <= last; j0 += kFew * by) {  // kFew parts' loads at a time
      f32x2 ml[kFew];
      f32x4 v[kFew];
      float top = m;
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        const int j = j0 + i * by;
        const bool here = live && (!few || j <= last);
        const int64_t s = slot_of(min(j, last));
        ml[i] = here ? reinterpret_cast<const f32x2*>(p.part_ml)[s] : f32x2{kNegInf, 0.f};
        v[i] = here ? *reinterpret_cast<const f32x4*>(p.part_o + s * D + col * 4) : f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int i = 0; i < kFew; ++i) top = fmaxf(top, ml[i][0]);
      const float keep = part_weight(m, top);
      o *= keep;
      l *= keep;
      m = top;
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        if (j0 + i * by > last) continue;
        const float f = part_weight(ml[i][0], m);
        o += v[i] * f;
        l += ml[i][1] * f;
      }
    }
    if (!few) {
      s_sum[slice][col] = o;
      if (col == 0) {
        s_l[slice] = l;
        s_m[slice] = m;
      }
      __syncthreads();
      if (slice == 0) {
#pragma unroll
        for (int i = 1; i < kSlices; ++i) m = fmaxf(m, s_m[i]);
        const float keep = part_weight(s_m[0], m);
        o *= keep;
        l *= keep;
#pragma unroll
        for (int i = 1; i < kSlices; ++i) {
          const float f = part_weight(s_m[i], m);
          o += s_sum[i][col] * f;
          l += s_l[i] * f;
        }
      }
    }
    if (live && (few || slice == 0)) {
      int depth = n;
      if (p.lse && p.slopes && p.parent && col == 0) {
        const int32_t* parent = p.parent + (int64_t)it.b * p.N;
        depth = 0;
        for (int a = n; a > 0; ++depth) {
          const int up = parent[a];
          if (up < 0 || up >= a) break;
          a = up;
        }
      }
      const float y[4] = {o[0], o[1], o[2], o[3]};
      finish<D, DT, 4>(p, it.b, n, head, col * 4, y, m, l, depth);
    }
    __syncthreads();
  }
}

template <int D, int DT, int TILES, int SPLIT>
bool run(const AttentionParams& p, hipStream_t s) {
  if (p.tiles != TILES || p.split != SPLIT) return false;
  attention_kernel<D, TILES, SPLIT, DT><<<(uint32_t)p.blocks, Form<TILES, SPLIT>::kThreads, 0, s>>>(p);
  return true;
}

// The forms that attention_form() chooses among.
template <int D, int DT>
hipError_t attention(const AttentionParams& p, hipStream_t s) {
  bool ran = run<D, DT, 1, 1>(p, s);
  if constexpr (D == 64)
    ran = ran || run<D, DT, 2, 1>(p, s) || run<D, DT, 3, 1>(p, s) || run<D, DT, 4, 1>(p, s) || run<D, DT, 3, 2>(p, s) ||
          run<D, DT, 4, 2>(p, s) || run<D, DT, 3, 4>(p, s) || run<D, DT, 4, 4>(p, s);
  if constexpr (D == 128)
    ran = ran || run<D, DT, 2, 1>(p, s) || run<D, DT, 3, 1>(p, s) || run<D, DT, 2, 2>(p, s) || run<D, DT, 3, 2>(p, s) ||
          run<D, DT, 2, 4>(p, s) || run<D, DT, 3, 4>(p, s);
  if constexpr (D == 256) ran = ran || run<D, DT, 1, 2>(p, s) || run<D, DT, 1, 4>(p, s);
  if (!ran) return hipErrorInvalidValue;
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  join_kernel<D, DT><<<kJoinBlocks, kJoinThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int D>
hipError_t attention(const AttentionParams& p, sv_dtype dt, hipStream_t s) {
  return dt == SV_BF16 ? attention<D, SV_BF16>(p, s) : attention<D, SV_F16>(p, s);
}

}  // namespace

hipError_t launch_kv_attention(const AttentionParams& p, sv_dtype dt, int D, hipStream_t s) {
  return D == 64 ? attention<64>(p, dt, s) : D == 128 ? attention<128>(p, dt, s) : attention<256>(p, dt, s);
}

}  // namespace sv
