// sv_kv.hip -- the 4-bit cache: writing, reading back, committing a path.
//
// All three move bytes.  A thread takes 8 neighbouring values of a key and of
// a value row: 16 bytes (32 in fp32) on one side, 4 on the other.  Threads are
// ordered (sequence, group of 4 slots, head, slot, 8 values), because the
// cache holds sixteenths of value rows for 4 tokens side by side: a wave then
// writes and reads whole lines of the cache.  Bound by memory for many tokens
// (16 x 2047 tokens of 8 heads of 128 in bf16 written 22 us and read back 19;
// 8 x 16384 in fp16 read back 97 us, 5.2 TB/s; a copy 4.9), by the launch for few
// (3 us each).  Sequences are the grid's second dimension, so that a thread finds its place by
// 32-bit divisions (by 64-bit ones of its number in the whole: 55 us for the former
// two, 129 us).
#include "sv_kv.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;

// A thread's place in a launch over the tokens start .. start + N - 1.
struct Place {
  int b, n, h, d8;
  int64_t token;
};

// Groups of 4 slots that N tokens from anywhere in a group on can touch.
__host__ __device__ inline int64_t slot_groups(int N) { return ((int64_t)N + 6) / 4; }

template <int D>
__device__ __forceinline__ bool place_of(const KvMoveParams& p, Place* at, int64_t* len, int* count, bool* first) {
  const uint32_t in = blockIdx.x * kThreads + threadIdx.x;  // of the sequence
  const int b = blockIdx.y;
  at->b = b;
  at->d8 = (int)(in % (D / 8));
  const uint32_t row = in / (D / 8), gh = row / 4, g = gh / (uint32_t)p.c.H;
  at->h = (int)(gh - g * p.c.H);
  *len = p.lens ? p.lens[b] : 0;
  *count = p.news ? p.news[b] : p.N;
  *first = in == 0;
  if (*len < 0 || *count < 0 || *count > p.N || *len + *count > p.c.room) {
    if (*first) flag(p.err, SV_DERR_RANGE);
    return false;
  }
  at->token = (*len / 4 + g) * 4 + row % 4;
  at->n = (int)(at->token - *len);
  return at->n >= 0 && at->n < *count;
}

// The head's part of the token's page, null where the page is none of the pool.
__device__ __forceinline__ char* page_of(const Kv& c, int b, int64_t token, int h) {
  const int32_t id = c.pages[(int64_t)b * c.max_pages + (token >> c.pshift)];
  if ((uint32_t)id >= (uint32_t)c.num_pages) return nullptr;
  return c.pool + id * c.page_stride + h * c.head;
}

template <int D, int DT>
__global__ __launch_bounds__(kThreads) void write_kernel(const KvMoveParams p) {
  Place at;
  int64_t len;
  int count;
  bool first;
  const bool live = place_of<D>(p, &at, &len, &count, &first);
  if (!live) return;  // whole rows: the 4 threads of a block of 32 values stay together
  constexpr int es = DT == SV_F32 ? 4 : 2;
  Eight<DT> in[2];
  in[0].load(p.k + at.b * p.st[0][0] + at.n * p.st[0][1] + at.h * p.st[0][2] + at.d8 * 8 * es);
  in[1].load(p.v + at.b * p.st[1][0] + at.n * p.st[1][1] + at.h * p.st[1][2] + at.d8 * 8 * es);
  char* page = page_of(p.c, at.b, at.token, at.h);
  const int64_t slot = at.token & (((int64_t)1 << p.c.pshift) - 1);
  uint32_t code[2], byte[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[8];
    in[i].get(x);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    // the largest of 4 threads' magnitudes, as bits: NaN counts as the largest
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor1, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor2, 0xF, 0xF, false));
    byte[i] = scale_byte(m);
    code[i] = byte[i] == 255 ? 0 : encode8(x, scale_of(byte[i]));
  }
  if (!page) {
    if (at.d8 == 0) flag(p.err, SV_DERR_RANGE);
    return;
  }
  *reinterpret_cast<uint32_t*>(page + key_at<D>(slot, at.d8)) = code[0];
  if constexpr (D == 64) {
    char* v = page + p.c.vc + value_at<D>(slot, at.d8);
    *reinterpret_cast<uint16_t*>(v) = (uint16_t)code[1];
    *reinterpret_cast<uint16_t*>(v + 8) = (uint16_t)(code[1] >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(page + p.c.vc + value_at<D>(slot, at.d8)) = code[1];
  }
  if (at.d8 % 4 == 0) {
    page[p.c.ks + key_scale_at<D>(slot, at.d8 / 4)] = (char)byte[0];
    page[p.c.vs + value_scale_at<D>(slot, at.d8 / 4)] = (char)byte[1];
  }
}

template <int D, int DT>
__global__ __launch_bounds__(kThreads) void read_kernel(const KvMoveParams p) {
  Place at;
  int64_t len;
  int count;
  bool first;
  if (!place_of<D>(p, &at, &len, &count, &first)) return;
  const char* page = page_of(p.c, at.b, at.token, at.h);
  if (!page) {
    if (at.d8 == 0) flag(p.err, SV_DERR_RANGE);
    return;
  }
  const int64_t slot = at.token & (((int64_t)1 << p.c.pshift) - 1);
  uint32_t code[2];
  code[0] = *reinterpret_cast<const uint32_t*>(page + key_at<D>(slot, at.d8));
  const char* v = page + p.c.vc + value_at<D>(slot, at.d8);
  if constexpr (D == 64)
    code[1] = *reinterpret_cast<const uint16_t*>(v) | (uint32_t)*reinterpret_cast<const uint16_t*>(v + 8) << 16;
  else
    code[1] = *reinterpret_cast<const uint32_t*>(v);
  const uint8_t sk = (uint8_t)page[p.c.ks + key_scale_at<D>(slot, at.d8 / 4)];
  const uint8_t sv = (uint8_t)page[p.c.vs + value_scale_at<D>(slot, at.d8 / 4)];
  constexpr int es = DT == SV_F32 ? 4 : 2;
  float x[8];
  Eight<DT> out;
  decode8(code[0], scale_of(sk), x);
  out.set(x);
  out.store(p.k + at.b * p.st[0][0] + at.n * p.st[0][1] + at.h * p.st[0][2] + at.d8 * 8 * es);
  decode8(code[1], scale_of(sv), x);
  out.set(x);
  out.store(p.v + at.b * p.st[1][0] + at.n * p.st[1][1] + at.h * p.st[1][2] + at.d8 * 8 * es);
}

// A block moves one sequence's path in one head of several layers, tokens in
// the path's order: a place is written after everything that stood in it and
// moves has been read, because a token moves to a lower place, past none of
// those behind it.  A thread takes one piece of a token -- 16 bytes of the keys'
// codes, a sixteenth of the values', the keys' scales, one of the values' -- and
// reads it from all of the block's layers before it writes: what a layer moves
// is little (8 tokens of 136 bytes), so the time is that of the loads one after
// another (lengths, path, pages, pieces), and layers share it: 32 paths of up to 8
// tokens in 64 layers of 8 heads take 13 us, 55 with a layer a block.
constexpr int kLayers = 8;

template <int BYTES>
struct Bits;
template <>
struct Bits<1> { using T = uint8_t; };
template <>
struct Bits<2> { using T = uint16_t; };
template <>
struct Bits<4> { using T = uint32_t; };
template <>
struct Bits<8> { using T = uint64_t; };

template <int D>
__global__ __launch_bounds__(kThreads) void commit_kernel(const KvCommitParams p) {
  const int h = blockIdx.x, b = blockIdx.z;
  const int layer0 = blockIdx.y * kLayers, layers = min(kLayers, p.c.layers - layer0);
  const int64_t len = p.lens[b];
  const int n = p.n[b];
  const int32_t* path = p.path ? p.path + (int64_t)b * p.M : nullptr;
  const int32_t* pages = p.c.pages + (int64_t)b * p.c.max_pages;
  // n is not bounded by M where there is no path
  bool range = n < -1 || (path && n > p.M) || len < 0 || (n >= 0 && len + 1 + (int64_t)n > p.c.room);
  bool tree = false;
  if (!range && path) {
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const int at = path[j], before = j ? path[j - 1] : 0;
      if (at <= before || at >= SV_MAX_N) {
        tree = true;
      } else if (len + at >= p.c.room) {
        range = true;
      } else {
        const uint32_t from = (uint32_t)pages[(len + at) >> p.c.pshift], to = (uint32_t)pages[(len + 1 + j) >> p.c.pshift];
        if (at != 1 + j && (from >= (uint32_t)p.c.num_pages || to >= (uint32_t)p.c.num_pages)) range = true;
      }
    }
  }
  range = __syncthreads_or(range);
  tree = path && __syncthreads_or(tree);
  const bool bad = range || tree;
  if (h == 0 && layer0 == 0 && threadIdx.x == 0) {  // the sequence's first block writes its length and flags
    p.out_lens[b] = bad || n < 0 ? (int32_t)len : (int32_t)(len + 1 + n);
    if (bad) flag(p.err, (range ? SV_DERR_RANGE : 0) | (tree ? SV_DERR_TREE : 0));
  }
  if (bad || !path || n <= 0) return;
  constexpr int w = D / 32;
  constexpr int kPieces = w + 16 + 1 + w;
  constexpr int kTokens = kThreads / kPieces;
  char* const base = p.c.pool + layer0 * p.c.layer_stride + h * p.c.head;
  const int64_t in_page = ((int64_t)1 << p.c.pshift) - 1;
  const int piece = threadIdx.x % kPieces;
  for (int j0 = 0; j0 < n; j0 += kTokens) {
    const int j = j0 + threadIdx.x / kPieces;
    const bool live = (int)threadIdx.x < kTokens * kPieces && j < n && path[min(j, n - 1)] != 1 + j;
    u32x4 held[kLayers];
    int64_t to = 0, from = 0;
    if (live) {
      const int64_t s = len + path[j], d = len + 1 + j;
      const int64_t ss = s & in_page, ds = d & in_page;
      if (piece < w) {
        from = ss * (D / 2) + piece * 16;
        to = ds * (D / 2) + piece * 16;
      } else if (piece < w + 16) {
        from = p.c.vc + ((ss / 4 * 16 + piece - w) * 4 + ss % 4) * w;
        to = p.c.vc + ((ds / 4 * 16 + piece - w) * 4 + ds % 4) * w;
      } else if (piece == w + 16) {
        from = p.c.ks + ss * w;
        to = p.c.ks + ds * w;
      } else {
        from = p.c.vs + value_scale_at<D>(ss, piece - w - 17);
        to = p.c.vs + value_scale_at<D>(ds, piece - w - 17);
      }
      from += pages[s >> p.c.pshift] * p.c.page_stride;
      to += pages[d >> p.c.pshift] * p.c.page_stride;
#pragma unroll
      for (int i = 0; i < kLayers; ++i) {
        const char* at = base + min(i, layers - 1) * p.c.layer_stride + from;
        if (piece < w)
          held[i] = *reinterpret_cast<const u32x4*>(at);
        else if (piece > w + 16)
          held[i][0] = (uint8_t)*at;
        else if constexpr (w == 8) {
          const uint64_t x = *reinterpret_cast<const uint64_t*>(at);
          held[i][0] = (uint32_t)x;
          held[i][1] = (uint32_t)(x >> 32);
        } else {
          held[i][0] = *reinterpret_cast<const typename Bits<w>::T*>(at);
        }
      }
    }
    __syncthreads();
    if (live) {
#pragma unroll
      for (int i = 0; i < kLayers; ++i) {
        if (i >= layers) break;
        char* at = base + i * p.c.layer_stride + to;
        if (piece < w)
          *reinterpret_cast<u32x4*>(at) = held[i];
        else if (piece > w + 16)
          *at = (char)held[i][0];
        else if constexpr (w == 8)
          *reinterpret_cast<uint64_t*>(at) = held[i][0] | (uint64_t)held[i][1] << 32;
        else
          *reinterpret_cast<typename Bits<w>::T*>(at) = (typename Bits<w>::T)held[i][0];
      }
    }
  }
}

template <int D>
hipError_t move(const KvMoveParams& p, sv_dtype dt, bool write, hipStream_t s) {
  const int64_t threads = slot_groups(p.N) * p.c.H * 4 * (D / 8);  // of a sequence
  const dim3 grid((uint32_t)((threads + kThreads - 1) / kThreads), (uint32_t)p.B);
  switch (dt) {
    case SV_BF16:
      write ? write_kernel<D, SV_BF16><<<grid, kThreads, 0, s>>>(p) : read_kernel<D, SV_BF16><<<grid, kThreads, 0, s>>>(p);
      break;
    case SV_F16:
      write ? write_kernel<D, SV_F16><<<grid, kThreads, 0, s>>>(p) : read_kernel<D, SV_F16><<<grid, kThreads, 0, s>>>(p);
      break;
    default:
      write ? write_kernel<D, SV_F32><<<grid, kThreads, 0, s>>>(p) : read_kernel<D, SV_F32><<<grid, kThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

hipError_t move(const KvMoveParams& p, sv_dtype dt, int D, bool write, hipStream_t s) {
  return D == 64 ? move<64>(p, dt, write, s) : D == 128 ? move<128>(p, dt, write, s) : move<256>(p, dt, write, s);
}

}  // namespace

hipError_t launch_kv_write(const KvMoveParams& p, sv_dtype dt, int D, hipStream_t s) { return move(p, dt, D, true, s); }
hipError_t launch_kv_read(const KvMoveParams& p, sv_dtype dt, int D, hipStream_t s) { return move(p, dt, D, false, s); }

hipError_t launch_kv_commit(const KvCommitParams& p, int D, hipStream_t s) {
  dim3 grid((uint32_t)p.c.H, (uint32_t)(p.c.layers + kLayers - 1) / kLayers, (uint32_t)p.B);
  if (!p.path) grid.x = grid.y = 1;  // nothing moves
  if (D == 64) commit_kernel<64><<<grid, kThreads, 0, s>>>(p);
  if (D == 128) commit_kernel<128><<<grid, kThreads, 0, s>>>(p);
  if (D == 256) commit_kernel<256><<<grid, kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace sv
