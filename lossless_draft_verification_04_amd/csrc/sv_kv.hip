// sv_kv.hip -- the 4-bit cache: writing, reading back, committing a path.
//
// All three move bytes.  A thread takes 8 neighbouring values of a key and of
// a value row: 16 bytes (32 in fp32) on one side, 4 on the other.  Threads are
// ordered (sequence, group of 4 slots, head, slot, 8 values), because the
// cache holds sixteenths of value rows for 4 tokens side by side: a wave then
// writes and reads whole lines of the cache.
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
  const int64_t per = slot_groups(p.N) * p.c.H * 4 * (D / 8);  // of a sequence
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t b = i / per;
  if (b >= p.B) return false;
  const int64_t in = i - b * per;
  at->b = (int)b;
  at->d8 = (int)(in % (D / 8));
  const int64_t row = in / (D / 8);
  const int64_t gh = row / 4;
  at->h = (int)(gh % p.c.H);
  const int64_t g = gh / p.c.H;
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

// A block moves one sequence's path in one layer's head, tokens in the path's
// order: a place is written after everything that stood in it and moves has
// been read, because a token moves to a lower place, past none of those behind
// it.  Threads of a pass take (token, piece): pieces of 4 bytes of the
// keys' codes, a sixteenth of the values', one byte of the scales.
template <int D>
__global__ __launch_bounds__(kThreads) void commit_kernel(const KvCommitParams p) {
  const int h = blockIdx.x % p.c.H;
  const int64_t lb = blockIdx.x / p.c.H;
  const int b = (int)(lb % p.B);
  const int64_t layer = lb / p.B;
  const int64_t len = p.lens[b];
  const int n = p.n[b];
  const bool speaks = h == 0 && layer == 0;  // the sequence's first block writes its length and flags
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
  tree = __syncthreads_or(tree);
  if (speaks && threadIdx.x == 0) {
    p.out_lens[b] = range || tree || n < 0 ? (int32_t)len : (int32_t)(len + 1 + n);
    if (range) flag(p.err, SV_DERR_RANGE);
    if (tree) flag(p.err, SV_DERR_TREE);
  }
  if (range || tree || !path || n <= 0) return;
  constexpr int kKeys = D / 8, kPieces = kKeys + 16 + 2 * (D / 32);
  constexpr int kPass = 4;  // pieces of a thread at a time
  constexpr int kTokens = kThreads * kPass / kPieces;
  char* base = p.c.pool + layer * p.c.layer_stride + h * p.c.head;
  const int64_t in_page = ((int64_t)1 << p.c.pshift) - 1;
  for (int j0 = 0; j0 < n; j0 += kTokens) {
    const int some = min(kTokens, n - j0) * kPieces;
    uint64_t held[kPass];
    char* to[kPass];
    int size[kPass];
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const int x = i * kThreads + threadIdx.x;
      size[i] = 0;
      if (x >= some) continue;
      const int j = j0 + x / kPieces, piece = x % kPieces;
      const int64_t s = len + path[j], d = len + 1 + j;
      if (s == d) continue;
      const char* sp = base + pages[s >> p.c.pshift] * p.c.page_stride;
      char* dp = base + pages[d >> p.c.pshift] * p.c.page_stride;
      const int64_t ss = s & in_page, ds = d & in_page;
      if (piece < kKeys) {
        size[i] = 4;
        held[i] = *reinterpret_cast<const uint32_t*>(sp + key_at<D>(ss, piece));
        to[i] = dp + key_at<D>(ds, piece);
      } else if (piece < kKeys + 16) {
        constexpr int w = D / 32;
        const int c = piece - kKeys;
        const char* f = sp + p.c.vc + ((ss / 4 * 16 + c) * 4 + ss % 4) * w;
        to[i] = dp + p.c.vc + ((ds / 4 * 16 + c) * 4 + ds % 4) * w;
        size[i] = w;
        if constexpr (w == 2) held[i] = *reinterpret_cast<const uint16_t*>(f);
        if constexpr (w == 4) held[i] = *reinterpret_cast<const uint32_t*>(f);
        if constexpr (w == 8) held[i] = *reinterpret_cast<const uint64_t*>(f);
      } else {
        const int c = (piece - kKeys - 16) / 2;
        const bool key = (piece - kKeys - 16) % 2 == 0;
        size[i] = 1;
        held[i] = (uint8_t)(key ? sp[p.c.ks + key_scale_at<D>(ss, c)] : sp[p.c.vs + value_scale_at<D>(ss, c)]);
        to[i] = key ? dp + p.c.ks + key_scale_at<D>(ds, c) : dp + p.c.vs + value_scale_at<D>(ds, c);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      if (size[i] == 1) *to[i] = (char)held[i];
      if (size[i] == 2) *reinterpret_cast<uint16_t*>(to[i]) = (uint16_t)held[i];
      if (size[i] == 4) *reinterpret_cast<uint32_t*>(to[i]) = (uint32_t)held[i];
      if (size[i] == 8) *reinterpret_cast<uint64_t*>(to[i]) = held[i];
    }
  }
}

template <int D>
hipError_t move(const KvMoveParams& p, sv_dtype dt, bool write, hipStream_t s) {
  const int64_t threads = (int64_t)p.B * slot_groups(p.N) * p.c.H * 4 * (D / 8);
  const dim3 grid((uint32_t)((threads + kThreads - 1) / kThreads));
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
  // without a path nothing moves: one block a sequence
  const int64_t blocks = p.path ? (int64_t)p.c.layers * p.B * p.c.H : (int64_t)p.B * p.c.H;
  const dim3 grid((uint32_t)blocks);
  if (D == 64) commit_kernel<64><<<grid, kThreads, 0, s>>>(p);
  if (D == 128) commit_kernel<128><<<grid, kThreads, 0, s>>>(p);
  if (D == 256) commit_kernel<256><<<grid, kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace sv
