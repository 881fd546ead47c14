// sv_pass_api.hip -- the C ABI of the verifier's pass (specverify_pass.h):
// host-side argument checks, workspace planning and kernel launches on the
// caller's stream.
//
// Every check below runs before any HIP call, so invalid arguments are
// rejected synchronously and nothing is enqueued.
#include <algorithm>
#include <cmath>

#include "sv_host.hpp"
#include "sv_pass.h"

namespace sv {

namespace {

bool bad_type(sv_dtype dt) { return dt != SV_F32 && dt != SV_BF16 && dt != SV_F16; }
int type_bytes(sv_dtype dt) { return dt == SV_F32 ? 4 : 2; }
bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

sv_status check_cache(const sv_kv_cache* c, bool layers, Kv* kv) {
  if (!c) return SV_EINVAL;
  if (c->H < 1 || c->page_tokens < 1 || c->max_pages < 1 || c->num_pages < 1) return SV_EINVAL;
  if ((c->page_tokens & (c->page_tokens - 1)) || c->page_tokens < 16) return SV_EINVAL;
  if (c->D != 64 && c->D != 128 && c->D != 256) return SV_EUNSUPPORTED;
  if (c->H > SV_MAX_HEADS || c->page_tokens > SV_MAX_PAGE_TOKENS) return SV_EUNSUPPORTED;
  int64_t page;
  const sv_status st = sv_kv_page_bytes(c->H, c->D, c->page_tokens, &page);
  if (st != SV_OK) return st;
  if (!c->pool || !c->pages || c->page_stride < page) return SV_EINVAL;
  if (misaligned(c->pool, 16) || c->page_stride % 16) return SV_EALIGN;
  int64_t span;  // of a layer's pages
  if (__builtin_mul_overflow((int64_t)c->num_pages - 1, c->page_stride, &span) ||
      __builtin_add_overflow(span, page, &span))
    return SV_EINVAL;
  kv->layers = 1;
  kv->layer_stride = 0;
  if (layers) {
    if (c->layers < 1) return SV_EINVAL;
    kv->layers = c->layers;
    if (c->layers > 1) {
      // layers one behind another, or within the pages' stride
      if (c->layer_stride < page || (c->layer_stride < span && c->num_pages > 1 &&
                                     ((c->layers - 1) > (c->page_stride - page) / c->layer_stride)))
        return SV_EINVAL;
      int64_t end;
      if (__builtin_mul_overflow((int64_t)c->layers - 1, c->layer_stride, &end) ||
          __builtin_add_overflow(end, span, &end))
        return SV_EINVAL;
      if (c->layer_stride % 16) return SV_EALIGN;
      kv->layer_stride = c->layer_stride;
    }
  }
  kv->pool = static_cast<char*>(c->pool);
  kv->pages = c->pages;
  kv->page_stride = c->page_stride;
  kv->head = page / c->H;
  const int64_t codes = (int64_t)c->page_tokens * c->D / 2, scales = (int64_t)c->page_tokens * c->D / 32;
  kv->ks = codes;
  kv->vc = codes + scales;
  kv->vs = 2 * codes + scales;
  kv->num_pages = c->num_pages;
  kv->max_pages = c->max_pages;
  kv->pshift = __builtin_ctz((unsigned)c->page_tokens);
  kv->H = c->H;
  // places are 32-bit numbers
  kv->room = std::min((int64_t)c->max_pages << kv->pshift, (int64_t)INT32_MAX - 1024);
  return SV_OK;
}

// Byte strides of a [B, N, heads, D] tensor and the bytes that it spans; a
// stride of a dimension of one is not read.  `apart`: whether rows cannot
// overlap.
sv_status check_tensor(const void* base, const int64_t* stride, int64_t B, int64_t N, int64_t heads, int64_t D, int es,
                       bool aligned, int64_t* bytes, int64_t* span, bool* apart) {
  if (!base || !stride) return SV_EINVAL;
  const int64_t n[3] = {B, N, heads};
  int o[3] = {0, 1, 2};
  int64_t end = D * es;
  for (int i = 0; i < 3; ++i) {
    bytes[i] = 0;
    if (n[i] <= 1) continue;
    if (stride[i] < 0 || __builtin_mul_overflow(stride[i], (int64_t)es, &bytes[i])) return SV_EINVAL;
  }
  std::sort(o, o + 3, [&](int x, int y) { return bytes[x] < bytes[y]; });
  *apart = true;
  for (int j = 0; j < 3; ++j) {
    const int i = o[j];
    if (n[i] <= 1) continue;
    if (bytes[i] < end) *apart = false;
    int64_t add;
    if (__builtin_mul_overflow(n[i] - 1, bytes[i], &add) || __builtin_add_overflow(end, add, &end)) return SV_EINVAL;
  }
  *span = end;
  if (misaligned(base, aligned ? 16 : es)) return SV_EALIGN;
  if (aligned)
    for (int i = 0; i < 3; ++i)
      if (bytes[i] % 16) return SV_EALIGN;
  return SV_OK;
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Whether two [B, N, heads, D] tensors that lie within one another share no
// value: views of one tensor, the heads of one behind those of the other.
// Strides and rows in bytes.
bool views_apart(const void* a, const int64_t* as, int64_t ha, const void* b, const int64_t* bs, int64_t hb, int64_t B,
                 int64_t N, int64_t row) {
  if (as[0] != bs[0] || as[1] != bs[1]) return false;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t ea = (ha - 1) * as[2] + row, eb = (hb - 1) * bs[2] + row;
  if (d >= 0 ? d < ea : -d < eb) return false;
  const int64_t both = d >= 0 ? d + eb : -d + ea;  // what a node's heads of both span
  const int64_t inner = N > 1 && B > 1 ? std::min(as[0], as[1]) : N > 1 ? as[1] : as[0];
  const int64_t outer = std::max(as[0], as[1]), count = as[0] < as[1] ? B : N;
  if (N == 1 && B == 1) return true;
  return both <= inner && (N == 1 || B == 1 || outer >= (count - 1) * inner + both);
}

struct PassPlan {
  size_t bytes;
  AttentionForm form;
  int32_t tiles;
  size_t off_desc, off_ml, off_o;
};

sv_status plan_attention(int32_t B, int32_t N, int32_t Hq, int32_t H, int32_t D, PassPlan* pl) {
  if (B < 0 || N < 1 || Hq < 1 || H < 1 || Hq % H) return SV_EINVAL;
  if (D != 64 && D != 128 && D != 256) return SV_EUNSUPPORTED;
  if (B > SV_MAX_SEQ || N > SV_MAX_N || Hq > SV_MAX_HEADS) return SV_EUNSUPPORTED;
  const int tiles = (N * (Hq / H) + 15) / 16;
  pl->form = attention_form(D, tiles);
  pl->tiles = tiles;
  const size_t rows = (size_t)2 * pl->form.blocks * pl->form.split * pl->form.tiles * 16;
  size_t off = kWsFixed;
  pl->off_desc = off;
  off = align_up(off + (size_t)pl->form.blocks * sizeof(AttentionItem), 256);
  pl->off_ml = off;
  off = align_up(off + rows * 2 * sizeof(float), 256);
  pl->off_o = off;
  off = align_up(off + rows * D * sizeof(float), 256);
  pl->bytes = off;
  return SV_OK;
}

sv_status check_space(const void* ws, size_t have, size_t want) {
  if (!ws || have < want) return SV_EWORKSPACE;
  return misaligned(ws, 256) ? SV_EALIGN : SV_OK;
}

sv_status kv_move(const void* k, const int64_t* ks, const void* v, const int64_t* vs, sv_dtype dt,
                  const sv_kv_cache* cache, const int32_t* lens, const int32_t* news, int32_t B, int32_t N, bool write,
                  void* ws, size_t ws_bytes, void* stream) {
  if (bad_type(dt)) return SV_EDTYPE;
  if (B < 0 || N < 0) return SV_EINVAL;
  if (B > SV_MAX_SEQ) return SV_EUNSUPPORTED;
  if (B == 0 || N == 0) return SV_OK;
  KvMoveParams p;
  sv_status st = check_cache(cache, false, &p.c);
  if (st != SV_OK) return st;
  if (write && !lens) return SV_EINVAL;
  int64_t nk, nv;
  bool ak, av;
  if ((st = check_tensor(k, ks, B, N, cache->H, cache->D, type_bytes(dt), true, p.st[0], &nk, &ak)) != SV_OK) return st;
  if ((st = check_tensor(v, vs, B, N, cache->H, cache->D, type_bytes(dt), true, p.st[1], &nv, &av)) != SV_OK) return st;
  if (!write && (!ak || !av)) return SV_EINVAL;
  if (!write && overlap(k, nk, v, nv) &&
      !views_apart(k, p.st[0], cache->H, v, p.st[1], cache->H, B, N, (int64_t)cache->D * type_bytes(dt)))
    return SV_EINVAL;
  if ((st = check_space(ws, ws_bytes, kWsFixed)) != SV_OK) return st;
  // threads of a sequence, 8 values of keys each, are counted in 32 bits
  if (((int64_t)N + 6) * cache->H * cache->D / 8 > INT32_MAX - 1024) return SV_EUNSUPPORTED;
  p.k = static_cast<char*>(const_cast<void*>(k));
  p.v = static_cast<char*>(const_cast<void*>(v));
  p.lens = lens;
  p.news = news;
  p.B = B;
  p.N = N;
  p.err = static_cast<int32_t*>(ws);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return (write ? launch_kv_write(p, dt, cache->D, s) : launch_kv_read(p, dt, cache->D, s)) == hipSuccess ? SV_OK
                                                                                                         : SV_EHIP;
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

sv_status sv_kv_page_bytes(int32_t H, int32_t D, int32_t page_tokens, int64_t* bytes) {
  if (!bytes || H < 1 || page_tokens < 16 || (page_tokens & (page_tokens - 1))) return SV_EINVAL;
  if (D != 64 && D != 128 && D != 256) return SV_EUNSUPPORTED;
  if (H > SV_MAX_HEADS || page_tokens > SV_MAX_PAGE_TOKENS) return SV_EUNSUPPORTED;
  *bytes = (int64_t)H * page_tokens * (D + D / 16);
  return SV_OK;
}

sv_status sv_pass_workspace_size(sv_pass_op op, int32_t B, int32_t N, int32_t Hq, int32_t H, int32_t D,
                                 size_t* bytes) {
  if (!bytes) return SV_EINVAL;
  if (op == SV_PASS_ATTENTION) {
    PassPlan pl;
    const sv_status st = plan_attention(B, N, Hq, H, D, &pl);
    if (st != SV_OK) return st;
    *bytes = pl.bytes;
    return SV_OK;
  }
  if (op != SV_PASS_ROPE && op != SV_PASS_WRITE && op != SV_PASS_READ && op != SV_PASS_COMMIT) return SV_EINVAL;
  *bytes = kWsFixed;
  return SV_OK;
}

sv_status sv_rope(const void* q, const int64_t* q_stride, const void* k, const int64_t* k_stride, sv_dtype dt,
                  int32_t B, int32_t N, int32_t Hq, int32_t Hk, int32_t D, int32_t R, const double* freq, float factor,
                  int32_t interleaved, int32_t inverse, const int32_t* positions, const int32_t* lens,
                  const int32_t* parent, void* out_q, const int64_t* out_q_stride, void* out_k,
                  const int64_t* out_k_stride, void* ws, size_t ws_bytes, void* stream) {
  if (bad_type(dt)) return SV_EDTYPE;
  if (B < 0 || N < 0 || Hq < 0 || Hk < 0 || D < 2 || R < 2 || R > D || R % 2) return SV_EINVAL;
  if (D > 8192 || Hq > SV_MAX_HEADS || Hk > SV_MAX_HEADS || (int64_t)B * N > INT32_MAX) return SV_EUNSUPPORTED;
  if (!std::isfinite(factor)) return SV_EINVAL;
  if (parent && !positions && N > SV_MAX_N) return SV_EUNSUPPORTED;
  if (B == 0 || N == 0 || Hq + Hk == 0) return SV_OK;
  if (!freq) return SV_EINVAL;
  if (misaligned(freq, 8)) return SV_EALIGN;
  RopeParams p;
  const void* in[2] = {q, k};
  void* out[2] = {out_q, out_k};
  const int64_t* is[2] = {q_stride, k_stride};
  const int64_t* os[2] = {out_q_stride, out_k_stride};
  const int32_t heads[2] = {Hq, Hk};
  int64_t ni[2] = {0, 0}, no[2] = {0, 0};
  sv_status st;
  for (int w = 0; w < 2; ++w) {
    p.heads[w] = heads[w];
    p.in[w] = static_cast<const char*>(in[w]);
    p.out[w] = static_cast<char*>(out[w]);
    if (!heads[w]) continue;
    bool ai, ao;
    if ((st = check_tensor(in[w], is[w], B, N, heads[w], D, type_bytes(dt), false, p.is[w], &ni[w], &ai)) != SV_OK) return st;
    if ((st = check_tensor(out[w], os[w], B, N, heads[w], D, type_bytes(dt), false, p.os[w], &no[w], &ao)) != SV_OK) return st;
    if (!ao) return SV_EINVAL;
  }
  // nothing that is written is read or written elsewhere; tensors may be views
  // of the heads of one, as a fused projection's are
  const int64_t row = (int64_t)D * type_bytes(dt);
  for (int w = 0; w < 2; ++w) {
    if (!heads[w]) continue;
    for (int x = 0; x < 2; ++x) {
      if (!heads[x]) continue;
      const bool in_place = x == w && in[w] == out[w] && std::equal(p.is[w], p.is[w] + 3, p.os[w]);
      if (!in_place && overlap(in[x], ni[x], out[w], no[w]) &&
          !views_apart(in[x], p.is[x], heads[x], out[w], p.os[w], heads[w], B, N, row))
        return SV_EINVAL;
    }
  }
  if (Hq && Hk && overlap(out_q, no[0], out_k, no[1]) &&
      !views_apart(out_q, p.os[0], Hq, out_k, p.os[1], Hk, B, N, row))
    return SV_EINVAL;
  if ((st = check_space(ws, ws_bytes, kWsFixed)) != SV_OK) return st;
  p.B = B;
  p.N = N;
  p.D = D;
  p.R = R;
  p.freq = freq;
  p.factor = factor;
  p.interleaved = interleaved != 0;
  p.inverse = inverse != 0;
  p.positions = positions;
  p.lens = lens;
  p.parent = parent;
  p.err = static_cast<int32_t*>(ws);
  return launch_rope(p, dt, static_cast<hipStream_t>(stream)) == hipSuccess ? SV_OK : SV_EHIP;
}

sv_status sv_rope_frequencies(sv_rope_kind kind, int32_t R, double theta, double scale, int32_t original, double fast,
                              double slow, double* out_freq, float* out_factor) {
  if (!out_freq || !out_factor || R < 2 || R % 2 || R > 8192) return SV_EINVAL;
  if (!(theta > 0) || !std::isfinite(theta) || !(scale >= 1) || !std::isfinite(scale)) return SV_EINVAL;
  if (kind < SV_ROPE_PLAIN || kind > SV_ROPE_PARTS) return SV_EINVAL;
  double low = 0, high = 0;
  if (kind == SV_ROPE_PARTS) {
    if (original < 1 || !(slow > 0) || !(fast > slow) || !std::isfinite(fast) || !(theta > 1)) return SV_EINVAL;
    // the pair that makes n turns over `original` positions: theta^(-2i/R) original = 2 pi n
    const auto pair = [&](double n) { return R * std::log(original / (n * 2 * M_PI)) / (2 * std::log(theta)); };
    low = std::max(std::floor(pair(fast)), 0.0);
    high = std::min(std::ceil(pair(slow)), (double)(R - 1));
    if (pair(slow) < 0) low = high = -1;  // the first pair is slow: all are
  }
  if (kind == SV_ROPE_BASE && R > 2) theta *= std::pow(scale, (double)R / (R - 2));
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / R);
    if (kind == SV_ROPE_LINEAR) f /= scale;
    if (kind == SV_ROPE_PARTS) {
      const double ramp = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
      f = f * (1 - ramp) + f / scale * ramp;
    }
    out_freq[i] = f;
  }
  *out_factor = kind == SV_ROPE_PARTS ? (float)(0.1 * std::log(scale) + 1) : 1.0f;
  return SV_OK;
}

sv_status sv_kv_write(const void* k, const int64_t* k_stride, const void* v, const int64_t* v_stride, sv_dtype dt,
                      const sv_kv_cache* cache, const int32_t* lens, const int32_t* news, int32_t B, int32_t N,
                      void* ws, size_t ws_bytes, void* stream) {
  return kv_move(k, k_stride, v, v_stride, dt, cache, lens, news, B, N, true, ws, ws_bytes, stream);
}

sv_status sv_kv_read(const sv_kv_cache* cache, const int32_t* start, const int32_t* count, int32_t B, int32_t N,
                     sv_dtype dt, void* out_k, const int64_t* k_stride, void* out_v, const int64_t* v_stride,
                     void* ws, size_t ws_bytes, void* stream) {
  return kv_move(out_k, k_stride, out_v, v_stride, dt, cache, start, count, B, N, false, ws, ws_bytes, stream);
}

sv_status sv_kv_attention(const void* q, const int64_t* q_stride, sv_dtype dt, const sv_kv_cache* cache,
                          const int32_t* lens, const int32_t* news, const int32_t* parent, int32_t B, int32_t N,
                          int32_t Hq, float scale, float cap, const float* slopes, int32_t reach, void* out,
                          const int64_t* out_stride, float* out_lse, void* ws, size_t ws_bytes, void* stream) {
  if (dt != SV_BF16 && dt != SV_F16) return SV_EDTYPE;
  if (B < 0 || N < 1 || Hq < 1) return SV_EINVAL;
  if (B > SV_MAX_SEQ || N > SV_MAX_N || Hq > SV_MAX_HEADS) return SV_EUNSUPPORTED;
  if (B == 0) return SV_OK;
  AttentionParams p;
  sv_status st = check_cache(cache, false, &p.c);
  if (st != SV_OK) return st;
  PassPlan pl;
  if ((st = plan_attention(B, N, Hq, cache->H, cache->D, &pl)) != SV_OK) return st;
  // (they are held as exponents of 2)
  if (!std::isfinite(scale * 1.5f) || !std::isfinite(cap * 1.5f) || cap < 0 || reach < 0) return SV_EINVAL;
  if (cap > 0 && !std::isfinite(2.9f / cap)) return SV_EINVAL;
  if (!lens) return SV_EINVAL;
  int64_t nq, no;
  bool aq, ao;
  if ((st = check_tensor(q, q_stride, B, N, Hq, cache->D, 2, true, p.qs, &nq, &aq)) != SV_OK) return st;
  if ((st = check_tensor(out, out_stride, B, N, Hq, cache->D, 2, true, p.os, &no, &ao)) != SV_OK) return st;
  if (!ao) return SV_EINVAL;
  if (overlap(q, nq, out, no) && !views_apart(q, p.qs, Hq, out, p.os, Hq, B, N, (int64_t)cache->D * 2)) return SV_EINVAL;
  if (out_lse) {
    const int64_t nl = (int64_t)B * N * Hq * (int64_t)sizeof(float);
    if (overlap(out_lse, nl, out, no) || overlap(out_lse, nl, q, nq)) return SV_EINVAL;
    if (misaligned(out_lse, 4)) return SV_EALIGN;
  }
  if ((st = check_space(ws, ws_bytes, pl.bytes)) != SV_OK) return st;
  char* w = static_cast<char*>(ws);
  p.q = static_cast<const char*>(q);
  p.out = static_cast<char*>(out);
  p.lse = out_lse;
  p.lens = lens;
  p.news = news;
  p.parent = parent;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.G = Hq / cache->H;
  p.scale = scale;
  p.cap = cap;
  p.slopes = slopes;
  p.reach = reach < p.c.room ? reach : 0;  // no two tokens are further apart
  p.err = reinterpret_cast<int32_t*>(w);
  p.tiles = pl.form.tiles;
  p.split = pl.form.split;
  p.groups = pl.form.groups;
  p.all_tiles = pl.tiles;
  p.blocks = pl.form.blocks;
  p.log_blocks = __builtin_ctz((unsigned)pl.form.blocks);
  p.desc = w + pl.off_desc;
  p.part_ml = reinterpret_cast<float*>(w + pl.off_ml);
  p.part_o = reinterpret_cast<float*>(w + pl.off_o);
  return launch_kv_attention(p, dt, cache->D, static_cast<hipStream_t>(stream)) == hipSuccess ? SV_OK : SV_EHIP;
}

sv_status sv_kv_commit(const sv_kv_cache* cache, const int32_t* lens, const int32_t* n, const int32_t* path, int32_t B,
                       int32_t M, int32_t* out_lens, void* ws, size_t ws_bytes, void* stream) {
  if (B < 0 || M < 0) return SV_EINVAL;
  if (B > SV_MAX_SEQ || M > SV_MAX_N) return SV_EUNSUPPORTED;
  if (B == 0) return SV_OK;
  KvCommitParams p;
  sv_status st = check_cache(cache, true, &p.c);
  if (st != SV_OK) return st;
  if (p.c.layers > SV_MAX_LAYERS) return SV_EUNSUPPORTED;
  if (!lens || !n || !out_lens) return SV_EINVAL;
  const int64_t row = (int64_t)B * (int64_t)sizeof(int32_t);
  if (overlap(lens, row, out_lens, row) || overlap(n, row, out_lens, row)) return SV_EINVAL;
  if (path && M && overlap(path, row * M, out_lens, row)) return SV_EINVAL;
  if ((st = check_space(ws, ws_bytes, kWsFixed)) != SV_OK) return st;
  p.lens = lens;
  p.n = n;
  p.path = path;
  p.B = B;
  p.M = M;
  p.out_lens = out_lens;
  p.err = static_cast<int32_t*>(ws);
  return launch_kv_commit(p, cache->D, static_cast<hipStream_t>(stream)) == hipSuccess ? SV_OK : SV_EHIP;
}

}  // extern "C"
