// sv_draft_api.hip -- the C ABI of the drafter-side entry points
// (specverify_draft.h): host-side argument checks, workspace planning and
// kernel launches on the caller's stream.
//
// Every check below runs before any HIP call, so invalid arguments are
// rejected synchronously and nothing is enqueued.
#include <algorithm>
#include <cmath>

#include "sv_device.hpp"
#include "sv_draft.h"
#include "sv_host.hpp"
#include "sv_topmass.hpp"

namespace sv {

namespace {

// Blocks of the top-value passes, and the smallest part of a row split for
// them: joining parts costs about as much as a block takes for 8192 vectors
// (17 x 32000 fp32 rows, 64 values: 12.4 us whole, 16.5 in parts of 2667;
// 17 x 152064 bf16 rows: 20.7 us in 2 parts, 21.4 in 4).  Beams are joined
// anyway (8 beams of 152064, 16 kept: 15.9 us in 4 parts each, 18.7 in 2).
constexpr int kTopBlocks = 256;
constexpr int kTopPartVecs = 8192, kBeamPartVecs = 4096;

// Blocks of the distillation passes.  A part of a loss costs a hand-off, so
// rows are split only until every compute unit has a block: 64 x 152064 bf16
// rows take 11.3 us in 256 blocks, 15.4 in 1024; 600 rows 37 us whole, 43 in
// 1200 parts; past 1000 rows the number does not matter.  Gradients need no
// joining and gain from many blocks in flight: 1100 rows take 140 us in 1100
// blocks, 133 in 2200, 129 in 4400; few rows, from parts of half the size
// (64 x 32000 fp32: 8.2 us in 448 parts, 7.3 in 960).
constexpr int kLossBlocks = 256;
constexpr int kGradBlocks = 4096;
constexpr int kGradFew = 1024;

// T and its log2(e) / T usable in 32 bits.
bool bad_scale(float T) { return bad_temperature(T) || !std::isfinite(log2e_over(T)) || !(log2e_over(T) > 0.f); }

sv_status plan_topmass(sv_dtype dt, int64_t rows, int32_t V, int32_t k, int64_t part, Plan* pl) {
  pl->nvec = (V + per_vec(dt) - 1) / per_vec(dt);
  // no more blocks than kTopBlocks, rows in equal numbers of parts: the few of a
  // second round take as long as the first (200 x 152064 bf16 rows: 32 us in
  // 400 blocks, 21.7 whole; 11 x 8 beams of 128256: 22.1 in 264, 19.7 in 176)
  split(rows, pl->nvec, rows > 0 ? (int)std::max(rows, kTopBlocks / rows * rows) : 1, &pl->nch1, &pl->vpc1, part);
  const int32_t most = std::min(kPartEntries / k, kMostParts);
  if (pl->nch1 > most) {
    pl->vpc1 = (pl->nvec + most - 1) / most;
    pl->nch1 = (int32_t)((pl->nvec + pl->vpc1 - 1) / pl->vpc1);
  }
  pl->grid1 = rows * pl->nch1;
  if (pl->grid1 > INT32_MAX) return SV_EUNSUPPORTED;
  size_t off = kWsFixed;
  pl->off_lists = off;
  off = align_up(off + (size_t)pl->grid1 * k * 8, 256);
  pl->off_part1 = off;
  off = align_up(off + (size_t)pl->grid1 * sizeof(Partial), 256);
  pl->bytes = off;
  return SV_OK;
}

sv_status plan_teacher(sv_dtype dt, int32_t R, int32_t V, int32_t k, Plan* pl) {
  if (bad_dtype(dt)) return SV_EDTYPE;
  if (R < 0 || V < 1 || k < 1) return SV_EINVAL;
  if (R > SV_MAX_ROWS || V > SV_MAX_V || k > SV_MAX_FANOUT) return SV_EUNSUPPORTED;
  return plan_topmass(dt, R, V, k, kTopPartVecs, pl);
}

sv_status plan_beam(sv_dtype dt, int32_t B, int32_t W, int32_t V, int32_t N, Plan* pl) {
  if (bad_dtype(dt)) return SV_EDTYPE;
  if (B < 0 || W < 1 || V < 1 || N < 1) return SV_EINVAL;
  if (W > SV_MAX_BEAMS || (int64_t)B * W > SV_MAX_ROWS || V > SV_MAX_V || N > SV_MAX_FANOUT) return SV_EUNSUPPORTED;
  return plan_topmass(dt, (int64_t)B * W, V, N, kBeamPartVecs, pl);
}

sv_status plan_distill(sv_dtype dt, int32_t R, int32_t V, int32_t k, Plan* pl) {
  if (bad_dtype(dt)) return SV_EDTYPE;
  if (R < 0 || V < 1 || k < 1) return SV_EINVAL;
  if (R > SV_MAX_ROWS || V > SV_MAX_V || k > SV_MAX_TEACHER) return SV_EUNSUPPORTED;
  pl->nvec = (V + per_vec(dt) - 1) / per_vec(dt);
  split(R, pl->nvec, kLossBlocks, &pl->nch1, &pl->vpc1);
  if (pl->vpc1 > kDistillPartVecs) {
    pl->vpc1 = kDistillPartVecs;
    pl->nch1 = (int32_t)((pl->nvec + pl->vpc1 - 1) / pl->vpc1);
  }
  split(R, pl->nvec, kGradBlocks, &pl->nch2, &pl->vpc2);
  if ((int64_t)R * pl->nch2 < kGradFew) split(R, pl->nvec, kGradFew, &pl->nch2, &pl->vpc2, kBlockVecs / 2);
  pl->grid1 = (int64_t)R * pl->nch1;
  pl->grid2 = (int64_t)R * pl->nch2;
  if (pl->grid1 > INT32_MAX || pl->grid2 > INT32_MAX) return SV_EUNSUPPORTED;
  size_t off = kWsFixed;
  pl->off_part1 = off;
  off = align_up(off + (size_t)pl->grid1 * sizeof(Partial), 256);
  pl->bytes = off;
  return SV_OK;
}

// Whether loss and gradient together hold rows in registers, a block a row:
// wherever a row fits, but for a few long ones, which many blocks finish
// sooner in two launches.  The fewer values a vector has, the sooner a block
// is through with a row, so fp32 rows are held from longer ones and fewer on.
// Held / in two launches, us:
//   bf16  82000 logits  17.7 / 16.9 (16 rows), 18.2 / 18.7 (48)
//        110000         20.0 / 17.4 (16), 20.7 / 20.8 (56), 20.9 / 23.2 (72)
//        152064         25.9 / 18.4 (16), 27.0 / 25.9 (72), 27.2 / 27.8 (80), 27.5 / 31.3 (96)
//        196608         32.7 / 18.4 (16), 35.8 / 35.5 (104), 36.1 / 39.8 (128)
//   fp32  48000         13.3 / 14.5 (4)
//         64128         15.9 / 14.6 (4), 16.5 / 16.9 (32), 16.7 / 18.5 (40)
//         76032         19.1 / 17.3 (16), 19.7 / 18.7 (40), 19.8 / 20.4 (48)
//         98304         25.0 / 17.4 (16), 27.2 / 25.5 (80), 27.6 / 30.3 (88)
// and many rows: 2000 bf16 of 128256 210 / 278, of 152064 254 / 330, of 196608
// 340 / 423; a little more than a block a compute unit at the greatest lengths
// is the worst of it (300 of 196608: 81 / 76).
bool hold_rows(sv_dtype dt, int32_t R, int64_t nvec) {
  if (nvec > kHeldVecs) return false;
  if (dt == SV_F32) return R > (nvec - 13000) / 140;
  return nvec <= 10000 || R > nvec / 240;
}

void plan_reorder(Plan* pl) { pl->bytes = kWsFixed; }

// The gradient's rows: z itself, or apart from it.
sv_status check_grad(const void* z, int64_t stride, const void* grad, int64_t gs, int32_t R, int32_t V, sv_dtype dt) {
  const sv_status st = check_rows(grad, gs, V, dt);
  if (st != SV_OK) return st;
  if (grad == z && gs == stride) return SV_OK;
  const int64_t es = elem_bytes(dt);
  const uintptr_t a = reinterpret_cast<uintptr_t>(z), b = reinterpret_cast<uintptr_t>(grad);
  const uintptr_t ae = a + (uintptr_t)(((int64_t)(R - 1) * stride + V) * es);
  const uintptr_t be = b + (uintptr_t)(((int64_t)(R - 1) * gs + V) * es);
  return a < be && b < ae ? SV_EINVAL : SV_OK;
}

bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

void fill_distill(DistillParams* p, const Plan& pl, const void* z, sv_dtype dt, int64_t stride, int32_t R, int32_t V,
                  const int32_t* ids, const float* vals, const float* rest, int32_t k, float T, const float* g,
                  void* grad, int64_t gs, void* ws) {
  char* w = static_cast<char*>(ws);
  p->z = z;
  p->sb = stride * elem_bytes(dt);
  p->R = R;
  p->V = V;
  p->k = k;
  p->ids = ids;
  p->vals = vals;
  p->rest = rest;
  p->c = log2e_over(T);
  p->invT = 1.0 / (double)T;
  p->g = g;
  p->out_loss = nullptr;
  p->out_stat = nullptr;
  p->stat = nullptr;
  p->grad = grad;
  p->gb = gs * elem_bytes(dt);
  p->err = reinterpret_cast<int32_t*>(w);
  p->cnt = reinterpret_cast<uint32_t*>(w + kWsHeader);
  p->parts = w + pl.off_part1;
  p->nch = pl.nch1;
  p->vpc = pl.vpc1;
  p->nch2 = pl.nch2;
  p->vpc2 = pl.vpc2;
  p->nvec = pl.nvec;
}

// The bytes from a tensor's base to its end, -1 if a stride is negative or
// the extent does not fit; `apart`: whether its rows cannot overlap.
int64_t extent(const int64_t* n, const int64_t* stride, int64_t run, bool* apart) {
  int64_t end = run;
  int o[4] = {0, 1, 2, 3};
  *apart = true;
  for (int i = 0; i < 4; ++i)
    if (n[i] > 1 && stride[i] < 0) return -1;
  std::sort(o, o + 4, [&](int x, int y) { return stride[x] < stride[y]; });
  for (int j = 0; j < 4; ++j) {
    const int i = o[j];
    if (n[i] <= 1) continue;
    if (stride[i] < end) *apart = false;
    int64_t add;
    if (__builtin_mul_overflow(n[i] - 1, stride[i], &add) || __builtin_add_overflow(end, add, &end)) return -1;
  }
  return end;
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

sv_status sv_draft_workspace_size(sv_draft_op op, sv_dtype dt, int32_t rows, int32_t W, int32_t V, int32_t k,
                                  size_t* bytes) {
  if (!bytes) return SV_EINVAL;
  Plan pl;
  sv_status st = SV_OK;
  switch (op) {
    case SV_DRAFT_TEACHER: st = plan_teacher(dt, rows, V, k, &pl); break;
    case SV_DRAFT_DISTILL: st = plan_distill(dt, rows, V, k, &pl); break;
    case SV_DRAFT_BEAM: st = plan_beam(dt, rows, W, V, k, &pl); break;
    case SV_DRAFT_REORDER: plan_reorder(&pl); break;
    default: return SV_EINVAL;
  }
  if (st != SV_OK) return st;
  *bytes = pl.bytes;
  return SV_OK;
}

sv_status sv_teacher_topk(const void* logits, sv_dtype dt, int64_t stride, int32_t R, int32_t V, int32_t k, float T,
                          int32_t* out_ids, float* out_vals, float* out_rest, void* ws, size_t ws_bytes,
                          void* stream) {
  Plan pl;
  sv_status st = plan_teacher(dt, R, V, k, &pl);
  if (st != SV_OK) return st;
  if (bad_scale(T)) return SV_EINVAL;
  if (R == 0) return SV_OK;
  if ((st = check_rows(logits, stride, V, dt)) != SV_OK) return st;
  if (!out_ids || !out_vals || !out_rest) return SV_EINVAL;
  if ((st = check_ws(ws, ws_bytes, pl)) != SV_OK) return st;
  char* w = static_cast<char*>(ws);
  TeacherParams p;
  p.logits = logits;
  p.sb = stride * elem_bytes(dt);
  p.R = R;
  p.V = V;
  p.k = k;
  p.c = log2e_over(T);
  p.invT = 1.0 / (double)T;
  p.out_ids = out_ids;
  p.out_vals = out_vals;
  p.out_rest = out_rest;
  p.cnt = reinterpret_cast<uint32_t*>(w + kWsHeader);
  p.lists = w + pl.off_lists;
  p.parts = w + pl.off_part1;
  p.nch = pl.nch1;
  p.vpc = pl.vpc1;
  p.nvec = pl.nvec;
  return launch_teacher(p, dt, static_cast<hipStream_t>(stream)) == hipSuccess ? SV_OK : SV_EHIP;
}

sv_status sv_distill_topk(const void* z, sv_dtype dt, int64_t stride, int32_t R, int32_t V, const int32_t* t_ids,
                          const float* t_vals, const float* t_rest, int32_t k, float T, const float* grad_loss,
                          float* out_loss, float* out_stat, void* out_grad, int64_t grad_stride, void* ws,
                          size_t ws_bytes, void* stream) {
  Plan pl;
  sv_status st = plan_distill(dt, R, V, k, &pl);
  if (st != SV_OK) return st;
  if (bad_scale(T)) return SV_EINVAL;
  if (R == 0) return SV_OK;
  if ((st = check_rows(z, stride, V, dt)) != SV_OK) return st;
  if (!t_ids || !t_vals || !out_loss || !out_stat) return SV_EINVAL;
  if (misaligned(out_stat, 16)) return SV_EALIGN;
  if (out_grad && (st = check_grad(z, stride, out_grad, grad_stride, R, V, dt)) != SV_OK) return st;
  if ((st = check_ws(ws, ws_bytes, pl)) != SV_OK) return st;
  DistillParams p;
  fill_distill(&p, pl, z, dt, stride, R, V, t_ids, t_vals, t_rest, k, T, grad_loss, out_grad, grad_stride, ws);
  p.out_loss = out_loss;
  p.out_stat = out_stat;
  p.stat = out_stat;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (out_grad && hold_rows(dt, R, pl.nvec)) return launch_distill_held(p, dt, s) == hipSuccess ? SV_OK : SV_EHIP;
  if (launch_distill_loss(p, dt, s) != hipSuccess) return SV_EHIP;
  if (out_grad && launch_distill_grad(p, dt, s) != hipSuccess) return SV_EHIP;
  return SV_OK;
}

sv_status sv_distill_topk_backward(const void* z, sv_dtype dt, int64_t stride, int32_t R, int32_t V,
                                   const int32_t* t_ids, const float* t_vals, const float* t_rest, int32_t k, float T,
                                   const float* stat, const float* grad_loss, void* out_grad, int64_t grad_stride,
                                   void* ws, size_t ws_bytes, void* stream) {
  Plan pl;
  sv_status st = plan_distill(dt, R, V, k, &pl);
  if (st != SV_OK) return st;
  if (bad_scale(T)) return SV_EINVAL;
  if (R == 0) return SV_OK;
  if ((st = check_rows(z, stride, V, dt)) != SV_OK) return st;
  if (!t_ids || !t_vals || !stat) return SV_EINVAL;
  if (misaligned(stat, 16)) return SV_EALIGN;
  if ((st = check_grad(z, stride, out_grad, grad_stride, R, V, dt)) != SV_OK) return st;
  if ((st = check_ws(ws, ws_bytes, pl)) != SV_OK) return st;
  DistillParams p;
  fill_distill(&p, pl, z, dt, stride, R, V, t_ids, t_vals, t_rest, k, T, grad_loss, out_grad, grad_stride, ws);
  p.stat = stat;
  return launch_distill_grad(p, dt, static_cast<hipStream_t>(stream)) == hipSuccess ? SV_OK : SV_EHIP;
}

sv_status sv_beam_select(const void* logits, sv_dtype dt, int64_t stride, const float* scores, const int32_t* finished,
                         int32_t B, int32_t W, int32_t V, float T, int32_t pad_tok, int32_t N, int32_t* out_beam,
                         int32_t* out_tok, float* out_score, void* ws, size_t ws_bytes, void* stream) {
  Plan pl;
  sv_status st = plan_beam(dt, B, W, V, N, &pl);
  if (st != SV_OK) return st;
  if (bad_scale(T)) return SV_EINVAL;
  if (B == 0) return SV_OK;
  if ((st = check_rows(logits, stride, V, dt)) != SV_OK) return st;
  if (!scores || !out_beam || !out_tok || !out_score) return SV_EINVAL;
  if ((st = check_ws(ws, ws_bytes, pl)) != SV_OK) return st;
  char* w = static_cast<char*>(ws);
  BeamParams p;
  p.logits = logits;
  p.sb = stride * elem_bytes(dt);
  p.scores = scores;
  p.finished = finished;
  p.B = B;
  p.W = W;
  p.V = V;
  p.N = N;
  p.pad = pad_tok;
  p.c = log2e_over(T);
  p.invT = 1.0 / (double)T;
  p.out_beam = out_beam;
  p.out_tok = out_tok;
  p.out_score = out_score;
  p.err = reinterpret_cast<int32_t*>(w);
  p.cnt = reinterpret_cast<uint32_t*>(w + kWsHeader);
  p.lists = w + pl.off_lists;
  p.parts = w + pl.off_part1;
  p.nch = pl.nch1;
  p.vpc = pl.vpc1;
  p.nvec = pl.nvec;
  return launch_beam(p, dt, static_cast<hipStream_t>(stream)) == hipSuccess ? SV_OK : SV_EHIP;
}

sv_status sv_beam_reorder(const void* src, const int64_t* src_stride, void* dst, const int64_t* dst_stride,
                          const int32_t* parent, const int32_t* lens, int32_t L, int32_t B, int32_t W, int32_t N,
                          int32_t H, int64_t S, int64_t pos_bytes, void* ws, size_t ws_bytes, void* stream) {
  if (L < 0 || B < 0 || W < 1 || N < 1 || H < 0 || S < 0 || pos_bytes < 1) return SV_EINVAL;
  if (W > SV_MAX_BEAMS || N > SV_MAX_BEAMS || S > INT32_MAX) return SV_EUNSUPPORTED;
  int64_t run;
  if (__builtin_mul_overflow(S, pos_bytes, &run)) return SV_EUNSUPPORTED;
  if (L == 0 || B == 0 || H == 0 || run == 0) return SV_OK;
  if (!src || !dst || !src_stride || !dst_stride || !parent) return SV_EINVAL;
  const int64_t ns[4] = {L, B, W, H}, nd[4] = {L, B, N, H};
  bool apart_s, apart_d;
  const int64_t es = extent(ns, src_stride, run, &apart_s), ed = extent(nd, dst_stride, run, &apart_d);
  if (es < 0 || ed < 0 || !apart_d) return SV_EINVAL;
  bool inplace = src == dst && N <= W;
  for (int i = 0; i < 4; ++i) inplace = inplace && (src_stride[i] == dst_stride[i] || (ns[i] == 1 && nd[i] == 1));
  if (inplace && !apart_s) return SV_EINVAL;  // a beam that no beam takes the place of could lie under one that moves
  const uintptr_t a = reinterpret_cast<uintptr_t>(src), b = reinterpret_cast<uintptr_t>(dst);
  if (!inplace && a < b + (uintptr_t)ed && b < a + (uintptr_t)es) return SV_EINVAL;
  Plan pl;
  plan_reorder(&pl);
  sv_status st;
  if ((st = check_ws(ws, ws_bytes, pl)) != SV_OK) return st;
  if (reorder_blocks(run, reorder_unit(N, inplace)) > kReorderMostBlocks / ((int64_t)L * B) / H) return SV_EUNSUPPORTED;
  ReorderParams p;
  p.src = static_cast<const char*>(src);
  p.dst = static_cast<char*>(dst);
  for (int i = 0; i < 4; ++i) {
    p.ss[i] = ns[i] > 1 ? src_stride[i] : 0;
    p.ds[i] = nd[i] > 1 ? dst_stride[i] : 0;
  }
  p.parent = parent;
  p.lens = lens;
  p.L = L;
  p.B = B;
  p.W = W;
  p.N = N;
  p.H = H;
  p.S = S;
  p.pos = pos_bytes;
  p.inplace = inplace;
  p.err = reinterpret_cast<int32_t*>(static_cast<char*>(ws));
  return launch_reorder(p, static_cast<hipStream_t>(stream)) == hipSuccess ? SV_OK : SV_EHIP;
}

}  // extern "C"
