// sv_draft.h -- launch parameters of the drafter-side entry points (not part
// of the public C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specverify_draft.h"

namespace sv {

// A part of a row: its list of k entries and the mass outside the list
// (Partial), merged by the row's last block.
struct TeacherParams {
  const void* logits;
  int64_t sb;
  int32_t R, V, k;
  float c;      // log2(e) / T
  double invT;  // 1 / T
  int32_t* out_ids;
  float* out_vals;
  float* out_rest;
  uint32_t* cnt;  // arrivals per row
  void* lists;    // [R][nch][k] entries (nch > 1)
  void* parts;    // [R][nch] partials (nch > 1)
  int32_t nch;
  int64_t vpc, nvec;
};

struct BeamParams {
  const void* logits;
  int64_t sb;
  const float* scores;
  const int32_t* finished;
  int32_t B, W, V, N, pad;
  float c;
  double invT;
  int32_t* out_beam;
  int32_t* out_tok;
  float* out_score;
  int32_t* err;
  uint32_t* cnt;  // arrivals per sequence
  void* lists;    // [B * W][nch][N] entries
  void* parts;    // [B * W][nch] partials
  int32_t nch;
  int64_t vpc, nvec;
};

struct DistillParams {
  const void* z;
  int64_t sb;
  int32_t R, V, k;
  const int32_t* ids;
  const float* vals;
  const float* rest;  // or null: no mass outside the teacher's tokens
  float c;
  double invT;
  const float* g;  // or null: all 1
  float* out_loss;
  float* out_stat;
  const float* stat;  // backward's input
  void* grad;
  int64_t gb;  // gradient row stride in bytes
  int32_t* err;
  uint32_t* cnt;  // arrivals per row
  void* parts;    // [R][nch] partials (nch > 1)
  int32_t nch, nch2;  // parts of a row: loss, gradient
  int64_t vpc, vpc2, nvec;
};
constexpr int64_t kDistillPartVecs = 32768;  // vectors of a loss part at most (a byte of LDS marks each)
constexpr int64_t kHeldVecs = 1024 * 24;  // vectors of a row that a block can hold in registers

struct ReorderParams {
  const char* src;
  char* dst;
  int64_t ss[4], ds[4];  // byte strides: layer, sequence, beam, segment
  const int32_t* parent;
  const int32_t* lens;
  int32_t L, B, W, N, H;
  int64_t S, pos;  // positions, bytes per position
  bool inplace;
  int32_t* err;
};

hipError_t launch_teacher(const TeacherParams& p, sv_dtype dt, hipStream_t s);
hipError_t launch_beam(const BeamParams& p, sv_dtype dt, hipStream_t s);
hipError_t launch_distill_loss(const DistillParams& p, sv_dtype dt, hipStream_t s);
hipError_t launch_distill_grad(const DistillParams& p, sv_dtype dt, hipStream_t s);
hipError_t launch_distill_held(const DistillParams& p, sv_dtype dt, hipStream_t s);
hipError_t launch_reorder(const ReorderParams& p, hipStream_t s);
constexpr int kReorderOdd = 6;  // places at a segment's end: of 4 bytes (3 at most) and of one (3)
constexpr int kReorderThreads = 256;
// Bytes of a place: in place every beam's piece is held at once; apart, 16 beams at a time.
inline int reorder_unit(int32_t N, bool inplace) { return N <= 16 || !inplace ? 16 : N <= 32 ? 8 : 4; }
// Blocks of a segment of `run` bytes, and of a launch at most (fewer than 2^32 threads).
inline int64_t reorder_blocks(int64_t run, int unit) {
  return (run / unit + kReorderOdd + kReorderThreads - 1) / kReorderThreads;
}
constexpr int64_t kReorderMostBlocks = UINT32_MAX / kReorderThreads;

}  // namespace sv
