// sv_host.hpp -- host-side helpers that the entry points' files share:
// argument checks and the splitting of rows over blocks.
#pragma once

#include <cmath>
#include <cstdlib>

#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kBlockVecs = 1024;   // smallest row part (vectors): 4 in flight per thread of a 256-thread block

inline int env_int(const char* name, int dflt) {
  const char* v = std::getenv(name);
  if (!v || !*v) return dflt;
  const int x = std::atoi(v);
  return x > 0 ? x : dflt;
}

// Blocks the streaming passes aim for (the chip has 256 CUs; four blocks of
// 256 threads per CU with four 16-byte loads in flight per thread keep the
// HBM busy; fewer, longer parts also mean fewer parts to merge).
// Overridable for tuning sweeps with SV_STATS_BLOCKS.
inline int stats_blocks() {
  static const int v = env_int("SV_STATS_BLOCKS", 1024);
  return v;
}
inline int per_vec(sv_dtype dt) { return dt == SV_BF16 ? 8 : 4; }
inline int elem_bytes(sv_dtype dt) { return dt == SV_BF16 ? 2 : 4; }

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Split rows of nvec vectors into parts of at least min_vecs vectors so that
// rows * parts ~ target.
inline void split(int64_t rows, int64_t nvec, int target, int32_t* nch, int64_t* vpc, int64_t min_vecs = kBlockVecs) {
  int64_t n = rows > 0 ? (target + rows - 1) / rows : 1;
  const int64_t cap = nvec / min_vecs > 1 ? nvec / min_vecs : 1;
  if (n > cap) n = cap;
  if (n < 1) n = 1;
  int64_t per = (nvec + n - 1) / n;
  if (per < 1) per = 1;
  *vpc = per;
  *nch = (int32_t)((nvec + per - 1) / per);
}

inline bool bad_dtype(sv_dtype dt) { return dt != SV_BF16 && dt != SV_F32; }

inline sv_status check_rows(const void* base, int64_t stride, int32_t V, sv_dtype dt) {
  if (!base) return SV_EINVAL;
  if (stride < V) return SV_EINVAL;
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0) return SV_EALIGN;
  if ((stride * elem_bytes(dt)) % 16 != 0) return SV_EALIGN;
  return SV_OK;
}

inline bool bad_temperature(float T) { return !(T > 0.f) || !std::isfinite(T); }

inline sv_status check_ws(const void* ws, size_t ws_bytes, const Plan& pl) {
  if (!ws || ws_bytes < pl.bytes) return SV_EWORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return SV_EALIGN;
  return SV_OK;
}

inline float log2e_over(float T) { return (float)(1.4426950408889634 / (double)T); }

}  // namespace

}  // namespace sv
