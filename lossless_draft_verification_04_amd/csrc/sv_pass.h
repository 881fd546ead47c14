// sv_pass.h -- launch parameters of the verifier's pass (not part of the
// public C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specverify_pass.h"

namespace sv {

// A cache as the kernels see it; offsets in bytes within a head's part of a page.
struct Kv {
  char* pool;
  const int32_t* pages;
  int64_t page_stride, layer_stride;
  int64_t head;          // bytes of a head in a page
  int64_t ks, vc, vs;    // where the keys' scales, the values, their scales begin
  int32_t num_pages, max_pages, pshift, H, layers;
  int64_t room;          // tokens that a sequence's table holds
};

struct RopeParams {
  const char* in[2];
  char* out[2];
  int64_t is[2][3], os[2][3];  // bytes: sequence, node, head
  int32_t B, N, heads[2], D, R;
  const double* freq;
  float factor;
  bool interleaved, inverse;
  const int32_t* positions;
  const int32_t* lens;
  const int32_t* parent;
  int32_t* err;
};

struct KvMoveParams {  // write, read
  Kv c;
  char* k;  // read by the write, written by the read
  char* v;
  int64_t st[2][3];  // bytes: sequence, token, head
  const int32_t* lens;
  const int32_t* news;
  int32_t B, N;
  int32_t* err;
};

struct KvCommitParams {
  Kv c;
  const int32_t* lens;
  const int32_t* n;
  const int32_t* path;
  int32_t B, M;
  int32_t* out_lens;
  int32_t* err;
};

struct AttentionParams {
  Kv c;
  const char* q;
  char* out;
  int64_t qs[3], os[3];  // bytes: sequence, node, head
  float* lse;
  const int32_t* lens;
  const int32_t* news;
  const int32_t* parent;
  int32_t B, N, Hq, G;  // G query heads of a key head
  float scale, cap;
  const float* slopes;
  int32_t reach;
  int32_t* err;
  int32_t tiles, split;  // a block's rows: `split` waves beside one another with so many tiles of 16 each
  int32_t groups, all_tiles;  // groups of so many rows, and all tiles
  int32_t blocks, log_blocks;
  float* part_o;  // [2 * blocks][split * tiles * 16][D]: a block's first and last item
  float* part_ml; // [2 * blocks][split * tiles * 16][2]: reference, sum
  void* desc;     // [blocks] of AttentionItem
};

// An item (a sequence's key head and group of rows) that several blocks share.
struct AttentionItem {
  int32_t b, h, group;  // b = -1: none
  int32_t news;         // of the sequence
  int32_t slot, last;   // of the first block's part; the last block
  int32_t unused[2];    // 32 bytes
};

hipError_t launch_rope(const RopeParams& p, sv_dtype dt, hipStream_t s);
hipError_t launch_kv_write(const KvMoveParams& p, sv_dtype dt, int D, hipStream_t s);
hipError_t launch_kv_read(const KvMoveParams& p, sv_dtype dt, int D, hipStream_t s);
hipError_t launch_kv_commit(const KvCommitParams& p, int D, hipStream_t s);
hipError_t launch_kv_attention(const AttentionParams& p, sv_dtype dt, int D, hipStream_t s);

// How `all` tiles of 16 rows (nodes x heads of a key head) are taken: as many
// in a wave as its registers hold (`most`: two at D = 256 would spill 114 to 198
// of them), more by two or four waves beside one another, which read the same
// tokens, more still by several blocks.  Waves beside one another against blocks
// of their own: 5 tiles of 128 values 119 against 127 us (32 chains of 17 nodes x
// 4 heads), 16 of 256 values 265 against 278 (trees of 64 x 4, 65536 tokens), 256 of
// 128 values as long (1024 nodes x 4 heads: 313 and 309).
struct AttentionForm {
  int tiles, split, groups, blocks;
};
inline AttentionForm attention_form(int D, int all) {
  const int most = D == 64 ? 4 : D == 128 ? 3 : 1;
  AttentionForm f;
  f.groups = (all + 4 * most - 1) / (4 * most);
  const int each = (all + f.groups - 1) / f.groups;
  f.split = each <= most ? 1 : each <= 2 * most ? 2 : 4;
  f.tiles = (each + f.split - 1) / f.split;
  f.groups = (all + f.split * f.tiles - 1) / (f.split * f.tiles);
  // as many blocks as are resident at once
  f.blocks = f.split > 1 ? 256 : f.tiles > 1 || D == 256 ? 512 : D == 64 ? 1024 : 768;
  return f;
}
constexpr int kAttentionBlocks = 1024;  // at most

}  // namespace sv
