// The packed sequences' plan: which workgroup takes which rows and keys.
// Shared by the attention kernels and the planner.
#pragma once

#include <mutex>
#include <vector>

#include "internal.h"

namespace st {

// One workgroup's share of one sequence, for one key-value head.  Rows are
// (query token, head of the group) pairs: row r is token r / group, head
// r % group, so the heads that share keys share a tile.
struct AttnItem {
  int32_t q0, lq, k0, lk;   // the sequence: first query and key token, lengths
  int32_t at;               // forward, dq: first row of the tile; dk, dv: first key
  int32_t lo, hi;           // forward, dq: keys [lo, hi); dk, dv: rows [lo, hi)
  int32_t part;             // slot of its partial result, -1: the result itself
};
// A tile whose keys (rows) were split: parts [first, first + count)
struct AttnJoin {
  int32_t q0, lq, k0, lk, at, first, count, pad;
};

// A kernel's launch: items for four waves and for one wave, and its joins
struct AttnList {
  std::vector<AttnItem> item[2];     // 0: four waves, 1: one wave
  std::vector<AttnJoin> join[2];
  int32_t tile[2] = {0, 0};          // rows (keys) of a tile
  int64_t parts[2] = {0, 0};         // partial slots
  const AttnItem* d_item[2] = {nullptr, nullptr};
  const AttnJoin* d_join[2] = {nullptr, nullptr};
};

enum { kListForward = 0, kListDq = 1, kListDkv = 2, kLists = 3 };

// Tile shapes of a kernel for one element type and padded head width
struct AttnShape {
  int tile[kLists][2];      // rows (keys) per tile: four waves, one wave
  int step[kLists];         // keys (rows) of one step of the loop
  int fill[kLists][2];      // workgroups that fill the GPU
};
inline int attn_padded_dim(int dim) { return dim <= 32 ? 32 : dim <= 64 ? 64 : dim <= 96 ? 96 : 128; }
AttnShape attn_shape(st_dtype dtype);

}  // namespace st

struct st_seqs {
  int32_t nseq, heads, kv_heads, group, dim, dp, causal;
  st_dtype dtype;
  int64_t total_q = 0, total_k = 0;
  st::AttnShape shape;
  st::AttnList list[st::kLists];
  std::mutex dev_mu;
  char* d_table = nullptr;
  int dev_id = -1;
};

namespace st {
// Uploads the work tables on first use (on the current device).
st_status seqs_device_table(st_seqs* s, hipStream_t stream);
}  // namespace st
