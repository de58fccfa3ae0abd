// kv8_prefix.hpp -- what the parts of kv8_prefix_attention share: its plan, its
// workspace, and the kernel, which is compiled per head_dim.
//
// Two lines of items (kv8_attn.hpp): the groups' shared keys, each item a block
// of query rows of all the group's requests, and each request's own keys from
// there on.  A workgroup takes its slice of the one and then its slice of the
// other, so that both load every CU alike whatever their share of the work, with
// no gap between them.  Each line leaves sums of its own for each row, in fp32;
// a second kernel puts them together.
#pragma once

#include "dfs_internal.hpp"

namespace dfs {

// Rows of a request up to which keys are shared: above, the rows of one request
// already fill what a wave takes at once.
constexpr int kPrefixRows = 32;

struct PrefixGroup {
  int32_t t0, n;   // its tokens
  int32_t p0, p1;  // lowest and highest position of them
  int32_t keys;    // shared keys, a multiple of the tile; 0: nothing is shared
  int32_t row;     // row of the page table
};
// One line's plan and parts.
struct PrefixLine {
  int64_t* first;  // where each entry starts, then the total
  int32_t* of;     // group or request of each entry
  int32_t* qblk;   // its block of rows
  int32_t* n;      // entries, and the most tiles of an item
  int32_t most;    // entries at most
  uint32_t* count;
  float* part_o;
  f2* part_ml;
  f2* group_ml;
  float* sum_o;    // [tokens * q_heads][D]: what the line gives for each row
  f2* sum_ml;
};
struct PrefixWs {
  PrefixGroup* groups;  // [n_groups]
  int32_t* live;        // [n_groups]: requests with tokens
  int32_t* group_of;    // [n_req]: group of each request, or -1
  int32_t* pos;         // [n_tok]: position of each token
  PrefixLine shared, own;
};
// The forms of the two lines.
struct PrefixCut {
  bool split;       // of the shared keys: the waves of a workgroup take tiles in turn
  int nq, qb;       // groups of 16 rows a wave, rows an item
  int nq_own;       // of the own keys, always in turn
  int slices;
};
struct PrefixLaunch {
  KvAttnLaunch a;
  int32_t n_groups;
  const int32_t *group_start, *shared;
};

template <int D>
void launch_prefix(const PrefixLaunch& p, const PrefixWs& w, const PrefixCut& c, hipStream_t s);

}  // namespace dfs
