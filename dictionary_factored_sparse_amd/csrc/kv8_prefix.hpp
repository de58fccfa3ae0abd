// kv8_prefix.hpp -- what the parts of kv8_prefix_attention share: its plan, its
// workspace, and the kernel, which is compiled per head_dim.
//
// Two lines of items (kv8_attn.hpp): the groups' shared keys, each item a block
// of query rows of all the group's requests, and each request's own keys from
// there on.  The workgroups are dealt out between the two by their work.  (With a
// slice of both for every workgroup, one after the other, the chain of reads that
// starts an item was paid twice.)  What an item or a part of one gives for its rows
// stays in fp32 sums; a second kernel, over all rows at once, joins them.
#pragma once

#include "dfs_internal.hpp"

namespace dfs {

// Keys are shared where the rows of a request, on the average, leave room in what
// kv8_attention would take them in: blocks of 32 rows, of 128 for more than 32.  64
// requests of 4 query heads a cached one behind 6007 shared tokens, in us, shared and
// not: 20 rows 112, 124; 24 rows 122, 120; 28 rows 134, 121; 36 rows 172, 309; 64 rows
// 251, 313; 96 rows 348, 341; 128 rows 465, 367 (8 requests behind 20000: 24 rows 56,
// 71; 36 rows 74, 141; 80 rows 121, 159).
constexpr int kPrefixRowsFew = 24, kPrefixRowsWave = 32, kPrefixRows = 96;

struct PrefixGroup {
  int32_t t0, n;   // its tokens
  int32_t p0, p1;  // lowest and highest position of them
  int32_t keys;    // shared keys, a multiple of the tile; 0: nothing is shared
  int32_t row;     // row of the page table: of its first request that shares
};
// One line's plan.
struct PrefixEntries {
  int64_t* first;  // where each entry starts, then the total
  int32_t* of;     // group or request of each entry
  int32_t* qblk;   // its block of rows
  int32_t* n;      // entries, and the most tiles of an item
};
// What the second kernel needs to know of a token: the first entries of its
// request and of its group, and the token's first row in them; -1: none.
struct PrefixToken {
  int32_t own, own_row, shared, shared_row;
};
// How a line was cut: positions a slice, and whether no item was split.
struct PrefixSlices {
  int64_t per;
  int32_t whole, none;
};
struct PrefixPlan {
  PrefixGroup* groups;  // [n_groups]
  int32_t* live;        // [n_groups]: requests with tokens
  int32_t* from;        // [n_req]: first key of its own
  int32_t* pos;         // [n_tok]: position of each token
  PrefixEntries shared, own;
};
// One line's sums.
struct PrefixSums {
  float* part_o;  // [2 * slices][rows][D], as run_line places them
  f2* part_ml;
  float* o;       // [tokens * q_heads][D]: of items that are not split
  f2* ml;
};
struct PrefixWs {
  PrefixPlan plan;
  PrefixToken* tokens;   // [n_tok]
  PrefixSlices* slices;  // [2]: of shared keys, of own ones
  PrefixSums shared, own;
  int32_t most_shared, most_own;  // entries at most
};
// The forms of the two lines.
struct PrefixCut {
  bool split;       // of the shared keys: the waves of a workgroup take tiles in turn
  int nq, qb;       // groups of 16 rows a wave, rows an item
  int nq_own;       // of the own keys, always in turn
  int slices;
  int in;           // the workgroups plan for themselves
};
struct PrefixLaunch {
  KvAttnLaunch a;
  int32_t n_groups;
  const int32_t *group_start, *shared;
};

// Up to these the workgroups plan for themselves, in LDS, and there is one launch less
// (four beams of 1561 tokens 17.9 us, 21.6 with a launch for the plan; 64 requests
// behind 6007 tokens 44.3, 48.5).  More would not fit beside the joins of two workgroups
// a CU.
constexpr int kPrefixInline = 128;         // requests
constexpr int kPrefixInlineTokens = 256;
constexpr int kPrefixInlineEntries = 128;  // of either line, at most
// Own keys: tiles up to which items are not split, but dealt out whole.  48 samples of
// 500 own tokens 62.5 us, 76.8 split; four beams of 500 own tokens 20.0, 18.7.
constexpr int kPrefixEach = 16;

template <int D>
void launch_prefix(const PrefixLaunch& p, const PrefixWs& w, const PrefixCut& c, hipStream_t s);

}  // namespace dfs
