// kv8_prefix_plan.hpp -- the plan of kv8_prefix_attention: which rows share which
// keys, and the entries of the two lines.
#pragma once

#include "kv8_attn.hpp"
#include "kv8_prefix.hpp"

namespace dfs {
namespace {

// The facts of a small batch, in LDS.
struct PrefixInline {
  int64_t tmp[kWaves];
  int32_t longest;
  Req facts[kPrefixInline];
  int32_t group_start[kPrefixInline + 1], shared[kPrefixInline];
  PrefixGroup groups[kPrefixInline];
  int32_t live[kPrefixInline], from[kPrefixInline], pos[kPrefixInlineTokens];
  int32_t group_of[kPrefixInline], first_entry[kPrefixInline], first_shared[kPrefixInline];
  struct Entries {
    int64_t first[kPrefixInlineEntries + 1];
    int32_t of[kPrefixInlineEntries], qblk[kPrefixInlineEntries], n[2];
  } line_shared, line_own;
};

// Entries of one line in order, and where each starts: blocks(i) blocks of rows of
// group or request i, of tiles(i, block) tiles each, `extra` counted beside them;
// at(i, entry) is told the first entry of each.
template <int T, typename B, typename F, typename G>
__device__ __forceinline__ void plan_line(const PrefixEntries& w, int most, int n, int heads, int extra, B blocks,
                                          F tiles, G at_first, int64_t* tmp, int* longest) {
  int n_entries = 0;
  for (int i0 = 0; i0 < n; i0 += T) {
    const int i = i0 + (int)threadIdx.x;
    const int nb = i < n ? min(blocks(i), most) : 0;
    int64_t total;
    const int64_t at = n_entries + block_scan<int64_t>(nb, tmp, &total, T);
    if (i < n) at_first(i, (int)min(at, (int64_t)most));
    for (int b = 0; b < nb && at + b < most; ++b) {
      w.of[at + b] = i;
      w.qblk[at + b] = b;
    }
    n_entries = (int)min(n_entries + total, (int64_t)most);
  }
  if (threadIdx.x == 0) *longest = 0;
  __syncthreads();
  int64_t base = 0;
  int top = 0;
  for (int e0 = 0; e0 < n_entries; e0 += T) {
    const int e = e0 + (int)threadIdx.x;
    int64_t t = 0;
    if (e < n_entries) {
      const int m = tiles(w.of[e], w.qblk[e]);
      top = max(top, m);
      t = ((int64_t)m + extra) * heads;
    }
    int64_t total;
    const int64_t at = base + block_scan<int64_t>(t, tmp, &total, T);
    if (e < n_entries) w.first[e] = at;
    base += total;
  }
  if (top > 0) atomicMax(longest, top);
  __syncthreads();
  if (threadIdx.x == 0) {
    w.first[n_entries] = base;
    w.n[0] = n_entries;
    w.n[1] = *longest;
  }
  __syncthreads();
}

// The plan, by one workgroup of T threads.  facts(r): request r; starts(i), shared(i):
// of group i; group_of, entry_own, entry_shared: scratch of one int a request, a
// request, a group; put_token takes what the second kernel needs.
template <int T, typename Q, typename S, typename H, typename P>
__device__ __forceinline__ void make_prefix_plan(const PrefixLaunch& p, const PrefixPlan& w, Q facts, S starts,
                                                 H shared, int32_t* group_of, int32_t* entry_own,
                                                 int32_t* entry_shared, int most_shared, int most_own, int qb,
                                                 int extra, int qb_own, int extra_own, P put_token,
                                                 int64_t* tmp, int* longest) {
  const KvAttnLaunch& a = p.a;
  const int tid = threadIdx.x, g = a.q_heads / a.kv.heads;
  // tokens that group i shares, as far as the table goes
  auto shared_of = [&](int i) {
    return (int)min((int64_t)max(shared(i), 0), (int64_t)a.b.table_pages * a.kv.page);
  };
  for (int i = tid; i < p.n_groups; i += T) {
    const int r = min(max(starts(i), 0), max(a.b.n_req - 1, 0));
    w.groups[i] = PrefixGroup{INT32_MAX, INT32_MIN, INT32_MAX, INT32_MIN, 0, r};
    w.live[i] = 0;
  }
  __syncthreads();
  for (int r = tid; r < a.b.n_req; r += T) {
    const Req q = facts(r);
    int lo = 0, hi = p.n_groups;  // the last group that starts at or before r, if any does
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (starts(mid) <= r) lo = mid;
      else hi = mid;
    }
    const bool in = starts(lo) <= r && r < starts(lo + 1) && q.len >= shared_of(lo);  // else it stands alone
    group_of[r] = in ? lo : -1;
    if (!in || q.n <= 0) continue;
    PrefixGroup* f = w.groups + lo;
    atomicMin(&f->t0, q.t0);
    atomicMax(&f->n, q.t0 + q.n);  // their end, for now
    atomicMin(&f->p0, q.len - q.n);
    atomicMax(&f->p1, q.len - 1);
    atomicAdd(w.live + lo, 1);
  }
  __syncthreads();
  for (int i = tid; i < p.n_groups; i += T) {
    PrefixGroup f = w.groups[i];
    f.keys = shared_of(i) / kTile * kTile;
    // worth it for two requests that see some of it
    if (w.live[i] < 2) f.keys = 0;
    else f.n -= f.t0;  // with the tokens between of requests that stand alone, whose sums nobody takes
    if (f.keys > 0) {
      const int hi = min(f.p1, f.keys - 1), lo = a.window > 0 && f.p0 >= a.window ? f.p0 - a.window + 1 : 0;
      if (hi < 0 || (hi < lo && a.sinks <= 0)) f.keys = 0;
    }
    w.groups[i].n = f.n;
    w.groups[i].keys = f.keys;
  }
  __syncthreads();
  for (int r = tid; r < a.b.n_req; r += T) {
    const int i = group_of[r];
    w.from[r] = i < 0 ? 0 : w.groups[i].keys;
  }
  plan_line<T>(
      w.shared, most_shared, p.n_groups, a.kv.heads, extra,
      [&](int i) {
        const PrefixGroup& f = w.groups[i];
        return f.keys > 0 ? (int)(((int64_t)f.n * g + qb - 1) / qb) : 0;
      },
      [&](int i, int) {
        const PrefixGroup& f = w.groups[i];
        return get_span(Req{f.t0, f.n, f.keys, f.keys}, f.p0, f.p1, a.window, a.sinks).n;
      },
      [&](int i, int e) { entry_shared[i] = e; }, tmp, longest);
  plan_line<T>(
      w.own, most_own, a.b.n_req, a.kv.heads, extra_own,
      [&](int r) { return (int)(((int64_t)facts(r).n * g + qb_own - 1) / qb_own); },
      [&](int r, int b) {
        const Req q = facts(r);
        const int i0 = (int)((int64_t)b * qb_own / g);
        const int i1 = (int)min(((int64_t)(b + 1) * qb_own - 1) / g, (int64_t)q.n - 1);
        return get_span(q, q.len - q.n + i0, q.len - q.n + i1, a.window, a.sinks, w.from[r]).n;
      },
      [&](int r, int e) { entry_own[r] = e; }, tmp, longest);
  for (int t = tid; t < a.b.n_tok; t += T) {
    int lo = 0, hi = a.b.n_req;  // the last request that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (facts(mid).t0 <= t) lo = mid;
      else hi = mid;
    }
    const Req q = facts(lo);
    w.pos[t] = q.len - q.n + (t - q.t0);
    PrefixToken k = {-1, 0, -1, 0};
    if (t >= q.t0 && t < q.t0 + q.n) {
      k.own = entry_own[lo];
      k.own_row = (t - q.t0) * g;
      const int i = group_of[lo];
      if (i >= 0 && w.groups[i].keys > 0) {
        k.shared = entry_shared[i];
        k.shared_row = (t - w.groups[i].t0) * g;
      }
    }
    put_token(t, k);
  }
  __syncthreads();
}

}  // namespace
}  // namespace dfs
