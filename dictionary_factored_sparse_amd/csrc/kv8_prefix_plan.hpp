// kv8_prefix_plan.hpp -- the plan of kv8_prefix_attention: which rows share which
// keys, and the entries of the two lines.
#pragma once

#include "kv8_attn.hpp"
#include "kv8_prefix.hpp"

namespace dfs {
namespace {

// The facts of a small batch, in LDS.
struct PrefixInline {
  int64_t tmp[kWaves][2];
  int32_t longest[2];
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

// Two sums over the threads before this one, and over all of them.
template <int T>
__device__ __forceinline__ void block_scan2(int64_t& x, int64_t& y, int64_t (*tmp)[2], int64_t& all_x,
                                            int64_t& all_y) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int64_t sx = x, sy = y;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t ux = __shfl_up(sx, o, kWave), uy = __shfl_up(sy, o, kWave);
    if (lane >= o) {
      sx += ux;
      sy += uy;
    }
  }
  if (lane == kWave - 1) {
    tmp[wave][0] = sx;
    tmp[wave][1] = sy;
  }
  __syncthreads();
  all_x = all_y = 0;
  x = sx - x;
  y = sy - y;
#pragma unroll
  for (int w = 0; w < T / kWave; ++w) {
    const int64_t ux = tmp[w][0], uy = tmp[w][1];
    if (w < wave) {
      x += ux;
      y += uy;
    }
    all_x += ux;
    all_y += uy;
  }
  __syncthreads();
}

// Workgroups that take shared keys, of all; the others take own ones.  By the two
// lines' work: a tile of shared keys takes as long as kTileCost of own ones where
// each wave has rows of its own (3.6 us, 1.5).
constexpr float kTileCost = 2.4f;
__device__ __forceinline__ int shared_slices(int64_t shared, int64_t own, bool split, int slices) {
  if (own <= 0) return slices;
  if (shared <= 0) return 0;
  const float x = (float)shared * (split ? 1.0f : kTileCost);
  return min(max((int)(x / (x + (float)own) * (float)slices + 0.5f), 1), slices - 1);
}

// The plan, by one workgroup of T threads.  facts(r): request r; starts(i), shared(i):
// of group i; group_of, entry_own, entry_shared: scratch of one int a request, a
// request, a group; put_token takes what the second kernel needs.
template <int T, typename Q, typename S, typename H, typename P>
__device__ __forceinline__ void make_prefix_plan(const PrefixLaunch& p, const PrefixPlan& w, Q facts, S starts,
                                                 H shared, int32_t* group_of, int32_t* entry_own,
                                                 int32_t* entry_shared, int most_shared, int most_own, int qb,
                                                 int extra, int qb_own, int extra_own, P put_token,
                                                 int64_t (*tmp)[2], int* longest) {
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
  // entries in order: first those of both lines' groups and requests, then where
  // each starts in its line
  auto put_entries = [&](const PrefixEntries& l, int64_t at, int nb, int most, int i) {
    for (int b = 0; b < nb && at + b < most; ++b) {
      l.of[at + b] = i;
      l.qblk[at + b] = b;
    }
  };
  const int n = max(p.n_groups, a.b.n_req);
  int64_t n_shared = 0, n_own = 0;
  for (int i0 = 0; i0 < n; i0 += T) {
    const int i = i0 + tid;
    int nb_shared = 0, nb_own = 0;
    if (i < p.n_groups && w.groups[i].keys > 0) nb_shared = (int)(((uint32_t)(w.groups[i].n * g) + qb - 1) / qb);
    if (i < a.b.n_req) nb_own = (int)(((uint32_t)(facts(i).n * g) + qb_own - 1) / qb_own);
    int64_t x = nb_shared, y = nb_own, all_x, all_y;
    block_scan2<T>(x, y, tmp, all_x, all_y);
    x += n_shared;
    y += n_own;
    if (i < p.n_groups) entry_shared[i] = (int)min(x, (int64_t)most_shared);
    if (i < a.b.n_req) entry_own[i] = (int)min(y, (int64_t)most_own);
    put_entries(w.shared, x, nb_shared, most_shared, i);
    put_entries(w.own, y, nb_own, most_own, i);
    n_shared += all_x;
    n_own += all_y;
  }
  n_shared = min(n_shared, (int64_t)most_shared);
  n_own = min(n_own, (int64_t)most_own);
  if (tid < 2) longest[tid] = 0;
  __syncthreads();
  int64_t base_shared = 0, base_own = 0;
  int top_shared = 0, top_own = 0;
  for (int e0 = 0; e0 < max(n_shared, n_own); e0 += T) {
    const int e = e0 + tid;
    int64_t x = 0, y = 0, all_x, all_y;
    if (e < n_shared) {
      const PrefixGroup& f = w.groups[w.shared.of[e]];
      const int m = get_span(Req{f.t0, f.n, f.keys, f.keys}, f.p0, f.p1, a.window, a.sinks).n;
      top_shared = max(top_shared, m);
      x = ((int64_t)m + extra) * a.kv.heads;
    }
    if (e < n_own) {
      const int r = w.own.of[e];
      const Req q = facts(r);
      const uint32_t r0 = w.own.qblk[e] * qb_own, r1 = min(r0 + qb_own, (uint32_t)(q.n * g)) - 1;
      const int p0 = q.len - q.n;
      const int m = get_span(q, p0 + (int)(r0 / g), p0 + (int)(r1 / g), a.window, a.sinks, w.from[r]).n;
      top_own = max(top_own, m);
      y = ((int64_t)m + extra_own) * a.kv.heads;
    }
    block_scan2<T>(x, y, tmp, all_x, all_y);
    if (e < n_shared) w.shared.first[e] = base_shared + x;
    if (e < n_own) w.own.first[e] = base_own + y;
    base_shared += all_x;
    base_own += all_y;
  }
  if (top_shared > 0) atomicMax(longest, top_shared);
  if (top_own > 0) atomicMax(longest + 1, top_own);
  __syncthreads();
  if (tid == 0) {
    w.shared.first[n_shared] = base_shared;
    w.own.first[n_own] = base_own;
    w.shared.n[0] = (int)n_shared;
    w.own.n[0] = (int)n_own;
    w.shared.n[1] = longest[0];
    w.own.n[1] = longest[1];
  }
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
