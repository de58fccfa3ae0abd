// kv8_prefix_plan.hpp -- the plan of kv8_prefix_attention: which rows share which
// keys, and the entries of the two lines.
#pragma once

#include "kv8_attn.hpp"
#include "kv8_prefix.hpp"

namespace dfs {
namespace {

// What the lanes before this one hold, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t moved(int64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), CTRL, ROWS, 0xF, false);
  return (int64_t)((uint64_t)(uint32_t)hi << 32 | lo);
}

// Three sums over the threads before this one, and over all of them.
struct Scan3 {
  int64_t v[3];
};
template <int T>
__device__ __forceinline__ Scan3 block_scan3(const Scan3& x, Scan3* tmp, Scan3& all) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  Scan3 s = x;
#pragma unroll
  for (int i = 0; i < 3; ++i) {  // from 1, 2, 4, 8 lanes before, then between rows of 16 lanes
    s.v[i] += moved<0x111, 0xF>(s.v[i]);
    s.v[i] += moved<0x112, 0xF>(s.v[i]);
    s.v[i] += moved<0x114, 0xF>(s.v[i]);
    s.v[i] += moved<0x118, 0xF>(s.v[i]);
    s.v[i] += moved<0x142, 0xA>(s.v[i]);
    s.v[i] += moved<0x143, 0xC>(s.v[i]);
  }
  if (lane == kWave - 1) tmp[wave] = s;
  __syncthreads();
  all = {};
#pragma unroll
  for (int i = 0; i < 3; ++i) s.v[i] -= x.v[i];
#pragma unroll 4
  for (int w = 0; w < T / kWave; ++w) {
    const Scan3 u = tmp[w];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      s.v[i] += w < wave ? u.v[i] : 0;
      all.v[i] += u.v[i];
    }
  }
  __syncthreads();
  return s;
}

// The facts of a small batch, in LDS.
struct PrefixInline {
  Scan3 tmp[kWaves];
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

// Workgroups that take shared keys, of all; the others take own ones.  By the two
// lines' work: a tile of shared keys takes as long as kTileCost of own ones where
// each wave has rows of its own (3.6 us, 1.5), and beside those, own items that are not
// split cost kWholeCost of what they count in the line, where `extra` stands for a join
// as well (24 questions to a document 92 us without, 88 so).
constexpr float kTileCost = 2.4f, kWholeCost = 0.6f;
__device__ __forceinline__ int shared_slices(int64_t shared, int64_t own, int longest, bool split, int slices) {
  if (own <= 0) return slices;
  if (shared <= 0) return 0;
  const float x = (float)shared * (split ? 1.0f : kTileCost);
  const float y = (float)own * (!split && longest <= kPrefixEach ? kWholeCost : 1.0f);
  return min(max((int)(x / (x + y) * (float)slices + 0.5f), 1), slices - 1);
}

// The plan, by one workgroup of T threads.  facts(r): request r; starts(i), shared(i):
// of group i; group_of, entry_own, entry_shared: scratch of one int a request, a
// request, a group; put_token takes what the second kernel needs.  Begins after a
// barrier that facts, starts and shared want.
template <int T, typename Q, typename S, typename H, typename P>
__device__ __forceinline__ void make_prefix_plan(const PrefixLaunch& p, const PrefixPlan& w, Q facts, S starts,
                                                 H shared, int32_t* group_of, int32_t* entry_own,
                                                 int32_t* entry_shared, int most_shared, int most_own, int qb,
                                                 int extra, int qb_own, int extra_own, P put_token,
                                                 Scan3* tmp, int* longest) {
  const KvAttnLaunch& a = p.a;
  const int tid = threadIdx.x, heads = a.kv.heads;
  const uint32_t g = a.q_heads / heads;
  // tokens that group i shares, as far as the table goes
  auto shared_of = [&](int i) {
    return (int)min((int64_t)max(shared(i), 0), (int64_t)a.b.table_pages * a.kv.page);
  };
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
    atomicMin(&f->row, r);  // the rows of requests that stand alone need not name the shared pages
    atomicAdd(w.live + lo, 1);
  }
  __syncthreads();
  // what a group shares: worth it for two requests that see some of it
  auto keys_of = [&](int i, const PrefixGroup& f) {
    const int keys = w.live[i] < 2 ? 0 : shared_of(i) / kTile * kTile;
    const int hi = min(f.p1, keys - 1), lo = a.window > 0 && f.p0 >= a.window ? f.p0 - a.window + 1 : 0;
    return hi < 0 || (hi < lo && a.sinks <= 0) ? 0 : keys;
  };
  const int n = max(p.n_groups, a.b.n_req);
  int64_t n_shared = 0, n_own = 0, base_shared = 0, base_own = 0;
  int top_shared = 0, top_own = 0;
  for (int i0 = 0; i0 < n; i0 += T) {
    const int i = i0 + tid;
    PrefixGroup f = {};
    Span fs = {}, rs = {};
    uint32_t nb_shared = 0, nb_own = 0;
    Scan3 x = {}, all;
    Req q = {};
    int from = 0;
    bool uniform = true;  // whether all blocks of a request have the same tiles
    auto span_of = [&](uint32_t b) {
      const uint32_t r0 = b * qb_own, r1 = min(r0 + qb_own, (uint32_t)q.n * g) - 1;
      const int p0 = q.len - q.n;
      return get_span(q, p0 + (int)(r0 / g), p0 + (int)(r1 / g), a.window, a.sinks, from);
    };
    if (i < p.n_groups) {
      f = w.groups[i];
      f.keys = keys_of(i, f);
      if (f.keys > 0) {
        f.n -= f.t0;  // with the tokens between of requests that stand alone, whose sums nobody takes
        nb_shared = ((uint32_t)f.n * g + qb - 1) / qb;
        fs = get_span(Req{f.t0, f.n, f.keys, f.keys}, f.p0, f.p1, a.window, a.sinks);
        top_shared = max(top_shared, fs.n);
      }
    }
    if (i < a.b.n_req) {
      q = facts(i);
      const int grp = group_of[i];
      if (grp >= 0) from = keys_of(grp, w.groups[grp]);
      w.from[i] = from;
      nb_own = ((uint32_t)q.n * g + qb_own - 1) / qb_own;
      uniform = nb_own <= 1;
      for (uint32_t b = 0; b < nb_own; ++b) {
        rs = span_of(b);
        top_own = max(top_own, rs.n);
        x.v[2] += ((int64_t)rs.n + extra_own) * heads;
      }
    }
    x.v[0] = (int64_t)nb_shared << 32 | nb_own;
    x.v[1] = ((int64_t)fs.n + extra) * heads * nb_shared;
    // before the barriers of the sums, after which the groups may be written
    const Scan3 at = block_scan3<T>(x, tmp, all);
    int64_t e = n_shared + (at.v[0] >> 32), o = n_own + (uint32_t)at.v[0];
    if (i < p.n_groups) {
      w.groups[i].n = f.n;
      w.groups[i].keys = f.keys;
      entry_shared[i] = (int)min(e, (int64_t)most_shared);
      for (uint32_t b = 0; b < nb_shared && e < most_shared; ++b, ++e) {
        w.shared.of[e] = i;
        w.shared.qblk[e] = b;
        w.shared.first[e] = base_shared + at.v[1] + (int64_t)b * (fs.n + extra) * heads;
      }
    }
    if (i < a.b.n_req) {
      entry_own[i] = (int)min(o, (int64_t)most_own);
      int64_t start = base_own + at.v[2];
      for (uint32_t b = 0; b < nb_own && o < most_own; ++b, ++o) {
        w.own.of[o] = i;
        w.own.qblk[o] = b;
        w.own.first[o] = start;
        start += ((int64_t)(uniform ? rs.n : span_of(b).n) + extra_own) * heads;
      }
    }
    n_shared += all.v[0] >> 32;
    n_own += (uint32_t)all.v[0];
    base_shared += all.v[1];
    base_own += all.v[2];
  }
  if (top_shared > 0) atomicMax(longest, top_shared);
  if (top_own > 0) atomicMax(longest + 1, top_own);
  if (tid == 0) {
    n_shared = min(n_shared, (int64_t)most_shared);
    n_own = min(n_own, (int64_t)most_own);
    w.shared.first[n_shared] = base_shared;
    w.own.first[n_own] = base_own;
    w.shared.n[0] = (int)n_shared;
    w.own.n[0] = (int)n_own;
  }
  __syncthreads();
  if (tid == 0) w.shared.n[1] = longest[0];
  if (tid == 0) w.own.n[1] = longest[1];
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
    // an entry past the last place is not there (starts that do not ascend can want more)
    auto there = [&](int e, int rows, int of, int most) { return e + (rows + of - 1) / of <= most; };
    if (t >= q.t0 && t < q.t0 + q.n && there(entry_own[lo], q.n * (int)g, qb_own, most_own)) {
      k.own = entry_own[lo];
      k.own_row = (t - q.t0) * (int)g;
      const int i = group_of[lo];
      if (i >= 0 && w.groups[i].keys > 0 && there(entry_shared[i], w.groups[i].n * (int)g, qb, most_shared)) {
        k.shared = entry_shared[i];
        k.shared_row = (t - w.groups[i].t0) * (int)g;
      }
    }
    put_token(t, k);
  }
  __syncthreads();
}
// What the plan starts from; a barrier follows.
template <int T>
__device__ __forceinline__ void clear_prefix_plan(const PrefixLaunch& p, const PrefixPlan& w, int* longest) {
  for (int i = threadIdx.x; i < p.n_groups; i += T) {
    w.groups[i] = PrefixGroup{INT32_MAX, INT32_MIN, INT32_MAX, INT32_MIN, 0, INT32_MAX};
    w.live[i] = 0;
  }
  if (threadIdx.x < 2) longest[threadIdx.x] = 0;
}

}  // namespace
}  // namespace dfs
