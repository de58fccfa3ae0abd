// kv8_prefix_attention.hip -- attention over the 8-bit paged cache where the
// requests of a group share their first tokens: plan, and the joining of the
// shared keys' part of each row with its own keys' part,
//   o = (o_s 2^(m_s - m) + o_r 2^(m_r - m)) / (l_s 2^(m_s - m) + l_r 2^(m_r - m)),
// m the larger of m_s and m_r.
#include "kv8_attn.hpp"
#include "kv8_prefix.hpp"

namespace dfs {
namespace {

constexpr int kPlanThreads = 1024;

// The group of request r, or -1.
__device__ __forceinline__ int group_of(const PrefixLaunch& p, int r) {
  int lo = 0, hi = p.n_groups;  // the last group that starts at or before r, if any does
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (*gptr(p.group_start + mid) <= r) lo = mid;
    else hi = mid;
  }
  return *gptr(p.group_start + lo) <= r && r < *gptr(p.group_start + lo + 1) ? lo : -1;
}

// Entries of one line in order, and where each starts: blocks(i) blocks of rows
// of group or request i, tiles(i, block) tiles each, `extra` counted beside them.
template <typename B, typename T>
__device__ __forceinline__ void plan_line(const PrefixLine& w, int n, int heads, int extra, B blocks, T tiles,
                                          int64_t* tmp, int* longest) {
  int n_entries = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + (int)threadIdx.x;
    const int nb = i < n ? min(blocks(i), w.most) : 0;
    int64_t total;
    const int64_t at = n_entries + block_scan<int64_t>(nb, tmp, &total, kPlanThreads);
    for (int b = 0; b < nb && at + b < w.most; ++b) {
      w.of[at + b] = i;
      w.qblk[at + b] = b;
    }
    n_entries = (int)min(n_entries + total, (int64_t)w.most);
  }
  if (threadIdx.x == 0) *longest = 0;
  __syncthreads();
  int64_t base = 0;
  int most = 0;
  for (int e0 = 0; e0 < n_entries; e0 += kPlanThreads) {
    const int e = e0 + (int)threadIdx.x;
    int64_t t = 0;
    if (e < n_entries) {
      const int m = tiles(w.of[e], w.qblk[e]);
      most = max(most, m);
      t = ((int64_t)m + extra) * heads;
    }
    int64_t total;
    const int64_t at = base + block_scan<int64_t>(t, tmp, &total, kPlanThreads);
    if (e < n_entries) w.first[e] = at;
    base += total;
  }
  if (most > 0) atomicMax(longest, most);
  __syncthreads();
  if (threadIdx.x == 0) {
    w.first[n_entries] = base;
    w.n[0] = n_entries;
    w.n[1] = *longest;
  }
  __syncthreads();
}

// Tokens that group i shares, as far as the table goes.
__device__ __forceinline__ int shared_of(const PrefixLaunch& p, int i) {
  return (int)min((int64_t)max(*gptr(p.shared + i), 0), (int64_t)p.a.b.table_pages * p.a.kv.page);
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PrefixLaunch p, PrefixWs ws, int qb, int extra,
                                                            int qb_own, int extra_own) {
  __shared__ int64_t tmp[kPlanThreads / kWave];
  __shared__ int longest;
  const KvAttnLaunch& a = p.a;
  const int tid = threadIdx.x, g = a.q_heads / a.kv.heads;
  for (int i = tid; i < p.n_groups; i += kPlanThreads) {
    const int r = min(max(*gptr(p.group_start + i), 0), max(a.b.n_req - 1, 0));
    ws.groups[i] = {INT32_MAX, INT32_MIN, INT32_MAX, INT32_MIN, 0, r};
    ws.live[i] = 0;
  }
  __syncthreads();
  for (int r = tid; r < a.b.n_req; r += kPlanThreads) {
    const Req q = get_req(a.b, a.kv.page, r);
    int i = group_of(p, r);
    if (i >= 0 && q.len < shared_of(p, i)) i = -1;  // it stands alone
    ws.group_of[r] = i;
    if (i < 0 || q.n <= 0) continue;
    PrefixGroup* f = ws.groups + i;
    atomicMin(&f->t0, q.t0);
    atomicMax(&f->n, q.t0 + q.n);  // their end, for now
    atomicMin(&f->p0, q.len - q.n);
    atomicMax(&f->p1, q.len - 1);
    atomicAdd(ws.live + i, 1);
  }
  for (int t = tid; t < a.b.n_tok; t += kPlanThreads) {
    // the request of token t
    int lo = 0, hi = a.b.n_req;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (*gptr(a.b.tok_start + mid) <= t) lo = mid;
      else hi = mid;
    }
    const Req q = get_req(a.b, a.kv.page, lo);
    ws.pos[t] = q.len - q.n + (t - q.t0);
  }
  __syncthreads();
  for (int i = tid; i < p.n_groups; i += kPlanThreads) {
    PrefixGroup f = ws.groups[i];
    f.keys = shared_of(p, i) / kTile * kTile;
    // worth it for two requests that see some of it
    if (ws.live[i] < 2) f.keys = 0;
    else f.n -= f.t0;  // with the tokens between of requests that stand alone, whose sums nobody takes
    if (f.keys > 0) {
      const int hi = min(f.p1, f.keys - 1), lo = a.window > 0 && f.p0 >= a.window ? f.p0 - a.window + 1 : 0;
      if (hi < 0 || (hi < lo && a.sinks <= 0)) f.keys = 0;
    }
    ws.groups[i] = f;
  }
  __syncthreads();
  plan_line(
      ws.shared, p.n_groups, a.kv.heads, extra,
      [&](int i) {
        const PrefixGroup& f = ws.groups[i];
        return f.keys > 0 ? (int)(((int64_t)f.n * g + qb - 1) / qb) : 0;
      },
      [&](int i, int) {
        const PrefixGroup& f = ws.groups[i];
        return get_span(Req{f.t0, f.n, f.keys, f.keys}, f.p0, f.p1, a.window, a.sinks).n;
      },
      tmp, &longest);
  plan_line(
      ws.own, a.b.n_req, a.kv.heads, extra_own,
      [&](int r) { return (int)(((int64_t)get_req(a.b, a.kv.page, r).n * g + qb_own - 1) / qb_own); },
      [&](int r, int b) {
        const Req q = get_req(a.b, a.kv.page, r);
        const int grp = ws.group_of[r], from = grp < 0 ? 0 : ws.groups[grp].keys;
        const int i0 = (int)((int64_t)b * qb_own / g);
        const int i1 = (int)min(((int64_t)(b + 1) * qb_own - 1) / g, (int64_t)q.n - 1);
        return get_span(q, q.len - q.n + i0, q.len - q.n + i1, a.window, a.sinks, from).n;
      },
      tmp, &longest);
}

// Row by row: the shared keys' sums and the own keys'.
template <typename T>
__global__ __launch_bounds__(256) void merge_kernel(KvAttnLaunch a, PrefixWs ws, int wide) {
  const int D = a.kv.head_dim, quads = D / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / quads;
  const int d = (int)(i % quads) * 4;
  const int tok = (int)(row / a.q_heads), h = (int)(row % a.q_heads);
  // rows of no request are left as they are
  const int t0 = min(max(*gptr(a.b.tok_start), 0), a.b.n_tok), t1 = min(*gptr(a.b.tok_start + a.b.n_req), a.b.n_tok);
  if (tok < t0 || tok >= t1) return;
  int lo = 0, hi = a.b.n_req;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (*gptr(a.b.tok_start + mid) <= tok) lo = mid;
    else hi = mid;
  }
  const int grp = *gptr(ws.group_of + lo);
  f4 v = *gptr((const f4*)(ws.own.sum_o + row * D + d));
  f2 w = *gptr(ws.own.sum_ml + row);
  if (grp >= 0 && *gptr(&ws.groups[grp].keys) > 0) {
    const f4 x = *gptr((const f4*)(ws.shared.sum_o + row * D + d));
    const f2 y = *gptr(ws.shared.sum_ml + row);
    const float m = fmaxf(w.x, y.x);
    const float fw = __builtin_amdgcn_exp2f(w.x - m), fy = __builtin_amdgcn_exp2f(y.x - m);
    v = v * fw + x * fy;
    w.y = w.y * fw + y.y * fy;
  }
  // rows that see nothing are 0; a sum that is NaN stays so
  const float inv = w.y == 0.0f ? 0.0f : 1.0f / w.y;
  typedef T T4 __attribute__((ext_vector_type(4)));
  const T4 r = {(T)(v[0] * inv), (T)(v[1] * inv), (T)(v[2] * inv), (T)(v[3] * inv)};
  T* out = (T*)a.O + tok * a.ldo + (int64_t)h * D + d;
  if (wide) {
    *gptr_w((T4*)out) = r;
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) *gptr_w(out + c) = r[c];
  }
}

bool shares(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads, int32_t n_groups) {
  return n_groups > 0 && (int64_t)n_tok * (q_heads / kv.heads) <= (int64_t)kPrefixRows * n_req;
}
PrefixCut get_cut(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads, int32_t n_groups) {
  PrefixCut c;
  const int64_t rows = (int64_t)n_tok * (q_heads / kv.heads);
  c.nq_own = rows <= 16 * (int64_t)n_req ? 1 : 2;
  c.split = rows <= 32 * (int64_t)n_groups;
  c.nq = c.split && rows <= 16 * (int64_t)n_groups && c.nq_own == 1 ? 1 : 2;
  c.qb = c.split ? 16 * c.nq : 16 * c.nq * kWaves;
  c.slices = kv.head_dim == 256 ? 256 : 512;  // as many workgroups as the device holds at once
  return c;
}
size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Places of the workspace's arrays; at: its next free byte.
struct Places {
  char* base;
  size_t at;
  template <typename T>
  T* take(int64_t n) {
    T* p = (T*)(base + at);
    at += up((size_t)n * sizeof(T));
    return p;
  }
};
// `most` entries, `qb` rows an item, `rows` rows in all.
void place_line(Places& p, PrefixLine& w, int64_t most, int qb, int64_t rows, int slices, int D) {
  w.first = p.take<int64_t>(most + 1);
  w.of = p.take<int32_t>(most);
  w.qblk = p.take<int32_t>(most);
  w.n = p.take<int32_t>(2);
  w.most = (int32_t)most;
  w.part_ml = p.take<f2>(2 * (int64_t)slices * qb);
  w.group_ml = p.take<f2>(2 * (int64_t)slices * qb);
  w.part_o = p.take<float>(2 * (int64_t)slices * qb * D);
  w.sum_ml = p.take<f2>(rows);
  w.sum_o = p.take<float>(rows * D);
}
struct Sizes {
  int64_t n_req, n_groups, n_tok, entries, entries_own;
  int qb, qb_own, slices;
};
size_t place(char* base, const dfs_kv8& kv, int32_t q_heads, const Sizes& s, PrefixWs* w) {
  Places p = {base, kCounterBytes};
  w->groups = p.take<PrefixGroup>(s.n_groups);
  w->live = p.take<int32_t>(s.n_groups);
  w->group_of = p.take<int32_t>(s.n_req);
  w->pos = p.take<int32_t>(s.n_tok);
  const int64_t rows = s.n_tok * q_heads;
  place_line(p, w->shared, s.entries, s.qb, rows, s.slices, kv.head_dim);
  place_line(p, w->own, s.entries_own, s.qb_own, rows, s.slices, kv.head_dim);
  w->shared.count = (uint32_t*)base;
  w->own.count = (uint32_t*)base + 3 * s.slices;
  return p.at;
}
Sizes get_sizes(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads, int32_t n_groups,
                const PrefixCut& c) {
  const int64_t rows = (int64_t)n_tok * (q_heads / kv.heads);
  const int qb_own = 16 * c.nq_own;
  return {n_req,
          n_groups,
          n_tok,
          std::min(n_groups, n_tok) + rows / c.qb,
          std::min(n_req, n_tok) + rows / qb_own,
          c.qb,
          qb_own,
          c.slices};
}

}  // namespace

size_t kv8_prefix_ws_need(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads, int32_t n_groups) {
  if (!shares(kv, n_req, n_tok, q_heads, n_groups)) return kv8_attention_ws_need(kv, n_req, n_tok, q_heads);
  PrefixWs w;
  return place(nullptr, kv, q_heads,
               get_sizes(kv, n_req, n_tok, q_heads, n_groups, get_cut(kv, n_req, n_tok, q_heads, n_groups)), &w);
}

// Enough for every call of up to n_req requests and n_tok tokens, whatever its
// groups: those that share have at most kPrefixRows rows a request, n_req groups,
// and an entry for each group or request and each full block of its rows.
size_t kv8_prefix_ws_bytes(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads) {
  const int64_t g = q_heads / kv.heads;
  const int64_t tok = std::min<int64_t>(n_tok, (int64_t)kPrefixRows * n_req / g);
  const int64_t most = std::min<int64_t>(n_req, tok) + tok * g / 16;
  PrefixWs w;
  const Sizes s = {n_req, n_req, tok, most, most, 32 * kWaves, 32, kv.head_dim == 256 ? 256 : 512};
  return std::max(place(nullptr, kv, q_heads, s, &w), kv8_attention_ws_bytes(kv, n_req, n_tok, q_heads));
}

hipError_t launch_kv8_prefix_attention(const KvAttnLaunch& a, int32_t n_groups, const int32_t* group_start,
                                       const int32_t* shared, void* ws, hipStream_t s) {
  if (!shares(a.kv, a.b.n_req, a.b.n_tok, a.q_heads, n_groups)) return launch_kv8_attention(a, ws, s);
  const PrefixLaunch p = {a, n_groups, group_start, shared};
  const PrefixCut c = get_cut(a.kv, a.b.n_req, a.b.n_tok, a.q_heads, n_groups);
  PrefixWs w;
  place((char*)ws, a.kv, a.q_heads, get_sizes(a.kv, a.b.n_req, a.b.n_tok, a.q_heads, n_groups, c), &w);
  using Split = Attn<DFS_INT8, 64, 1, true, false, false>;
  using Each = Attn<DFS_INT8, 64, 2, false, false, false>;
  hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, w, c.qb,
                     c.split ? Split::kExtra : Each::kExtra, 16 * c.nq_own, Split::kExtra);
  if (a.kv.head_dim == 64) launch_prefix<64>(p, w, c, s);
  else if (a.kv.head_dim == 96) launch_prefix<96>(p, w, c, s);
  else if (a.kv.head_dim == 128) launch_prefix<128>(p, w, c, s);
  else launch_prefix<256>(p, w, c, s);
  const int wide = (uintptr_t)a.O % (a.odt == DFS_F32 ? 16 : 8) == 0 && a.ldo % 4 == 0;
  const int64_t quads = (int64_t)a.b.n_tok * a.q_heads * (a.kv.head_dim / 4);
  const dim3 grid((unsigned)((quads + 255) / 256));
  if (a.odt == DFS_F32) hipLaunchKernelGGL(merge_kernel<float>, grid, dim3(256), 0, s, a, w, wide);
  else hipLaunchKernelGGL(merge_kernel<_Float16>, grid, dim3(256), 0, s, a, w, wide);
  return hipGetLastError();
}

}  // namespace dfs
