// kv8_prefix_attention.hip -- attention over the 8-bit paged cache where the
// requests of a group share their first tokens: plan, and the joining of the
// shared keys' part of each row with its own keys' part,
//   o = (o_s 2^(m_s - m) + o_r 2^(m_r - m)) / (l_s 2^(m_s - m) + l_r 2^(m_r - m)),
// m the larger of m_s and m_r.
#include "kv8_prefix_plan.hpp"

namespace dfs {
namespace {

constexpr int kPlanThreads = 512;

// The plan of a batch that is too large for every workgroup to make its own.  Up
// to kPlanNear requests what it looks up again and again is in LDS.
constexpr int kPlanNear = 1024;
struct PlanNear {
  Req facts[kPlanNear];
  PrefixGroup groups[kPlanNear];
  int32_t group_start[kPlanNear + 1], shared[kPlanNear], live[kPlanNear];
  int32_t group_of[kPlanNear], first_entry[kPlanNear], first_shared[kPlanNear];
};

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PrefixLaunch p, PrefixWs ws, int32_t* scratch, int qb,
                                                            int extra, int qb_own, int extra_own) {
  __shared__ Scan3 tmp[kPlanThreads / kWave];
  __shared__ int longest[2];
  __shared__ PlanNear lds;
  const int n = p.a.b.n_req, tid = threadIdx.x;
  auto put = [&](int t, const PrefixToken& k) { ws.tokens[t] = k; };
  if (n <= kPlanNear) {  // n_groups <= n_req
    PrefixPlan w = ws.plan;
    w.groups = lds.groups;
    w.live = lds.live;
    for (int i = tid; i <= p.n_groups; i += kPlanThreads) lds.group_start[i] = *gptr(p.group_start + i);
    for (int i = tid; i < p.n_groups; i += kPlanThreads) lds.shared[i] = *gptr(p.shared + i);
    for (int i = tid; i < n; i += kPlanThreads) lds.facts[i] = get_req(p.a.b, p.a.kv.page, i);
    clear_prefix_plan<kPlanThreads>(p, w, longest);
    __syncthreads();
    make_prefix_plan<kPlanThreads>(
        p, w, [&](int r) { return lds.facts[r]; }, [&](int i) { return lds.group_start[i]; },
        [&](int i) { return lds.shared[i]; }, lds.group_of, lds.first_entry, lds.first_shared, ws.most_shared,
        ws.most_own, qb, extra, qb_own, extra_own, put, tmp, longest);
    for (int i = tid; i < p.n_groups; i += kPlanThreads) ws.plan.groups[i] = lds.groups[i];
    return;
  }
  clear_prefix_plan<kPlanThreads>(p, ws.plan, longest);
  __syncthreads();
  make_prefix_plan<kPlanThreads>(
      p, ws.plan, [&](int r) { return get_req(p.a.b, p.a.kv.page, r); },
      [&](int i) { return *gptr(p.group_start + i); }, [&](int i) { return *gptr(p.shared + i); }, scratch,
      scratch + n, scratch + 2 * n, ws.most_shared, ws.most_own, qb, extra, qb_own, extra_own, put, tmp, longest);
}

// What the second kernel knows of a line.
struct LineCut {
  const int64_t* first;
  PrefixSums sums;
  int qb, extra;
};

// What one line gives for row `row` (counted from its entry's first one) of kv head
// kh: m, l and four sums at dim d.  The parts of a split item are read by the
// waves in turn, part u by wave u % kWaves: each returns its own share.
__device__ __forceinline__ void line_sums(const LineCut& c, const PrefixSlices& cut, int first_entry, int row, int kh,
                                          int heads, int64_t at, int D, int d, int wave, float& m, float& l, f4& v) {
  const int e = first_entry + row / c.qb, r = row % c.qb;
  const int64_t f0 = *gptr(c.first + e), f1 = *gptr(c.first + e + 1);
  const int64_t line = (f1 - f0) / heads, item0 = f0 + kh * line, item1 = item0 + line - c.extra;
  const int w0 = (int)(item0 / cut.per), w1 = (int)((item1 - 1) / cut.per);
  m = -1e30f;
  l = 0.0f;
  v = f4{0, 0, 0, 0};
  if (cut.whole || w0 == w1) {
    if (wave == 0) {
      const f2 w = *gptr(c.sums.ml + at);
      m = w.x;
      l = w.y;
      v = *gptr((const f4*)(c.sums.o + at * D + d));
    }
    return;
  }
  constexpr int kAhead = 4;
#pragma unroll 1
  for (int u = w0 + wave; u <= w1; u += kAhead * kWaves) {
    f2 pm[kAhead];
    f4 po[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int w = min(u + i * kWaves, w1);
      // the item is the last one of its first slice, and the first of the others
      const int64_t pr = (2 * (int64_t)w + (w == w0)) * c.qb + r;
      pm[i] = *gptr(c.sums.part_ml + pr);
      po[i] = *gptr((const f4*)(c.sums.part_o + pr * D + d));
    }
    float mb = m;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) mb = fmaxf(mb, pm[i].x);
    const float old = __builtin_amdgcn_exp2f(m - mb);
    l *= old;
    v *= old;
    m = mb;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float f = u + i * kWaves <= w1 ? __builtin_amdgcn_exp2f(pm[i].x - mb) : 0.0f;
      l += pm[i].y * f;
      v += po[i] * f;
    }
  }
}

// The rows of one token, 64 places of four dims a workgroup: the sums of both
// lines, each wave's share, joined in the waves' order.
template <typename T>
__global__ __launch_bounds__(kThreads) void merge_kernel(KvAttnLaunch a, const PrefixToken* tokens,
                                                         const PrefixSlices* slices, LineCut shared, LineCut own,
                                                         int wide) {
  __shared__ f2 ml[kWaves][kWave];
  __shared__ f4 sum[kWaves][kWave];
  const int D = a.kv.head_dim, quads = D / 4, g = a.q_heads / a.kv.heads;
  const int lane = threadIdx.x % kWave, wave = uni(threadIdx.x / kWave), tok = blockIdx.x;
  const PrefixToken k = tokens[tok];
  const PrefixSlices cut_shared = slices[0], cut_own = slices[1];
  if (k.own < 0) return;  // of no request: left as it is
  const int place = blockIdx.y * kWave + lane;
  const bool real = place < a.q_heads * quads;
  const int h = real ? place / quads : 0, d = real ? place % quads * 4 : 0, kh = h / g;
  const int64_t at = (int64_t)tok * a.q_heads + h;
  float m, l;
  f4 v;
  line_sums(own, cut_own, k.own, k.own_row + h - kh * g, kh, a.kv.heads, at, D, d, wave, m, l, v);
  if (k.shared >= 0) {
    float y, z;
    f4 x;
    line_sums(shared, cut_shared, k.shared, k.shared_row + h - kh * g, kh, a.kv.heads, at, D, d, wave, y, z, x);
    const float top = fmaxf(m, y);
    const float fm = __builtin_amdgcn_exp2f(m - top), fy = __builtin_amdgcn_exp2f(y - top);
    l = l * fm + z * fy;
    v = v * fm + x * fy;
    m = top;
  }
  ml[wave][lane] = f2{m, l};
  sum[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || !real) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, ml[w][lane].x);
  l = 0.0f;
  v = f4{0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float f = __builtin_amdgcn_exp2f(ml[w][lane].x - m);
    l += ml[w][lane].y * f;
    v += sum[w][lane] * f;
  }
  // rows that see nothing are 0; a sum that is NaN stays so
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
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
  const int64_t rows = (int64_t)n_tok * (q_heads / kv.heads), n = n_req;
  return n_groups > 0 && (rows <= kPrefixRowsFew * n || (rows > kPrefixRowsWave * n && rows <= kPrefixRows * n));
}
int64_t most_entries(int32_t n, int32_t n_tok, int64_t rows, int qb) { return std::min(n, n_tok) + rows / qb; }
PrefixCut get_cut(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads, int32_t n_groups) {
  PrefixCut c;
  const int64_t rows = (int64_t)n_tok * (q_heads / kv.heads);
  c.nq_own = rows <= 16 * (int64_t)n_req ? 1 : 2;
  // Up to 64 rows a group the waves take the tiles in turn: 16 requests of 3 tokens
  // with 48 rows to a group of heads of 64 dims 40 us, 48 where each wave has rows of its
  // own; a document asked by 24 requests 64 us with 60 rows, and with 65 rows 71 in rows of
  // their own.
  c.split = rows <= 64 * (int64_t)n_groups;
  c.nq = c.split && rows <= 16 * (int64_t)n_groups && c.nq_own == 1 ? 1 : 2;
  c.qb = c.split ? 16 * c.nq : 16 * c.nq * kWaves;
  c.slices = kv.head_dim == 256 ? 256 : 512;  // as many workgroups as the device holds at once
  c.in = n_req <= kPrefixInline && n_tok <= kPrefixInlineTokens &&
         most_entries(n_groups, n_tok, rows, c.qb) <= kPrefixInlineEntries &&
         most_entries(n_req, n_tok, rows, 16 * c.nq_own) <= kPrefixInlineEntries;
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
void place_entries(Places& p, PrefixEntries& e, int64_t most) {
  e.first = p.take<int64_t>(most + 1);
  e.of = p.take<int32_t>(most);
  e.qblk = p.take<int32_t>(most);
  e.n = p.take<int32_t>(2);
}
void place_sums(Places& p, PrefixSums& s, int qb, int64_t rows, int slices, int D) {
  s.part_ml = p.take<f2>(2 * (int64_t)slices * qb);
  s.part_o = p.take<float>(2 * (int64_t)slices * qb * D);
  s.ml = p.take<f2>(rows);
  s.o = p.take<float>(rows * D);
}
struct Sizes {
  int64_t n_req, n_groups, n_tok, most_shared, most_own;
  int qb, qb_own, slices;
};
size_t place(char* base, const dfs_kv8& kv, int32_t q_heads, const Sizes& s, PrefixWs* w, int32_t** scratch) {
  Places p = {base, kCounterBytes};
  w->plan.groups = p.take<PrefixGroup>(s.n_groups);
  w->plan.live = p.take<int32_t>(s.n_groups);
  w->plan.from = p.take<int32_t>(s.n_req);
  w->plan.pos = p.take<int32_t>(s.n_tok);
  *scratch = p.take<int32_t>(2 * s.n_req + s.n_groups);
  w->tokens = p.take<PrefixToken>(s.n_tok);
  w->slices = p.take<PrefixSlices>(2);
  place_entries(p, w->plan.shared, s.most_shared);
  place_entries(p, w->plan.own, s.most_own);
  const int64_t rows = s.n_tok * q_heads;
  place_sums(p, w->shared, s.qb, rows, s.slices, kv.head_dim);
  place_sums(p, w->own, s.qb_own, rows, s.slices, kv.head_dim);
  w->most_shared = (int32_t)s.most_shared;
  w->most_own = (int32_t)s.most_own;
  return p.at;
}
Sizes get_sizes(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads, int32_t n_groups,
                const PrefixCut& c) {
  const int64_t rows = (int64_t)n_tok * (q_heads / kv.heads);
  const int qb_own = 16 * c.nq_own;
  return {n_req, n_groups, n_tok, most_entries(n_groups, n_tok, rows, c.qb), most_entries(n_req, n_tok, rows, qb_own),
          c.qb,  qb_own,   c.slices};
}

}  // namespace

size_t kv8_prefix_ws_need(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads, int32_t n_groups) {
  if (!shares(kv, n_req, n_tok, q_heads, n_groups)) return kv8_attention_ws_need(kv, n_req, n_tok, q_heads);
  PrefixWs w;
  int32_t* scratch;
  return place(nullptr, kv, q_heads,
               get_sizes(kv, n_req, n_tok, q_heads, n_groups, get_cut(kv, n_req, n_tok, q_heads, n_groups)), &w,
               &scratch);
}

// Enough for every call of up to n_req requests and n_tok tokens, whatever its
// groups: those that share have at most kPrefixRows rows a request, n_req groups,
// and an entry for each group or request and each full block of its rows.
size_t kv8_prefix_ws_bytes(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads) {
  const int64_t g = q_heads / kv.heads;
  const int64_t tok = std::min<int64_t>(n_tok, (int64_t)kPrefixRows * n_req / g);
  const int64_t most = std::min<int64_t>(n_req, tok) + tok * g / 16;
  PrefixWs w;
  int32_t* scratch;
  const Sizes s = {n_req, n_req, tok, most, most, 32 * kWaves, 32, kv.head_dim == 256 ? 256 : 512};
  return std::max(place(nullptr, kv, q_heads, s, &w, &scratch), kv8_attention_ws_bytes(kv, n_req, n_tok, q_heads));
}

hipError_t launch_kv8_prefix_attention(const KvAttnLaunch& a, int32_t n_groups, const int32_t* group_start,
                                       const int32_t* shared, void* ws, hipStream_t s) {
  if (!shares(a.kv, a.b.n_req, a.b.n_tok, a.q_heads, n_groups)) return launch_kv8_attention(a, ws, s);
  const PrefixLaunch p = {a, n_groups, group_start, shared};
  const PrefixCut c = get_cut(a.kv, a.b.n_req, a.b.n_tok, a.q_heads, n_groups);
  PrefixWs w;
  int32_t* scratch;
  place((char*)ws, a.kv, a.q_heads, get_sizes(a.kv, a.b.n_req, a.b.n_tok, a.q_heads, n_groups, c), &w, &scratch);
  using Turns = Attn<DFS_INT8, 64, 1, true, false, false>;
  using Alone = Attn<DFS_INT8, 64, 2, false, false, false>;
  const int extra = c.split ? Turns::kExtra : Alone::kExtra;
  if (!c.in)
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, w, scratch, c.qb, extra, 16 * c.nq_own,
                       Turns::kExtra);
  if (a.kv.head_dim == 64) launch_prefix<64>(p, w, c, s);
  else if (a.kv.head_dim == 96) launch_prefix<96>(p, w, c, s);
  else if (a.kv.head_dim == 128) launch_prefix<128>(p, w, c, s);
  else launch_prefix<256>(p, w, c, s);
  const LineCut shared_cut = {w.plan.shared.first, w.shared, c.qb, extra};
  const LineCut own_cut = {w.plan.own.first, w.own, 16 * c.nq_own, Turns::kExtra};
  const int wide = (uintptr_t)a.O % (a.odt == DFS_F32 ? 16 : 8) == 0 && a.ldo % 4 == 0;
  const dim3 grid(a.b.n_tok, (a.q_heads * (a.kv.head_dim / 4) + kWave - 1) / kWave);
  if (a.odt == DFS_F32)
    hipLaunchKernelGGL(merge_kernel<float>, grid, dim3(kThreads), 0, s, a, w.tokens, w.slices, shared_cut, own_cut,
                       wide);
  else
    hipLaunchKernelGGL(merge_kernel<_Float16>, grid, dim3(kThreads), 0, s, a, w.tokens, w.slices, shared_cut, own_cut,
                       wide);
  return hipGetLastError();
}

}  // namespace dfs
