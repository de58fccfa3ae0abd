// kv8_prefix_kernel.hpp -- the kernel of kv8_prefix_attention, one head_dim a
// translation unit.
//
// What bounds it (head_dim 128, both launches).  Many rows a group: the vector units,
// by conversions of codes, exponentials and weights' halves, for 32 rows a wave (64
// requests of 4 heads a cached one behind 6007 tokens 45 us, 0.15 PFLOP/s; 24 requests
// of 5 behind 65500 tokens 94 us, 0.34 PFLOP/s: vector units 65 to 70% busy, matrix
// cores 40%, and as long where every page is the same, from a cache).  Few rows a
// group: memory (48 samples of 6 prompts 63 us, 4.0 TB/s).  Few requests: the chain of
// reads, plan, pages, codes, sums (four beams of 1561 tokens 18 us).
#pragma once

#include "kv8_prefix_plan.hpp"

namespace dfs {
namespace {

// The plan, where it is.
struct PrefixAt {
  const PrefixPlan* ws;
  const PrefixInline* lds;
  bool in;  // in LDS
};

// The items of one line; complete rows are sums of it.
template <typename B, bool SHARED>
struct Part : B {
  static constexpr bool kJoinHere = false;
  static constexpr int kEach = SHARED ? 0 : kPrefixEach, kKeep = 0;
  const PrefixAt& at_;
  const PrefixSums& sums;
  __device__ __forceinline__ Part(const KvAttnLaunch& a, const PrefixAt& p, const PrefixSums& s)
      : B(a), at_(p), sums(s) {}
  __device__ __forceinline__ const PrefixInline::Entries& lds() const {
    return SHARED ? at_.lds->line_shared : at_.lds->line_own;
  }
  __device__ __forceinline__ const PrefixEntries& far() const { return SHARED ? at_.ws->shared : at_.ws->own; }
  __device__ __forceinline__ int entries() const { return at_.in ? lds().n[0] : *gptr(far().n); }
  __device__ __forceinline__ int64_t first(int e) const { return at_.in ? lds().first[e] : *gptr(far().first + e); }
  __device__ __forceinline__ int longest() const { return uni(at_.in ? lds().n[1] : *gptr(far().n + 1)); }
  __device__ __forceinline__ int ready(int e, int kh) {
    const int i = uni(at_.in ? lds().of[e] : *gptr(far().of + e));
    const int qblk = uni(at_.in ? lds().qblk[e] : *gptr(far().qblk + e));
    if constexpr (SHARED) {
      const PrefixGroup f = at_.in ? at_.lds->groups[i] : at_.ws->groups[i];
      const int t0 = uni(f.t0), keys = uni(f.keys);
      B::template begin_by<true>(Req{t0, f.n, keys, keys}, uni(f.row), qblk, kh, 0, uni(f.p0), uni(f.p1),
                                 [&](int tok) { return at_.in ? at_.lds->pos[t0 + tok] : *gptr(at_.ws->pos + t0 + tok); });
    } else {
      B::begin(at_.in ? at_.lds->facts[i] : get_req(B::a.b, B::a.kv.page, i), i, qblk, kh,
               uni(at_.in ? at_.lds->from[i] : *gptr(at_.ws->from + i)));
    }
    return qblk;
  }
  __device__ __forceinline__ int64_t at(int row) const {
    const int g = B::a.q_heads / B::a.kv.heads;
    const int tok = row / g, h = B::kh * g + row - tok * g;
    return (int64_t)(B::rq.t0 + tok) * B::a.q_heads + h;
  }
  __device__ __forceinline__ void put(int64_t at, int d, const f4& v, float m, float l) const {
    *gptr_w((f4*)(sums.o + at * B::kD + d)) = v;
    if (d == 0) {  // as one whole number: see put2
      *gptr_w((uint64_t*)(sums.ml + at)) = (uint64_t)__float_as_uint(l) << 32 | __float_as_uint(m);
    }
  }
  __device__ __forceinline__ void put_nan(int64_t at, int d) const {
    *gptr_w(sums.o + at * B::kD + d) = __builtin_nanf("");
  }
};
__device__ __forceinline__ Line line_of(const PrefixSums& p) { return {nullptr, p.part_o, p.part_ml, nullptr}; }

// Short items, one a wave, where there are two for every workgroup: wave `at` of n takes
// items at, at + n, ... of the line; there is no barrier and nothing to join (48 samples
// of 500 own tokens 57.9 us, 63.4 with the waves of a workgroup at one item; 64 requests
// of 700 37.8, 41.8).
template <typename A>
__device__ __forceinline__ void run_lone(A& t, int n_entries, int at, int n) {
  const int heads = t.a.kv.heads;
  const int64_t items = (int64_t)n_entries * heads;
  for (int64_t x = at; x < items; x += n) {
    const int e = uni((int)((uint32_t)x / (uint32_t)heads)), kh = uni((int)x - e * heads);
    const int n_tiles = uni((int)((t.first(e + 1) - t.first(e)) / heads)) - A::kExtra;
    t.ready(e, kh);
    t.template tiles<false>(0, n_tiles, 1);
    const bool nans = A::kNan && t.any_nan();
    if (A::kNan && nans) {
      t.ready(e, kh);
      t.template tiles<true>(0, n_tiles, 1);
    }
    t.finish();
#pragma unroll
    for (int i = 0; i < A::kNq; ++i) {
      const int row = 16 * i + t.r16;
      if (row < t.nrows) {
        const int64_t at = t.at(t.row0 + row);
#pragma unroll
        for (int d = 0; d < A::kDims; ++d) t.put(at, d * 16 + t.q4 * 4, t.o[i][d], t.m[i], t.l[i]);
      }
    }
    if (A::kNan && nans)
      t.spread_nan(0, n_tiles, 1, [&](int i, int d) {
        const int row = 16 * i + t.r16;
        if (row < t.nrows) t.put_nan(t.at(t.row0 + row), d);
      });
  }
}

template <int KIND, int D, int NQ, bool SPLIT, int OWN, bool BIG>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2)
void prefix_kernel(PrefixLaunch p, PrefixWs ws, int slices, int in) {
  using P = Part<Attn<KIND, D, NQ, SPLIT, false, BIG>, true>;
  using S = Part<Attn<KIND, D, OWN, true, false, BIG>, false>;
  __shared__ union {
    typename P::Work p;
    typename S::Work s;
  } sh;
  __shared__ PrefixInline lds;
  const KvAttnLaunch& a = p.a;
  const PrefixAt at = {&ws.plan, &lds, in != 0};
  if (in) {
    const int tid = threadIdx.x;
    const PrefixPlan w = {lds.groups, lds.live, lds.from, lds.pos,
                          {lds.line_shared.first, lds.line_shared.of, lds.line_shared.qblk, lds.line_shared.n},
                          {lds.line_own.first, lds.line_own.of, lds.line_own.qblk, lds.line_own.n}};
    const int start = tid <= p.n_groups ? *gptr(p.group_start + tid) : 0;
    const int shared = tid < p.n_groups ? *gptr(p.shared + tid) : 0;
    if (tid < a.b.n_req) lds.facts[tid] = get_req(a.b, a.kv.page, tid);
    if (tid <= p.n_groups) lds.group_start[tid] = start;
    if (tid < p.n_groups) lds.shared[tid] = shared;
    clear_prefix_plan<kThreads>(p, w, lds.longest);
    __syncthreads();
    make_prefix_plan<kThreads>(
        p, w, [&](int r) { return lds.facts[r]; }, [&](int i) { return lds.group_start[i]; },
        [&](int i) { return lds.shared[i]; }, lds.group_of, lds.first_entry, lds.first_shared, ws.most_shared,
        ws.most_own, P::kQb, P::kExtra, S::kQb, S::kExtra,
        [&](int t, const PrefixToken& k) {
          if (blockIdx.x == 0) ws.tokens[t] = k;
        },
        lds.tmp, lds.longest);
    if (blockIdx.x == 0) {  // what the second kernel reads of it
      for (int i = tid; i <= lds.line_shared.n[0]; i += kThreads) ws.plan.shared.first[i] = lds.line_shared.first[i];
      for (int i = tid; i <= lds.line_own.n[0]; i += kThreads) ws.plan.own.first[i] = lds.line_own.first[i];
    }
  }
  auto length = [&](const PrefixInline::Entries& e, const PrefixEntries& f) {
    return in ? e.first[e.n[0]] : *gptr(f.first + *gptr(f.n));
  };
  const int n = shared_slices(length(lds.line_shared, ws.plan.shared), length(lds.line_own, ws.plan.own),
                              in ? lds.line_own.n[1] : *gptr(ws.plan.own.n + 1), SPLIT, slices);
  const int slice = blockIdx.x;
  if (slice == 0 && threadIdx.x < 2) {  // for the second kernel
    const bool own = threadIdx.x != 0;
    const int64_t total = own ? length(lds.line_own, ws.plan.own) : length(lds.line_shared, ws.plan.shared);
    const int longest = own ? (in ? lds.line_own.n[1] : *gptr(ws.plan.own.n + 1)) : INT32_MAX;
    const int of = max(own ? slices - n : n, 1);
    ws.slices[threadIdx.x] = {max((int64_t)(own || SPLIT ? kWaves : 1), (total + of - 1) / of),
                              longest <= kPrefixEach, 0};
  }
  if (slice < n) {
    P t(a, at, ws.shared);
    run_line(t, sh.p, line_of(ws.shared), t.entries(), SPLIT ? kWaves : 1, slice, n);
  } else {
    S t(a, at, ws.own);
    const int entries = t.entries(), longest = t.longest();
    const int64_t items = (int64_t)entries * a.kv.heads;
    if (longest <= kPrefixEach && items >= 2 * (slices - n))
      run_lone(t, entries, slice - n + t.wave * (slices - n), (slices - n) * kWaves);
    else
      run_line(t, sh.s, line_of(ws.own), entries, kWaves, slice - n, slices - n);
  }
}

template <int KIND, int D, int NQ, bool SPLIT, int OWN>
void go(const PrefixLaunch& p, const PrefixWs& w, const PrefixCut& c, hipStream_t s) {
  if (p.a.kv.page >= kTile)
    hipLaunchKernelGGL((prefix_kernel<KIND, D, NQ, SPLIT, OWN, true>), dim3(c.slices), dim3(kThreads), 0,
                       s, p, w, c.slices, c.in);
  else
    hipLaunchKernelGGL((prefix_kernel<KIND, D, NQ, SPLIT, OWN, false>), dim3(c.slices), dim3(kThreads), 0,
                       s, p, w, c.slices, c.in);
}
template <int KIND, int D>
void go_cut(const PrefixLaunch& p, const PrefixWs& w, const PrefixCut& c, hipStream_t s) {
  if (!c.split) {
    if (c.nq_own == 1) go<KIND, D, 2, false, 1>(p, w, c, s);
    else go<KIND, D, 2, false, 2>(p, w, c, s);
  } else if (c.nq == 1) {
    go<KIND, D, 1, true, 1>(p, w, c, s);
  } else {
    if (c.nq_own == 1) go<KIND, D, 2, true, 1>(p, w, c, s);
    else go<KIND, D, 2, true, 2>(p, w, c, s);
  }
}

}  // namespace

template <int D>
void launch_prefix(const PrefixLaunch& p, const PrefixWs& w, const PrefixCut& c, hipStream_t s) {
  if (p.a.kv.dtype == DFS_FP8) go_cut<DFS_FP8, D>(p, w, c, s);
  else go_cut<DFS_INT8, D>(p, w, c, s);
}

}  // namespace dfs
