// kv8_prefix_kernel.hpp -- the kernel of kv8_prefix_attention, one head_dim a
// translation unit.
#pragma once

#include "kv8_attn.hpp"
#include "kv8_prefix.hpp"

namespace dfs {
namespace {

// Complete sums of a line.
template <typename A>
struct Sums {
  const A& t;
  float* o;
  f2* ml;
  __device__ __forceinline__ int64_t at(int row) const {
    const int g = t.a.q_heads / t.a.kv.heads;
    const int tok = row / g, h = t.kh * g + row - tok * g;
    return (int64_t)(t.rq.t0 + tok) * t.a.q_heads + h;
  }
  __device__ __forceinline__ void put(int64_t at, int d, const f4& v, f2 w) const {
    *gptr_w((f4*)(o + at * A::kD + d)) = v;
    if (d == 0) *gptr_w(ml + at) = w;
  }
  __device__ __forceinline__ void put_nan(int64_t at, int d) const {
    *gptr_w(o + at * A::kD + d) = __builtin_nanf("");
  }
};
__device__ __forceinline__ Line line_of(const PrefixLine& p) {
  return {p.count, p.part_o, p.part_ml, p.group_ml};
}

template <int KIND, int D, int NQ, bool SPLIT, int OWN, bool BIG>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2)
void prefix_kernel(KvAttnLaunch a, PrefixWs ws, int slices) {
  using P = Attn<KIND, D, NQ, SPLIT, false, BIG>;
  using S = Attn<KIND, D, OWN, true, false, BIG>;
  __shared__ union {
    typename P::Work p;
    typename S::Work s;
  } sh;
  const int g = a.q_heads / a.kv.heads;
  {
    P t(a);
    const PrefixLine& w = ws.shared;
    run_line(
        t, sh.p, line_of(w), *gptr(w.n), [&](int e) { return *gptr(w.first + e); },
        [&] { return uni(*gptr(w.n + 1)); },
        [&](int e, int kh) {
          const int i = uni(*gptr(w.of + e)), qblk = uni(*gptr(w.qblk + e));
          const PrefixGroup* f = ws.groups + i;
          const int t0 = uni(*gptr(&f->t0)), keys = uni(*gptr(&f->keys));
          const Req q = {t0, uni(*gptr(&f->n)), keys, keys};
          const Span s = get_span(q, uni(*gptr(&f->p0)), uni(*gptr(&f->p1)), a.window, a.sinks);
          t.template begin<true>(q, s, uni(*gptr(&f->row)), qblk, kh,
                                 [&](int tok) { return *gptr(ws.pos + t0 + tok); });
          return qblk;
        },
        Sums<P>{t, w.sum_o, w.sum_ml}, SPLIT ? kWaves : 1, (int)blockIdx.x, slices);
  }
  __syncthreads();
  {
    S t(a);
    const PrefixLine& w = ws.own;
    run_line(
        t, sh.s, line_of(w), *gptr(w.n), [&](int e) { return *gptr(w.first + e); },
        [&] { return uni(*gptr(w.n + 1)); },
        [&](int e, int kh) {
          const int req = uni(*gptr(w.of + e)), qblk = uni(*gptr(w.qblk + e));
          const int grp = uni(*gptr(ws.group_of + req));
          const int from = grp < 0 ? 0 : uni(*gptr(&ws.groups[grp].keys));
          const Req f = get_req(a.b, a.kv.page, req);
          const Req q = {uni(f.t0), uni(f.n), uni(f.len), uni(f.keys)};
          const int pos0 = q.len - q.n, i0 = qblk * S::kQb, i1 = min(i0 + S::kQb, q.n * g);
          const Span s = get_span(q, pos0 + i0 / g, pos0 + (i1 - 1) / g, a.window, a.sinks, from);
          t.template begin<false>(q, s, req, qblk, kh, [&](int tok) { return pos0 + tok; });
          return qblk;
        },
        Sums<S>{t, w.sum_o, w.sum_ml}, kWaves, (int)blockIdx.x, slices);
  }
}

template <int KIND, int D, int NQ, bool SPLIT, int OWN>
void go(const KvAttnLaunch& a, const PrefixWs& w, const PrefixCut& c, hipStream_t s) {
  if (a.kv.page >= kTile)
    hipLaunchKernelGGL((prefix_kernel<KIND, D, NQ, SPLIT, OWN, true>), dim3(c.slices), dim3(kThreads), 0,
                       s, a, w, c.slices);
  else
    hipLaunchKernelGGL((prefix_kernel<KIND, D, NQ, SPLIT, OWN, false>), dim3(c.slices), dim3(kThreads), 0,
                       s, a, w, c.slices);
}
template <int KIND, int D>
void go_cut(const KvAttnLaunch& a, const PrefixWs& w, const PrefixCut& c, hipStream_t s) {
  if (!c.split) {
    if (c.nq_own == 1) go<KIND, D, 2, false, 1>(a, w, c, s);
    else go<KIND, D, 2, false, 2>(a, w, c, s);
  } else if (c.nq == 1) {
    go<KIND, D, 1, true, 1>(a, w, c, s);
  } else {
    if (c.nq_own == 1) go<KIND, D, 2, true, 1>(a, w, c, s);
    else go<KIND, D, 2, true, 2>(a, w, c, s);
  }
}

}  // namespace

template <int D>
void launch_prefix(const PrefixLaunch& p, const PrefixWs& w, const PrefixCut& c, hipStream_t s) {
  if (p.a.kv.dtype == DFS_FP8) go_cut<DFS_FP8, D>(p.a, w, c, s);
  else go_cut<DFS_INT8, D>(p.a, w, c, s);
}

}  // namespace dfs
