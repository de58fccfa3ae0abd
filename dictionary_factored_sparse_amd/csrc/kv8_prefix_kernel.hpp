// kv8_prefix_kernel.hpp -- the kernel of kv8_prefix_attention, one head_dim a
// translation unit.
#pragma once

#include "kv8_attn.hpp"
#include "kv8_prefix.hpp"

namespace dfs {
namespace {

// The items of one line; complete rows are sums of it.
template <typename B>
struct Part : B {
  const PrefixWs& ws;
  const PrefixLine& w;
  __device__ __forceinline__ Part(const KvAttnLaunch& a, const PrefixWs& s, const PrefixLine& l)
      : B(a), ws(s), w(l) {}
  __device__ __forceinline__ int64_t first(int e) const { return *gptr(w.first + e); }
  __device__ __forceinline__ int longest() const { return uni(*gptr(w.n + 1)); }
  __device__ __forceinline__ int64_t at(int row) const {
    const int g = B::a.q_heads / B::a.kv.heads;
    const int tok = row / g, h = B::kh * g + row - tok * g;
    return (int64_t)(B::rq.t0 + tok) * B::a.q_heads + h;
  }
  __device__ __forceinline__ void put(int64_t at, int d, const f4& v, float m, float l) const {
    *gptr_w((f4*)(w.sum_o + at * B::kD + d)) = v;
    if (d == 0) *gptr_w(w.sum_ml + at) = f2{m, l};
  }
  __device__ __forceinline__ void put_nan(int64_t at, int d) const {
    *gptr_w(w.sum_o + at * B::kD + d) = __builtin_nanf("");
  }
};
// The keys that groups share.
template <typename B>
struct SharedPart : Part<B> {
  using P = Part<B>;
  __device__ __forceinline__ SharedPart(const KvAttnLaunch& a, const PrefixWs& s) : P(a, s, s.shared) {}
  __device__ __forceinline__ int ready(int e, int kh) {
    const int i = uni(*gptr(P::w.of + e)), qblk = uni(*gptr(P::w.qblk + e));
    const PrefixGroup* f = P::ws.groups + i;
    const int t0 = uni(*gptr(&f->t0)), keys = uni(*gptr(&f->keys));
    const int32_t* pos = P::ws.pos + t0;
    B::template begin_by<true>(Req{t0, uni(*gptr(&f->n)), keys, keys}, uni(*gptr(&f->row)), qblk, kh, 0,
                               uni(*gptr(&f->p0)), uni(*gptr(&f->p1)),
                               [=](int tok) { return *gptr(pos + tok); });
    return qblk;
  }
};
// Each request's own keys.
template <typename B>
struct OwnPart : Part<B> {
  using P = Part<B>;
  __device__ __forceinline__ OwnPart(const KvAttnLaunch& a, const PrefixWs& s) : P(a, s, s.own) {}
  __device__ __forceinline__ int ready(int e, int kh) {
    const int req = uni(*gptr(P::w.of + e)), qblk = uni(*gptr(P::w.qblk + e));
    const int grp = uni(*gptr(P::ws.group_of + req));
    const int from = grp < 0 ? 0 : uni(*gptr(&P::ws.groups[grp].keys));
    B::begin(get_req(B::a.b, B::a.kv.page, req), req, qblk, kh, from);
    return qblk;
  }
};
__device__ __forceinline__ Line line_of(const PrefixLine& p) {
  return {p.count, p.part_o, p.part_ml, p.group_ml};
}

template <int KIND, int D, int NQ, bool SPLIT, int OWN, bool BIG>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2)
void prefix_kernel(KvAttnLaunch a, PrefixWs ws, int slices) {
  using P = SharedPart<Attn<KIND, D, NQ, SPLIT, false, BIG>>;
  using S = OwnPart<Attn<KIND, D, OWN, true, false, BIG>>;
  __shared__ union {
    typename P::Work p;
    typename S::Work s;
  } sh;
  {
    P t(a, ws);
    run_line(t, sh.p, line_of(ws.shared), *gptr(ws.shared.n), SPLIT ? kWaves : 1, (int)blockIdx.x, slices);
  }
  __syncthreads();
  {
    S t(a, ws);
    run_line(t, sh.s, line_of(ws.own), *gptr(ws.own.n), kWaves, (int)blockIdx.x, slices);
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
