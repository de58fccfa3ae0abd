// kv8_attention.hip -- attention of new tokens over the 8-bit paged cache,
// with a sliding window and first tokens that stay visible.
//
// For query row q of a kv head: o = sum_j w_j v_j / sum_j w_j with
// w_j = 2^(t_j - m), t_j = (q . code_j) kscale_j sm_scale log2(e), m the
// running maximum of t: one pass over the keys.
//
// The products, the softmax and the split of the work stand in kv8_attn.hpp.
//
// What bounds it, as measured (head_dim 128 unless stated; times of a call among
// others).  Decode: the codes, read once.  32 requests of 646 to 8192 tokens, 32
// heads: 191 us for 1.05 GB, 5.5 TB/s (a plain read of 1 GiB: 5.84); 4 tokens over
// 131071, 8 kv heads for 32: 65 us, 4.1 TB/s; 24 int8 requests under a window of
// 4096, pages of 16: 50 us, 3.9 TB/s; these two end with a join.  One request of
// 777 tokens: 10.3 us, chain of plan, pages, codes, join.  Prompts: the vector
// units are busy 61% of the time (conversions, exponentials, masks), the matrix
// cores 37%, neither full.  3 chunks of 1500 to 2048 tokens over 495 to 1021
// cached ones: 261 us, 0.55 PFLOP/s.  Sharing the converted codes of a tile
// between the waves through LDS costs a barrier per tile: 303 us where each wave
// converting for itself took 281.  head_dim 256: 32 requests to 8000 tokens, 8 kv
// heads for 16, 117 us; 3 chunks to 1024 tokens over to 500, 4 for 16, 163 us.
#include "kv8_attn.hpp"

namespace dfs {
namespace {

constexpr int kInlinePlan = 256;         // entries up to which every workgroup plans for itself

struct AttnWs {
  Line line;
  int64_t* first;    // plan: first tile of each entry, then the total
  int32_t* req;      // plan: request of each entry
  int32_t* qblk;     // plan: its block of query rows
  int32_t* n_entries;  // plan: entries, and the most tiles of an item
  int32_t max_entries;
};

// The plan of a small batch, in LDS.
struct Plan {
  int64_t tmp[kWaves];
  int32_t longest;
  int64_t first[kInlinePlan + 1];
  int32_t req[kInlinePlan], qblk[kInlinePlan];
  Req facts[kInlinePlan];
};

// The items of a batch; complete rows go to the output.
template <int KIND, int D, int NQ, bool SPLIT, bool F32, bool BIG>
struct Batch : Attn<KIND, D, NQ, SPLIT, F32, BIG> {
  using A = Attn<KIND, D, NQ, SPLIT, F32, BIG>;
  const AttnWs& ws;
  const Plan& plan;
  const int inline_plan;
  __device__ __forceinline__ Batch(const KvAttnLaunch& a, const AttnWs& w, const Plan& p, int in)
      : A(a), ws(w), plan(p), inline_plan(in) {}
  __device__ __forceinline__ int64_t first(int e) const { return inline_plan ? plan.first[e] : *gptr(ws.first + e); }
  __device__ __forceinline__ int longest() const { return uni(inline_plan ? plan.longest : *gptr(ws.n_entries + 1)); }
  __device__ __forceinline__ int ready(int e, int kh) {
    const int req = uni(inline_plan ? plan.req[e] : *gptr(ws.req + e));
    const int qblk = uni(inline_plan ? plan.qblk[e] : *gptr(ws.qblk + e));
    A::begin(inline_plan ? plan.facts[req] : get_req(A::a.b, A::a.kv.page, req), req, qblk, kh);
    return qblk;
  }
  __device__ __forceinline__ int64_t at(int row) const { return A::out_at(row); }
  __device__ __forceinline__ void put(int64_t at, int d, const f4& v, float, float l) const { A::store(at + d, v, l); }
  __device__ __forceinline__ void put_nan(int64_t at, int d) const { A::store_nan(at + d); }
};

// Entries (request, block of qb query rows) in order and the first tile of
// each, by one workgroup; first[entries] is the total, *longest the most tiles
// that an item has.  Returns the entries:
// at most `most`, which a tok_start that is not ascending could pass.
// `extra` tiles stand for what an item costs besides its tiles.  facts: of the
// requests, if there is room for them.
template <typename T>  // of the entry counts: 256 requests of at most 256 entries fit int
__device__ int make_plan(const KvAttnLaunch& a, int qb, int extra, int most, int64_t* first,
                         int32_t* req, int32_t* qblk, Req* facts, int32_t* longest, int64_t* tmp, int threads) {
  const int g = a.q_heads / a.kv.heads;
  int n_entries = 0;
  for (int r0 = 0; r0 < a.b.n_req; r0 += threads) {
    const int r = r0 + (int)threadIdx.x;
    int nb = 0;
    if (r < a.b.n_req) {
      const Req q = get_req(a.b, a.kv.page, r);
      if (facts) facts[r] = q;
      nb = (int)min<int64_t>(((int64_t)q.n * g + qb - 1) / qb, most);
    }
    T total;
    const T at = n_entries + block_scan<T>(nb, (T*)tmp, &total, threads);
    for (int i = 0; i < nb && at + i < most; ++i) {
      req[at + i] = r;
      qblk[at + i] = i;
    }
    n_entries = (int)min<T>(n_entries + total, most);
  }
  __syncthreads();
  int64_t base = 0;
  int most_tiles = 0;
  if (threadIdx.x == 0) *longest = 0;
  for (int e0 = 0; e0 < n_entries; e0 += threads) {
    const int e = e0 + (int)threadIdx.x;
    int64_t t = 0;
    if (e < n_entries) {
      const Req q = facts ? facts[req[e]] : get_req(a.b, a.kv.page, req[e]);
      const int i0 = (int)((int64_t)qblk[e] * qb / g);
      const int i1 = (int)min<int64_t>(((int64_t)(qblk[e] + 1) * qb - 1) / g, q.n - 1);
      const int tiles = get_span(q, q.len - q.n + i0, q.len - q.n + i1, a.window, a.sinks).n;
      most_tiles = max(most_tiles, tiles);
      t = ((int64_t)tiles + extra) * a.kv.heads;
    }
    int64_t total;
    const int64_t at = base + block_scan<int64_t>(t, tmp, &total, threads);
    if (e < n_entries) first[e] = at;
    base += total;
  }
  if (threadIdx.x == 0) first[n_entries] = base;
  if (most_tiles > 0) atomicMax(longest, most_tiles);
  __syncthreads();
  return n_entries;
}

constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(KvAttnLaunch a, AttnWs w, int qb,
                                                            int extra) {
  __shared__ int64_t tmp[kPlanThreads / kWave];
  __shared__ int32_t longest;
  const int n = make_plan<int64_t>(a, qb, extra, w.max_entries, w.first, w.req, w.qblk, nullptr, &longest,
                                   tmp, kPlanThreads);
  if (threadIdx.x == 0) {
    w.n_entries[0] = n;
    w.n_entries[1] = longest;
  }
}

template <int KIND, int D, int NQ, bool SPLIT, bool F32, bool BIG>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2)
void attn_kernel(KvAttnLaunch a, AttnWs ws, int least, int slices, int inline_plan) {
  using A = Batch<KIND, D, NQ, SPLIT, F32, BIG>;
  __shared__ typename A::Work sh;
  __shared__ Plan plan;
  A t(a, ws, plan, inline_plan);
  const int n_entries =
      inline_plan ? make_plan<int>(a, A::kQb, A::kExtra, ws.max_entries, plan.first, plan.req, plan.qblk,
                                   plan.facts, &plan.longest, plan.tmp, kThreads)
                  : *gptr(ws.n_entries);
  run_line(t, sh, ws.line, n_entries, least, (int)blockIdx.x, slices);
}

// How a call is cut: query rows per item, workgroups, entries at most.
struct Cut {
  bool split;
  int nq, qb;
  int slices;
  int64_t entries;
};
Cut get_cut(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads) {
  Cut c;
  const int64_t g = q_heads / kv.heads;
  // By the rows of a request, on average.  Up to 16 one group of rows: 10.5 us
  // at one request, 191 at 32 long ones, against 11.6 and 196 with two groups.
  // Up to 32 the waves share the rows: 40.8 us at 20 rows of 8 requests to 16000
  // tokens, 42.0 where each wave has its own; 191, 209 at one row of 32; at 48
  // rows both take 60 to 63 us, and prompts 403 us shared, 254 with rows of their own.
  const double rows = (double)n_tok * g / std::max(n_req, 1);
  c.split = rows <= 32;
  c.nq = c.split && rows <= 16 ? 1 : 2;
  c.qb = c.split ? 16 * c.nq : 16 * c.nq * 4;
  c.entries = std::min<int64_t>(n_req, n_tok) + (int64_t)n_tok * g / c.qb;
  // as many workgroups as the device holds at once: two per CU, one where a
  // wave needs more than half of a SIMD's registers (half as many: 269 against
  // 254 us for prompts, 71 against 64 with a window, 197 against 191 at decode;
  // head_dim 256 with 512: 230 against 163 for prompts, 124 against 117 at decode)
  c.slices = kv.head_dim == 256 ? 256 : 512;
  return c;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t first, req, qblk, n, part_ml, group_ml, part_o, total;
};
Layout get_layout(const Cut& c, int D) {
  Layout l;
  l.first = kCounterBytes;
  l.req = l.first + up((c.entries + 1) * 8);
  l.qblk = l.req + up(c.entries * 4);
  l.n = l.qblk + up(c.entries * 4);
  l.part_ml = l.n + 256;
  l.group_ml = l.part_ml + up((size_t)2 * c.slices * c.qb * 8);
  l.part_o = l.group_ml + up((size_t)2 * c.slices * c.qb * 8);
  l.total = l.part_o + (size_t)2 * c.slices * c.qb * D * 4;
  return l;
}

template <int KIND, int D, int NQ, bool SPLIT>
void go(const KvAttnLaunch& a, const AttnWs& w, const Cut& c, hipStream_t s) {
  const int in = c.entries <= kInlinePlan && a.b.n_req <= kInlinePlan;
  using A = Attn<KIND, D, NQ, SPLIT, false, false>;
  if (!in) hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, w, c.qb,
                              A::kExtra);
  static_assert(A::kQb == (SPLIT ? 16 * NQ : 64 * NQ), "get_cut");
  const int least = SPLIT ? kWaves : 1;
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(c.slices), dim3(kThreads), 0, s, a, w, least, c.slices, in);
  };
  const bool big = a.kv.page >= kTile;
  if (a.odt == DFS_F32) {
    if (big) run(attn_kernel<KIND, D, NQ, SPLIT, true, true>);
    else run(attn_kernel<KIND, D, NQ, SPLIT, true, false>);
  } else {
    if (big) run(attn_kernel<KIND, D, NQ, SPLIT, false, true>);
    else run(attn_kernel<KIND, D, NQ, SPLIT, false, false>);
  }
}
template <int KIND, int D>
void go_d(const KvAttnLaunch& a, const AttnWs& w, const Cut& c, hipStream_t s) {
  if (!c.split) go<KIND, D, 2, false>(a, w, c, s);
  else if (c.nq == 1) go<KIND, D, 1, true>(a, w, c, s);
  else go<KIND, D, 2, true>(a, w, c, s);
}
template <int KIND>
void go_kind(const KvAttnLaunch& a, const AttnWs& w, const Cut& c, hipStream_t s) {
  if (a.kv.head_dim == 64) go_d<KIND, 64>(a, w, c, s);
  else if (a.kv.head_dim == 96) go_d<KIND, 96>(a, w, c, s);
  else if (a.kv.head_dim == 128) go_d<KIND, 128>(a, w, c, s);
  else go_d<KIND, 256>(a, w, c, s);
}

}  // namespace

size_t kv8_attention_ws_need(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads) {
  return get_layout(get_cut(kv, n_req, n_tok, q_heads), kv.head_dim).total;
}

// Enough for every call of up to n_req requests and n_tok tokens: fewer requests
// have more rows each, so that blocks can be larger than this call's, and the
// smallest blocks are for at most 16 rows a request.
size_t kv8_attention_ws_bytes(const dfs_kv8& kv, int32_t n_req, int32_t n_tok, int32_t q_heads) {
  const int64_t rows = (int64_t)n_tok * (q_heads / kv.heads);
  Cut c = get_cut(kv, 1, n_tok, q_heads);  // the largest blocks
  c.entries = std::min(n_req, n_tok) +
              std::max(std::min<int64_t>(rows / 16, std::max(n_req, 1)), rows / 128);
  return get_layout(c, kv.head_dim).total;
}

hipError_t launch_kv8_attention(const KvAttnLaunch& a, void* ws, hipStream_t s) {
  const Cut c = get_cut(a.kv, a.b.n_req, a.b.n_tok, a.q_heads);
  const Layout l = get_layout(c, a.kv.head_dim);
  char* p = (char*)ws;
  const AttnWs w = {{(uint32_t*)p, (float*)(p + l.part_o), (f2*)(p + l.part_ml), (f2*)(p + l.group_ml)},
                    (int64_t*)(p + l.first),
                    (int32_t*)(p + l.req),
                    (int32_t*)(p + l.qblk),
                    (int32_t*)(p + l.n),
                    (int32_t)c.entries};
  if (a.kv.dtype == DFS_FP8) go_kind<DFS_FP8>(a, w, c, s);
  else go_kind<DFS_INT8>(a, w, c, s);
  return hipGetLastError();
}

}  // namespace dfs
