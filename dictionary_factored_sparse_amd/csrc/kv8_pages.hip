// kv8_pages.hip -- who owns which page of the 8-bit cache: page tables and
// slot maps from request lengths, rows given back, rows forked or reordered,
// and the copies of pages that this asks for.
//
// The pool's state is one count per page, refs[p]: the table entries that name
// it, 0 where it is free.  Pages are handed out lowest first, in the order of
// rows and entries, so that what a call does depends on its inputs alone.
//
// What bounds it.  Tables and reorders: a chain of reads, sums and searches in one
// workgroup, which alone can hand pages out in order without a wait between workgroups
// (32 decoding requests over 2777 pages 8.3 us, 203 requests with 1116 new entries over
// 90001 pages 9.4 and 3.7 for the maps; 13 rows forked to 104 8.5).  Giving back: launch
// and one pass (2.8).  Copies: memory (104 halves of pages of 8 heads in 4 layers, 127
// MB, 17.7 us, 7.2 TB/s).
#include <algorithm>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kLoads = 32;                        // refs a lane holds at once
constexpr int kWords = kWaves * kLoads;           // 64 pages each
constexpr int kRound = kWords * kWave;            // pages looked at in one round
// Tokens up to which the workgroup of the tables maps them: 32 tokens 8.3 us, 10.0 in a
// launch of their own; some 4000 12.3, 11.4 and the other launch's start.
constexpr int kInlineTokens = 4 * kThreads;

__device__ __forceinline__ int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ bool is_page(int p, int n) { return p >= 0 && p < n; }

// Pages that rows of `len` tokens take.
__device__ __forceinline__ int pages_of(int64_t len, int page, int most) {
  return (int)least((len + page - 1) / page, most);
}

// Sums that stop at 2^32 - 1 are as good as longer ones where a smaller bound is
// applied to them, and adding so is associative.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Lane l's sum over the lanes up to it, in its row of 16 lanes or (WAVE) in the wave.
// The lanes' registers are read in place (by shuffles, which go through LDS, and a
// second barrier a sum 32 decoding requests took 10.9 us, so 8.6; a reorder of 4 rows
// 8.2, so 7.2).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}
template <bool WAVE>
__device__ __forceinline__ uint32_t lane_scan(uint32_t x) {
  x = add(x, moved<0x111, 0xF>(x));  // from 1, 2, 4, 8 lanes before
  x = add(x, moved<0x112, 0xF>(x));
  x = add(x, moved<0x114, 0xF>(x));
  x = add(x, moved<0x118, 0xF>(x));
  if constexpr (WAVE) {
    x = add(x, moved<0x142, 0xA>(x));  // row 0's last lane to row 1, row 2's to row 3
    x = add(x, moved<0x143, 0xC>(x));  // row 1's last lane to rows 2 and 3
  }
  return x;
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) { return __builtin_amdgcn_readlane(v, l); }

// Sums over the threads before this one, and over all of them, one barrier each: two
// calls in a row use different places.
struct Scan {
  uint32_t tmp[2][kWaves];
};
struct Scanner {
  Scan& sh;
  int at = 0;
  __device__ __forceinline__ Scanner(Scan& s) : sh(s) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t v, uint32_t* total) {
    static_assert(kWaves == 16, "a row of lanes");
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t x = lane_scan<true>(v);
    if (lane == kWave - 1) sh.tmp[at][wave] = x;
    __syncthreads();
    const uint32_t w = lane_scan<false>(sh.tmp[at][lane % kWaves]);
    at ^= 1;
    *total = lane_of(w, kWaves - 1);
    // the sum before this lane is that up to the lane before it
    const uint32_t before = moved<0x138, 0xF>(x);
    return add(wave > 0 ? lane_of(w, wave - 1) : 0u, before);
  }
};

// The free pages in order, as one workgroup finds them: a round of kRound pages
// at a time, held as one bit a page.  Every call is made by all threads.
struct FreePages {
  struct Shared {
    uint64_t bits[kWords];
    int before[kWords];  // free pages of the round before this word
    uint32_t sum[kWaves];
    Scan scan;
  };
  Shared& sh;
  const int32_t* refs;
  const int n_pages;
  Scanner scan;
  uint32_t next = 0;       // first page not looked at
  int64_t lo = 0, hi = 0;  // ranks of the free pages of this round: lo .. hi - 1

  __device__ __forceinline__ FreePages(Shared& s, const int32_t* r, int n)
      : sh(s), refs(r), n_pages(n), scan(s.scan) {}
  __device__ __forceinline__ bool more() const { return next < (uint32_t)n_pages; }
  // The counts that this lane looks at in the next round.
  struct Ahead {
    int32_t v[kLoads];
  };
  __device__ __forceinline__ uint32_t mine() const {
    return next + threadIdx.x / kWave * kLoads * kWave + threadIdx.x % kWave;
  }
  __device__ __forceinline__ Ahead ahead() const {
    const uint32_t p0 = mine();
    Ahead x;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)  // pages are below 2^28: byte offsets fit 32 bits
      x.v[i] = *gptr((const int32_t*)((const char*)refs + 4 * min(p0 + i * kWave, (uint32_t)n_pages - 1)));
    return x;
  }
  __device__ __forceinline__ void round() { round(ahead()); }
  __device__ __forceinline__ void round(const Ahead& x) {
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t p0 = mine();
    uint64_t word = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint64_t m = __ballot(x.v[i] == 0 && p0 + i * kWave < (uint32_t)n_pages);
      if (lane == i) word = m;
    }
    // the words of a wave are in its lanes 0 .. kLoads - 1
    const uint32_t own = __popcll(word), upto = lane_scan<true>(own);
    if (next > 0) __syncthreads();  // the last round's words have been read
    if (lane < kLoads) sh.bits[wave * kLoads + lane] = word;
    if (lane == kLoads - 1) sh.sum[wave] = upto;
    __syncthreads();
    const uint32_t w = lane_scan<false>(sh.sum[lane % kWaves]);
    if (lane < kLoads) sh.before[wave * kLoads + lane] = (int)((wave > 0 ? lane_of(w, wave - 1) : 0u) + upto - own);
    __syncthreads();
    lo = hi;
    hi += lane_of(w, kWaves - 1);
    page0 = next;
    next += kRound;
  }
  // The free page of rank r, lo <= r < hi.
  __device__ __forceinline__ int page(int64_t r) const {
    const int k = (int)(r - lo);
    int w = 0;
    for (int s = kWords / 2; s > 0; s >>= 1)
      if (sh.before[w + s] <= k) w += s;
    uint64_t m = sh.bits[w];
    int i = k - sh.before[w], at = 0;  // its place among the word's set bits, by halves
#pragma unroll
    for (int s = kWave / 2; s > 0; s >>= 1) {
      const int low = __popcll(m & ((1ull << s) - 1));
      if (i >= low) {
        i -= low;
        at += s;
        m >>= s;
      }
    }
    return (int)(page0 + w * kWave + at);
  }
  // Hands pages to the threads that want one, lowest rank first; `done` ranks
  // went out before.  -1 where there are none left.
  __device__ __forceinline__ int take(bool want, int64_t& done) {
    uint32_t total;
    const uint32_t at = scan(want ? 1 : 0, &total);
    const int64_t r = done + at;
    int got = -1;
    done += total;
    if (total == 0) return -1;
    for (;;) {
      if (want && r >= lo && r < hi) got = page(r);
      if (done <= hi || !more()) return got;
      round();
    }
  }

 private:
  uint32_t page0 = 0;
};

// ------------------------------------------------------------------ tables

__device__ __forceinline__ void map_token(const KvTables& a, int t, int r, int start, int cached) {
  int pos = -1;
  int64_t slot = -1;
  if (r >= 0) {
    const int64_t p = (int64_t)max(cached, 0) + (t - start);
    pos = (int)least(p, INT32_MAX);
    const int i = pos / a.page;
    if (i < a.table_pages) {
      const int pg = a.table[r * a.ldt + i];
      if (is_page(pg, a.n_pages)) slot = (int64_t)pg * a.page + pos % a.page;
    }
  }
  if (a.tok_req) a.tok_req[t] = r;
  if (a.tok_pos) a.tok_pos[t] = pos;
  if (a.slot) a.slot[t] = slot;
}
// The request of token t: the last one that starts at or before it and is not
// empty; -1 behind the last one's tokens.  starts(i), i = 0 .. n_req, ascends.
template <typename F>
__device__ __forceinline__ int request_of(int t, int n_req, F starts) {
  if (t >= starts(n_req)) return -1;
  int lo = 0, hi = n_req;  // starts(lo) <= t < starts(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (starts(mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Starts, lengths and pages of all requests, by one workgroup; the tokens' maps
// too where MAP.
template <bool MAP>
__global__ __launch_bounds__(kThreads) void tables_kernel(KvTables a) {
  __shared__ FreePages::Shared fs;
  __shared__ int first[kThreads], entry[kThreads], start[kThreads + 1], have[kThreads];
  FreePages pages(fs, a.refs, a.n_pages);
  const int tid = threadIdx.x;
  int64_t ranks = 0;
  uint32_t tok = 0;  // tokens so far, up to 2^32 - 1
  int ci = tid < a.n_req ? *gptr(a.cached + tid) : 0, ni = tid < a.n_req ? *gptr(a.n_new + tid) : 0;
  pages.round();  // its reads go with those of the first requests
  for (int r0 = 0; r0 < a.n_req; r0 += kThreads) {
    const int r = r0 + tid;
    if (r0 > 0) {
      ci = r < a.n_req ? *gptr(a.cached + r) : 0;
      ni = r < a.n_req ? *gptr(a.n_new + r) : 0;
    }
    const int64_t c = max(ci, 0);
    int64_t n = max(ni, 0);
    uint32_t all;
    const int64_t at = add(tok, pages.scan((uint32_t)n, &all));
    const int64_t t0 = least(at, a.n_tok);
    n = least(at + n, a.n_tok) - t0;
    tok = add(tok, all);
    if (r < a.n_req) {
      a.tok_start[r] = (int)t0;
      a.length[r] = (int)least(c + n, INT32_MAX);
      if (MAP) {
        start[tid] = (int)t0;
        have[tid] = ci;
      }
    }
    const int i0 = pages_of(c, a.page, a.table_pages);
    const int many = pages_of(c + n, a.page, a.table_pages) - i0;
    uint32_t total;
    first[tid] = (int)pages.scan((uint32_t)many, &total);
    entry[tid] = i0;
    __syncthreads();
    for (int e0 = 0; e0 < (int)total; e0 += kThreads) {
      const int e = e0 + tid;
      int32_t* p = nullptr;
      if (e < (int)total) {
        int j = 0;
        for (int s = kThreads / 2; s > 0; s >>= 1)
          if (first[j + s] <= e) j += s;
        p = a.table + (int64_t)(r0 + j) * a.ldt + entry[j] + (e - first[j]);
      }
      const bool want = p && !is_page(*p, a.n_pages);
      const int got = pages.take(want, ranks);
      if (want) {
        *p = got;
        if (got >= 0) a.refs[got] = 1;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    const int end = (int)least(tok, a.n_tok);
    a.tok_start[a.n_req] = end;
    if (MAP) start[a.n_req] = end;
    a.missing[0] = (int)max(ranks - pages.hi, (int64_t)0);
  }
  if constexpr (MAP) {
    __syncthreads();
    for (int t = tid; t < a.n_tok; t += kThreads) {
      const int r = request_of(t, a.n_req, [&](int i) { return start[i]; });
      map_token(a, t, r, r < 0 ? 0 : start[r], r < 0 ? 0 : have[r]);
    }
  }
}

__global__ __launch_bounds__(256) void map_kernel(KvTables a) {
  const int t = blockIdx.x * 256 + (int)threadIdx.x;
  if (t >= a.n_tok) return;
  const int r = request_of(t, a.n_req, [&](int i) { return *gptr(a.tok_start + i); });
  map_token(a, t, r, r < 0 ? 0 : *gptr(a.tok_start + r), r < 0 ? 0 : *gptr(a.cached + r));
}

// ------------------------------------------------------------------ release

__global__ __launch_bounds__(256) void release_kernel(KvRelease a, int row0) {
  const int r = row0 + (int)blockIdx.y;
  const int i0 = a.first ? min(max(*gptr(a.first + r), 0), a.table_pages) : 0;  // the sums below stay in 32 bits
  const int i1 = a.last ? min(*gptr(a.last + r), a.table_pages) : a.table_pages;
  for (int i = i0 + (int)(blockIdx.x * 256 + threadIdx.x); i < i1; i += (int)gridDim.x * 256) {
    int32_t* p = a.table + r * a.ldt + i;
    const int pg = *p;
    if (is_page(pg, a.n_pages)) atomicSub(a.refs + pg, 1);
    *p = -1;
  }
}

// ------------------------------------------------------------------ reorder

// Entry i of out row r: its parent's.
__device__ __forceinline__ void out_entry(const KvReorder& a, int r, int i) {
  const int p = *gptr(a.parent + r);
  const bool real = p >= 0 && p < a.n_in;
  const int len = real ? max(*gptr(a.length + p), 0) : 0;
  const int pg = i < pages_of(len, a.page, a.table_pages) ? *gptr(a.table + p * a.ldt + i) : -1;
  a.out[r * a.ldo + i] = is_page(pg, a.n_pages) ? pg : -1;
  if (i == 0) {
    a.length_out[r] = len;
    a.src[r] = -1;
    a.dst[r] = -1;
  }
}
// Entry i of in row r, which has c children: what they and the row's own end do to the
// page's count.
__device__ __forceinline__ void in_entry(const KvReorder& a, int r, int c, int i) {
  const int pg = *gptr(a.table + r * a.ldt + i);
  const int used = pages_of(max(*gptr(a.length + r), 0), a.page, a.table_pages);
  const int delta = (i < used ? c : 0) - (a.keep ? 0 : 1);
  if (delta != 0 && is_page(pg, a.n_pages)) atomicAdd(a.refs + pg, delta);
}

__global__ __launch_bounds__(256) void rows_kernel(KvReorder a, int32_t* children, int32_t* eldest,
                                                   int row0) {
  const int r = row0 + (int)blockIdx.y, tid = threadIdx.x;
  const int at = (int)blockIdx.x * 256 + tid, step = (int)gridDim.x * 256;
  if (r < a.n_out)
    for (int i = at; i < a.table_pages; i += step) out_entry(a, r, i);
  if (r < a.n_in) {
    __shared__ int count, eld;
    if (tid == 0) {
      count = 0;
      eld = INT32_MAX;
    }
    __syncthreads();
    int c = 0, e = INT32_MAX;
    for (int b = tid; b < a.n_out; b += 256)
      if (*gptr(a.parent + b) == r) {
        ++c;
        e = min(e, b);
      }
    if (c > 0) {
      atomicAdd(&count, c);
      atomicMin(&eld, e);
    }
    __syncthreads();
    if (at == 0) {
      children[r] = count;
      eldest[r] = eld;
    }
    for (int i = at; i < a.table_pages; i += step) in_entry(a, r, count, i);
  }
}

// The pages that out rows would write next and do not own alone, by one workgroup.
// children(p), eldest(p): of in row p.
template <typename F, typename G>
__device__ __forceinline__ void split_rows(const KvReorder& a, FreePages& pages, F children, G eldest) {
  int64_t ranks = 0;
  // the entry in question of row b, or null
  auto entry = [&](int b, int& p) -> int32_t* {
    if (b >= a.n_out) return nullptr;
    p = *gptr(a.parent + b);
    if (p < 0 || p >= a.n_in) return nullptr;
    const int len = max(*gptr(a.length + p), 0);
    if (len % a.page == 0 || len / a.page >= a.table_pages) return nullptr;
    return a.out + b * a.ldo + len / a.page;
  };
  for (int b0 = 0; b0 < a.n_out; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    int p = 0;
    int32_t* at = entry(b, p);
    const int pg = at ? *at : -1;
    const bool want = pg >= 0 && (eldest(p) != b || a.refs[pg] != children(p));
    const int got = pages.take(want, ranks);
    if (want) {
      *at = got;
      if (got >= 0) {
        a.refs[got] = 1;
        a.src[b] = pg;
        a.dst[b] = got;
      }
    }
  }
  if (threadIdx.x == 0) a.missing[0] = (int)max(ranks - pages.hi, (int64_t)0);
  __syncthreads();
  // only now may the pages that rows have left count as less used
  for (int b = threadIdx.x; b < a.n_out; b += kThreads) {
    int p = 0;
    const int32_t* at = entry(b, p);
    if (!at) continue;
    const int was = *gptr(a.table + p * a.ldt + (at - (a.out + b * a.ldo)));
    if (is_page(was, a.n_pages) && *at != was) atomicSub(a.refs + was, 1);
  }
}

__global__ __launch_bounds__(kThreads) void split_kernel(KvReorder a, const int32_t* children,
                                                         const int32_t* eldest) {
  __shared__ FreePages::Shared fs;
  FreePages pages(fs, a.refs, a.n_pages);
  pages.round();
  split_rows(a, pages, [&](int p) { return *gptr(children + p); }, [&](int p) { return *gptr(eldest + p); });
}

// All of a small call in one launch: what the last step asks of a row is read at
// the start (4 rows of 15 entries 8.2 us, 8.9 where each step
// read what it needed, with the same sums).
constexpr int kSmallRows = kThreads, kSmallEntries = 4096;
__global__ __launch_bounds__(kThreads) void small_kernel(KvReorder a) {
  __shared__ FreePages::Shared fs;
  __shared__ int children[kSmallRows], eldest[kSmallRows];
  const int b = threadIdx.x;
  children[b] = 0;
  eldest[b] = INT32_MAX;
  __syncthreads();
  int p = b < a.n_out ? *gptr(a.parent + b) : -1, part = -1, pg = -1;
  if (p >= 0 && p < a.n_in) {
    atomicAdd(children + p, 1);
    atomicMin(eldest + p, b);
    const int len = max(*gptr(a.length + p), 0);
    if (len % a.page != 0 && len / a.page < a.table_pages) {  // the page that is partly filled
      part = len / a.page;
      pg = *gptr(a.table + p * a.ldt + part);
    }
  }
  __syncthreads();
  for (int e = b; e < a.n_out * a.table_pages; e += kThreads) out_entry(a, e / a.table_pages, e % a.table_pages);
  for (int e = b; e < a.n_in * a.table_pages; e += kThreads)
    in_entry(a, e / a.table_pages, children[e / a.table_pages], e % a.table_pages);
  // the counts are read below by plain loads: what has been added is in the L2
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  FreePages pages(fs, a.refs, a.n_pages);
  const FreePages::Ahead ahead = pages.ahead();
  const bool want = is_page(pg, a.n_pages) && (eldest[p] != b || *gptr(a.refs + pg) != children[p]);
  pages.round(ahead);
  int64_t ranks = 0;
  const int got = pages.take(want, ranks);
  if (want) {
    a.out[b * a.ldo + part] = got;
    if (got >= 0) {
      a.refs[got] = 1;
      a.src[b] = pg;
      a.dst[b] = got;
    }
  }
  if (b == 0) a.missing[0] = (int)max(ranks - pages.hi, (int64_t)0);
  __syncthreads();
  // only now may the pages that rows have left count as less used
  if (want) atomicSub(a.refs + pg, 1);
}

// ------------------------------------------------------------------ copies

__global__ __launch_bounds__(256) void copy_kernel(KvCopy a, int row0) {
  const dfs_kv8& kv = a.kv[blockIdx.z];
  const int b = row0 + (int)blockIdx.y, h = blockIdx.x;
  const int s = *gptr(a.src + b), d = *gptr(a.dst + b);
  if (!is_page(s, kv.n_pages) || !is_page(d, kv.n_pages) || s == d) return;
  const int P = kv.page, D = kv.head_dim;
  const int full = a.length ? max(*gptr(a.length + b), 0) % P : 0;
  const int wide = full == 0 ? P / 16 : (full + 15) / 16;  // pieces of 16 tokens
  const int64_t from = (int64_t)s * kv.heads + h, to = (int64_t)d * kv.heads + h;
  const u4* ks = (const u4*)(kv.k + from * P * D);
  u4* kd = (u4*)(kv.k + to * P * D);
  for (int i = threadIdx.x; i < wide * D; i += 256) *gptr_w(kd + i) = *gptr(ks + i);
  const u4* vs = (const u4*)(kv.v + from * P * D);
  u4* vd = (u4*)(kv.v + to * P * D);
  for (int i = threadIdx.x; i < wide * D; i += 256) {
    const int at = i / wide * (P / 16) + i % wide;
    *gptr_w(vd + at) = *gptr(vs + at);
  }
  if (threadIdx.x == 0) {
    kv.kscale[to] = kv.kscale[from];
    kv.vscale[to] = kv.vscale[from];
  }
}

// Rows of a grid's y axis, which ends at 65535.
template <typename F>
void by_rows(int64_t rows, F launch) {
  for (int64_t y = 0; y < rows; y += 65535) launch((unsigned)std::min<int64_t>(rows - y, 65535), (int)y);
}

}  // namespace

hipError_t launch_kv8_tables(const KvTables& a, hipStream_t s) {
  const bool map = a.tok_req || a.tok_pos || a.slot;
  if (map && a.n_tok <= kInlineTokens && a.n_req <= kThreads) {
    hipLaunchKernelGGL(tables_kernel<true>, dim3(1), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(tables_kernel<false>, dim3(1), dim3(kThreads), 0, s, a);
  if (map && a.n_tok > 0)
    hipLaunchKernelGGL(map_kernel, dim3((unsigned)(((int64_t)a.n_tok + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv8_release(const KvRelease& a, hipStream_t s) {
  by_rows(a.n_req, [&](unsigned n, int r0) {
    hipLaunchKernelGGL(release_kernel, dim3(std::min((a.table_pages + 255) / 256, 64), n), dim3(256), 0,
                       s, a, r0);
  });
  return hipGetLastError();
}

hipError_t launch_kv8_reorder(const KvReorder& a, int32_t* ws, hipStream_t s) {
  // one launch while one workgroup is done with the rows in a few rounds: 4 rows of 15
  // entries 7.2 us so, 2.7 and 6.6 in two launches; 13 rows of 10 forked to 104 8.6 us,
  // 4.5 and 6.9
  if (std::max(a.n_in, a.n_out) <= kSmallRows && ((int64_t)a.n_in + a.n_out) * a.table_pages <= kSmallEntries) {
    hipLaunchKernelGGL(small_kernel, dim3(1), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  by_rows(std::max(a.n_in, a.n_out), [&](unsigned n, int r0) {
    hipLaunchKernelGGL(rows_kernel, dim3(std::min((a.table_pages + 255) / 256, 64), n), dim3(256), 0, s,
                       a, ws, ws + a.n_in, r0);
  });
  hipLaunchKernelGGL(split_kernel, dim3(1), dim3(kThreads), 0, s, a, (const int32_t*)ws,
                     (const int32_t*)ws + a.n_in);
  return hipGetLastError();
}

hipError_t launch_kv8_copy(const KvCopy& a, hipStream_t s) {
  by_rows(a.n, [&](unsigned n, int r0) {
    hipLaunchKernelGGL(copy_kernel, dim3(a.kv[0].heads, n, a.n_kv), dim3(256), 0, s, a, r0);
  });
  return hipGetLastError();
}

}  // namespace dfs
