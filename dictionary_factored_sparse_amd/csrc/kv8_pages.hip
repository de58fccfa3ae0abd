// kv8_pages.hip -- who owns which page of the 8-bit cache: page tables and
// slot maps from request lengths, rows given back, rows forked or reordered,
// and the copies of pages that this asks for.
//
// The pool's state is one count per page, refs[p]: the table entries that name
// it, 0 where it is free.  Pages are handed out lowest first, in the order of
// rows and entries, so that what a call does depends on its inputs alone.
#include <algorithm>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kLoads = 32;                        // refs a lane holds at once
constexpr int kWords = kWaves * kLoads;           // 64 pages each
constexpr int kRound = kWords * kWave;            // pages looked at in one round
constexpr int kInlineTokens = 4 * kThreads;       // tokens up to which one workgroup maps them

__device__ __forceinline__ int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ bool is_page(int p, int n) { return p >= 0 && p < n; }

// Pages that rows of `len` tokens take.
__device__ __forceinline__ int pages_of(int64_t len, int page, int most) {
  return (int)least((len + page - 1) / page, most);
}

// Sum of v over the threads before this one, and over all of them.  The waves' sums
// are added by the lanes of each wave.
template <typename T>
__device__ __forceinline__ T scan(T v, T* tmp, T* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  T x = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const T y = __shfl_up(x, o, kWave);
    x += lane >= o ? y : 0;
  }
  if (lane == kWave - 1) tmp[wave] = x;
  __syncthreads();
  T w = tmp[lane % kWaves];
#pragma unroll
  for (int o = 1; o < kWaves; o <<= 1) {
    const T y = __shfl_up(w, o, kWaves);
    w += lane % kWaves >= o ? y : 0;
  }
  __syncthreads();
  *total = __shfl(w, kWaves - 1, kWave);
  return (wave > 0 ? __shfl(w, wave - 1, kWave) : 0) + x - v;
}

// The free pages in order, as one workgroup finds them: a round of kRound pages
// at a time, held as one bit a page.  Every call is made by all threads.
struct FreePages {
  struct Shared {
    uint64_t bits[kWords];
    int before[kWords];  // free pages of the round before this word
    int sum[kWaves];
  };
  Shared& sh;
  const int32_t* refs;
  const int n_pages;
  uint32_t next = 0;       // first page not looked at
  int64_t lo = 0, hi = 0;  // ranks of the free pages of this round: lo .. hi - 1

  __device__ __forceinline__ FreePages(Shared& s, const int32_t* r, int n)
      : sh(s), refs(r), n_pages(n) {}
  __device__ __forceinline__ bool more() const { return next < (uint32_t)n_pages; }
  __device__ __forceinline__ void round() {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint32_t p0 = next + wave * kLoads * kWave + lane;
    int32_t v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)  // pages are below 2^28: byte offsets fit 32 bits
      v[i] = *gptr((const int32_t*)((const char*)refs + 4 * min(p0 + i * kWave, (uint32_t)n_pages - 1)));
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint64_t m = __ballot(v[i] == 0 && p0 + i * kWave < (uint32_t)n_pages);
      if (lane == i) mine = m;
    }
    // the words of a wave are in its lanes 0 .. kLoads - 1
    int x = __popcll(mine);
    const int own = x;
#pragma unroll
    for (int o = 1; o < kLoads; o <<= 1) {
      const int y = __shfl_up(x, o, kWave);
      if (lane >= o) x += y;
    }
    __syncthreads();  // the last round's words have been read
    if (lane < kLoads) sh.bits[wave * kLoads + lane] = mine;
    if (lane == kLoads - 1) sh.sum[wave] = x;
    __syncthreads();
    int w = sh.sum[lane % kWaves];
#pragma unroll
    for (int o = 1; o < kWaves; o <<= 1) {
      const int y = __shfl_up(w, o, kWaves);
      w += lane % kWaves >= o ? y : 0;
    }
    const int all = __shfl(w, kWaves - 1, kWave), base = wave > 0 ? __shfl(w, wave - 1, kWave) : 0;
    if (lane < kLoads) sh.before[wave * kLoads + lane] = base + x - own;
    __syncthreads();
    lo = hi;
    hi += all;
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
  __device__ __forceinline__ int take(bool want, int64_t& done, int* tmp) {
    int total;
    const int at = scan<int>(want ? 1 : 0, tmp, &total);
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
  __shared__ int64_t tmp[kWaves];
  __shared__ int first[kThreads], entry[kThreads], start[kThreads + 1], have[kThreads];
  FreePages pages(fs, a.refs, a.n_pages);
  const int tid = threadIdx.x;
  int64_t tok = 0, ranks = 0;
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
    int64_t all;
    const int64_t at = tok + scan<int64_t>(n, tmp, &all);
    const int64_t t0 = least(at, a.n_tok);
    n = least(at + n, a.n_tok) - t0;
    tok += all;
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
    int total;
    first[tid] = scan<int>(many, (int*)tmp, &total);
    entry[tid] = i0;
    __syncthreads();
    for (int e0 = 0; e0 < total; e0 += kThreads) {
      const int e = e0 + tid;
      int32_t* p = nullptr;
      if (e < total) {
        int j = 0;
        for (int s = kThreads / 2; s > 0; s >>= 1)
          if (first[j + s] <= e) j += s;
        p = a.table + (int64_t)(r0 + j) * a.ldt + entry[j] + (e - first[j]);
      }
      const bool want = p && !is_page(*p, a.n_pages);
      const int got = pages.take(want, ranks, (int*)tmp);
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
__device__ __forceinline__ void split_rows(const KvReorder& a, FreePages& pages, int* tmp, F children, G eldest) {
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
    const int got = pages.take(want, ranks, tmp);
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
  __shared__ int tmp[kWaves];
  FreePages pages(fs, a.refs, a.n_pages);
  pages.round();
  split_rows(a, pages, tmp, [&](int p) { return *gptr(children + p); }, [&](int p) { return *gptr(eldest + p); });
}

// All of a small call in one launch.
constexpr int kSmallRows = 1024, kSmallEntries = 4096;
__global__ __launch_bounds__(kThreads) void small_kernel(KvReorder a) {
  __shared__ FreePages::Shared fs;
  __shared__ int tmp[kWaves], children[kSmallRows], eldest[kSmallRows];
  const int tid = threadIdx.x;
  if (tid < a.n_in) {
    children[tid] = 0;
    eldest[tid] = INT32_MAX;
  }
  __syncthreads();
  for (int b = tid; b < a.n_out; b += kThreads) {
    const int p = *gptr(a.parent + b);
    if (p < 0 || p >= a.n_in) continue;
    atomicAdd(children + p, 1);
    atomicMin(eldest + p, b);
  }
  __syncthreads();
  for (int e = tid; e < a.n_out * a.table_pages; e += kThreads) out_entry(a, e / a.table_pages, e % a.table_pages);
  for (int e = tid; e < a.n_in * a.table_pages; e += kThreads)
    in_entry(a, e / a.table_pages, children[e / a.table_pages], e % a.table_pages);
  // the counts are read below by plain loads: what has been added is in the L2
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  FreePages pages(fs, a.refs, a.n_pages);
  pages.round();
  split_rows(a, pages, tmp, [&](int p) { return children[p]; }, [&](int p) { return eldest[p]; });
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
  // entries 9.3 us so, 2.6 and 7.4 in two launches; 13 rows of 10 forked to 104 10.9 us,
  // 4.8 and 7.8
  if (a.n_in <= kSmallRows && ((int64_t)a.n_in + a.n_out) * a.table_pages <= kSmallEntries) {
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
