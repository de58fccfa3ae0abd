// kv8_attention.hip -- attention of new tokens over the 8-bit paged cache,
// with a sliding window and first tokens that stay visible.
//
// For query row q of a kv head: o = sum_j w_j v_j / sum_j w_j with
// w_j = 2^(t_j - m), t_j = (q . code_j) kscale_j sm_scale log2(e), m the
// running maximum of t: one pass over the keys.
//
// Layout of the products.  A wave takes 64 keys and NQ groups of 16 query
// rows (a row is one query token of one query head; the heads that share a kv
// head, and the tokens of a request, are rows of the same item, so a cached
// byte is read once for all of them).  Both products are
// v_mfma_f32_16x16x32_f16 on transposed operands, S^T = K Q^T and
// O^T = V^T W^T, so that the codes come from memory straight into the A
// operand in 16-byte loads and the softmax weights pass from the first
// product's result to the second one's B operand in their own lanes:
//   - K row of A row x in key group mm: key 16 (x / 4) + 4 mm + x % 4.  Then
//     lane (r = lane % 16, q = lane / 16) of S^T holds, for query row r, the
//     keys 16 q .. 16 q + 15: mm and the accumulator index count them.
//   - the second product takes k slots q * 8 + e as keys 16 q + 8 kk + e,
//     which is what that lane holds, and V^T rows are dims whose 16 keys
//     16 q .. are contiguous in a page (dfs_kv8 stores values so).
// Codes become f16 exactly (every E4M3 and int8 value is an f16 value); the
// page scales multiply the fp32 scores, and for values they enter the weights:
// w'_j = 2^(t_j + log2(vscale_j) - c), c the running maximum over the row's own
// keys of t_j + log2(vscale_j), so that a row's sums keep their bits whatever
// the scales of pages that it does not see or hardly weighs (with one exponent
// of vscale per wave, rows beside a page of 2^24 times their values lost 1e-4 of
// theirs, of 2^40 times all).  The sums are in units of 2^c, those of the
// weights themselves in units of 2^m.
//
// Rounding.  w' enters the second product as the sum of two f16 values: f16
// output is then as near to exact as its own rounding allows (2.1e-4 of the
// norm).  One f16 value gave 3.2e-4 and took 238 us for the prompts below where
// two took 256; for few rows two cost at most 2% (24 windowed requests 48.0 us
// with one, 49.0; 32 long ones 190.0, 190.7).  Weights are kept at 2^13 times their
// value so that f16's normal range reaches 2^-27 of the largest, and c is
// raised only when a key passes it by more than 2 (weights stay below 2^15),
// which spares most rescales of the sums.  m may lag by 32: nothing is held in
// few bits there, and finding its maximum over the lanes for every tile took the
// prompts below from 259 to 283 us.
//
// Work split.  The tiles of 64 keys of all items (request, block of query
// rows, kv head) form one line, cut into equal slices, one per workgroup: the
// lengths are read on the device, and a batch of uneven lengths or a single
// long request loads every CU alike.  An item that lies in several slices is
// joined by the workgroup that finishes last, in slice order, so results do
// not depend on which that is.
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
#include <algorithm>
#include <type_traits>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 64;                // keys per tile
constexpr int kInlinePlan = 256;         // entries up to which every workgroup plans for itself
constexpr int kCounterBytes = 65536;     // per-slice counters at the start of the workspace
constexpr int kWhole = 8;                // tiles up to which an item of a prompt is not split
constexpr float kWeightBits = 13.0f;     // weights are held at 2^13 times their value
constexpr float kSlack = 2.0f;           // the reference of the sums may lag by this (log2),
constexpr float kFar = 32.0f;            // that of the weights' own sum by this
constexpr float kLeast = 72.0f;          // 2^(13 + kFar - kLeast) is 0 in f16, 2^(13 - kLeast) far
                                         // above the least normal fp32
constexpr float kLog2e = 1.44269504088896340736f;

struct AttnWs {
  uint32_t* count;   // [3 * slices]: parts of a group that are done, groups of an item
  int64_t* first;    // plan: first tile of each entry, then the total
  int32_t* req;      // plan: request of each entry
  int32_t* qblk;     // plan: its block of query rows
  int32_t* n_entries;  // plan: entries, and the most tiles of an item
  int32_t max_entries;
  float* part_o;     // [2 * slices][rows][D]
  f2* part_ml;       // [2 * slices][rows]: reference of the weights, their sum
  f2* group_ml;      // the same of a group of slices, at its first slice's slot
};

// A request's rows in the batch, clamped to what the arrays hold.
struct Req {
  int t0, n, len, keys;
};
__device__ __forceinline__ Req get_req(const KvBatch& b, int page, int r) {
  Req q;
  q.t0 = min(max(b.tok_start[r], 0), b.n_tok);
  q.n = min(max(b.tok_start[r + 1], q.t0), b.n_tok) - q.t0;
  q.len = max(b.have[r], 0);
  q.keys = min(q.len, b.table_pages * page);
  return q;
}

// A value that is the same in all lanes, as the compiler is to know: addresses
// and bounds made of it then cost scalar instructions.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Tiles that some row of an entry sees: the first `ns` tiles hold first
// tokens, the others run from tile `ta`.
struct Span {
  int ns, ta, n;
  __device__ __forceinline__ int tile(int u) const { return u < ns ? u : u - ns + ta; }
};
__device__ __forceinline__ Span get_span(const Req& q, int p0, int p1, int window, int sinks) {
  Span s;
  const int hi = min(p1, q.keys - 1);                                // last visible key
  const int lo = window > 0 && p0 >= window ? p0 - window + 1 : 0;   // first one of the window
  const int sk = min(sinks, hi + 1);
  s.ta = lo / kTile;
  s.ns = sk > 0 ? min((sk - 1) / kTile + 1, s.ta) : 0;
  s.n = s.ns + (hi >= lo ? hi / kTile - s.ta + 1 : 0);
  if (s.n <= 0) s = {0, 0, 1};  // rows that see nothing still get their zeros
  return s;
}

template <typename T>
__device__ __forceinline__ T block_scan(T v, T* tmp, T* total, int threads) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  T x = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const T y = __shfl_up(x, o, kWave);
    if (lane >= o) x += y;
  }
  if (lane == kWave - 1) tmp[wave] = x;
  __syncthreads();
  T base = 0, sum = 0;
  for (int w = 0; w < threads / kWave; ++w) {
    if (w < wave) base += tmp[w];
    sum += tmp[w];
  }
  __syncthreads();
  *total = sum;
  return base + x - v;  // exclusive
}

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

// Eight codes to f16, exactly.
template <int KIND>
__device__ __forceinline__ h8 codes_h8(uint32_t lo, uint32_t hi) {
  h8 v;
  if constexpr (KIND == DFS_FP8) {
    const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    v = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
  } else {
    // byte b ^ 0x80 = b + 128 under the exponent of 1024: 1152 + b, exactly
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    u4 w;
    w.x = __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u);
    w.y = __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u);
    w.z = __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u);
    w.w = __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u);
    v = __builtin_bit_cast(h8, w) - (_Float16)1152.0f;
  }
  return v;
}

// The top bit of each byte that is an E4M3 NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t c) {
  return ((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Parts of an item pass between workgroups of different XCDs, whose L2s are
// not coherent for plain accesses: they are written and read by accesses of
// device scope, which do not stay in an L2, so no cache has to be written back
// or invalidated.  A fence of device scope does both, for the whole L2: with
// fences, 4 drafted tokens over 131071 took 107 us (65 without), a windowed
// decode batch of 24 requests 106 (49), one request of 777 tokens 24 (14.7).
// A part counts as done when its stores have completed (stores_done, then the
// barrier, then the counter).
__device__ __forceinline__ void put2(f2* p, f2 v) {
  __hip_atomic_store((uint64_t*)p, __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f2 get2(const f2* p) {
  return __builtin_bit_cast(f2, __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT));
}
__device__ __forceinline__ void put4(float* p, f4 v) {
  // one store of device scope (there is no builtin of 16 bytes); the wait state
  // keeps the next instruction off its operands
  asm volatile("global_store_dwordx4 %0, %1, off sc1\n\ts_nop 1" ::"v"(p), "v"(v) : "memory");
}
__device__ __forceinline__ f4 get4(const float* p) {
  const f2 a = get2((const f2*)p), b = get2((const f2*)p + 1);
  return f4{a.x, a.y, b.x, b.y};
}
__device__ __forceinline__ void stores_done() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Called by a whole workgroup after its stores: whether it is the last of n.
// That one leaves the counter zero.
__device__ __forceinline__ bool arrive(uint32_t* count, int n, int* last) {
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0) {
    *last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
            (uint32_t)(n - 1);
    if (*last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *last != 0;
}

// Joins n parts of an item: every thread calls put(row, dim, four sums,
// reference of the weights and their sum) for its share of the rows.  ml and o
// are indexed by slot(part) * stride + row.  E places of P parts each are in
// flight at once: the loads go past the L2, so that their latency is what a
// join costs.
constexpr int kJoin = 8;
template <int D, int E, typename F, typename G>
__device__ __forceinline__ void join_by(const f2* ml, const float* o, int stride, int rows, int n,
                                        F slot, G put) {
  constexpr int P = kJoin / E;
  const int places = rows * (D / 4);
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < places; i0 += E * kThreads) {
    float mm[E], l[E];
    f4 v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      mm[e] = -INFINITY;
      l[e] = 0.0f;
      v[e] = f4{0, 0, 0, 0};
    }
#pragma unroll 1
    for (int b = 0; b < n; b += P) {
      f2 pm[E][P];
      f4 po[E][P];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = min(i0 + e * kThreads, places - 1);
        const int row = at / (D / 4), d = at % (D / 4) * 4;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int64_t pr = slot(min(b + i, n - 1)) * stride + row;
          pm[e][i] = get2(ml + pr);
          po[e][i] = get4(o + pr * D + d);
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float mb = mm[e];
#pragma unroll
        for (int i = 0; i < P; ++i) mb = fmaxf(mb, pm[e][i].x);
        const float old = __builtin_amdgcn_exp2f(mm[e] - mb);
        l[e] *= old;
        v[e] *= old;
        mm[e] = mb;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float f = b + i < n ? __builtin_amdgcn_exp2f(pm[e][i].x - mb) : 0.0f;
          l[e] += pm[e][i].y * f;
          v[e] += po[e][i] * f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = i0 + e * kThreads;
      if (at < places) put(at / (D / 4), at % (D / 4) * 4, v[e], f2{mm[e], l[e]});
    }
  }
}
template <int D, typename F, typename G>
__device__ __forceinline__ void join(const f2* ml, const float* o, int stride, int rows, int n,
                                     F slot, G put) {
  if (n <= 2 && rows * (D / 4) > kThreads) join_by<D, 4>(ml, o, stride, rows, n, slot, put);
  else join_by<D, 1>(ml, o, stride, rows, n, slot, put);
}

// Maximum and sum over the four lanes that hold one query row (lane % 16).
__device__ __forceinline__ float max4(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum4(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// SPLIT: the waves of a workgroup take the tiles of an item in turn, all for
// the same NQ * 16 query rows (few rows, long caches).  Otherwise each wave
// has NQ * 16 rows of its own and all take every tile (prompts).
// BIG: a tile lies in one page (pages of 64 or 128 tokens), whose address and
// scales are then the same for all lanes.
template <int KIND, int D, int NQ, bool SPLIT, bool F32, bool BIG>
struct Attn {
  // what an item costs besides its tiles, in tiles (see make_plan): its first
  // reads and its results (32 requests to 8192 tokens: 202 us where items
  // counted by tiles alone, 191 so; one of 777 tokens: 14.1, 10.5; prompts
  // under a window of 512: 74, 64)
  static constexpr int kExtra = SPLIT ? 4 : 3;
  static constexpr int kRows = 16 * NQ;                      // per wave
  static constexpr int kQb = SPLIT ? kRows : kRows * kWaves;  // per item
  static constexpr int kSteps = D / 32;                      // first product, per key group
  static constexpr int kDims = D / 16;                       // 16-dim groups of the second
  static constexpr int kWide = D / 64;                       // 16-byte pieces of a lane's K row

  struct Shared {
    union {
      float o[SPLIT ? kWaves * kRows * D : 1];  // each wave's sums
      int64_t tmp[kWaves];
    };
    float m[kWaves][kRows], l[kWaves][kRows];
    int last;
    int32_t longest;
    int64_t first[kInlinePlan + 1];
    int32_t req[kInlinePlan], qblk[kInlinePlan];
    Req facts[kInlinePlan];
  };

  // one wave's state
  h8 qf[NQ][kSteps];
  f4 o[NQ][kDims];
  float m[NQ], l[NQ];
  float c[NQ];  // o is in units of 2^(c - 13), l of 2^(m - 13); whole numbers, so
                // that what they put into exponents and factors is exact
  uint32_t kraw[4][D / 16];  // K codes of the tile to come
  float ks, vs;              // and the scales of this lane's key block in it
  // pages of a tile: of this lane's K rows, and of its key block
  struct Pages {
    int k, v;
  } pg0, pg1;  // of that tile, and of the one after it

  const KvAttnLaunch& a;
  const int lane, wave, r16, q4;
  const bool wide;  // whether O takes four elements at once
  Req rq;
  Span sp;
  int kh, row0, nrows;      // this wave's first row of the request, its rows (may be <= 0)
  int pos[NQ], pmin, pmax;  // positions of the rows
  const int32_t* tab;

  __device__ __forceinline__ Attn(const KvAttnLaunch& a_)
      : a(a_), lane(threadIdx.x % kWave), wave(uni(threadIdx.x / kWave)), r16(lane & 15),
        q4(lane >> 4),
        wide((uintptr_t)a_.O % (F32 ? 16 : 8) == 0 && a_.ldo % 4 == 0) {}

  __device__ __forceinline__ Pages load_pages(int u) const {
    const int kb = sp.tile(u) * kTile;
    const int sh = __builtin_ctz(a.kv.page);
    const int last = a.b.table_pages - 1;
    if constexpr (BIG) {
      const int pg = *gptr(tab + min(kb >> sh, last));
      return {pg, pg};
    }
    return {*gptr(tab + min((kb + 16 * (r16 >> 2)) >> sh, last)),
            *gptr(tab + min((kb + 16 * q4) >> sh, last))};
  }
  // Pages that have arrived.
  static __device__ __forceinline__ Pages settle(Pages p) {
    return BIG ? Pages{uni(p.k), uni(p.v)} : p;
  }
  // A page that is none is read as page 0 and masked.
  __device__ __forceinline__ bool valid(int pg) const { return pg >= 0 && pg < a.kv.n_pages; }

  // K codes and the scales of tile u; if there is none (!real) every lane
  // reads the same bytes at the start of the cache, which costs nothing.
  __device__ __forceinline__ void load_k(int u, bool real) {
    const int kb = sp.tile(u) * kTile;
    const int P = a.kv.page;
    const int pg = valid(pg0.k) ? pg0.k : 0;
    const uint8_t* base = a.kv.k;
    uint32_t off = 0;  // of this lane
    if constexpr (BIG) {
      base += (((int64_t)pg * a.kv.heads + kh) * P + (kb & (P - 1))) * D;
      off = real ? (16 * (r16 >> 2) + (r16 & 3)) * D + q4 * 16 : 0;
    } else {
      const int64_t at = (((int64_t)pg * a.kv.heads + kh) * P + ((kb + 16 * (r16 >> 2)) & (P - 1)) +
                          (r16 & 3)) * D + q4 * 16;
      base += real ? at : 0;
    }
    const int q8 = real ? 8 * q4 : 0;
#pragma unroll
    for (int mm = 0; mm < 4; ++mm) {
      const uint8_t* p = base + 4 * mm * D;
#pragma unroll
      for (int c = 0; c < kWide; ++c) {
        const u4 w = ld16<u4>(p + off + 64 * c);
        kraw[mm][4 * c] = w.x;
        kraw[mm][4 * c + 1] = w.y;
        kraw[mm][4 * c + 2] = w.z;
        kraw[mm][4 * c + 3] = w.w;
      }
      if constexpr (D % 64 != 0) {
        const u2 w = *gptr((const u2*)(p + off + 64 * kWide - q8));
        kraw[mm][4 * kWide] = w.x;
        kraw[mm][4 * kWide + 1] = w.y;
      }
    }
    const int64_t ph = (int64_t)(valid(pg0.v) ? pg0.v : 0) * a.kv.heads + kh;
    ks = *gptr(a.kv.kscale + ph);
    vs = *gptr(a.kv.vscale + ph);
  }

  __device__ __forceinline__ void begin(const Req& facts, int req, int qblk, int kh_) {
    const int g = a.q_heads / a.kv.heads;
    kh = kh_;
    rq = {uni(facts.t0), uni(facts.n), uni(facts.len), uni(facts.keys)};
    tab = a.b.table + (int64_t)req * a.b.ldt;
    const int rows = rq.n * g;  // < 2^31: n_tok rows of q_heads * head_dim elements exist
    const int item0 = qblk * kQb, item1 = min(item0 + kQb, rows);
    row0 = item0 + (SPLIT ? 0 : wave * kRows);
    nrows = min(item1 - row0, kRows);
    const int pos0 = rq.len - rq.n;
    sp = get_span(rq, pos0 + item0 / g, pos0 + (item1 - 1) / g, a.window, a.sinks);
    pmin = pos0 + min(row0, item1 - 1) / g;
    pmax = pos0 + (min(row0 + kRows, item1) - 1) / g;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      // rows past the end repeat the last one and are not written
      const int row = min(row0 + 16 * i + r16, item1 - 1);
      const int tok = row / g, h = kh * g + row - tok * g;
      pos[i] = pos0 + tok;
      const _Float16* qp = a.Q + (int64_t)(rq.t0 + tok) * a.ldq + (int64_t)h * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d = s < 2 * kWide ? (s >> 1) * 64 + q4 * 16 + (s & 1) * 8 : 64 * kWide + q4 * 8;
        qf[i][s] = ld16<h8>(qp + d);
      }
      m[i] = c[i] = -1e30f;
      l[i] = 0.0f;
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[i][d] = f4{0, 0, 0, 0};
    }
  }

  // Bits of this lane's 16 keys, from j0 on, that lie below key `end`.
  static __device__ __forceinline__ uint32_t below(int end, int j0) {
    return (1u << min(max(end - j0, 0), 16)) - 1u;
  }
  // Bits of the keys from j0 on that a row whose window starts at `low` and
  // whose keys end before `high` sees.
  __device__ __forceinline__ uint32_t seen(int low, int high, int j0) const {
    return below(high, j0) & (~below(low, j0) | below(a.sinks, j0));
  }
  // First key of the window of a row at position p.
  __device__ __forceinline__ int window_low(int p) const {
    return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
  }

  // What some row of the wave sees of this lane's 16 keys from j0 on, in page pv.
  __device__ __forceinline__ uint32_t seen_by_any(int pv, int j0) const {
    return valid(pv) ? seen(window_low(pmin), min(pmax + 1, rq.keys), j0) : 0u;
  }
  // This lane's V codes of the tile that starts at key kb: its row of the first
  // 16 dims, and the others 16 P bytes apart.
  __device__ __forceinline__ const uint8_t* v_codes(int kb, int pv, uint32_t& off) const {
    const int P = a.kv.page;
    const int64_t ph = (int64_t)(valid(pv) ? pv : 0) * a.kv.heads + kh;
    const uint8_t* base = a.kv.v + ph * D * P;
    off = r16 * P + 16 * q4;
    if constexpr (BIG) {
      base += kb & (P - 1);
    } else {
      base += off + (((kb + 16 * q4) & (P - 1)) - 16 * q4);
      off = 0;
    }
    return base;
  }

  // Tile u, whose K codes are in kraw.  The tile `next` is loaded meanwhile,
  // and the pages of the tile `after`.  The loads are in the order in which
  // they are waited for, with no branch around them: a wait then leaves the
  // later ones in flight.
  template <bool CAREFUL>
  __device__ __forceinline__ void tile(int u, int next, int after, bool more) {
    const int kb = sp.tile(u) * kTile;
    const int pv = pg0.v;
    u4 vraw[kDims];
    {
      uint32_t off;
      const uint8_t* base = v_codes(kb, pv, off);
#pragma unroll
      for (int d = 0; d < kDims; ++d) vraw[d] = ld16<u4>(base + d * 16 * a.kv.page + off);
    }
    f4 s[NQ][4];
#pragma unroll
    for (int mm = 0; mm < 4; ++mm) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) s[i][mm] = f4{0, 0, 0, 0};
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const h8 kf = codes_h8<KIND>(kraw[mm][2 * st], kraw[mm][2 * st + 1]);
#pragma unroll
        for (int i = 0; i < NQ; ++i)
          s[i][mm] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[i][st], s[i][mm], 0, 0, 0);
      }
    }
    float kscale = ks * (a.sm_scale * kLog2e), vscale = vs;
    pg0 = settle(pg1);
    load_k(next, more);
    pg1 = load_pages(after);
    const bool plain = kb + kTile - 1 <= pmin && kb + kTile <= rq.keys &&
                       (a.window <= 0 || pmax - kb < a.window || kb + kTile <= a.sinks) &&
                       __ballot(!valid(pv) || !(vscale > 0.0f && vscale < INFINITY)) == 0;
    if (!plain) {
      const int j0 = kb + 16 * q4;
      // what some row of the wave sees
      const uint32_t any = seen_by_any(pv, j0);
      if (any == 0) vscale = 0.0f;
      // A scale that is not finite makes NaN of the rows that see a key of its
      // page, by their scores, and of no other.
      const float odd = vscale - vscale;
      if (odd != 0.0f) vscale = 0.0f;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const uint32_t see = any & seen(window_low(pos[i]), pos[i] + 1, j0);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          s[i][x >> 2][x & 3] = see >> x & 1u ? s[i][x >> 2][x & 3] * kscale + odd : -INFINITY;
      }
      kscale = 1.0f;
      // codes of keys that nobody sees may be NaN, and a scale of 0 makes 0 of
      // any code
      const uint32_t used = vscale == 0.0f ? 0u : any;
      u4 keep;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        keep[w] = ((used >> (4 * w) & 15u) * 0x00204081u & 0x01010101u) * 0xFFu;
#pragma unroll
      for (int d = 0; d < kDims; ++d) vraw[d] &= keep;
      if constexpr (CAREFUL) {
#pragma unroll
        for (int d = 0; d < kDims; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t n = nan_codes(vraw[d][x]);
            vraw[d][x] &= ~(n - (n >> 7));
          }
      }
    }
    // vscale = 2^(ve + lf), lf = -inf for a scale of 0.  A lane's keys lie in one
    // page, so that what its scale adds to the weights' exponents goes out of
    // their sum again by one factor.
    const float ve = __builtin_amdgcn_frexp_expf(vscale);
    const float lf =
        __builtin_amdgcn_logf(__builtin_amdgcn_ldexpf(vscale, -__builtin_amdgcn_frexp_expf(vscale)));
    float mx[NQ];
    bool far = false, rescale = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      mx[i] = s[i][0][0];
#pragma unroll
      for (int x = 1; x < 16; ++x) mx[i] = fmaxf(mx[i], s[i][x >> 2][x & 3]);
      mx[i] *= kscale;
      far = far || mx[i] > m[i] + kFar;
    }
    if (__ballot(far) != 0) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const float top = fmaxf(ceilf(max4(mx[i])), m[i]);
        l[i] *= __builtin_amdgcn_exp2f(m[i] - top);
        m[i] = top;
      }
    }
    h8 w[NQ][2], wl[NQ][2];
    float alpha[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const float mo = ceilf(max4(mx[i] + (ve + lf)));
      const bool up = mo > c[i] + kSlack;
      alpha[i] = up ? __builtin_amdgcn_exp2f(c[i] - mo) : 1.0f;
      c[i] = up ? mo : c[i];
      rescale = rescale || up;
      // Contributions below 2^(kFar - kLeast) of the largest may count as that: as
      // f16 they are 0, and the sum of the weights keeps its part of them.
      const float add = fmaxf((ve + kWeightBits - c[i]) + lf, kWeightBits - kLeast - m[i]);
      const float back = __builtin_amdgcn_exp2f((kWeightBits - m[i]) - add);
      float sum = 0.0f;
#pragma unroll
      for (int x = 0; x < 16; ++x)
        s[i][x >> 2][x & 3] =
            __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][x >> 2][x & 3], kscale, add));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 0; x < 8; x += 2) {
          const f2 p = {s[i][2 * h + (x >> 2)][x & 3], s[i][2 * h + (x >> 2)][(x & 3) + 1]};
          const h2 hi = __builtin_convertvector(p, h2);
          w[i][h][x] = hi.x;
          w[i][h][x + 1] = hi.y;
          const f2 rest = {p.x - (float)hi.x, p.y - (float)hi.y};
          const h2 lo = __builtin_convertvector(rest, h2);
          wl[i][h][x] = lo.x;
          wl[i][h][x + 1] = lo.y;
          sum += p.x + p.y;
        }
      }
      l[i] = __builtin_fmaf(sum, back, l[i]);
    }
    if (__ballot(rescale) != 0) {
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int d = 0; d < kDims; ++d) o[i][d] *= alpha[i];
    }
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
      const h8 v0 = codes_h8<KIND>(vraw[d].x, vraw[d].y);
      const h8 v1 = codes_h8<KIND>(vraw[d].z, vraw[d].w);
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w[i][0], o[i][d], 0, 0, 0);
        o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w[i][1], o[i][d], 0, 0, 0);
        o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, wl[i][0], o[i][d], 0, 0, 0);
        o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, wl[i][1], o[i][d], 0, 0, 0);
      }
    }
  }

  // The sum of a row's weights over its four lanes, in units (2^m from here on)
  // that bring it to 1/2 .. 1, and o in the same.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      l[i] = sum4(l[i]);
      const int e = __builtin_amdgcn_frexp_expf(l[i]);
      l[i] = __builtin_amdgcn_ldexpf(l[i], -e);
      const int by = (int)fmaxf(c[i] - m[i], -1000.0f) - e;
      m[i] += (float)e - kWeightBits;
#pragma unroll
      for (int d = 0; d < kDims; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          o[i][d][x] = __builtin_amdgcn_ldexpf(o[i][d][x], by);
    }
  }

  // tiles u0, u0 + step, ... below u1
  template <bool CAREFUL>
  __device__ __forceinline__ void tiles(int u0, int u1, int step) {
    if (u0 >= u1) return;
    const int last = u0 + (u1 - 1 - u0) / step * step;
    pg0 = settle(load_pages(u0));
    pg1 = load_pages(min(u0 + step, last));
    load_k(u0, true);
    for (int u = u0; u <= last; u += step)
      tile<CAREFUL>(u, min(u + step, last), min(u + 2 * step, last), u < last);
  }

  // NaN codes of V in a tile that some rows see only in part: a weight of 0 does
  // not keep them out of the rows that do not see their keys.  The sums tell, and
  // cost nothing on the way; where some are NaN, the tiles are taken once more in
  // a careful form, with such codes as 0, and spread_nan makes NaN of the sums
  // that they belong to.  (Looked for in the tiles themselves, they took 3% of
  // the time for prompts and for one short request; so, 0 to 1%.)
  __device__ __forceinline__ bool any_nan() const {
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int d = 0; d < kDims; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x) z = __builtin_fmaf(o[i][d][x], 0.0f, z);
    return __ballot(z != z) != 0;
  }
  // A product of ones counts, for each row and dim, the NaN codes that the row
  // sees; put(i, d) is called where there are some, i the group of rows.  u0, u1
  // and step as for tiles().
  template <typename F>
  __device__ __forceinline__ void spread_nan(int u0, int u1, int step, F put) const {
    stores_done();
#pragma unroll 1
    for (int u = u0; u < u1; u += step) {
      const int kb = sp.tile(u) * kTile, j0 = kb + 16 * q4, pv = settle(load_pages(u)).v;
      const uint32_t any = seen_by_any(pv, j0);
      uint32_t off;
      const uint8_t* base = v_codes(kb, pv, off);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {  // eight of the lane's keys at a time
        const uint32_t some = any >> (8 * h) & 0xFFu;
        h8 w[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const uint32_t see = some & seen(window_low(pos[i]), pos[i] + 1, j0) >> (8 * h);
#pragma unroll
          for (int x = 0; x < 8; ++x) w[i][x] = see >> x & 1u ? (_Float16)1.0f : (_Float16)0.0f;
        }
#pragma unroll 1
        for (int d = 0; d < kDims; ++d) {
          const u2 c = *gptr((const u2*)(base + d * 16 * a.kv.page + off + 8 * h));
          // 0x08 where there is one: 2^-6
          const h8 v = codes_h8<KIND>(nan_codes(c.x) >> 4, nan_codes(c.y) >> 4);
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            const f4 n = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[i], f4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (n[x] > 0.0f) put(i, d * 16 + q4 * 4 + x);
          }
        }
      }
    }
  }

  // One row's destination.
  __device__ __forceinline__ int64_t out_at(int row) const {
    const int g = a.q_heads / a.kv.heads;
    const int tok = row / g, h = kh * g + row - tok * g;
    return (int64_t)(rq.t0 + tok) * a.ldo + (int64_t)h * D;
  }
  using T = typename std::conditional<F32, float, _Float16>::type;
  __device__ __forceinline__ void store_nan(int64_t at) const {
    *gptr_w((T*)a.O + at) = (T)__builtin_nanf("");
  }
  __device__ __forceinline__ void store(int64_t at, const f4& v, float l) const {
    // rows that see nothing are 0; a sum that is NaN stays so
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    typedef T T4 __attribute__((ext_vector_type(4)));
    const T4 w = {(T)(v[0] * inv), (T)(v[1] * inv), (T)(v[2] * inv), (T)(v[3] * inv)};
    if (wide) {
      *gptr_w((T4*)((T*)a.O + at)) = w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) *gptr_w((T*)a.O + at + c) = w[c];
    }
  }
};

template <int KIND, int D, int NQ, bool SPLIT, bool F32, bool BIG>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2)
void attn_kernel(KvAttnLaunch a, AttnWs ws, int least, int slices, int inline_plan) {
  using A = Attn<KIND, D, NQ, SPLIT, F32, BIG>;
  __shared__ typename A::Shared sh;
  A t(a);
  const int n_entries =
      inline_plan ? make_plan<int>(a, A::kQb, A::kExtra, ws.max_entries, sh.first, sh.req, sh.qblk,
                                   sh.facts, &sh.longest, sh.tmp, kThreads)
                  : *gptr(ws.n_entries);
  auto first = [&](int e) { return inline_plan ? sh.first[e] : *gptr(ws.first + e); };
  if (n_entries == 0) return;
  const int64_t total = first(n_entries);
  const int64_t per = max((int64_t)least, (total + slices - 1) / slices);
  const int64_t xs = blockIdx.x * per, xe = min(xs + per, total);
  if (xs >= total) return;
  // the entry e with first(e) <= xs < first(e + 1)
  int e = 0;
  for (int n = n_entries; n > 1;) {
    const int stride = (n + kThreads - 1) / kThreads;
    const int at = (int)threadIdx.x * stride;
    const int below = __syncthreads_count(at < n && first(e + at) <= xs);
    e += (below - 1) * stride;
    n = min(stride, n_entries - e);
  }
  // Items of few tiles are not split: a slice then takes those that start in it,
  // whole.  A part and its join cost as much as some tiles (four prompts of 500
  // tokens, 8 tiles at most: 46 us split, 38 us whole; windows of 512 tokens, 11
  // tiles: 70 us split, 82 us whole).
  const bool keep =
      !SPLIT && uni(inline_plan ? sh.longest : *gptr(ws.n_entries + 1)) <= kWhole;
  for (int64_t x = xs; x < xe;) {
    while (first(e + 1) <= x) ++e;
    const int64_t fe = first(e);
    // an item is its tiles, and then the extra ones
    const int n_line = uni((int)((first(e + 1) - fe) / a.kv.heads)), n_tiles = n_line - A::kExtra;
    const int kh = uni((int)((x - fe) / n_line));
    const int64_t item0 = fe + (int64_t)kh * n_line, item1 = item0 + n_tiles;
    if (keep ? x > item0 : x >= item1) {  // another slice's, or only extra ones are left of it
      x = item0 + n_line;
      continue;
    }
    const int req = uni(inline_plan ? sh.req[e] : *gptr(ws.req + e));
    const int qblk = uni(inline_plan ? sh.qblk[e] : *gptr(ws.qblk + e));
    const int u0 = uni((int)(x - item0)), u1 = uni(keep ? n_tiles : (int)(min(item1, xe) - item0));
    x = u1 == n_tiles ? item0 + n_line : item0 + u1;
    t.begin(inline_plan ? sh.facts[req] : get_req(a.b, a.kv.page, req), req, qblk, kh);
    const int v0 = SPLIT ? u0 + t.wave : u0, step = SPLIT ? kWaves : 1;
    const int v1 = SPLIT || t.nrows > 0 ? u1 : u0;  // this wave's tiles: v0, v0 + step, ... below v1
    t.template tiles<false>(v0, v1, step);
    const bool nans = KIND == DFS_FP8 && t.any_nan();
    if (KIND == DFS_FP8 && nans) {
      t.begin(inline_plan ? sh.facts[req] : get_req(a.b, a.kv.page, req), req, qblk, kh);
      t.template tiles<true>(v0, v1, step);
    }
    t.finish();
    const bool whole = u0 == 0 && u1 == n_tiles;
    // a slice has at most two items that are not whole: its first and its last
    const int64_t slot = 2 * (int64_t)blockIdx.x + (u0 == 0 ? 1 : 0);
    const int rows = min(A::kQb, t.rq.n * (a.q_heads / a.kv.heads) - qblk * A::kQb);
    if constexpr (SPLIT) {
      // join the waves
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int row = 16 * i + t.r16;
        if (row < rows) {
          if (t.q4 == 0) {
            sh.m[t.wave][row] = t.m[i];
            sh.l[t.wave][row] = t.l[i];
          }
#pragma unroll
          for (int d = 0; d < A::kDims; ++d)
            *(f4*)&sh.o[(t.wave * A::kRows + row) * D + d * 16 + t.q4 * 4] = t.o[i][d];
        }
      }
      if (KIND == DFS_FP8 && nans) t.spread_nan(v0, v1, step, [&](int i, int d) {
        sh.o[(t.wave * A::kRows + 16 * i + t.r16) * D + d] = __builtin_nanf("");
      });
      __syncthreads();
      for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kThreads) {
        const int row = idx / (D / 4), d = idx % (D / 4) * 4;
        float mm = sh.m[0][row];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, sh.m[w][row]);
        float l = 0.0f;
        f4 v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(sh.m[w][row] - mm);
          l += sh.l[w][row] * f;
          v += *(f4*)&sh.o[(w * A::kRows + row) * D + d] * f;
        }
        if (whole) {
          t.store(t.out_at(t.row0 + row) + d, v, l);
        } else {
          put4(&ws.part_o[(slot * A::kQb + row) * D + d], v);
          if (d == 0) put2(&ws.part_ml[slot * A::kQb + row], f2{mm, l});
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int row = 16 * i + t.r16;
        if (row < t.nrows) {
          const int64_t at = whole ? t.out_at(t.row0 + row) : 0;
          const int64_t pr = slot * A::kQb + t.wave * A::kRows + row;
#pragma unroll
          for (int d = 0; d < A::kDims; ++d) {
            if (whole) t.store(at + d * 16 + t.q4 * 4, t.o[i][d], t.l[i]);
            else put4(&ws.part_o[pr * D + d * 16 + t.q4 * 4], t.o[i][d]);
          }
          if (!whole && t.q4 == 0) put2(&ws.part_ml[pr], f2{t.m[i], t.l[i]});
        }
      }
      if (KIND == DFS_FP8 && nans)
        t.spread_nan(v0, v1, step, [&](int i, int d) {
          const int row = 16 * i + t.r16;
          if (row >= t.nrows) return;
          if (whole) {
            t.store_nan(t.out_at(t.row0 + row) + d);
          } else {
            const int64_t pr = slot * A::kQb + t.wave * A::kRows + row;
            __hip_atomic_store(&ws.part_o[pr * D + d], __builtin_nanf(""), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
          }
        });
    }
    if (!whole) {
      // The parts of an item are joined in groups of kJoin slices, each by the
      // slice of the group that comes last, then the groups' results by the
      // group that comes last: always in slice order.
      const int w0 = (int)(item0 / per), w1 = (int)((item1 - 1) / per);
      const int me = (int)blockIdx.x - w0;
      const int groups = (w1 - w0) / kJoin + 1, grp = me / kJoin;
      const int g0 = w0 + grp * kJoin, g1 = min(g0 + kJoin - 1, w1);
      // the item starts in slice w0 as that slice's last item (slot 1), and is
      // the first one of the others
      auto slot_of = [&](int w) { return 2 * (int64_t)w + (w == w0); };
      if (arrive(&ws.count[slot_of(g0)], g1 - g0 + 1, &sh.last)) {
        join<D>(ws.part_ml, ws.part_o, A::kQb, rows, g1 - g0 + 1,
                [&](int i) { return slot_of(g0 + i); }, [&](int row, int d, const f4& v, f2 ml) {
                  if (groups == 1) {
                    t.store(t.out_at(qblk * A::kQb + row) + d, v, ml.y);
                  } else {
                    const int64_t pr = slot_of(g0) * A::kQb + row;
                    put4(ws.part_o + pr * D + d, v);
                    if (d == 0) put2(ws.group_ml + pr, ml);
                  }
                });
        if (groups > 1 && arrive(&ws.count[2 * gridDim.x + w0], groups, &sh.last))
          join<D>(ws.group_ml, ws.part_o, A::kQb, rows, groups,
                  [&](int i) { return slot_of(w0 + i * kJoin); },
                  [&](int row, int d, const f4& v, f2 ml) {
                    t.store(t.out_at(qblk * A::kQb + row) + d, v, ml.y);
                  });
      }
    }
    __syncthreads();
  }
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
  const AttnWs w = {(uint32_t*)p,          (int64_t*)(p + l.first), (int32_t*)(p + l.req),
                    (int32_t*)(p + l.qblk), (int32_t*)(p + l.n),     (int32_t)c.entries,
                    (float*)(p + l.part_o), (f2*)(p + l.part_ml),
                    (f2*)(p + l.group_ml)};
  if (a.kv.dtype == DFS_FP8) go_kind<DFS_FP8>(a, w, c, s);
  else go_kind<DFS_INT8>(a, w, c, s);
  return hipGetLastError();
}

}  // namespace dfs
