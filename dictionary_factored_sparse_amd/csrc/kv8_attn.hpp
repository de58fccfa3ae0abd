// kv8_attn.hpp -- the attention of query rows over tiles of the 8-bit paged
// cache, and lines of such work cut into equal slices; shared by kv8_attention
// and kv8_prefix_attention.
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
#pragma once

#include <algorithm>
#include <type_traits>

#include "dfs_internal.hpp"

namespace dfs {
namespace {


constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 64;                // keys per tile
constexpr int kCounterBytes = 65536;     // counters at the start of the workspace
constexpr int kWhole = 8;                // tiles up to which an item of a prompt is not split
constexpr float kWeightBits = 13.0f;     // weights are held at 2^13 times their value
constexpr float kSlack = 2.0f;           // the reference of the sums may lag by this (log2),
constexpr float kFar = 32.0f;            // that of the weights' own sum by this
constexpr float kLeast = 72.0f;          // 2^(13 + kFar - kLeast) is 0 in f16, 2^(13 - kLeast) far
                                         // above the least normal fp32
constexpr float kLog2e = 1.44269504088896340736f;

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

// Tiles that some row of an entry sees: the first `ns` tiles, from tile `t0` on,
// hold first tokens, the others run from tile `ta`.
struct Span {
  int t0, ns, ta, n;
  __device__ __forceinline__ int tile(int u) const { return u < ns ? t0 + u : u - ns + ta; }
};
__device__ __forceinline__ Span get_span(const Req& q, int p0, int p1, int window, int sinks,
                                         int from = 0) {
  Span s;
  const int hi = min(p1, q.keys - 1);                                // last visible key
  const int lo = max(window > 0 && p0 >= window ? p0 - window + 1 : 0, from);  // first of the window
  const int sk = min(sinks, hi + 1);
  s.t0 = from / kTile;
  s.ta = lo / kTile;
  s.ns = sk > from ? min((sk - 1) / kTile + 1, s.ta) - s.t0 : 0;
  s.n = s.ns + (hi >= lo ? hi / kTile - s.ta + 1 : 0);
  if (s.n <= 0) {  // rows that see nothing still get their zeros
    s.ns = 0;
    s.ta = s.t0;
    s.n = 1;
  }
  return s;
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

// p - hi, rounded to f16: one instruction an element, where the compiler takes two
// conversions and a difference (the prompts below 255 us so, 252; a document of 65500
// tokens for 24 requests 89 us, 87).
__device__ __forceinline__ h2 rest(h2 hi, f2 p) {
  uint32_t r;
  const uint32_t x = __builtin_bit_cast(uint32_t, hi);
  asm("v_fma_mixlo_f16 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixhi_f16 %0, %1, -1.0, %3 op_sel:[1,0,0] op_sel_hi:[1,0,0]"
      : "=&v"(r) : "v"(x), "v"(p.x), "v"(p.y));
  return __builtin_bit_cast(h2, r);
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
// The same of two numbers that are not a pair: made as whole numbers, for else the
// arrays that they come from are kept in memory.
__device__ __forceinline__ void put2(f2* p, float x, float y) {
  const uint64_t v = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
  __hip_atomic_store((uint64_t*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
  static constexpr bool kSplit = SPLIT, kNan = KIND == DFS_FP8;  // kNan: codes may be NaN
  static constexpr bool kJoinHere = true;
  static constexpr int kEach = 0;          // items of at most so many tiles are dealt out whole
  static constexpr int kKeep = SPLIT ? 0 : kWhole;  // or taken whole by the slice they start in
  static constexpr int kD = D, kNq = NQ;
  static constexpr int kRows = 16 * NQ;                      // per wave
  static constexpr int kQb = SPLIT ? kRows : kRows * kWaves;  // per item
  static constexpr int kSteps = D / 32;                      // first product, per key group
  static constexpr int kDims = D / 16;                       // 16-dim groups of the second
  static constexpr int kWide = D / 64;                       // 16-byte pieces of a lane's K row

  struct Work {
    float o[SPLIT ? kWaves * kRows * D : 1];  // each wave's sums
    float m[kWaves][kRows], l[kWaves][kRows];
    int last;
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

  // The item of block qblk of `facts`' rows and kv head kh_, over the keys from
  // `from` on in the pages of row `req` of the table.
  __device__ __forceinline__ void begin(const Req& facts, int req, int qblk, int kh_, int from = 0) {
    begin_by<false>(facts, req, qblk, kh_, from, 0, 0, [&](int tok) { return rq.len - rq.n + tok; });
  }
  // The same where pos_of(token) is a token's position, p0 the lowest of them all
  // and p1 the highest (ANY: they do not ascend).
  template <bool ANY, typename P>
  __device__ __forceinline__ void begin_by(const Req& facts, int req, int qblk, int kh_, int from, int p0,
                                           int p1, P pos_of) {
    const int g = a.q_heads / a.kv.heads;
    kh = kh_;
    rq = {uni(facts.t0), uni(facts.n), uni(facts.len), uni(facts.keys)};
    tab = a.b.table + (int64_t)req * a.b.ldt;
    const int rows = rq.n * g;  // < 2^31: n_tok rows of q_heads * head_dim elements exist
    const int item0 = qblk * kQb, item1 = min(item0 + kQb, rows);
    row0 = item0 + (SPLIT ? 0 : wave * kRows);
    nrows = min(item1 - row0, kRows);
    if constexpr (!ANY) {
      sp = get_span(rq, pos_of(item0 / g), pos_of((item1 - 1) / g), a.window, a.sinks, from);
      pmin = pos_of(min(row0, item1 - 1) / g);
      pmax = pos_of((min(row0 + kRows, item1) - 1) / g);
    } else {
      sp = get_span(rq, p0, p1, a.window, a.sinks, from);
      pmin = INT32_MAX;
      pmax = INT32_MIN;
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      // rows past the end repeat the last one and are not written
      const int row = min(row0 + 16 * i + r16, item1 - 1);
      const int tok = row / g, h = kh * g + row - tok * g;
      pos[i] = pos_of(tok);
      if constexpr (ANY) {
        pmin = min(pmin, pos[i]);
        pmax = max(pmax, pos[i]);
      }
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
    if constexpr (ANY) {  // the same for all rows of the wave
#pragma unroll
      for (int s = 1; s < 16; s <<= 1) {
        pmin = min(pmin, __shfl_xor(pmin, s, kWave));
        pmax = max(pmax, __shfl_xor(pmax, s, kWave));
      }
      pmin = uni(pmin);
      pmax = uni(pmax);
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
    float alpha[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const float mo = ceilf(max4(mx[i] + (ve + lf)));
      const bool up = mo > c[i] + kSlack;
      alpha[i] = up ? __builtin_amdgcn_exp2f(c[i] - mo) : 1.0f;
      c[i] = up ? mo : c[i];
      rescale = rescale || up;
    }
    if (__ballot(rescale) != 0) {
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int d = 0; d < kDims; ++d) o[i][d] *= alpha[i];
    }
    h8 w[NQ][2], wl[NQ][2];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
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
          const h2 lo = rest(hi, p);
          wl[i][h][x] = lo.x;
          wl[i][h][x + 1] = lo.y;
          sum += p.x + p.y;
        }
      }
      l[i] = __builtin_fmaf(sum, back, l[i]);
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


// The parts of a line's items, two to a slice: slot 2 w + 1 for the last item of
// slice w, 2 w for its first one.
struct Line {
  uint32_t* count;  // [3 * slices]: parts of a group that are done, groups of an item
  float* part_o;    // [2 * slices][rows][D]
  f2* part_ml;      // [2 * slices][rows]: reference of the weights, their sum
  f2* group_ml;     // the same of a group of slices, at its first slice's slot
};

// A part, for this kernel's other workgroups or for a later kernel.
template <typename A>
__device__ __forceinline__ void put_part(float* p, const f4& v) {
  if constexpr (A::kJoinHere) put4(p, v);
  else *gptr_w((f4*)p) = v;
}
template <typename A>
__device__ __forceinline__ void put_part(f2* p, float x, float y) {
  if constexpr (A::kJoinHere) put2(p, x, y);
  else *gptr_w((uint64_t*)p) = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
}

// Slice `slice` of a line of items.  A is an Attn that knows its line as well:
// first(e) is the line's position where entry e starts (a plan has made it),
// first(n_entries) its end; longest() the most tiles an item has; ready(e, kv head)
// readies t for an item and returns its block of rows; the rows that are complete
// go to at(row of the entry's requests), by put(at, dim, four sums, reference of
// the weights, their sum) and put_nan(at, dim).  Where A::kJoinHere, the parts of an
// item are joined as they come; else they stay where they are for a later kernel.
template <typename A>
__device__ __forceinline__ void run_line(A& t, typename A::Work& sh, const Line& ln, int n_entries, int least,
                                         int slice, int slices) {
  if (n_entries == 0) return;
  const bool each = A::kEach > 0 && t.longest() <= A::kEach;
  const int64_t total = t.first(n_entries);
  const int64_t per = max((int64_t)least, (total + slices - 1) / slices);
  const int64_t xs = each ? slice : slice * per;
  const int64_t xe = each ? (int64_t)n_entries * t.a.kv.heads : min(xs + per, total);
  if (xs >= (each ? xe : total)) return;
  // the entry e with first(e) <= xs < first(e + 1)
  int e = 0;
  for (int n = each ? 1 : n_entries; n > 1;) {
    const int stride = (n + kThreads - 1) / kThreads;
    const int at = (int)threadIdx.x * stride;
    const int below = __syncthreads_count(at < n && t.first(e + at) <= xs);
    e += (below - 1) * stride;
    n = min(stride, n_entries - e);
  }
  // Items of few tiles are not split: a slice then takes those that start in it,
  // whole.  A part and its join cost as much as some tiles (four prompts of 500
  // tokens, 8 tiles at most: 46 us split, 38 us whole; windows of 512 tokens, 11
  // tiles: 70 us split, 82 us whole).
  const bool keep = A::kKeep > 0 && t.longest() <= A::kKeep;
  for (int64_t x = xs; x < xe;) {
    if (each) e = (int)(x / t.a.kv.heads);
    else
      while (t.first(e + 1) <= x) ++e;
    const int64_t fe = t.first(e);
    // an item is its tiles, and then the extra ones
    const int n_line = uni((int)((t.first(e + 1) - fe) / t.a.kv.heads)), n_tiles = n_line - A::kExtra;
    const int kh = uni(each ? (int)(x % t.a.kv.heads) : (int)((x - fe) / n_line));
    const int64_t item0 = fe + (int64_t)kh * n_line, item1 = item0 + n_tiles;
    if (!each && (keep ? x > item0 : x >= item1)) {  // another slice's, or only extra ones are left of it
      x = item0 + n_line;
      continue;
    }
    const int u0 = uni(each ? 0 : (int)(x - item0));
    const int u1 = uni(each || keep ? n_tiles : (int)(min(item1, xe) - item0));
    if (each) x += slices;
    else x = u1 == n_tiles ? item0 + n_line : item0 + u1;
    const int qblk = t.ready(e, kh);
    const int v0 = A::kSplit ? u0 + t.wave : u0, step = A::kSplit ? kWaves : 1;
    const int v1 = A::kSplit || t.nrows > 0 ? u1 : u0;  // this wave's tiles: v0, v0 + step, ... below v1
    t.template tiles<false>(v0, v1, step);
    const bool nans = A::kNan && t.any_nan();
    if (A::kNan && nans) {
      t.ready(e, kh);
      t.template tiles<true>(v0, v1, step);
    }
    t.finish();
    const bool whole = u0 == 0 && u1 == n_tiles;
    // a slice has at most two items that are not whole: its first and its last
    const int64_t slot = 2 * (int64_t)slice + (u0 == 0 ? 1 : 0);
    const int rows = min(A::kQb, t.rq.n * (t.a.q_heads / t.a.kv.heads) - qblk * A::kQb);
    if constexpr (A::kSplit) {
      // join the waves
#pragma unroll
      for (int i = 0; i < A::kNq; ++i) {
        const int row = 16 * i + t.r16;
        if (row < rows) {
          if (t.q4 == 0) {
            sh.m[t.wave][row] = t.m[i];
            sh.l[t.wave][row] = t.l[i];
          }
#pragma unroll
          for (int d = 0; d < A::kDims; ++d)
            *(f4*)&sh.o[(t.wave * A::kRows + row) * A::kD + d * 16 + t.q4 * 4] = t.o[i][d];
        }
      }
      if (A::kNan && nans) t.spread_nan(v0, v1, step, [&](int i, int d) {
        sh.o[(t.wave * A::kRows + 16 * i + t.r16) * A::kD + d] = __builtin_nanf("");
      });
      __syncthreads();
      for (int idx = threadIdx.x; idx < rows * (A::kD / 4); idx += kThreads) {
        const int row = idx / (A::kD / 4), d = idx % (A::kD / 4) * 4;
        float mm = sh.m[0][row];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, sh.m[w][row]);
        float l = 0.0f;
        f4 v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(sh.m[w][row] - mm);
          l += sh.l[w][row] * f;
          v += *(f4*)&sh.o[(w * A::kRows + row) * A::kD + d] * f;
        }
        if (whole) {
          t.put(t.at(t.row0 + row), d, v, mm, l);
        } else {
          put_part<A>(&ln.part_o[(slot * A::kQb + row) * A::kD + d], v);
          if (d == 0) put_part<A>(&ln.part_ml[slot * A::kQb + row], mm, l);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < A::kNq; ++i) {
        const int row = 16 * i + t.r16;
        if (row < t.nrows) {
          const int64_t at = whole ? t.at(t.row0 + row) : 0;
          const int64_t pr = slot * A::kQb + t.wave * A::kRows + row;
#pragma unroll
          for (int d = 0; d < A::kDims; ++d) {
            if (whole) t.put(at, d * 16 + t.q4 * 4, t.o[i][d], t.m[i], t.l[i]);
            else put_part<A>(&ln.part_o[pr * A::kD + d * 16 + t.q4 * 4], t.o[i][d]);
          }
          if (!whole && t.q4 == 0) put_part<A>(&ln.part_ml[pr], t.m[i], t.l[i]);
        }
      }
      if (A::kNan && nans)
        t.spread_nan(v0, v1, step, [&](int i, int d) {
          const int row = 16 * i + t.r16;
          if (row >= t.nrows) return;
          if (whole) {
            t.put_nan(t.at(t.row0 + row), d);
          } else {
            const int64_t pr = slot * A::kQb + t.wave * A::kRows + row;
            __hip_atomic_store(&ln.part_o[pr * A::kD + d], __builtin_nanf(""), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
          }
        });
    }
    if (A::kJoinHere && !whole) {
      // The parts of an item are joined in groups of kJoin slices, each by the
      // slice of the group that comes last, then the groups' results by the
      // group that comes last: always in slice order.
      const int w0 = (int)(item0 / per), w1 = (int)((item1 - 1) / per);
      const int me = slice - w0;
      const int groups = (w1 - w0) / kJoin + 1, grp = me / kJoin;
      const int g0 = w0 + grp * kJoin, g1 = min(g0 + kJoin - 1, w1);
      // the item starts in slice w0 as that slice's last item (slot 1), and is
      // the first one of the others
      auto slot_of = [&](int w) { return 2 * (int64_t)w + (w == w0); };
      if (arrive(&ln.count[slot_of(g0)], g1 - g0 + 1, &sh.last)) {
        join<A::kD>(ln.part_ml, ln.part_o, A::kQb, rows, g1 - g0 + 1,
                [&](int i) { return slot_of(g0 + i); }, [&](int row, int d, const f4& v, f2 ml) {
                  if (groups == 1) {
                    t.put(t.at(qblk * A::kQb + row), d, v, ml.x, ml.y);
                  } else {
                    const int64_t pr = slot_of(g0) * A::kQb + row;
                    put4(ln.part_o + pr * A::kD + d, v);
                    if (d == 0) put2(ln.group_ml + pr, ml);
                  }
                });
        if (groups > 1 && arrive(&ln.count[2 * slices + w0], groups, &sh.last))
          join<A::kD>(ln.group_ml, ln.part_o, A::kQb, rows, groups,
                  [&](int i) { return slot_of(w0 + i * kJoin); },
                  [&](int row, int d, const f4& v, f2 ml) {
                    t.put(t.at(qblk * A::kQb + row), d, v, ml.x, ml.y);
                  });
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace dfs
