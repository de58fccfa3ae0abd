// beam_select.hip -- the next beams of beam search: of the width * vocab
// continuations of a request, the `width` best.
//
// total(w, v) = score_w + x_wv - lse_w, lse_w = m_w + log sum_v 2^((x_wv - m_w) log2 e),
// ranked by total * norm_w.
//
// One launch, one pass over the logits.  A wave takes a part of a row, a step of 8
// or 32 elements a lane at a time with the next step's loads on their way, sums the
// exponentials and keeps what may be among the part's `width` largest elements
// (within a row the order of the totals is that of the logits); there is no barrier
// on the way.  The workgroup that comes last of a request's joins the sums and picks
// from what the parts offer.
//
// The largest elements of a part.  The width-th largest of the lanes' maxima of the
// first step bounds the width-th largest element from below; it takes 20 steps of a
// compare and a count of the lanes, no memory.  The elements above the bound go to a
// list in LDS; where it fills, the same count over the list raises the bound.  In the
// end what reaches the list's width-th largest is ranked by broadcasts of registers.
// (Ranking a list by reads of LDS took 330 us for 256 rows of 131072 and width 32.)
// If too many are equal for that, the elements are taken one by one, from memory.
//
// What bounds it.  Many rows: the exponentials, bounds and lists of the pass (120 rows of
// 50021 in fp32 19.6 us, 1.2 TB/s), and for wide beams also the choice, by one
// workgroup a request (256 rows of 131072 in f16, 32 beams, 45 us, 1.5 TB/s; a read of
// them takes 14).  Few rows: the chain of reads, sums, arrival and choice (4 rows of
// 32000 in f16 11.9 us).
//
// Precision.  Beams of different rows compete by sums that may be close: the
// exponentials, with the rounding error of their arguments put back in, are added
// in pairs in 32 bits and from there on in 64, and totals are compared in 64 bits.
#include <algorithm>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kList = 512;
constexpr size_t kCounterBytes = 65536;
static_assert(2 * kMaxBeamRows * 4 == kCounterBytes, "counters");
constexpr uint32_t kNone = 0x007FFFFFu;  // key of -inf: no continuation

struct BeamWs {
  uint32_t* count;  // [kMaxBeamRows]: rows of each request that are done; then workgroups of each row
  uint64_t* part;   // [rows][chunks][waves]: key of the reference, sum of the exponentials
  uint64_t* cand;   // [rows][chunks][width]: key of a logit, complement of its token
};

// Keys whose order is the values'.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  return __longlong_as_double((int64_t)(k ^ ((uint64_t)((int64_t)~k >> 63) | 0x8000000000000000ull)));
}

// The largest t, of bits kLow and above, that at least n lanes of the wave reach (0
// where fewer have a key): eleven bits of a number's fraction bound closely enough.
constexpr int kLow = 12, kLow64 = 9;  // of a float's key, of the upper half of a double's
template <int LOW>
__device__ __forceinline__ uint32_t nth_largest(uint32_t k, int n) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= LOW; --b) {
    const uint32_t u = t | 1u << b;
    if (__popcll(__ballot(k >= u)) >= n) t = u;
  }
  return t;
}
// The same of a list's `many` keys, f(i) being key i.
template <int LOW, int PER, typename F>
__device__ __forceinline__ uint32_t nth_of(int many, int n, F f) {
  const int lane = threadIdx.x % kWave;
  uint32_t k[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) k[j] = lane + j * kWave < many ? f(lane + j * kWave) : 0;
  uint32_t t = 0;
#pragma unroll 1
  for (int b = 31; b >= LOW; --b) {
    const uint32_t u = t | 1u << b;
    int c = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c += __popcll(__ballot(k[j] >= u));
    if (c >= n) t = u;
  }
  return t;
}
template <int LOW, typename F>
__device__ __forceinline__ uint32_t nth_of_list(int many, int n, F f) {
  if (many <= kWave) return 0;  // all of them can be ranked
  return many <= 4 * kWave ? nth_of<LOW, 4>(many, n, f) : nth_of<LOW, kList / kWave>(many, n, f);
}
// The first 64 of the list's places whose key reaches t, in order, to `to`; how many
// do.  By one wave.
template <typename F>
__device__ __forceinline__ int gather(int many, uint32_t t, F f, int* to) {
  const int lane = threadIdx.x % kWave;
  int m = 0;
  for (int i0 = 0; i0 < many; i0 += kWave) {
    const int i = i0 + lane;
    const bool hit = i < many && f(i) >= t;
    const uint64_t mask = __ballot(hit);
    const int at = m + __popcll(mask & ((1ull << lane) - 1));
    if (hit && at < kWave) to[at] = i;
    m += __popcll(mask);
  }
  return m;
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ uint64_t lane_of(uint64_t v, int l) {
  return (uint64_t)lane_of((uint32_t)(v >> 32), l) << 32 | lane_of((uint32_t)v, l);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, kWave));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// One candidate of a request: its rank key, row and element.
struct Cand {
  uint64_t key;   // of the ranked total
  uint64_t elem;  // key of the logit, then the complement of its token
  uint32_t row;   // of the request
  __device__ __forceinline__ bool above(const Cand& o) const {
    if (key != o.key) return key > o.key;
    if (row != o.row) return row < o.row;
    return elem > o.elem;
  }
};

constexpr int kPart = 256;  // entries of a wave's list
struct Shared {
  uint32_t bound[kWaves];
  int n, last, picked;
  int pick[kWave], rank[kWaves][kWave];
  union {
    struct {
      uint64_t list[kPart], best[kMaxBeams];
      int many, pick[kWave];
    } part[kWaves];
    struct {
      double lse[kMaxBeams], score[kMaxBeams], norm[kMaxBeams];
      int state[kMaxBeams];  // 0: no continuation, 1: its logits', 2: its eos
      uint64_t key[kList], elem[kList];
      uint32_t row[kList];
      Cand top[kWaves];
    } f;
  };
};

// What a wave has written to LDS, its lanes may read.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void put(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether a row offers continuations, and which: its three facts are read at once.
struct RowFacts {
  float score, norm;
  int done;
  __device__ __forceinline__ RowFacts(const BeamLaunch& a, int64_t row)
      : score(*gptr(a.score + row)), norm(a.norm ? *gptr(a.norm + row) : 1.0f),
        done(a.done ? *gptr(a.done + row) : 0) {}
  __device__ __forceinline__ int state() const {
    const bool fine = score > -INFINITY && score < INFINITY && norm > 0.0f && norm < INFINITY;
    return !fine ? 0 : done != 0 ? 2 : 1;
  }
};

// Adds a piece's sum (in units of its largest exponential) to another.
__device__ __forceinline__ void join_sums(uint32_t& top, double& sum, uint32_t k, double s) {
  if (k <= kNone) return;
  const uint32_t m = max(top, k);
  if (top <= kNone) {
    sum = s;
  } else {
    const double f = exp((double)value_of(min(top, k)) - (double)value_of(m));
    sum = m == top ? sum + s * f : sum * f + s;
  }
  top = m;
}

// The request's choice, by the workgroup that came last.
__device__ __forceinline__ void choose(const BeamLaunch& a, const BeamWs& ws, Shared& sh, int req, int chunks) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, W = a.width;
  const int64_t row0 = (int64_t)req * W;
  const int per_row = chunks * W, all = per_row * W;
  const uint64_t* cands = ws.cand + row0 * per_row;
  // the first candidates of this thread's first piece, on their way while the sums
  // are joined (those of a row without logits are not used)
  constexpr int kAhead = 8;
  uint64_t x[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) x[k] = get(cands + min(tid * W, all - W) + min(k, W - 1));
  // each row's sum, by 8 to 64 lanes of a wave
  int lanes = kWave;
  while (lanes * W > kThreads) lanes /= 2;
  const int w = tid / lanes, sub = tid % lanes;
  if (w < W) {
    const RowFacts f(a, row0 + w);
    const int parts = chunks * kWaves;
    const uint64_t* p = ws.part + (row0 + w) * parts * 2;
    uint32_t k = (uint32_t)get(p + 2 * min(sub, parts - 1));
    double s = __longlong_as_double((int64_t)get(p + 2 * min(sub, parts - 1) + 1));
    const int st = f.state();
    uint32_t top = 0;
    double sum = 0.0;
    for (int c = sub; st == 1 && c < parts; c += lanes) {
      if (c != sub) {
        k = (uint32_t)get(p + 2 * c);
        s = __longlong_as_double((int64_t)get(p + 2 * c + 1));
      }
      join_sums(top, sum, k, s);
    }
    uint32_t best = top;
    for (int o = lanes / 2; o > 0; o >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, o, kWave));
    if (top != best) sum *= top > kNone ? exp((double)value_of(top) - (double)value_of(best)) : 0.0;
    for (int o = lanes / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    top = best;
    if (sub == 0) {
      sh.f.lse[w] = top > kNone ? (double)value_of(top) + log(sum) : 0.0;
      sh.f.score[w] = f.score;
      sh.f.norm[w] = f.norm;
      sh.f.state[w] = st;
    }
  }
  if (tid == 0) sh.n = 0;
  __syncthreads();
  auto total_of = [&](const Cand& c) {
    return sh.f.state[c.row] == 2 ? sh.f.score[c.row]
                                  : sh.f.score[c.row] + ((double)value_of((uint32_t)(c.elem >> 32)) - sh.f.lse[c.row]);
  };
  // A candidate of a row whose element is x, `first` in its list of the row's first
  // piece (rows without logits have one, their eos); key 0: none.
  auto cand_of = [&](int w, uint64_t x, bool first) {
    Cand c;
    c.key = 0;
    c.row = w;
    c.elem = x;
    const int st = sh.f.state[w];
    if (st != 1) c.elem = st == 2 && first ? (uint64_t)(kNone + 1) << 32 | (uint32_t)~a.eos : 0;
    if ((uint32_t)(c.elem >> 32) > kNone) c.key = key_of(total_of(c) * sh.f.norm[w]);
    return c;
  };
  auto cand_at = [&](int i) {
    const int w = i / per_row;
    return cand_of(w, sh.f.state[w] == 1 ? get(cands + i) : 0, i == w * per_row);
  };
  // A piece's candidates descend: the width-th largest of the first ones of a wave's
  // pieces bounds those to look at; of the first eight, where the pieces are few or the
  // width is large (8 requests of width 32 with heads alone: 600 candidates and 62 us).
  const int lists = W * chunks;
  uint32_t bound = 0;
  for (int deep = W > kAhead ? 1 : 0; deep < 2 && bound == 0; ++deep) {
    uint32_t best = 0;
    for (int j0 = 0; j0 < lists; j0 += kThreads) {
      const int j = j0 + tid, w = min(j / chunks, W - 1);
      if (lists > kThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k] = get(cands + min(j, lists - 1) * W + min(k, W - 1));
      }
      auto key = [&](int k) {
        return j < lists && k < W ? (uint32_t)(cand_of(w, x[k], k == 0 && j == w * chunks).key >> 32) : 0;
      };
      uint32_t t = 0;
      if (deep == 0) {
        t = nth_largest<kLow64>(key(0), W);
      } else {
        uint32_t keys[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) keys[k] = key(k);
#pragma unroll 1
        for (int b = 31; b >= kLow64; --b) {
          const uint32_t u = t | 1u << b;
          int c = 0;
#pragma unroll
          for (int k = 0; k < kAhead; ++k) c += __popcll(__ballot(keys[k] >= u));
          if (c >= W) t = u;
        }
      }
      best = max(best, t);
    }
    __syncthreads();  // an earlier round's bounds have been read
    if (lane == 0) sh.bound[wave] = best;
    __syncthreads();
    for (int v = 0; v < kWaves; ++v) bound = max(bound, sh.bound[v]);
    if (lists * W <= kList / 4) break;  // few enough to look at them all
  }
  for (bool again = false;; again = true) {
    for (int j = tid; j < lists; j += kThreads) {
      const int w = j / chunks;
      bool more = true;
      for (int k0 = 0; k0 < W && more; k0 += kAhead) {
        if (k0 > 0 || again || lists > kThreads) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k) x[k] = get(cands + j * W + min(k0 + k, W - 1));
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (!more || k0 + k >= W) continue;
          const Cand c = cand_of(w, x[k], k0 + k == 0 && j == w * chunks);
          more = c.key != 0 && (uint32_t)(c.key >> 32) >= bound;
          if (!more) continue;
          const int at = atomicAdd(&sh.n, 1);
          if (at < kList) {
            sh.f.key[at] = c.key;
            sh.f.elem[at] = c.elem;
            sh.f.row[at] = c.row;
          }
        }
      }
    }
    __syncthreads();
    // too many: the width-th largest of those that the list holds is a higher bound
    if (sh.n <= kList) break;
    const uint32_t t = nth_of<kLow64, kList / kWave>(kList, W, [&](int i) { return (uint32_t)(sh.f.key[i] >> 32); });
    if (t <= bound) break;  // they are equal
    bound = t;
    __syncthreads();
    if (tid == 0) sh.n = 0;
    __syncthreads();
  }
  const int n = sh.n;
  auto write = [&](int rank, const Cand& c) {
    const int64_t o = row0 + rank;
    const int token = (int)~(uint32_t)c.elem;
    a.parent[o] = (int)(row0 + c.row);
    a.token[o] = token;
    a.score_out[o] = (float)total_of(c);
    if (a.done_out) a.done_out[o] = sh.f.state[c.row] == 2 || token == a.eos;
  };
  int found = min(n, W);
  auto listed = [&](int i) { return Cand{sh.f.key[i], sh.f.elem[i], sh.f.row[i]}; };
  if (n <= kList) {
    if (wave == 0) {
      auto hi = [&](int i) { return (uint32_t)(sh.f.key[i] >> 32); };
      const int m = gather(n, nth_of_list<kLow64>(n, W, hi), hi, sh.pick);
      if (lane == 0) sh.picked = m;
    }
    __syncthreads();
    const int m = sh.picked;
    if (m > kWave) {
      for (int i = tid; i < n; i += kThreads) {
        const Cand c = listed(i);
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += listed(j).above(c);
        if (rank < W) write(rank, c);
      }
    } else {  // each wave counts a quarter of those above
      const Cand c = listed(lane < m ? sh.pick[lane] : 0);
      int rank = 0;
      for (int j = wave; j < m; j += kWaves)
        rank += Cand{lane_of(c.key, j), lane_of(c.elem, j), lane_of(c.row, j)}.above(c);
      sh.rank[wave][lane] = rank;
      __syncthreads();
      if (wave == 0) {
        for (int v = 1; v < kWaves; ++v) rank += sh.rank[v][lane];
        if (lane < m && rank < W) write(rank, c);
      }
    }
  } else {
    // more than the list holds reach the bound: one after the other
    Cand limit = {~0ull, ~0ull, 0};
    for (int k = 0; k < W; ++k) {
      Cand c = {0, 0, 0};
      for (int i = tid; i < all; i += kThreads) {
        const Cand x = cand_at(i);
        if (x.key != 0 && limit.above(x) && (c.key == 0 || x.above(c))) c = x;
      }
      for (int o = 32; o > 0; o >>= 1) {
        const Cand x = {(uint64_t)__shfl_xor((unsigned long long)c.key, o, kWave),
                        (uint64_t)__shfl_xor((unsigned long long)c.elem, o, kWave),
                        (uint32_t)__shfl_xor((int)c.row, o, kWave)};
        if (x.key != 0 && (c.key == 0 || x.above(c))) c = x;
      }
      __syncthreads();
      if (lane == 0) sh.f.top[wave] = c;
      __syncthreads();
      for (int w = 0; w < kWaves; ++w)
        if (sh.f.top[w].key != 0 && (c.key == 0 || sh.f.top[w].above(c))) c = sh.f.top[w];
      if (tid == 0) write(k, c);
      limit = c;
    }
  }
  for (int k = found + tid; k < W; k += kThreads) {  // fewer continuations than beams
    a.parent[row0 + k] = (int)row0;
    a.token[row0 + k] = -1;
    a.score_out[row0 + k] = -INFINITY;
    if (a.done_out) a.done_out[row0 + k] = 0;
  }
}

// A part's `width` largest, taken one by one from memory.
template <typename T>
__device__ void one_by_one(const T* x, int64_t from, int64_t to, int W, uint64_t* out) {
  const int lane = threadIdx.x % kWave;
  uint64_t limit = ~0ull;
  for (int k = 0; k < W; ++k) {
    uint64_t c = 0;
#pragma unroll 8
    for (int64_t i = from + lane; i < to; i += kWave) {
      const float v = fminf(fmaxf((float)*gptr(x + i), -INFINITY), 3.402823466e38f) + 0.0f;
      const uint64_t y = (uint64_t)key_of(v) << 32 | (uint32_t)~(uint32_t)i;
      if (y < limit && y > c) c = y;
    }
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t y = (uint64_t)__shfl_xor((unsigned long long)c, o, kWave);
      c = y > c ? y : c;
    }
    if (lane == 0) out[k] = c;
    limit = c;
  }
}

template <typename T, int E>
__global__ __launch_bounds__(kThreads) void beam_kernel(BeamLaunch a, BeamWs ws, int chunks, int steps) {
  constexpr int kN = 16 / sizeof(T), kPieces = E / kN;
  // Which lane takes an element depends on its place in the row alone, so that
  // equal rows give equal sums: loads are of 16 bytes wherever the row starts.
  typedef T V __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid % kWave, W = a.width;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int row = blockIdx.y, chunk = (int)blockIdx.x, req = row / W;
  const T* x = (const T*)a.logits + row * a.ldl;
  const int64_t step = (int64_t)kWave * E, from = ((int64_t)chunk * kWaves + wave) * steps * step;
  const int64_t to = from + steps * step < a.vocab ? from + steps * step : a.vocab;
  V raw[kPieces];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int64_t i0 = at + (p * kWave + lane) * kN;
      if (i0 + kN <= a.vocab) {
        raw[p] = *(const __attribute__((address_space(1))) V*)(x + i0);
      } else {
#pragma unroll
        for (int c = 0; c < kN; ++c) raw[p][c] = i0 + c < a.vocab ? *gptr(x + i0 + c) : (T)-INFINITY;
      }
    }
  };
  // few rows: the logits come while the row's state is looked up; else rows without
  // continuations of their own are not read
  constexpr bool kEarly = E <= 8;
  if (kEarly && from < to) load(from);
  if (RowFacts(a, row).state() == 1) {
    if (!kEarly && from < to) load(from);
    uint64_t* list = sh.part[wave].list;
    uint64_t* best = sh.part[wave].best;  // the part's largest, in order
    float bound = -3.402823466e38f, ref = -INFINITY;  // the bound; what exponentials are relative to
    double sum = 0.0;
    int n = 0;
    bool full = false, first = true;
#pragma unroll 1
    for (int64_t at = from; at < to; at += step) {
      // NaN counts as no continuation (a maximum passes over it), infinity as the
      // largest number
      float v[E], big = -INFINITY;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        V w = __builtin_elementwise_max(raw[p], (V)((T)-INFINITY));
        if constexpr (sizeof(T) == 4) w = __builtin_elementwise_min(w, (V)((T)3.402823466e38f));
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          float y = (float)w[c];
          if constexpr (sizeof(T) == 2) y = fminf(y, 3.402823466e38f);
          v[p * kN + c] = y;
          big = fmaxf(big, y);
        }
      }
      if (at + step < to) load(at + step);
      if (__ballot(big > ref + 40.0f) != 0) {
        const float m = value_of(wave_max(key_of(big)));
        if (ref > -INFINITY) sum *= exp((double)ref - (double)m);
        ref = m;
      }
      if (ref == -INFINITY) continue;
      if (first) {
        bound = fmaxf(bound, value_of(max(nth_largest<kLow>(key_of(big), W), kNone + 1)));
        first = false;
      }
      constexpr double kLn2 = 0.69314718055994530942;
      constexpr float kHi = (float)(1.0 / kLn2), kLo = (float)((1.0 / kLn2 - (double)kHi) * kLn2);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float d = fmaxf(v[e + i] - ref, -1000.0f);
          const float t = d * kHi;
          // what the product's rounding lost, and the rest of 1 / ln 2, as a factor
          const float lost = __builtin_fmaf(d, kLo, __builtin_fmaf(d, kHi, -t) * (float)kLn2);
          const float z = __builtin_amdgcn_exp2f(t);
          y[i] = __builtin_fmaf(z, lost, z);
        }
        sum += (double)(y[0] + y[1]);
      }
      // what may be among the largest
      if (full) continue;
      auto add = [&](int c) {  // as far as the list goes; how many it would hold
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint64_t hits = __ballot(v[e] >= bound);
          if (hits != 0) {
            const uint32_t i = (uint32_t)(at + ((e / kN) * kWave + lane) * kN + e % kN);
            const int to = c + __popcll(hits & ((1ull << lane) - 1));
            // zeros of either sign are equal
            if (v[e] >= bound && to < kPart) list[to] = (uint64_t)key_of(v[e] + 0.0f) << 32 | ~i;
            c += __popcll(hits);
          }
        }
        wave_sync();
        return c;
      };
      const int was = n;
      n = add(was);
      if (n > kPart) {
        // of those before, only what reaches their own width-th largest; then once more
        auto hi = [&](int i) { return (uint32_t)(list[i] >> 32); };
        const uint32_t t = nth_of<kLow, kPart / kWave>(was, W, hi);
        uint64_t keep[kPart / kWave];
#pragma unroll
        for (int j = 0; j < kPart / kWave; ++j) keep[j] = lane + j * kWave < was ? list[lane + j * kWave] : 0;
        n = 0;
#pragma unroll
        for (int j = 0; j < kPart / kWave; ++j) {
          const bool hit = keep[j] != 0 && (uint32_t)(keep[j] >> 32) >= t;
          const uint64_t mask = __ballot(hit);
          if (hit) list[n + __popcll(mask & ((1ull << lane) - 1))] = keep[j];
          n += __popcll(mask);
        }
        wave_sync();
        bound = fmaxf(bound, value_of(max(t, kNone + 1)));
        n = add(n);
        full = n > kPart;
      }
    }
    sum = wave_sum(sum);
    auto hi = [&](int i) { return (uint32_t)(list[i] >> 32); };
    int m = 0;
    if (!full) {
      m = gather(n, n <= kWave ? 0 : nth_of<kLow, kPart / kWave>(n, W, hi), hi, sh.part[wave].pick);
      wave_sync();
    }
    if (lane < W) best[lane] = 0;
    wave_sync();
    if (full) {
      one_by_one(x, from, to, W, best);
    } else if (m > kWave) {
      for (int i = lane; i < n; i += kWave) {
        const uint64_t k = list[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += list[j] > k;
        if (rank < W) best[rank] = k;
      }
    } else {
      const uint64_t k = list[lane < m ? sh.part[wave].pick[lane] : 0];
      int rank = 0;
      for (int j = 0; j < m; ++j) rank += lane_of(k, j) > k;
      if (lane < m && rank < W) best[rank] = k;
    }
    if (lane == 0) {
      sh.part[wave].many = full ? W : min(n, W);
      uint64_t* p = ws.part + (((int64_t)row * chunks + chunk) * kWaves + wave) * 2;
      put(p, key_of(ref));
      put(p + 1, (uint64_t)__double_as_longlong(sum));
    }
    __syncthreads();
    // the waves' parts together: an element's rank is its own in its part and how many
    // of each other part are above it
    uint64_t* out = ws.cand + ((int64_t)row * chunks + chunk) * W;
    if (tid < kWaves * W) {
      const int own = tid / W, i = tid - own * W;
      const uint64_t k = sh.part[own].best[i];
      int rank = i;
      for (int w = 0; w < kWaves; ++w) {
        if (w == own) continue;
        int lo = 0, hi = W;  // how many are above k
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (sh.part[w].best[mid] > k) lo = mid + 1;
          else hi = mid;
        }
        rank += lo;
      }
      if (i < sh.part[own].many && rank < W) put(out + rank, k);
    } else if (tid >= kThreads - kWave) {
      int all = 0;
      for (int w = 0; w < kWaves; ++w) all += sh.part[w].many;
      for (int i = all + lane; i < W; i += kWave) put(out + i, 0);
    }
  }
  // the stores have completed before this workgroup counts as done
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    // first the row's counter, then its last one the request's: the arrivals at one
    // address follow each other at some 0.1 us (24 requests of 5 beams 30 us with one
    // counter a request, 22 so)
    auto last_of = [](uint32_t* count, uint32_t n) {
      if (__hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != n - 1) return false;
      __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      return true;
    };
    sh.last = last_of(ws.count + kMaxBeamRows + row, (uint32_t)chunks) && last_of(ws.count + req, (uint32_t)W);
  }
  __syncthreads();
  if (sh.last) choose(a, ws, sh, req, chunks);
}

// How a call is cut: 64 bytes a lane and step (32 f16 elements, 16 fp32 ones; with 32
// fp32 ones, 137 registers and 24 us for 24 requests of 5 beams, 20 so) where that still
// gives every CU a wave, else 8 elements (4 rows of 32000 11.9 us, 14.0 with 32); steps
// of a part as many as leave four waves to a SIMD.  A workgroup takes four parts of a row.
constexpr int kBytes = 64, kFew = 8;
struct Cut {
  int e, steps;
  int64_t chunks;
};
int many_of(int32_t dtype) { return kBytes / (dtype == DFS_F16 ? 2 : 4); }
int64_t chunks_of(int32_t vocab, int e, int steps) {
  const int64_t per = (int64_t)kWave * e * steps * kWaves;
  return (vocab + per - 1) / per;
}
Cut get_cut(int64_t rows, int32_t vocab, int32_t dtype) {
  Cut c;
  const int many = many_of(dtype);
  c.e = rows * chunks_of(vocab, many, 1) >= 64 ? many : kFew;
  c.steps = c.e == kFew ? 1 : (int)std::max<int64_t>(1, rows * vocab / ((int64_t)kWave * many * 4096));
  c.chunks = chunks_of(vocab, c.e, c.steps);
  return c;
}
size_t layout(int64_t parts, int32_t width, size_t* cand) {
  *cand = kCounterBytes + (size_t)parts * kWaves * 16;
  return *cand + (size_t)parts * width * 8;
}

}  // namespace

size_t beam_ws_need(int32_t n_req, int32_t width, int32_t vocab, int32_t dtype) {
  const int64_t rows = (int64_t)n_req * width;
  size_t cand;
  return layout(rows * get_cut(rows, vocab, dtype).chunks, width, &cand);
}
// Of any smaller call: where few rows take small steps, these make at most four times
// as many pieces as the 63 that large ones would.
size_t beam_ws_bytes(int32_t n_req, int32_t width, int32_t vocab) {
  const int64_t rows = (int64_t)n_req * width;
  size_t cand;
  return layout(std::max(rows * chunks_of(vocab, kBytes / 4, 1), std::min<int64_t>(rows * chunks_of(vocab, kFew, 1), 4 * 63)),
                width, &cand);
}

hipError_t launch_beam_select(const BeamLaunch& a, void* ws, hipStream_t s) {
  const int64_t rows = (int64_t)a.n_req * a.width;
  const Cut c = get_cut(rows, a.vocab, a.dtype);
  size_t cand;
  layout(rows * c.chunks, a.width, &cand);
  const BeamWs w = {(uint32_t*)ws, (uint64_t*)((char*)ws + kCounterBytes), (uint64_t*)((char*)ws + cand)};
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)c.chunks, (unsigned)rows), dim3(kThreads), 0, s, a, w,
                       (int)c.chunks, c.steps);
  };
  if (a.dtype == DFS_F16) {
    if (c.e == kFew) run(beam_kernel<_Float16, kFew>);
    else run(beam_kernel<_Float16, kBytes / 2>);
  } else {
    if (c.e == kFew) run(beam_kernel<float, kFew>);
    else run(beam_kernel<float, kBytes / 4>);
  }
  return hipGetLastError();
}

}  // namespace dfs
