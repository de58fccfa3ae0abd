// beam_select.hip -- the next beams of beam search: of the width * vocab
// continuations of a request, the `width` best.
//
// total(w, v) = score_w + x_wv - lse_w, lse_w = m_w + log sum_v 2^((x_wv - m_w) log2 e),
// ranked by total * norm_w.
//
// One launch, one pass over the logits: a workgroup takes a piece of a row and
// keeps its elements in registers, sums its exponentials and finds its `width`
// largest elements (within a row the order of the totals is that of the
// logits).  The workgroup that comes last of a request's joins the sums and
// picks from what the pieces offer.
//
// The largest elements of a piece.  The width-th largest of the 64 lanes'
// maxima of one wave bounds the width-th largest element from below; it takes
// 32 steps of a compare and a count of the lanes, no memory.  The few elements
// above the bound go to a list in LDS, where each is ranked by counting those
// above it.  If more than the list holds are equal to the bound, the elements
// are taken one by one.
//
// Precision.  Beams of different rows compete by sums that may be close: the
// exponentials are summed in 64 bits, with the rounding error of their
// arguments put back in, and totals are compared in 64 bits.
#include <algorithm>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kList = 1024;
constexpr size_t kCounterBytes = 65536;
constexpr uint32_t kNone = 0x007FFFFFu;  // key of -inf: no continuation

struct BeamWs {
  uint32_t* count;  // [n_req]: workgroups that are done
  uint64_t* part;   // [rows][chunks]: key of the largest logit, sum of the exponentials
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

// The largest t that at least n lanes of the wave reach (0 where fewer have a key).
__device__ __forceinline__ uint32_t nth_largest(uint32_t k, int n) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 0; --b) {
    const uint32_t u = t | 1u << b;
    if (__popcll(__ballot(k >= u)) >= n) t = u;
  }
  return t;
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

struct Shared {
  uint32_t wmax[kWaves], bound[kWaves];
  double wsum[kWaves];
  int n, last;
  uint64_t best[kWaves];
  union {
    uint64_t list[kList];
    struct {
      double lse[kMaxBeams], score[kMaxBeams], norm[kMaxBeams];
      int state[kMaxBeams];  // 0: no continuation, 1: its logits', 2: its eos
      uint64_t key[kList], elem[kList];
      uint32_t row[kList];
      Cand top[kWaves];
    } f;
  };
};

__device__ __forceinline__ void put(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether a row offers continuations, and which.
__device__ __forceinline__ int state_of(const BeamLaunch& a, int row) {
  const float sc = *gptr(a.score + row);
  const float nm = a.norm ? *gptr(a.norm + row) : 1.0f;
  if (!(sc > -INFINITY && sc < INFINITY) || !(nm > 0.0f && nm < INFINITY)) return 0;
  return a.done && *gptr(a.done + row) != 0 ? 2 : 1;
}

// The request's choice, by the workgroup that came last.
__device__ __forceinline__ void choose(const BeamLaunch& a, const BeamWs& ws, Shared& sh, int req, int chunks) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, W = a.width;
  const int64_t row0 = (int64_t)req * W;
  for (int w = wave; w < W; w += kWaves) {
    const int st = state_of(a, (int)(row0 + w));
    double lse = 0.0;
    if (st == 1) {
      const uint64_t* p = ws.part + (row0 + w) * chunks * 2;
      uint32_t m = 0;
      for (int c = lane; c < chunks; c += kWave) m = max(m, (uint32_t)get(p + 2 * c));
      m = wave_max(m);
      const double top = value_of(m);
      double s = 0.0;
      if (m > kNone)
        for (int c = lane; c < chunks; c += kWave) {
          const uint32_t k = (uint32_t)get(p + 2 * c);
          if (k > kNone) s += __longlong_as_double((int64_t)get(p + 2 * c + 1)) * exp((double)value_of(k) - top);
        }
      s = wave_sum(s);
      lse = top + log(s);
    }
    if (lane == 0) {
      sh.f.lse[w] = lse;
      sh.f.score[w] = a.score[row0 + w];
      sh.f.norm[w] = a.norm ? a.norm[row0 + w] : 1.0f;
      sh.f.state[w] = st;
    }
  }
  if (tid == 0) sh.n = 0;
  __syncthreads();
  const int per_row = chunks * W, all = per_row * W;
  const uint64_t* cands = ws.cand + row0 * per_row;
  auto total_of = [&](const Cand& c) {
    return sh.f.state[c.row] == 2 ? sh.f.score[c.row]
                                  : sh.f.score[c.row] + ((double)value_of((uint32_t)(c.elem >> 32)) - sh.f.lse[c.row]);
  };
  // candidate i; key 0: none
  auto cand_at = [&](int i) {
    Cand c;
    c.key = 0;
    c.row = i / per_row;
    c.elem = 0;
    const int st = sh.f.state[c.row];
    if (st == 1) c.elem = get(cands + i);
    if (st == 2 && i % per_row == 0) c.elem = (uint64_t)(kNone + 1) << 32 | (uint32_t)~a.eos;
    if ((uint32_t)(c.elem >> 32) > kNone) c.key = key_of(total_of(c) * sh.f.norm[c.row]);
    return c;
  };
  uint32_t mine = 0;
  for (int i = tid; i < all; i += kThreads) mine = max(mine, (uint32_t)(cand_at(i).key >> 32));
  const uint32_t b = nth_largest(mine, W);
  if (lane == 0) sh.bound[wave] = b;
  __syncthreads();
  uint32_t bound = 0;
  for (int w = 0; w < kWaves; ++w) bound = max(bound, sh.bound[w]);
  for (int i = tid; i < all; i += kThreads) {
    const Cand c = cand_at(i);
    if (c.key != 0 && (uint32_t)(c.key >> 32) >= bound) {
      const int at = atomicAdd(&sh.n, 1);
      if (at < kList) {
        sh.f.key[at] = c.key;
        sh.f.elem[at] = c.elem;
        sh.f.row[at] = c.row;
      }
    }
  }
  __syncthreads();
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
  if (n <= kList) {
    for (int i = tid; i < n; i += kThreads) {
      const Cand c = {sh.f.key[i], sh.f.elem[i], sh.f.row[i]};
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += Cand{sh.f.key[j], sh.f.elem[j], sh.f.row[j]}.above(c);
      if (rank < W) write(rank, c);
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

template <typename T, int E>
__global__ __launch_bounds__(kThreads) void beam_kernel(BeamLaunch a, BeamWs ws, int chunks) {
  constexpr int kN = 16 / sizeof(T), kPieces = E / kN;
  // Which thread takes an element depends on its place in the row alone, so that
  // equal rows give equal sums: loads are of 16 bytes wherever the row starts.
  typedef T V __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, W = a.width;
  const int row = blockIdx.y, chunk = blockIdx.x, req = row / W;
  if (state_of(a, row) == 1) {
    const T* x = (const T*)a.logits + row * a.ldl;
    float v[E];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int64_t i0 = ((int64_t)(chunk * kPieces + p) * kThreads + tid) * kN;
      if (i0 + kN <= a.vocab) {
        const V w = *gptr((const V*)(x + i0));
#pragma unroll
        for (int c = 0; c < kN; ++c) v[p * kN + c] = (float)w[c];
      } else {
#pragma unroll
        for (int c = 0; c < kN; ++c)
          v[p * kN + c] = i0 + c < a.vocab ? (float)*gptr(x + i0 + c) : -INFINITY;
      }
    }
    uint32_t best = kNone;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      // NaN counts as no continuation, infinity as the largest number
      v[e] = v[e] != v[e] ? -INFINITY : fminf(v[e], 3.402823466e38f);
      best = max(best, key_of(v[e]));
    }
    const uint32_t wm = wave_max(best), wb = nth_largest(best, W);
    if (lane == 0) {
      sh.wmax[wave] = wm;
      sh.bound[wave] = wb;
    }
    if (tid == 0) sh.n = 0;
    __syncthreads();
    uint32_t top = 0, bound = kNone + 1;
    for (int w = 0; w < kWaves; ++w) {
      top = max(top, sh.wmax[w]);
      bound = max(bound, sh.bound[w]);
    }
    const float m = value_of(top);
    double sum = 0.0;
    if (top > kNone) {
      constexpr double kLog2e = 1.44269504088896340736;
      constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = v[e] - m;
        const float t = d * kHi;
        // what the product's rounding lost, and the rest of log2 e
        const float lost = d > -1e4f ? __builtin_fmaf(d, kHi, -t) + d * kLo : 0.0f;
        const float y = __builtin_amdgcn_exp2f(t);
        sum += (double)__builtin_fmaf(y, lost * 0.69314718f, y);
      }
    }
    sum = wave_sum(sum);
    if (lane == 0) sh.wsum[wave] = sum;
    // what may be among the largest
    auto elem_of = [&](int e) {
      const int64_t i = ((int64_t)(chunk * kPieces + e / kN) * kThreads + tid) * kN + e % kN;
      return (uint64_t)key_of(v[e]) << 32 | (uint32_t)~(uint32_t)i;
    };
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (key_of(v[e]) >= bound) {
        const int at = atomicAdd(&sh.n, 1);
        if (at < kList) sh.list[at] = elem_of(e);
      }
    __syncthreads();
    const int n = sh.n;
    uint64_t* out = ws.cand + ((int64_t)row * chunks + chunk) * W;
    if (n <= kList) {
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t k = sh.list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.list[j] > k;
        if (rank < W) put(out + rank, k);
      }
      for (int i = n + tid; i < W; i += kThreads) put(out + i, 0);
    } else {
      uint64_t limit = ~0ull;
      for (int k = 0; k < W; ++k) {
        uint64_t c = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint64_t y = elem_of(e);
          if (y < limit && y > c) c = y;
        }
        for (int o = 32; o > 0; o >>= 1) {
          const uint64_t y = (uint64_t)__shfl_xor((unsigned long long)c, o, kWave);
          c = y > c ? y : c;
        }
        __syncthreads();
        if (lane == 0) sh.best[wave] = c;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) c = sh.best[w] > c ? sh.best[w] : c;
        if (tid == 0) put(out + k, c);
        limit = c;
      }
    }
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < kWaves; ++w) s += sh.wsum[w];
      uint64_t* p = ws.part + ((int64_t)row * chunks + chunk) * 2;
      put(p, top);
      put(p + 1, (uint64_t)__double_as_longlong(s));
    }
  }
  // the stores have completed before this workgroup counts as done
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    const uint32_t all = (uint32_t)(W * chunks);
    sh.last = __hip_atomic_fetch_add(ws.count + req, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == all - 1;
    if (sh.last) __hip_atomic_store(ws.count + req, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (sh.last) choose(a, ws, sh, req, chunks);
}

// Elements a thread: 32 where that still fills the device, else 8.
constexpr int kMany = 32, kFew = 8;
int64_t chunks_of(int32_t vocab, int32_t dtype, int e) {
  const int64_t n = dtype == DFS_F16 ? 8 : 4;
  const int64_t pieces = (vocab + n - 1) / n;
  const int64_t per = (int64_t)kThreads * (e / n);
  return (pieces + per - 1) / per;
}
int elements(int64_t rows, int32_t vocab, int32_t dtype) {
  return rows * chunks_of(vocab, dtype, kMany) >= 256 ? kMany : kFew;
}
size_t layout(int64_t rows, int64_t chunks, int32_t width, size_t* cand) {
  *cand = kCounterBytes + (size_t)rows * chunks * 16;
  return *cand + (size_t)rows * chunks * width * 8;
}

}  // namespace

size_t beam_ws_need(int32_t n_req, int32_t width, int32_t vocab, int32_t dtype) {
  const int64_t rows = (int64_t)n_req * width;
  size_t cand;
  return layout(rows, chunks_of(vocab, dtype, elements(rows, vocab, dtype)), width, &cand);
}
// Of any smaller call: one with few rows takes small pieces.
size_t beam_ws_bytes(int32_t n_req, int32_t width, int32_t vocab) {
  const int64_t rows = (int64_t)n_req * width;
  size_t cand;
  return layout(rows, chunks_of(vocab, DFS_F32, kFew), width, &cand);
}

hipError_t launch_beam_select(const BeamLaunch& a, void* ws, hipStream_t s) {
  const int64_t rows = (int64_t)a.n_req * a.width;
  const int e = elements(rows, a.vocab, a.dtype);
  const int chunks = (int)chunks_of(a.vocab, a.dtype, e);
  size_t cand;
  layout(rows, chunks, a.width, &cand);
  const BeamWs w = {(uint32_t*)ws, (uint64_t*)((char*)ws + kCounterBytes), (uint64_t*)((char*)ws + cand)};
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(chunks, (unsigned)rows), dim3(kThreads), 0, s, a, w, chunks);
  };
  if (a.dtype == DFS_F16) {
    if (e == kMany) run(beam_kernel<_Float16, kMany>);
    else run(beam_kernel<_Float16, kFew>);
  } else {
    if (e == kMany) run(beam_kernel<float, kMany>);
    else run(beam_kernel<float, kFew>);
  }
  return hipGetLastError();
}

}  // namespace dfs
