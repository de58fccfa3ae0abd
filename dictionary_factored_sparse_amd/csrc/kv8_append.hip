// kv8_append.hip -- new keys and values into the 8-bit paged cache, one fp32
// scale per page and head (the recipe stands in dictfs.h).  Compiled without
// FMA contraction: each step of the recipe is one correctly rounded fp32
// operation.
//
// One workgroup per page that gets tokens, head, and keys or values: a first
// pass over the new elements for the largest size, a second (from L1: a page's
// new elements are 4 to 128 KB) for the codes.  Workgroups of neighbouring
// heads read neighbouring bytes and are neighbours in the grid.  Values are
// stored with the page's tokens contiguous, so a lane takes 16 tokens of a few
// dims and packs codes across the tokens in registers: no transposition
// through LDS.
//
// What bounds it: prompts, the bytes (source read, codes written); single
// tokens, the chain of dependent reads (requests, page table, scale).
#include <algorithm>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr uint32_t kTop = 0x477FE000u;  // 65504: larger elements count as this

// value / scale, correctly rounded, for many values: with r the correctly
// rounded reciprocal of the scale, v r is within two units of the quotient;
// the remainder of a candidate is exact in one FMA, and the second of two
// corrections by remainder * r then rounds correctly (Markstein).  Quotients
// below 2^-10 may lose bits where remainders underflow; their code is 0 in any
// case.  Scales so small that the reciprocal leaves the normal range are
// divided by.
struct Quotient {
  float scale, r;
  uint32_t sign;  // the bit that comes from the value: none where the scale is 0
  bool fast;
  __device__ __forceinline__ explicit Quotient(float s)
      : scale(s), r(s > 0.0f ? 1.0f / s : 0.0f), sign(s > 0.0f ? 0x80000000u : 0u),
        fast(s >= 0x1p-60f || s == 0.0f) {}
  __device__ __forceinline__ float operator()(float v) const {
    if (!fast) return v / scale;
    float q = v * r;
    q = __builtin_fmaf(__builtin_fmaf(-q, scale, v), r, q);
    q = __builtin_fmaf(__builtin_fmaf(-q, scale, v), r, q);
    // the corrections lose the sign of a zero
    return __uint_as_float((__float_as_uint(v) & sign) | (__float_as_uint(q) & ~sign));
  }
};

// Codes of four quotients, the first in the low byte.
template <int KIND>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (KIND == DFS_FP8) {
    auto in = [](float q) { return __builtin_amdgcn_fmed3f(q, -448.0f, 448.0f); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(in(a), in(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(in(c), in(d), w, true);
  } else {
    // adding 1.5 * 2^23 rounds to the nearest whole number, ties to even, which
    // then stands in the low bits
    auto in = [](float q) {
      return __float_as_uint(__builtin_amdgcn_fmed3f(q, -127.0f, 127.0f) + 12582912.0f);
    };
    const uint32_t lo = __builtin_amdgcn_perm(in(b), in(a), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(in(d), in(c), 0x04000c0cu);
    return lo | hi;
  }
}
template <int KIND>
__device__ __forceinline__ float decode8(uint32_t c) {
  if constexpr (KIND == DFS_FP8) return e4m3_to_f32(c & 0xFFu);
  return (float)(int8_t)c;
}

// What an element counts as: NaN 0, the rest within +-65504.
__device__ __forceinline__ float tamed(float v) {
  return v != v ? 0.0f : __builtin_amdgcn_fmed3f(v, -65504.0f, 65504.0f);
}

// 16 bytes of source elements.
template <typename T>
struct Piece {
  static constexpr int kN = 16 / sizeof(T);
  typedef T VT __attribute__((ext_vector_type(16 / sizeof(T))));
  VT v;
  __device__ __forceinline__ void load(const T* p, bool vec) {
    if (vec) {
      v = *gptr((const VT*)p);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = *gptr(p + i);
    }
  }
  // the largest size's bits; NaN and infinities come out above kTop
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = max(m, __float_as_uint((float)v[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ float at(int i, bool tame) const {
    return tame ? tamed((float)v[i]) : (float)v[i];
  }
};

__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
  __syncthreads();
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = max(m, red[w]);
  return m;
}

// The request and page that slot `slot` stands for (slots count the pages that
// get tokens, request after request).
struct Job {
  int req, t0, n, cached, page;  // page: of the request
};
__device__ __forceinline__ bool find_job(const KvBatch& b, int P, int slot, Job& j) {
  const int lane = threadIdx.x % kWave;
  int base = 0;
  for (int r0 = 0; r0 < b.n_req; r0 += kWave) {
    const int r = r0 + lane;
    int t0 = 0, n = 0, c = 0;
    if (r < b.n_req) {
      t0 = min(max(*gptr(b.tok_start + r), 0), b.n_tok);
      n = min(max(*gptr(b.tok_start + r + 1), t0), b.n_tok) - t0;
      c = max(*gptr(b.have + r), 0);
    }
    const int m = n > 0 ? (int)(((int64_t)c + n - 1) / P - c / P + 1) : 0;
    int x = m;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int y = __shfl_up(x, o, kWave);
      if (lane >= o) x += y;
    }
    const uint64_t hit = __ballot(slot >= base + x - m && slot < base + x);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      j.req = r0 + l;
      j.t0 = __builtin_amdgcn_readlane(t0, l);
      j.n = __builtin_amdgcn_readlane(n, l);
      j.cached = __builtin_amdgcn_readlane(c, l);
      j.page = j.cached / P + slot - base - __builtin_amdgcn_readlane(x - m, l);
      return true;
    }
    base += __builtin_amdgcn_readlane(x, kWave - 1);
  }
  return false;
}

template <int KIND, typename T>
__global__ __launch_bounds__(kThreads) void append_kernel(dfs_kv8 kv, KvBatch b, const T* K,
                                                          int64_t ldk, const T* V, int64_t ldv,
                                                          int vec, int slot0) {
  constexpr int kN = Piece<T>::kN;
  __shared__ uint32_t red[kWaves];
  const int P = kv.page, D = kv.head_dim, h = blockIdx.x;
  const bool values = blockIdx.z != 0;
  Job j;
  if (!find_job(b, P, slot0 + (int)blockIdx.y, j) || j.page >= b.table_pages) return;
  const int pg = *gptr(b.table + j.req * b.ldt + j.page);
  // slots lo .. hi - 1 of the page are new; slot s is row row0 + s of the source
  const int64_t p0 = (int64_t)j.page * P;
  const int lo = (int)max((int64_t)j.cached - p0, (int64_t)0);
  const int hi = (int)min((int64_t)j.cached + j.n - p0, (int64_t)P);
  const int64_t ld = values ? ldv : ldk;
  const T* src = (values ? V : K) + (int64_t)h * D + (j.t0 + p0 - j.cached) * ld;
  const int per_row = D / kN;
  uint32_t top = 0;
#pragma unroll 4
  for (int e = threadIdx.x; e < (hi - lo) * per_row; e += kThreads) {
    const int s = e / per_row;
    Piece<T> x;
    x.load(src + (lo + s) * ld + (e - s * per_row) * kN, vec);
    top = max(top, x.top());
  }
  top = block_max(top, red);
  const bool tame = top > kTop;
  if (tame) {  // something is not finite or too large: once more, with what it counts as
    top = 0;
#pragma unroll 1
    for (int e = threadIdx.x; e < (hi - lo) * D; e += kThreads)
      top = max(top, __float_as_uint(fabsf(tamed((float)src[(lo + e / D) * ld + e % D]))));
    top = block_max(top, red);
  }
  if (pg < 0 || pg >= kv.n_pages) return;
  const int64_t ph = (int64_t)pg * kv.heads + h;
  uint8_t* codes = (values ? kv.v : kv.k) + ph * P * D;
  float* scale = (values ? kv.vscale : kv.kscale) + ph;
  const float need = __uint_as_float(top) / (KIND == DFS_FP8 ? 448.0f : 127.0f);
  const float old = lo > 0 ? *scale : 0.0f;
  const float sc = need > old ? need : old;
  const Quotient q(sc);
  if (need > old && lo > 0) {
    // a larger scale: the codes of the tokens already there, four at a time
    // (keys: of four dims; values: of four tokens, of which some may be new or
    // later and stay)
    const int words = values ? (lo + 3) / 4 : D / 4, rows = values ? D : lo;
#pragma unroll 1
    for (int e = threadIdx.x; e < rows * words; e += kThreads) {
      const int row = e / words, w = e - row * words;
      uint32_t* p = (uint32_t*)(codes + row * (values ? P : D)) + w;
      const uint32_t c = *p;
      const int held = values ? lo - 4 * w : 4;  // bytes that are older tokens'
      const uint32_t keep = held >= 4 ? 0u : 0xFFFFFFFFu << (8 * held);
      const uint32_t n = encode4<KIND>(q(decode8<KIND>(c) * old), q(decode8<KIND>(c >> 8) * old),
                                       q(decode8<KIND>(c >> 16) * old),
                                       q(decode8<KIND>(c >> 24) * old));
      *p = (c & keep) | (n & ~keep);
    }
    __syncthreads();  // new tokens' bytes go into the same words
  }
  if (threadIdx.x == 0) *scale = sc;
  if (!values) {
#pragma unroll 2
    for (int e = threadIdx.x; e < (hi - lo) * per_row; e += kThreads) {
      const int s = e / per_row, d = (e - s * per_row) * kN;
      Piece<T> x;
      x.load(src + (lo + s) * ld + d, vec);
      uint32_t* p = (uint32_t*)(codes + (lo + s) * D + d);
#pragma unroll
      for (int i = 0; i < kN; i += 4)
        p[i / 4] = encode4<KIND>(q(x.at(i, tame)), q(x.at(i + 1, tame)), q(x.at(i + 2, tame)),
                                 q(x.at(i + 3, tame)));
    }
  } else {
    // groups of 16 slots: whole ones by 16-byte stores, others token by token
    const int g0 = lo / 16, groups = (hi + 15) / 16 - g0;
#pragma unroll 1
    for (int e = threadIdx.x; e < groups * per_row; e += kThreads) {
      const int g = e / per_row, d = (e - g * per_row) * kN, s0 = (g0 + g) * 16;
      uint8_t* p = codes + d * P + s0;
      if (s0 >= lo && s0 + 16 <= hi) {
        Piece<T> x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i].load(src + (s0 + i) * ld + d, vec);
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          u4 w;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = encode4<KIND>(q(x[4 * i].at(k, tame)), q(x[4 * i + 1].at(k, tame)),
                                 q(x[4 * i + 2].at(k, tame)), q(x[4 * i + 3].at(k, tame)));
          *gptr_w((u4*)(p + k * P)) = w;
        }
      } else {
#pragma unroll 1
        for (int s = max(s0, lo); s < min(s0 + 16, hi); ++s) {
          Piece<T> x;
          x.load(src + s * ld + d, vec);
#pragma unroll
          for (int k = 0; k < kN; k += 4) {
            const uint32_t w = encode4<KIND>(q(x.at(k, tame)), q(x.at(k + 1, tame)),
                                             q(x.at(k + 2, tame)), q(x.at(k + 3, tame)));
#pragma unroll
            for (int i = 0; i < 4; ++i) p[(k + i) * P + s - s0] = (uint8_t)(w >> (8 * i));
          }
        }
      }
    }
  }
}

template <int KIND, typename T>
void go(const dfs_kv8& kv, const KvBatch& b, const void* K, int64_t ldk, const void* V, int64_t ldv,
        hipStream_t s) {
  // n tokens of a request touch at most (n - 2) / page + 2 pages, and one if n is 1
  const int64_t most = std::min<int64_t>(b.n_tok, b.n_tok / kv.page + 2 * (int64_t)b.n_req);
  const int vec = ((uintptr_t)K | (uintptr_t)V) % 16 == 0 && ldk * sizeof(T) % 16 == 0 &&
                  ldv * sizeof(T) % 16 == 0;
  // the y axis of a grid ends at 65535: one launch but for millions of tokens
  for (int64_t y = 0; y < most; y += 65535)
    hipLaunchKernelGGL((append_kernel<KIND, T>),
                       dim3(kv.heads, (unsigned)std::min<int64_t>(most - y, 65535), 2),
                       dim3(kThreads), 0, s, kv, b, (const T*)K, ldk, (const T*)V, ldv, vec, (int)y);
}

}  // namespace

hipError_t launch_kv8_append(const dfs_kv8& kv, const KvBatch& b, const void* K, int64_t ldk,
                             const void* V, int64_t ldv, int32_t dtype, hipStream_t s) {
  if (dtype == DFS_F16) {
    if (kv.dtype == DFS_FP8) go<DFS_FP8, _Float16>(kv, b, K, ldk, V, ldv, s);
    else go<DFS_INT8, _Float16>(kv, b, K, ldk, V, ldv, s);
  } else {
    if (kv.dtype == DFS_FP8) go<DFS_FP8, float>(kv, b, K, ldk, V, ldv, s);
    else go<DFS_INT8, float>(kv, b, K, ldk, V, ldv, s);
  }
  return hipGetLastError();
}

}  // namespace dfs
