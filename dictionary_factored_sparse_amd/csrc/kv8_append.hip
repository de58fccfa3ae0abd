// kv8_append.hip -- new keys and values into the 8-bit paged cache, one fp32
// scale per page and head (the recipe stands in dictfs.h).  Compiled without
// FMA contraction: each step of the recipe is one correctly rounded fp32
// operation.
//
// One workgroup per page that gets tokens and head: a first pass over the new
// elements for the largest sizes, a second for the codes, with the elements
// kept in registers between them where they fit.  Workgroups of neighbouring
// heads read neighbouring bytes and are neighbours in the grid.  Values are
// stored with the page's tokens contiguous: a lane packs the codes of four
// tokens into a word, and the words go out through LDS.
//
// What bounds it: prompts, the bytes (source read, codes written): 7191 tokens
// of 32 heads of 128 from f16 take 58 us, 3.0 TB/s over 177 MB, against 83
// with a workgroup for K and one for V and value codes stored without LDS.
// Single tokens, the chain of dependent reads (requests, page table, scale):
// 10.8 us for 32 requests of 32 heads, 7.7 for 346 tokens of 8 heads on pages of
// 16 (with plain divisions, and FP8 codes made by bit operations and stored one
// by one, 21.6 and 13.1; prompts 254).  These are calls whose pages keep their
// scales.  Where the new tokens raise some, older codes of those pages are coded
// anew: 15.5 and 8.4 us for the kernel alone, against 11.2 and 7.8.
#include <algorithm>
#include <type_traits>

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

typedef uint16_t us8 __attribute__((ext_vector_type(8)));
// Running maxima of sizes as bits (their order is the values'), f16 in pairs.
template <typename T>
struct Tops {
  typename std::conditional<sizeof(T) == 2, us8, u4>::type m = 0;
  // fp32 bits; NaN and infinities come out above kTop
  __device__ __forceinline__ uint32_t bits() const {
    if constexpr (sizeof(T) == 2) {
      uint16_t h = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) h = max(h, m[i]);
      return h >= 0x7C00 ? 0x7F800000u
                         : __float_as_uint((float)__builtin_bit_cast(_Float16, h));
    } else {
      return m[0];
    }
  }
};

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
  // Folds the sizes' bits into m; Tops turns them into fp32 bits.
  __device__ __forceinline__ void fold(Tops<T>& t) const {
    if constexpr (sizeof(T) == 2) {
      const us8 b = __builtin_bit_cast(us8, v) & (uint16_t)0x7FFF;
      t.m = __builtin_elementwise_max(t.m, b);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        t.m[0] = max(t.m[0], __float_as_uint((float)v[i]) & 0x7FFFFFFFu);
    }
  }
  __device__ __forceinline__ float at(int i, bool tame) const {
    return tame ? tamed((float)v[i]) : (float)v[i];
  }
};

// Maxima of k and v over the workgroup.
__device__ __forceinline__ void block_max(uint32_t& k, uint32_t& v, uint32_t (*red)[2]) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    k = max(k, (uint32_t)__shfl_xor((int)k, o, kWave));
    v = max(v, (uint32_t)__shfl_xor((int)v, o, kWave));
  }
  __syncthreads();
  if (threadIdx.x % kWave == 0) {
    red[threadIdx.x / kWave][0] = k;
    red[threadIdx.x / kWave][1] = v;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    k = max(k, red[w][0]);
    v = max(v, red[w][1]);
  }
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

// Four slots' pieces of a few dims, zero for slots outside [lo, hi).
template <typename T>
struct Item {
  Piece<T> x[4];
  __device__ __forceinline__ void load(const T* src, int64_t ld, int s0, int lo, int hi, bool vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i].v = typename Piece<T>::VT{};
      if (s0 + i >= lo && s0 + i < hi) x[i].load(src + (s0 + i) * ld, vec);
    }
  }
  __device__ __forceinline__ void fold(Tops<T>& t) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i].fold(t);
  }
};

// Four codes under a new scale.
template <int KIND>
__device__ __forceinline__ uint32_t again4(uint32_t c, float old, const Quotient& q) {
  return encode4<KIND>(q(decode8<KIND>(c) * old), q(decode8<KIND>(c >> 8) * old),
                       q(decode8<KIND>(c >> 16) * old), q(decode8<KIND>(c >> 24) * old));
}

template <int KIND, typename T>
__global__ __launch_bounds__(kThreads) void append_kernel(dfs_kv8 kv, KvBatch b, const T* K,
                                                          int64_t ldk, const T* V, int64_t ldv,
                                                          int vec, int slot0) {
  constexpr int kN = Piece<T>::kN;
  __shared__ uint32_t red[kWaves][2];
  extern __shared__ uint32_t words[];  // new value codes, [dim][word of four slots]
  const int P = kv.page, D = kv.head_dim, h = blockIdx.x;
  Job j;
  if (!find_job(b, P, slot0 + (int)blockIdx.y, j) || j.page >= b.table_pages) return;
  const int32_t* entry = b.table + j.req * b.ldt + j.page;
  const int pg = *gptr(entry);
  // slots lo .. hi - 1 of the page are new; slot s is row row0 + s of the source
  const int64_t p0 = (int64_t)j.page * P, row0 = j.t0 + p0 - j.cached;
  const int lo = (int)max((int64_t)j.cached - p0, (int64_t)0);
  const int hi = (int)min((int64_t)j.cached + j.n - p0, (int64_t)P);
  const T* ksrc = K + (int64_t)h * D + row0 * ldk;
  const T* vsrc = V + (int64_t)h * D + row0 * ldv;
  // an item is four slots of kN dims; a thread's first one stays in registers
  // (all of them do for up to 256 items: 64 tokens of 128 f16 dims)
  const int per_row = D / kN, w0 = lo / 4, w1 = (hi + 3) / 4, items = (w1 - w0) * per_row;
  auto slot_of = [&](int e) { return 4 * (w0 + e / per_row); };
  auto dim_of = [&](int e) { return e % per_row * kN; };
  Item<T> k0, v0;
  Tops<T> kt, vt;
  if ((int)threadIdx.x < items) {
    const int s0 = slot_of(threadIdx.x), d = dim_of(threadIdx.x);
    k0.load(ksrc + d, ldk, s0, lo, hi, vec);
    v0.load(vsrc + d, ldv, s0, lo, hi, vec);
  }
  const bool real = pg >= 0 && pg < kv.n_pages;
  const int64_t ph = (int64_t)(real ? pg : 0) * kv.heads + h;
  const float kold = lo > 0 ? *gptr(kv.kscale + ph) : 0.0f;
  const float vold = lo > 0 ? *gptr(kv.vscale + ph) : 0.0f;
  // what the value codes' first word holds now, if it keeps some of it
  uint32_t was0 = 0;
  if ((int)threadIdx.x < D * (w1 - w0) && real) {
    const int w = w0 + (int)threadIdx.x % (w1 - w0);
    if (4 * w < lo || 4 * w + 4 > hi)
      was0 = *gptr((uint32_t*)(kv.v + (ph * D + (int)threadIdx.x / (w1 - w0)) * P) + w);
  }
  if ((int)threadIdx.x < items) {
    k0.fold(kt);
    v0.fold(vt);
  }
#pragma unroll 1
  for (int e = threadIdx.x + kThreads; e < items; e += kThreads) {
    const int s0 = slot_of(e), d = dim_of(e);
    Item<T> x, y;
    x.load(ksrc + d, ldk, s0, lo, hi, vec);
    y.load(vsrc + d, ldv, s0, lo, hi, vec);
    x.fold(kt);
    y.fold(vt);
  }
  uint32_t ktop = kt.bits(), vtop = vt.bits();
  block_max(ktop, vtop, red);
  const bool tame = max(ktop, vtop) > kTop;
  if (tame) {  // something is not finite or too large: once more, with what it counts as
    ktop = vtop = 0;
#pragma unroll 1
    for (int e = threadIdx.x; e < (hi - lo) * D; e += kThreads) {
      const int s = lo + e / D, d = e % D;
      ktop = max(ktop, __float_as_uint(fabsf(tamed((float)ksrc[s * ldk + d]))));
      vtop = max(vtop, __float_as_uint(fabsf(tamed((float)vsrc[s * ldv + d]))));
    }
    block_max(ktop, vtop, red);
  }
  if (!real) return;
  constexpr float kMax = KIND == DFS_FP8 ? 448.0f : 127.0f;
  const float kneed = __uint_as_float(ktop) / kMax, vneed = __uint_as_float(vtop) / kMax;
  const Quotient kq(kneed > kold ? kneed : kold), vq(vneed > vold ? vneed : vold);
  if (threadIdx.x == 0) {
    kv.kscale[ph] = kq.scale;
    kv.vscale[ph] = vq.scale;
  }
  uint8_t* kc = kv.k + ph * P * D;
  uint8_t* vc = kv.v + ph * P * D;
  if (kneed > kold && lo > 0) {
    // a larger scale: the codes of the tokens already there
    constexpr int kAhead = 8;
    uint32_t* p = (uint32_t*)kc;
#pragma unroll 1
    for (int e = threadIdx.x; e < lo * D / 4; e += kAhead * kThreads) {
      uint32_t c[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) c[i] = *gptr(p + min(e + i * kThreads, lo * D / 4 - 1));
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (e + i * kThreads < lo * D / 4) *gptr_w(p + e + i * kThreads) = again4<KIND>(c[i], kold, kq);
    }
  }
  const int ldw = P / 4 + 1;
#pragma unroll 1
  for (int e = threadIdx.x; e < items; e += kThreads) {
    const int s0 = slot_of(e), d = dim_of(e);
    if (e >= kThreads) {
      k0.load(ksrc + d, ldk, s0, lo, hi, vec);
      v0.load(vsrc + d, ldv, s0, lo, hi, vec);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Piece<T>& x = k0.x[i];
      if (s0 + i < lo || s0 + i >= hi) continue;
      typedef uint32_t CT __attribute__((ext_vector_type(kN / 4)));
      CT w;
#pragma unroll
      for (int c = 0; c < kN; c += 4)
        w[c / 4] = encode4<KIND>(kq(x.at(c, tame)), kq(x.at(c + 1, tame)), kq(x.at(c + 2, tame)),
                                 kq(x.at(c + 3, tame)));
      *gptr_w((CT*)(kc + (s0 + i) * D + d)) = w;
    }
#pragma unroll
    for (int c = 0; c < kN; ++c)
      words[(d + c) * ldw + s0 / 4] =
          encode4<KIND>(vq(v0.x[0].at(c, tame)), vq(v0.x[1].at(c, tame)), vq(v0.x[2].at(c, tame)),
                        vq(v0.x[3].at(c, tame)));
  }
  __syncthreads();
  // value codes by words of four slots, dim after dim.  A word may hold older
  // tokens (first bytes) and later slots (last bytes), which stay.
  const bool grown = vneed > vold && lo > 0;
  const int first = grown ? 0 : w0, n = w1 - first;
#pragma unroll 4
  for (int e = threadIdx.x; e < D * n; e += kThreads) {
    const int d = e / n, w = first + e % n;
    uint32_t* p = (uint32_t*)(vc + d * P) + w;
    const int older = min(max(lo - 4 * w, 0), 4), later = min(max(4 * w + 4 - hi, 0), 4);
    uint32_t c = w >= w0 ? words[d * ldw + w] : 0u;
    if (older + later > 0) {
      const uint32_t was = !grown && e < kThreads ? was0 : *gptr(p);
      const uint32_t om = older == 4 ? 0xFFFFFFFFu : (1u << (8 * older)) - 1u;
      const uint32_t lm = later == 0 ? 0u : 0xFFFFFFFFu << (8 * (4 - later));
      c &= ~(om | lm);
      c |= was & lm;
      c |= (grown && older > 0 ? again4<KIND>(was, vold, vq) : was) & om;
    }
    *gptr_w(p) = c;
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
                       dim3(kv.heads, (unsigned)std::min<int64_t>(most - y, 65535)),
                       dim3(kThreads), (kv.page / 4 + 1) * kv.head_dim * 4, s, kv, b, (const T*)K, ldk, (const T*)V, ldv, vec, (int)y);
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
