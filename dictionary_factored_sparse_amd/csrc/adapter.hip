// adapter.hip -- low-rank adapters of many requests beside a shared
// projection: Y[t] = base[t] + scale_a ((X[t] A_a^T) B_a^T), a = ids[t].
//
// Tokens of one adapter are taken 16 at a time (a tile), wherever they stand
// in the batch: the 16 columns of v_mfma_f32_16x16x32_f16, whose rows are
// ranks in the first product (U^T = A X^T) and outputs in the second
// (Y^T = B U^T), so that A and B come straight from memory as operands.
//
// What bounds it.  At decode the adapters' own bytes, once per adapter
// (2 r (d_in + d_out)), and a chain of dependent reads: ids, X and A, then B.
// For prompts X, base and Y, each read or written once.  Hence one launch
// that keeps U in LDS: a workgroup computes its tile's U with K split over its
// waves and then a chunk of the outputs.  With few tiles several workgroups
// take chunks of one tile and each computes U anew: A is then read from L2 by
// all of them, which costs less than a second launch as long as A is small
// (see split_ranks).  Otherwise a first launch splits K over workgroups.
//
// Rounding.  X, A and B are f16 and products of them exact in fp32; sums are
// fp32.  U enters the second product as the sum of two f16 values, 22 bits,
// after a scaling of each token's U by a power of two that brings the largest
// of its ranks near the top of f16's range: neither a large nor a small U
// leaves that range.
#include <algorithm>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kTok = 16;       // tokens per tile
constexpr int kChunk = 64;     // elements of d_in, or outputs, that a wave takes at once
constexpr int kGroup = 64;     // ranks that one pass over X computes
constexpr int kSmallT = 256;   // tokens up to which every workgroup finds its own tile
constexpr int kPartLd = kGroup + 4;
constexpr int kULd = kMaxAdapterRank + 8;

struct AdapterWs {
  int32_t* perm;    // tokens in order of their adapter
  int32_t* tiles;   // per tile: first place in perm, tokens, adapter (-1: none)
  int32_t* n_tiles;
  float* u;         // [slices][T][rank_ld] partial products X A^T of the split form
  int32_t slices;   // of d_in; 0: not split
  int32_t rank_ld;
};

struct Shared {
  float part[kWaves][kTok][kPartLd];
  float u[kTok][kULd];
  _Float16 hi[kTok][kULd], lo[kTok][kULd];
  int32_t exp[kTok];  // hi + lo = u 2^-exp
  int32_t tok[kTok];
  int32_t key, count;
};

__device__ __forceinline__ int key_of(const AdapterLaunch& a, int t) {
  const int id = a.ids[t];
  return id >= 0 && id < a.ad.n ? id : -1;
}

// The tile of workgroup `x` of the tile axis: its adapter and tokens.  For few
// tokens workgroup x stands for token x and has a tile if that token's place
// among those of its adapter is a multiple of 16; for many, x indexes the
// plan's tiles.
__device__ bool find_tile(const AdapterLaunch& a, const AdapterWs& ws, int x, Shared& sh) {
  if (a.T <= kSmallT) {
    if (x >= a.T) return false;
    if (threadIdx.x < kWave) {
      const int lane = threadIdx.x;
      int key[kSmallT / kWave];
#pragma unroll
      for (int c = 0; c < kSmallT / kWave; ++c) {
        const int t = c * kWave + lane;
        key[c] = t < a.T ? key_of(a, t) : -2;
      }
      int mine = -2, place = 0, before = 0;
#pragma unroll
      for (int c = 0; c < kSmallT / kWave; ++c)
        if (c == x / kWave) mine = __builtin_amdgcn_readlane(key[c], x % kWave);
      uint64_t match[kSmallT / kWave];
#pragma unroll
      for (int c = 0; c < kSmallT / kWave; ++c) {
        match[c] = __ballot(key[c] == mine);
        const int first = c * kWave;
        if (x >= first + kWave) place += __popcll(match[c]);
        else if (x >= first) place += __popcll(match[c] & ((1ull << (x - first)) - 1));
      }
      const bool leads = place % kTok == 0;
#pragma unroll
      for (int c = 0; c < kSmallT / kWave; ++c) {
        const int at = before + __popcll(match[c] & ((1ull << lane) - 1)) - place;
        if (key[c] == mine && at >= 0 && at < kTok) sh.tok[at] = c * kWave + lane;
        before += __popcll(match[c]);
      }
      if (lane == 0) {
        sh.key = mine;
        sh.count = leads ? min(before - place, kTok) : 0;
      }
    }
    __syncthreads();
    return sh.count > 0;
  }
  if (x >= *ws.n_tiles) return false;
  const int first = ws.tiles[3 * x], count = ws.tiles[3 * x + 1];
  if (threadIdx.x < count) sh.tok[threadIdx.x] = ws.perm[first + threadIdx.x];
  if (threadIdx.x == 0) {
    sh.key = ws.tiles[3 * x + 2];
    sh.count = count;
  }
  __syncthreads();
  return true;
}

// Eight elements of a row from element d on, zero from `end` on.
__device__ __forceinline__ h8 row8(const _Float16* row, int d, int end) {
  if (d + 8 <= end) return ld16<h8>(row + d);
  h8 v = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (d + i < end) v[i] = *gptr(row + d + i);
  return v;
}

// This wave's share of U^T for ranks g0 .. g0 + 16 NT - 1 over the 64-element
// chunks c0 + wave, + kWaves, ... below c1, into sh.part.
template <int NT>
__device__ __forceinline__ void shrink_ranks(const AdapterLaunch& a, int r, int g0, int c0, int c1,
                                             Shared& sh) {
  constexpr int kAhead = 4 / NT;  // chunks whose loads are in flight together
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int r16 = lane & 15, q4 = lane >> 4;
  const _Float16* x = a.X + (int64_t)sh.tok[min(r16, sh.count - 1)] * a.ldx;
  const _Float16* A = (const _Float16*)a.ad.A + sh.key * a.ad.stride_a;
  const _Float16* w[NT];
  f4 u[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    w[i] = A + (int64_t)min(g0 + 16 * i + r16, r - 1) * a.ad.lda;
    u[i] = f4{0, 0, 0, 0};
  }
  const int full = min(c1, a.ad.d_in / kChunk);
  int c = c0 + wave;
  for (; c + (kAhead - 1) * kWaves < full; c += kAhead * kWaves) {
    h8 xv[kAhead][2], wv[kAhead][NT][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int d = (c + k * kWaves) * kChunk + q4 * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xv[k][h] = ld16<h8>(x + d + 8 * h);
#pragma unroll
        for (int i = 0; i < NT; ++i) wv[k][i][h] = ld16<h8>(w[i] + d + 8 * h);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          u[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv[k][i][h], xv[k][h], u[i], 0, 0, 0);
  }
  for (; c < c1; c += kWaves) {  // what is left, and the piece at the end of the rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = c * kChunk + q4 * 16 + 8 * h;
      const h8 xv = row8(x, d, a.ad.d_in);
#pragma unroll
      for (int i = 0; i < NT; ++i)
        u[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(row8(w[i], d, a.ad.d_in), xv, u[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) *(f4*)&sh.part[wave][r16][16 * i + 4 * q4] = u[i];
}
__device__ __forceinline__ void shrink(const AdapterLaunch& a, int r, int g0, int c0, int c1,
                                       Shared& sh) {
  if (r - g0 <= 16) shrink_ranks<1>(a, r, g0, c0, c1, sh);
  else if (r - g0 <= 32) shrink_ranks<2>(a, r, g0, c0, c1, sh);
  else shrink_ranks<4>(a, r, g0, c0, c1, sh);
}

// sh.u to sh.hi + sh.lo, zeros from rank r to r32 on (32 threads per token).
__device__ __forceinline__ void halve_u(int r, int r32, Shared& sh) {
  constexpr int kPer = kThreads / kTok;
  const int tok = threadIdx.x / kPer, at = threadIdx.x % kPer;
  float top = 0.0f;
  for (int k = at; k < r; k += kPer) top = fmaxf(top, fabsf(sh.u[tok][k]));
#pragma unroll
  for (int o = 1; o < kPer; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
  const int e = __builtin_amdgcn_frexp_expf(top) - 14;  // 0 - 14 for 0, infinities and NaN
  for (int k = at; k < r32; k += kPer) {
    const float v = k < r ? __builtin_amdgcn_ldexpf(sh.u[tok][k], -e) : 0.0f;
    const _Float16 hi = (_Float16)v;
    const float rest = v - (float)hi;
    sh.hi[tok][k] = hi;
    sh.lo[tok][k] = (_Float16)(rest == rest ? rest : 0.0f);  // an infinity has no rest
  }
  if (at == 0) sh.exp[tok] = e;
}

template <typename YT>
__device__ __forceinline__ void load16(const YT* p, bool vec, int n, float* v) {
  if (vec && n == 16) {
    constexpr int kPer = 16 / sizeof(YT);
    typedef YT VT __attribute__((ext_vector_type(kPer)));
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      const VT w = *gptr((const VT*)p + i);
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[i * kPer + k] = (float)w[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? (float)*gptr(p + i) : 0.0f;
  }
}
template <typename YT>
__device__ __forceinline__ void store16(YT* p, bool vec, int n, const float* v) {
  if (vec && n == 16) {
    constexpr int kPer = 16 / sizeof(YT);
    typedef YT VT __attribute__((ext_vector_type(kPer)));
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      VT w;
#pragma unroll
      for (int k = 0; k < kPer; ++k) w[k] = (YT)v[i * kPer + k];
      *gptr_w((VT*)p + i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) *gptr_w(p + i) = (YT)v[i];
  }
}

// Outputs [j0, j1) of a tile from sh.hi + sh.lo, 64 per wave and step.
template <typename YT>
__device__ __forceinline__ void expand(const AdapterLaunch& a, int r, int j0, int j1, bool vec,
                                       Shared& sh) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int steps = (r + 31) / 32;
  const float scale = r > 0 ? a.ad.scale[sh.key] : 0.0f;
  const bool mine = r16 < sh.count;
  const int e = sh.exp[r16];
  const int64_t t = sh.tok[min(r16, sh.count - 1)];
  const _Float16* B = (const _Float16*)a.ad.B + max(sh.key, 0) * a.ad.stride_b;
  for (int jb = j0 + wave * kChunk; jb < j1; jb += kWaves * kChunk) {
    const int j = jb + 16 * q4, n = min(j1 - j, 16);  // this lane's outputs of its token
    f4 acc[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[m] = f4{0, 0, 0, 0};
    float y[16];
    if (a.base && mine && n > 0) {
      load16((const YT*)a.base + t * a.ldbase + j, vec, n, y);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0.0f;
    }
    for (int s = 0; s < steps; ++s) {
      const int k = s * 32 + q4 * 8;
      const h8 uh = *(const h8*)&sh.hi[r16][k], ul = *(const h8*)&sh.lo[r16][k];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        // A row x is output 16 (x / 4) + 4 m + x % 4: a lane's results are then
        // 16 outputs in a row
        const int row = min(jb + (r16 >> 2) * 16 + 4 * m + (r16 & 3), a.ad.d_out - 1);
        const h8 w = k < r ? row8(B + row * a.ad.ldb, k, r) : h8{};
        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, uh, acc[m], 0, 0, 0);
        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, ul, acc[m], 0, 0, 0);
      }
    }
    if (r > 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) 
        y[i] = __builtin_fmaf(scale, __builtin_amdgcn_ldexpf(acc[i >> 2][i & 3], e), y[i]);
    }
    if (mine && n > 0) store16((YT*)a.Y + t * a.ldy + j, vec, n, y);
  }
}

__device__ __forceinline__ int rank_of(const AdapterLaunch& a, int key) {
  return key >= 0 ? min(max(a.ad.rank[key], 0), a.ad.r_max) : 0;
}

// SPLIT: U comes from the partial products of shrink_kernel.
template <typename YT, bool SPLIT>
__global__ __launch_bounds__(kThreads, 4) void adapter_kernel(AdapterLaunch a, AdapterWs ws,
                                                              int chunk, int vec) {
  __shared__ Shared sh;
  if (!find_tile(a, ws, blockIdx.x, sh)) return;
  const int r = rank_of(a, sh.key);
  const int r32 = (r + 31) / 32 * 32;
  if constexpr (SPLIT) {
    for (int e = threadIdx.x; e < kTok * r; e += kThreads) {
      const int tok = e / r, rank = e % r;
      float v = 0.0f;
      if (tok < sh.count) {
        const float* p = ws.u + (int64_t)sh.tok[tok] * ws.rank_ld + rank;
        for (int s = 0; s < ws.slices; ++s) v += *gptr(p + (int64_t)s * a.T * ws.rank_ld);
      }
      sh.u[tok][rank] = v;
    }
    __syncthreads();
  } else {
    for (int g0 = 0; g0 < r; g0 += kGroup) {
      shrink(a, r, g0, 0, (a.ad.d_in + kChunk - 1) / kChunk, sh);
      __syncthreads();
      for (int e = threadIdx.x; e < kTok * kGroup; e += kThreads) {
        const int tok = e / kGroup, rank = e % kGroup;
        if (g0 + rank >= r) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += sh.part[w][tok][rank];
        sh.u[tok][g0 + rank] = v;
      }
      __syncthreads();
    }
  }
  if (r > 0) {
    halve_u(r, r32, sh);
    __syncthreads();
  }
  const int j0 = blockIdx.y * chunk;
  expand<YT>(a, r, j0, min(j0 + chunk, a.ad.d_out), vec != 0, sh);
}

// Slice blockIdx.y of K of a tile's U, into ws.u.
__global__ __launch_bounds__(kThreads, 4) void shrink_kernel(AdapterLaunch a, AdapterWs ws) {
  __shared__ Shared sh;
  if (!find_tile(a, ws, blockIdx.x, sh)) return;
  const int r = rank_of(a, sh.key);
  const int chunks = (a.ad.d_in + kChunk - 1) / kChunk;
  const int c0 = (int)((int64_t)chunks * blockIdx.y / ws.slices);
  const int c1 = (int)((int64_t)chunks * (blockIdx.y + 1) / ws.slices);
  for (int g0 = 0; g0 < r; g0 += kGroup) {
    shrink(a, r, g0, c0, c1, sh);
    __syncthreads();
    for (int e = threadIdx.x; e < sh.count * kGroup; e += kThreads) {
      const int tok = e / kGroup, rank = e % kGroup;
      if (g0 + rank >= r) continue;
      float v = 0.0f;
      for (int w = 0; w < kWaves; ++w) v += sh.part[w][tok][rank];
      *gptr_w(ws.u + ((int64_t)blockIdx.y * a.T + sh.tok[tok]) * ws.rank_ld + g0 + rank) = v;
    }
    __syncthreads();
  }
}

// The tokens in order of their adapter, and the tiles: one workgroup.  The
// order of tokens within an adapter is free (a token's result does not depend
// on its tile), so places are handed out by atomics.
constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(AdapterLaunch a, AdapterWs ws) {
  extern __shared__ int32_t place[];  // per adapter, and for no adapter: its count, then its place
  __shared__ int32_t tmp[2][kPlanThreads / kWave];
  const int n = a.ad.n + 1, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) place[i] = 0;
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int t0 = 0; t0 < a.T; t0 += kPlanThreads) {
      const int t = t0 + (int)threadIdx.x;
      const int key = t < a.T ? key_of(a, t) + 1 : -1;
      // one atomic per wave and key
      for (uint64_t left = __ballot(key >= 0); left != 0;) {
        const int k = __builtin_amdgcn_readlane(key, __builtin_ctzll(left));
        const uint64_t same = __ballot(key == k);
        left &= ~same;
        int at = 0;
        if (lane == __builtin_ctzll(same)) at = atomicAdd(&place[k], __popcll(same));
        at = __builtin_amdgcn_readlane(at, __builtin_ctzll(same));
        if (pass == 1 && key == k) ws.perm[at + __popcll(same & ((1ull << lane) - 1))] = t;
      }
    }
    __syncthreads();
    if (pass == 1) break;
    int tok0 = 0, tile0 = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
      const int i = i0 + (int)threadIdx.x;
      const int c = i < n ? place[i] : 0, tiles = (c + kTok - 1) / kTok;
      int x = c, y = tiles;
      for (int o = 1; o < kWave; o <<= 1) {
        const int p = __shfl_up(x, o, kWave), q = __shfl_up(y, o, kWave);
        if (lane >= o) {
          x += p;
          y += q;
        }
      }
      if (lane == kWave - 1) {
        tmp[0][wave] = x;
        tmp[1][wave] = y;
      }
      __syncthreads();
      int st = tok0, sy = tile0;
      for (int w = 0; w < kPlanThreads / kWave; ++w) {
        if (w < wave) {
          st += tmp[0][w];
          sy += tmp[1][w];
        }
        tok0 += tmp[0][w];
        tile0 += tmp[1][w];
      }
      st += x - c;
      sy += y - tiles;
      if (i < n) {
        place[i] = st;
        for (int k = 0; k < tiles; ++k) {
          ws.tiles[3 * (sy + k)] = st + k * kTok;
          ws.tiles[3 * (sy + k) + 1] = min(c - k * kTok, kTok);
          ws.tiles[3 * (sy + k) + 2] = i - 1;
        }
      }
      __syncthreads();
    }
    if (threadIdx.x == 0) *ws.n_tiles = tile0;
    __syncthreads();
  }
}

// How a call is cut.
struct Cut {
  int tiles;   // workgroups of the tile axis
  int chunk;   // outputs per workgroup
  int slices;  // of K in a launch of its own; 0: U is computed where it is used
};
Cut get_cut(int32_t T, const dfs_adapters& ad) {
  Cut c;
  c.tiles = T <= kSmallT ? (T + 7) / 8 * 8 : (int)(T / kTok + std::min<int64_t>(ad.n + 1, T));
  // tiles that have work, at most
  const int busy = std::min<int64_t>(T, T / kTok + std::min<int64_t>(ad.n + 1, T));
  const int most = (ad.d_out + kWaves * kChunk - 1) / (kWaves * kChunk);
  const int chunks = std::max(1, std::min(most, 512 / busy));
  c.chunk = ((ad.d_out + chunks - 1) / chunks + kChunk - 1) / kChunk * kChunk;
  c.slices = 0;
  if ((int64_t)ad.r_max * ad.d_in > 512 * 1024 / 2 && busy < 256)
    c.slices = std::max(1, std::min((ad.d_in + kWaves * kChunk - 1) / (kWaves * kChunk),
                                    512 / busy));
  if (c.slices == 1) c.slices = 0;
  return c;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }
struct Layout {
  size_t tiles, n, u, total;
  int rank_ld;
};
Layout get_layout(int32_t T, const dfs_adapters& ad, const Cut& c) {
  Layout l;
  const bool plan = T > kSmallT;
  l.tiles = plan ? up((size_t)T * 4) : 0;
  l.n = l.tiles + (plan ? up((size_t)c.tiles * 12) : 0);
  l.u = l.n + (plan ? 256 : 0);
  l.rank_ld = (ad.r_max + 3) / 4 * 4;
  l.total = l.u + (size_t)c.slices * T * l.rank_ld * 4;
  return l;
}

template <typename YT>
void go(const AdapterLaunch& a, const AdapterWs& w, const Cut& c, hipStream_t s) {
  const int vec = ((uintptr_t)a.Y | (uintptr_t)a.base) % 16 == 0 && a.ldy * sizeof(YT) % 16 == 0 &&
                  (!a.base || a.ldbase * sizeof(YT) % 16 == 0);
  const dim3 grid(c.tiles, (a.ad.d_out + c.chunk - 1) / c.chunk);
  if (c.slices > 0) {
    hipLaunchKernelGGL(shrink_kernel, dim3(c.tiles, c.slices), dim3(kThreads), 0, s, a, w);
    hipLaunchKernelGGL((adapter_kernel<YT, true>), grid, dim3(kThreads), 0, s, a, w, c.chunk, vec);
  } else {
    hipLaunchKernelGGL((adapter_kernel<YT, false>), grid, dim3(kThreads), 0, s, a, w, c.chunk,
                       vec);
  }
}

}  // namespace

size_t adapter_ws_bytes(int32_t T, const dfs_adapters& ad) {
  return T > 0 ? get_layout(T, ad, get_cut(T, ad)).total : 0;
}

hipError_t launch_adapter(const AdapterLaunch& a, void* ws, hipStream_t s) {
  const Cut c = get_cut(a.T, a.ad);
  const Layout l = get_layout(a.T, a.ad, c);
  char* p = (char*)ws;
  const AdapterWs w = {(int32_t*)p, (int32_t*)(p + l.tiles), (int32_t*)(p + l.n),
                       (float*)(p + l.u), c.slices, l.rank_ld};
  if (a.T > kSmallT)
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)(a.ad.n + 1) * 4, s, a,
                       w);
  if (a.ydt == DFS_F16) go<_Float16>(a, w, c, s);
  else go<float>(a, w, c, s);
  return hipGetLastError();
}

}  // namespace dfs
