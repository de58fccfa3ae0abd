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
// For prompts X, base and Y, each read or written once.  For small A one launch
// keeps U in LDS: a workgroup computes its tile's U with K split over its waves
// and then a chunk of the outputs; several workgroups take chunks of one tile
// and each computes U anew.  Otherwise a first launch splits K over workgroups
// and a second one does the outputs (get_cut holds both sides' times).
//
// Measured: 4 tokens of 4 adapters of rank 16, 4096 -> 4096: 9.2 us.  61 tokens
// of 24 adapters of ranks to 64, 11008 -> 4096 (37 MB): 15.6 and 10.5 us, 25.8 a
// call among others; the first reads 16 rows of A, 64 bytes each, per
// instruction, and takes 10.7 if A lies in the order of those reads.  4099 tokens
// of 7 prompts, ranks to 32, 4096 -> 4096 (102 MB): 19.5 and 22.1 us, 46.5 a call
// (2.2 TB/s): 5 go between and about the two launches, and finding the tiles
// takes 3 of the first.
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

constexpr int kTok = 16;       // tokens of one matrix instruction
constexpr int kMany = 4;       // groups of 16 tokens in a tile of a large batch
constexpr int kChunk = 64;     // elements of d_in, or outputs, that a wave takes at once
constexpr int kSmallT = 256;   // tokens up to which a workgroup stands for a token
constexpr int kMidT = 8192;    // tokens and
constexpr int kMidN = 4095;    // adapters up to which every workgroup finds its own tile

// A tile: up to 16 NG tokens of one adapter.
struct TileHead {
  int32_t key, count;  // adapter (-1: none), tokens; no tokens: no tile
  int32_t rank;
  float scale;
};
template <int NG>
struct Tile : TileHead {
  int32_t tok[kTok * NG];
};
struct AdapterWs {
  int32_t* perm;    // tokens in order of their adapter
  int32_t* plan;    // per tile: first place in perm, tokens, adapter
  int32_t* n_tiles;
  char* tiles;      // of the first launch, for the second
  float* u;         // [slices][T][rank_ld] partial products X A^T of the split form
  int32_t slices;   // of d_in
  int32_t rank_ld;
};

template <int W>
struct FindShared {
  int32_t hist[kMidN + 1];  // tokens of no adapter, and of each
  int16_t key[kMidT];       // 0: no adapter, -1: no token; a wave's tokens stand together
  int32_t scan[W];
  int32_t first;
};
// Ranks that one pass over X computes: 16 NT.
template <int NT, int NG, int W>
struct Part {
  float u[W][kTok * NG][16 * NT + 4];
};
template <int NT, int NG, int W>
struct ShrinkShared {
  Tile<NG> tile;
  union {
    Part<NT, NG, W> part;
    FindShared<W> find;
  };
};
template <int NG, int W>
struct ExpandShared {
  static constexpr int kULd = (NG == 1 ? kMaxAdapterRank : 64) + 8;
  Tile<NG> tile;
  union {
    float u[kTok * NG][kULd];          // until it is halved; then
    float stage[W][kTok][kChunk + 4];  // a step's outputs, where they are written one by one
  };
  _Float16 hi[kTok * NG][kULd], lo[kTok * NG][kULd];
  int32_t exp[kTok * NG];  // hi + lo = u 2^-exp
};
template <int NT, int W>
struct BothShared : ExpandShared<1, W> {
  Part<NT, 1, W> part;
};

__device__ __forceinline__ int key_of(const AdapterLaunch& a, int t) {
  const int id = a.ids[t];
  return id >= 0 && id < a.ad.n ? id : -1;
}

// Count a wave's keys (-1: none): one atomic where they are all equal, as in
// the rows of one request.
__device__ __forceinline__ void count_keys(int32_t* hist, int key) {
  const uint64_t any = __ballot(key >= 0);
  if (any == 0) return;
  const int k = __builtin_amdgcn_readlane(key, __builtin_ctzll(any));
  if (__ballot(key == k) == any) {
    if ((int)(threadIdx.x % kWave) == __builtin_ctzll(any)) atomicAdd(&hist[k], __popcll(any));
  } else if (key >= 0) {
    atomicAdd(&hist[key], 1);
  }
}

// Exclusive sum over the workgroup's threads; *total gets the whole.
template <int W>
__device__ __forceinline__ int block_sum(int v, int32_t* tmp, int* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int x = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int y = __shfl_up(x, o, kWave);
    if (lane >= o) x += y;
  }
  if (lane == kWave - 1) tmp[wave] = x;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wave) base += tmp[w];
    sum += tmp[w];
  }
  __syncthreads();
  *total = sum;
  return base + x - v;
}

__device__ __forceinline__ int rank_of(const AdapterLaunch& a, int key) {
  return key >= 0 ? min(max(*gptr(a.ad.rank + key), 0), a.ad.r_max) : 0;
}

// Tile x of up to kMidT tokens: counts of every adapter say which one tile x
// belongs to, and the places of that adapter's tokens, in order, which of them
// it has.  Every workgroup does this for itself, for less than a launch that
// does it for all of them would take.  A wave holds the keys of tokens that
// follow each other.
template <int NG, int W>
__device__ void find_tile_mid(const AdapterLaunch& a, int x, Tile<NG>& tile, FindShared<W>& sh) {
  constexpr int kThreads = W * kWave, kKeys = kMidT / kThreads, kSize = kTok * NG;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int n = a.ad.n + 1;
  const int keys = (a.T + kThreads - 1) / kThreads;  // of a lane
  const int t0 = wave * keys * kWave + lane;
  int16_t* mykey = sh.key + t0;
  int id[kKeys];  // all loads at once, no branch between them
#pragma unroll
  for (int i = 0; i < kKeys; ++i) id[i] = *gptr(a.ids + min(t0 + i * kWave, a.T - 1));
  for (int i = threadIdx.x; i < n; i += kThreads) sh.hist[i] = 0;
#pragma unroll
  for (int i = 0; i < kKeys; ++i)
    if (i < keys)
      mykey[i * kWave] = (int16_t)(t0 + i * kWave >= a.T ? -1 : id[i] >= 0 && id[i] < a.ad.n ? id[i] + 1 : 0);
  __syncthreads();
  // (loops that are not unrolled: code that runs once costs its own fetch)
#pragma unroll 1
  for (int i = 0; i < keys; ++i) count_keys(sh.hist, mykey[i * kWave]);
  __syncthreads();
  // every wave looks for the tile, 64 adapters at a time
  int tile0 = 0, mine = -1, first = 0, count = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n && mine < 0; i0 += kWave) {
    const int i = i0 + lane;
    const int c = i < n ? sh.hist[i] : 0, tiles = (c + kSize - 1) / kSize;
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int y = __shfl_up(sum, o, kWave);
      if (lane >= o) sum += y;
    }
    const int at = tile0 + sum - tiles;
    const uint64_t hit = __ballot(x >= at && x < at + tiles);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      mine = i0 + l;
      first = (x - __builtin_amdgcn_readlane(at, l)) * kSize;
      count = min(__builtin_amdgcn_readlane(c, l) - first, kSize);
    }
    tile0 += __builtin_amdgcn_readlane(sum, kWave - 1);
  }
  if (mine < 0) return;  // every wave leaves
  const int r = rank_of(a, mine - 1);
  const float scale = mine > 0 ? *gptr(a.ad.scale + mine - 1) : 0.0f;
  int had = 0;  // this wave's tokens of the adapter
#pragma unroll 1
  for (int i = 0; i < keys; ++i) had += __popcll(__ballot(mykey[i * kWave] == mine));
  if (lane == 0) sh.scan[wave] = had;
  __syncthreads();
  int at = -first;
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < wave) at += sh.scan[w];
#pragma unroll 1
  for (int i = 0; i < keys; ++i) {
    const bool hit = mykey[i * kWave] == mine;
    const uint64_t match = __ballot(hit);
    const int place = at + __popcll(match & ((1ull << lane) - 1));
    if (hit && place >= 0 && place < kSize) tile.tok[place] = t0 + i * kWave;
    at += __popcll(match);
  }
  if (threadIdx.x == 0) {
    tile.key = mine - 1;
    tile.count = count;
    tile.rank = r;
    tile.scale = scale;
  }
  __syncthreads();
}

// Tile x of up to kSmallT tokens, by one wave: x stands for a token, which has
// a tile if its place among those of its adapter is a multiple of 16.
__device__ __forceinline__ void find_tile_small(const AdapterLaunch& a, int x, Tile<1>& tile) {
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    int key[kSmallT / kWave];
#pragma unroll
    for (int c = 0; c < kSmallT / kWave; ++c)
      key[c] = *gptr(a.ids + min(c * kWave + lane, a.T - 1));
#pragma unroll
    for (int c = 0; c < kSmallT / kWave; ++c)
      key[c] = c * kWave + lane >= a.T ? -2 : key[c] >= 0 && key[c] < a.ad.n ? key[c] : -1;
    int mine = -2, place = 0, before = 0;
#pragma unroll
    for (int c = 0; c < kSmallT / kWave; ++c)
      if (c == x / kWave) mine = __builtin_amdgcn_readlane(key[c], x % kWave);
    const int r = rank_of(a, mine);
    const float scale = mine >= 0 ? *gptr(a.ad.scale + mine) : 0.0f;
    uint64_t match[kSmallT / kWave];
#pragma unroll
    for (int c = 0; c < kSmallT / kWave; ++c) {
      match[c] = __ballot(key[c] == mine);
      const int first = c * kWave;
      if (x >= first + kWave) place += __popcll(match[c]);
      else if (x >= first) place += __popcll(match[c] & ((1ull << (x - first)) - 1));
    }
#pragma unroll
    for (int c = 0; c < kSmallT / kWave; ++c) {
      const int at = before + __popcll(match[c] & ((1ull << lane) - 1)) - place;
      if (key[c] == mine && at >= 0 && at < kTok) tile.tok[at] = c * kWave + lane;
      before += __popcll(match[c]);
    }
    if (lane == 0) {
      tile.key = mine;
      tile.count = x < a.T && place % kTok == 0 ? min(before - place, kTok) : 0;
      tile.rank = r;
      tile.scale = scale;
    }
  }
  __syncthreads();
}

// Eight elements of a row from element d on (a multiple of 8), zero from `end`
// on; rows are readable in whole pieces of eight.  No branch: a lane past the
// end reads the last piece and drops it.
__device__ __forceinline__ h8 row8(const _Float16* row, int d, int end) {
  const u4 v = ld16<u4>(row + min(d, (end - 1) & ~7));
  const int n = min(max(end - d, 0), 8);  // elements that count
  u4 keep;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    keep[i] = n >= 2 * i + 2 ? 0xFFFFFFFFu : (n == 2 * i + 1 ? 0xFFFFu : 0u);
  return __builtin_bit_cast(h8, v & keep);
}

// This wave's share of U^T for ranks g0 .. g0 + 16 NT - 1 over the 64-element
// chunks c0 + wave, + kWaves, ... below c1, into part.
template <int NT, int NG, int W>
__device__ __forceinline__ void shrink(const AdapterLaunch& a, const Tile<NG>& tile, int g0, int c0,
                                       int c1, Part<NT, NG, W>& part) {
  constexpr int kAhead = NG > 1 ? 1 : NT == 1 ? 4 : 2;  // chunks whose loads are in flight together
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int r16 = lane & 15, q4 = lane >> 4;
  const _Float16* x[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
    x[g] = a.X + (int64_t)tile.tok[min(g * kTok + r16, tile.count - 1)] * a.ldx;
  const _Float16* A = (const _Float16*)a.ad.A + tile.key * a.ad.stride_a;
  const _Float16* w[NT];
  f4 u[NG][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    w[i] = A + (int64_t)min(g0 + 16 * i + r16, tile.rank - 1) * a.ad.lda;
#pragma unroll
    for (int g = 0; g < NG; ++g) u[g][i] = f4{0, 0, 0, 0};
  }
  const int full = min(c1, a.ad.d_in / kChunk);
  int c = c0 + wave;
#pragma unroll 1
  for (; c + (kAhead - 1) * W < full; c += kAhead * W) {
    h8 xv[kAhead][2][NG], wv[kAhead][2][NT];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int d = (c + k * W) * kChunk + q4 * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int g = 0; g < NG; ++g) xv[k][h][g] = ld16<h8>(x[g] + d + 32 * h);
#pragma unroll
        for (int i = 0; i < NT; ++i) wv[k][h][i] = ld16<h8>(w[i] + d + 32 * h);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int g = 0; g < NG; ++g)
            u[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv[k][h][i], xv[k][h][g], u[g][i], 0,
                                                             0, 0);
  }
#pragma unroll 1
  for (; c < c1; c += W) {  // what is left, and the piece at the end of the rows
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int d = c * kChunk + q4 * 8 + 32 * h;
      h8 xv[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) xv[g] = row8(x[g], d, a.ad.d_in);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const h8 wv = row8(w[i], d, a.ad.d_in);
#pragma unroll
        for (int g = 0; g < NG; ++g)
          u[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, xv[g], u[g][i], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int i = 0; i < NT; ++i) *(f4*)&part.u[wave][g * kTok + r16][16 * i + 4 * q4] = u[g][i];
}

// sh.u to sh.hi + sh.lo, zeros from the rank to the end of the blocks of 32 that
// Expand takes (at least KS); some lanes per token.
template <int KS, int NG, int W>
__device__ __forceinline__ void halve_u(ExpandShared<NG, W>& sh) {
  constexpr int kPer = W * kWave / (kTok * NG);
  const int tok = threadIdx.x / kPer, at = threadIdx.x % kPer;
  const int r = sh.tile.rank, r32 = max((r + 31) / 32, KS) * 32;
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

// A lane's 16 outputs of a step, of 64: 16 bytes in a row at a time, so that the
// four lanes of a token and one access cover 64 bytes.
template <typename YT>
struct Row16 {
  static constexpr int kPer = 16 / sizeof(YT);  // elements of one access
  typedef YT VT __attribute__((ext_vector_type(16 / sizeof(YT))));
  VT v[16 / kPer];
  // Place in the step of the lane's first output of access i.
  static __device__ __forceinline__ int at(int i, int q4) { return (4 * i + q4) * kPer; }
  // The output of the step that row x of the operand of product m is.
  static __device__ __forceinline__ int output(int m, int x) {
    return kPer == 4 ? 16 * m + x : (m >> 1) * 32 + (x >> 2) * 8 + (m & 1) * 4 + (x & 3);
  }
  __device__ __forceinline__ void load(const YT* p, int q4) {
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) v[i] = *gptr((const VT*)(p + at(i, q4)));
  }
  __device__ __forceinline__ void store(YT* p, int q4) const {
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) *gptr_w((VT*)(p + at(i, q4))) = v[i];
  }
};

// The second product: outputs of a tile, 64 per wave and step, one group of 16
// tokens after the other.  What a group needs (base; B for the first KS blocks
// of 32 ranks, kept for the groups of a step) is loaded while the one before
// it is worked on, and the first one's before U is known.
template <typename YT, int KS, int NG, int W>
struct Expand {
  const AdapterLaunch& a;
  ExpandShared<NG, W>& sh;
  const int r, j0, j1, steps, vec, wave, lane, r16, q4;
  const _Float16* B;
  h8 wt[KS][4];
  Row16<YT> y;

  __device__ __forceinline__ Expand(const AdapterLaunch& a_, ExpandShared<NG, W>& sh_, int j0_,
                                    int j1_, int vec_)
      : a(a_), sh(sh_), r(sh_.tile.rank), j0(j0_), j1(j1_),
        steps((j1_ - j0_ + kChunk - 1) / kChunk), vec(vec_), wave(threadIdx.x / kWave),
        lane(threadIdx.x % kWave), r16(lane & 15), q4(lane >> 4),
        B((const _Float16*)a_.ad.B + max(sh_.tile.key, 0) * a_.ad.stride_b) {}

  // Steps start elsewhere in each tile: rows that lie a power of two apart
  // would otherwise keep every workgroup on the same memory channels.
  __device__ __forceinline__ int place(int i) const {
    return j0 + (int)((i + 3u * blockIdx.x) % (unsigned)steps) * kChunk;
  }
  __device__ __forceinline__ h8 weight(int jb, int m, int s) const {
    const int row = min(jb + Row16<YT>::output(m, r16), a.ad.d_out - 1);
    return row8(B + row * a.ad.ldb, s * 32 + q4 * 8, r);
  }
  // Whether the step's outputs are read and written in 16-byte pieces.
  __device__ __forceinline__ bool wide(int jb) const { return vec && jb + kChunk <= j1; }
  __device__ __forceinline__ void load_w(int jb) {
    if (r > 0) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int m = 0; m < 4; ++m) wt[s][m] = weight(jb, m, s);
    }
  }
  // Lanes past the tile's tokens repeat the last one and store nothing.
  __device__ __forceinline__ int64_t token(int g) const {
    return sh.tile.tok[min(g * kTok + r16, sh.tile.count - 1)];
  }
  __device__ __forceinline__ void load_y(int jb, int g) {
    if (a.base && wide(jb)) y.load((const YT*)a.base + token(g) * a.ldbase + jb, q4);
  }
  __device__ __forceinline__ void load_first() {
    if (wave < steps) {
      load_w(place(wave));
      load_y(place(wave), 0);
    }
  }
  __device__ __forceinline__ void run() {
    const float scale = sh.tile.scale;
    const int groups = (sh.tile.count + kTok - 1) / kTok;
    constexpr int kPer = Row16<YT>::kPer;
#pragma unroll 1
    for (int i = wave, g = 0; i < steps;) {
      const int jb = place(i), at = g * kTok;
      const int e = r > 0 ? sh.exp[at + r16] : 0;
      f4 acc[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = f4{0, 0, 0, 0};
      const Row16<YT> base = y;
      if (r > 0) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const h8 uh = *(const h8*)&sh.hi[at + r16][s * 32 + q4 * 8];
          const h8 ul = *(const h8*)&sh.lo[at + r16][s * 32 + q4 * 8];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wt[s][m], uh, acc[m], 0, 0, 0);
            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wt[s][m], ul, acc[m], 0, 0, 0);
          }
        }
        if constexpr (KS == 2 && NG == 1) {
#pragma unroll 1
          for (int s = KS; s * 32 < r; ++s) {
            const h8 uh = *(const h8*)&sh.hi[at + r16][s * 32 + q4 * 8];
            const h8 ul = *(const h8*)&sh.lo[at + r16][s * 32 + q4 * 8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const h8 x = weight(jb, m, s);
              acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, uh, acc[m], 0, 0, 0);
              acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, ul, acc[m], 0, 0, 0);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[m][c] = __builtin_amdgcn_ldexpf(acc[m][c], e);
      }
      const int64_t t = token(g);
      const bool mine = at + r16 < sh.tile.count;
      if (++g == groups) {
        g = 0;
        i += W;
        if (i < steps) load_w(place(i));
      }
      if (i < steps) load_y(place(i), g);
      if (wide(jb)) {
        Row16<YT> out;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float b = a.base ? (float)base.v[c / kPer][c % kPer] : 0.0f;
          out.v[c / kPer][c % kPer] = (YT)(r > 0 ? __builtin_fmaf(scale, acc[c >> 2][c & 3], b) : b);
        }
        if (mine) out.store((YT*)a.Y + t * a.ldy + jb, q4);
      } else {
        // the end of a row, or rows without 16-byte places: by single outputs,
        // lane after lane
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            sh.stage[wave][r16][Row16<YT>::output(m, 4 * q4 + c)] = acc[m][c];
        __builtin_amdgcn_wave_barrier();
        const int j = jb + lane;
#pragma unroll 1
        for (int k = 0; k < min(sh.tile.count - at, kTok); ++k) {
          const int64_t row = sh.tile.tok[at + k];
          if (j < j1) {
            const float b = a.base ? (float)*gptr((const YT*)a.base + row * a.ldbase + j) : 0.0f;
            const float v = sh.stage[wave][k][lane];
            *gptr_w((YT*)a.Y + row * a.ldy + j) = (YT)(r > 0 ? __builtin_fmaf(scale, v, b) : b);
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
};

// One launch, for few tokens and r_max <= 16 NT <= 32: workgroup (x, y)
// computes U of tile x, then chunk y of its outputs.
constexpr int kBothWaves = 8;
template <typename YT, int NT>
__global__ __launch_bounds__(kBothWaves* kWave, 2) void adapter_kernel(AdapterLaunch a, int chunk,
                                                                       int vec) {
  constexpr int W = kBothWaves;
  __shared__ BothShared<NT, W> sh;
  find_tile_small(a, blockIdx.x, sh.tile);
  if (sh.tile.count == 0) return;
  const int j0 = blockIdx.y * chunk;
  Expand<YT, 1, 1, W> x(a, sh, j0, min(j0 + chunk, a.ad.d_out), vec);
  x.load_first();
  if (sh.tile.rank > 0) {
    shrink<NT, 1, W>(a, sh.tile, 0, 0, (a.ad.d_in + kChunk - 1) / kChunk, sh.part);
    __syncthreads();
    for (int e = threadIdx.x; e < kTok * 16 * NT; e += W * kWave) {
      const int tok = e / (16 * NT), rank = e % (16 * NT);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += sh.part.u[w][tok][rank];
      sh.u[tok][rank] = v;
    }
    __syncthreads();
    halve_u<1, 1, W>(sh);
    __syncthreads();
  }
  x.run();
}

// Two launches.  First: slice blockIdx.y of K of a tile's U into ws.u, and the
// tile into ws.tiles.  FIND: how a workgroup comes by its tile.
constexpr int kShrinkWaves = 8;
enum { kFindSmall, kFindMid, kFindPlanned };
template <int FIND, int NT, int NG>
__global__ __launch_bounds__(kShrinkWaves* kWave, 2) void shrink_kernel(AdapterLaunch a,
                                                                        AdapterWs ws) {
  constexpr int W = kShrinkWaves;
  __shared__ ShrinkShared<NT, NG, W> sh;
  const int x = blockIdx.x;
  if (threadIdx.x == 0) sh.tile.count = 0;
  if constexpr (FIND == kFindSmall) {
    find_tile_small(a, x, sh.tile);
  } else if constexpr (FIND == kFindMid) {
    find_tile_mid<NG, W>(a, x, sh.tile, sh.find);
  } else {
    const bool have = x < *ws.n_tiles;
    const int count = have ? ws.plan[3 * x + 1] : 0;
    if ((int)threadIdx.x < count) sh.tile.tok[threadIdx.x] = ws.perm[ws.plan[3 * x] + threadIdx.x];
    if (threadIdx.x == 0) {
      const int key = have ? ws.plan[3 * x + 2] : -1;
      sh.tile.key = key;
      sh.tile.count = count;
      sh.tile.rank = rank_of(a, key);
      sh.tile.scale = key >= 0 ? a.ad.scale[key] : 0.0f;
    }
  }
  __syncthreads();
  Tile<NG>* out = (Tile<NG>*)ws.tiles + x;
  if (blockIdx.y == 0 && threadIdx.x < sizeof(Tile<NG>) / 4)
    ((int32_t*)out)[threadIdx.x] = ((const int32_t*)&sh.tile)[threadIdx.x];
  if (sh.tile.count == 0) return;
  const int r = sh.tile.rank;
  const int chunks = (a.ad.d_in + kChunk - 1) / kChunk;
  const int c0 = (int)((int64_t)chunks * blockIdx.y / ws.slices);
  const int c1 = (int)((int64_t)chunks * (blockIdx.y + 1) / ws.slices);
#pragma unroll 1
  for (int g0 = 0; g0 < r; g0 += 16 * NT) {
    shrink<NT, NG, W>(a, sh.tile, g0, c0, c1, sh.part);
    __syncthreads();
    // four ranks at a time; rows of ws.u have room for whole fours
    for (int e = threadIdx.x; e < sh.tile.count * 4 * NT; e += W * kWave) {
      const int tok = e / (4 * NT), rank = e % (4 * NT) * 4;
      f4 v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < W; ++w) v += *(const f4*)&sh.part.u[w][tok][rank];
      if (g0 + rank < r)
        *gptr_w((f4*)(ws.u + ((int64_t)blockIdx.y * a.T + sh.tile.tok[tok]) * ws.rank_ld + g0 +
                      rank)) = v;
    }
    __syncthreads();
  }
}

// Second: chunk blockIdx.y of the outputs of a tile.
constexpr int kExpandWaves = 4;
template <typename YT, int KS, int NG>
__global__ __launch_bounds__(kExpandWaves* kWave, 3) void expand_kernel(AdapterLaunch a,
                                                                        AdapterWs ws, int chunk,
                                                                        int vec) {
  constexpr int W = kExpandWaves;
  __shared__ ExpandShared<NG, W> sh;
  const Tile<NG>* in = (const Tile<NG>*)ws.tiles + blockIdx.x;
  if (threadIdx.x < sizeof(Tile<NG>) / 4)
    ((int32_t*)&sh.tile)[threadIdx.x] = ((const int32_t*)in)[threadIdx.x];
  __syncthreads();
  if (sh.tile.count == 0) return;
  const int r = sh.tile.rank;
  const int j0 = blockIdx.y * chunk;
  Expand<YT, KS, NG, W> x(a, sh, j0, min(j0 + chunk, a.ad.d_out), vec);
  x.load_first();
  if (r > 0) {
    const int fours = (r + 3) / 4;
#pragma unroll 1
    for (int e = threadIdx.x; e < sh.tile.count * fours; e += W * kWave) {
      const int tok = e / fours, rank = e % fours * 4;
      const float* p = ws.u + (int64_t)sh.tile.tok[tok] * ws.rank_ld + rank;
      f4 v = {0, 0, 0, 0};
#pragma unroll 4
      for (int s = 0; s < ws.slices; ++s) v += *gptr((const f4*)(p + (int64_t)s * a.T * ws.rank_ld));
      *(f4*)&sh.u[tok][rank] = v;
    }
    __syncthreads();
    halve_u<KS, NG, W>(sh);
    __syncthreads();
  }
  x.run();
}

// The tokens in order of their adapter, and the tiles: one workgroup.  The
// order of tokens within an adapter is free (a token's result does not depend
// on its tile), so places are handed out by atomics.
constexpr int kPlanWaves = 16;
__global__ __launch_bounds__(kPlanWaves* kWave) void plan_kernel(AdapterLaunch a, AdapterWs ws,
                                                                 int size) {
  extern __shared__ int32_t place[];  // per adapter, and for no adapter: its count, then its place
  __shared__ int32_t tmp[kPlanWaves];
  const int n = a.ad.n + 1;
  for (int i = threadIdx.x; i < n; i += kPlanWaves * kWave) place[i] = 0;
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int t0 = 0; t0 < a.T; t0 += kPlanWaves * kWave) {
      const int t = t0 + (int)threadIdx.x;
      const int key = t < a.T ? key_of(a, t) + 1 : -1;
      if (pass == 0) {
        count_keys(place, key);
      } else if (key >= 0) {
        ws.perm[atomicAdd(&place[key], 1)] = t;
      }
    }
    __syncthreads();
    if (pass == 1) break;
    int tok0 = 0, tile0 = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanWaves * kWave) {
      const int i = i0 + (int)threadIdx.x;
      const int c = i < n ? place[i] : 0, tiles = (c + size - 1) / size;
      int st, sy;
      const int at_tok = tok0 + block_sum<kPlanWaves>(c, tmp, &st), at_tile = tile0 + block_sum<kPlanWaves>(tiles, tmp, &sy);
      tok0 += st;
      tile0 += sy;
      if (i < n) {
        place[i] = at_tok;
        for (int k = 0; k < tiles; ++k) {
          ws.plan[3 * (at_tile + k)] = at_tok + k * size;
          ws.plan[3 * (at_tile + k) + 1] = min(c - k * size, size);
          ws.plan[3 * (at_tile + k) + 2] = i - 1;
        }
      }
    }
    if (threadIdx.x == 0) *ws.n_tiles = tile0;
    __syncthreads();
  }
}

// How a call is cut.
struct Cut {
  int groups;    // of 16 tokens in a tile: 1 or kMany
  int tiles;     // workgroups of the tile axis
  int chunk;     // outputs per workgroup
  int slices;    // of K in a launch of its own; 0: one launch
  bool planned;  // whether a launch before finds the tiles
};
constexpr int kSlots = 384;  // workgroups of the first launch, while there are fewer tiles
int most_slices(const dfs_adapters& ad) {
  return (ad.d_in + 2 * kShrinkWaves * kChunk - 1) / (2 * kShrinkWaves * kChunk);
}
Cut get_cut(int32_t T, const dfs_adapters& ad) {
  Cut c;
  // Tiles of 64 tokens read A and B a quarter as often, if adapters have that
  // many: rank 32, 4096 -> 4096, 41.4 us against 44.7 in tiles of 16 at 455
  // tokens per adapter, 48.8 and 52.6 at 129, 32.4 and 34.1 at 65, 28.4 and 25.1 at 32.
  c.groups = T > kSmallT && ad.r_max <= 64 && T >= (int64_t)kMany * kTok * (ad.n + 1) ? kMany : 1;
  const int size = c.groups * kTok;
  // tiles that have work, at most
  const int busy = (int)std::min<int64_t>(T, T / size + std::min<int64_t>(ad.n + 1, T));
  c.tiles = T <= kSmallT ? (T + 7) / 8 * 8 : busy;
  // One launch while the A that every workgroup reads is small.  4 tokens, the
  // kernels' own time without what lies between two: rank 8 over 4096, 7.9 us
  // against 8.8 in two launches; 16 over 4096, 9.2 and 9.1; 32 over 2048, 9.0 and
  // 9.4; 32 over 4096, 12.7 and 9.9; 32 over 8192, 20.5 and 9.9.
  const bool both =
      T <= kSmallT && ad.r_max <= 32 && (int64_t)ad.r_max * ad.d_in <= 64 * 1024;
  const int per = (both ? kBothWaves : kExpandWaves) * kChunk;  // outputs of one step
  const int most = (ad.d_out + per - 1) / per;
  const int chunks = std::max(1, std::min(most, (both ? 512 : 1024) / busy));
  c.chunk = ((ad.d_out + chunks - 1) / chunks + kChunk - 1) / kChunk * kChunk;
  c.slices = both ? 0 : std::max(1, std::min(most_slices(ad), kSlots / busy));
  // A launch that plans costs 5.1 us at 1100 tokens and 9.9 at 4099, what the
  // workgroups do instead about 2 and 3; it is for what their LDS cannot hold.
  c.planned = T > kMidT || (T > kSmallT && ad.n > kMidN);
  return c;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }
struct Layout {
  size_t plan, n, tiles, u, total;
  int rank_ld;
};
Layout get_layout(int32_t T, const dfs_adapters& ad, const Cut& c) {
  Layout l;
  l.plan = c.planned ? up((size_t)T * 4) : 0;
  l.n = l.plan + (c.planned ? up((size_t)c.tiles * 12) : 0);
  l.tiles = l.n + (c.planned ? 256 : 0);
  const size_t tile = c.groups == 1 ? sizeof(Tile<1>) : sizeof(Tile<kMany>);
  l.u = l.tiles + (c.slices > 0 ? up(c.tiles * tile) : 0);
  l.rank_ld = (ad.r_max + 3) / 4 * 4;
  l.total = l.u + (size_t)c.slices * T * l.rank_ld * 4;
  return l;
}

template <int FIND, int NG>
void go_shrink(const AdapterLaunch& a, const AdapterWs& w, const Cut& c, hipStream_t s) {
  const dim3 grid(c.tiles, c.slices), block(kShrinkWaves * kWave);
  if (a.ad.r_max <= 16) hipLaunchKernelGGL((shrink_kernel<FIND, 1, NG>), grid, block, 0, s, a, w);
  else if (a.ad.r_max <= 32)
    hipLaunchKernelGGL((shrink_kernel<FIND, 2, NG>), grid, block, 0, s, a, w);
  else hipLaunchKernelGGL((shrink_kernel<FIND, 4, NG>), grid, block, 0, s, a, w);
}

template <typename YT>
void go(const AdapterLaunch& a, const AdapterWs& w, const Cut& c, hipStream_t s) {
  const int vec = ((uintptr_t)a.Y | (uintptr_t)a.base) % 16 == 0 && a.ldy * sizeof(YT) % 16 == 0 &&
                  (!a.base || a.ldbase * sizeof(YT) % 16 == 0);
  const dim3 grid(c.tiles, (a.ad.d_out + c.chunk - 1) / c.chunk);
  if (c.slices == 0) {
    const dim3 block(kBothWaves * kWave);
    if (a.ad.r_max <= 16)
      hipLaunchKernelGGL((adapter_kernel<YT, 1>), grid, block, 0, s, a, c.chunk, vec);
    else
      hipLaunchKernelGGL((adapter_kernel<YT, 2>), grid, block, 0, s, a, c.chunk, vec);
    return;
  }
  if (c.planned)
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanWaves * kWave), (size_t)(a.ad.n + 1) * 4, s,
                       a, w, c.groups * kTok);
  if (a.T <= kSmallT) go_shrink<kFindSmall, 1>(a, w, c, s);
  else if (!c.planned && c.groups == 1) go_shrink<kFindMid, 1>(a, w, c, s);
  else if (!c.planned) go_shrink<kFindMid, kMany>(a, w, c, s);
  else if (c.groups == 1) go_shrink<kFindPlanned, 1>(a, w, c, s);
  else go_shrink<kFindPlanned, kMany>(a, w, c, s);
  const dim3 block(kExpandWaves * kWave);
  auto second = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, w, c.chunk, vec);
  };
  if (c.groups == 1) {
    if (a.ad.r_max <= 32) second(expand_kernel<YT, 1, 1>);
    else second(expand_kernel<YT, 2, 1>);
  } else {
    if (a.ad.r_max <= 32) second(expand_kernel<YT, 1, kMany>);
    else second(expand_kernel<YT, 2, kMany>);
  }
}

}  // namespace

size_t adapter_ws_need(int32_t T, const dfs_adapters& ad) {
  return T > 0 ? get_layout(T, ad, get_cut(T, ad)).total : 0;
}

// Enough for every call of up to T tokens.  A call's own need does not rise with
// its tokens throughout: slices fall in whole steps, and tiles of 64 tokens are
// fewer.  So each part is taken at the most that it can be.
size_t adapter_ws_bytes(int32_t T, const dfs_adapters& ad) {
  if (T <= 0) return 0;
  const Cut c = get_cut(T, ad);
  if (T <= kSmallT && c.slices == 0) return 0;  // so is every smaller batch
  const bool planned = T > kMidT || (T > kSmallT && ad.n > kMidN);
  const bool many = c.groups == kMany;
  // tiles of 16 tokens end where those of 64 begin
  const int64_t t16 = many ? std::min<int64_t>(T, std::max<int64_t>(kSmallT, (int64_t)kMany * kTok * (ad.n + 1)))
                           : T;
  auto busy = [&](int64_t t, int size) {
    return std::min<int64_t>(t, t / size + std::min<int64_t>(ad.n + 1, t));
  };
  const int64_t tiles16 = std::max<int64_t>((std::min<int64_t>(T, kSmallT) + 7) / 8 * 8, busy(t16, kTok));
  const int64_t tiles64 = many ? busy(T, kTok * kMany) : 0;
  size_t bytes = 0;
  if (planned) bytes += up((size_t)T * 4) + up((size_t)std::max(tiles16, tiles64) * 12) + 256;
  bytes += std::max(up(tiles16 * sizeof(Tile<1>)), up(tiles64 * sizeof(Tile<kMany>)));
  // slices * tokens: slices are at most kSlots / busy (or 1), busy is at least
  // tokens / size
  const int64_t rows = std::max<int64_t>(
      T, std::min<int64_t>((int64_t)most_slices(ad) * T, (int64_t)kSlots * (many ? kTok * kMany : kTok)));
  return bytes + (size_t)rows * get_layout(T, ad, c).rank_ld * 4;
}

hipError_t launch_adapter(const AdapterLaunch& a, void* ws, hipStream_t s) {
  const Cut c = get_cut(a.T, a.ad);
  const Layout l = get_layout(a.T, a.ad, c);
  char* p = (char*)ws;
  const AdapterWs w = {(int32_t*)p, (int32_t*)(p + l.plan), (int32_t*)(p + l.n),
                       p + l.tiles, (float*)(p + l.u),      c.slices,
                       l.rank_ld};
  if (a.ydt == DFS_F16) go<_Float16>(a, w, c, s);
  else go<float>(a, w, c, s);
  return hipGetLastError();
}

}  // namespace dfs
