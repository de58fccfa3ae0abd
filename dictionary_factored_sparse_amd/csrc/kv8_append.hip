// kv8_append.hip -- new keys and values into the 8-bit paged cache, one fp32
// scale per page and head.  Compiled without FMA contraction: each step of
// the recipe in dictfs.h is one correctly rounded fp32 operation.
// One workgroup per page that gets tokens and head.
#include <algorithm>

#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 256;

template <int KIND>
__device__ __forceinline__ uint8_t encode8(float v, float sc) {
  if (sc == 0.0f) return 0;
  const float q = v / sc;
  if constexpr (KIND == DFS_FP8)
    return (uint8_t)(e4m3_rne_satfinite(fabsf(q)) | ((__float_as_uint(v) >> 24) & 0x80u));
  return (uint8_t)(int8_t)(int)fminf(fmaxf(__builtin_rintf(q), -127.0f), 127.0f);
}
template <int KIND>
__device__ __forceinline__ float decode8(uint8_t c) {
  if constexpr (KIND == DFS_FP8) return e4m3_to_f32(c);
  return (float)(int8_t)c;
}

// What an element counts as: NaN 0, the rest within +-65504.
__device__ __forceinline__ float tamed(float v) {
  return v != v ? 0.0f : fminf(fmaxf(v, -65504.0f), 65504.0f);
}

template <int KIND, typename T>
__global__ __launch_bounds__(kThreads) void append_kernel(dfs_kv8 kv, KvBatch b, const T* K,
                                                          int64_t ldk, const T* V, int64_t ldv) {
  __shared__ float red[kThreads / kWave];
  const int P = kv.page, D = kv.head_dim, h = blockIdx.y;
  int slot = blockIdx.x, r = 0, t0 = 0, n = 0, c = 0;
  for (; r < b.n_req; ++r) {
    t0 = min(max(b.tok_start[r], 0), b.n_tok);
    n = min(max(b.tok_start[r + 1], t0), b.n_tok) - t0;
    c = max(b.have[r], 0);
    if (n == 0) continue;
    const int m = (int)(((int64_t)c + n - 1) / P - c / P + 1);
    if (slot < m) break;
    slot -= m;
  }
  if (r == b.n_req) return;
  const int lp = c / P + slot;
  if (lp >= b.table_pages) return;
  const int pg = b.table[r * b.ldt + lp];
  if (pg < 0 || pg >= kv.n_pages) return;
  const int64_t p0 = (int64_t)lp * P;
  const int lo = (int)(max((int64_t)c, p0) - p0);
  const int hi = (int)(min((int64_t)c + n, p0 + P) - p0);
  const int64_t row0 = t0 + p0 - c;  // row of slot 0
  const int64_t ph = (int64_t)pg * kv.heads + h;
  for (int which = 0; which < 2; ++which) {
    const T* src = which ? V : K;
    const int64_t ld = which ? ldv : ldk;
    uint8_t* codes = (which ? kv.v : kv.k) + ph * P * D;
    float* scale = (which ? kv.vscale : kv.kscale) + ph;
    const int ts = which ? 1 : D, ds = which ? P : 1;
    float m = 0.0f;
    for (int e = threadIdx.x; e < (hi - lo) * D; e += kThreads)
      m = fmaxf(m, fabsf(tamed((float)src[(row0 + lo + e / D) * ld + (int64_t)h * D + e % D])));
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = m;
    __syncthreads();
    for (int w = 0; w < kThreads / kWave; ++w) m = fmaxf(m, red[w]);
    const float need = m / (KIND == DFS_FP8 ? 448.0f : 127.0f);
    const float old = lo > 0 ? *scale : 0.0f;
    const float sc = fmaxf(need, old);
    __syncthreads();
    if (need > old)
      for (int e = threadIdx.x; e < lo * D; e += kThreads) {
        uint8_t* q = codes + (e / D) * ts + (e % D) * ds;
        *q = encode8<KIND>(decode8<KIND>(*q) * old, sc);
      }
    for (int e = threadIdx.x; e < (hi - lo) * D; e += kThreads) {
      const float v = tamed((float)src[(row0 + lo + e / D) * ld + (int64_t)h * D + e % D]);
      codes[(lo + e / D) * ts + (e % D) * ds] = encode8<KIND>(v, sc);
    }
    if (threadIdx.x == 0) *scale = sc;
  }
}

}  // namespace

hipError_t launch_kv8_append(const dfs_kv8& kv, const KvBatch& b, const void* K, int64_t ldk,
                             const void* V, int64_t ldv, int32_t dtype, hipStream_t s) {
  // n tokens of a request touch at most (n - 2) / page + 2 pages, and one if n is 1
  const int64_t most =
      std::min<int64_t>(b.n_tok, b.n_tok / kv.page + 2 * (int64_t)b.n_req);
  const dim3 grid((unsigned)most, kv.heads);
  auto go = [&](auto kernel, auto* k, auto* v) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, kv, b, k, ldk, v, ldv);
  };
  if (dtype == DFS_F16) {
    if (kv.dtype == DFS_FP8)
      go(append_kernel<DFS_FP8, _Float16>, (const _Float16*)K, (const _Float16*)V);
    else
      go(append_kernel<DFS_INT8, _Float16>, (const _Float16*)K, (const _Float16*)V);
  } else {
    if (kv.dtype == DFS_FP8)
      go(append_kernel<DFS_FP8, float>, (const float*)K, (const float*)V);
    else
      go(append_kernel<DFS_INT8, float>, (const float*)K, (const float*)V);
  }
  return hipGetLastError();
}

}  // namespace dfs
