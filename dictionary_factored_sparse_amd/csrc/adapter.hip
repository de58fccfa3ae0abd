// adapter.hip -- low-rank adapters of many requests beside a shared
// projection: Y[t] = base[t] + scale_a ((X[t] A_a^T) B_a^T), a = ids[t].
// One workgroup per token.
#include "dfs_internal.hpp"

namespace dfs {
namespace {

constexpr int kThreads = 256;

template <typename YT>
__global__ __launch_bounds__(kThreads) void adapter_kernel(AdapterLaunch a) {
  __shared__ float u[kMaxAdapterRank];
  const int t = blockIdx.x;
  const int id = a.ids[t];
  const bool have = id >= 0 && id < a.ad.n;
  const int r = have ? min(max(a.ad.rank[id], 0), a.ad.r_max) : 0;
  const _Float16* x = a.X + (int64_t)t * a.ldx;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  for (int i = wave; i < r; i += kThreads / kWave) {
    const _Float16* w = (const _Float16*)a.ad.A + id * a.ad.stride_a + i * a.ad.lda;
    float s = 0.0f;
    for (int c = lane; c < a.ad.d_in; c += kWave) s += (float)x[c] * (float)w[c];
    s = wave_sum(s);
    if (lane == 0) u[i] = s;
  }
  __syncthreads();
  const float sc = have ? a.ad.scale[id] : 0.0f;
  for (int j = threadIdx.x; j < a.ad.d_out; j += kThreads) {
    float s = 0.0f;
    if (r > 0) {
      const _Float16* w = (const _Float16*)a.ad.B + id * a.ad.stride_b + j * a.ad.ldb;
      for (int i = 0; i < r; ++i) s += u[i] * (float)w[i];
    }
    float y = a.base ? (float)((const YT*)a.base)[t * a.ldbase + j] : 0.0f;
    if (r > 0) y += sc * s;
    ((YT*)a.Y)[t * a.ldy + j] = (YT)y;
  }
}

}  // namespace

size_t adapter_ws_bytes(int32_t, const dfs_adapters&) { return 0; }

hipError_t launch_adapter(const AdapterLaunch& a, void*, hipStream_t s) {
  if (a.ydt == DFS_F16)
    hipLaunchKernelGGL(adapter_kernel<_Float16>, dim3(a.T), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL(adapter_kernel<float>, dim3(a.T), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace dfs
