// kv8_attention.hip -- attention over the 8-bit paged cache, with a sliding
// window and first tokens that stay visible.  One wave per query token and
// head, 64 keys at a time: one pass with the running maximum and sum of the
// softmax.
#include "dfs_internal.hpp"

namespace dfs {
namespace {

template <int KIND>
__device__ __forceinline__ float decode8(uint8_t c) {
  if constexpr (KIND == DFS_FP8) return e4m3_to_f32(c);
  return (float)(int8_t)c;
}

template <int KIND, typename OT>
__global__ __launch_bounds__(kWave) void attn_kernel(KvAttnLaunch a) {
  const dfs_kv8& kv = a.kv;
  const KvBatch& b = a.b;
  const int P = kv.page, D = kv.head_dim, row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  const int kh = h / (a.q_heads / kv.heads);
  __shared__ float q[256];
  int r = 0;
  for (; r < b.n_req; ++r)
    if (row >= b.tok_start[r] && row < b.tok_start[r + 1]) break;
  if (r == b.n_req) return;
  const int n = min(b.tok_start[r + 1], b.n_tok) - max(b.tok_start[r], 0);
  const int64_t len = max(b.have[r], 0), pos = len - n + (row - max(b.tok_start[r], 0));
  const int64_t keys = min(len, (int64_t)b.table_pages * P);
  for (int d = lane; d < D; d += kWave)
    q[d] = (float)a.Q[row * a.ldq + (int64_t)h * D + d] * a.sm_scale;
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
  for (int64_t j0 = 0; j0 < keys; j0 += kWave) {
    const int64_t j = j0 + lane;
    bool seen = j < keys && j <= pos && (a.window <= 0 || pos - j < a.window || j < a.sinks);
    int pg = -1;
    if (seen) pg = b.table[r * b.ldt + j / P];
    seen = pg >= 0 && pg < kv.n_pages;
    if (__ballot(seen) == 0) continue;
    float s = -INFINITY, vs = 0.0f;
    const int64_t ph = (int64_t)pg * kv.heads + kh;
    if (seen) {
      const uint8_t* k = kv.k + (ph * P + j % P) * D;
      s = 0.0f;
      for (int d = 0; d < D; ++d) s += q[d] * decode8<KIND>(k[d]);
      s *= kv.kscale[ph];
      vs = kv.vscale[ph];
    }
    float mx = s;
    for (int x = 32; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor(mx, x, kWave));
    const float mn = fmaxf(m, mx), alpha = expf(m - mn);
    const float p = seen ? expf(s - mn) : 0.0f;
    m = mn;
    l = l * alpha + wave_sum(p);
    for (int i = 0; i < 4; ++i) o[i] *= alpha;
    const float pv = p * vs;
    for (int x = 0; x < kWave; ++x) {
      const float w = __shfl(pv, x, kWave);
      const int64_t pj = __shfl((int)seen, x, kWave) ? __shfl(ph, x, kWave) : -1;
      if (pj < 0) continue;
      for (int i = 0; i < 4; ++i)
        if (lane + i * kWave < D)
          o[i] += w * decode8<KIND>(kv.v[(pj * D + lane + i * kWave) * P + (j0 + x) % P]);
    }
  }
  for (int i = 0; i < 4; ++i)
    if (lane + i * kWave < D)
      ((OT*)a.O)[row * a.ldo + (int64_t)h * D + lane + i * kWave] =
          (OT)(l > 0.0f ? o[i] / l : 0.0f);
}

}  // namespace

size_t kv8_attention_ws_bytes(const dfs_kv8&, int32_t, int32_t, int32_t) { return 65536; }

hipError_t launch_kv8_attention(const KvAttnLaunch& a, void*, hipStream_t s) {
  const dim3 grid(a.b.n_tok, a.q_heads);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kWave), 0, s, a); };
  if (a.odt == DFS_F16) {
    if (a.kv.dtype == DFS_FP8) go(attn_kernel<DFS_FP8, _Float16>);
    else go(attn_kernel<DFS_INT8, _Float16>);
  } else {
    if (a.kv.dtype == DFS_FP8) go(attn_kernel<DFS_FP8, float>);
    else go(attn_kernel<DFS_INT8, float>);
  }
  return hipGetLastError();
}

}  // namespace dfs
