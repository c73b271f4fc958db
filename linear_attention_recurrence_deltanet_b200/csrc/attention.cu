// Causal attention over the 4-bit paged cache (kv4.cuh): for query token i of a
// sequence of `len` cached tokens, of which the last `new` are the queries' own,
//   o = sum_t p_t v_t,  p = softmax over t <= len - new + i of scale q . k_t.
//
// One warp per (token, query head): a key a lane for the scores of 32 keys, then
// D / 32 channels a lane for their values.
#include "../../include/gdn.h"
#include "internal.h"
#include "kv4.cuh"

namespace gdn {
namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128) attention_kernel(AttnProblem a, KvCache cache, int32_t* status) {
  __shared__ float s_q[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + warp;
  if (row >= (int64_t)a.T * a.Hq) return;
  const int t = (int)(row / a.Hq), hq = (int)(row - (int64_t)t * a.Hq), h = hq / (a.Hq / cache.Hkv);
  const int n = seq_of(a.cu, a.N, t), len = cache.lens[n];
  const int seen = len - (a.cu[n + 1] - t) + 1;  // keys this query sees
  for (int c = lane; c < D; c += 32) s_q[warp][c] = to_f(((const T*)a.q)[t * a.ldq + (int64_t)hq * D + c]);
  __syncwarp();
  constexpr int CL = D / 32;
  float m = -INFINITY, l = 0.0f, o[CL];
#pragma unroll
  for (int i = 0; i < CL; ++i) o[i] = 0.0f;
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const int j = j0 + lane;
    const int64_t at = j < seen ? kv_tile_at(cache, D, n, j, h) : -1;
    if (j < seen && at < 0) set_status(status, kStatusBadPage | (GDN_K_ATTENTION << 8));
    float s = -INFINITY;
    if (at >= 0) {
      const unsigned char* tile = cache.pool + at;
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(tile + kv_scale_off(D)) + j % kKvTile;
      s = 0.0f;
      for (int c = 0; c < D; c += 8) {
        float k[8];
        dequantise8(*reinterpret_cast<const uint32_t*>(tile + (c / 64) * 512 + (j % kKvTile) * 32 + (c % 64) / 2),
                    sc[(c / kKGroup) * kKvTile], k);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(s_q[warp][c + i], k[i], s);
      }
      s *= a.scale;
    }
    float mx = s;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float p = at >= 0 ? expf(s - mn) : 0.0f, r = expf(m - mn);
    l = l * r + warp_sum(p);
#pragma unroll
    for (int i = 0; i < CL; ++i) o[i] *= r;
    m = mn;
    for (int u = 0; u < 32; ++u) {
      const int64_t au = __shfl_sync(0xffffffffu, at, u);
      const float pu = __shfl_sync(0xffffffffu, p, u);
      if (au < 0) continue;
      const unsigned char* tile = cache.pool + au;
      const int ju = (j0 + u) % kKvTile, c = lane * CL;
      const uint32_t sw = reinterpret_cast<const uint32_t*>(tile + kv_scale_off(D))[(D / kKGroup + c / v_group(D)) * kKvTile + ju];
      const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + kv_v_off(D) + (c / 64) * 512 + v_row(ju) * 32 + (c % 64) / 8 * 4);
      float v[8];
      dequantise8(w >> (4 * (c % 8)), sw, v);
#pragma unroll
      for (int i = 0; i < CL; ++i) o[i] = fmaf(pu, v[i], o[i]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
#pragma unroll
  for (int i = 0; i < CL; ++i) ((T*)a.o)[row * D + lane * CL + i] = from_f<T>(o[i] * inv);
  if (a.lse && lane == 0) a.lse[row] = m == -INFINITY ? -INFINITY : m + logf(l);
}

template <typename T>
void attention_d(const AttnProblem& p, const KvCache& c, int grid, int32_t* status, cudaStream_t st) {
  if (p.D == 64) attention_kernel<T, 64><<<grid, 128, 0, st>>>(p, c, status);
  else if (p.D == 128) attention_kernel<T, 128><<<grid, 128, 0, st>>>(p, c, status);
  else attention_kernel<T, 256><<<grid, 128, 0, st>>>(p, c, status);
}

}  // namespace

size_t attention_ws_bytes(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

cudaError_t launch_attention(const AttnProblem& p, const KvCache& cache, void*, int32_t* status, cudaStream_t stream) {
  const int grid = (int)(((int64_t)p.T * p.Hq + 3) / 4);
  LaunchScope scope(GDN_K_ATTENTION, stream);
  if (p.bf16) attention_d<__nv_bfloat16>(p, cache, grid, status, stream);
  else attention_d<float>(p, cache, grid, status, stream);
  return cudaGetLastError();
}

}  // namespace gdn
