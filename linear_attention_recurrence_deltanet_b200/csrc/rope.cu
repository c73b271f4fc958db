// Rotary positions over several axes, and the 4-bit paged cache's writer and
// reader (the attention side of the hybrid stack: "Qwen RoPE", DS4Server issue
// #95, Implementation; mRoPE, Core AI model card).
//
// All three stream their rows once: a lane owns eight channels of a head (16
// bytes of bf16), D / 8 lanes a head, whole heads per warp.  The partner half
// of a rotated pair is read by the lane that needs it (an L1 hit) rather than
// exchanged.  A token's angles are shared by its heads: a block computes those of
// its tokens once, in shared memory, and a lane keeps the eight it needs in
// registers while its warp passes over the token's heads.
#include "../../include/gdn.h"
#include "internal.h"
#include "kv4.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTok = 8;     // tokens of a block
constexpr int kMaxHalf = GDN_ROPE_MAX_PAIRS;

struct RopeArgs {
  const void* x;
  void* out;
  int64_t ldx, ldo;  // elements between tokens
  const int32_t* pos;
  int32_t T, H, D, inverse;
};

// float2 j of a token's angles, one padded every eight: the lanes of a head read 16 different bank pairs
__device__ __forceinline__ int at8(int j) { return j + (j >> 3); }
constexpr int kLdCs = kMaxHalf + kMaxHalf / 8;

// The angles of one lane's channels c .. c + 7, sines with the sign of its half, and the pairs' other channels.
struct LaneAngles {
  float c[8], s[8];
  int partner;  // channel of the first partner; -1: not rotated, -2: half is not a multiple of 8, one by one
  __device__ __forceinline__ void load(const float2* cs, int ch, int half) {
    partner = ch >= 2 * half ? -1 : (half & 7) ? -2 : ch < half ? ch + half : ch - half;
    if (partner < 0) return;
    const int j = ch < half ? ch : ch - half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = cs[at8(j + i)];
      c[i] = t.x, s[i] = ch < half ? -t.y : t.y;
    }
  }
};
// Products and sums are rounded one by one (see quantise8).
template <typename T>
__device__ __forceinline__ void rotate(const T* head, int ch, int half, const LaneAngles& a, const float2* cs, float (&x)[8]) {
  load8(head + ch, x);
  if (a.partner >= 0) {
    float y[8];
    load8(head + a.partner, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], a.c[i]), __fmul_rn(y[i], a.s[i]));
  } else if (a.partner == -2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = ch + i;
      if (e >= 2 * half) break;
      const bool first = e < half;
      const int j = first ? e : e - half;
      const float2 t = cs[at8(j)];
      const float p = __fmul_rn(x[i], t.x), q = __fmul_rn(to_f(head[first ? e + half : j]), t.y);
      x[i] = first ? __fsub_rn(p, q) : __fadd_rn(p, q);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ gdn_rope_plan plan, RopeArgs a, int tok) {
  __shared__ float2 cs[kMaxTok][kLdCs];
  const int half = plan.rotary_dim / 2, t0 = blockIdx.x * tok, nt = min(tok, a.T - t0);
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    const int p = a.pos[(int64_t)plan.axis[j] * a.T + t0 + t];
    const float2 r = rope_angle(plan, j, p);
    cs[t][at8(j)] = make_float2(r.x, a.inverse ? -r.y : r.y);
  }
  __syncthreads();
  const int lph = a.D / 8, hpw = 32 / lph;  // lanes a head, heads a warp
  const int lane = threadIdx.x & 31, sub = lane / lph, c = (lane - sub * lph) * 8;
  const int wpt = kWarps / tok, t = (threadIdx.x >> 5) / wpt;  // warps a token; this warp's token
  if (t >= nt) return;
  LaneAngles ang;
  ang.load(cs[t], sub < hpw ? c : a.D, half);
  const T* x_row = (const T*)a.x + (int64_t)(t0 + t) * a.ldx;
  T* o_row = (T*)a.out + (int64_t)(t0 + t) * a.ldo;
#pragma unroll 2
  for (int h = ((threadIdx.x >> 5) % wpt) * hpw + sub; h - sub < a.H; h += wpt * hpw) {
    const bool on = sub < hpw && h < a.H;
    float x[8];
    if (on) rotate(x_row + h * a.D, c, half, ang, cs[t], x);
    __syncwarp();  // out may be x: every lane has read its head before one writes
    if (on) store8(o_row + h * a.D + c, x);
  }
}

struct AppendArgs {
  const void *q, *k, *v;
  void* q_out;
  int64_t ldq, ldk, ldv, ldqo;
  const int32_t *pos, *cu;
  int32_t T, N, Hq;  // Hq = 0: no queries
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const __grid_constant__ gdn_rope_plan plan, AppendArgs a, KvCache cache, int tok, int32_t* status) {
  __shared__ float2 cs[kMaxTok][kLdCs];
  __shared__ int s_seq[kMaxTok], s_at[kMaxTok];
  const int half = plan.rotary_dim / 2, t0 = blockIdx.x * tok, nt = min(tok, a.T - t0);
  // the tokens' sequences: every thread looks at some (one round of loads), beyond 1024 by bisection (ten or more, but
  // a few threads)
  if (a.N <= 4 * kThreads) {
    for (int n = threadIdx.x; n < a.N; n += kThreads) {
      const int lo = max(a.cu[n], t0), hi = min(a.cu[n + 1], t0 + nt);
      for (int t = lo; t < hi; ++t) s_seq[t - t0] = n;
    }
    __syncthreads();
  } else if (threadIdx.x < nt) {
    s_seq[threadIdx.x] = seq_of(a.cu, a.N, t0 + threadIdx.x);
  }
  if (threadIdx.x < nt) {
    const int n = s_seq[threadIdx.x];
    s_at[threadIdx.x] = cache.lens[n] - (a.cu[n + 1] - (t0 + threadIdx.x));  // position in the cache; negative: not stored
  }
  if (!a.pos) __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    cs[t][at8(j)] = rope_angle(plan, j, a.pos ? a.pos[(int64_t)plan.axis[j] * a.T + t0 + t] : s_at[t]);
  }
  __syncthreads();
  constexpr int lph = D / 8, hpw = 32 / lph;
  const int lane = threadIdx.x & 31, sub = lane / lph, c = (lane % lph) * 8;
  const int uq = (a.Hq + hpw - 1) / hpw, uk = (cache.Hkv + hpw - 1) / hpw, upt = uq + 2 * uk;
  const int wpt = kWarps / tok, t = (threadIdx.x >> 5) / wpt;  // warps a token; this warp's token
  if (t >= nt) return;
  LaneAngles ang;
  ang.load(cs[t], c, half);
  const int64_t row = t0 + t;
#pragma unroll 2
  for (int w = (threadIdx.x >> 5) % wpt; w < upt; w += wpt) {
    float x[8];
    if (w < uq) {
      const int h = w * hpw + sub;
      const bool on = h < a.Hq;
      if (on) rotate((const T*)a.q + row * a.ldq + h * D, c, half, ang, cs[t], x);
      __syncwarp();  // q_out may be q
      if (on) store8((T*)a.q_out + row * a.ldqo + h * D + c, x);
      continue;
    }
    const bool key = w < uq + uk;
    const int h = (key ? w - uq : w - uq - uk) * hpw + sub;
    const bool on = h < cache.Hkv;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    if (on && key)
      rotate((const T*)a.k + row * a.ldk + h * D, c, half, ang, cs[t], x);
    else if (on)
      load8((const T*)a.v + row * a.ldv + h * D + c, x);
    uint32_t sw;
    const uint32_t word = quantise8(x, (key ? kKGroup : v_group(D)) / 8, sw);
    const int p = s_at[t];
    if (!on || p < 0) continue;
    const int64_t at = kv_tile_at(cache, D, s_seq[t], p, h);
    if (at < 0) {
      set_status(status, kStatusBadPage | (GDN_K_KV_APPEND << 8));
      continue;
    }
    unsigned char* tile = cache.pool + at;
    const int r = p % kKvTile;
    const int block = (c / 64) * (kKvTile * 32) + (c % 64) / 2;
    if (key) {
      *reinterpret_cast<uint32_t*>(tile + block + r * 32) = word;
      if (c % kKGroup == 0)
        *reinterpret_cast<uint32_t*>(tile + kv_scale_off(D) + (c / kKGroup) * (kKvTile * 4) + r * 4) = sw;
    } else {
      *reinterpret_cast<uint32_t*>(tile + kv_v_off(D) + block + v_row(r) * 32) = word;
      if (c % v_group(D) == 0)
        *reinterpret_cast<uint32_t*>(tile + kv_scale_off(D) + (D / kKGroup + c / v_group(D)) * (kKvTile * 4) + r * 4) = sw;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    read_kernel(const int32_t* __restrict__ cu, int T_tot, int N, KvCache cache, T* __restrict__ k_out,
                T* __restrict__ v_out, int32_t* status) {
  constexpr int lph = D / 8, hpw = 32 / lph;
  const int lane = threadIdx.x & 31, sub = lane / lph, c = (lane % lph) * 8;
  const int upt = (cache.Hkv + hpw - 1) / hpw;
  const int64_t units = (int64_t)T_tot * upt;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(u / upt), h = (int)(u - (int64_t)t * upt) * hpw + sub;
    if (h >= cache.Hkv) continue;
    const int n = seq_of(cu, N, t), p = cache.lens[n] - (cu[n + 1] - t);
    float k[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.0f;
    const int64_t at = p < 0 ? -1 : kv_tile_at(cache, D, n, p, h);
    if (at >= 0) {
      const unsigned char* tile = cache.pool + at;
      const int r = p % kKvTile, block = (c / 64) * (kKvTile * 32) + (c % 64) / 2;
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(tile + block + r * 32);
      const uint32_t vw = *reinterpret_cast<const uint32_t*>(tile + kv_v_off(D) + block + v_row(r) * 32);
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(tile + kv_scale_off(D)) + r;
      dequantise8(kw, sc[(c / kKGroup) * kKvTile], k);
      dequantise8(vw, sc[(D / kKGroup + c / v_group(D)) * kKvTile], v);
    } else if (p >= 0) {
      set_status(status, kStatusBadPage | (GDN_K_KV_READ << 8));
    }
    const int64_t o = ((int64_t)t * cache.Hkv + h) * D + c;
    store8(k_out + o, k);
    store8(v_out + o, v);
  }
}

// Tokens a block: a warp each, which then reads its angles once for all heads, when there are enough to fill the SMs
// (16384 tokens of 26 heads: 95 us with four tokens' heads dealt out to all warps); else the warps share a token's heads.
int tokens_per_block(int32_t T) { return T >= 4 * 148 * kMaxTok ? kMaxTok : T >= 148 * 16 ? 4 : T >= 148 * 8 ? 2 : 1; }

template <typename T>
void append_d(int D, int grid, const gdn_rope_plan& plan, const AppendArgs& a, const KvCache& c, int tok, int32_t* status,
              cudaStream_t st) {
  if (D == 64) append_kernel<T, 64><<<grid, kThreads, 0, st>>>(plan, a, c, tok, status);
  else if (D == 128) append_kernel<T, 128><<<grid, kThreads, 0, st>>>(plan, a, c, tok, status);
  else append_kernel<T, 256><<<grid, kThreads, 0, st>>>(plan, a, c, tok, status);
}
template <typename T>
void read_d(int D, int grid, const int32_t* cu, int32_t T_tot, int32_t N, const KvCache& c, void* k, void* v,
            int32_t* status, cudaStream_t st) {
  if (D == 64) read_kernel<T, 64><<<grid, kThreads, 0, st>>>(cu, T_tot, N, c, (T*)k, (T*)v, status);
  else if (D == 128) read_kernel<T, 128><<<grid, kThreads, 0, st>>>(cu, T_tot, N, c, (T*)k, (T*)v, status);
  else read_kernel<T, 256><<<grid, kThreads, 0, st>>>(cu, T_tot, N, c, (T*)k, (T*)v, status);
}

}  // namespace

cudaError_t launch_rope(const gdn_rope_plan& plan, bool bf16, const void* x, int64_t ldx, const int32_t* pos, int32_t T,
                        int32_t H, int32_t D, bool inverse, void* out, int64_t ldo, cudaStream_t stream) {
  const RopeArgs a{x, out, ldx, ldo, pos, T, H, D, inverse ? 1 : 0};
  const int tok = tokens_per_block(T), grid = (T + tok - 1) / tok;
  LaunchScope scope(GDN_K_ROPE, stream);
  if (bf16) rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(plan, a, tok);
  else rope_kernel<float><<<grid, kThreads, 0, stream>>>(plan, a, tok);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const gdn_rope_plan& plan, bool bf16, int32_t D, int32_t Hq, const void* q, int64_t ldq,
                             const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* pos,
                             const int32_t* cu, int32_t T, int32_t N, const KvCache& cache, void* q_out, int64_t ldqo,
                             int32_t* status, cudaStream_t stream) {
  const AppendArgs a{q, k, v, q_out, ldq, ldk, ldv, ldqo, pos, cu, T, N, q ? Hq : 0};
  const int tok = tokens_per_block(T), grid = (T + tok - 1) / tok;
  LaunchScope scope(GDN_K_KV_APPEND, stream);
  if (bf16) append_d<__nv_bfloat16>(D, grid, plan, a, cache, tok, status, stream);
  else append_d<float>(D, grid, plan, a, cache, tok, status, stream);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(bool bf16, int32_t D, const int32_t* cu, int32_t T, int32_t N, const KvCache& cache,
                           void* k_out, void* v_out, int32_t* status, cudaStream_t stream) {
  const int64_t heads_per_warp = 256 / D, units = (int64_t)T * ((cache.Hkv + heads_per_warp - 1) / heads_per_warp);
  const int64_t blocks = (units + kWarps - 1) / kWarps;
  const int grid = (int)(blocks < 148 * 32 ? blocks : 148 * 32);
  LaunchScope scope(GDN_K_KV_READ, stream);
  if (bf16) read_d<__nv_bfloat16>(D, grid, cu, T, N, cache, k_out, v_out, status, stream);
  else read_d<float>(D, grid, cu, T, N, cache, k_out, v_out, status, stream);
  return cudaGetLastError();
}

}  // namespace gdn
