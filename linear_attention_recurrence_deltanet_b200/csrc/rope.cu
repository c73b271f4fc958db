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
// Eight channels of a head and their partners, as loaded: the loads of several heads go out together, before the
// stores of the first, which may be to the same rows.
template <typename T>
struct Loaded {
  static constexpr int V = sizeof(T) / 2;  // 16-byte pieces of eight channels
  uint4 x[V], y[V];
  const T* head;
  __device__ __forceinline__ void load(const T* h, int ch, const LaneAngles& a) {
    head = h;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = ld16_rw(h + ch + 8 / V * i);
      if (a.partner >= 0) y[i] = ld16_rw(h + a.partner + 8 / V * i);
    }
  }
  // the rotated channels.  Products and sums are rounded one by one (see quantise8).
  __device__ __forceinline__ void rotate(int ch, int half, const LaneAngles& a, const float2* cs, float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) Vec16<T>::unpack(x[i], o + 8 / V * i);
    if (a.partner >= 0) {
      float p[8];
#pragma unroll
      for (int i = 0; i < V; ++i) Vec16<T>::unpack(y[i], p + 8 / V * i);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __fadd_rn(__fmul_rn(o[i], a.c[i]), __fmul_rn(p[i], a.s[i]));
    } else if (a.partner == -2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = ch + i;
        if (e >= 2 * half) break;
        const bool first = e < half;
        const int j = first ? e : e - half;
        const float2 t = cs[at8(j)];
        const float p = __fmul_rn(o[i], t.x), q = __fmul_rn(to_f(head[first ? e + half : j]), t.y);
        o[i] = first ? __fsub_rn(p, q) : __fadd_rn(p, q);
      }
    }
  }
};

// Heads h0, h0 + step, .. of one token's row, rotated from x to out (which may be x): U of them in flight.
template <int U, typename T>
__device__ __forceinline__ void rotate_heads_by(const T* x, T* out, int h0, int step, int H, int D, bool lane_on, int c, int half,
                                                const LaneAngles& a, const float2* cs) {
  for (; __any_sync(0xffffffffu, h0 < H); h0 += U * step) {
    Loaded<T> in[U];
    float o[8];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (lane_on && h0 + u * step < H) in[u].load(x + (h0 + u * step) * D, c, a);
    if (U == 1 && lane_on && h0 < H) in[0].rotate(c, half, a, cs, o);  // partners read one by one: before the store
    __syncwarp();  // every lane has read its heads before one writes
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (lane_on && h0 + u * step < H) {
        if (U > 1) in[u].rotate(c, half, a, cs, o);
        store8(out + (h0 + u * step) * D + c, o);
      }
  }
}
template <typename T>
__device__ __forceinline__ void rotate_heads(const T* x, T* out, int h0, int step, int H, int D, bool lane_on, int c, int half,
                                             const LaneAngles& a, const float2* cs) {
  if (half & 7) rotate_heads_by<1>(x, out, h0, step, H, D, lane_on, c, half, a, cs);
  else rotate_heads_by<8 / sizeof(T)>(x, out, h0, step, H, D, lane_on, c, half, a, cs);
}

// The angles of a block's tokens.  A plan is read from parameter space, one lane after the other where their pairs
// differ; several tokens read it from shared memory (16384 tokens: 58 -> 50 us).
template <typename F>
__device__ __forceinline__ void make_angles(const gdn_rope_plan& plan, float2 (*cs)[kLdCs], int half, int nt, const F& pos_of) {
  __shared__ uint64_t s_turn[kMaxHalf];
  __shared__ uint8_t s_axis[kMaxHalf];
  if (nt > 1) {
    for (int j = threadIdx.x; j < half; j += kThreads) s_turn[j] = plan.turn[j], s_axis[j] = plan.axis[j];
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half, j = i - t * half;
      cs[t][at8(j)] = rope_angle(s_turn[j], pos_of(t, s_axis[j]));
    }
  } else {
    for (int j = threadIdx.x; j < half; j += kThreads) cs[0][at8(j)] = rope_angle(plan.turn[j], pos_of(0, plan.axis[j]));
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ gdn_rope_plan plan, RopeArgs a, int tok) {
  __shared__ float2 cs[kMaxTok][kLdCs];
  const int half = plan.rotary_dim / 2, t0 = blockIdx.x * tok, nt = min(tok, a.T - t0);
  make_angles(plan, cs, half, nt, [&](int t, int axis) {
    const int64_t p = a.pos[(int64_t)axis * a.T + t0 + t];
    return a.inverse ? -p : p;  // the inverse turns back
  });
  const int lph = a.D / 8, hpw = 32 / lph;  // lanes a head, heads a warp
  const int lane = threadIdx.x & 31, sub = lane / lph, c = (lane - sub * lph) * 8;
  const int wpt = kWarps / tok, t = (threadIdx.x >> 5) / wpt;  // warps a token; this warp's token
  if (t >= nt) return;
  LaneAngles ang;
  ang.load(cs[t], sub < hpw ? c : a.D, half);
  rotate_heads((const T*)a.x + (int64_t)(t0 + t) * a.ldx, (T*)a.out + (int64_t)(t0 + t) * a.ldo,
               ((threadIdx.x >> 5) % wpt) * hpw + sub, wpt * hpw, a.H, a.D, sub < hpw, c, half, ang, cs[t]);
}

struct AppendArgs {
  const void *q, *k, *v;
  void* q_out;
  int64_t ldq, ldk, ldv, ldqo;
  const int32_t *pos, *cu;
  int32_t T, N, Hq;  // Hq = 0: no queries
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 3)
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
    // (a cu_seqlens that leaves a token out is not the host's copy: the token may go wrong, not the address)
    const int n = s_seq[threadIdx.x] = min((uint32_t)s_seq[threadIdx.x], (uint32_t)a.N - 1u);
    s_at[threadIdx.x] = kv_len(cache, n) - (a.cu[n + 1] - (t0 + threadIdx.x));  // position in the cache; negative: not stored
  }
  if (!a.pos) __syncthreads();
  make_angles(plan, cs, half, nt, [&](int t, int axis) {
    return (int64_t)(a.pos ? a.pos[(int64_t)axis * a.T + t0 + t] : s_at[t]);
  });
  constexpr int lph = D / 8, hpw = 32 / lph;
  const int lane = threadIdx.x & 31, sub = lane / lph, c = (lane % lph) * 8;
  const int uq = (a.Hq + hpw - 1) / hpw, uk = (cache.Hkv + hpw - 1) / hpw;
  const int wpt = kWarps / tok, t = (threadIdx.x >> 5) / wpt;  // warps a token; this warp's token
  if (t >= nt) return;
  LaneAngles ang;
  ang.load(cs[t], c, half);
  const int64_t row = t0 + t;
  const int w0 = (threadIdx.x >> 5) % wpt;
  if (a.Hq)
    rotate_heads((const T*)a.q + row * a.ldq, (T*)a.q_out + row * a.ldqo, w0 * hpw + sub, wpt * hpw, a.Hq, D, true, c, half,
                 ang, cs[t]);
  // keys, then values; the warps that had a query step less begin
  for (int w = (w0 + wpt - uq % wpt) % wpt; w < 2 * uk; w += wpt) {
    const bool key = w < uk;
    const int h = (key ? w : w - uk) * hpw + sub;
    const bool on = h < cache.Hkv;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    if (on && key) {
      Loaded<T> in;
      in.load((const T*)a.k + row * a.ldk + h * D, c, ang);
      in.rotate(c, half, ang, cs[t], x);
    } else if (on) {
      load8((const T*)a.v + row * a.ldv + h * D + c, x);
    }
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
    const int n = seq_of(cu, N, t), p = kv_len(cache, n) - (cu[n + 1] - t);
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
