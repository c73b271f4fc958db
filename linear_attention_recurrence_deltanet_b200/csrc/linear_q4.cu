// Y[M, N] = X[M, K] W[N, K]^T with W in 4 bits: w = scale * code + bias, scale
// and bias (bf16) shared by a group of 32, 64 or 128 input features ("Q4" and
// "MLX affine" weights: DS4Server issues #88, Scope, and #95, implementation
// comment).  Per group
//   y = sum_g scale_ng (x_g . code_ng) + bias_ng sum(x_g).
//
// Packed weights (gdn_q4_pack), zero-filled to whole tiles:
//   codes   [N / 16 tiles][K / 64 blocks][32 lanes] 16 bytes: lane 4r + q holds the
//           words of channels 16q .. 16q+7 and 16q+8 .. 16q+15 of row r, then of
//           row r + 8, of its block -- a warp's fragment of the tile in one
//           16-byte load a lane.  A word holds channel 2i in its nibble i and
//           channel 2i + 1 in its nibble 4 + i, so that masking the word gives
//           pairs of neighbouring channels.
//   scales  [N / 16 tiles][groups][16 rows] words, scale low, bias high
//   rows    [N / 16 tiles][16] floats: the power of two that brings the row's
//           largest weight below 2^11
#include <algorithm>

#include "../../include/gdn.h"
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"
#include "vec.cuh"

namespace gdn {
namespace {

constexpr int kTile = 16, kBlock = 64;

__global__ void q4_pack_kernel(const unsigned char* __restrict__ codes, const unsigned short* __restrict__ scales,
                               const unsigned short* __restrict__ biases, int N, int K, int group, int64_t row_bytes,
                               Q4Layout L, uint32_t* __restrict__ out) {
  const int64_t words = (int64_t)L.row_off / 4, scale_words = (int64_t)L.scale_off / 4;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x) {
    uint32_t w = 0;
    if (i < scale_words) {
      const int64_t blk = i / 128;
      const int in = (int)(i - blk * 128), lane = in / 4, part = in & 3;
      const int64_t n = blk / L.blocks * kTile + lane / 4 + (part >> 1) * 8;
      const int64_t k0 = blk % L.blocks * kBlock + (lane & 3) * 16 + (part & 1) * 8;
      if (n < N)
        for (int b = 0; b < 4; ++b)
          if (k0 + 2 * b < K) {
            const uint32_t byte = codes[n * row_bytes + k0 / 2 + b];
            const uint32_t odd = k0 + 2 * b + 1 < K ? byte >> 4 : 0;
            w |= (byte & 15u) << (4 * b) | odd << (16 + 4 * b);
          }
    } else {
      const int64_t j = i - scale_words, n = j / 16 / L.groups * kTile + j % 16, g = j / 16 % L.groups;
      if (n < N)
        w = (uint32_t)scales[n * L.groups + g] | ((uint32_t)biases[n * L.groups + g] << 16);
    }
    out[i] = w;
  }
}

// a warp a row: the power of two that brings the row's largest finite weight, at code 0 or 15, below 2^11
__global__ void q4_rows_kernel(const unsigned short* __restrict__ scales, const unsigned short* __restrict__ biases, int N,
                               Q4Layout L, float* __restrict__ rows) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= L.tiles * kTile) return;
  uint32_t top = 0;
  if (n < N)
    for (int g = lane; g < L.groups; g += 32) {
      const float s = __uint_as_float((uint32_t)scales[(int64_t)n * L.groups + g] << 16);
      const float b = __uint_as_float((uint32_t)biases[(int64_t)n * L.groups + g] << 16);
      const uint32_t e0 = __float_as_uint(b) & 0x7fffffffu, e1 = __float_as_uint(fmaf(15.0f, s, b)) & 0x7fffffffu;
      const uint32_t e2 = __float_as_uint(s) & 0x7fffffffu;
      if (e0 < 0x7f800000u) top = max(top, e0);
      if (e1 < 0x7f800000u) top = max(top, e1);
      if (e2 < 0x7f800000u) top = max(top, e2);
    }
  top = __reduce_max_sync(0xffffffffu, top);
  const int e = max(-100, (int)(top >> 23) - 127);
  if (lane == 0) rows[n] = __uint_as_float((uint32_t)(127 + 10 - e) << 23);
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The weight stream: each warp copies chunks of B blocks of its 16 rows, and their groups' scale words, into a ring of
// its own, so that the copies run ahead of the products whatever the other warps do.
template <int B, int S>
struct Ring {
  static constexpr int kSlot = B * 512 + 64 * 2 * B;  // groups of 32: two a block
  unsigned char* smem;
  uint64_t* full;  // [S]
  int head = 0;    // chunks asked for
  __device__ __forceinline__ void fetch(const unsigned char* packed, const Q4Layout& L, int lg, int64_t tile, int block) {
    const int nb = min(B, L.blocks - block), g0 = (block * kBlock) >> lg;
    const int ng = min(L.groups, (((block + nb) * kBlock - 1) >> lg) + 1) - g0;
    unsigned char* d = smem + (head % S) * kSlot;
    uint64_t* m = full + head % S;
    tc::mbar_expect_tx(m, nb * 512 + ng * 64);
    tc::bulk_load(d, packed + (tile * L.blocks + block) * 512, nb * 512, m);
    tc::bulk_load(d + B * 512, packed + L.scale_off + (tile * L.groups + g0) * 64, ng * 64, m);
    ++head;
  }
};
constexpr int64_t kWaitCycles = 4000000000ll;  // about two seconds
constexpr int kSms = 148;

// ------------------------------------------------------------------ few rows
// Up to 8 MT rows of x a block: the codes go to the tensor cores as bf16
// integers (A: 16 weight rows, B: 8 rows of x), each group's products are scaled
// in fp32, so nothing but the sums is rounded.  bf16 io takes 128 + code (one
// mask a pair), fp32 io code - 8 and three bf16 parts of x.
//
// A block takes 16 weight rows; its warps, and those of the `S` blocks of its
// cluster, deal the groups of K out and join in shared memory.  The weight
// stream bounds it: a warp keeps 2 KB of codes in flight ahead of the products.
constexpr int kSmallWarps = 8, kSmallThreads = kSmallWarps * 32;

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool F32>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {  // channels 2i, 2i + 1 of a word
  const uint32_t c = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  if constexpr (!F32) return c;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(c), "r"(0x43084308u));
  return r;
}

constexpr int kSmallB = 2, kSmallS = 4;  // blocks of a chunk, chunks of a warp's ring

template <typename T, int MT, int G>
__global__ void __launch_bounds__(kSmallThreads, 2)
    linear_small_kernel(const T* __restrict__ x, int M, int K, const unsigned char* __restrict__ packed, Q4Layout L,
                        int N, T* __restrict__ y, int S, int32_t* status) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int P = F32 ? 3 : 1;                 // bf16 parts of x
  constexpr int NB = G == 128 ? 2 : 1;           // 64-channel blocks that are scaled together
  constexpr int SUB = G == 32 ? 2 : 1;           // groups of a block
  constexpr int LG = G == 32 ? 5 : G == 64 ? 6 : 7;
  using R = Ring<kSmallB, kSmallS>;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ uint64_t s_full[kSmallWarps][kSmallS];
  __shared__ float s_part[kSmallWarps][MT * 4][32];
  __shared__ float s_sum[MT * 128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  const int rank = (int)blockIdx.x % S, m0 = (int)blockIdx.y * MT * 8;
  const int first = (int)blockIdx.x / S, stride = (int)gridDim.x / S;  // row tiles of this cluster
  const int chunks = (L.blocks + kSmallB - 1) / kSmallB, step = S * kSmallWarps, w0 = rank * kSmallWarps + warp;

  if (threadIdx.x < kSmallWarps * kSmallS) tc::mbar_init(&s_full[threadIdx.x / kSmallS][threadIdx.x % kSmallS], 1);
  tc::mbar_init_fence();
  __syncthreads();
  R ring{ring_smem + warp * kSmallS * R::kSlot, s_full[warp]};
  int ft = first, fc = w0;  // the next chunk to ask for
  auto fetch = [&]() {
    if (fc < chunks && ft < L.tiles) {
      if (lane == 0) ring.fetch(packed, L, LG, ft, fc * kSmallB);
      fc += step;
      if (fc >= chunks) fc = w0, ft += stride;
    }
  };
  for (int i = 0; i < kSmallS; ++i) fetch();
  int used = 0;
  bool dead = false;

  for (int tile = first; tile < L.tiles; tile += stride) {
  float acc[MT][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.0f;

  for (int c = w0; c < chunks && !dead; c += step) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait_cycles(ring.full + used % kSmallS, (used / kSmallS) & 1, kWaitCycles))) {
      set_status(status, kStatusWaitTimeout | (GDN_K_LINEAR_Q4 << 8));
      dead = true;
      break;
    }
    const unsigned char* slot = ring.smem + (used % kSmallS) * R::kSlot;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(slot + kSmallB * 512);
#pragma unroll
    for (int i = 0; i < kSmallB / NB; ++i) {
      const int u = c * (kSmallB / NB) + i;
      if (u * NB >= L.blocks) break;
      float p[SUB][MT][4], xs[SUB][MT][4];
#pragma unroll
      for (int g = 0; g < SUB; ++g)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[g][t][e] = xs[g][t][e] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (u * NB + b >= L.blocks) break;
        const uint4 cw = *reinterpret_cast<const uint4*>(slot + (i * NB + b) * 512 + lane * 16);
        uint32_t a[8][2];  // pairs of the lane's 16 channels, rows r and r + 8
        const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j][0] = code_pair<F32>(w[j >> 2], j & 3);
          a[j][1] = code_pair<F32>(w[2 + (j >> 2)], j & 3);
        }
        const int k = (u * NB + b) * kBlock + q * 16;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const int m = m0 + t * 8 + r;
          const T* src = x + (int64_t)m * K + k;
          uint32_t f[P][8];
          if constexpr (!F32) {
            uint4 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              v[h] = m < M && k + 8 * h < K ? ld16(src + 8 * h) : make_uint4(0, 0, 0, 0);
            f[0][0] = v[0].x, f[0][1] = v[0].y, f[0][2] = v[0].z, f[0][3] = v[0].w;
            f[0][4] = v[1].x, f[0][5] = v[1].y, f[0][6] = v[1].z, f[0][7] = v[1].w;
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint4 v = m < M && k + 4 * h < K ? ld16(src + 4 * h) : make_uint4(0, 0, 0, 0);
              float e[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
#pragma unroll
              for (int part = 0; part < P; ++part)
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                  const uint32_t z = bf16x2(e[2 * d], e[2 * d + 1]);
                  f[part][2 * h + d] = z;
                  e[2 * d] -= lo_bf16(z), e[2 * d + 1] -= hi_bf16(z);
                }
            }
          }
#pragma unroll
          for (int part = 0; part < P; ++part)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int g = 0; g < SUB; ++g) {
                // groups of 32: lanes q < 2 hold the first, q >= 2 the second
                const bool on = SUB == 1 || (q >> 1) == g;
                const uint32_t b0 = on ? f[part][2 * j] : 0u, b1 = on ? f[part][2 * j + 1] : 0u;
                mma(p[g][t], a[2 * j][0], a[2 * j][1], a[2 * j + 1][0], a[2 * j + 1][1], b0, b1);
                mma(xs[g][t], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, b0, b1);
              }
        }
      }
#pragma unroll
      for (int g = 0; g < SUB; ++g) {
        if (u * SUB + g >= L.groups) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w = sc[(i * SUB + g) * 16 + r + 8 * h];
          const float s = lo_bf16(w), z = fmaf(F32 ? 8.0f : -128.0f, s, hi_bf16(w));
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              acc[t][2 * h + e] = fmaf(s, p[g][t][2 * h + e], fmaf(z, xs[g][t][e], acc[t][2 * h + e]));
        }
      }
    }
    ++used;
    __syncwarp();  // the slot is read before lane 0 refills it
    fetch();
  }

#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_part[warp][t * 4 + e][lane] = acc[t][e];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 128; i += kSmallThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) v += s_part[w][i >> 5][i & 31];
    s_sum[i] = v;
  }
  if (S > 1) tc::cluster_sync();
  else __syncthreads();
  if (rank == 0) {
    for (int i = threadIdx.x; i < MT * 128; i += kSmallThreads) {
      const int n_in = i & 15, m_in = i >> 4;  // neighbouring threads write neighbouring outputs
      const int at = ((m_in >> 3) * 4 + (n_in >> 3) * 2 + (m_in & 1)) * 32 + (n_in & 7) * 4 + ((m_in & 7) >> 1);
      float v = s_sum[at];
      for (int o = 1; o < S; ++o) {
        float f;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(tc::mapa_shared(tc::smem_u32(&s_sum[at]), o)));
        v += f;
      }
      const int n = tile * kTile + n_in, m = m0 + m_in;
      if (n < N && m < M) y[(int64_t)m * N + n] = from_f<T>(v);
    }
  }
  if (S > 1) tc::cluster_sync();  // the leader has read the others' sums
  }
  if (dead && lane == 0)  // the copies still in flight land before the block exits
    for (int j = used; j < ring.head; ++j) tc::mbar_wait_cycles(ring.full + j % kSmallS, (j / kSmallS) & 1, kWaitCycles / 100);
}

// ------------------------------------------------------------------ many rows
// Rows past kSmallRows (bf16 io): tcgen05 products of 128 weight rows (A) and
// `tn` rows of x (B), in fp16.  Weights are expanded to fp16 tiles in shared
// memory by eight warps, one of the tile's 16-row strips each; scaled by a power of two a row (q4_pack) so that
// the row's largest value is below 2^11, a weight is off by half a step, 2^-11,
// against 2^-8 in bf16.  x goes through x_half_kernel: fp16 with a power of two
// a row, exact but for elements 2^-25 of the row's largest and smaller, laid out
// as the tiles that the products read.
//
// Warp 0 loads x, warp 1 issues the products, warps 2-5 write the accumulator
// out, warps 6-13 expand.  Two accumulators, so that one tile's output overlaps
// the next one's products.  With fewer tiles than SMs a cluster of S blocks
// splits K and joins in the leader's shared memory.
constexpr int kBM = 128, kExpandWarps = 8, kBigThreads = (6 + kExpandWarps) * 32;
constexpr int kBigB = 4, kBigS = 3;  // blocks of a chunk, chunks of a warp's ring
using BigRing = Ring<kBigB, kBigS>;
constexpr int kWStage = kBM * kBlock * 2, kMaxRing = 8;
constexpr int kCodeRing = kExpandWarps * kBigS * BigRing::kSlot;  // 60 KB
constexpr int kBigRing = 147456, kBigSmem = kBigRing + kCodeRing + 1024;  // 144 KB: three stages at 256 rows of x
static_assert(kBigSmem + 2048 <= 232448, "shared memory of a block");

struct BigArgs {
  const unsigned char* packed;
  Q4Layout L;
  const unsigned char* xh;  // [blocks][mp][128 bytes]
  const float* xf;          // [mp]: power of two of each row
  __nv_bfloat16* y;
  int32_t M, N, mp, tn, lg_group, S;
  int32_t* status;
};

// one block a row of x: fp16 scaled to below 2^11, into the layout of the products' operand
__global__ void __launch_bounds__(256) x_half_kernel(const __nv_bfloat16* __restrict__ x, int M, int K, int blocks, int mp,
                                                     unsigned char* __restrict__ xh, float* __restrict__ xf) {
  __shared__ uint32_t s_top[8];
  const int m = blockIdx.x;
  const int chunks = blocks * 8;
  const __nv_bfloat16* row = x + (int64_t)m * K;
  uint32_t top = 0;  // largest finite magnitude, as bits
  if (m < M)
    for (int c = threadIdx.x; c * 8 < K; c += 256) {
      const uint4 v = ld16(row + c * 8);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = (w[i] << 16) & 0x7fff0000u, b = w[i] & 0x7fff0000u;
        if (a < 0x7f800000u) top = max(top, a);
        if (b < 0x7f800000u) top = max(top, b);
      }
    }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = max(top, s_top[w]);
  asm volatile("griddepcontrol.launch_dependents;");
  // exponent e of the largest: values times 2^(10 - e) are below 2^11
  const int e = max(-100, (int)(top >> 23) - 127);
  const float f = __uint_as_float((uint32_t)(127 + 10 - e) << 23);
  if (threadIdx.x == 0) xf[m] = __uint_as_float((uint32_t)(127 + e - 10) << 23);
  for (int c = threadIdx.x; c < chunks; c += 256) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (m < M && c * 8 < K) Vec16<__nv_bfloat16>::unpack(ld16(row + c * 8), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= f;
    *reinterpret_cast<uint4*>(xh + ((int64_t)(c >> 3) * mp + m) * 128 + (((c & 7) ^ (m & 7)) << 4)) = tc::pack8h(v);
  }
}

// codes of a word -> eight fp16 weights s code + b (one rounding).  Nibbles 0, 2 (and 4, 6) are masked into 1024 + c,
// nibbles 1, 3 into 1024 + 16 c, which saves their shift.
__device__ __forceinline__ uint4 expand(uint32_t w, __half2 s, __half2 b) {
  uint32_t o[4];
  const __half2 k1024 = __half2half2(__ushort_as_half(0x6400)), k16 = __half2half2(__ushort_as_half(0x2c00)),
                k64 = __half2half2(__ushort_as_half(0xd400));  // 1024, 1/16, -64
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = (w & 0x000f000fu) | 0x64006400u, hi = (w & 0x00f000f0u) | 0x64006400u;
    const __half2 cl = __hsub2(*reinterpret_cast<const __half2*>(&lo), k1024);
    const __half2 ch = __hfma2(*reinterpret_cast<const __half2*>(&hi), k16, k64);
    const __half2 wl = __hfma2(cl, s, b), wh = __hfma2(ch, s, b);
    o[2 * i] = *reinterpret_cast<const uint32_t*>(&wl);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&wh);
    w >>= 8;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kBigThreads, 1) linear_big_kernel(const __grid_constant__ BigArgs a) {
  using namespace tc;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full_c[kExpandWarps][kBigS], full_x[kMaxRing], full_w[kMaxRing], empty[kMaxRing], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tslot;
  bool bad = false;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int xbytes = a.tn * 128, stage_bytes = kWStage + xbytes;
  const int stages = min(kMaxRing, kBigRing / stage_bytes);
  const int mt = a.mp / a.tn, nt = (a.N + kBM - 1) / kBM;
  const int rank = a.S > 1 ? (int)cluster_ctarank() : 0;
  const int tiles = mt * nt, first = (int)blockIdx.x / a.S, stride = (int)gridDim.x / a.S;
  auto slice = [&](int i) { return i == a.S ? a.L.blocks : (int)((int64_t)a.L.blocks * i / a.S) & ~1; };  // whole groups
  const int kb0 = slice(rank), nk = slice(rank + 1) - kb0;

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full_x[s], 1);
      mbar_init(&full_w[s], kExpandWarps);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kExpandWarps * kBigS; ++s) mbar_init(&full_c[s / kBigS][s % kBigS], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(&drain, 1);
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(&tslot, 512);
  sync_tc();
  const uint32_t tbase = tslot;

  if (warp == 0) {
    if (lane == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // x_half_kernel's output
      int i = 0, last[kMaxRing];
      for (int s = 0; s < kMaxRing; ++s) last[s] = -1;
      for (int t = first; t < tiles && !bad; t += stride) {
        const int m0 = (t % mt) * a.tn;
        for (int kb = 0; kb < nk; ++kb, ++i) {
          const int s = i % stages;
          if (i >= stages && !mbar_wait_cycles(&empty[s], ((i / stages) & 1) ^ 1, kWaitCycles)) {
            bad = true;
            break;
          }
          mbar_expect_tx(&full_x[s], xbytes);
          bulk_load(sm + s * stage_bytes + kWStage, a.xh + ((int64_t)(kb0 + kb) * a.mp + m0) * 128, xbytes, &full_x[s]);
          last[s] = i;
        }
      }
      if (bad)  // let the copies already issued land before the block exits
        for (int s = 0; s < stages; ++s)
          if (last[s] >= 0) mbar_wait_cycles(&full_x[s], (last[s] / stages) & 1, kWaitCycles);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id = idesc_f16(kBM, a.tn, false, false);
      int i = 0, j = 0;
      for (int t = first; t < tiles && !bad; t += stride, ++j) {
        const int ab = j & 1;
        if (j >= 2 && !mbar_wait_cycles(&acc_empty[ab], ((j >> 1) & 1) ^ 1, kWaitCycles)) {
          bad = true;
          break;
        }
        fence_after();
        const uint32_t d = tbase + 256 * ab;
        for (int kb = 0; kb < nk; ++kb, ++i) {
          const int s = i % stages;
          if (!mbar_wait_cycles(&full_x[s], (i / stages) & 1, kWaitCycles) || !mbar_wait_cycles(&full_w[s], (i / stages) & 1, kWaitCycles)) {
            bad = true;
            break;
          }
          fence_after();
          const uint32_t w = smem_u32(sm + s * stage_bytes), x = w + kWStage;
#pragma unroll
          for (int kk = 0; kk < kBlock / 16; ++kk)
            mma_f16(d, desc_kmaj(w, kBM, kk), desc_kmaj(x, a.tn, kk), id, (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&empty[s]);
        }
        if (!bad) mma_commit(&acc_full[ab]);
      }
      // every product issued has finished before TMEM is released
      mma_commit(&drain);
      mbar_wait_cycles(&drain, 0, kWaitCycles);
    }
  } else if (warp >= 6) {
    const int strip = warp - 6, r = lane >> 2, q = lane & 3;
    const float* row_inv = reinterpret_cast<const float*>(a.packed + a.L.row_off);
    BigRing ring{sm + kBigRing + strip * kBigS * BigRing::kSlot, full_c[strip]};
    // a strip behind the last row of weights has no chunks: its rows are zeros
    int ft = first, fb = 0;  // the next chunk to ask for
    auto fetch = [&]() {
      while (ft < tiles) {
        const int tile = (ft / mt) * (kBM / kTile) + strip, block = kb0 + fb;
        if ((fb += kBigB) >= nk) fb = 0, ft += stride;
        if (tile >= a.L.tiles) continue;
        if (lane == 0) ring.fetch(a.packed, a.L, a.lg_group, tile, block);
        return;
      }
    };
    for (int i = 0; i < kBigS; ++i) fetch();
    int s = 0, used = 0;
    uint32_t round = 0;
    for (int t = first; t < tiles && !bad; t += stride) {
      const int tile = (t / mt) * (kBM / kTile) + strip;
      const bool on = tile < a.L.tiles;
      float inv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) inv[h] = on ? __ldg(row_inv + tile * kTile + r + 8 * h) : 0.0f;
      for (int k0 = 0; k0 < nk && !bad; k0 += kBigB) {
        const unsigned char* slot = ring.smem + (used % kBigS) * BigRing::kSlot;
        if (on) {
          const bool ok = mbar_wait_cycles(ring.full + used % kBigS, (used / kBigS) & 1, kWaitCycles);
          if (__any_sync(0xffffffffu, !ok)) {
            bad = true;
            break;
          }
        }
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(slot + kBigB * 512) - (((kb0 + k0) * kBlock) >> a.lg_group) * 16;
#pragma unroll
        for (int e = 0; e < kBigB; ++e) {
          if (k0 + e >= nk) break;
          uint4 c = make_uint4(0, 0, 0, 0);
          __half2 sh[2], bh[2];
          if (on) {
            c = *reinterpret_cast<const uint4*>(slot + e * 512 + lane * 16);
            const int g = min(((kb0 + k0 + e) * kBlock + q * 16) >> a.lg_group, a.L.groups - 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = sc[g * 16 + r + 8 * h];
              sh[h] = __float2half2_rn(lo_bf16(w) * inv[h]);
              bh[h] = __float2half2_rn(hi_bf16(w) * inv[h]);
            }
          } else {
            sh[0] = sh[1] = bh[0] = bh[1] = __float2half2_rn(0.0f);
          }
          if (round > 0) {
            const bool ok = mbar_wait_cycles(&empty[s], (round & 1) ^ 1, kWaitCycles);
            if (__any_sync(0xffffffffu, !ok)) {
              bad = true;
              break;
            }
          }
          unsigned char* row = sm + s * stage_bytes + strip * 2048 + r * 128;
          *reinterpret_cast<uint4*>(row + (((2 * q) ^ r) << 4)) = expand(c.x, sh[0], bh[0]);
          *reinterpret_cast<uint4*>(row + (((2 * q + 1) ^ r) << 4)) = expand(c.y, sh[0], bh[0]);
          *reinterpret_cast<uint4*>(row + 1024 + (((2 * q) ^ r) << 4)) = expand(c.z, sh[1], bh[1]);
          *reinterpret_cast<uint4*>(row + 1024 + (((2 * q + 1) ^ r) << 4)) = expand(c.w, sh[1], bh[1]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full_w[s]);
          if (++s == stages) s = 0, ++round;
        }
        if (on && !bad) {
          ++used;
          __syncwarp();  // the slot is read before lane 0 refills it
          fetch();
        }
      }
    }
    if (bad && lane == 0)  // the copies still in flight land before the block exits
      for (int j = used; j < ring.head; ++j) mbar_wait_cycles(ring.full + j % kBigS, (j / kBigS) & 1, kWaitCycles / 100);
  } else if (a.S == 1) {  // warp w reads TMEM lanes 32 (w % 4) .. + 31: weight rows 32 q + lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q = warp & 3;
    const float* row_inv = reinterpret_cast<const float*>(a.packed + a.L.row_off);
    int j = 0;
    for (int t = first; t < tiles; t += stride, ++j) {
      const int ab = j & 1, m0 = (t % mt) * a.tn, n = (t / mt) * kBM + 32 * q + lane;
      const float wf = n < a.N ? 1.0f / __ldg(row_inv + n) : 0.0f;
      const bool ok = mbar_wait_cycles(&acc_full[ab], (j >> 1) & 1, kWaitCycles);
      if (__any_sync(0xffffffffu, !ok)) {  // the whole warp leaves together (the TMEM loads are warp-wide)
        bad = true;
        break;
      }
      fence_after();
      const uint32_t src = tbase + 256 * ab + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
      for (int c = 0; c < a.tn; c += 16) {
        float v[16];
        tmem_ld16(src + c, v);
        if (n < a.N)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (m0 + c + e < a.M) a.y[(int64_t)(m0 + c + e) * a.N + n] = __float2bfloat16_rn(v[e] * wf * a.xf[m0 + c + e]);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
    }
  }
  if (a.S > 1) {  // one tile a cluster: the others' sums, [tn][128] floats each, go to the leader's ring
    const int q = warp & 3, row = 32 * q + lane;
    const bool epi = warp >= 2 && warp < 6;
    if (epi) {
      const bool ok = mbar_wait_cycles(&acc_full[0], 0, kWaitCycles);
      if (__any_sync(0xffffffffu, !ok)) bad = true;
      fence_after();
    }
    fence_before();
    __syncwarp();
    cluster_sync();  // every product of the cluster is done: the leader's ring is free
    fence_after();
    const uint32_t src = tbase + ((uint32_t)(32 * q) << 16);
    if (epi && rank > 0 && !bad) {
      const uint32_t slot = mapa_shared(smem_u32(sm), 0) + (uint32_t)(((rank - 1) * a.tn) * kBM + row) * 4;
#pragma unroll 1
      for (int c = 0; c < a.tn; c += 16) {
        float v[16];
        tmem_ld16(src + c, v);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(slot + (uint32_t)(c + e) * kBM * 4), "f"(v[e]) : "memory");
      }
    }
    fence_before();
    __syncwarp();
    cluster_sync();
    fence_after();
    if (epi && rank == 0 && !bad) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const int m0 = (first % mt) * a.tn, n = (first / mt) * kBM + row;
      const float wf = n < a.N ? 1.0f / __ldg(reinterpret_cast<const float*>(a.packed + a.L.row_off) + n) : 0.0f;
#pragma unroll 1
      for (int c = 0; c < a.tn; c += 16) {
        float v[16];
        tmem_ld16(src + c, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          for (int o = 0; o < a.S - 1; ++o) v[e] += reinterpret_cast<const float*>(sm)[(o * a.tn + c + e) * kBM + row];
          if (n < a.N && m0 + c + e < a.M)
            a.y[(int64_t)(m0 + c + e) * a.N + n] = __float2bfloat16_rn(v[e] * wf * a.xf[m0 + c + e]);
        }
      }
    }
  }
  if (sync_tc_any(bad) && tid == 0) set_status(a.status, kStatusWaitTimeout | (GDN_K_LINEAR_Q4 << 8));
  if (warp == 0) tmem_dealloc(tbase, 512);
}

}  // namespace

Q4Layout q4_layout(int32_t N, int32_t K, int32_t group) {
  Q4Layout L;
  L.tiles = (N + kTile - 1) / kTile;
  L.blocks = (K + kBlock - 1) / kBlock;
  L.groups = (K + group - 1) / group;
  L.scale_off = (size_t)L.tiles * L.blocks * 512;
  L.row_off = L.scale_off + (size_t)L.tiles * L.groups * 64;
  L.total_bytes = L.row_off + (size_t)L.tiles * kTile * 4;
  return L;
}

cudaError_t launch_q4_pack(const void* codes, const void* scales, const void* biases, int32_t N, int32_t K,
                           int32_t group, void* packed, cudaStream_t stream) {
  const Q4Layout L = q4_layout(N, K, group);
  const int64_t blocks = ((int64_t)L.row_off / 4 + 255) / 256;
  LaunchScope scope(GDN_K_Q4_PACK, stream);
  q4_pack_kernel<<<(unsigned)(blocks < 148 * 64 ? blocks : 148 * 64), 256, 0, stream>>>(
      (const unsigned char*)codes, (const unsigned short*)scales, (const unsigned short*)biases, N, K, group,
      (int64_t)L.groups * group / 2, L, (uint32_t*)packed);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  q4_rows_kernel<<<(unsigned)(L.tiles * kTile / 8), 256, 0, stream>>>((const unsigned short*)scales, (const unsigned short*)biases, N,
                                                            L, (float*)((unsigned char*)packed + L.row_off));
  return cudaGetLastError();
}

namespace {

constexpr int kSmallRows = 16;  // bf16 io: more rows run linear_big_kernel

template <typename T, int MT, int G>
cudaError_t run_small(const T* x, int32_t M, int32_t K, const unsigned char* packed, const Q4Layout& L, int32_t N, T* y,
                      int32_t* status, cudaStream_t stream) {
  using R = Ring<kSmallB, kSmallS>;
  constexpr int smem = kSmallWarps * kSmallS * R::kSlot;
  const int mg = (M + MT * 8 - 1) / (MT * 8), chunks = (L.blocks + kSmallB - 1) / kSmallB;
  int S = 1;  // K over more blocks while row tiles leave SMs without one and a warp keeps two chunks
  while (S < 8 && (int64_t)L.tiles * mg * S < 4 * kSms && chunks >= 4 * S * kSmallWarps) S *= 2;
  const int per_row = std::max(1, 2 * kSms / mg / S);  // two blocks an SM
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min(L.tiles, per_row) * S), (unsigned)mg);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = S > 1 ? 1 : 0;
  cudaError_t e = cudaFuncSetAttribute(linear_small_kernel<T, MT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  LaunchScope scope(GDN_K_LINEAR_Q4, stream);
  return cudaLaunchKernelEx(&cfg, linear_small_kernel<T, MT, G>, x, M, K, packed, L, N, y, S, status);
}
template <typename T, int MT>
cudaError_t run_small_g(const T* x, int32_t M, int32_t K, const unsigned char* packed, const Q4Layout& L, int32_t N,
                        int32_t group, T* y, int32_t* status, cudaStream_t stream) {
  if (group == 32) return run_small<T, MT, 32>(x, M, K, packed, L, N, y, status, stream);
  if (group == 64) return run_small<T, MT, 64>(x, M, K, packed, L, N, y, status, stream);
  return run_small<T, MT, 128>(x, M, K, packed, L, N, y, status, stream);
}

struct BigPlan {
  int tn, mp, S, grid;
};
// Rows of x a tile: one that leaves the fewest columns of products on the fullest SM.  A 64-channel step takes 2 cycles
// a column, and 160 for the expansion of its weights at least.
BigPlan big_plan(int32_t M, const Q4Layout& L) {
  const int64_t nt = (L.tiles * kTile + kBM - 1) / kBM;
  BigPlan b{};
  int64_t best = INT64_MAX;
  for (int tn = 16; tn <= 256; tn += 16) {
    const int64_t mt = (M + tn - 1) / tn, rounds = (nt * mt + kSms - 1) / kSms, cost = rounds * std::max(160, 2 * tn);
    if (cost < best || (cost == best && nt * mt < nt * (b.mp / b.tn))) best = cost, b.tn = tn, b.mp = (int)(mt * tn);
  }
  const int64_t tiles = nt * (b.mp / b.tn);
  b.S = 1;
  while (b.S < 8 && tiles * (b.S + 1) <= kSms && L.blocks >= 4 * (b.S + 1) && b.S * b.tn * kBM * 4 <= kBigRing) ++b.S;
  b.grid = b.S > 1 ? (int)tiles * b.S : (int)std::min<int64_t>(tiles, kSms);
  return b;
}

}  // namespace

size_t linear_q4_ws_bytes(int32_t M, int32_t N, int32_t K, int32_t group, bool bf16) {
  if (!bf16 || M <= kSmallRows || N == 0) return 0;
  const Q4Layout L = q4_layout(N, K, group);
  const BigPlan b = big_plan(M, L);
  return (size_t)b.mp * (L.blocks * 128 + 4);
}

cudaError_t launch_linear_q4(bool bf16, const void* x, int32_t M, int32_t K, const void* packed, int32_t N,
                             int32_t group, void* y, void* ws, int32_t* status, cudaStream_t stream) {
  const Q4Layout L = q4_layout(N, K, group);
  const unsigned char* w = (const unsigned char*)packed;
  if (!bf16 || M <= kSmallRows) {
    for (int32_t m0 = 0; m0 < M; m0 += 65535 * 8) {  // grid.y
      const int32_t m = std::min(M - m0, 65535 * 8);
      cudaError_t e;
      if (!bf16) e = run_small_g<float, 1>((const float*)x + (int64_t)m0 * K, m, K, w, L, N, group, (float*)y + (int64_t)m0 * N, status, stream);
      else if (M <= 8) e = run_small_g<__nv_bfloat16, 1>((const __nv_bfloat16*)x, M, K, w, L, N, group, (__nv_bfloat16*)y, status, stream);
      else e = run_small_g<__nv_bfloat16, 2>((const __nv_bfloat16*)x, M, K, w, L, N, group, (__nv_bfloat16*)y, status, stream);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const BigPlan b = big_plan(M, L);
  unsigned char* xh = (unsigned char*)ws;
  float* xf = (float*)(xh + (size_t)b.mp * L.blocks * 128);
  {
    LaunchScope scope(GDN_K_X_HALF, stream);
    x_half_kernel<<<(unsigned)b.mp, 256, 0, stream>>>((const __nv_bfloat16*)x, M, K, L.blocks, b.mp, xh, xf);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(linear_big_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBigSmem)) != cudaSuccess) return e;
  const BigArgs a{w, L, xh, xf, (__nv_bfloat16*)y, M, N, b.mp, b.tn, group == 32 ? 5 : group == 64 ? 6 : 7, b.S, status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)b.grid);
  cfg.blockDim = dim3(kBigThreads);
  cfg.dynamicSmemBytes = kBigSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = b.S, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = b.S > 1 ? 2 : 1;
  LaunchScope scope(GDN_K_LINEAR_Q4, stream);
  return cudaLaunchKernelEx(&cfg, linear_big_kernel, a);
}

}  // namespace gdn
