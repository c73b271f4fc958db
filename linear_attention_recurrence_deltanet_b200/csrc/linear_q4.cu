// Y[M, N] = X[M, K] W[N, K]^T with W in 4 bits: w = scale * code + bias, scale
// and bias (bf16) shared by a group of 32, 64 or 128 input features ("Q4" and
// "MLX affine" weights: DS4Server issues #88, Scope, and #95, implementation
// comment).  Per group
//   y = sum_g scale_ng (x_g . code_ng) + bias_ng sum(x_g).
//
// Packed weights (gdn_q4_pack), zero-filled to whole tiles of 128 rows and blocks
// of 64 channels, so that both kernels stream them with a few large copies:
//   codes   [tiles][blocks][8 strips of 16 rows][32 lanes] 16 bytes: lane 4r + q
//           holds the words of channels 16q .. 16q+7 and 16q+8 .. 16q+15 of row r,
//           then of row r + 8 -- a warp's fragment of the strip in one 16-byte load
//           a lane.  A word holds channel 2i in its nibble i and channel 2i + 1 in
//           its nibble 4 + i, so that masking the word gives pairs of neighbours.
//   scales  [tiles][groups of whole blocks][128 rows] words, scale low, bias high
//   rows    [tiles][128] floats: the power of two that brings the row's largest
//           weight below 2^11
#include <algorithm>

#include "../../include/gdn.h"
#include "common.cuh"
#include "internal.h"
#include "tc.cuh"
#include "vec.cuh"

namespace gdn {
namespace {

constexpr int kTile = 128, kStrip = 16, kStrips = 8, kBlock = 64;
constexpr int kBlockBytes = kTile * kBlock / 2, kGroupBytes = kTile * 4;  // of a tile's codes, of its scale words

__global__ void q4_pack_kernel(const unsigned char* __restrict__ codes, const unsigned short* __restrict__ scales,
                               const unsigned short* __restrict__ biases, int N, int K, int group, int64_t row_bytes,
                               Q4Layout L, uint32_t* __restrict__ out) {
  const int64_t words = (int64_t)L.row_off / 4, scale_words = (int64_t)L.scale_off / 4;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x) {
    uint32_t w = 0;
    if (i < scale_words) {
      const int64_t blk = i / (kBlockBytes / 4);
      const int in = (int)(i % (kBlockBytes / 4)), lane = in / 4 & 31, part = in & 3;
      const int64_t n = blk / L.blocks * kTile + in / 128 * kStrip + lane / 4 + (part >> 1) * 8;
      const int64_t k0 = blk % L.blocks * kBlock + (lane & 3) * 16 + (part & 1) * 8;
      if (n < N)
        for (int b = 0; b < 4; ++b)
          if (k0 + 2 * b < K) {
            const uint32_t byte = codes[n * row_bytes + k0 / 2 + b];
            const uint32_t odd = k0 + 2 * b + 1 < K ? byte >> 4 : 0;
            w |= (byte & 15u) << (4 * b) | odd << (16 + 4 * b);
          }
    } else {
      const int64_t j = i - scale_words, n = j / kTile / L.row_groups * kTile + j % kTile, g = j / kTile % L.row_groups;
      if (n < N && g < L.groups)
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

// The weight stream: one lane copies `nb` blocks of a tile and their groups' scale words into a slot, kScaleAt bytes
// apart, both completing on `full`.
struct Stream {
  const unsigned char *codes, *scales;  // of the tile
  int lg;
  __device__ __forceinline__ Stream(const unsigned char* packed, const Q4Layout& L, int tile, int lg_group)
      : codes(packed + (int64_t)tile * L.blocks * kBlockBytes),
        scales(packed + L.scale_off + (int64_t)tile * L.row_groups * kGroupBytes), lg(lg_group) {}
  __device__ __forceinline__ void fetch(unsigned char* slot, int scale_at, int block, int nb, uint64_t* full) const {
    const int g0 = (block * kBlock) >> lg, ng = (((block + nb) * kBlock - 1) >> lg) + 1 - g0;
    tc::mbar_expect_tx(full, nb * kBlockBytes + ng * kGroupBytes);
    tc::bulk_load(slot, codes + (int64_t)block * kBlockBytes, nb * kBlockBytes, full);
    tc::bulk_load(slot + scale_at, scales + (int64_t)g0 * kGroupBytes, ng * kGroupBytes, full);
  }
};
constexpr int kSms = 148;

// One output by its definition, in fp64: sum_k x_k (s code_k + b).  The kernels for few rows take scale and bias out of the
// sums, which turns an infinity in x, or values whose multiple by 128 passes fp32, into inf - inf.  Results that are not
// finite come here once all are written, and mostly leave as they came (at most 1 % of a call without any, 2 % for 16 rows).
template <typename T>
__device__ __forceinline__ float by_definition(const T* x, int K, const unsigned char* packed, const Q4Layout& L, int lg, int n) {
  const int tile = n / kTile, row = n % kTile;
  const unsigned char* codes = packed + (int64_t)tile * L.blocks * kBlockBytes + row / kStrip * 512 + row % 8 * 64 + row / 8 % 2 * 8;
  const uint32_t* scales = reinterpret_cast<const uint32_t*>(packed + L.scale_off + (int64_t)tile * L.row_groups * kGroupBytes) + row;
  double v = 0.0;
#pragma unroll 1
  for (int k = 0; k < K && v == v; k += 8) {  // a word: channels 16 q + 8 part of the block, pairs in nibbles i and 4 + i
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (int64_t)(k / kBlock) * kBlockBytes + k / 16 % 4 * 16 + k / 8 % 2 * 4);
    const uint32_t sw = scales[(int64_t)(k >> lg) * kTile];
    const double s = lo_bf16(sw), b = hi_bf16(sw);
#pragma unroll 1
    for (int i = 0; i < 8; ++i) v += (double)to_f(x[k + i]) * (s * (double)((w >> (4 * (i / 2) + 16 * (i % 2))) & 15u) + b);
  }
  return (float)v;
}

// ------------------------------------------------------------------ few rows
// Eight rows of x a block: the codes go to the tensor cores as bf16
// integers (A: 16 weight rows, B: 8 rows of x), each group's products are scaled
// in fp32, so nothing but the sums is rounded.  bf16 io takes 128 + code (one
// mask a pair), fp32 io code - 8 and three bf16 parts of x.
//
// A block takes 128 weight rows; its eight warps, and those of the S blocks of its
// cluster, deal the 64-channel blocks of K out.  A warp streams its blocks (4 KB
// of codes and their scales) through a ring of its own and multiplies all 128
// rows with the x it holds in registers; the warps join in shared memory.  The
// weight stream bounds it.
constexpr int kSmallWarps = 8, kSmallThreads = kSmallWarps * 32;

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Channels 2i, 2i + 1 of a word as bf16: 128 + code, or code - 8 for fp32 io.  The mask and the exponent sit in registers
// whose values the compiler does not know (a kernel argument that is 0 is in them), so that one instruction takes both.
template <bool F32>
struct CodePair {
  uint32_t mask, magic;
  __device__ __forceinline__ explicit CodePair(uint32_t zero) : mask(0x000f000fu + zero), magic(0x43004300u + zero) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t w, int i) const {
    uint32_t c;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(c) : "r"(w >> (4 * i)), "r"(mask), "r"(magic));  // (w & mask) | magic
    if constexpr (!F32) return c;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(c), "r"(0x43084308u));
    return r;
  }
};

__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {  // C = 0
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

constexpr int kSmallSlots = 2, kSmallSlot = kBlockBytes + 2 * kGroupBytes;  // groups of 32: two a block
constexpr int kSmallSmem = kSmallWarps * kSmallSlots * kSmallSlot;           // 80 KB: two blocks an SM
constexpr int kRedLd = kTile + 4;                                            // floats between columns of the join

template <typename T, int G>
__global__ void __launch_bounds__(kSmallThreads, 2)
    linear_small_kernel(const T* __restrict__ x, int M, int K, const unsigned char* __restrict__ packed, Q4Layout L,
                        int N, T* __restrict__ y, int S, int32_t* status, uint32_t zero) {
  constexpr bool F32 = sizeof(T) == 4;
  const CodePair<F32> code_pair(zero);
  constexpr int P = F32 ? 3 : 1;                 // bf16 parts of x
  constexpr int SUB = G == 32 ? 2 : 1;           // groups of a block
  constexpr int LG = G == 32 ? 5 : G == 64 ? 6 : 7;
  static_assert(kSmallWarps * 8 * kRedLd * 4 <= kSmallSmem, "the join uses the rings");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t s_full[kSmallWarps][kSmallSlots];
  __shared__ float s_sum[8 * kTile];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3, m0 = (int)blockIdx.y * 8;
  const int rank = (int)blockIdx.x % S, tile = (int)blockIdx.x / S;
  const int step = S * kSmallWarps, first = rank * kSmallWarps + warp;  // this warp's blocks

  if (threadIdx.x < kSmallWarps * kSmallSlots) tc::mbar_init(&s_full[threadIdx.x / kSmallSlots][threadIdx.x % kSmallSlots], 1);
  tc::mbar_init_fence();
  __syncthreads();
  unsigned char* ring = smem + warp * kSmallSlots * kSmallSlot;
  const Stream stream(packed, L, tile, LG);
  if (lane == 0)
    for (int i = 0, b = first; i < kSmallSlots && b < L.blocks; ++i, b += step)
      stream.fetch(ring + i * kSmallSlot, kBlockBytes, b, 1, &s_full[warp][i]);

  float acc[kStrips][4];
#pragma unroll
  for (int i = 0; i < kStrips; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
  const bool here = m0 + r < M;
  const int kmax = here ? K - q * 16 : 0;  // channels of this lane from block 0 on
  const T* xp = x + (int64_t)(here ? m0 + r : 0) * K + q * 16;

  int slot_i = 0;
  uint32_t phase = 0;
  for (int b = first; b < L.blocks; b += step) {
    // x as B fragments, and its sums over the groups as the product with ones
    uint32_t f[P][8];
    float xs[SUB][4];
    const T* src = xp + (int64_t)b * kBlock;
    const int left = kmax - b * kBlock;
#pragma unroll
    for (int h = 0; h < (F32 ? 4 : 2); ++h) {
      const uint4 v = (F32 ? 4 : 8) * h < left ? ld16(src + (F32 ? 4 : 8) * h) : make_uint4(0, 0, 0, 0);
      if constexpr (!F32) {
        f[0][4 * h] = v.x, f[0][4 * h + 1] = v.y, f[0][4 * h + 2] = v.z, f[0][4 * h + 3] = v.w;
      } else {
        float e[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
#pragma unroll
        for (int pt = 0; pt < P; ++pt)
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const uint32_t z = bf16x2(e[2 * d], e[2 * d + 1]);
            f[pt][2 * h + d] = z;
            e[2 * d] -= lo_bf16(z), e[2 * d + 1] -= hi_bf16(z);
          }
      }
    }
#pragma unroll
    for (int g = 0; g < SUB; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) xs[g][e] = 0.0f;
#pragma unroll
    for (int pt = 0; pt < P; ++pt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int g = 0; g < SUB; ++g) {  // groups of 32: lanes q < 2 hold the first, q >= 2 the second
          const bool on = SUB == 1 || (q >> 1) == g;
          mma(xs[g], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, on ? f[pt][2 * j] : 0u,
              on ? f[pt][2 * j + 1] : 0u);
        }
    if (!tc::mbar_wait_warp(&s_full[warp][slot_i], phase)) {
      set_status(status, kStatusWaitTimeout | (GDN_K_LINEAR_Q4 << 8));
      break;
    }
    const unsigned char* slot = ring + slot_i * kSmallSlot;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(slot + kBlockBytes) + r;
#pragma unroll
    for (int i = 0; i < kStrips; ++i) {
      const uint4 cw = *reinterpret_cast<const uint4*>(slot + i * 512 + lane * 16);
      const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
      uint32_t a[8][2];  // pairs of the lane's 16 channels, rows r and r + 8
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j][0] = code_pair(w[j >> 2], j & 3);
        a[j][1] = code_pair(w[2 + (j >> 2)], j & 3);
      }
#pragma unroll
      for (int g = 0; g < SUB; ++g) {
        float p[4];
#pragma unroll
        for (int pt = 0; pt < P; ++pt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool on = SUB == 1 || (q >> 1) == g;
            const uint32_t f0 = on ? f[pt][2 * j] : 0u, f1 = on ? f[pt][2 * j + 1] : 0u;
            if (pt == 0 && j == 0) mma0(p, a[0][0], a[0][1], a[1][0], a[1][1], f0, f1);
            else mma(p, a[2 * j][0], a[2 * j][1], a[2 * j + 1][0], a[2 * j + 1][1], f0, f1);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t sw = sc[g * kTile + i * kStrip + 8 * h];
          const float s = lo_bf16(sw), z = fmaf(F32 ? 8.0f : -128.0f, s, hi_bf16(sw));
#pragma unroll
          for (int e = 0; e < 2; ++e) acc[i][2 * h + e] = fmaf(s, p[2 * h + e], fmaf(z, xs[g][e], acc[i][2 * h + e]));
        }
      }
    }
    __syncwarp();  // the slot is read before lane 0 refills it
    const int nb = b + kSmallSlots * step;
    if (lane == 0 && nb < L.blocks) stream.fetch(ring + slot_i * kSmallSlot, kBlockBytes, nb, 1, &s_full[warp][slot_i]);
    if (++slot_i == kSmallSlots) slot_i = 0, phase ^= 1;
  }
  // (after a wait that ran out) every copy has landed before the rings take the sums
  for (int i = 0; i < kSmallSlots; ++i) {
    const int mine = first < L.blocks ? (L.blocks - first + step - 1) / step : 0, uses = (mine - i + kSmallSlots - 1) / kSmallSlots;
    if (uses > 0) tc::mbar_wait_warp(&s_full[warp][i], (uses & 1) ^ 1, tc::kWaitTries / 64);
  }
  __syncthreads();

  float* red = reinterpret_cast<float*>(smem);  // [warp][column of x][row]
#pragma unroll
  for (int i = 0; i < kStrips; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[(warp * 8 + 2 * q + (e & 1)) * kRedLd + i * kStrip + r + 8 * (e >> 1)] = acc[i][e];
  __syncthreads();
  bool odd = false;
  auto put = [&](int i, float v) {
    const int n = tile * kTile + i % kTile, m = m0 + i / kTile;
    if (n >= N || m >= M) return;
    odd |= !isfinite(v);
    y[(int64_t)m * N + n] = from_f<T>(v);
  };
  for (int i = threadIdx.x; i < 8 * kTile; i += kSmallThreads) {
    if (m0 + i / kTile >= M) break;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) v += red[(w * 8 + i / kTile) * kRedLd + i % kTile];
    if (S == 1) put(i, v);
    else s_sum[i] = v;
  }
  auto mend = [&](int first, int step) {
    if (!odd) return;
    for (int i = first; i < 8 * kTile; i += step) {
      const int n = tile * kTile + i % kTile, m = m0 + i / kTile;
      if (n < N && m < M && !isfinite(to_f(y[(int64_t)m * N + n])))
        y[(int64_t)m * N + n] = from_f<T>(by_definition(x + (int64_t)m * K, K, packed, L, LG, n));
    }
  };
  if (S == 1) return mend(threadIdx.x, kSmallThreads);
  tc::cluster_sync();
  if (rank == 0)
    for (int i = threadIdx.x; i < 8 * kTile; i += kSmallThreads) {
      if (m0 + i / kTile >= M) break;
      float v = s_sum[i];
      for (int o = 1; o < S; ++o) {
        float f;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(tc::mapa_shared(tc::smem_u32(&s_sum[i]), o)));
        v += f;
      }
      put(i, v);
    }
  tc::cluster_sync();  // the leader has read the others' sums
  mend(threadIdx.x, kSmallThreads);
}

// 9 to 32 rows of bf16 io (8 MT).  A warp takes SPW of the tile's eight strips, so that its sums stay in registers, and
// every KW-th 64-channel block; the block copies x of KW blocks at a time, in the order of B fragments, some steps ahead
// (5120 x 6144, 16 rows: 16.8 us, 18 with weights from memory; with x read by each warp 26).
constexpr int strips_per_warp(int MT) { return MT == 2 ? 8 : 4; }
constexpr int rows_slots(int MT) { return MT == 2 ? 2 : 4; }
constexpr int rows_kw(int MT) { return strips_per_warp(MT); }  // eight warps / (8 / SPW)
constexpr int rows_stages(int MT) { return MT == 2 ? 2 : 3; }
constexpr int rows_slot_bytes(int MT, int G) { return strips_per_warp(MT) * (512 + 64 * (G == 32 ? 2 : 1)); }
constexpr int rows_smem(int MT, int G) {
  const int rings = kSmallWarps * rows_slots(MT) * rows_slot_bytes(MT, G) + rows_stages(MT) * rows_kw(MT) * MT * 1024;
  const int join = (rows_kw(MT) * MT * 8 * kRedLd + MT * 8 * kTile) * 4;
  return rings > join ? rings : join;
}
constexpr int rows_blocks(int MT, int G) { return 2 * (rows_smem(MT, G) + 2048) <= 232448 && MT == 2 ? 2 : 1; }  // an SM

template <int MT, int G>
__global__ void __launch_bounds__(kSmallThreads, rows_blocks(MT, G))
    linear_rows_kernel(const __nv_bfloat16* __restrict__ x, int M, int K, const unsigned char* __restrict__ packed, Q4Layout L,
                       int N, __nv_bfloat16* __restrict__ y, int S, int32_t* status, uint32_t zero) {
  constexpr int SPW = strips_per_warp(MT), SG = kStrips / SPW, KW = kSmallWarps / SG, SLOTS = rows_slots(MT);
  constexpr int SUB = G == 32 ? 2 : 1, LG = G == 32 ? 5 : G == 64 ? 6 : 7;
  constexpr int STAGES = rows_stages(MT), SLOT = rows_slot_bytes(MT, G), STAGE = KW * MT * 1024;
  static_assert(KW == rows_kw(MT), "warps");
  const CodePair<false> code_pair(zero);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t s_full[kSmallWarps][SLOTS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  const int sg = warp % SG, kw = warp / SG;
  const int rank = (int)blockIdx.x % S, tile = (int)blockIdx.x / S;
  const int steps = (L.blocks + S * KW - 1) / (S * KW);  // step i: blocks (i S + rank) KW ..
  if (threadIdx.x < kSmallWarps * SLOTS) tc::mbar_init(&s_full[threadIdx.x / SLOTS][threadIdx.x % SLOTS], 1);
  tc::mbar_init_fence();
  __syncthreads();

  unsigned char* ring = smem + warp * SLOTS * SLOT;
  unsigned char* xs_base = smem + kSmallWarps * SLOTS * SLOT;
  const unsigned char* codes = packed + (int64_t)tile * L.blocks * kBlockBytes + sg * SPW * 512;
  const unsigned char* scales = packed + L.scale_off + (int64_t)tile * L.row_groups * kGroupBytes + sg * SPW * 64;
  auto fetch = [&](int step, int slot) {  // one lane: this warp's strips of its block
    const int b = (step * S + rank) * KW + kw;
    if (b >= L.blocks) return;
    uint64_t* m = &s_full[warp][slot];
    unsigned char* d = ring + slot * SLOT;
    tc::mbar_expect_tx(m, SPW * 512 + SUB * SPW * 64);
    tc::bulk_load(d, codes + (int64_t)b * kBlockBytes, SPW * 512, m);
#pragma unroll
    for (int g = 0; g < SUB; ++g)
      tc::bulk_load(d + SPW * 512 + g * SPW * 64, scales + (int64_t)(((b * kBlock) >> LG) + g) * kGroupBytes, SPW * 64, m);
  };
  // x of a step's blocks: chunk c (eight channels) of row m of block k goes to lane (m % 8, c / 2), half c % 2
  auto copy_x = [&](int step) {
    if (step < steps)
      for (int i = threadIdx.x; i < KW * MT * 64; i += kSmallThreads) {
        const int c = i & 7, m = (i >> 3) % (MT * 8), k = (i >> 3) / (MT * 8);
        const int ch = ((step * S + rank) * KW + k) * kBlock + c * 8;
        const bool on = m < M && ch < K;
        tc::cp_async16(xs_base + (step % STAGES) * STAGE + k * MT * 1024 +
                           ((((m >> 3) * 2 + (c & 1)) * 32) + (m & 7) * 4 + (c >> 1)) * 16,
                       on ? x + (int64_t)m * K + ch : x, on ? 16 : 0);
      }
    tc::cp_async_commit();
  };
  if (lane == 0)
    for (int i = 0; i < SLOTS && i < steps; ++i) fetch(i, i);
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) copy_x(i);

  float acc[SPW][MT][4];
#pragma unroll
  for (int i = 0; i < SPW; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.0f;

  int slot_i = 0;
  uint32_t phase = 0;
  bool dead = false;
  for (int step = 0; step < steps; ++step) {
    tc::cp_async_wait<STAGES - 2>();
    __syncthreads();  // everybody's copies of this step have landed, and the stage of the last one is read
    copy_x(step + STAGES - 1);
    const bool here = (step * S + rank) * KW + kw < L.blocks && !dead;
    if (here && !tc::mbar_wait_warp(&s_full[warp][slot_i], phase)) {
      set_status(status, kStatusWaitTimeout | (GDN_K_LINEAR_Q4 << 8));
      dead = true;
    }
    if (here && !dead) {
      const uint4* xs = reinterpret_cast<const uint4*>(xs_base + (step % STAGES) * STAGE + kw * MT * 1024) + lane;
      uint32_t f[MT][8];
      float sum[SUB][MT][4];  // x over the groups, as the product with ones
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint4 v0 = xs[(2 * t) * 32], v1 = xs[(2 * t + 1) * 32];
        f[t][0] = v0.x, f[t][1] = v0.y, f[t][2] = v0.z, f[t][3] = v0.w;
        f[t][4] = v1.x, f[t][5] = v1.y, f[t][6] = v1.z, f[t][7] = v1.w;
#pragma unroll
        for (int g = 0; g < SUB; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // groups of 32: lanes q < 2 hold the first, q >= 2 the second
            const bool on = SUB == 1 || (q >> 1) == g;
            const uint32_t f0 = on ? f[t][2 * j] : 0u, f1 = on ? f[t][2 * j + 1] : 0u;
            if (j == 0) mma0(sum[g][t], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, f0, f1);
            else mma(sum[g][t], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, f0, f1);
          }
      }
      const unsigned char* slot = ring + slot_i * SLOT;
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(slot + SPW * 512) + r;
#pragma unroll
      for (int i = 0; i < SPW; ++i) {
        const uint4 cw = *reinterpret_cast<const uint4*>(slot + i * 512 + lane * 16);
        const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
        uint32_t a[8][2];  // pairs of the lane's 16 channels, rows r and r + 8
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j][0] = code_pair(w[j >> 2], j & 3), a[j][1] = code_pair(w[2 + (j >> 2)], j & 3);
#pragma unroll
        for (int g = 0; g < SUB; ++g) {
          float s[2], z[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sw = sc[g * SPW * 16 + i * kStrip + 8 * h];
            s[h] = lo_bf16(sw), z[h] = fmaf(-128.0f, s[h], hi_bf16(sw));
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool on = SUB == 1 || (q >> 1) == g;
              const uint32_t f0 = on ? f[t][2 * j] : 0u, f1 = on ? f[t][2 * j + 1] : 0u;
              if (j == 0) mma0(p, a[0][0], a[0][1], a[1][0], a[1][1], f0, f1);
              else mma(p, a[2 * j][0], a[2 * j][1], a[2 * j + 1][0], a[2 * j + 1][1], f0, f1);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                acc[i][t][2 * h + e] = fmaf(s[h], p[2 * h + e], fmaf(z[h], sum[g][t][e], acc[i][t][2 * h + e]));
          }
        }
      }
      __syncwarp();  // the slot is read before lane 0 refills it
    }
    if (lane == 0 && !dead && step + SLOTS < steps) fetch(step + SLOTS, slot_i);
    if (++slot_i == SLOTS) slot_i = 0, phase ^= 1;
  }
  tc::cp_async_wait<0>();
  if (dead)  // the copies still in flight land before the block goes on
    for (int i = 0; i < SLOTS; ++i)
      for (uint32_t ph = 0; ph < 2; ++ph) tc::mbar_wait_warp(&s_full[warp][i], ph, tc::kWaitTries / 64);
  __syncthreads();

  float* red = reinterpret_cast<float*>(smem);  // [K part][column of x][row]
  float* s_sum = red + KW * MT * 8 * kRedLd;
#pragma unroll
  for (int i = 0; i < SPW; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[(kw * MT * 8 + t * 8 + 2 * q + (e & 1)) * kRedLd + (sg * SPW + i) * kStrip + r + 8 * (e >> 1)] = acc[i][t][e];
  __syncthreads();
  bool odd = false;
  auto put = [&](int i, float v) {
    const int n = tile * kTile + i % kTile;
    if (n >= N) return;
    odd |= !isfinite(v);
    y[(int64_t)(i / kTile) * N + n] = __float2bfloat16_rn(v);
  };
  for (int i = threadIdx.x; i < M * kTile; i += kSmallThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) v += red[(w * MT * 8 + i / kTile) * kRedLd + i % kTile];
    if (S == 1) put(i, v);
    else s_sum[i] = v;
  }
  auto mend = [&](int first, int step) {
    if (!odd) return;
    for (int i = first; i < M * kTile; i += step) {
      const int n = tile * kTile + i % kTile;
      __nv_bfloat16* d = y + (int64_t)(i / kTile) * N + n;
      if (n < N && !isfinite(to_f(*d))) *d = __float2bfloat16_rn(by_definition(x + (int64_t)(i / kTile) * K, K, packed, L, LG, n));
    }
  };
  if (S == 1) return mend(threadIdx.x, kSmallThreads);
  tc::cluster_sync();
  // each block of the cluster adds up its share of the rows
  for (int i = rank * kSmallThreads + threadIdx.x; i < M * kTile; i += S * kSmallThreads) {
    float v = 0.0f;
    for (int o = 0; o < S; ++o) {
      float f;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(tc::mapa_shared(tc::smem_u32(&s_sum[i]), o)));
      v += f;
    }
    put(i, v);
  }
  tc::cluster_sync();  // the others have read this block's sums
  mend(rank * kSmallThreads + threadIdx.x, S * kSmallThreads);
}

// ------------------------------------------------------------------ many rows
// More rows (bf16 io): tcgen05 products of 128 weight rows (A) and
// `tn` rows of x (B), in fp16.  Weights are expanded to fp16 into TMEM by eight
// warps, one of the tile's 16-row strips each; scaled by a power of two a row
// (q4_pack) so that the row's largest value is below 2^11, a weight is off by half a
// step, 2^-11, against 2^-8 in bf16.  x goes through x_half_kernel: fp16 with a power
// of two a row, exact but for elements 2^-25 of the row's largest and smaller, laid
// out as the tiles that the products read, with the channels of a block in the order
// in which a warp's TMEM store leaves the weights.
//
// Shared memory is what the products and the copies of x share: weights that went
// through it as well took 96 KB a step of 256 rows, more than it moves in the
// products' 512 cycles.  In TMEM they leave 256 columns: two accumulators of 128, so
// that one tile's output overlaps the next one's products, or one of 256.
//
// Warp 0 loads x, warp 1 issues the products, warps 2-5 write the accumulator
// out, warp 6 loads codes and scales, warps 8-31 expand: three groups of
// eight, a warp each 16-row strip, take the blocks in turn, since a block's way
// through a warp takes longer than its products.
// Rounds of whole tiles, then the remaining tiles in S slices of K each: their
// sums go to the workspace, and the block that comes last adds them in the order
// of the slices.
//
// Measured (x_half included): 2048 rows of 5120 -> 8192 148 us, 1160 TFLOP/s (weights in
// shared memory 167, an output loop of nine instructions a value 175, rounds chosen
// without the output's cost 164); 64 rows of 6144 -> 5120 24 us (25), 26 with weights
// from memory.  What is left
// beside the products, which keep the tensor pipe active for 66 %: the output of the
// single accumulator, start, x_half and the slices' join; for few rows the handshake
// of a step and 9 us of start, x_half and join.  A pair of
// blocks a tile, which halves the copies of x, took 250 us: its handshake is longer
// than a step.
constexpr int kGroups = 3, kExpandWarps = kGroups * kStrips, kBigThreads = (8 + kExpandWarps) * 32;
constexpr int kBigB = kGroups, kMaxSlots = 4;  // blocks of a chunk, chunks ahead
constexpr int kChunk = kBigB * kBlockBytes + 2 * kBigB * kGroupBytes;
constexpr int kMaxRing = 8, kWAt = 256, kWCols = kBlock / 2;  // columns of TMEM where the weights begin, and of a stage of them
// accumulators (of 128 columns, or one of 256) in front of the weights
__host__ __device__ constexpr int big_accs(int tn) { return tn <= 128 ? 2 : 1; }
constexpr int kBigRing = 229376, kBigSmem = kBigRing + 1024;  // chunks and stages: 224 KB
static_assert(kBigSmem + 2048 <= 232448, "shared memory of a block");
static_assert(kWAt + kMaxRing * kWCols == 512, "TMEM: accumulators, then the weights' stages");
// chunks: many where tiles of x leave room (and weights come from memory), few beside six stages of 256 rows
__host__ __device__ constexpr int big_slots(int tn) { return tn <= 128 ? kMaxSlots : 2; }

struct BigArgs {
  const unsigned char* packed;
  Q4Layout L;
  const unsigned char* xh;  // [blocks][mp][128 bytes]
  const float* xf;          // [mp]: power of two of each row
  float* part;              // [blocks of the last round][tn][128] sums of a slice
  int32_t* count;           // [tiles of the last round] slices written, 0 at the start
  __nv_bfloat16* y;
  int32_t M, N, mp, tn, lg_group, full, S;  // rounds of whole tiles; slices of a tile of the last round
  int32_t* status;
  uint32_t zero;  // 0, unknown to the compiler
};

// one block a row of x: fp16 scaled to below 2^11, into the layout of the products' operand
__global__ void __launch_bounds__(256) x_half_kernel(const __nv_bfloat16* __restrict__ x, int M, int K, int blocks, int mp,
                                                     unsigned char* __restrict__ xh, float* __restrict__ xf,
                                                     int32_t* __restrict__ count, int counts) {
  __shared__ uint32_t s_top[8];
  const int m = blockIdx.x;
  if (m == 0)
    for (int i = threadIdx.x; i < counts; i += 256) count[i] = 0;
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
    // channels 16 q + 4 i .. + 3 of 64 go to 16 i + 4 q, where the weights have them
    const uint4 h = tc::pack8h(v);
    unsigned char* d = xh + ((int64_t)(c >> 3) * mp + m) * 128 + 8 * ((c >> 1) & 1);
    const int at = 4 * (c & 1) + ((c >> 2) & 1);
    *reinterpret_cast<uint2*>(d + ((at ^ (m & 7)) << 4)) = make_uint2(h.x, h.y);
    *reinterpret_cast<uint2*>(d + (((at + 2) ^ (m & 7)) << 4)) = make_uint2(h.z, h.w);
  }
}

// Codes of a word -> eight fp16 weights s code + b (one rounding).  Nibbles 0, 2 (and 4, 6) are masked into 1024 + c,
// nibbles 1, 3 into 1024 + 16 c, which saves their shift; masks and exponent as in CodePair.
struct Expand {
  uint32_t lo, hi, magic;
  __device__ __forceinline__ explicit Expand(uint32_t zero)
      : lo(0x000f000fu + zero), hi(0x00f000f0u + zero), magic(0x64006400u + zero) {}
  __device__ __forceinline__ uint4 operator()(uint32_t w, __half2 s, __half2 b) const {
    uint32_t o[4];
    const __half2 k1024 = __half2half2(__ushort_as_half(0x6400)), k16 = __half2half2(__ushort_as_half(0x2c00)),
                  k64 = __half2half2(__ushort_as_half(0xd400));  // 1024, 1/16, -64
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t x, y;
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "r"(lo), "r"(magic));
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "r"(hi), "r"(magic));
      const __half2 cl = __hsub2(*reinterpret_cast<const __half2*>(&x), k1024);
      const __half2 ch = __hfma2(*reinterpret_cast<const __half2*>(&y), k16, k64);
      const __half2 wl = __hfma2(cl, s, b), wh = __hfma2(ch, s, b);
      o[2 * i] = *reinterpret_cast<const uint32_t*>(&wl);
      o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&wh);
      w >>= 8;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

// The TMEM accesses below are .sync.aligned and, unlike those of tc.cuh, do not reconverge the warp themselves, which would
// cost 3 % of the kernel: what only some lanes do ends with a __syncwarp() before them.
// products with the weights (A) in TMEM; b: the lower half of the descriptor of x
__device__ __forceinline__ void mma_ts_low(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 y;\nmov.b64 y, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(acc), "n"(tc::kDescHigh));
}
// 16 TMEM lanes x 32 columns: lane (r, q) of the warp has lanes r (a, b) and r + 8 (c, d), columns 8 i + 2 q and the next
// of each i < 4; waits until they are there
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, uint4 a, uint4 b, uint4 c, uint4 d) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(a.x), "r"(a.y), "r"(c.x), "r"(c.y), "r"(a.z), "r"(a.w), "r"(c.z), "r"(c.w), "r"(b.x), "r"(b.y), "r"(d.x), "r"(d.y),
      "r"(b.z), "r"(b.w), "r"(d.z), "r"(d.w)
      : "memory");
}

// 16 columns of this thread's TMEM lane, on their way until ld_wait, which names the registers that the load fills
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

__global__ void __launch_bounds__(kBigThreads, 1) linear_big_kernel(const __grid_constant__ BigArgs a) {
  using namespace tc;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // (an offset, so that the accesses stay shared ones)
  __shared__ uint64_t full_c[kMaxSlots], free_c[kMaxSlots];
  __shared__ uint64_t full[kMaxRing], empty[kMaxRing], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tslot;
  __shared__ __align__(16) float s_xf[256];
  __shared__ int s_last;  // this block's slice came last: it adds the tile up
  bool bad = false;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stage_bytes = a.tn * 128, accs = big_accs(a.tn);
  const int slots = big_slots(a.tn), stages = min(kMaxRing, (kBigRing - slots * kChunk) / stage_bytes);
  unsigned char* chunks = sm + stages * stage_bytes;
  const int mt = a.mp / a.tn, tiles = mt * a.L.tiles;
  // this block's pieces: whole tiles, then a slice of one
  struct Piece {
    int tile, k0, k1;
  };
  auto piece = [&](int i, Piece& p) {
    if (i < a.full) {
      p = Piece{i * (int)gridDim.x + (int)blockIdx.x, 0, a.L.blocks};
      return true;
    }
    const int t = a.full * (int)gridDim.x + (int)blockIdx.x / a.S, j = (int)blockIdx.x % a.S;
    if (i > a.full || t >= tiles) return false;
    auto slice = [&](int v) { return v == a.S ? a.L.blocks : (int)((int64_t)a.L.blocks * v / a.S) & ~1; };  // whole groups
    p = Piece{t, slice(j), slice(j + 1)};
    return true;
  };
  Piece p;

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 2);  // x, and the warps that expand its weights
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < slots; ++s) {
      mbar_init(&full_c[s], 1);
      mbar_init(&free_c[s], kGroups);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(&drain, 1);
    mbar_init_fence();
    s_last = 0;
  }
  if (warp == 0) tmem_alloc(&tslot, 512);
  sync_tc();
  const uint32_t tbase = tslot;

  if (warp == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // x_half_kernel's output
    int i = 0, s = 0;
    uint32_t phase = 1;
    for (int j = 0; piece(j, p) && !bad; ++j) {
      const unsigned char* src = a.xh + ((int64_t)p.k0 * a.mp + (p.tile % mt) * a.tn) * 128;
      for (int kb = p.k0; kb < p.k1; ++kb, ++i, src += (int64_t)a.mp * 128) {
        if (i >= stages && !mbar_wait_warp(&empty[s], phase)) {
          bad = true;
          break;
        }
        if (elect_one()) {
          mbar_expect_tx(&full[s], stage_bytes);
          bulk_load(sm + s * stage_bytes, src, stage_bytes, &full[s]);
        }
        __syncwarp();
        if (++s == stages) s = 0, phase ^= 1;
      }
    }
    if (bad)  // let the copies already issued land before the block exits
      for (int j = max(0, i - stages); j < i; ++j) mbar_wait_warp(&full[j % stages], (j / stages) & 1, tc::kWaitTries / 64);
  } else if (warp == 1) {
    const uint32_t id = idesc_f16(kTile, a.tn, false, false);
    const uint32_t dx = (uint32_t)desc_kmaj(smem_u32(sm), a.tn, 0);
    const int stage16 = stage_bytes >> 4;  // addresses count in 16 bytes
    int s = 0;
    uint32_t phase = 0;
    for (int j = 0; piece(j, p) && !bad; ++j) {
      const int ab = j % accs;
      if (j >= accs && !mbar_wait_warp(&acc_empty[ab], ((j / accs) & 1) ^ 1)) {
        bad = true;
        break;
      }
      fence_after();
      const uint32_t d = tbase + 128 * ab;
      for (int kb = p.k0; kb < p.k1; ++kb) {
        if (!mbar_wait_warp(&full[s], phase)) {
          bad = true;
          break;
        }
        fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kBlock / 16; ++kk)  // 32 bytes further in each row
            mma_ts_low(d, tbase + kWAt + kWCols * s + 8 * kk, dx + (uint32_t)(s * stage16 + 2 * kk), id, (kb > p.k0 || kk > 0) ? 1u : 0u);
          mma_commit(&empty[s]);
          if (kb + 1 == p.k1) mma_commit(&acc_full[ab]);
        }
        __syncwarp();
        if (++s == stages) s = 0, phase ^= 1;
      }
    }
    // every product issued has finished before TMEM is released
    if (elect_one()) mma_commit(&drain);
    __syncwarp();
    mbar_wait_warp(&drain, 0);
  } else if (warp == 6) {
    int i = 0, c = 0;
    uint32_t phase = 1;
    for (int j = 0; piece(j, p) && !bad; ++j) {
      const Stream stream(a.packed, a.L, p.tile / mt, a.lg_group);
      for (int k0 = p.k0; k0 < p.k1; k0 += kBigB, ++i) {
        if (i >= slots && !mbar_wait_warp(&free_c[c], phase)) {
          bad = true;
          break;
        }
        if (elect_one()) stream.fetch(chunks + c * kChunk, kBigB * kBlockBytes, k0, min(kBigB, p.k1 - k0), &full_c[c]);
        __syncwarp();
        if (++c == slots) c = 0, phase ^= 1;
      }
    }
    if (bad)  // let the copies already issued land before the block exits
      for (int j = max(0, i - slots); j < i; ++j) mbar_wait_warp(&full_c[j % slots], (j / slots) & 1, tc::kWaitTries / 64);
  } else if (warp >= 8) {
    const Expand expand(a.zero);
    // a warp writes the TMEM lanes of its number's remainder by four: two strips of 16 rows
    const int grp = (warp - 8) >> 3, strip = 2 * (warp & 3) + ((warp >> 2) & 1), r = lane >> 2, q = lane & 3;
    const bool polls = (warp & 7) == 0;
    const float* row_inv = reinterpret_cast<const float*>(a.packed + a.L.row_off) + strip * kStrip + r;
    const unsigned char* code_at = chunks + grp * kBlockBytes + strip * 512 + lane * 16;
    const unsigned char* scale_at = chunks + kBigB * kBlockBytes + (strip * kStrip + r) * 4;
    const uint32_t w_at = tbase + kWAt + ((uint32_t)(16 * strip) << 16);
    int s = 0, c = 0;                    // stage of the next chunk's first block; chunk slot
    uint32_t round = 0, slot_phase = 0;  // rounds of the stages; phase of the slot
    for (int j = 0; piece(j, p) && !bad; ++j) {
      float inv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) inv[h] = __ldg(row_inv + (p.tile / mt) * kTile + 8 * h);
      for (int k0 = p.k0; k0 < p.k1; k0 += kBigB) {
        const bool here = k0 + grp < p.k1;
        int se = s + grp;
        uint32_t re = round;
        if (se >= stages) se -= stages, ++re;
        if (!group_wait(2 + grp, 32 * kStrips, polls, &full_c[c], slot_phase, here && re > 0 ? &empty[se] : nullptr,
                        (re & 1) ^ 1)) {
          bad = true;
          break;
        }
        if (here) {
          const uint4 w = *reinterpret_cast<const uint4*>(code_at + c * kChunk);
          const int g = (((k0 + grp) * kBlock + q * 16) >> a.lg_group) - ((k0 * kBlock) >> a.lg_group);
          const unsigned char* sc = scale_at + c * kChunk + g * kGroupBytes;
          __half2 sh[2], bh[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(sc + 32 * h);
            sh[h] = __float2half2_rn(lo_bf16(v) * inv[h]);
            bh[h] = __float2half2_rn(hi_bf16(v) * inv[h]);
          }
          const uint4 o0 = expand(w.x, sh[0], bh[0]), o1 = expand(w.y, sh[0], bh[0]);  // row r, eight channels each
          const uint4 o2 = expand(w.z, sh[1], bh[1]), o3 = expand(w.w, sh[1], bh[1]);  // row r + 8
          fence_after();
          tmem_st_16x8(w_at + kWCols * se, o0, o1, o2, o3);
          fence_before();
        }
        bar_sync(2 + grp, 32 * kStrips);
        if (polls) {
          if (here) mbar_arrive_if(&full[se], lane == 0);
          mbar_arrive_if(&free_c[c], lane == 0);
        }
        s += min(kBigB, p.k1 - k0);
        if (s >= stages) s -= stages, ++round;
        if (++c == slots) c = 0, slot_phase ^= 1;
      }
    }
  } else if (warp < 6) {  // warp w reads TMEM lanes 32 (w % 4) .. + 31: weight rows 32 q + lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q = warp & 3, row = 32 * q + lane;
    const float* row_inv = reinterpret_cast<const float*>(a.packed + a.L.row_off);
    for (int j = 0; piece(j, p); ++j) {
      const int ab = j % accs, m0 = (p.tile % mt) * a.tn, n = (p.tile / mt) * kTile + row;
      const bool split = p.k1 - p.k0 < a.L.blocks;
      const float wf = 1.0f / __ldg(row_inv + n);  // (whole tiles of them are laid out)
      bar_sync(1, 128);  // the last tile's factors are read
      for (int c = tid - 64; c < a.tn; c += 128) s_xf[c] = a.xf[m0 + c];
      __syncwarp();
      if (!group_wait(1, 128, warp == 2, &acc_full[ab], (j / accs) & 1, nullptr, 0)) {  // the four warps leave together
        bad = true;
        break;
      }
      fence_after();
      const uint32_t src = tbase + 128 * ab + ((uint32_t)(32 * q) << 16);
      // 16 columns at a time, the next ones on their way
      uint32_t raw[2][16];
      const int cols = split ? a.tn : min(a.tn, (a.M - m0 + 15) & ~15);
      tmem_ld16_async(src, raw[0]);
      auto columns = [&](auto&& out) {
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = c + 16 * h;
            if (at < cols) {
              ld_wait(raw[h]);
              if (at + 16 < cols) tmem_ld16_async(src + at + 16, raw[h ^ 1]);
              out(at, raw[h]);
            }
          }
        }
      };
      if (split) {  // always a block's last piece: no other waits for the accumulator
        float* mine = a.part + (int64_t)blockIdx.x * a.tn * kTile + row;
        columns([&](int c, const uint32_t (&v)[16]) {
#pragma unroll
          for (int e = 0; e < 16; ++e) __stcg(mine + (c + e) * kTile, __uint_as_float(v[e]));
        });
        __threadfence();
        bar_sync(1, 128);
        if (tid == 64) s_last = atomicAdd(a.count + blockIdx.x / a.S, 1) == a.S - 1;
        break;
      }
      __nv_bfloat16* y = a.y + (int64_t)m0 * a.N + n;
      const bool ragged = n - lane + 32 > a.N;  // some of the warp's rows are past the last
      columns([&](int c, const uint32_t (&v)[16]) {
        const int left = a.M - m0 - c;
        auto put = [&](auto all) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 f = *reinterpret_cast<const float2*>(&s_xf[c + e]);
            const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(v[e]) * wf * f.x, __uint_as_float(v[e + 1]) * wf * f.y);
            if (all || e < left) y[0] = two.x;
            if (all || e + 1 < left) y[a.N] = two.y;
            y += 2 * (int64_t)a.N;
          }
        };
        if (ragged) {
          if (n < a.N) put(std::false_type{});
          __syncwarp();
        } else if (left >= 16) {
          put(std::true_type{});
        } else {
          put(std::false_type{});
        }
      });
      fence_before();
      __syncwarp();
      mbar_arrive_if(&acc_empty[ab], lane == 0);
    }
  }
  const bool any_bad = sync_tc_any(bad);
  if (any_bad && tid == 0) set_status(a.status, kStatusWaitTimeout | (GDN_K_LINEAR_Q4 << 8));
  if (warp == 0) tmem_dealloc(tbase, 512);
  if (!s_last) return;
  // the slices' sums in their order, by all threads: neighbours take neighbouring weight rows
  __threadfence();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tile = a.full * (int)gridDim.x + (int)blockIdx.x / a.S, m0 = tile % mt * a.tn, n0 = tile / mt * kTile;
  const float* parts = a.part + (int64_t)(blockIdx.x / a.S) * a.S * a.tn * kTile;
  const float* row_inv = reinterpret_cast<const float*>(a.packed + a.L.row_off);
  const int cols = min(a.tn, a.M - m0), rows = min(kTile, a.N - n0);
#pragma unroll 4
  for (int i = tid; i < cols * kTile; i += kBigThreads) {
    const int c = i / kTile, r = i % kTile;
    float p[8];
#pragma unroll
    for (int o = 0; o < 8; ++o) p[o] = o < a.S ? __ldcg(parts + (int64_t)o * a.tn * kTile + i) : 0.0f;
    float v = p[0];
#pragma unroll
    for (int o = 1; o < 8; ++o) v += p[o];
    if (r < rows) a.y[(int64_t)(m0 + c) * a.N + n0 + r] = __float2bfloat16_rn(v * (1.0f / __ldg(row_inv + n0 + r)) * a.xf[m0 + c]);
  }
}

}  // namespace

Q4Layout q4_layout(int32_t N, int32_t K, int32_t group) {
  Q4Layout L;
  L.tiles = (N + kTile - 1) / kTile;
  L.blocks = (K + kBlock - 1) / kBlock;
  L.groups = (K + group - 1) / group;
  L.row_groups = std::max(L.groups, L.blocks * kBlock / group);  // groups of 32: two for each block
  L.scale_off = (size_t)L.tiles * L.blocks * kBlockBytes;
  L.row_off = L.scale_off + (size_t)L.tiles * L.row_groups * kGroupBytes;
  L.total_bytes = L.row_off + (size_t)L.tiles * kTile * 4;
  return L;
}

cudaError_t launch_q4_pack(const void* codes, const void* scales, const void* biases, int32_t N, int32_t K,
                           int32_t group, void* packed, cudaStream_t stream) {
  const Q4Layout L = q4_layout(N, K, group);
  const int64_t blocks = ((int64_t)L.row_off / 4 + 255) / 256;
  {
    LaunchScope scope(GDN_K_Q4_PACK, stream);
    q4_pack_kernel<<<(unsigned)(blocks < 148 * 64 ? blocks : 148 * 64), 256, 0, stream>>>(
        (const unsigned char*)codes, (const unsigned short*)scales, (const unsigned short*)biases, N, K, group,
        (int64_t)L.groups * group / 2, L, (uint32_t*)packed);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  LaunchScope scope(GDN_K_Q4_PACK, stream);
  q4_rows_kernel<<<(unsigned)(L.tiles * kTile / 8), 256, 0, stream>>>((const unsigned short*)scales, (const unsigned short*)biases, N,
                                                            L, (float*)((unsigned char*)packed + L.row_off));
  return cudaGetLastError();
}

namespace {

// bf16 io: whether the products go by the kernels for few rows, which round no weight.  17 to 32 rows do where the weight is
// small; the border is in 128 x 64 blocks.  us, exact | rounded (linear_big_kernel), 17 and 32 rows: 1024 x 2048 (256 blocks)
// 6.0 | 11.3, 7.0 | 11.3; 2048 x 2048 (512) 10.9 | 12.2, 12.7 | 12.5; 4096 x 2048 (1024) 16.4 | 12.9, 18.8 | 13.5; 2560 x 5120
// (1600) 17.8 | 14.7, 19.9 | 15.8; 3840 x 3840 (1800) 14.9 | 15.9, 16.9 | 16.7; 5120 x 6144 (3840) 27.7 | 20.4, 30.9 | 20.8.
// Between 512 and 1500 up to 40 % are paid for exact products.
bool few_rows(int32_t M, const Q4Layout& L) { return M <= 16 || (M <= 32 && (int64_t)L.tiles * L.blocks <= 1500); }

// Blocks a tile: a block for each SM, while every warp keeps two blocks of K.  (Twice as many put 320 blocks of 5120 x
// 6144 in two rounds: one row 11.9 us against 9.3.)
int cluster_blocks(int64_t tiles, int blocks, int kw) {
  int S = 1;
  while (S < 8 && tiles * S < kSms + 2 && blocks >= 2 * S * kw) S *= 2;
  return S;
}
cudaLaunchConfig_t cluster_config(dim3 grid, int S, int smem, cudaStream_t stream, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = (unsigned)S, at->val.clusterDim.y = 1, at->val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = S > 1 ? 1 : 0;
  return cfg;
}

template <typename T, int G>
cudaError_t run_small(const T* x, int32_t M, int32_t K, const unsigned char* packed, const Q4Layout& L, int32_t N, T* y,
                      int32_t* status, cudaStream_t stream) {
  const int mg = (M + 7) / 8, S = cluster_blocks((int64_t)L.tiles * mg, L.blocks, kSmallWarps);
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(L.tiles * S), (unsigned)mg), S, kSmallSmem, stream, &at);
  cudaError_t e = cudaFuncSetAttribute(linear_small_kernel<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
  if (e != cudaSuccess) return e;
  LaunchScope scope(GDN_K_LINEAR_Q4, stream);
  return cudaLaunchKernelEx(&cfg, linear_small_kernel<T, G>, x, M, K, packed, L, N, y, S, status, 0u);
}
template <int MT, int G>
cudaError_t run_rows(const __nv_bfloat16* x, int32_t M, int32_t K, const unsigned char* packed, const Q4Layout& L, int32_t N,
                     __nv_bfloat16* y, int32_t* status, cudaStream_t stream) {
  constexpr int smem = rows_smem(MT, G);
  static_assert((smem + 2048) * rows_blocks(MT, G) <= 232448, "shared memory of an SM");
  const int S = cluster_blocks(L.tiles, L.blocks, rows_kw(MT));
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(L.tiles * S)), S, smem, stream, &at);
  cudaError_t e = cudaFuncSetAttribute(linear_rows_kernel<MT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  LaunchScope scope(GDN_K_LINEAR_Q4, stream);
  return cudaLaunchKernelEx(&cfg, linear_rows_kernel<MT, G>, x, M, K, packed, L, N, y, S, status, 0u);
}
template <int G>
cudaError_t run_few(bool bf16, const void* x, int32_t M, int32_t K, const unsigned char* w, const Q4Layout& L, int32_t N, void* y,
                    int32_t* status, cudaStream_t stream) {
  if (!bf16) {
    for (int32_t m0 = 0; m0 < M; m0 += 65535 * 8) {  // grid.y
      const cudaError_t e = run_small<float, G>((const float*)x + (int64_t)m0 * K, std::min(M - m0, 65535 * 8), K, w, L, N,
                                       (float*)y + (int64_t)m0 * N, status, stream);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const __nv_bfloat16* xb = (const __nv_bfloat16*)x;
  __nv_bfloat16* yb = (__nv_bfloat16*)y;
  if (M <= 8) return run_small<__nv_bfloat16, G>(xb, M, K, w, L, N, yb, status, stream);
  if (M <= 16) return run_rows<2, G>(xb, M, K, w, L, N, yb, status, stream);
  return run_rows<4, G>(xb, M, K, w, L, N, yb, status, stream);
}

struct BigPlan {
  int tn, mp, full, S, grid, rem;
};
// Rows of x a tile, rounds of whole tiles and slices of the rest: the fewest cycles on the fullest SM.  A 64-channel
// step takes 2 cycles a column in the products and about 300 for the expansion of its weights at least; the output
// of a tile 4000 where there is one accumulator; the slices' join 16 a column and slice (1100 rows of 5120 -> 17408:
// 167 us, with 8 of them 218).
BigPlan big_plan(int32_t M, const Q4Layout& L) {
  const int64_t nt = L.tiles;
  BigPlan best{};
  double least = 1e30;
  for (int tn = 16; tn <= 256; tn += 16) {
    BigPlan b;
    const int64_t mt = (M + tn - 1) / tn, tiles = nt * mt;
    b.tn = tn, b.mp = (int)(mt * tn), b.full = (int)(tiles / kSms), b.rem = (int)(tiles % kSms), b.S = 1;
    if (b.rem) b.S = (int)std::min<int64_t>(std::min(kSms / b.rem, 8), std::max(1, L.blocks / 4));
    b.grid = b.full ? kSms : b.rem * b.S;
    const double steps = b.full * (double)L.blocks + (b.rem ? (double)L.blocks / b.S : 0.0);
    const double cost = steps * std::max(300, 2 * tn) + (big_accs(tn) == 1 ? 4000.0 * b.full : 0.0) + (b.S > 1 ? 1000.0 + 16.0 * b.S * tn : 0.0);
    if (cost < least * 0.995) least = cost, best = b;
  }
  return best;
}
struct BigWs {
  size_t xf, part, count, total;
};
BigWs big_ws(const BigPlan& b, const Q4Layout& L) {
  BigWs w;
  w.xf = (size_t)b.mp * L.blocks * 128;
  w.part = (w.xf + (size_t)b.mp * 4 + 255) / 256 * 256;
  w.count = w.part + (b.S > 1 ? (size_t)b.rem * b.S * b.tn * kTile * 4 : 0);
  w.total = w.count + (size_t)b.rem * 4;
  return w;
}

}  // namespace

size_t linear_q4_ws_bytes(int32_t M, int32_t N, int32_t K, int32_t group, bool bf16) {
  const Q4Layout L = q4_layout(N, K, group);
  if (!bf16 || N == 0 || few_rows(M, L)) return 0;
  return big_ws(big_plan(M, L), L).total;
}

cudaError_t launch_linear_q4(bool bf16, const void* x, int32_t M, int32_t K, const void* packed, int32_t N,
                             int32_t group, void* y, void* ws, int32_t* status, cudaStream_t stream) {
  const Q4Layout L = q4_layout(N, K, group);
  const unsigned char* w = (const unsigned char*)packed;
  if (!bf16 || few_rows(M, L)) {
    if (group == 32) return run_few<32>(bf16, x, M, K, w, L, N, y, status, stream);
    if (group == 64) return run_few<64>(bf16, x, M, K, w, L, N, y, status, stream);
    return run_few<128>(bf16, x, M, K, w, L, N, y, status, stream);
  }
  const BigPlan b = big_plan(M, L);
  const BigWs bw = big_ws(b, L);
  unsigned char* xh = (unsigned char*)ws;
  float* xf = (float*)(xh + bw.xf);
  int32_t* count = (int32_t*)(xh + bw.count);
  {
    LaunchScope scope(GDN_K_X_HALF, stream);
    x_half_kernel<<<(unsigned)b.mp, 256, 0, stream>>>((const __nv_bfloat16*)x, M, K, L.blocks, b.mp, xh, xf, count, b.rem);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(linear_big_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBigSmem)) != cudaSuccess) return e;
  const BigArgs a{w, L, xh, xf, (float*)(xh + bw.part), count, (__nv_bfloat16*)y, M, N, b.mp, b.tn,
                  group == 32 ? 5 : group == 64 ? 6 : 7, b.full, b.S, status, 0};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)b.grid);
  cfg.blockDim = dim3(kBigThreads);
  cfg.dynamicSmemBytes = kBigSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  LaunchScope scope(GDN_K_LINEAR_Q4, stream);
  return cudaLaunchKernelEx(&cfg, linear_big_kernel, a);
}

}  // namespace gdn
