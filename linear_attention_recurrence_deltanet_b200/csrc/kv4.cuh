// The 4-bit key/value cache: page layout, quantisation of a group and the angles
// of the rotation, shared by the kernels that write and read it.
//
// A page holds page_size tokens (a multiple of 16) of every key/value head as
//   [Hkv][page_size / 16] tiles of 16 tokens, tile_bytes each:
//     K codes   [D / 64 groups][16 tokens][32 bytes]
//     V codes   [D / 64 blocks][16 rows][32 bytes], token t of the tile in row v_row(t)
//     K scales  [D / 64][16 tokens] words, V scales [D / v_group][16 tokens] words
// Eight channels are one 32-bit word of codes, channel i in bits 4i .. 4i+3.  A
// scale word holds the group's scale (low half) and bias (high half) in bf16;
// a code c stands for scale * c + bias.
//
// One tile is one contiguous piece, so a reader streams a head's tokens with
// large copies.  Rows of 32 bytes are whole sectors for the writer.  The order
// of the V rows (the even tokens of each eight before the odd ones) lets the
// four lanes that need tokens 2q of a tile read 32 different banks.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/gdn.h"
#include "common.cuh"
#include "vec.cuh"

namespace gdn {

constexpr int kKvTile = 16;     // tokens of a tile
constexpr int kKGroup = 64;     // channels that share a key scale

__host__ __device__ constexpr int v_group(int D) { return D < 128 ? D : 128; }
__host__ __device__ constexpr int kv_groups(int D) { return D / kKGroup + D / v_group(D); }
__host__ __device__ constexpr int kv_tile_bytes(int D) { return kKvTile * (D + 4 * kv_groups(D)); }
__host__ __device__ constexpr int kv_v_off(int D) { return kKvTile * D / 2; }
__host__ __device__ constexpr int kv_scale_off(int D) { return kKvTile * D; }
__host__ __device__ constexpr int v_row(int t) { return (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3); }

// A paged cache as the kernels see it (sizes validated on the host; page ids
// and lengths are device data and checked where they are used).
struct KvCache {
  unsigned char* pool;
  const int32_t* table;   // [N, width] page ids
  const int32_t* lens;    // [N] tokens of each sequence, the new ones included
  int64_t page_bytes;
  int32_t width, num_pages, page_size, Hkv;
};

// Tokens of a sequence, the new ones included.  A negative number holds none, as 0 does; positions counted back from it stay
// within int32.
__device__ __forceinline__ int kv_len(const KvCache& c, int n) { return max(c.lens[n], -(1 << 30)); }

// Bytes of the pool before the tile of (head h, position p) of sequence n, or
// -1 when p has no page: past the table's row, or a page id outside the pool.
__device__ __forceinline__ int64_t kv_tile_at(const KvCache& c, int D, int n, int p, int h) {
  const int pg = p / c.page_size;
  if (pg >= c.width) return -1;
  const int id = c.table[(int64_t)n * c.width + pg];
  if (id < 0 || id >= c.num_pages) return -1;
  return (int64_t)id * c.page_bytes +
         ((int64_t)h * (c.page_size / kKvTile) + (p - pg * c.page_size) / kKvTile) * kv_tile_bytes(D);
}

// the sequence of packed token t: the last n with cu[n] <= t (empty sequences are passed over)
__device__ __forceinline__ int seq_of(const int32_t* cu, int N, int t) {
  int lo = 0, hi = N;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// NaN-propagating minimum and maximum
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Quantises one group spread over `lanes` neighbouring lanes, eight channels a
// lane: the word of codes, and the scale word (the same in every lane).
//   bias = bf16(min), scale = bf16((max - min) * fl32(1/15)),
//   code = clamp(rint((x - bias) / scale), 0, 15)
// Every step is a correctly rounded fp32 operation without contraction, so that
// the codes, which step at their borders, do not depend on the compiler.  A
// group with a value that is not finite (or whose range is not) stands for NaN.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], int lanes, uint32_t& scale_word) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = min_nan(lo, x[i]), hi = max_nan(hi, x[i]);
  for (int o = 1; o < lanes; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float range = __fsub_rn(hi, lo);
  __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(range, 1.0f / 15.0f));
  __nv_bfloat16 bb = __float2bfloat16_rn(lo);
  if (!isfinite(range) || !isfinite(__bfloat162float(bb))) sb = bb = __ushort_as_bfloat16(0x7fc0);
  scale_word = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(bb) << 16);
  const float s = __bfloat162float(sb), b = __bfloat162float(bb);
  uint32_t w = 0;
  if (s > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = rintf(__fdiv_rn(__fsub_rn(x[i], b), s));
      w |= (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f) << (4 * i);
    }
  }
  return w;
}

// what eight codes stand for
__device__ __forceinline__ void dequantise8(uint32_t w, uint32_t scale_word, float (&x)[8]) {
  const float s = __uint_as_float(scale_word << 16), b = __uint_as_float(scale_word & 0xffff0000u);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(s, (float)((w >> (4 * i)) & 15u), b);
}

// eight consecutive io elements at a 16-byte aligned address
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    Vec16<T>::unpack(ld16_rw(p), x);
  } else {
    Vec16<T>::unpack(ld16_rw(p), x);
    Vec16<T>::unpack(ld16_rw(p + 4), x + 4);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    st16(p, Vec16<T>::pack(x));
  } else {
    st16(p, Vec16<T>::pack(x));
    st16(p + 4, Vec16<T>::pack(x + 4));
  }
}

// Cosine and sine of a pair at a position.  turn is the frequency in turns per
// position as a 64-bit fraction, so pos * turn mod 2^64 is the angle's
// fraction of a turn without a range reduction: its error is |pos| * 2^-65
// turns, at any position.  Evaluated in fp64 and rounded once.
__device__ __forceinline__ float2 rope_angle(uint64_t turn, int64_t pos) {
  const uint64_t ph = (uint64_t)pos * turn;
  double s, c;
  sincospi((double)(int64_t)ph * 1.0842021724855044e-19, &s, &c);  // 2^-63: half turns
  return make_float2((float)c, (float)s);
}

}  // namespace gdn
