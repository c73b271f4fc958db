// What the two attention kernels over the 4-bit cache share: the rows of a
// sequence's query tiles, the cutting of their cache tiles into equal quotas, one
// a block, and the partial rows that the blocks leave.
//
// Groups.  The query rows of a (sequence, key/value head) are (query token, query
// head) pairs, cut into row tiles of RT rows; a group is one row tile and counts
// GU units, for its queries and its output, and one unit for each TT keys that its
// last row sees.  The units of all groups, end to end, are cut into equal quotas,
// so that ragged lengths fill the SMs evenly.  A group that crosses blocks leaves
// unnormalised partial rows in the workspace for a combine kernel.
//
// A launch takes the sequences whose rows a key/value head lie in its range and passes
// over the others, which have no units in it: so a sequence's rounding, and what a short
// one computes, does not depend on whether the call holds long ones.
#pragma once

#include "../../include/gdn.h"
#include "internal.h"
#include "kv4.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;  // how far (powers of two) a score may pass the running maximum before it moves
constexpr int kAttnSms = 148;

// Partial rows of the blocks: slot 2b holds block b's part of a group that starts in an earlier block, slot 2b + 1
// that of a group that starts in b and leaves it.
struct AttnWorkspace {
  float* o;     // [2 * blocks][rows][D]
  float2* ml;   // [2 * blocks][rows]: running maximum (log2 units) and sum
  int4* split;  // [blocks]: (sequence, head, row tile, last block) of the group that starts in b and leaves it, or last -1
};

struct AttnArgs {
  AttnProblem p;
  KvCache cache;
  AttnWorkspace ws;
  int32_t G;  // blocks
  int32_t least, most;  // rows a key/value head of the sequences that this launch takes
  int32_t* status;
  uint32_t zero;  // 0, unknown to the compiler
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {  // 2^x to 2 ulp, subnormal results as zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// rows of a sequence's query tiles and the keys they see
struct AttnRows {
  int32_t rows;   // new * (Hq / Hkv); 0 where another launch takes the sequence
  int32_t first;  // keys that query token 0 sees: len - new + 1
  int32_t cap;    // positions that the page table's row covers
};
__device__ __forceinline__ AttnRows rows_of(const AttnArgs& a, int n) {
  const int nw = a.p.cu[n + 1] - a.p.cu[n];
  const int rows = nw * (a.p.Hq / a.cache.Hkv);
  return AttnRows{rows >= a.least && rows <= a.most ? rows : 0, kv_len(a.cache, n) - nw + 1, a.cache.width * a.cache.page_size};
}

// inclusive sum over the block's threads
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += s_warp[w];
  return v;
}

// A block's walk over the pieces of its quota.
template <int RT, int TT, int GU, int MIN>
struct AttnWalk {
  int64_t u, u_end, at, quota;  // units: here, the quota's end, into the group, a quota
  int n, h, rt, tiles;          // sequence, head, row tile; the group's tiles
  int t0, t1;                   // the piece's tiles
  AttnRows rw;

  __device__ __forceinline__ static int tiles_of(const AttnArgs& a, const AttnRows& r, int i) {
    const int last = min(r.rows, (i + 1) * RT) - 1;  // the tile's last row sees most
    const int seen = min(r.first + last / (a.p.Hq / a.cache.Hkv), r.cap);
    return max(1, (seen + TT - 1) / TT);  // at least one: somebody writes the rows
  }
  __device__ __forceinline__ static int64_t head_units(const AttnArgs& a, const AttnRows& r) {  // of one head
    int64_t x = 0;
    for (int j = 0; j * RT < r.rows; ++j) x += GU + tiles_of(a, r, j);
    return x;
  }
  __device__ __forceinline__ static int64_t div(int64_t x, int64_t y) {  // of positive numbers; 64-bit division is slow
    return ((x | y) >> 31) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
  }
  // Every thread of the block; false: nothing to do.  s_warp: a word a warp, s_found: four (the sum; the sequence, the
  // units before it, those of a head).  Up to as many sequences as threads are looked at once; more, in rounds, twice:
  // for the sum, then for the sequence that holds u.
  __device__ __forceinline__ bool start(const AttnArgs& a, int threads, int64_t* s_warp, int64_t* s_found) {
    const int tid = threadIdx.x;
    int64_t total = 0, own = 0, upto = 0, head = 0;
    for (int n0 = 0; n0 < a.p.N; n0 += threads) {
      head = n0 + tid < a.p.N ? head_units(a, rows_of(a, n0 + tid)) : 0;
      own = head * a.cache.Hkv;
      upto = block_scan(own, s_warp);
      if (tid == threads - 1) s_found[0] = upto;
      __syncthreads();
      total += s_found[0];
    }
    quota = max((int64_t)MIN, div(total + a.G - 1, a.G));
    u = quota * blockIdx.x;
    u_end = min(total, u + quota);
    if (tid == 0) a.ws.split[blockIdx.x] = make_int4(0, 0, 0, -1);
    if (u >= u_end) return false;
    if (a.p.N <= threads) {
      if (upto - own <= u && u < upto) s_found[1] = tid, s_found[2] = upto - own, s_found[3] = head;
      __syncthreads();
    } else {
      int64_t before = 0;
      for (int n0 = 0; n0 < a.p.N; n0 += threads) {
        head = n0 + tid < a.p.N ? head_units(a, rows_of(a, n0 + tid)) : 0;
        own = head * a.cache.Hkv;
        upto = before + block_scan(own, s_warp);
        __syncthreads();
        if (upto - own <= u && u < upto) s_found[1] = n0 + tid, s_found[2] = upto - own, s_found[3] = head;
        if (tid == threads - 1) s_warp[0] = upto;
        __syncthreads();
        before = s_warp[0];
        __syncthreads();
        if (before > u) break;
      }
    }
    n = (int)s_found[1];
    at = u - s_found[2];
    rw = rows_of(a, n);
    h = (int)div(at, s_found[3]), rt = 0;
    at -= h * s_found[3];
    for (int w; at >= (w = GU + tiles_of(a, rw, rt)); ++rt) at -= w;
    return true;
  }
  // the piece at u; false when the quota holds none of the group's tiles
  __device__ __forceinline__ bool piece(const AttnArgs& a) {
    tiles = tiles_of(a, rw, rt);
    const int64_t left = at + (u_end - u) - GU;  // the quota's end, from the group's first tile
    t0 = (int)max((int64_t)0, at - GU), t1 = (int)max((int64_t)0, min((int64_t)tiles, left));
    return t0 < t1;
  }
  __device__ __forceinline__ int rows_here() const { return min(RT, rw.rows - rt * RT); }
  __device__ __forceinline__ int last_block() const { return (int)div(u - at + GU + tiles - 1, quota); }  // of the group
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    u += GU + tiles - at;
    at = 0;
    if (u >= u_end) return false;
    if ((rt + 1) * RT < rw.rows) {
      ++rt;
      return true;
    }
    rt = 0;
    if (++h == a.cache.Hkv) {
      h = 0;
      do rw = rows_of(a, ++n); while (rw.rows == 0);  // a sequence without rows here has no units
    }
    return true;
  }
};

// the x-th block that started a group and did not finish it, or -1 (256 threads; s_count: a word a warp and round)
constexpr int kSplitPer = 3;  // blocks a thread looks at: up to 768
__device__ __forceinline__ int split_group(const AttnArgs& a, int x, int* s_count, int* s_first) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) *s_first = -1;
  uint32_t ball[kSplitPer];
#pragma unroll
  for (int i = 0; i < kSplitPer; ++i) {
    const int b = i * 256 + threadIdx.x;
    ball[i] = __ballot_sync(0xffffffffu, b < a.G && a.ws.split[b].w >= 0);
    if (lane == 0) s_count[i * 8 + warp] = __popc(ball[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSplitPer; ++i) {
    int before = __popc(ball[i] & ((1u << lane) - 1u));
    for (int w = 0; w < i * 8 + warp; ++w) before += s_count[w];
    if (((ball[i] >> lane) & 1u) && before == x) *s_first = i * 256 + threadIdx.x;
  }
  __syncthreads();
  return *s_first;
}

// attention_prefill.cu: bf16 io, the sequences with more than prefill_from(D) rows
constexpr int prefill_rows(int D) { return D <= 128 ? 256 : 128; }  // a block's
cudaError_t launch_attention_prefill(const AttnArgs& a, cudaStream_t stream);

}  // namespace gdn
