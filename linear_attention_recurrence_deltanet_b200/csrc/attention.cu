// Causal attention over the 4-bit paged cache (kv4.cuh): for query token i of a
// sequence of `len` cached tokens, of which the last `new` are the queries' own,
//   o = sum_t p_t v_t,  p = softmax over t <= len - new + i of scale q . k_t.
//
// The codes go to the tensor cores as they are, as small integers, and the
// scales and biases of their groups are applied outside the products:
//   q . k_t = sum_g s_tg (q_g . (c_tg - 8)) + (b_tg + 8 s_tg) sum(q_g),
//   o = sum_t (p_t s_t) (c_t - 8) + sum_t p_t (b_t + 8 s_t),
// with the codes less 8 exact in 16 bits.  bf16 io: fp16 operands, query rows brought
// below 2^8 by a power of two each (exactly, but for elements 2^-22 of the row's
// largest), and nothing rounded but p_t s_t, to fp16 under a power of two of the
// warp's largest s_t: 2^-11 of it, or, where it is below 2^-17 of that largest, 2^-28
// of the largest.  The outputs' bf16 rounds by 2^-8; a second part of p_t s_t cost 8 %.
// fp32 io: bf16 operands, queries and p_t s_t in three parts.
//
// Keys and values are the A operand (16 keys x 16 channels, 16 channels x 16
// keys), eight query rows the B operand: a lane then scales two keys for all rows,
// and a tile of eight rows wastes nothing.  The probabilities turn from an output
// into an operand by movmatrix.
//
// Row tiles of 16 rows, 8 where no sequence has more; tiles of 16 keys
// (attention.cuh has the cutting).  The four warps of a block take every fourth
// tile of its piece and join at the piece's end.
#include <algorithm>

#include "attention.cuh"
#include "tc.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kGroupUnits = 20;  // what a group costs beside its tiles, in tiles
// the least quota: short contexts are spread over more blocks, whose parts have to be joined (one token over 2000 keys, 24 / 2
// heads of 128: 4 14.1 us, 7 14.6, 10 15.0, 20 16.8; over 8000: 16.8, 16.0, 16.0, 17.4; 16 of them over 300: 16.4, 16.0, 17.2, 18.7)
constexpr int kMinUnits = 7;

constexpr int stages(int D) { return D == 64 ? 8 : 4; }
// what registers and shared memory allow (all_fit below; a third block of 256 x 8 rows waited for a place, and every quota
// was two thirds of one: 64 requests of 16 / 2 heads of 256 68.7 us, two blocks 51.8)
constexpr int blocks_per_sm(int D, int RT) { return D == 256 ? 2 : RT == 8 ? 4 : 3; }
// queries in shared memory where a warp's copy would take too many registers
constexpr bool q_in_smem(int D, int RT, int TQ) { return D * TQ * (RT / 8) > 128; }
constexpr int smem_bytes(int D, int RT, int TQ) {
  return kWarps * stages(D) * kv_tile_bytes(D) + (q_in_smem(D, RT, TQ) ? D / 16 * TQ * 512 : 0);
}

// Codes less 8 of a word's nibbles 0 and 4 (lo) and 1 and 5 (hi), as pairs of bf16 or fp16.  A mask and an exponent turn a
// nibble into the low mantissa bits of 128 (bf16) or 1024 (fp16, nibble 1 as 16 c, which saves its shift).  They sit in
// registers whose values the compiler does not know (a kernel argument that is 0 is in them), so that one instruction
// takes both.
template <bool F32>
struct Codes {
  uint32_t mask_lo, mask_hi, magic;
  __device__ __forceinline__ explicit Codes(uint32_t zero)
      : mask_lo(0x000f000fu + zero), mask_hi(0x00f000f0u + zero), magic((F32 ? 0x43004300u : 0x64006400u) + zero) {}
  __device__ __forceinline__ uint32_t lo(uint32_t w) const {
    uint32_t r;
    if constexpr (F32)
      asm("{\n.reg .b32 t;\nlop3.b32 t, %1, %2, %3, 0xEA;\nsub.rn.bf16x2 %0, t, %4;\n}\n"  // ((w & mask) | magic) - 136
          : "=r"(r)
          : "r"(w), "r"(mask_lo), "r"(magic), "r"(0x43084308u));
    else
      asm("{\n.reg .b32 t;\nlop3.b32 t, %1, %2, %3, 0xEA;\nadd.rn.f16x2 %0, t, %4;\n}\n"  // ((w & mask) | magic) - 1032
          : "=r"(r)
          : "r"(w), "r"(mask_lo), "r"(magic), "r"(0xe408e408u));
    return r;
  }
  __device__ __forceinline__ uint32_t hi(uint32_t w) const {
    if constexpr (F32) return lo(w >> 4);
    uint32_t r;
    asm("{\n.reg .b32 t;\nlop3.b32 t, %1, %2, %3, 0xEA;\nfma.rn.f16x2 %0, t, %4, %5;\n}\n"  // (1024 + 16 c) / 16 - 72
        : "=r"(r)
        : "r"(w), "r"(mask_hi), "r"(magic), "r"(0x2c002c00u), "r"(0xd480d480u));
    return r;
  }
};
template <bool F32>
__device__ __forceinline__ uint32_t pair(float lo, float hi) {  // the operand type
  if constexpr (F32) return bf16x2(lo, hi);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
template <bool F32>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F32)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool F32>
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {  // C = 0
  if constexpr (F32)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {  // of bf16: lane (r, q) has row r, columns 2q, 2q + 1
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D, RT)) attn_kernel(const __grid_constant__ AttnArgs a) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int TQ = F32 ? 3 : 1;          // parts of a query
  constexpr int TP = F32 ? 3 : 1;          // parts of p_t s_t
  constexpr int GK = D / kKGroup, GV = D / v_group(D), CB = D / 64, NM = D / 16;
  constexpr int S = stages(D), TB = kv_tile_bytes(D);
  constexpr bool QS = q_in_smem(D, RT, TQ);
  constexpr int NR = RT / 8;               // groups of eight rows: a lane has rows 2q, 2q + 1 of each
  static_assert(!F32 || RT == 16, "fp32 io runs 16-row tiles");

  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t s_full[kWarps][S];
  __shared__ int64_t s_warp[kWarps];
  __shared__ int64_t s_found[4];
  __shared__ float2 s_ml[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  unsigned char* ring = smem + warp * (S * TB);
  uint4* s_q = reinterpret_cast<uint4*>(smem + kWarps * S * TB);
  const AttnProblem& p = a.p;
  const int Gq = p.Hq / a.cache.Hkv;

  if (threadIdx.x < kWarps * S) tc::mbar_init(&s_full[threadIdx.x / S][threadIdx.x % S], 1);
  tc::mbar_init_fence();

  AttnWalk<RT, kKvTile, kGroupUnits, kMinUnits> walk;
  if (!walk.start(a, kThreads, s_warp, s_found)) return;
  const float c_log2 = p.scale * kLog2e;
  const Codes<F32> codes(a.zero);
  uint32_t used = 0;  // tiles this warp has passed: stage used % S, phase used / S
  bool dead = false;

  while (true) {
    if (walk.piece(a)) {
    const int n = walk.n, h = walk.h, rt = walk.rt, t_begin = walk.t0, t_end = walk.t1;
    const AttnRows rw = walk.rw;
    const int row_last = min(rw.rows, (rt + 1) * RT) - 1;
    const int whole = min(rw.first + rt * RT / Gq, rw.cap) / kKvTile;  // every row of the group sees the tiles before this one
    const int seen_tiles = (max(0, min(rw.first + row_last / Gq, rw.cap)) + kKvTile - 1) / kKvTile;

    // This warp's tiles: t_begin + warp + 4 j.  Every 32 of them, lane j looks up the place of the j-th, and asks for it
    // when its turn comes, S - 1 tiles ahead.  A tile without a page passes through the ring as an empty stage.
    const int stop = min(t_end, seen_tiles);
    const int count = !dead && t_begin + warp < stop ? (stop - t_begin - warp + kWarps - 1) / kWarps : 0;
    int64_t place = -1;
    auto look_up = [&](int j0) {
      const int t = t_begin + warp + kWarps * (j0 + lane);
      place = -1;
      if (j0 + lane < count) {
        place = kv_tile_at(a.cache, D, n, t * kKvTile, h);
        if (place < 0) set_status(a.status, kStatusBadPage | (GDN_K_ATTENTION << 8));
      }
    };
    auto fetch = [&](int j) {  // by the lane that looked tile j up
      if (lane == (j & 31) && j < count) {
        const uint32_t s = (used + j) & (S - 1);  // (used: before the piece)
        if (place >= 0) {
          tc::mbar_expect_tx(&s_full[warp][s], TB);
          tc::bulk_load(ring + s * TB, a.cache.pool + place, TB, &s_full[warp][s]);
        } else {
          tc::mbar_arrive(&s_full[warp][s]);
        }
      }
    };
    look_up(0);
    uint32_t valid = __ballot_sync(0xffffffffu, place >= 0), valid_next = valid;  // of the 32 tiles around the use side
#pragma unroll 1
    for (int j = 0; j < S - 1; ++j) fetch(j);

    // keys that this lane's rows see; a row that is none sees all and is not written
    int lim[NR][2];
#pragma unroll
    for (int k = 0; k < NR; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = rt * RT + 8 * k + 2 * q + e;
        lim[k][e] = row < rw.rows ? max(0, min(rw.first + row / Gq, rw.cap)) : 0x7fffffff;
        if (row < rw.rows && rw.first + row / Gq > rw.cap) set_status(a.status, kStatusBadPage | (GDN_K_ATTENTION << 8));
      }
    // queries as B fragments: lane (r, q) holds channels 16q .. 16q+15 of each 64 of row r, paired (c, c + 4) as the
    // codes are; [group], [2 + group]
    uint32_t qf[QS ? 1 : NM][4];
    float qsum[NR][2][GK], unit[NR][2];  // sums of the row as it went into the operand; what that is a multiple of
    if constexpr (QS) __syncthreads();   // the last piece's reads of s_q
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = rt * RT + r + 8 * i;
      const bool on = i < NR && row < rw.rows;
      const T* src = (const T*)p.q + (int64_t)(p.cu[n] + (on ? row / Gq : 0)) * p.ldq + (int64_t)(h * Gq + (on ? row % Gq : 0)) * D;
      float scale = 1.0f;
      if constexpr (!F32) {
        if (i < NR) {
          uint32_t top = 0;  // largest finite magnitude of the row, as bits
#pragma unroll
          for (int c = 0; c < 2 * GK; ++c) {
            const uint4 v = on ? ld16_rw(src + (c >> 1) * 64 + q * 16 + (c & 1) * 8) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = (w[e] << 16) & 0x7fff0000u, hi = w[e] & 0x7fff0000u;
              if (lo < 0x7f800000u) top = max(top, lo);
              if (hi < 0x7f800000u) top = max(top, hi);
            }
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = max(-100, (int)(top >> 23) - 127);
          scale = pow2(7 - e);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (i < NR) unit[i < NR ? i : 0][e] = F32 ? 1.0f : 1.0f / __shfl_sync(0xffffffffu, scale, (2 * q + e) * 4);
#pragma unroll
      for (int g = 0; g < GK; ++g) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.0f;
        if (on) {
          float y[8];
          load8(src + g * 64 + q * 16, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = F32 ? y[e] : y[e] * scale;
          load8(src + g * 64 + q * 16 + 8, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[8 + e] = F32 ? y[e] : y[e] * scale;
        }
        if (i < NR) {
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) s += x[e];
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
          for (int e = 0; e < 2; ++e) qsum[i < NR ? i : 0][e][g] = __shfl_sync(0xffffffffu, s, (2 * q + e) * 4);
        }
#pragma unroll
        for (int term = 0; term < TQ; ++term) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int e = 8 * (m >> 1) + 2 * (m & 1);
            const uint32_t f0 = pair<F32>(x[e], x[e + 4]), f1 = pair<F32>(x[e + 1], x[e + 5]);
            if constexpr (F32) {
              x[e] -= lo_bf16(f0), x[e + 4] -= hi_bf16(f0), x[e + 1] -= lo_bf16(f1), x[e + 5] -= hi_bf16(f1);
            }
            if constexpr (QS) {
              if (g % kWarps == warp) {
                uint32_t* d = reinterpret_cast<uint32_t*>(s_q + ((g * 4 + m) * TQ + term) * 32 + lane);
                d[i] = f0, d[2 + i] = f1;
              }
            } else if (i < NR) {
              qf[g * 4 + m][i] = f0, qf[g * 4 + m][2 + i] = f1;
            }
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) unit[k][0] *= c_log2, unit[k][1] *= c_log2;
    if constexpr (QS) __syncthreads();

    float o[NR][CB][4][4];                   // [channels 8r + 2j, + 1 of each 64][two channels x two rows]
    float mx[NR][2], l[NR][2], ob[NR][2][GV];
    // bf16 io: p_t s_t times v_scale = 2^(6 - v_ref), where s_t < v_lim = 2^(v_ref + 1)
    int v_ref = -100;
    float v_scale = F32 ? 1.0f : 0.0f, v_lim = 0.0f;
    const int seen_all = min(rw.first + row_last / Gq, rw.cap);  // keys that some row sees
#pragma unroll
    for (int k = 0; k < NR; ++k) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[k][e] = -INFINITY, l[k][e] = 0.0f;
#pragma unroll
        for (int g = 0; g < GV; ++g) ob[k][e][g] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[k][cb][j][e] = 0.0f;
      }
    }

    int done = count;  // tiles passed (fewer after a wait that ran out)
    for (int j = 0; j < count; ++j) {
      const int jf = j + S - 1;
      if ((jf & 31) == 0) {
        look_up(jf);
        valid_next = __ballot_sync(0xffffffffu, place >= 0);
      }
      if ((j & 31) == 0) valid = valid_next;
      fetch(jf);
      const uint32_t stage = (used + j) & (S - 1);
      if (!tc::mbar_wait_warp(&s_full[warp][stage], ((used + j) / S) & 1)) {
        set_status(a.status, kStatusWaitTimeout | (GDN_K_ATTENTION << 8));
        dead = true;
        done = j;
        break;
      }
      if (!((valid >> (j & 31)) & 1u)) continue;
      const int t = t_begin + warp + kWarps * j;
      const unsigned char* tile = ring + stage * TB;
      const uint32_t* scales = reinterpret_cast<const uint32_t*>(tile + kv_scale_off(D)) + r;  // of keys r and r + 8

      // scores: [group][key r or r + 8][row 2q or 2q + 1]
      float s[NR][2][2];
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) s[k][i][0] = s[k][i][1] = 0.0f;
#pragma unroll
      for (int g = 0; g < GK; ++g) {
        float acc[NR][4];
        uint2 kw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) kw[i] = *reinterpret_cast<const uint2*>(tile + g * 512 + (8 * i + r) * 32 + q * 8);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int sh = 8 * (m & 1);
          uint32_t c0[2], c1[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = (m < 2 ? kw[i].x : kw[i].y) >> sh;
            c0[i] = codes.lo(w), c1[i] = codes.hi(w);
          }
#pragma unroll
          for (int term = 0; term < TQ; ++term) {
            uint32_t f[4];
            if constexpr (QS) {
              const uint4 v = s_q[((g * 4 + m) * TQ + term) * 32 + lane];
              f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = qf[g * 4 + m][e];
            }
#pragma unroll
            for (int k = 0; k < NR; ++k) {
              if (m == 0 && term == 0) mma0<F32>(acc[k], c0[0], c0[1], c1[0], c1[1], f[k], f[2 + k]);
              else mma<F32>(acc[k], c0[0], c0[1], c1[0], c1[1], f[k], f[2 + k]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = scales[g * kKvTile + 8 * i];
          const float sk = lo_bf16(w), z = fmaf(8.0f, sk, hi_bf16(w));
#pragma unroll
          for (int k = 0; k < NR; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[k][i][e] = fmaf(sk, acc[k][2 * i + e], fmaf(z, qsum[k][e][g], s[k][i][e]));
        }
      }
      // online softmax in powers of two.  The running maximum moves only when a score passes it by kSlack, which is
      // rare after the first tiles; until then exponentials are at most 2^kSlack.
      const bool masked = t >= whole;
      const int key = t * kKvTile + r;
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) s[k][i][0] *= unit[k][0], s[k][i][1] *= unit[k][1];
      if (masked) {
        __syncwarp();  // (keeps the branch a branch)
#pragma unroll
        for (int k = 0; k < NR; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (key + 8 * i >= lim[k][e]) s[k][i][e] = -INFINITY;
      }
      float sv[GV][2], bv[GV][2];  // of the values of keys r and r + 8: scale, and bias moved to code 8
#pragma unroll
      for (int gv = 0; gv < GV; ++gv)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = scales[(GK + gv) * kKvTile + 8 * i];
          sv[gv][i] = lo_bf16(w), bv[gv][i] = fmaf(8.0f, sv[gv][i], hi_bf16(w));
        }
      bool over = false;
      if constexpr (!F32) {
#pragma unroll
        for (int gv = 0; gv < GV; ++gv)
#pragma unroll
          for (int i = 0; i < 2; ++i) over |= fabsf(sv[gv][i]) >= v_lim && (!masked || key + 8 * i < seen_all);
      }
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) over |= fmaxf(s[k][0][e], s[k][1][e]) > mx[k][e] + kSlack;
      if (__any_sync(0xffffffffu, over)) {
        float fv = 1.0f;
        if constexpr (!F32) {  // a larger scale than all before moves the reference, by three powers of two more
          uint32_t top = 0;
#pragma unroll
          for (int gv = 0; gv < GV; ++gv)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (!masked || key + 8 * i < seen_all) {
                const uint32_t bits = __float_as_uint(fabsf(sv[gv][i]));
                if (bits < 0x7f800000u) top = max(top, bits);  // (NaN reaches the rows that see it by itself)
              }
          top = __reduce_max_sync(0xffffffffu, top);
          const int e = max(-100, (int)(top >> 23) - 127);
          if (e > v_ref || v_lim == 0.0f) {
            const int before = v_ref;
            v_ref = min(e + 3, 120);
            fv = exp2f((float)(before - v_ref));
            v_scale = pow2(6 - v_ref), v_lim = pow2(v_ref + 1);
          }
        }
#pragma unroll
        for (int k = 0; k < NR; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[k][0][e], s[k][1][e]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            m = fmaxf(m, mx[k][e]);
            const float f = m == mx[k][e] ? 1.0f : ex2(mx[k][e] - m);
            mx[k][e] = m;
            l[k][e] *= f;
#pragma unroll
            for (int g = 0; g < GV; ++g) ob[k][e][g] *= f;
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[k][cb][x][e] *= f * fv, o[k][cb][x][2 + e] *= f * fv;
          }
      }
#pragma unroll
      for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m = mx[k][e] == -INFINITY ? 0.0f : mx[k][e];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float pe = F32 ? exp2f(s[k][i][e] - m) : ex2(s[k][i][e] - m);
            s[k][i][e] = pe;
            l[k][e] += pe;
          }
        }
      // values: p_t s_t, in parts and turned into B fragments, against the codes
#pragma unroll
      for (int gv = 0; gv < GV; ++gv) {
        uint32_t f[NR][TP][2];
#pragma unroll
        for (int k = 0; k < NR; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x[2], y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) x[e] = s[k][i][e] * (F32 ? sv[gv][i] : sv[gv][i] * v_scale), y[e] = s[k][i][e] * bv[gv][i];
            if (masked) {  // what a row does not see may hold anything
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (key + 8 * i >= lim[k][e]) x[e] = y[e] = 0.0f;
            }
            ob[k][0][gv] += y[0], ob[k][1][gv] += y[1];
#pragma unroll
            for (int tp = 0; tp < TP; ++tp) {
              const uint32_t w = pair<F32>(x[0], x[1]);
              f[k][tp][i] = transpose8x8(w);
              if constexpr (F32) x[0] -= lo_bf16(w), x[1] -= hi_bf16(w);
            }
          }
#pragma unroll
        for (int cb = gv * (CB / GV); cb < (gv + 1) * (CB / GV); ++cb) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = *reinterpret_cast<const uint32_t*>(tile + kv_v_off(D) + cb * 512 + ((e >> 1) * 8 + (e & 1) * 4 + q) * 32 + r * 4);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7632 : 0x5410;
            const uint32_t w01 = __byte_perm(w[0], w[1], sel), w23 = __byte_perm(w[2], w[3], sel);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {  // channels 8r + 4 half + 2 jj and the next
              uint32_t c[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                c[e] = e ? codes.hi(w01 >> (8 * jj)) : codes.lo(w01 >> (8 * jj));
                c[2 + e] = e ? codes.hi(w23 >> (8 * jj)) : codes.lo(w23 >> (8 * jj));
              }
#pragma unroll
              for (int k = 0; k < NR; ++k)
#pragma unroll
                for (int tp = 0; tp < TP; ++tp)
                  mma<F32>(o[k][cb][2 * half + jj], c[0], c[1], c[2], c[3], f[k][tp][0], f[k][tp][1]);
            }
          }
        }
      }
      __syncwarp();  // the stage is read before it is refilled
    }
    if (dead)  // the copies still in flight land before the ring is used for the join
      for (int j = done; j < min(count, done + S); ++j)
        tc::mbar_wait_warp(&s_full[warp][(used + j) & (S - 1)], ((used + j) / S) & 1, tc::kWaitTries / 64);
    used += count;

    // the join: every warp's rows (unnormalised, bias added) into its ring, then all threads over rows and channels
    float* mine = reinterpret_cast<float*>(ring);
    constexpr int LD = D + 4;
    static_assert(RT * LD * 4 <= S * TB, "the join uses the ring");
#pragma unroll
    for (int k = 0; k < NR; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * k + 2 * q + e;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[k][e] += __shfl_xor_sync(0xffffffffu, l[k][e], x);
#pragma unroll
          for (int g = 0; g < GV; ++g) ob[k][e][g] += __shfl_xor_sync(0xffffffffu, ob[k][e][g], x);
        }
        if (r == 0) s_ml[warp][row] = make_float2(mx[k][e], l[k][e]);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float b = ob[k][e][cb * GV / CB], u = F32 ? 1.0f : pow2(v_ref - 6);
            *reinterpret_cast<float4*>(mine + row * LD + cb * 64 + 8 * r + 4 * half) =
                make_float4(fmaf(u, o[k][cb][2 * half][e], b), fmaf(u, o[k][cb][2 * half][2 + e], b),
                            fmaf(u, o[k][cb][2 * half + 1][e], b), fmaf(u, o[k][cb][2 * half + 1][2 + e], b));
          }
      }
    __syncthreads();
    const bool from_start = t_begin == 0, to_end = t_end == walk.tiles;
    const int rows_here = row_last - rt * RT + 1;
    const int slot = 2 * blockIdx.x + (from_start ? 1 : 0);
    for (int x = threadIdx.x; x < rows_here * (D / 4); x += kThreads) {
      const int row = x / (D / 4), c = (x - row * (D / 4)) * 4;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w][row].x);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float sl = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w][row];
        if (ml.x == -INFINITY && ml.y == 0.0f) continue;
        const float f = exp2f(ml.x - m);
        const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * (S * TB)) + row * LD + c);
        v.x = fmaf(f, y.x, v.x), v.y = fmaf(f, y.y, v.y), v.z = fmaf(f, y.z, v.z), v.w = fmaf(f, y.w, v.w);
        sl = fmaf(f, ml.y, sl);
      }
      if (from_start && to_end) {
        const int gr = rt * RT + row, tok = p.cu[n] + gr / Gq;
        const int64_t out = (int64_t)tok * p.Hq + h * Gq + gr % Gq;
        const float inv = sl == 0.0f ? 0.0f : 1.0f / sl;
        T* d = (T*)p.o + out * D + c;
        if constexpr (F32) {
          *reinterpret_cast<float4*>(d) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        } else {
          *reinterpret_cast<uint2*>(d) = make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
        }
        if (c == 0 && p.lse) p.lse[out] = sl == 0.0f ? -INFINITY : (m + log2f(sl)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(a.ws.o + ((int64_t)slot * 16 + row) * D + c) = v;
        if (c == 0) a.ws.ml[slot * 16 + row] = make_float2(m, sl);
      }
    }
    if (threadIdx.x == 0 && from_start && !to_end) a.ws.split[blockIdx.x] = make_int4(n, h, rt, walk.last_block());
    }  // a piece with tiles
    if (!walk.next(a)) break;
    tc::fence_async_all();  // the join's writes to the ring, before the next piece's copies into it
    __syncthreads();
  }
}

// One block per (split group, row, D / gridDim.z channels): joins the partial rows that the group's blocks have left.
// Block x takes the x-th of the blocks that started a group and did not finish it.  Four channels a thread, the weights
// 2^(m_i - m) of all parts first, so that the loads of the rows do not wait on one another.
constexpr int kCombineThreads = 256, kCombineWarps = kCombineThreads / 32, kMaxBlocks = 256 * kSplitPer;
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kCombineThreads) attn_combine_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ float4 s_o[kCombineThreads];
  __shared__ float s_w[kMaxBlocks], s_m[kCombineWarps], s_l[kCombineWarps];
  __shared__ int s_count[kMaxBlocks / 32], s_first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y;
  const int first = split_group(a, blockIdx.x, s_count, &s_first);
  if (first < 0) return;
  const int4 sp = a.ws.split[first];
  const AttnRows rw = rows_of(a, sp.x);
  const int gr = sp.z * RT + row;
  if (gr >= rw.rows) return;
  const int Gq = a.p.Hq / a.cache.Hkv, parts = sp.w - first + 1;
  auto slot_of_part = [&](int i) { return (int64_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * 16 + row; };
  float2 ml[kSplitPer];
  float m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kSplitPer; ++i) {
    const int x = i * kCombineThreads + threadIdx.x;
    ml[i] = x < parts ? a.ws.ml[slot_of_part(x)] : make_float2(-INFINITY, 0.0f);
    m = fmaxf(m, ml[i].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_m[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) m = fmaxf(m, s_m[w]);
#pragma unroll
  for (int i = 0; i < kSplitPer; ++i) {
    const bool none = ml[i].x == -INFINITY && ml[i].y == 0.0f;  // a part whose tokens the row does not see
    const float f = none ? -1.0f : exp2f(ml[i].x - m);
    if (!none) l = fmaf(f, ml[i].y, l);
    s_w[i * kCombineThreads + threadIdx.x] = f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  const int quads = D / 4 / gridDim.z, sub = threadIdx.x / quads, subs = kCombineThreads / quads;
  const int c = (blockIdx.z * quads + threadIdx.x - sub * quads) * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = sub; i < parts; i += subs) {
    const float f = s_w[i];
    if (f < 0.0f) continue;
    const float4 y = *reinterpret_cast<const float4*>(a.ws.o + slot_of_part(i) * D + c);
    v.x = fmaf(f, y.x, v.x), v.y = fmaf(f, y.y, v.y), v.z = fmaf(f, y.z, v.z), v.w = fmaf(f, y.w, v.w);
  }
  s_o[threadIdx.x] = v;
  __syncthreads();
  if (sub > 0) return;
  float sl = 0.0f;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) sl += s_l[w];
  for (int i = 1; i < min(subs, parts); ++i) {
    const float4 y = s_o[i * quads + threadIdx.x];
    v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
  }
  const float inv = sl == 0.0f ? 0.0f : 1.0f / sl;
  const int64_t out = (int64_t)(a.p.cu[sp.x] + gr / Gq) * a.p.Hq + sp.y * Gq + gr % Gq;
  T* d = (T*)a.p.o + out * D + c;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(d) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  } else {
    *reinterpret_cast<uint2*>(d) = make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
  }
  if (c == 0 && a.p.lse) a.p.lse[out] = sl == 0.0f ? -INFINITY : (m + log2f(sl)) * kLn2;
}

int grid_of(int D, int RT) { return kAttnSms * blocks_per_sm(D, RT); }
// the quotas count on a place for every block: 228 KB an SM, 1 KB of each block the driver's
constexpr bool all_fit(int D, int RT, int TQ) { return blocks_per_sm(D, RT) * (smem_bytes(D, RT, TQ) + 1024 + 1024) <= 228 * 1024; }
static_assert(all_fit(64, 8, 1) && all_fit(128, 8, 1) && all_fit(256, 8, 1), "8-row tiles");
static_assert(all_fit(64, 16, 1) && all_fit(128, 16, 1) && all_fit(256, 16, 1), "16-row tiles");
static_assert(all_fit(64, 16, 3) && all_fit(128, 16, 3) && all_fit(256, 16, 3), "16-row tiles, fp32");
static_assert(kAttnSms * blocks_per_sm(64, 8) <= kMaxBlocks, "split_group looks at kSplitPer blocks a thread");

struct WsLayout {
  size_t o, ml, split, total;
};
WsLayout ws_layout(int D, int blocks, int rows) {
  const size_t g = (size_t)blocks;
  WsLayout w;
  w.o = 0;
  w.ml = w.o + g * 2 * rows * D * sizeof(float);
  w.split = w.ml + g * 2 * rows * sizeof(float2);
  w.total = (w.split + g * sizeof(int4) + 255) / 256 * 256;
  return w;
}
AttnWorkspace ws_at(const WsLayout& w, void* ws) {
  unsigned char* b = (unsigned char*)ws;
  return AttnWorkspace{(float*)(b + w.o), (float2*)(b + w.ml), (int4*)(b + w.split)};
}

// bf16 io: sequences with more rows a key/value head than this take the long row tiles.  One border a head size, since a
// sequence's rounding goes by it and must not depend on the call's other sequences; which side is faster does.  16 / 2 heads,
// short | long tiles, us:
//   D = 128, one sequence over 4000 keys: 56 rows 18 | 27, 96 22 | 28, 192 23 | 38; 16 of them: 40 rows 41 | 40, 56 50 | 41, 72 58 | 41
//   D = 64, one over 20000: 56 rows 19 | 35, 192 32 | 54; 16 of them: 40 rows 81 | 89, 56 104 | 89, 72 126 | 90
//   D = 256, one over 20000: 56 rows 36 | 54, 128 57 | 57, 160 58 | 53; 16 of them: 24 rows 143 | 135, 72 328 | 143, 128 514 | 152
constexpr int prefill_from(int D) { return D <= 128 ? 64 : 128; }

// What a call's sequences ask for: of those with up to `border` rows a key/value head, their rows, how many and the longest;
// whether there are others.
struct Split {
  int64_t rows;
  int32_t seqs, longest;
  bool longer;
};
Split split_at(const AttnProblem& p, int32_t Hkv, int64_t border) {
  Split s{};
  for (int32_t n = 0; n < p.N; ++n) {
    const int64_t rows = (int64_t)(p.cu_host[n + 1] - p.cu_host[n]) * (p.Hq / Hkv);
    if (rows > border) s.longer = true;
    else if (rows > 0) s.rows += rows, ++s.seqs, s.longest = std::max(s.longest, (int32_t)rows);
  }
  return s;
}

template <typename T, int D, int RT>
cudaError_t run(const AttnProblem& p, const KvCache& cache, const Split& s, void* ws, int32_t* status, cudaStream_t stream) {
  const AttnArgs a{p, cache, ws_at(ws_layout(D, grid_of(D, RT), 16), ws), grid_of(D, RT), 1, s.longest, status, 0};
  constexpr int bytes = smem_bytes(D, RT, sizeof(T) == 4 ? 3 : 1);
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<T, D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  {
    LaunchScope scope(GDN_K_ATTENTION, stream);
    attn_kernel<T, D, RT><<<a.G, kThreads, bytes, stream>>>(a);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // as many split groups as there are groups, or blocks; rows of the longest sequence's tile
  const int64_t groups = (s.rows / RT + s.seqs) * cache.Hkv;
  const int rows = std::min(RT, s.longest);
  const int64_t x = std::min<int64_t>(groups, a.G);
  // few rows have many parts: the channels go to D / 32 blocks (131072 tokens, 24 rows: 15.6 -> 6.3 us); many rows have
  // few, and the blocks that find no group cost more (64 sequences of 8 heads: 6.6 us against 14.4)
  const int z = x * rows <= 2 * kAttnSms ? D / 32 : 1;
  LaunchScope scope(GDN_K_ATTN_COMBINE, stream);
  attn_combine_kernel<T, D, RT><<<dim3((unsigned)x, rows, z), kCombineThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_d(const AttnProblem& p, const KvCache& c, const Split& s, void* ws, int32_t* status, cudaStream_t st) {
  if (!p.bf16) return run<float, D, 16>(p, c, s, ws, status, st);
  // a tile of 8 rows is half the products of one of 16, whose second half would be empty
  if (s.longest <= 8) return run<__nv_bfloat16, D, 8>(p, c, s, ws, status, st);
  return run<__nv_bfloat16, D, 16>(p, c, s, ws, status, st);
}

}  // namespace

size_t attention_ws_bytes(int32_t T, int32_t, int32_t Hq, int32_t Hkv, int32_t D, bool bf16) {
  size_t w = ws_layout(D, grid_of(D, 8), 16).total;  // the larger grid
  if (bf16 && (int64_t)T * (Hq / Hkv) > prefill_from(D)) w = std::max(w, ws_layout(D, kAttnSms, prefill_rows(D)).total);
  return w;
}

cudaError_t launch_attention(const AttnProblem& p, const KvCache& cache, void* ws, int32_t* status,
                             cudaStream_t stream) {
  const int32_t border = p.bf16 ? prefill_from(p.D) : 0x7fffffff;
  const Split s = split_at(p, cache.Hkv, border);
  // one after the other: both may use the workspace
  if (s.longer) {
    const cudaError_t e = launch_attention_prefill(
        AttnArgs{p, cache, ws_at(ws_layout(p.D, kAttnSms, prefill_rows(p.D)), ws), kAttnSms, border + 1, 0x7fffffff, status, 0}, stream);
    if (e != cudaSuccess || s.seqs == 0) return e;
  }
  if (p.D == 64) return run_d<64>(p, cache, s, ws, status, stream);
  if (p.D == 128) return run_d<128>(p, cache, s, ws, status, stream);
  return run_d<256>(p, cache, s, ws, status, stream);
}

}  // namespace gdn
