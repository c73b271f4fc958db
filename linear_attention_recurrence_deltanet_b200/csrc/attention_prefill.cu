// Causal attention over the 4-bit paged cache for many query rows (chunked
// prefill; bf16 io, heads of 64 or 128 channels), on tcgen05:
//   S = Q K^T, P = 2^(S - m) and O = P V on tiles of 128 rows x 128 keys.
//
// Operands are fp16, with powers of two over them: query rows are brought below 2^8
// (exactly, but for elements 2^-22 of the row's largest), keys and values below
// 2^12 by the largest of the block so far.  Keys go as s (c - 8), which is exact in
// 11 bits, and the rest, b + 8 s by group, times the sums of the query's groups, as
// 16 more channels in high and low parts:
//   q . k_t = sum_g q_g . s_tg (c_tg - 8) + (b_tg + 8 s_tg) sum(q_g),
// so that scores, and the log of their sum, are those of fp32.  (Keys as s c + b
// in fp16 put 2^-12 of a score into the log of a short row's sum.)  Values,
// s c + b, and probabilities are off by half a step of fp16, 2^-11, against 2^-8
// in bf16, at the same rate.  A value group that stands for NaN is expanded as
// zeros and noted by token, so that it reaches the rows that see it and no other.
//
// A block takes two tiles of 128 query rows (tokens x the heads that share a
// key/value head) through the same keys.  Warps 0-3 and 4-7 are the softmax of
// either tile, a thread a row; warps 8-15 expand, 16 keys each; warp 16 issues the
// products (17-19 fill its group up).  While one tile's softmax runs the other's products do.  S is 128
// columns of TMEM, P overwrites its first 64 in fp16 and is the A operand of P V.
// O stays in TMEM; the running maximum moves only when a score passes it by
// kSlack, and only then is O rescaled.
#include <cuda_fp16.h>

#include "attention.cuh"
#include "tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kRows = kPrefillRows, kKeys = 128;
constexpr int kSoftWarps = 8, kExpandWarps = 8, kThreads = (kSoftWarps + kExpandWarps + 4) * 32;
// Registers a thread after the start: 640 threads begin with 96, 61440 in all; these come to 60416.
constexpr int kSoftRegs = 128, kExpandRegs = 80, kProductRegs = 56;
static_assert((kSoftWarps * kSoftRegs + kExpandWarps * kExpandRegs + 4 * kProductRegs) * 32 <= kThreads * 96, "register split");
template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
using Walk = AttnWalk<kRows, kKeys, 3, 6>;     // a group's queries and output cost about three tiles

constexpr int tile_bytes(int D) { return kKeys * D * 2; }
constexpr int kSide = kKeys * 32;  // the 16 more channels of a tile: 32 bytes a row, 32-byte swizzle
constexpr int smem_bytes(int D) {  // one block an SM, which takes all of its TMEM
  return 6 * tile_bytes(D) + 4 * kSide + 1024 < 120000 ? 120000 : 6 * tile_bytes(D) + 4 * kSide + 1024;
}
// byte offset of eight of a row's 16 more channels, and the descriptor of such a tile (K-major, 8 rows a 256-byte group)
__device__ __forceinline__ uint32_t side_chunk(int row, int i) { return (uint32_t)(row * 32 + ((i ^ (row >> 2)) & 1) * 16); }
__device__ __forceinline__ uint64_t desc_side(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | (1ull << 16) | (16ull << 32) | (1ull << 46) | (6ull << 61);
}
// x in two halves: its fp16 and the fp16 of the rest
__device__ __forceinline__ uint32_t high_low(float x) {
  const __half h = __float2half_rn(x), l = __float2half_rn(x - __half2float(h));
  return (uint32_t)__half_as_ushort(h) | ((uint32_t)__half_as_ushort(l) << 16);
}

// what the expanding warps say of a key tile
struct alignas(16) Meta {
  float k_unit;          // a key's value = its operand times this
  float v_unit;          // the same of the values, of this tile and all before
  float v_step;          // v_unit before / after this tile: O is rescaled by it
  uint32_t rare;         // some keys have no page (1), some values are NaN (2); the four are read as one uint4
  uint8_t valid[8];      // 16 keys each: they have a page
  uint16_t v_nan[8];     // by key: its value is NaN
};

// Eight codes as values s c + b or keys s (c - 8), in the order 0 4 1 5 2 6 3 7.  Nibbles 1, 3, .. are masked into 1024 + 16 c, which saves their
// shift.  The masks sit in registers whose values the compiler does not know (a kernel argument that is 0 is in them),
// so that one instruction takes a mask and the exponent.
struct Expand {
  uint32_t lo, hi, magic;
  __device__ __forceinline__ explicit Expand(uint32_t zero)
      : lo(0x000f000fu + zero), hi(0x00f000f0u + zero), magic(0x64006400u + zero) {}
  template <typename F>
  __device__ __forceinline__ uint4 by(uint32_t w, float off, const F& f) const {  // f of the codes less `off`
    uint32_t o[4];
    const __half2 kl = __float2half2_rn(-1024.0f - off), k16 = __float2half2_rn(0.0625f), kh = __float2half2_rn(-64.0f - off);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t x, y;
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "r"(lo), "r"(magic));  // (w & mask) | magic
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "r"(hi), "r"(magic));
      const __half2 wl = f(__hadd2(*reinterpret_cast<const __half2*>(&x), kl));
      const __half2 wh = f(__hfma2(*reinterpret_cast<const __half2*>(&y), k16, kh));
      o[2 * i] = *reinterpret_cast<const uint32_t*>(&wl);
      o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&wh);
      w >>= 8;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
  __device__ __forceinline__ uint4 value(uint32_t w, __half2 s, __half2 b) const {
    return by(w, 0.0f, [&](__half2 c) { return __hfma2(c, s, b); });
  }
  __device__ __forceinline__ uint4 key(uint32_t w, __half2 s) const {
    return by(w, 8.0f, [&](__half2 c) { return __hmul2(c, s); });
  }
};
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// exponent of a finite magnitude's bits, at least -100
__device__ __forceinline__ int exponent(uint32_t bits) { return max(-100, (int)(bits >> 23) - 127); }
__device__ __forceinline__ bool finite_word(uint32_t w) {
  return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}
// bound of the magnitudes that a finite scale word's codes stand for (twice the largest at most)
__device__ __forceinline__ float reach(uint32_t w) { return fmaf(15.0f, fabsf(lo_bf16(w)), fabsf(hi_bf16(w))); }

__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}
// 32 columns of this thread's lane, not waited for; ld_wait() ends all loads in flight
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// the wait names the registers that the load fills, so that no use moves before it
__device__ __forceinline__ void ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
// a b + c and a + b of two floats in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 x, y, z, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\nfma.rn.f32x2 w, x, y, z;\n"
      "mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 x, y, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 w, x, y;\nmov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int GK = D / kKGroup, CB = D / 64, TB = kv_tile_bytes(D), TILE = tile_bytes(D);
  constexpr uint32_t kO = 256;  // TMEM: S of either tile at 0 and 128, O at 256 and 256 + D
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], o_full[2], kv_full[2], kv_free[2], drain;
  __shared__ Meta meta[2];
  __shared__ uint2 s_top[kExpandWarps];
  __shared__ int64_t s_warp[kThreads / 32], s_found[4];
  __shared__ uint32_t tslot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnProblem& p = a.p;
  const int Gq = p.Hq / a.cache.Hkv;

  Walk walk;
  if (!walk.start(a, kThreads, s_warp, s_found)) return;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_free[i], 1);
    }
    mbar_init(&drain, 1);
    mbar_init_fence();
  }
  if (warp == kSoftWarps + kExpandWarps) tmem_alloc(&tslot, 512);
  sync_tc();
  const uint32_t tbase = tslot;
  bool bad = false;
  int kt = 0;  // key tiles before this one, over all pieces: stage kt & 1

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    more_regs<kSoftRegs>();
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lanes + 128 * x, to = tbase + lanes + kO + D * x;
    unsigned char* sq = sm + x * TILE;
    const float c_log2 = fabsf(p.scale) * kLog2e;
    uint32_t ph_s = 0, ph_o = 0;
    do {
      if (!walk.piece(a)) continue;
      const int tiles = walk.t1 - walk.t0;
      if (x == 1 && walk.rows_here() <= 128) {  // no rows in the second tile
        kt += tiles;
        continue;
      }
      const AttnRows rw = walk.rw;
      const int row = walk.rt * kRows + x * 128 + r;
      const bool on = row < rw.rows;
      const int tok = p.cu[walk.n] + (on ? row / Gq : 0), head = walk.h * Gq + (on ? row % Gq : 0);
      // keys this row sees; a row that is none sees all there are and is not written
      const int lim = on ? max(0, min(rw.first + row / Gq, rw.cap)) : 0x7fffffff;
      const int whole = min(rw.first + (walk.rt * kRows + x * 128) / Gq, rw.cap);  // every row of the tile sees these
      if (on && rw.first + row / Gq > rw.cap) set_status(a.status, kStatusBadPage | (GDN_K_ATTENTION << 8));
      // the query row as an operand; a negative scale turns its sign
      float unit = 0.0f;
      {
        const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)p.q + (int64_t)tok * p.ldq + (int64_t)head * D);
        uint32_t top = 0;
        if (on) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = src[c];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = (w[e] << 16) & 0x7fff0000u, hi = w[e] & 0x7fff0000u;
              if (lo < 0x7f800000u) top = max(top, lo);
              if (hi < 0x7f800000u) top = max(top, hi);
            }
          }
        }
        const int e = exponent(top);
        unit = pow2(e - 7);
        const float f = p.scale < 0.0f ? -pow2(7 - e) : pow2(7 - e);
        float sum[GK];
#pragma unroll
        for (int g = 0; g < GK; ++g) sum[g] = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          float v[8], z[8];
          Vec16<__nv_bfloat16>::unpack(on ? src[c] : make_uint4(0, 0, 0, 0), v);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = v[(j >> 1) + 4 * (j & 1)] * f, sum[c / 8] += z[j];  // channels in the order of Expand
          *reinterpret_cast<uint4*>(sq + kmaj_chunk(128, r, c * 8)) = pack8h(z);
        }
        uint32_t side[4] = {0, 0, 0, 0};  // high, low, high, low by group
#pragma unroll
        for (int g = 0; g < GK; ++g) side[2 * g] = side[2 * g + 1] = high_low(sum[g]);
        unsigned char* row_side = sm + 6 * TILE + x * kSide;
        *reinterpret_cast<uint4*>(row_side + side_chunk(r, 0)) = make_uint4(side[0], side[1], side[2], side[3]);
        *reinterpret_cast<uint4*>(row_side + side_chunk(r, 1)) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[x]);
      }
      float m = -INFINITY, l = 0.0f, v_unit = 1.0f;
      bool nan = false;
      for (int t = walk.t0; t < walk.t1; ++t, ++kt) {
        if (!group_wait(1 + x, 128, (warp & 3) == 0, &s_full[x], ph_s, nullptr, 0)) {
          bad = true;
          break;
        }
        ph_s ^= 1;
        fence_after();
        const Meta& mt = meta[kt & 1];
        const uint4 units = *reinterpret_cast<const uint4*>(&mt);
        const float f = unit * __uint_as_float(units.x) * c_log2, v_step = __uint_as_float(units.z);
        v_unit = __uint_as_float(units.y);
        uint2 valid = make_uint2(0x01010101u, 0x01010101u);
        const int left = lim - t * kKeys;  // keys of this tile that the row sees
        const bool masked = (t + 1) * kKeys > whole || (units.w & 1u);
        if (units.w & 1u) valid = *reinterpret_cast<const uint2*>(mt.valid);
        auto seen = [&](int c) { return c < left && ((c < 64 ? valid.x >> (8 * (c >> 4)) : valid.y >> (8 * ((c >> 4) - 4))) & 1u); };
        if (units.w & 2u) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int k = left - 16 * i;
            nan |= (mt.v_nan[i] & (k >= 16 ? 0xffffu : k <= 0 ? 0u : (1u << k) - 1u)) != 0;
          }
        }
        // S is read twice, 32 columns at a time and the next ones on their way: for the largest product, then for the
        // probabilities
        uint32_t raw[2][32];
        tmem_ld32_async(ts, raw[0]);
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t(&cur)[32] = raw[c & 1];
          ld_wait(cur);
          tmem_ld32_async(ts + 32 * ((c + 1) & 3), raw[(c + 1) & 1]);  // the last: the first again
          if (masked) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 32; ++e) cur[e] = seen(32 * c + e) ? cur[e] : 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) top = fmaxf(top, fmaxf(__uint_as_float(cur[e]), __uint_as_float(cur[e + 1])));
        }
        top = top == -INFINITY ? top : top * f;
        if (__any_sync(0xffffffffu, top > m + kSlack || v_step != 1.0f)) {
          const float m2 = fmaxf(m, top), g = m2 == m ? 1.0f : ex2(m - m2);
          m = m2;
          l *= g;
          if (t > walk.t0) {  // the product of the last tile is done: S came after it
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              float z[16];
              uint32_t w[16];
              tmem_ld16(to + c0, z);
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(z[e] * (g * v_step));
              tmem_st16(to + c0, w);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : -m;
        float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t(&cur)[32] = raw[c & 1];
          ld_wait(cur);
          if (c < 3) tmem_ld32_async(ts + 32 * (c + 1), raw[(c + 1) & 1]);
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 z = fma2(make_float2(__uint_as_float(cur[e]), __uint_as_float(cur[e + 1])), make_float2(f, f),
                                  make_float2(base, base));
            v[e] = ex2(z.x), v[e + 1] = ex2(z.y);
          }
          if (masked) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = seen(32 * c + e) ? v[e] : 0.0f;
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], make_float2(v[e], v[e + 1]));
            const __half2 h = __floats2half2_rn(v[e], v[e + 1]);
            w[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
          }
          __syncwarp();
          tmem_st16(ts + 16 * c, w);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (bad || !group_wait(1 + x, 128, (warp & 3) == 0, &o_full[x], ph_o, nullptr, 0)) {
        bad = true;
        break;
      }
      ph_o ^= 1;
      fence_after();
      // rows out: whole, or unnormalised to the workspace
      const bool from_start = walk.t0 == 0, to_end = walk.t1 == walk.tiles;
      const bool is_whole = from_start && to_end;
      const int64_t out = (int64_t)tok * p.Hq + head;
      const int64_t slot = ((int64_t)(2 * blockIdx.x + (from_start ? 1 : 0)) * kRows + x * 128 + r);
      const float f = nan ? __int_as_float(0x7fc00000) : is_whole ? (l == 0.0f ? 0.0f : v_unit / l) : v_unit;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float v[32];
        tmem_ld32(to + c0, v);
        if (!on) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float z[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) z[(j >> 1) + 4 * (j & 1)] = v[8 * c + j] * f;
          if (is_whole) {
            st16((__nv_bfloat16*)p.o + out * D + c0 + 8 * c, Vec16<__nv_bfloat16>::pack(z));
          } else {
            float4* d = reinterpret_cast<float4*>(a.ws.o + slot * D + c0 + 8 * c);
            d[0] = make_float4(z[0], z[1], z[2], z[3]);
            d[1] = make_float4(z[4], z[5], z[6], z[7]);
          }
        }
      }
      if (on) {
        if (is_whole) {
          if (p.lse) p.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
          a.ws.ml[slot] = make_float2(m, l);
        }
      }
      if (tid == 0 && from_start && !to_end)
        a.ws.split[blockIdx.x] = make_int4(walk.n, walk.h, walk.rt, walk.last_block());
      fence_before();  // O is read before the next piece's first product, which waits for p_full
    } while (walk.next(a));
  } else if (warp < kSoftWarps + kExpandWarps) {
    // ------------------------------------------------------------- expansion
    fewer_regs<kExpandRegs>();
    const int w = warp - kSoftWarps, half = lane & 1, tk = lane >> 1;
    const int tv = (tk & 8) | ((tk & 3) << 1) | ((tk >> 2) & 1);  // the token of V row tk (v_row's inverse)
    int k_ref = -100, v_ref = -100;                               // exponents of the largest values so far
    float k_lim = -1.0f, v_lim = -1.0f, fk = 0.0f, fv = 0.0f;     // what they hold, and their scales
    const Expand expand(a.zero);
    // where this lane's four chunks of 64 channels go, of keys and of values
    const bool odd = (tv >> 2) & 1;  // pairs of words in turn: the eight lanes of a store then hit all banks
    uint32_t at_k[4], at_v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      at_k[j] = 2 * TILE + kmaj_chunk(kKeys, 16 * w + tk, (half * 4 + j) * 8);
      at_v[j] = 3 * TILE + mnmaj_chunk(kKeys, 16 * w + tv, (half * 4 + (j ^ (odd ? 1 : 0))) * 8);
    }
    do {
      if (!walk.piece(a)) continue;
      const int n = walk.n, h = walk.h;
      const int all = max(0, min(walk.rw.first + (walk.rt * kRows + walk.rows_here() - 1) / Gq, walk.rw.cap));  // keys anybody sees
      uint4 kc[CB], vc[CB], kn[CB], vnx[CB];
      uint32_t ks[GK], vs, ksn[GK], vsn;
      bool ok, okn;
      int64_t place = -1;
      // this warp's 16 keys of tile t; every 32 tiles lane j looks the j-th of them up
      auto load = [&](int t, uint4 (&k4)[CB], uint4 (&v4)[CB], uint32_t (&sk)[GK], uint32_t& sv, bool& there) {
        if ((t - walk.t0) % 32 == 0) {
          const int pos = (t + lane) * kKeys + 16 * w;
          place = -1;
          if (t + lane < walk.t1 && pos < all) {
            place = kv_tile_at(a.cache, D, n, pos, h);
            if (place < 0) set_status(a.status, kStatusBadPage | (GDN_K_ATTENTION << 8));
          }
        }
        const int64_t at = __shfl_sync(0xffffffffu, place, (t - walk.t0) % 32);
        const int pos = t * kKeys + 16 * w;
        there = at >= 0 || pos >= all;
#pragma unroll
        for (int g = 0; g < CB; ++g) k4[g] = v4[g] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int g = 0; g < GK; ++g) sk[g] = 0;
        sv = 0;
        if (at >= 0) {
          const unsigned char* tile = a.cache.pool + at;
          const uint32_t* sc = reinterpret_cast<const uint32_t*>(tile + kv_scale_off(D));
#pragma unroll
          for (int g = 0; g < CB; ++g) {
            k4[g] = *reinterpret_cast<const uint4*>(tile + g * 512 + lane * 16);
            v4[g] = *reinterpret_cast<const uint4*>(tile + kv_v_off(D) + g * 512 + lane * 16);
          }
          if (pos + tk < all) {  // behind the last key the codes may be anything
#pragma unroll
            for (int g = 0; g < GK; ++g) sk[g] = sc[g * kKvTile + tk];
          }
          if (pos + tv < all) sv = sc[GK * kKvTile + tv];
        }
      };
      load(walk.t0, kc, vc, ks, vs, ok);
      for (int t = walk.t0; t < walk.t1; ++t, ++kt) {
        if (t + 1 < walk.t1) load(t + 1, kn, vnx, ksn, vsn, okn);
        const int st = kt & 1;
        // Mostly the tile's keys and values stay within the references and are finite, and every key has a page: one
        // barrier says so, which the wait for the stage needs anyway.
        float rk = 0.0f;
#pragma unroll
        for (int g = 0; g < GK; ++g) rk = fmaxf(rk, reach(ks[g]));
        const float rv = reach(vs);
        bool odd_k = false;
#pragma unroll
        for (int g = 0; g < GK; ++g) odd_k |= !finite_word(ks[g]);
        const bool v_bad = !finite_word(vs);
        const bool plain = rk <= k_lim && rv <= v_lim && !odd_k && !v_bad && ok;
        bool waited = true;
        if (kt >= 2 && w == 0) waited = mbar_wait_warp(&kv_free[st], ((kt >> 1) & 1) ^ 1);
        if (bar_or(3, 32 * kExpandWarps, !plain || !waited)) {
          // the rest of it: whether the wait ran out, the tile's largest finite key and value, what is odd
          uint32_t top_k = 0;
#pragma unroll
          for (int g = 0; g < GK; ++g)
            if (finite_word(ks[g])) top_k = max(top_k, __float_as_uint(reach(ks[g])));
          top_k = __reduce_max_sync(0xffffffffu, top_k);
          uint32_t top_v = __reduce_max_sync(0xffffffffu, v_bad ? 0u : __float_as_uint(rv));
          const uint32_t nans = __reduce_or_sync(0xffffffffu, v_bad ? 1u << tv : 0u);
          if (v_bad) vs = 0;
          if (lane == 0) {
            s_top[w] = make_uint2(top_k, top_v);
            meta[st].valid[w] = ok ? 1 : 0;
            meta[st].v_nan[w] = (uint16_t)nans;
          }
          if (bar_or(3, 32 * kExpandWarps, !waited)) {
            bad = true;
            break;
          }
          const bool no_page = bar_or(3, 32 * kExpandWarps, !ok), any_nan = bar_or(3, 32 * kExpandWarps, nans != 0);
#pragma unroll
          for (int i = 0; i < kExpandWarps; ++i) top_k = max(top_k, s_top[i].x), top_v = max(top_v, s_top[i].y);
          // a larger exponent than all before moves the reference, by three more
          const int ek = exponent(min(top_k, 0x7f7fffffu)), ev = exponent(min(top_v, 0x7f7fffffu)), v_old = v_ref;
          if (ek > k_ref) k_ref = min(ek + 3, 127);
          if (ev > v_ref) v_ref = min(ev + 3, 127);
          fk = pow2(11 - k_ref), fv = pow2(11 - v_ref);
          k_lim = k_ref >= 127 ? 3.0e38f : pow2(k_ref + 1) * 0.99f, v_lim = v_ref >= 127 ? 3.0e38f : pow2(v_ref + 1) * 0.99f;
          if (w == 0 && lane == 0) {
            meta[st].v_step = v_old == v_ref ? 1.0f : exp2f((float)(v_old - v_ref));
            meta[st].rare = (no_page ? 1u : 0u) | (any_nan ? 2u : 0u);
          }
          bar_sync(3, 32 * kExpandWarps);  // s_top is read
        } else if (w == 0 && lane == 0) {
          meta[st].v_step = 1.0f, meta[st].rare = 0;
        }
        if (w == 0 && lane == 0) meta[st].k_unit = pow2(k_ref - 11), meta[st].v_unit = pow2(v_ref - 11);
        unsigned char* stage = sm + 2 * st * TILE;
        constexpr int kBlock64 = kKeys * 128;  // bytes of 64 channels of a tile, in either layout
        uint32_t side[4] = {0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < CB; ++g) {
          const float sk = lo_bf16(ks[g]) * fk;
          const uint32_t z = high_low(fmaf(8.0f, sk, hi_bf16(ks[g]) * fk));
          side[2 * g] = __byte_perm(z, z, 0x1010), side[2 * g + 1] = __byte_perm(z, z, 0x3232);  // high, high, low, low
          const __half2 s = __float2half2_rn(sk);
          const uint32_t c[4] = {kc[g].x, kc[g].y, kc[g].z, kc[g].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(stage + at_k[j] + g * kBlock64) = expand.key(c[j], s);
        }
        *reinterpret_cast<uint4*>(sm + 6 * TILE + (2 + st) * kSide + side_chunk(16 * w + tk, half)) =
            half ? make_uint4(0, 0, 0, 0) : make_uint4(side[0], side[1], side[2], side[3]);
        const __half2 s = __float2half2_rn(lo_bf16(vs) * fv), b = __float2half2_rn(hi_bf16(vs) * fv);
#pragma unroll
        for (int g = 0; g < CB; ++g) {
          const uint32_t c[4] = {odd ? vc[g].y : vc[g].x, odd ? vc[g].x : vc[g].y, odd ? vc[g].w : vc[g].z, odd ? vc[g].z : vc[g].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(stage + at_v[j] + g * kBlock64) = expand.value(c[j], s, b);
        }
        fence_async_smem();
        bar_sync(3, 32 * kExpandWarps);
        if (w == 0 && lane == 0) mbar_arrive(&kv_full[st]);
#pragma unroll
        for (int g = 0; g < CB; ++g) kc[g] = kn[g], vc[g] = vnx[g];
#pragma unroll
        for (int g = 0; g < GK; ++g) ks[g] = ksn[g];
        vs = vsn, ok = okn;
      }
    } while (!bad && walk.next(a));
  } else {
    // ------------------------------------------------------------- products
    fewer_regs<kProductRegs>();
    if (warp == kSoftWarps + kExpandWarps) {
    const uint32_t id_s = idesc_f16(128, kKeys, false, false), id_o = idesc_f16(128, D, false, true);
    const uint64_t dq = desc_kmaj(smem_u32(sm), 128, 0), dk = desc_kmaj(smem_u32(sm) + 2 * TILE, kKeys, 0);
    const uint64_t dv = desc_mnmaj(smem_u32(sm) + 3 * TILE, kKeys, 0);
    const uint64_t dqs = desc_side(smem_u32(sm) + 6 * TILE), dks = desc_side(smem_u32(sm) + 6 * TILE + 2 * kSide);
    auto scores = [&](int x, int st) {
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint32_t off = ((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4;  // 64 channels a block of the operands
        mma_f16(tbase + 128 * x, dq + (uint32_t)((x * TILE >> 4) + off), dk + (uint32_t)((2 * st * TILE >> 4) + off), id_s, s > 0);
      }
      mma_f16(tbase + 128 * x, dqs + (uint32_t)(x * kSide >> 4), dks + (uint32_t)(st * kSide >> 4), id_s, 1u);
      mma_commit(&s_full[x]);
    };
    auto values = [&](int x, int st, bool more) {
#pragma unroll
      for (int s = 0; s < kKeys / 16; ++s)
        mma_ts(tbase + kO + D * x, tbase + 128 * x + 8 * s, dv + (uint32_t)((2 * st * TILE >> 4) + s * 128), id_o,
               more || s > 0 ? 1u : 0u);
    };
    uint32_t ph_q[2] = {0, 0}, ph_p[2] = {0, 0};
    do {
      if (!walk.piece(a)) continue;
      const int both = walk.rows_here() > 128 ? 2 : 1;
      for (int x = 0; x < both && !bad; ++x) {
        if (!mbar_wait_warp(&q_full[x], ph_q[x])) bad = true;
        ph_q[x] ^= 1;
      }
      if (!bad && !mbar_wait_warp(&kv_full[kt & 1], (kt >> 1) & 1)) bad = true;
      if (bad) break;
      fence_after();
      if (elect_one()) {
        scores(0, kt & 1);
        if (both == 2) scores(1, kt & 1);
      }
      __syncwarp();
      for (int t = walk.t0; t < walk.t1 && !bad; ++t, ++kt) {
        const bool more = t + 1 < walk.t1;
        for (int x = 0; x < both; ++x) {
          if (!mbar_wait_warp(&p_full[x], ph_p[x]) ||
              (x == 0 && more && !mbar_wait_warp(&kv_full[(kt + 1) & 1], ((kt + 1) >> 1) & 1))) {
            bad = true;
            break;
          }
          ph_p[x] ^= 1;
          fence_after();
          if (elect_one()) {
            values(x, kt & 1, t > walk.t0);
            if (x + 1 == both) mma_commit(&kv_free[kt & 1]);
            if (more) scores(x, (kt + 1) & 1);
            else mma_commit(&o_full[x]);
          }
          __syncwarp();
        }
      }
    } while (!bad && walk.next(a));
    if (elect_one()) mma_commit(&drain);  // every product issued has finished before TMEM is released
    __syncwarp();
    mbar_wait_warp(&drain, 0);
    }
  }
  if (sync_tc_any(bad) && tid == 0) set_status(a.status, kStatusWaitTimeout | (GDN_K_ATTENTION << 8));
  if (warp == kSoftWarps + kExpandWarps) tmem_dealloc(tbase, 512);
}

// A warp a row of a split group: joins the partial rows of its blocks.
template <int D>
__global__ void __launch_bounds__(256) attn_prefill_combine_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ int s_count[8 * kSplitPer], s_first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = split_group(a, blockIdx.x, s_count, &s_first);
  if (first < 0) return;
  const int4 sp = a.ws.split[first];
  const AttnRows rw = rows_of(a, sp.x);
  const int Gq = a.p.Hq / a.cache.Hkv, parts = sp.w - first + 1;
  constexpr int V = D / 32;  // channels of a lane
  for (int row = blockIdx.y * 8 + warp; row < kRows; row += gridDim.y * 8) {
    const int gr = sp.z * kRows + row;
    if (gr >= rw.rows) break;
    auto slot = [&](int i) { return (int64_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * kRows + row; };
    float m = -INFINITY, l = 0.0f, v[V];
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = 0.0f;
    for (int i = 0; i < parts; ++i) m = fmaxf(m, a.ws.ml[slot(i)].x);
#pragma unroll 2
    for (int i = 0; i < parts; ++i) {
      const float2 ml = a.ws.ml[slot(i)];
      const float f = ml.x == -INFINITY && ml.y == 0.0f ? 0.0f : exp2f(ml.x - m);
      const float2* o = reinterpret_cast<const float2*>(a.ws.o + slot(i) * D + lane * V);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        const float2 y = o[c];
        v[2 * c] = fmaf(f, y.x, v[2 * c]), v[2 * c + 1] = fmaf(f, y.y, v[2 * c + 1]);
      }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t out = (int64_t)(a.p.cu[sp.x] + gr / Gq) * a.p.Hq + sp.y * Gq + gr % Gq;
    uint32_t* d = reinterpret_cast<uint32_t*>((__nv_bfloat16*)a.p.o + out * D + lane * V);
#pragma unroll
    for (int c = 0; c < V; c += 2) d[c / 2] = bf16x2(v[c] * inv, v[c + 1] * inv);
    if (lane == 0 && a.p.lse) a.p.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <int D>
cudaError_t run(const AttnArgs& a, cudaStream_t stream) {
  constexpr int bytes = smem_bytes(D);
  cudaError_t e = cudaFuncSetAttribute(attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  {
    LaunchScope scope(GDN_K_ATTENTION, stream);
    attn_prefill_kernel<D><<<a.G, kThreads, bytes, stream>>>(a);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  LaunchScope scope(GDN_K_ATTN_COMBINE, stream);
  attn_prefill_combine_kernel<D><<<dim3((unsigned)a.G, 16), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_prefill(const AttnArgs& a, cudaStream_t stream) {
  return a.p.D == 64 ? run<64>(a, stream) : run<128>(a, stream);
}

}  // namespace gdn
