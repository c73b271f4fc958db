// Causal attention over the 4-bit paged cache for many query rows (chunked
// prefill; bf16 io), on tcgen05:
//   S = Q K^T, P = 2^(S - m) and O = P V on tiles of 128 rows x 128 keys.
//
// Operands are fp16, with powers of two over them: query rows are brought below 2^8
// (exactly, but for elements 2^-22 of the row's largest), keys and values below
// 2^12 by the largest of the piece so far.  Keys go as s (c - 8), which is exact in
// 11 bits, and the rest, b + 8 s by group, times the sums of the query's groups, as
// 16 more channels in high and low parts:
//   q . k_t = sum_g q_g . s_tg (c_tg - 8) + (b_tg + 8 s_tg) sum(q_g),
// so that scores, and the log of their sum, are those of fp32 but for 2^-32 of the
// piece's largest key, half a step below fp16's normal numbers.  (Keys as s c + b in
// fp16 put 2^-12 of a score into the log of a short row's sum.)  Values,
// s c + b, and probabilities are off by half a step of fp16, 2^-11, against 2^-8
// in bf16, at the same rate.  A value group that stands for NaN is expanded as
// zeros and noted by token, so that it reaches the rows that see it and no other.
//
// Heads of up to 128 channels: a block takes two tiles of 128 query rows (tokens x
// the heads that share a key/value head) through the same keys.  Warps 0-3 and 4-7
// are the softmax of either tile, a thread a row; eight warps expand, 16 keys each;
// one warp issues the products (three more fill its group up).  While one tile's
// softmax runs the other's products do.  S is 128 columns of TMEM, P overwrites its
// first 64 in fp16 and is the A operand of P V.  O stays in TMEM; the running maximum
// moves only when a score passes it by kSlack, and only then is O rescaled.
//
// Heads of 256: O of one tile is half of TMEM, and queries, keys and values of one
// tile are 192 KB, so a block takes one tile of rows.  Two buffers of S alternate
// from key tile to key tile: S of tile t + 1 is made while the softmax of t runs.
// Keys and values have one stage each, filled in turn: keys of t + 1 once S of t is made,
// values of t once P V of t - 1 is.
//
// Measured, 2048 tokens over 6144, 24 / 2 heads: D = 128 287 us (floor 107, by the
// products), D = 256 508 us (floor 214; 2310 with attn_kernel), D = 64 246 us.
// D = 128: a tile's chain of products, wake-ups, maximum and exponentials is longer than
// the other tile's work.
// D = 256: the chain is a tile's expansion, with shared memory half taken by operands.
// Tried there, against 487 then: two threads a row 497, the keys in two parts 515,
// sixteen warps that expand half the channels each 494, eight for keys and eight for
// values 604 (products and stores then meet in shared memory).
#include <cuda_fp16.h>

#include "attention.cuh"
#include "tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kKeys = 128;
constexpr float kFar = 1048576.0f;  // a maximum whose rounding is a score's own: 2^-4 powers of two and more
constexpr bool two_tiles(int D) { return D <= 128; }  // row tiles of a block: two, or one with two buffers of S
constexpr int rows_of_block(int D) { return prefill_rows(D); }
constexpr int soft_warps(int D) { return two_tiles(D) ? 8 : 4; }
constexpr int kExpandWarps = 8;
constexpr int threads_of(int D) { return (soft_warps(D) + kExpandWarps + 4) * 32; }
// Registers a thread after the start, heads of up to 128: 640 threads begin with 96, 61440 in all; these come to 60416.
// Heads of 256: 512 threads have 128 each and keep them.
constexpr int kSoftRegs = 128, kExpandRegs = 80, kProductRegs = 56;
static_assert((8 * kSoftRegs + kExpandWarps * kExpandRegs + 4 * kProductRegs) * 32 <= threads_of(128) * 96, "register split");
static_assert(kSoftRegs >= 96 && kExpandRegs <= 96 && kProductRegs <= 96, "setmaxnreg.inc must not lower, .dec not raise");
template <int N>
__device__ __forceinline__ void more_regs() {
  __syncwarp();
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
  __syncwarp();
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int D>
using Walk = AttnWalk<rows_of_block(D), kKeys, 3, 3>;  // a group's queries and output cost about three tiles; at least three a block (six: 64 tokens over 500 40 -> 55 us)

constexpr int tile_bytes(int D) { return kKeys * D * 2; }
constexpr int kSide = kKeys * 32;  // the 16 more channels of a tile: 32 bytes a row, 32-byte swizzle
// shared memory, in tiles: queries 0 (and 1), then stages of keys and values in turn; in sides: queries, then stages of keys
constexpr int q_tiles(int D) { return two_tiles(D) ? 2 : 1; }
constexpr int stages_of(int D) { return two_tiles(D) ? 2 : 1; }
constexpr int all_tiles(int D) { return q_tiles(D) + 2 * stages_of(D); }
constexpr int smem_bytes(int D) {  // one block an SM, which takes all of its TMEM
  return all_tiles(D) * tile_bytes(D) + 4 * kSide + 1024 < 120000 ? 120000 : all_tiles(D) * tile_bytes(D) + 4 * kSide + 1024;
}
static_assert(smem_bytes(256) <= 227 * 1024 - 2048, "shared memory of a block");
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
  float v_unit;          // the same of the values, of this tile and the piece's before
  float v_step;          // v_unit before / after this tile: O is rescaled by it
  uint32_t rare;         // some keys have no page (1), some values are NaN (2); the four are read as one uint4
  uint8_t valid[8];      // 16 keys each: they have a page
  uint16_t v_nan[2][8];  // by value group and key: its value is NaN
};

// Eight codes as values s c + b or keys s (c - 8), in the order 0 4 1 5 2 6 3 7.  Nibbles 1, 3, .. are masked into
// 1024 + 16 c, which saves their shift.  The masks sit in registers whose values the compiler does not know (a kernel argument that is 0 is in them),
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
// The TMEM accesses below are .sync.aligned and, unlike those of tc.cuh, do not reconverge the warp themselves, which would
// cost 3 % of the kernel: what only some lanes do ends with a __syncwarp() before them.
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

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(threads_of(D), 1) attn_prefill_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int GK = D / kKGroup, GV = D / v_group(D), CB = D / 64, TILE = tile_bytes(D);
  constexpr bool kTwo = two_tiles(D);
  constexpr int kSoftWarps = soft_warps(D), kThreads = threads_of(D), kRows = rows_of_block(D);
  constexpr int kKv = q_tiles(D) * TILE, kSides = all_tiles(D) * TILE;  // where stages and sides begin
  constexpr int kPSplit = kTwo ? 2 : 1;  // parts of P that are multiplied as they are written (2048 tokens over 6144: 300 -> 289 us)
  constexpr int kMeta = kTwo ? 2 : 4;  // key tiles that are spoken of at a time
  // TMEM: S of either row tile, or of either key tile in turn, at 0 and 128; O at 256 (and 256 + D).  P is in the first
  // half of its S, which is made anew only when the product that reads P is done: products of different shapes or into
  // different columns need not run in the order of their issue (the wait costs 10 of 287 us; heads of 256 were wrong without).  Heads of 64 leave columns for P apart from S, and
  // nothing waits.
  constexpr uint32_t kO = 256;
  constexpr bool kPApart = D == 64;
  constexpr uint32_t kP = kPApart ? kO + 2 * D : 0, kPStep = kPApart ? 64 : 128;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  // two row tiles: q, s, p, o by row tile, kv by stage.  One: s and p by key tile, kv_full of the keys and of the values,
  // o_full[0] of every key tile, o_full[1] of a piece's last.
  __shared__ uint64_t q_full[2], s_full[2], p_full[kPSplit][2], o_full[2], kv_full[2], kv_free[2], drain;
  __shared__ Meta meta[kMeta];
  __shared__ uint2 s_top[kExpandWarps];
  __shared__ int64_t s_warp[kThreads / 32], s_found[4];
  __shared__ uint32_t tslot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnProblem& p = a.p;
  const int Gq = p.Hq / a.cache.Hkv;

  Walk<D> walk;
  if (!walk.start(a, kThreads, s_warp, s_found)) return;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      for (int j = 0; j < kPSplit; ++j) mbar_init(&p_full[j][i], 4);
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
  int kt = 0;  // key tiles before this one, over all pieces

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    if constexpr (kTwo) more_regs<kSoftRegs>();
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;  // row tile, row
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tbase + lanes + kO + D * x;
    unsigned char* sq = sm + x * TILE;
    const float c_log2 = fabsf(p.scale) * kLog2e;
    uint32_t ph_s = 0, o_done = 0;  // o_done: phases of the o_full that ends a piece
    bool late = false;  // a wait of this warp alone ran out
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
        uint32_t side[8] = {};  // high, low, high, low by group
#pragma unroll
        for (int g = 0; g < GK; ++g) side[2 * g] = side[2 * g + 1] = high_low(sum[g]);
        unsigned char* row_side = sm + kSides + x * kSide;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<uint4*>(row_side + side_chunk(r, i)) =
              make_uint4(side[4 * i], side[4 * i + 1], side[4 * i + 2], side[4 * i + 3]);
        fence_async_smem();
        __syncwarp();
        mbar_arrive_if(&q_full[x], lane == 0);
      }
      float m = -INFINITY, l = 0.0f, v_unit = 1.0f;
      bool nan[GV] = {};
      auto p_done = [&](uint64_t* full) {  // what this warp has written of P may be multiplied
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before();
        __syncwarp();
        mbar_arrive_if(full, lane == 0);
      };
      for (int t = walk.t0; t < walk.t1; ++t, ++kt) {
        const int buf = kTwo ? x : kt & 1;
        const uint32_t ts = tbase + lanes + 128 * buf, tp = tbase + lanes + kP + kPStep * buf;
        if (!group_wait(1 + x, 128, (warp & 3) == 0, &s_full[buf], kTwo ? ph_s : (uint32_t)(kt >> 1) & 1u, nullptr, 0)) {
          bad = true;
          break;
        }
        ph_s ^= 1;
        fence_after();
        const Meta& mt = meta[kt % kMeta];
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
#pragma unroll
            for (int g = 0; g < GV; ++g) nan[g] |= (mt.v_nan[g][i] & (k >= 16 ? 0xffffu : k <= 0 ? 0u : (1u << k) - 1u)) != 0;
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
            __syncwarp();
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) top = fmaxf(top, fmaxf(__uint_as_float(cur[e]), __uint_as_float(cur[e + 1])));
        }
        top = top == -INFINITY ? top : top * f;
        if (__any_sync(0xffffffffu, top > m + kSlack || v_step != 1.0f || fabsf(m) >= kFar)) {
          const float m2 = fmaxf(m, top), g = m2 == m ? 1.0f : ex2(m - m2);
          m = m2;
          l *= g;
          if (t > walk.t0) {
            // the product of the last tile is done: S came after it.  With one row tile S came before, and O is waited for.
            if constexpr (!kTwo) {
              late |= !mbar_wait_warp(&o_full[0], (uint32_t)(kt - 1) & 1u);
              fence_after();
            }
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
          // S f - m in one step keeps what the rounding of m left out.  That is the same for all keys of the row, and nothing
          // beside scores of a few powers of two, but past the exponents' range where m is: from kFar on products are rounded
          // as m was.
          if (__any_sync(0xffffffffu, fabsf(m) >= kFar && m != -INFINITY)) {
            ld_wait(raw[0]);
            const float base = m == -INFINITY ? 0.0f : -m;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float z[16];
              uint32_t w[8];
              tmem_ld16(ts + 16 * c, z);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                float v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  v[i] = seen(16 * c + e + i) ? ex2(__fadd_rn(__fmul_rn(z[e + i], f), base)) : 0.0f;
                  l += v[i];
                }
                const __half2 h = __floats2half2_rn(v[0], v[1]);
                w[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
              }
              __syncwarp();
              tmem_st8(tp + 8 * c, w);
              if (c % (8 / kPSplit) == 8 / kPSplit - 1) p_done(&p_full[c / (8 / kPSplit)][buf]);
            }
            continue;
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
          tmem_st16(tp + 16 * c, w);
          if (c % (4 / kPSplit) == 4 / kPSplit - 1) p_done(&p_full[c / (4 / kPSplit)][buf]);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // The products of the piece are done.  A parity tells a phase from the one before it only: with two row tiles the
      // last S followed the product before the last (heads of 64: one phase a piece).  With one row tile it followed the
      // product before that, whose successor may still run, and o_full[0] would pass for it; waiting for both phases in
      // turn could miss the first, which the second may overtake once the last P is out.  So the last product of a piece
      // completes o_full[1], one phase a piece, none of them passed over.
      o_done += kTwo && !kPApart ? tiles : 1;
      if (bad || !group_wait(1 + x, 128, (warp & 3) == 0, &o_full[kTwo ? x : 1], (o_done - 1) & 1u, nullptr, 0)) {
        bad = true;
        break;
      }
      fence_after();
      // rows out: whole, or unnormalised to the workspace
      const bool from_start = walk.t0 == 0, to_end = walk.t1 == walk.tiles;
      const bool is_whole = from_start && to_end;
      const int64_t out = (int64_t)tok * p.Hq + head;
      const int64_t slot = ((int64_t)(2 * blockIdx.x + (from_start ? 1 : 0)) * kRows + x * 128 + r);
      const float f_row = is_whole ? (l == 0.0f ? 0.0f : v_unit / l) : v_unit;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        const float f = (GV > 1 && c0 >= v_group(D) ? nan[GV - 1] : nan[0]) ? __int_as_float(0x7fc00000) : f_row;
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
    bad |= late;
  } else if (warp < kSoftWarps + kExpandWarps) {
    // ------------------------------------------------------------- expansion
    if constexpr (kTwo) fewer_regs<kExpandRegs>();
    const int w = warp - kSoftWarps, half = lane & 1, tk = lane >> 1;  // 16 keys a warp
    constexpr int kGroup = 32 * kExpandWarps, kBar = 3;
    const int tv = (tk & 8) | ((tk & 3) << 1) | ((tk >> 2) & 1);  // the token of V row tk (v_row's inverse)
    const Expand expand(a.zero);
    constexpr int kBlock64 = kKeys * 128;  // bytes of 64 channels of a tile, in either layout
    // where this lane's four chunks of 64 channels go, of keys and of values
    const bool odd = (tv >> 2) & 1;  // pairs of words in turn: the eight lanes of a store then hit all banks
    uint32_t at_k[4], at_v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      at_k[j] = kKv + kmaj_chunk(kKeys, 16 * w + tk, (half * 4 + j) * 8);
      at_v[j] = kKv + TILE + mnmaj_chunk(kKeys, 16 * w + tv, (half * 4 + (j ^ (odd ? 1 : 0))) * 8);
    }
    do {
      if (!walk.piece(a)) continue;
      const int n = walk.n, h = walk.h;
      // References: exponents of the piece's largest values so far, what they hold, and their scales.  They begin anew with
      // every piece, or one request's magnitudes would leave the next one's values no bits.
      int k_ref = -100, v_ref = -100;
      float k_lim = -1.0f, v_lim = -1.0f, fk = 0.0f, fv = 0.0f;
      const int all = max(0, min(walk.rw.first + (walk.rt * kRows + walk.rows_here() - 1) / Gq, walk.rw.cap));  // keys anybody sees
      int64_t place = -1;
      // Where this warp's 16 keys of tile t are, -1: nowhere.  Every 32 tiles lane j looks the j-th of them up.
      auto find = [&](int t) {
        if ((t - walk.t0) % 32 == 0) {
          const int pos = (t + lane) * kKeys + 16 * w;
          place = -1;
          if (t + lane < walk.t1 && pos < all) {
            place = kv_tile_at(a.cache, D, n, pos, h);
            if (place < 0) set_status(a.status, kStatusBadPage | (GDN_K_ATTENTION << 8));
          }
        }
        return __shfl_sync(0xffffffffu, place, (t - walk.t0) % 32);
      };
      auto load_codes = [&](int64_t at, int off, uint4 (&c)[CB]) {
        const unsigned char* from = a.cache.pool + at + off + lane * 16;
#pragma unroll
        for (int g = 0; g < CB; ++g) c[g] = at >= 0 ? *reinterpret_cast<const uint4*>(from + g * 512) : make_uint4(0, 0, 0, 0);
      };
      auto load_scales = [&](int t, int64_t at, uint32_t (&sk)[GK], uint32_t (&sv)[GV], bool& there) {
        const int pos = t * kKeys + 16 * w;
        there = at >= 0 || pos >= all;
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(a.cache.pool + at + kv_scale_off(D));
        const bool see_k = pos + tk < all, see_v = pos + tv < all;  // behind the last key they may be anything
#pragma unroll
        for (int g = 0; g < GK; ++g) {
          const uint32_t v = at >= 0 ? sc[g * kKvTile + tk] : 0;
          sk[g] = see_k ? v : 0;
        }
#pragma unroll
        for (int g = 0; g < GV; ++g) {
          const uint32_t v = at >= 0 ? sc[(GK + g) * kKvTile + tv] : 0;
          sv[g] = see_v ? v : 0;
        }
      };
      // Brings the references up to a tile's keys and values and fills mt; false: a wait ran out (a warp passes waited =
      // false).  Mostly the tile stays within the references and is finite, and every key has a page: one barrier says
      // so, which the wait for the stage needs anyway.  A value that is NaN gets the scale 0.
      auto agree = [&](Meta& mt, bool waited, const uint32_t (&ks)[GK], uint32_t (&vs)[GV], bool ok) {
        float rk = 0.0f, rv = 0.0f;
        bool odd_k = false, odd_v = false;
#pragma unroll
        for (int g = 0; g < GK; ++g) rk = fmaxf(rk, reach(ks[g])), odd_k |= !finite_word(ks[g]);
#pragma unroll
        for (int g = 0; g < GV; ++g) rv = fmaxf(rv, reach(vs[g])), odd_v |= !finite_word(vs[g]);
        const bool plain = rk <= k_lim && rv <= v_lim && !odd_k && !odd_v && ok;
        if (bar_or(kBar, kGroup, !plain || !waited)) {
          // the rest of it: whether the wait ran out, the tile's largest finite key and value, what is odd
          uint32_t top_k = 0, top_v = 0, nans[GV];
          bool any = false;
#pragma unroll
          for (int g = 0; g < GK; ++g)
            if (finite_word(ks[g])) top_k = max(top_k, __float_as_uint(reach(ks[g])));
#pragma unroll
          for (int g = 0; g < GV; ++g) {
            const bool v_bad = !finite_word(vs[g]);
            if (v_bad) vs[g] = 0;
            else top_v = max(top_v, __float_as_uint(reach(vs[g])));
            nans[g] = __reduce_or_sync(0xffffffffu, v_bad ? 1u << tv : 0u);
            any |= nans[g] != 0;
          }
          top_k = __reduce_max_sync(0xffffffffu, top_k);
          top_v = __reduce_max_sync(0xffffffffu, top_v);
          if (lane == 0) {
            s_top[w] = make_uint2(top_k, top_v);
            mt.valid[w] = ok ? 1 : 0;
#pragma unroll
            for (int g = 0; g < GV; ++g) mt.v_nan[g][w] = (uint16_t)nans[g];
          }
          __syncwarp();
          if (bar_or(kBar, kGroup, !waited)) return false;
          const bool no_page = bar_or(kBar, kGroup, !ok), any_nan = bar_or(kBar, kGroup, any);
#pragma unroll
          for (int i = 0; i < 8; ++i) top_k = max(top_k, s_top[i].x), top_v = max(top_v, s_top[i].y);
          // a larger exponent than all before moves the reference, by three more
          const int ek = exponent(min(top_k, 0x7f7fffffu)), ev = exponent(min(top_v, 0x7f7fffffu)), v_old = v_ref;
          if (ek > k_ref) k_ref = min(ek + 3, 127);
          if (ev > v_ref) v_ref = min(ev + 3, 127);
          fk = pow2(11 - k_ref), fv = pow2(11 - v_ref);
          k_lim = k_ref >= 127 ? 3.0e38f : pow2(k_ref + 1) * 0.99f, v_lim = v_ref >= 127 ? 3.0e38f : pow2(v_ref + 1) * 0.99f;
          if (w == 0 && lane == 0) {
            mt.v_step = v_old == v_ref ? 1.0f : exp2f((float)(v_old - v_ref));
            mt.rare = (no_page ? 1u : 0u) | (any_nan ? 2u : 0u);
          }
          __syncwarp();
          bar_sync(kBar, kGroup);  // s_top is read
        } else if (w == 0 && lane == 0) {
          mt.v_step = 1.0f, mt.rare = 0;
        }
        if (w == 0) {
          if (lane == 0) mt.k_unit = pow2(k_ref - 11), mt.v_unit = pow2(v_ref - 11);
          __syncwarp();
        }
        return true;
      };
      auto put_keys = [&](int st, const uint4 (&kc)[CB], const uint32_t (&ks)[GK]) {
#pragma unroll
        for (int g = 0; g < CB; ++g) {
          const __half2 s = __float2half2_rn(lo_bf16(ks[g]) * fk);
          const uint32_t c[4] = {kc[g].x, kc[g].y, kc[g].z, kc[g].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(sm + 2 * st * TILE + at_k[j] + g * kBlock64) = expand.key(c[j], s);
        }
        uint32_t side[8] = {};
#pragma unroll
        for (int g = 0; g < GK; ++g) {
          const uint32_t z = high_low(fmaf(8.0f, lo_bf16(ks[g]) * fk, hi_bf16(ks[g]) * fk));
          side[2 * g] = __byte_perm(z, z, 0x1010), side[2 * g + 1] = __byte_perm(z, z, 0x3232);  // high, high, low, low
        }
        *reinterpret_cast<uint4*>(sm + kSides + (q_tiles(D) + st) * kSide + side_chunk(16 * w + tk, half)) =
            half ? make_uint4(side[4], side[5], side[6], side[7]) : make_uint4(side[0], side[1], side[2], side[3]);
      };
      auto put_values = [&](int st, const uint4 (&vc)[CB], const __half2 (&s)[GV], const __half2 (&b)[GV]) {
#pragma unroll
        for (int g = 0; g < CB; ++g) {
          const uint32_t c[4] = {odd ? vc[g].y : vc[g].x, odd ? vc[g].x : vc[g].y, odd ? vc[g].w : vc[g].z, odd ? vc[g].z : vc[g].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(sm + 2 * st * TILE + at_v[j] + g * kBlock64) = expand.value(c[j], s[g * GV / CB], b[g * GV / CB]);
        }
      };
      auto value_scales = [&](const uint32_t (&vs)[GV], __half2 (&s)[GV], __half2 (&b)[GV]) {
#pragma unroll
        for (int g = 0; g < GV; ++g) s[g] = __float2half2_rn(lo_bf16(vs[g]) * fv), b[g] = __float2half2_rn(hi_bf16(vs[g]) * fv);
      };
      auto full = [&](uint64_t* m) {  // what the warps have written may be read
        fence_async_smem();
        bar_sync(kBar, kGroup);
        if (w == 0) mbar_arrive_if(m, lane == 0);
      };
      uint4 kc[CB], vc[CB], kn[CB], vnx[CB];
      uint32_t ks[GK], vs[GV], ksn[GK], vsn[GV];
      __half2 v_s[GV], v_b[GV];
      bool ok, okn;
      int64_t at = find(walk.t0);
      load_codes(at, 0, kc);
      load_scales(walk.t0, at, ks, vs, ok);
      if constexpr (kTwo) {
        load_codes(at, kv_v_off(D), vc);
        for (int t = walk.t0; t < walk.t1; ++t, ++kt) {
          if (t + 1 < walk.t1) {
            at = find(t + 1);
            load_codes(at, 0, kn);
            load_codes(at, kv_v_off(D), vnx);
            load_scales(t + 1, at, ksn, vsn, okn);
          }
          const int st = kt & 1;
          bool waited = true;
          if (kt >= 2 && w == 0) waited = mbar_wait_warp(&kv_free[st], ((kt >> 1) & 1) ^ 1);
          if (!agree(meta[kt % kMeta], waited, ks, vs, ok)) {
            bad = true;
            break;
          }
          value_scales(vs, v_s, v_b);
          put_keys(st, kc, ks);
          put_values(st, vc, v_s, v_b);
          full(&kv_full[st]);
#pragma unroll
          for (int g = 0; g < CB; ++g) kc[g] = kn[g], vc[g] = vnx[g];
#pragma unroll
          for (int g = 0; g < GK; ++g) ks[g] = ksn[g];
#pragma unroll
          for (int g = 0; g < GV; ++g) vs[g] = vsn[g];
          ok = okn;
        }
      } else {
        // Keys of tile t, then values of tile t - 1 (kt: of tile t).  The waits say that the products which read the
        // last ones are done: S of the tile before, O of the tile before.
        for (int t = walk.t0; t <= walk.t1; ++t) {
          const int64_t at_here = at;
          if (t + 1 < walk.t1) {
            at = find(t + 1);
            load_codes(at, 0, kn);
            load_scales(t + 1, at, ksn, vsn, okn);
          }
          if (t < walk.t1) load_codes(at_here, kv_v_off(D), vnx);
          __half2 s_next[GV], b_next[GV];
          if (t < walk.t1) {
            bool waited = true;
            if (kt >= 1 && w == 0) waited = mbar_wait_warp(&s_full[(kt - 1) & 1], (uint32_t)((kt - 1) >> 1) & 1u);
            if (!agree(meta[kt % kMeta], waited, ks, vs, ok)) {
              bad = true;
              break;
            }
            value_scales(vs, s_next, b_next);
            put_keys(0, kc, ks);
            full(&kv_full[0]);
          }
          if (t > walk.t0) {
            if (kt >= 2 && !group_wait(kBar, kGroup, w == 0, &o_full[0], (uint32_t)(kt - 2) & 1u, nullptr, 0)) {
              bad = true;
              break;
            }
            put_values(0, vc, v_s, v_b);
            full(&kv_full[1]);
          }
          if (t == walk.t1) break;
          ++kt;
#pragma unroll
          for (int g = 0; g < CB; ++g) kc[g] = kn[g], vc[g] = vnx[g];
#pragma unroll
          for (int g = 0; g < GK; ++g) ks[g] = ksn[g];
#pragma unroll
          for (int g = 0; g < GV; ++g) vs[g] = vsn[g], v_s[g] = s_next[g], v_b[g] = b_next[g];
          ok = okn;
        }
      }
    } while (!bad && walk.next(a));
  } else {
    // ------------------------------------------------------------- products
    if constexpr (kTwo) fewer_regs<kProductRegs>();
    if (warp == kSoftWarps + kExpandWarps) {
    const uint32_t id_s = idesc_f16(128, kKeys, false, false), id_o = idesc_f16(128, D, false, true);
    const uint64_t dq = desc_kmaj(smem_u32(sm), 128, 0), dk = desc_kmaj(smem_u32(sm) + kKv, kKeys, 0);
    const uint64_t dv = desc_mnmaj(smem_u32(sm) + kKv + TILE, kKeys, 0);
    const uint64_t dqs = desc_side(smem_u32(sm) + kSides), dks = desc_side(smem_u32(sm) + kSides + q_tiles(D) * kSide);
    auto scores = [&](int x, int st, int buf) {  // row tile, stage, buffer of S
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint32_t off = ((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4;  // 64 channels a block of the operands
        mma_f16(tbase + 128 * buf, dq + (uint32_t)((x * TILE >> 4) + off), dk + (uint32_t)((2 * st * TILE >> 4) + off), id_s, s > 0);
      }
      mma_f16(tbase + 128 * buf, dqs + (uint32_t)(x * kSide >> 4), dks + (uint32_t)(st * kSide >> 4), id_s, 1u);
      mma_commit(&s_full[buf]);
    };
    auto values = [&](int x, int st, int buf, bool more, int part) {
#pragma unroll
      for (int s = part * (8 / kPSplit); s < (part + 1) * (8 / kPSplit); ++s)
        mma_ts(tbase + kO + D * x, tbase + kP + kPStep * buf + 8 * s, dv + (uint32_t)((2 * st * TILE >> 4) + s * 128), id_o,
               more || s > 0 ? 1u : 0u);
    };
    uint32_t ph_q[2] = {0, 0}, ph_p[2] = {0, 0}, ph_o[2] = {0, 0};
    do {
      if (!walk.piece(a)) continue;
      if constexpr (kTwo) {
        const int both = walk.rows_here() > 128 ? 2 : 1;
        for (int x = 0; x < both && !bad; ++x) {
          if (!mbar_wait_warp(&q_full[x], ph_q[x])) bad = true;
          ph_q[x] ^= 1;
        }
        if (!bad && !mbar_wait_warp(&kv_full[kt & 1], (kt >> 1) & 1)) bad = true;
        if (bad) break;
        fence_after();
        if (elect_one()) {
          scores(0, kt & 1, 0);
          if (both == 2) scores(1, kt & 1, 1);
        }
        __syncwarp();
        for (int t = walk.t0; t < walk.t1 && !bad; ++t, ++kt) {
          const bool more = t + 1 < walk.t1;
          for (int x = 0; x < both; ++x) {
#pragma unroll
            for (int j = 0; j < kPSplit - 1; ++j) {
              bad = bad || !mbar_wait_warp(&p_full[j][x], ph_p[x]);
              if (bad) break;
              fence_after();
              if (elect_one()) values(x, kt & 1, x, t > walk.t0, j);
              __syncwarp();
            }
            if (bad || !mbar_wait_warp(&p_full[kPSplit - 1][x], ph_p[x]) ||
                (x == 0 && more && !mbar_wait_warp(&kv_full[(kt + 1) & 1], ((kt + 1) >> 1) & 1))) {
              bad = true;
              break;
            }
            ph_p[x] ^= 1;
            fence_after();
            if (elect_one()) {
              values(x, kt & 1, x, t > walk.t0, kPSplit - 1);
              if (x + 1 == both) mma_commit(&kv_free[kt & 1]);
              if (kPApart && more) scores(x, (kt + 1) & 1, x);
              if (!kPApart || !more) mma_commit(&o_full[x]);
            }
            __syncwarp();
            if (!kPApart && more) {
              if (!mbar_wait_warp(&o_full[x], ph_o[x])) {
                bad = true;
                break;
              }
              fence_after();
              if (elect_one()) scores(x, (kt + 1) & 1, x);
              __syncwarp();
            }
            if (!kPApart || !more) ph_o[x] ^= 1;
          }
        }
      } else {
        // S of two tiles ahead of the probabilities; a buffer is made anew once the product that reads P there is done
        auto next_scores = [&](int k) {  // of key tile k (over all pieces)
          if (!mbar_wait_warp(&kv_full[0], (uint32_t)k & 1u)) return false;
          fence_after();
          if (elect_one()) scores(0, 0, k & 1);
          __syncwarp();
          return true;
        };
        bad = !mbar_wait_warp(&q_full[0], ph_q[0]);
        ph_q[0] ^= 1;
        bad = bad || !next_scores(kt) || (walk.t0 + 1 < walk.t1 && !next_scores(kt + 1));
        for (int t = walk.t0; t < walk.t1 && !bad; ++t, ++kt) {
          if (!mbar_wait_warp(&p_full[0][kt & 1], (uint32_t)(kt >> 1) & 1u) || !mbar_wait_warp(&kv_full[1], (uint32_t)kt & 1u)) {
            bad = true;
            break;
          }
          fence_after();
          if (elect_one()) {
            values(0, 0, kt & 1, t > walk.t0, 0);
            mma_commit(&o_full[0]);
            if (t + 1 == walk.t1) mma_commit(&o_full[1]);
          }
          __syncwarp();
          if (t + 2 < walk.t1) bad = !mbar_wait_warp(&o_full[0], (uint32_t)kt & 1u) || !next_scores(kt + 2);
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
  constexpr int V = D / 32, kRows = rows_of_block(D);  // channels of a lane
  constexpr int kParts = (kAttnSms + 31) / 32;         // parts of a lane
  for (int row = blockIdx.y * 8 + warp; row < kRows; row += gridDim.y * 8) {
    const int gr = sp.z * kRows + row;
    if (gr >= rw.rows) break;
    auto slot = [&](int i) { return (int64_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * kRows + row; };
    // the weights 2^(m_i - m) of all parts first, a part a lane, so that the loads of the rows do not wait on one another
    // (24 tokens over 20000, 16 / 2 heads of 256: 69 -> 56 us)
    float2 ml[kParts];
    float m = -INFINITY, l = 0.0f, v[V];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const int i = 32 * k + lane;
      ml[k] = i < parts ? a.ws.ml[slot(i)] : make_float2(-INFINITY, 0.0f);
      m = fmaxf(m, ml[k].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      ml[k].x = ml[k].x == -INFINITY && ml[k].y == 0.0f ? 0.0f : exp2f(ml[k].x - m);
      l = fmaf(ml[k].x, ml[k].y, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = 0.0f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const int here = min(32, parts - 32 * k);
#pragma unroll 8
      for (int i = 0; i < here; ++i) {
        const float f = __shfl_sync(0xffffffffu, ml[k].x, i);
        const float2* o = reinterpret_cast<const float2*>(a.ws.o + slot(32 * k + i) * D + lane * V);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
          const float2 y = o[c];
          v[2 * c] = fmaf(f, y.x, v[2 * c]), v[2 * c + 1] = fmaf(f, y.y, v[2 * c + 1]);
        }
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
    attn_prefill_kernel<D><<<a.G, threads_of(D), bytes, stream>>>(a);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  LaunchScope scope(GDN_K_ATTN_COMBINE, stream);
  attn_prefill_combine_kernel<D><<<dim3((unsigned)a.G, 16), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_prefill(const AttnArgs& a, cudaStream_t stream) {
  return a.p.D == 64 ? run<64>(a, stream) : a.p.D == 128 ? run<128>(a, stream) : run<256>(a, stream);
}

}  // namespace gdn
