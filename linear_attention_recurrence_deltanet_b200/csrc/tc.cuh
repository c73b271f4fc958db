// sm_100a primitives: tcgen05 MMA / TMEM, TMA tensor loads, mbarriers, and
// the shared-memory operand layouts the MMAs read.
//
// Operand layouts (fp16 elements, 128-byte swizzle; every tile base is
// 1024-byte aligned):
//   K-major tile of R rows x K (K a multiple of 64): K-blocks of 64 elements
//     are stored one after another (R*128 bytes each); inside a block, 8-row
//     groups are 1024 bytes apart, rows 128 bytes apart, and the 16-byte
//     chunk index is XORed with (row % 8).
//     Descriptor: LBO 16 B (unused), SBO 1024 B; an MMA step of K=16 starts
//     32 bytes further inside the block.
//   MN-major tile of K rows x N (N contiguous, N a multiple of 64): N-blocks
//     of 64 elements, each holding K/8 groups of 8 rows x 128 bytes (1024 B),
//     same 16-byte-chunk swizzle with (k % 8).
//     Descriptor: LBO = stride between N-blocks = (K/8)*1024 B, SBO 1024 B;
//     an MMA step of K=16 starts 2048 bytes further.
// Accumulators (fp32 in TMEM): M=128 puts row r in lane r; M=64 puts row r in
// lane (r % 16) + 32*(r / 16).  Column c of the accumulator is TMEM column
// base + c.  Warp w may only touch lanes 32*(w % 4) .. 32*(w % 4) + 31.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace gdn {
namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// byte offset of element (row, k) in a K-major SW128 tile with `rows` rows
__host__ __device__ __forceinline__ uint32_t kmaj(int rows, int row, int k) {
  return (uint32_t)((k >> 6) * (rows * 128) + (row >> 3) * 1024 + (row & 7) * 128 + ((((k & 63) >> 3) ^ (row & 7)) << 4) +
                    (k & 7) * 2);
}
// byte offset of the 16-byte chunk holding elements (row, k..k+7), k % 8 == 0
__host__ __device__ __forceinline__ uint32_t kmaj_chunk(int rows, int row, int k) {
  return (uint32_t)((k >> 6) * (rows * 128) + (row >> 3) * 1024 + (row & 7) * 128 + ((((k & 63) >> 3) ^ (row & 7)) << 4));
}
// byte offset of element (k, n) in an MN-major SW128 tile with K rows
__host__ __device__ __forceinline__ uint32_t mnmaj(int K, int k, int n) {
  return (uint32_t)((n >> 6) * ((K >> 3) * 1024) + (k >> 3) * 1024 + (k & 7) * 128 + ((((n & 63) >> 3) ^ (k & 7)) << 4) +
                    (n & 7) * 2);
}
__host__ __device__ __forceinline__ uint32_t mnmaj_chunk(int K, int k, int n) {
  return (uint32_t)((n >> 6) * ((K >> 3) * 1024) + (k >> 3) * 1024 + (k & 7) * 128 + ((((n & 63) >> 3) ^ (k & 7)) << 4));
}

// shared-memory matrix descriptor: SW128, version 1
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46) | (2ull << 61);
}
// descriptor of MMA step s (K = 16 elements per step) of a K-major tile with `rows` rows
__device__ __forceinline__ uint64_t desc_kmaj(uint32_t base, int rows, int s) {
  const int k0 = s * 16;
  return sdesc(base + (k0 >> 6) * (rows * 128) + (k0 & 63) * 2, 16, 1024);
}
// descriptor of MMA step s of an MN-major tile with K rows
__device__ __forceinline__ uint64_t desc_mnmaj(uint32_t base, int K, int s) {
  return sdesc(base + s * 2048, (K >> 3) * 1024, 1024);
}

// instruction descriptor, kind::f16: fp16 A and B, fp32 accumulator
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// The upper half of a descriptor with a 128-byte swizzle and 1024 bytes between 8-row groups; address and leading offset are
// the lower one.
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_commit(uint64_t* mbar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(mbar))
               : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// generic-proxy shared-memory writes -> visible to the tensor core (async proxy)
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// the same for every state space (e.g. generic global writes read back by a bulk copy)
__device__ __forceinline__ void fence_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// The tcgen05 alloc / dealloc / ld / st instructions are .sync.aligned: every lane
// of the warp must execute them together.  Each helper first reconverges the
// warp, since callers reach them after lane-dependent work (a lane that issued
// and then waits for bulk copies, rows that only some lanes own).
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t ncols) {
  __syncwarp();
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  __syncwarp();
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// 32 consecutive fp32 columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 consecutive fp32 columns of this thread's lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// store 32 consecutive fp32 columns of this thread's lane
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])),
      "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])), "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])),
      "r"(__float_as_uint(v[20])), "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
      "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])), "r"(__float_as_uint(v[27])),
      "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])), "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mbar_init(uint64_t* m, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(m)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_expect_tx(uint64_t* m, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(m)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* m, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(m)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Wait for phase `parity` of `m`, for at most `limit_ns`; false on timeout.
__device__ __forceinline__ bool mbar_wait(uint64_t* m, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(m, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(m, parity)) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}

// The wait of a whole warp, all lanes together: true for all lanes or for none.  A converged warp is suspended in the
// instruction until the phase ends (about 110 cycles from the arrival) or something else arrives, 3900 cycles at most; a
// lane that polls alone is not, and its polls take the issue slots of the warps that work.  For the same reason the limit
// counts tries, the loop's cheapest measure: 20 to 3900 cycles each, so kWaitTries are 40 ms at least, some seconds at most.
constexpr int kWaitTries = 1 << 22;
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* m, uint32_t parity, int tries = kWaitTries) {
  bool ok = mbar_try_wait(m, parity);
  while (!ok && --tries > 0) ok = mbar_try_wait(m, parity);
  return __all_sync(0xffffffffu, ok);
}

// Named barriers of n threads, aligned like the instructions above: whole warps, converged (a branch that only some lanes
// take is closed by __syncwarp() before them).  bar_or: whether any thread passed true.
__device__ __forceinline__ bool bar_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, %2, %3, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// A group of warps (n threads, barrier id) waits for up to two mbarriers: one warp polls, the others wait at the barrier.
// An arrival at any mbarrier wakes every warp that polls one; with 20 of them polling, their tries took more issue
// slots than the work (the 4-bit product of 2048 rows).  True for all threads or for none.
__device__ __forceinline__ bool group_wait(int id, int n, bool polls, uint64_t* m0, uint32_t p0, uint64_t* m1, uint32_t p1) {
  bool ok = true;
  if (polls) ok = mbar_wait_warp(m0, p0) && (!m1 || mbar_wait_warp(m1, p1));
  return !bar_or(id, n, !ok);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(m)) : "memory");
}

// The arrival of the threads that pass true, without a branch: the warp stays converged for an aligned instruction behind it.
__device__ __forceinline__ void mbar_arrive_if(uint64_t* m, bool v) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %1, 0;\n@p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_u32(m)),
               "r"((uint32_t)v)
               : "memory");
}

// True in one lane of a converged warp.  Branching on it (rather than on a lane number) lets the compiler keep the
// operands of tcgen05 and bulk-copy instructions in uniform registers without a loop over the lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// ---------------------------------------------------------------- TMA
// 1D bulk copy global -> shared (both 16-byte aligned, size a multiple of 16),
// completing `bytes` on mbarrier m.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* m) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"((uint64_t)src), "r"(bytes), "r"(smem_u32(m))
               : "memory");
}

// 1D bulk copy shared -> global (both 16-byte aligned, size a multiple of 16)
// in the issuing thread's bulk async-group; bulk_commit closes the group,
// bulk_wait_read<N> waits until at most N groups still read shared memory and
// bulk_wait<N> until at most N groups are incomplete.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"((uint64_t)dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}

// 16-byte asynchronous copy global -> shared through the load/store path (L2
// only); src_bytes = 0 fills the 16 bytes with zeros and reads nothing
__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"((uint64_t)src),
               "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// L2 prefetch of `bytes` (a multiple of 16) at a 16-byte aligned global address
__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"((uint64_t)src), "r"(bytes) : "memory");
}

// 2D tiled load of the box at (x = inner coordinate, y = row) into shared memory,
// completing `bytes` on mbarrier m (no multicast).
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* m) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(smem_u32(m))
      : "memory");
}

// ---------------------------------------------------------------- operand packing
// four / eight fp32 values -> fp16, one 8- / 16-byte store
__device__ __forceinline__ void st8(unsigned char* p, float a, float b, float c, float d) {
  __half2 h0 = __floats2half2_rn(a, b), h1 = __floats2half2_rn(c, d);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&h0);
  u.y = *reinterpret_cast<uint32_t*>(&h1);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ uint4 pack8h(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void st16h(unsigned char* p, const float* v) { *reinterpret_cast<uint4*>(p) = pack8h(v); }

// SiLU(y) = y / (1 + e^-y) with the fast exponential and division
__device__ __forceinline__ float silu_fast(float y) { return __fdividef(y, 1.0f + __expf(-y)); }

// block barrier that orders tcgen05 operations before / after it
__device__ __forceinline__ void sync_tc() {
  fence_before();
  __syncthreads();
  fence_after();
}
// the same barrier, returning whether any thread of the block passed `pred` true
// (a block-uniform decision, taken in the barrier itself)
__device__ __forceinline__ bool sync_tc_any(bool pred) {
  fence_before();
  const int r = __syncthreads_or(pred ? 1 : 0);
  fence_after();
  return r != 0;
}

// ---------------------------------------------------------------- thread-block clusters
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the shared::cluster address of this CTA's shared variable at `saddr` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t mapa_shared(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// store to another CTA of the cluster that completes 4 bytes of transaction on its mbarrier `cmbar`
__device__ __forceinline__ void st_async_f32(uint32_t caddr, float v, uint32_t cmbar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(caddr), "f"(v),
               "r"(cmbar)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* m, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, "
      "p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(m)), "r"(parity)
      : "memory");
  return ok != 0;
}
// as mbar_wait, with cluster-scope acquire (the arrivals come from another CTA)
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* m, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait_cluster(m, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_cluster(m, parity)) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}
// every thread of every CTA of the cluster; also a block barrier
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace tc
}  // namespace gdn
