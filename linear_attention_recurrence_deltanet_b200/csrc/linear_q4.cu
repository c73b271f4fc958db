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
//   scales  [N / 16 tiles][groups / 4][16 rows][4] words, scale low, bias high
#include "../../include/gdn.h"
#include "internal.h"
#include "vec.cuh"

namespace gdn {
namespace {

constexpr int kTile = 16, kBlock = 64;

__global__ void q4_pack_kernel(const unsigned char* __restrict__ codes, const unsigned short* __restrict__ scales,
                               const unsigned short* __restrict__ biases, int N, int K, int group, int64_t row_bytes,
                               Q4Layout L, uint32_t* __restrict__ out) {
  const int64_t words = (int64_t)L.total_bytes / 4, scale_words = (int64_t)L.scale_off / 4;
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
      const int64_t j = i - scale_words, g4 = (L.groups + 3) / 4;
      const int in = (int)(j % 64);
      const int64_t n = j / 64 / g4 * kTile + in / 4, g = j / 64 % g4 * 4 + (in & 3);
      if (n < N && g < L.groups)
        w = (uint32_t)scales[n * L.groups + g] | ((uint32_t)biases[n * L.groups + g] << 16);
    }
    out[i] = w;
  }
}

// one warp per output: lanes stride over the words of the row
template <typename T>
__global__ void __launch_bounds__(128) linear_kernel(const T* __restrict__ x, int M, int K, const uint32_t* __restrict__ packed,
                                                     Q4Layout L, int N, int group, T* __restrict__ y) {
  const int lane = threadIdx.x & 31, n = blockIdx.x * 4 + (threadIdx.x >> 5), m = blockIdx.y;
  if (n >= N) return;
  const uint32_t* codes = packed + (int64_t)(n / kTile) * L.blocks * 128;
  const uint32_t* scales = packed + L.scale_off / 4 + (int64_t)(n / kTile) * ((L.groups + 3) / 4) * 64 + (n % kTile) * 4;
  const int r = n % kTile;
  float acc = 0.0f;
  for (int k = lane * 8; k < K; k += 256) {
    const int in = k % kBlock;
    const uint32_t w = codes[(int64_t)(k / kBlock) * 128 + ((r & 7) * 4 + in / 16) * 4 + (r >> 3) * 2 + (in / 8 & 1)];
    const int g = k / group;
    const uint32_t sw = scales[(g / 4) * 64 + (g & 3)];
    const float s = __uint_as_float(sw << 16), b = __uint_as_float(sw & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = (w >> (4 * (i >> 1) + 16 * (i & 1))) & 15u;
      if (k + i < K) acc = fmaf(to_f(x[(int64_t)m * K + k + i]), fmaf(s, (float)c, b), acc);
    }
  }
  acc = warp_sum(acc);
  if (lane == 0) y[(int64_t)m * N + n] = from_f<T>(acc);
}

}  // namespace

Q4Layout q4_layout(int32_t N, int32_t K, int32_t group) {
  Q4Layout L;
  L.tiles = (N + kTile - 1) / kTile;
  L.blocks = (K + kBlock - 1) / kBlock;
  L.groups = (K + group - 1) / group;
  L.scale_off = (size_t)L.tiles * L.blocks * 512;
  L.total_bytes = L.scale_off + (size_t)L.tiles * ((L.groups + 3) / 4) * 256;
  return L;
}

cudaError_t launch_q4_pack(const void* codes, const void* scales, const void* biases, int32_t N, int32_t K,
                           int32_t group, void* packed, cudaStream_t stream) {
  const Q4Layout L = q4_layout(N, K, group);
  const int64_t blocks = ((int64_t)L.total_bytes / 4 + 255) / 256;
  LaunchScope scope(GDN_K_Q4_PACK, stream);
  q4_pack_kernel<<<(unsigned)(blocks < 148 * 64 ? blocks : 148 * 64), 256, 0, stream>>>(
      (const unsigned char*)codes, (const unsigned short*)scales, (const unsigned short*)biases, N, K, group,
      (int64_t)L.groups * group / 2, L, (uint32_t*)packed);
  return cudaGetLastError();
}

size_t linear_q4_ws_bytes(int32_t, int32_t, int32_t, int32_t, bool) { return 0; }

cudaError_t launch_linear_q4(bool bf16, const void* x, int32_t M, int32_t K, const void* packed, int32_t N,
                             int32_t group, void* y, void*, int32_t*, cudaStream_t stream) {
  const Q4Layout L = q4_layout(N, K, group);
  LaunchScope scope(GDN_K_LINEAR_Q4, stream);
  for (int32_t m0 = 0; m0 < M; m0 += 65535) {
    const int32_t m = M - m0 < 65535 ? M - m0 : 65535;
    const dim3 grid((unsigned)((N + 3) / 4), (unsigned)m);
    if (bf16)
      linear_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>((const __nv_bfloat16*)x + (int64_t)m0 * K, m, K,
                                                             (const uint32_t*)packed, L, N, group,
                                                             (__nv_bfloat16*)y + (int64_t)m0 * N);
    else
      linear_kernel<float><<<grid, 128, 0, stream>>>((const float*)x + (int64_t)m0 * K, m, K, (const uint32_t*)packed,
                                                     L, N, group, (float*)y + (int64_t)m0 * N);
  }
  return cudaGetLastError();
}

}  // namespace gdn
