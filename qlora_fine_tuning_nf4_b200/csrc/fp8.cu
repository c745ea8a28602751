// Quantisers of the 8-bit formats (fp8.cuh): rows with one scale per 128
// columns, weights with one per 128 x 128 block.  HBM-bound, one pass: 8192 x 4096 rows
// 18 us (5.6 TB/s), a 14336 x 4096 weight from HBM 31.7 us (5.5 TB/s, 0.86 of the copy
// rate), 4096 x 4096 11.1 us (4.5 TB/s).
#include "fp8.cuh"

namespace ql {

// A CTA takes 32 rows x 256 columns; a warp has four rows in flight, each lane 8
// columns of each (16-byte loads, 8-byte stores).  The scales of the 32 rows meet
// in shared memory and leave as whole lines of scale[block][row].
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const bf16* __restrict__ X, int M, int K, int ncb,
                                                                uint8_t* __restrict__ codes,
                                                                float* __restrict__ scale) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float ss[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = (blockIdx.x / ncb) * 32, c0 = (blockIdx.x % ncb) * 256;
  const int c = c0 + lane * 8;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = r0 + warp * 4 + i;
    v[i] = row < M && c < K ? __ldg(reinterpret_cast<const uint4*>(X + static_cast<size_t>(row) * K + c))
                            : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = r0 + warp * 4 + i;
    float f[8], s, inv;
    unpack_bf16x8(v[i], f);
    fp8_scale(half_warp_max(absmax8(f)), s, inv);
    if (row < M && c < K) *reinterpret_cast<uint2*>(codes + static_cast<size_t>(row) * K + c) = e4m3x8(f, inv);
    if ((lane & 15) == 0) ss[lane >> 4][warp * 4 + i] = s;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int kb = c0 / kFp8Block + (threadIdx.x >> 5);
    const int row = r0 + (threadIdx.x & 31);
    if (kb * kFp8Block < K && row < M) scale[static_cast<size_t>(kb) * M + row] = ss[threadIdx.x >> 5][threadIdx.x & 31];
  }
}

// One CTA per 128 x 128 block, held in registers (eight 16-byte chunks per thread).
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const bf16* __restrict__ w, int N, int K, int nkb,
                                                           uint8_t* __restrict__ codes, float* __restrict__ scale) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[8];
  const int nb = blockIdx.x / nkb, kb = blockIdx.x % nkb;
  const int r = nb * kFp8Block + (threadIdx.x >> 4), c = kb * kFp8Block + (threadIdx.x & 15) * 8;
  uint4 v[8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = r + i * 16 < N && c < K ? __ldg(reinterpret_cast<const uint4*>(w + static_cast<size_t>(r + i * 16) * K + c))
                                   : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack_bf16x8(v[i], f);
    m = fmaxf(m, absmax8(f));
  }
  m = half_warp_max(m);
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
  float s, inv;
  fp8_scale(m, s, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r + i * 16 >= N || c >= K) break;
    float f[8];
    unpack_bf16x8(v[i], f);
    *reinterpret_cast<uint2*>(codes + static_cast<size_t>(r + i * 16) * K + c) = e4m3x8(f, inv);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

cudaError_t launch_fp8_quantize_rows(const bf16* X, int64_t M, int64_t K, uint8_t* codes, float* scale,
                                     cudaStream_t st) {
  const int64_t ncb = (K + 255) / 256, grid = ncb * ((M + 31) / 32);
  return launch_pdl(fp8_quantize_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, X, (int)M, (int)K,
                    (int)ncb, codes, scale);
}
cudaError_t launch_fp8_quantize(const bf16* w, int64_t N, int64_t K, uint8_t* codes, float* scale, cudaStream_t st) {
  const int64_t nkb = (K + kFp8Block - 1) / kFp8Block, grid = nkb * ((N + kFp8Block - 1) / kFp8Block);
  return launch_pdl(fp8_quantize_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, w, (int)N, (int)K,
                    (int)nkb, codes, scale);
}

}  // namespace ql
