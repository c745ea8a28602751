// The block-scaled 8-bit product for a few rows (at most 32), with the LoRA term:
//   Y = X W^T + (s X A) B  (BWD = false)  or  dX = dY W + (s dY B^T) A^T  (BWD = true)
// with the operands and scales of gemm_fp8.cu.
//
// The weight's bytes bound it (each is read once), and with few rows the latency of
// reading them: a CTA takes 32 output columns and all of the reduction, and one
// thread streams the weight's blocks (32 x 128 bytes) by TMA into a 24-stage ring, so
// two CTAs keep up to 192 KB per SM on their way.  Eight warps take the blocks in
// turn.  Their fragments of warp-level MMAs (m16n8k32) need 4 consecutive reduction
// elements per lane, but which ones is free as long as both operands agree, so lanes
// read 16 bytes and call them two fragments.  For dX the reduction runs down the
// columns of W: lane q of a quad reads words (4 columns) of the rows q, q + 4, ..., and
// bytes are transposed 4 x 4 with byte permutes; the rows of dY, read as 32 bytes per
// lane, are brought to the same order by a transpose across the quad.
//
// Each block's product is formed in fp32 from zero, scaled and added to the warp's
// sums; the warps' sums meet in shared memory and are added in warp order.
//
// With weights that come from HBM: 16 rows, 4096 -> 4096 FWD_US us, 4096 -> 14336 (59 MB, 9.1 us at
// the copy rate) BIG_US us.
#include "kernels.cuh"
#include "ptx.cuh"

namespace ql {

constexpr int FEW_WARPS = 8;                      // consumer warps; one more streams the weight
constexpr int FEW_THREADS = (FEW_WARPS + 1) * 32;
constexpr int FEW_COLS = 32;                      // output columns per CTA
constexpr int FEW_STAGES = 24;
constexpr int FEW_BLOCK = FEW_COLS * 128;         // bytes of a weight block
constexpr int FEW_OFF_BAR = FEW_STAGES * FEW_BLOCK;
constexpr int FEW_SMEM = FEW_OFF_BAR + 2 * FEW_STAGES * 8 + 1024;  // + alignment slack
// The warps' sums [warp][16 MT rows][32 columns] take the ring's place at the end.
static_assert(FEW_WARPS * 32 * FEW_COLS * 4 <= FEW_OFF_BAR, "the sums fit over the ring");

// 4 x 4 bytes: word i holds row i; afterwards word j holds column j.
QL_DEV void transpose4x4(uint32_t& w0, uint32_t& w1, uint32_t& w2, uint32_t& w3) {
  const uint32_t a = prmt(w0, w1, 0x5140u), b = prmt(w0, w1, 0x7362u);  // r0c0 r1c0 r0c1 r1c1 | c2, c3
  const uint32_t c = prmt(w2, w3, 0x5140u), d = prmt(w2, w3, 0x7362u);
  w0 = prmt(a, c, 0x5410u);
  w1 = prmt(a, c, 0x7632u);
  w2 = prmt(b, d, 0x5410u);
  w3 = prmt(b, d, 0x7632u);
}
// Across a quad of lanes: lane q's word s becomes lane s's word q.
QL_DEV void quad_transpose(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, int q) {
  auto swap = [q](uint32_t& lo, uint32_t& hi, int bit) {
    const bool up = (q & bit) != 0;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
    if (up) lo = y;
    else hi = y;
  };
  swap(r0, r1, 1);
  swap(r2, r3, 1);
  swap(r0, r2, 2);
  swap(r1, r3, 2);
}

struct FewArgs {
  const uint8_t* x;   // e4m3 [M, red]
  const float* sa;    // [blocks, M]
  const float* sb;    // weight scales, strides per reduction block and per 128 output columns
  int sb_k, sb_n;
  int M, red, cols;   // rows, reduction length, output columns
  const bf16 *L, *R;  // LoRA operands: L [M, r]; R = B [r, n_out] or A [k_in, r]
  int r;              // 0: no adapter
  bf16* out;          // [M, cols]
  int* status;
};

// The lane's 32 bytes of row m in block kb.
template <bool BWD>
QL_DEV void few_load_x(const FewArgs& a, int kb, int m, int q, uint32_t (&v)[8]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int k = kb * 128 + (BWD ? q * 32 + c * 16 : c * 64 + q * 16);
    const uint4 u = m < a.M && k < a.red
                        ? __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(m) * a.red + k))
                        : make_uint4(0, 0, 0, 0);
    v[c * 4] = u.x;
    v[c * 4 + 1] = u.y;
    v[c * 4 + 2] = u.z;
    v[c * 4 + 3] = u.w;
  }
}

// MT: row tiles of 16 (1 or 2).  map: e4m3 weight [n_out, k_in], box {128, 32} with 128B swizzle
// (forward) or {32, 128} (dX).
template <bool BWD, int MT>
__global__ void __launch_bounds__(FEW_THREADS, MT == 1 ? 2 : 1)
    gemm_fp8_few_kernel(const __grid_constant__ CUtensorMap map, const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * FEW_COLS;
  const int nkb = (a.red + 127) / 128;
  auto full_bar = [&](int s) { return sbase + FEW_OFF_BAR + 8u * s; };
  auto empty_bar = [&](int s) { return sbase + FEW_OFF_BAR + 8u * (FEW_STAGES + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < FEW_STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  float acc[MT][4][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][j][i] = 0.f;
  const int g = lane >> 2, q = lane & 3;
  if (warp == FEW_WARPS) {
    bool ok = true;
    for (int kb = 0; kb < nkb && ok; ++kb) {
      const int s = kb % FEW_STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(s), ((kb / FEW_STAGES) & 1) ^ 1, a.status));
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(full_bar(s), FEW_BLOCK);
        if (BWD) tma_load_2d(sbase + s * FEW_BLOCK, &map, full_bar(s), n0, kb * 128);
        else tma_load_2d(sbase + s * FEW_BLOCK, &map, full_bar(s), kb * 128, n0);
      }
      __syncwarp();
    }
    if (!ok) settle_inflight();  // loads already issued land before the CTA can exit
  } else {
    const float* sb = a.sb + static_cast<size_t>(n0 / 128) * a.sb_n;  // 32 columns lie in one block of 128
    uint32_t xn[MT][2][8];  // one block ahead
    float scn[MT][2], swn = 0.f;
    auto request = [&](int kb) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = t * 16 + h * 8 + g;
          few_load_x<BWD>(a, kb, m, q, xn[t][h]);
          scn[t][h] = m < a.M ? __ldg(a.sa + static_cast<size_t>(kb) * a.M + m) : 0.f;
        }
      swn = __ldg(sb + static_cast<size_t>(kb) * a.sb_k);
    };
    if (warp < nkb) request(warp);
    for (int kb = warp; kb < nkb; kb += FEW_WARPS) {
      uint32_t w[32], x[MT][2][8];
      float sc[MT][2];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[t][h][i] = xn[t][h][i];
          sc[t][h] = scn[t][h] * swn;
          if constexpr (BWD) {
            // bytes of the lane's 32 consecutive elements -> bytes q, q + 4, q + 8, q + 12 of every 16
            transpose4x4(x[t][h][0], x[t][h][1], x[t][h][2], x[t][h][3]);
            transpose4x4(x[t][h][4], x[t][h][5], x[t][h][6], x[t][h][7]);
            quad_transpose(x[t][h][0], x[t][h][1], x[t][h][2], x[t][h][3], q);
            quad_transpose(x[t][h][4], x[t][h][5], x[t][h][6], x[t][h][7], q);
          }
        }
      if (kb + FEW_WARPS < nkb) request(kb + FEW_WARPS);
      const int s = kb % FEW_STAGES;
      if (!__all_sync(0xffffffffu, mbar_wait(full_bar(s), (kb / FEW_STAGES) & 1, a.status))) break;
      const uint8_t* blk = sgen + s * FEW_BLOCK;
      if constexpr (!BWD) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 u = *reinterpret_cast<const uint4*>(blk + (j * 8 + g) * 128 + (((c * 4 + q) ^ g) << 4));
            w[j * 8 + c * 4] = u.x;
            w[j * 8 + c * 4 + 1] = u.y;
            w[j * 8 + c * 4 + 2] = u.z;
            w[j * 8 + c * 4 + 3] = u.w;
          }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = *reinterpret_cast<const uint32_t*>(blk + (i * 4 + q) * 32 + g * 4);
#pragma unroll
        for (int i = 0; i < 32; i += 4) transpose4x4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float tmp[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) tmp[t][i] = 0.f;
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // 32 reduction elements each
          const uint32_t b0 = BWD ? w[p * 8 + j] : w[j * 8 + 2 * p];
          const uint32_t b1 = BWD ? w[p * 8 + 4 + j] : w[j * 8 + 2 * p + 1];
          constexpr int kLo = BWD ? 1 : 2, kHi = BWD ? 4 : 1;  // word of step p, and the distance to its second
#pragma unroll
          for (int t = 0; t < MT; ++t)
            mma_e4m3_16832(tmp[t], x[t][0][kLo * p], x[t][1][kLo * p], x[t][0][kLo * p + kHi], x[t][1][kLo * p + kHi],
                           b0, b1);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(tmp[t][i], sc[t][i >> 1], acc[t][j][i]);
      }
      // Released once the products have consumed what was read from it (an arrive right after the
      // loads could overtake them).
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(s));
    }
  }
  __syncthreads();  // every block has been used: the sums may take the ring's place
  float* part = reinterpret_cast<float*>(sgen);
  if (warp < FEW_WARPS) {
    // columns of the fragments: group j is columns 8 j .. 8 j + 7 (forward), or j, j + 4, ... (dX)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 2 * q + (i & 1), m = t * 16 + (i >> 1) * 8 + g;
          part[(warp * 16 * MT + m) * FEW_COLS + (BWD ? c * 4 + j : j * 8 + c)] = acc[t][j][i];
        }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * MT * FEW_COLS; i += FEW_THREADS) {
    const int m = i / FEW_COLS, n = n0 + i % FEW_COLS;
    if (m >= a.M) break;
    if (n >= a.cols) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < FEW_WARPS; ++k) v += part[k * 16 * MT * FEW_COLS + i];
    for (int k = 0; k < a.r; ++k)
      v = fmaf(__bfloat162float(a.L[static_cast<size_t>(m) * a.r + k]),
               __bfloat162float(BWD ? a.R[static_cast<size_t>(n) * a.r + k] : a.R[static_cast<size_t>(k) * a.cols + n]), v);
    a.out[static_cast<size_t>(m) * a.cols + n] = __float2bfloat16(v);
  }
}

template <bool BWD, int MT>
static cudaError_t launch_few(const CUtensorMap& map, const FewArgs& a, cudaStream_t st) {
  auto kern = gemm_fp8_few_kernel<BWD, MT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static bool set[64] = {false};
  if (!set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  return launch_pdl(kern, dim3((a.cols + FEW_COLS - 1) / FEW_COLS), dim3(FEW_THREADS), FEW_SMEM, st, map, a);
}

cudaError_t launch_gemm_fp8_few(bool bwd, const CUtensorMap& map, const uint8_t* x, const float* sa, const float* sb,
                                int sb_k, int sb_n, int M, int red, int cols, const bf16* L, const bf16* R, int r,
                                bf16* out, int* status, cudaStream_t st) {
  const FewArgs a = {x, sa, sb, sb_k, sb_n, M, red, cols, L, R, r, out, status};
  if (M > 32) return cudaErrorInvalidValue;
  if (M > 16) return bwd ? launch_few<true, 2>(map, a, st) : launch_few<false, 2>(map, a, st);
  return bwd ? launch_few<true, 1>(map, a, st) : launch_few<false, 1>(map, a, st);
}

}  // namespace ql
