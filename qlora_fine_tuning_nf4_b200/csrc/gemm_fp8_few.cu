// The block-scaled 8-bit product for a few rows (at most 64), with the LoRA term:
//   Y = X W^T + (s X A) B  (BWD = false)  or  dX = dY W + (s dY B^T) A^T  (BWD = true)
// with the operands and scales of gemm_fp8.cu.
//
// The weight's bytes bound it (each is read once), and with few rows the latency of
// reading them: so a CTA takes 32 output columns and all of the reduction, its eight
// warps take its 128-wide blocks in turn, and each lane has a whole block of weight
// in registers before the previous one is used (64 KB in flight per SM).  Warp-level
// MMAs (m16n8k32) read their fragments straight from those registers: a fragment
// needs 4 consecutive reduction elements per lane, but which ones is free as long
// as both operands agree, so lanes load 16 bytes and call them two fragments.  For
// dX the reduction runs down the columns of W: a lane loads a word (4 columns) of
// 32 rows and transposes 4 x 4 bytes with byte permutes.
//
// Each block's product is formed in fp32 from zero, scaled and added to the warp's
// sums; the warps' sums meet in shared memory and are added in warp order.
#include "kernels.cuh"
#include "ptx.cuh"

namespace ql {

constexpr int FEW_COLS = 32;  // output columns per CTA

// 4 x 4 bytes: word i holds row i; afterwards word j holds column j.
QL_DEV void transpose4x4(uint32_t& w0, uint32_t& w1, uint32_t& w2, uint32_t& w3) {
  const uint32_t a = prmt(w0, w1, 0x5140u), b = prmt(w0, w1, 0x7362u);  // r0c0 r1c0 r0c1 r1c1 | c2, c3
  const uint32_t c = prmt(w2, w3, 0x5140u), d = prmt(w2, w3, 0x7362u);
  w0 = prmt(a, c, 0x5410u);
  w1 = prmt(a, c, 0x7632u);
  w2 = prmt(b, d, 0x5410u);
  w3 = prmt(b, d, 0x7632u);
}

struct FewArgs {
  const uint8_t* x;   // e4m3 [M, red]
  const float* sa;    // [blocks, M]
  const uint8_t* w;   // e4m3 [n_out, k_in]
  const float* sb;    // weight scales, strides per reduction block and per 128 output columns
  int sb_k, sb_n;
  int M, red, cols;   // rows, reduction length, output columns
  int ldw;            // k_in
  const bf16 *L, *R;  // LoRA operands: L [M, r]; R = B [r, n_out] or A [k_in, r]
  int r;              // 0: no adapter
  bf16* out;          // [M, cols]
};

// Block kb of the weight, as fragments: v[2 (4 s + j) + i] is half i of the B fragment of reduction
// step s and column group j.  (The words are laid out by their use: see few_wfrag.)
template <bool BWD>
QL_DEV void few_load_w(const FewArgs& a, int kb, int n0, int g, int q, uint32_t (&v)[32]) {
  if constexpr (!BWD) {
    // rows n0 + 8 j + g; the lane's 16 bytes of each 64-byte half of the block
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + j * 8 + g;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = kb * 128 + c * 64 + q * 16;
        const uint4 u = n < a.cols && k < a.red
                            ? __ldg(reinterpret_cast<const uint4*>(a.w + static_cast<size_t>(n) * a.ldw + k))
                            : make_uint4(0, 0, 0, 0);
        v[j * 8 + c * 4] = u.x;
        v[j * 8 + c * 4 + 1] = u.y;
        v[j * 8 + c * 4 + 2] = u.z;
        v[j * 8 + c * 4 + 3] = u.w;
      }
    }
  } else {
    // rows 32 q .. 32 q + 31 of the block; columns n0 + 4 g .. n0 + 4 g + 3
    const int col = n0 + g * 4;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int n = kb * 128 + q * 32 + i;
      v[i] = n < a.red && col < a.cols
                 ? __ldg(reinterpret_cast<const uint32_t*>(a.w + static_cast<size_t>(n) * a.ldw + col))
                 : 0u;
    }
  }
}
// The lane's 32 bytes of row m in block kb, as the words of reduction steps 0..3 (two each).
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

// MT: row tiles of 16 (1 or 2).  FEW_WARPS: 16 or 8 per CTA.
template <bool BWD, int MT, int FEW_WARPS>
__global__ void __launch_bounds__(FEW_WARPS * 32, MT == 1 ? 16 / FEW_WARPS : 1) gemm_fp8_few_kernel(const FewArgs a) {
  extern __shared__ float part[];  // [warp][16 MT rows][32 columns]
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * FEW_COLS;
  const int nkb = (a.red + 127) / 128;
  const float* sb = a.sb + static_cast<size_t>(n0 / 128) * a.sb_n;  // 32 columns lie in one block of 128
  float acc[MT][4][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][j][i] = 0.f;
  uint32_t wn[32];  // one block of weight ahead
  if (warp < nkb) few_load_w<BWD>(a, warp, n0, g, q, wn);
  for (int kb = warp; kb < nkb; kb += FEW_WARPS) {
    uint32_t w[32], x[MT][2][8];
    float sc[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = t * 16 + h * 8 + g;
        few_load_x<BWD>(a, kb, m, q, x[t][h]);
        sc[t][h] = m < a.M ? __ldg(a.sa + static_cast<size_t>(kb) * a.M + m) : 0.f;
      }
    const float sw = __ldg(sb + static_cast<size_t>(kb) * a.sb_k);
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = wn[i];
    if (kb + FEW_WARPS < nkb) few_load_w<BWD>(a, kb + FEW_WARPS, n0, g, q, wn);
    if constexpr (BWD) {
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
      for (int s = 0; s < 4; ++s) {
        const uint32_t b0 = BWD ? w[s * 8 + j] : w[j * 8 + 2 * s];
        const uint32_t b1 = BWD ? w[s * 8 + 4 + j] : w[j * 8 + 2 * s + 1];
#pragma unroll
        for (int t = 0; t < MT; ++t)
          mma_e4m3_16832(tmp[t], x[t][0][2 * s], x[t][1][2 * s], x[t][0][2 * s + 1], x[t][1][2 * s + 1], b0, b1);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(tmp[t][i], sc[t][i >> 1] * sw, acc[t][j][i]);
    }
  }
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
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * MT * FEW_COLS; i += FEW_WARPS * 32) {
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

template <bool BWD, int MT, int FEW_WARPS>
static cudaError_t launch_few(const FewArgs& a, cudaStream_t st) {
  constexpr int smem = FEW_WARPS * 16 * MT * FEW_COLS * 4;
  static_assert(smem <= 48 * 1024, "no opt-in needed");
  return launch_pdl(gemm_fp8_few_kernel<BWD, MT, FEW_WARPS>, dim3((a.cols + FEW_COLS - 1) / FEW_COLS), dim3(FEW_WARPS * 32), smem,
                    st, a);
}

cudaError_t launch_gemm_fp8_few(bool bwd, const uint8_t* x, const float* sa, const uint8_t* w, const float* sb,
                                int sb_k, int sb_n, int M, int red, int cols, int ldw, const bf16* L, const bf16* R,
                                int r, bf16* out, int sms, cudaStream_t st) {
  const FewArgs a = {x, sa, w, sb, sb_k, sb_n, M, red, cols, ldw, L, R, r, out};
  if (M > 16) return bwd ? launch_few<true, 2, 8>(a, st) : launch_few<false, 2, 8>(a, st);
  if ((cols + FEW_COLS - 1) / FEW_COLS > sms) return bwd ? launch_few<true, 1, 8>(a, st) : launch_few<false, 1, 8>(a, st);
  return bwd ? launch_few<true, 1, 16>(a, st) : launch_few<false, 1, 16>(a, st);
}

}  // namespace ql
