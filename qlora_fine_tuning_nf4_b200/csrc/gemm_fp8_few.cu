// The block-scaled 8-bit product for a few rows (at most 64), with the LoRA term:
//   Y = X W^T + (s X A) B  (BWD = false)  or  dX = dY W + (s dY B^T) A^T  (BWD = true)
// with the operands and scales of gemm_fp8.cu.
//
// The weight's bytes bound it: each is read once.  So the weight is the MMA's 128-row
// operand and the few rows are its N (16, 32 or 64; rows past M are zeros from the
// TMA): out^T = W X^T.  A cluster takes 128 output columns and its CTAs deal the
// 128-wide reduction blocks among themselves, as many CTAs as fill the GPU.  Per CTA:
//   warp 0       TMA producer: weight tiles (128 x 128 bytes) and the rows' blocks
//   warp 1       TMEM allocation; issues tcgen05.mma, a fresh accumulator per block
//   warp 2       scales: sa * sw of a block's rows into a shared-memory ring
//   warps 4-7    accumulate: TMEM -> scale -> registers
// Eight accumulators of 16 or 32 columns (four of 64) hide the way from the MMA to the
// accumulating warps and back.  The CTAs' sums meet through distributed shared memory, are added in
// rank order and leave as bf16.  The LoRA term is two more blocks of the last CTA, the
// halves of the low-rank pair (gemm_fp8.cu): bf16 operands (kind::f16) and scale 1.
//
// With weights that come from HBM: one row, 4096 -> 14336 (59 MB, 9.1 us at the copy
// rate) 13.1 us, 4096 -> 4096 (17 MB, 2.6 us) 6.6 us; 64 rows 15.9 and 8.3 us; dX of the
// same weights 13.3 and 6.7, 17.1 and 8.6 us.  Warp-level
// MMAs fed by the same ring of TMA loads took 17.5 us for the former: an e4m3
// m16n8k32 occupies a scheduler for about 64 cycles, so they were bound by it.  Stages
// for two CTAs per SM rather than one: the next CTA (or the next launch's) sets up
// while this one drains (64 rows, 4096 -> 4096: 12.1 -> 8.5 us).
#include "kernels.cuh"
#include "ptx.cuh"

namespace ql {

template <int NT>
struct FewCfg {
  static constexpr int BM = 128;                 // output columns per cluster (the MMA's rows)
  static constexpr int W_BYTES = BM * 128;       // a block of the weight
  static constexpr int X_BYTES = NT * 128;       // a block of the rows
  static constexpr int S = NT == 64 ? 4 : 5;     // operand stages: two CTAs fit on an SM
  static constexpr int ACCS = NT == 64 ? 4 : 8;
  static constexpr int SR = S + ACCS + 2;        // scale slots (as in gemm_fp8.cu)
  static constexpr int G = 8;                    // blocks whose scales are requested together
  static constexpr int OFF_X = S * W_BYTES;
  static constexpr int OFF_SC = OFF_X + S * X_BYTES;
  static constexpr int OFF_BAR = OFF_SC + SR * NT * 4;
  static constexpr int NBAR = 2 * S + 2 * ACCS + 1;
  static constexpr int SMEM_BYTES = OFF_BAR + NBAR * 8 + 16 + 1024;  // + alignment slack
  static constexpr int THREADS = 256;
  static constexpr int TMEM_COLS = ACCS * NT;
  static_assert(SMEM_BYTES <= 232448 / 2 - 1024 && 2 * TMEM_COLS <= 512, "two CTAs per SM");
  static_assert(NT * BM * 4 <= S * W_BYTES, "a CTA's sums fit over the stages");
};

struct FewArgs {
  const float* sa;    // [blocks, M]
  const float* sb;    // weight scales, strides per reduction block and per 128 output columns
  int sb_k, sb_n;
  int M, nkb, cols;   // rows, reduction blocks, output columns
  int cluster;        // CTAs that share a tile's reduction
  int lora_k16;       // 16-wide reduction steps of a LoRA block (rank / 16), 0 = no adapter
  bf16* out;          // [M, cols]
  int* status;
};

template <bool BWD, int NT>
__global__ void __launch_bounds__(FewCfg<NT>::THREADS, 2)
    gemm_fp8_few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  using C = FewCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x % a.cluster);
  const int n0 = static_cast<int>(blockIdx.x / a.cluster) * C::BM;
  const int own = (a.nkb - rank + a.cluster - 1) / a.cluster;  // blocks rank, rank + cluster, ...
  const int mine = own + (a.lora_k16 > 0 && rank == a.cluster - 1 ? 2 : 0);

  if (!dev_check(a.M > 0 && a.M <= NT && a.cols > 0 && a.cluster >= 1 && a.cluster <= 8 && a.nkb >= a.cluster &&
                     a.lora_k16 >= 0 && a.lora_k16 <= 4 &&
                     static_cast<int>(gridDim.x) == (a.cols + C::BM - 1) / C::BM * a.cluster,
                 a.status)) {
    grid_dep_wait();
    return;
  }

  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::S + s); };
  const uint32_t acc_full0 = bar0 + 8u * (2 * C::S);
  const uint32_t acc_empty0 = acc_full0 + 8u * C::ACCS;
  const uint32_t drain_bar = acc_empty0 + 8u * C::ACCS;
  float* const scales = reinterpret_cast<float*>(sgen + C::OFF_SC);  // [slot][row]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sgen + C::OFF_BAR + C::NBAR * 8);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(full_bar(s), 2);  // the loads, and the scales
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < C::ACCS; ++b) {
      mbar_init(acc_full0 + 8u * b, 1);
      mbar_init(acc_empty0 + 8u * b, 4);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  grid_dep_wait();
  grid_dep_launch();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    bool ok = true;
    int s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < mine; ++i) {
      const int kb = rank + i * a.cluster;
      ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(s), ph, a.status));
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(full_bar(s), C::W_BYTES + C::X_BYTES);
        const uint32_t w = sbase + s * C::W_BYTES, x = sbase + C::OFF_X + s * C::X_BYTES;
        if (i < own) {
          // W rows x reduction bytes (K-major), or reduction rows x output columns (MN-major)
          if (BWD) tma_load_2d(w, &maps.w, full_bar(s), n0, kb * 128);
          else tma_load_2d(w, &maps.w, full_bar(s), kb * 128, n0);
          tma_load_2d(x, &maps.x, full_bar(s), kb * 128, 0);
        } else {
          // LoRA operands, 64 wide (the MMAs read the rank's): A [128 columns, r] K-major (dX) or
          // B [r, 128 columns] MN-major in chunks of 64 columns (forward), and half i - own of the pair
          if (BWD) {
            tma_load_2d(w, &maps.r, full_bar(s), 0, n0);
          } else {
            tma_load_2d(w, &maps.r, full_bar(s), n0, 0);
            tma_load_2d(w + 8192, &maps.r, full_bar(s), n0 + 64, 0);
          }
          tma_load_2d(x, &maps.l, full_bar(s), (i - own) * a.lora_k16 * 16, 0);
        }
      }
      __syncwarp();
      if (++s == C::S) s = 0, ph ^= 1;
    }
    if (!ok) settle_inflight();  // loads already issued land before the CTA can exit
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA -----
    bool ok = true;
    constexpr uint32_t idesc = idesc_e4m3(C::BM, NT, BWD, false);
    constexpr uint32_t idesc_lora = idesc_bf16(C::BM, NT, !BWD, false);
    const uint64_t wd0 = smem_desc(sbase, BWD ? C::W_BYTES : 16, 1024, QL_SWZ_128B);
    const uint64_t xd0 = smem_desc(sbase + C::OFF_X, 16, 1024, QL_SWZ_128B);
    const uint64_t rd0 = smem_desc(sbase, BWD ? 16 : 8192, 1024, QL_SWZ_128B);
    int s = 0, b = 0;
    uint32_t ph = 0, aph = 1;
    for (int i = 0; i < mine; ++i) {
      ok = mbar_wait(full_bar(s), ph, a.status) && mbar_wait(acc_empty0 + 8u * b, aph, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t wo = static_cast<uint64_t>(s) * (C::W_BYTES >> 4);
        const uint64_t xd = xd0 + static_cast<uint64_t>(s) * (C::X_BYTES >> 4);
        if (i < own) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 reduction elements each
            umma_e4m3<1>(tmem + b * NT, wd0 + wo + kk * (BWD ? 256 : 2), xd + kk * 2, idesc, kk != 0);
        } else {
          for (int kk = 0; kk < a.lora_k16; ++kk)
            umma_bf16<1>(tmem + b * NT, rd0 + wo + kk * (BWD ? 2 : 128), xd + kk * 2, idesc_lora, kk != 0);
        }
        umma_commit<1>(empty_bar(s));
        umma_commit<1>(acc_full0 + 8u * b);
      }
      __syncwarp();
      if (++s == C::S) s = 0, ph ^= 1;
      if (++b == C::ACCS) b = 0, aph ^= 1;
    }
    // let every issued MMA finish before TMEM can be released (after an error too)
    if (elect_one()) umma_commit<1>(drain_bar);
    __syncwarp();
    mbar_drain(drain_bar, 0);
  } else if (warp == 2) {
    // ------------------------------------------------------ scales -----
    bool ok = true;
    int s = 0, sl = 0;
    uint32_t ph = 1;
    const float* sb = a.sb + static_cast<size_t>(n0 / 128) * a.sb_n;
    for (int i0 = 0; i0 < mine && ok; i0 += C::G) {
      float v[C::G][NT / 32 + (NT < 32)];
#pragma unroll
      for (int g = 0; g < C::G; ++g) {
        const int kb = rank + (i0 + g) * a.cluster;
        const float lora = i0 + g >= own ? 1.f : 0.f;
        const float w = kb < a.nkb ? __ldg(sb + static_cast<size_t>(kb) * a.sb_k) : 0.f;
#pragma unroll
        for (int h = 0; h < NT / 32 + (NT < 32); ++h) {
          const int m = h * 32 + lane;
          v[g][h] = kb < a.nkb && m < a.M ? w * __ldg(a.sa + static_cast<size_t>(kb) * a.M + m) : lora;
        }
      }
#pragma unroll
      for (int g = 0; g < C::G; ++g) {
        if (i0 + g >= mine) break;
        ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(s), ph, a.status));
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < NT / 32 + (NT < 32); ++h)
          if (h * 32 + lane < NT) scales[sl * NT + h * 32 + lane] = v[g][h];
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar(s));
        if (++s == C::S) s = 0, ph ^= 1;
        if (++sl == C::SR) sl = 0;
      }
    }
  }
  float acc[NT];
  if (warp >= 4) {
    // ------------------------------------------------------ accumulate ---
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = 0.f;
    const uint32_t quad = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int b = 0, sl = 0;
    uint32_t ph = 0;
    for (int i = 0; i < mine; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(acc_full0 + 8u * b, ph, a.status))) break;
      tc_fence_after();
      const float4* sc = reinterpret_cast<const float4*>(scales + sl * NT);
      if (++sl == C::SR) sl = 0;
      constexpr int CH = NT < 32 ? NT : 32;  // columns loaded at a time
#pragma unroll
      for (int c0 = 0; c0 < NT; c0 += CH) {
        uint32_t v[CH];
#pragma unroll
        for (int c = 0; c < CH; c += 16) tmem_ld_32x32b_x16_async(tmem + quad + b * NT + c0 + c, v + c);
#pragma unroll
        for (int c = 0; c < CH; c += 16) tmem_wait_ld16(v + c);
#pragma unroll
        for (int c = 0; c < CH; c += 4) {
          const float4 x = sc[(c0 + c) / 4];
          acc[c0 + c] = fmaf(__uint_as_float(v[c]), x.x, acc[c0 + c]);
          acc[c0 + c + 1] = fmaf(__uint_as_float(v[c + 1]), x.y, acc[c0 + c + 1]);
          acc[c0 + c + 2] = fmaf(__uint_as_float(v[c + 2]), x.z, acc[c0 + c + 2]);
          acc[c0 + c + 3] = fmaf(__uint_as_float(v[c + 3]), x.w, acc[c0 + c + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty0 + 8u * b);
      if (++b == C::ACCS) b = 0, ph ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();  // every block has been added: the sums may take the stages' place
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, C::TMEM_COLS);
  }
  float* red = reinterpret_cast<float*>(sgen);  // [row][128 columns]
  if (warp >= 4) {
#pragma unroll
    for (int i = 0; i < NT; ++i) red[i * C::BM + (warp & 3) * 32 + lane] = acc[i];
  }
  cluster_sync();
  // each CTA finishes every cluster-th row, four columns per thread (cols % 16 == 0)
  for (int i = threadIdx.x; i < (a.M - rank + a.cluster - 1) / a.cluster * (C::BM / 4); i += C::THREADS) {
    const int m = rank + i / (C::BM / 4) * a.cluster, c = i % (C::BM / 4) * 4, n = n0 + c;
    if (n >= a.cols || !dev_check(m < a.M && n + 4 <= a.cols, a.status)) continue;
    float4 x[8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (p < a.cluster) x[p] = ld_cluster_f32x4(mapa_shared(sbase + (m * C::BM + c) * 4, static_cast<uint32_t>(p)));
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (p < a.cluster) v[0] += x[p].x, v[1] += x[p].y, v[2] += x[p].z, v[3] += x[p].w;
    *reinterpret_cast<uint2*>(a.out + static_cast<size_t>(m) * a.cols + n) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
  cluster_sync();  // no CTA leaves while another still reads its sums
}

template <bool BWD, int NT>
static cudaError_t launch_few(const FewMaps& maps, const FewArgs& a, cudaStream_t st) {
  using C = FewCfg<NT>;
  auto kern = gemm_fp8_few_kernel<BWD, NT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static bool set[64] = {false};
  if (!set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.cols + C::BM - 1) / C::BM * a.cluster));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

// Rows per MMA (the box of the rows' tensor map): M rounded up to 16, 32 or 64.
int gemm_fp8_few_rows(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : 64); }

cudaError_t launch_gemm_fp8_few(bool bwd, const FewMaps& maps, const float* sa, const float* sb, int sb_k, int sb_n,
                                int M, int red, int cols, int cluster, int r, bf16* out, int* status,
                                cudaStream_t st) {
  const FewArgs a = {sa, sb, sb_k, sb_n, M, (red + 127) / 128, cols, cluster, r / 16, out, status};
  if (M > 64) return cudaErrorInvalidValue;
  if (M > 32) return bwd ? launch_few<true, 64>(maps, a, st) : launch_few<false, 64>(maps, a, st);
  if (M > 16) return bwd ? launch_few<true, 32>(maps, a, st) : launch_few<false, 32>(maps, a, st);
  return bwd ? launch_few<true, 16>(maps, a, st) : launch_few<false, 16>(maps, a, st);
}

}  // namespace ql
