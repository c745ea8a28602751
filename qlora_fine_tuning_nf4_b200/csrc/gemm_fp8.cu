// Block-scaled 8-bit GEMM for sm_100a with the LoRA term in the same pass:
//   forward  Y  = X W^T + (s X A) B     (BWD = false, reduction over k_in)
//   dX       dX = dY W  + (s dY B^T) A^T (BWD = true, reduction over n_out)
// X, dY and W are e4m3; X and dY carry one fp32 scale per row and 128 reduction
// columns, W one per 128 x 128 block.  With x_kb and w_kb the codes of reduction
// block kb,
//   Y[m, n] = sum_kb sa[kb, m] sw[n / 128, kb] * (x_kb w_kb^T)[m, n].
// The scales are any fp32 numbers, so they cannot ride on the tensor core's own
// block scaling (powers of two): each block's product is an MMA group of its own
// into a fresh TMEM accumulator, and the epilogue warps add it, scaled, to the
// output tile they hold in registers in fp32.
//
// Structure (persistent; one 256 x 256 output tile at a time per CTA pair):
//   warp 0       TMA producer: A and W tiles (128 x 128 bytes each), LoRA operands
//   warp 1       TMEM allocation; the leader CTA's issues tcgen05.mma
//   warp 2       scales: sa * sw of a block's rows and two column blocks into a
//                shared-memory ring, ahead of the MMA
//   warps 4-11   accumulate: TMEM -> scale -> registers; at the tile's end
//                registers -> bf16 -> shared memory -> TMA store
// Two TMEM accumulators of 256 columns alternate per reduction block, so the MMA
// of one block runs while the previous one is being added.  The LoRA term is two
// more blocks with bf16 operands (kind::f16) and scale 1: the fp32 sums s X A (or
// s dY B^T) come as a pair of bf16 numbers, the rounded value and what the rounding
// leaves, each times the same factor, so that they enter Y (or dX) with 16 bits.
//
// What bounds it.  Per block and SM the tensor core needs 512 cycles, 32 KB come
// from L2 (64 bytes a cycle: 512 as well), and the accumulating warps 256 cycles
// of fma and as many of TMEM loads per scheduler.  8192 x 4096 x 11008 takes 0.30
// to 0.35 ms in bursts of ten (2.1 to 2.4 PFLOP/s, by the box) and 0.37 ms (2.0) in a
// long run of calls, under the 1 kW power cap; the same kernel without the scaling,
// adding the blocks in TMEM, 0.24 ms where this one took 0.31.  On the way there, each
// measured on that product:
//  * issuing from one elected thread of a converged warp (elect.sync) instead of
//    under `lane == 0`: 0.39 -> 0.35 ms.  Under a divergent branch every MMA,
//    commit and TMA load costs tens of cycles more, and the issue loop is one
//    serial chain that every block passes through;
//  * scales through shared memory from a warp of their own: 0.35 -> 0.31 ms.
//    Loaded by the accumulating warps themselves, even four blocks ahead, they
//    make those warps wait for an L2 round trip along with their TMEM loads;
//  * 160 columns with three accumulators, or two accumulators of 192: fewer
//    stalls between accumulators, but 15-30% more bytes from L2 per product:
//    0.38 ms;
//  * sixteen accumulating warps: slower, 0.31 -> 0.33-0.345 ms; packed pairs of
//    fma: no gain.
#include "kernels.cuh"
#include "ptx.cuh"

namespace ql {

// BN: output columns per tile, 256 or 128.
template <int BN>
struct Gemm8Cfg {
  static constexpr int BM = 128;    // rows per CTA
  static constexpr int BNT = BN;
  static constexpr int BNC = BN / 2;  // columns of W each CTA of the pair loads; columns per accumulating warp
  static constexpr int BK = 128;    // reduction block: one scale, one 128-byte row
  static constexpr int ACCS = 512 / BN;  // TMEM accumulators
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = BNC * BK;
  static constexpr int S = BN == 256 ? 6 : 8;  // operand stages
  // Scale slots.  A slot is written once its block's operand stage is free, at most S blocks ahead of
  // the MMA, which is at most ACCS ahead of the accumulating warps, which read a block's scale before
  // they release its accumulator: S + ACCS + 2 slots need no barrier of their own.
  static constexpr int SR = S + ACCS + 2;
  static constexpr int NBLK = BN / 128;     // weight blocks side by side in a tile
  static constexpr int SC_FLOATS = NBLK * BM;  // [weight block][row]
  static constexpr int G = 4;       // blocks whose scales are requested together
  static constexpr int EPI_WARPS = 8;
  static constexpr int EPI_WARP0 = 4;  // warp 3 fills the first warp group
  static constexpr int EPI_SLOT = 32 * 32 * 2;
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + S * A_BYTES;
  static constexpr int OFF_EPI = OFF_B + S * B_BYTES;
  static constexpr int OFF_SC = OFF_EPI + EPI_WARPS * EPI_SLOT;
  static constexpr int OFF_BAR = OFF_SC + SR * SC_FLOATS * 4;
  static constexpr int NBAR = 2 * S + 2 * ACCS + 1;
  static constexpr int SMEM_BYTES = OFF_BAR + NBAR * 8 + 16 + 1024;  // + alignment slack
  static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
  static constexpr int TMEM_COLS = 512;
  // The accumulating warps hold up to 128 sums and two 32-register TMEM loads each: more than the 168
  // registers a thread that 384 threads leave.  Warp group 0 gives up what it does not need:
  // 40 + 2 * 232 = 3 * 168.
  static constexpr int REGS_PRODUCER = 40, REGS_EPI = 232, REGS_LAUNCH = 168;
  static_assert(BN == 256 || BN == 128, "tile width");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(THREADS == 384 && REGS_PRODUCER + 2 * REGS_EPI == 3 * REGS_LAUNCH && REGS_LAUNCH * THREADS <= 65536,
                "the warp groups' registers add up to the launch's");
};

template <bool BWD, int BN>
__global__ void __launch_bounds__(Gemm8Cfg<BN>::THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ Gemm8Maps maps, const Gemm8Args args) {
  using C = Gemm8Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  const int n_tiles = (args.N + C::BNT - 1) / C::BNT;
  const int m_tiles = (args.M + 2 * C::BM - 1) / (2 * C::BM);
  // units of work: a tile, or one of `splits` parts of a tile's reduction
  const int units = n_tiles * m_tiles * args.splits;
  const int cluster = blockIdx.x / 2;
  const int clusters = gridDim.x / 2;
  if (!dev_check(args.M > 0 && args.N > 0 && args.nkb > 0 && args.group_m >= 1 && args.lora_k16 >= 0 &&
                     args.lora_k16 <= 4 && args.splits >= 1 && args.splits <= args.nkb,
                 args.status)) {
    grid_dep_wait();
    return;
  }

  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::S + s); };
  const uint32_t acc_full0 = bar0 + 8u * (2 * C::S);
  const uint32_t acc_empty0 = acc_full0 + 8u * C::ACCS;
  const uint32_t drain_bar = acc_empty0 + 8u * C::ACCS;
  float* const scales = reinterpret_cast<float*>(sgen + C::OFF_SC);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sgen + C::OFF_BAR + C::NBAR * 8);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(full_bar(s), 3);  // the loads, and each CTA's scales
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < C::ACCS; ++b) {
      mbar_init(acc_full0 + 8u * b, 1);
      mbar_init(acc_empty0 + 8u * b, 2 * C::EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  const uint32_t lead0 = mapa_shared(bar0, 0);  // the leader CTA's barriers
  grid_dep_wait();
  grid_dep_launch();

  // Tiles in groups of group_m row tiles, rows fastest inside a group (as the bf16 GEMM); a tile's
  // parts side by side.  Blocks [k0, k1) of the reduction; the last part takes the LoRA blocks (nkb, nkb + 1).
  auto unit_coords = [&](int u, int& m0, int& n0, int& k0, int& k1) {
    const int t = u / args.splits, p = u - t * args.splits;
    const int gsz = args.group_m * n_tiles;
    const int first = (t / gsz) * args.group_m;
    const int gm = min(m_tiles - first, args.group_m);
    const int r = t - (first / args.group_m) * gsz;
    m0 = (first + r % gm) * 2 * C::BM + static_cast<int>(rank) * C::BM;
    n0 = (r / gm) * C::BNT;
    k0 = static_cast<int>(static_cast<int64_t>(args.nkb) * p / args.splits);
    k1 = static_cast<int>(static_cast<int64_t>(args.nkb) * (p + 1) / args.splits);
    if (p == args.splits - 1 && args.lora_k16 > 0) k1 += 2;
  };

  if (warp < C::EPI_WARP0) {
    setmaxnreg_dec<C::REGS_PRODUCER>();
    if (warp == 0) {
      // ---------------------------------------------------- TMA producer --
      bool ok = true;
      int s = 0;
      uint32_t ph = 1;
      for (int u = cluster; u < units && ok; u += clusters) {
        int m0, n0, k0, k1;
        unit_coords(u, m0, n0, k0, k1);
        const int col = n0 + static_cast<int>(rank) * C::BNC;  // this CTA's share of the tile's columns
        for (int kb = k0; kb < k1; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(s), ph, args.status));
          if (!ok) break;
          if (elect_one()) {
            // both CTAs' loads complete on the leader's barrier
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * (C::A_BYTES + C::B_BYTES));
            const uint32_t bar = lead0 + 8u * s;
            const uint32_t a = sbase + C::OFF_A + s * C::A_BYTES, b = sbase + C::OFF_B + s * C::B_BYTES;
            if (kb < args.nkb) {
              tma_load_2d_pair(a, &maps.a, bar, kb * C::BK, m0);
              // W rows x reduction bytes (K-major), or reduction rows x output columns (MN-major)
              if (BWD) tma_load_2d_pair(b, &maps.b, bar, col, kb * C::BK);
              else tma_load_2d_pair(b, &maps.b, bar, kb * C::BK, col);
            } else {
              // LoRA operands, 64 wide (the MMAs read the rank's): half kb - nkb of the pair, and A [BNC
              // columns, r] K-major (dX) or B [r, BNC columns] MN-major in chunks of 64 columns (forward)
              tma_load_2d_pair(a, &maps.la, bar, (kb - args.nkb) * args.lora_k16 * 16, m0);
              if (BWD) {
                tma_load_2d_pair(b, &maps.lb, bar, 0, col);
              } else {
                for (int c = 0; c < C::BNC / 64; ++c) tma_load_2d_pair(b + c * 8192, &maps.lb, bar, col + c * 64, 0);
              }
            }
          }
          __syncwarp();
          if (++s == C::S) s = 0, ph ^= 1;
        }
      }
      if (!ok) settle_inflight();  // loads already issued land before the CTA can exit
    } else if (warp == 1 && rank == 0) {
      // --------------------------------------------------------- MMA -----
      // Descriptors and phases are carried along: this loop is one serial chain.
      bool ok = true;
      constexpr uint32_t idesc = idesc_e4m3(2 * C::BM, C::BNT, false, BWD);
      constexpr uint32_t idesc_lora = idesc_bf16(2 * C::BM, C::BNT, false, !BWD);
      const uint64_t ad0 = smem_desc(sbase + C::OFF_A, 16, 1024, QL_SWZ_128B);
      // W for dX: reduction rows of BNC bytes (MN-major, one swizzle atom wide)
      const uint64_t bd0 = BWD ? smem_desc(sbase + C::OFF_B, C::B_BYTES, 8 * C::BNC, C::BNC == 128 ? QL_SWZ_128B : QL_SWZ_64B)
                               : smem_desc(sbase + C::OFF_B, 16, 1024, QL_SWZ_128B);
      const uint64_t bl0 = smem_desc(sbase + C::OFF_B, BWD ? 16 : 8192, 1024, QL_SWZ_128B);
      int s = 0, b = 0;
      uint32_t ph = 0, aph = 1;  // phases of the operand ring and of the accumulators
      for (int u = cluster; u < units && ok; u += clusters) {
        int m0, n0, k0, k1;
        unit_coords(u, m0, n0, k0, k1);
        for (int kb = k0; kb < k1; ++kb) {
          ok = mbar_wait(full_bar(s), ph, args.status) && mbar_wait(acc_empty0 + 8u * b, aph, args.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t acc = tmem + b * C::BNT;
            const uint64_t ao = static_cast<uint64_t>(s) * (C::A_BYTES >> 4), bo = static_cast<uint64_t>(s) * (C::B_BYTES >> 4);
            if (kb < args.nkb) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 32 reduction elements each
                umma_e4m3<2>(acc, ad0 + ao + kk * 2, bd0 + bo + kk * (BWD ? 2 * C::BNC : 2), idesc, kk != 0);
            } else {
              for (int kk = 0; kk < args.lora_k16; ++kk)
                umma_bf16<2>(acc, ad0 + ao + kk * 2, bl0 + bo + kk * (BWD ? 2 : 128), idesc_lora, kk != 0);
            }
            umma_commit<2>(empty_bar(s));
            umma_commit<2>(acc_full0 + 8u * b);
          }
          __syncwarp();
          if (++s == C::S) s = 0, ph ^= 1;
          if (++b == C::ACCS) b = 0, aph ^= 1;
        }
      }
      // let every issued MMA finish before TMEM can be released (after an error too)
      if (elect_one()) umma_commit<2>(drain_bar);
      __syncwarp();
      mbar_drain(drain_bar, 0);
    } else if (warp == 2) {
      // ------------------------------------------------------ scales -----
      // G blocks' scales are requested at once and written as their operand stages come free.  The
      // arrival on the stage's full barrier orders them before the block's MMA, and so before its
      // accumulator is handed over.  Rows past the last one add zeros: any scale will do.
      bool ok = true;
      int s = 0, sl = 0;
      uint32_t ph = 1;
      for (int u = cluster; u < units && ok; u += clusters) {
        int m0, n0, k0, k1;
        unit_coords(u, m0, n0, k0, k1);
        const int nb = min(n0 / 128 + (lane & 1), (args.N - 1) / 128);
        const float* sb = args.sb + static_cast<size_t>(nb) * args.sb_n;
        for (int kb = k0; kb < k1 && ok; kb += C::G) {
          float va[C::G][4];
#pragma unroll
          for (int g = 0; g < C::G; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = m0 + i * 32 + lane;
              va[g][i] = kb + g < args.nkb && row < args.M
                             ? __ldg(args.sa + static_cast<size_t>(kb + g) * args.M + row)
                             : 1.f;
            }
          const int kw = kb + (lane >> 1);
          const float vb = lane < 2 * C::G && kw < args.nkb ? __ldg(sb + static_cast<size_t>(kw) * args.sb_k) : 1.f;
#pragma unroll
          for (int g = 0; g < C::G; ++g) {
            if (kb + g >= k1) break;
            ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(s), ph, args.status));
            if (!ok) break;
            const float w0 = __shfl_sync(0xffffffffu, vb, 2 * g), w1 = __shfl_sync(0xffffffffu, vb, 2 * g + 1);
            float* d = scales + sl * C::SC_FLOATS + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              d[i * 32] = va[g][i] * w0;
              if constexpr (C::NBLK == 2) d[C::BM + i * 32] = va[g][i] * w1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead0 + 8u * s);
            if (++s == C::S) s = 0, ph ^= 1;
            if (++sl == C::SR) sl = 0;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------ accumulate ---
    setmaxnreg_inc<C::REGS_EPI>();
    const int ew = warp - C::EPI_WARP0;
    const int lg = warp & 3;    // TMEM lane quadrant this warp may access
    const int half = ew >> 2;   // its BNC columns of the tile: one weight scale per reduction block
    const uint32_t stg = sbase + C::OFF_EPI + ew * C::EPI_SLOT;
    uint8_t* stg_g = sgen + C::OFF_EPI + ew * C::EPI_SLOT;
    const uint64_t pol = l2_policy_evict_first();
    const float* my_scale = scales + (C::NBLK == 2 ? half * C::BM : 0) + lg * 32 + lane;
    int b = 0, sl = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = cluster; u < units && ok; u += clusters) {
      int m0, n0, k0, k1;
      unit_coords(u, m0, n0, k0, k1);
      float acc[C::BNC];
#pragma unroll
      for (int i = 0; i < C::BNC; ++i) acc[i] = 0.f;
      for (int kb = k0; kb < k1; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full0 + 8u * b, ph, args.status));
        if (!ok) break;
        tc_fence_after();
        const float sc = my_scale[sl * C::SC_FLOATS];
        if (++sl == C::SR) sl = 0;
        const uint32_t tacc = tmem + b * C::BNT + half * C::BNC + (static_cast<uint32_t>(lg * 32) << 16);
        uint32_t v[2][32];  // 32 columns are loaded while the previous 32 are added
        tmem_ld_32x32b_x32_async(tacc, v[0]);
#pragma unroll
        for (int c = 0; c < C::BNC / 32; ++c) {
          tmem_wait_ld(v[c & 1]);
          if (c + 1 < C::BNC / 32) {
            tmem_ld_32x32b_x32_async(tacc + (c + 1) * 32, v[(c + 1) & 1]);
          } else {  // every value is in registers: the MMA may have the accumulator back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead0 + (acc_empty0 - bar0) + 8u * b);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c * 32 + i] = fmaf(__uint_as_float(v[c & 1][i]), sc, acc[c * 32 + i]);
        }
        if (++b == C::ACCS) b = 0, ph ^= 1;
      }
      if (!ok) break;
      if (args.splits > 1) {
        // a part's fp32 sums, in 16 x 32 chunks (128B swizzle) into its own rows of the partials
        const int prow = (u % args.splits) * args.prows + m0 + lg * 32;
#pragma unroll
        for (int c = 0; c < C::BNC / 32; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            if ((lane >> 4) == h) {
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float* v = acc + c * 32 + q * 4;
                *reinterpret_cast<float4*>(stg_g + (lane & 15) * 128 + ((q ^ (lane & 7)) << 4)) =
                    make_float4(v[0], v[1], v[2], v[3]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.part, stg, n0 + half * C::BNC + c * 32, prow + h * 16, pol);
              bulk_commit_group();
            }
          }
        }
        continue;
      }
      // 32 x 32 chunks through this warp's shared slot (64B swizzle); the TMA store clips at the edges
#pragma unroll
      for (int c = 0; c < C::BNC / 32; ++c) {
        if (lane == 0) bulk_wait_group_read<0>();  // the previous chunk's store has read the slot
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float* v = acc + c * 32 + q * 8;
          *reinterpret_cast<uint4*>(stg_g + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&maps.out, stg, n0 + half * C::BNC + c * 32, m0 + lg * 32, pol);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();  // output stores complete before the CTA exits
  }

  // ------------------------------------------------------------ teardown --
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem, C::TMEM_COLS);
  }
}

template <bool BWD, int BN>
static cudaError_t launch_one8(const Gemm8Maps& maps, const Gemm8Args& args, cudaStream_t stream) {
  using C = Gemm8Cfg<BN>;
  auto kern = gemm_fp8_kernel<BWD, BN>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static int resident[64] = {0};  // co-resident CTAs (even) per device
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (!resident[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int n = sms / 2, clusters = 0;
    cfg.gridDim = dim3(static_cast<unsigned>(sms - sms % 2), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0 && clusters < n)
      n = clusters;
    cudaGetLastError();
    resident[dev] = n * 2;
  }
  const int total = ((args.M + 255) / 256) * ((args.N + BN - 1) / BN) * args.splits;
  const int ctas = apply_grid_cap(total * 2 < resident[dev] ? total * 2 : resident[dev], 2);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, maps, args);
}

// out[m, n] = sum of the parts in order; eight columns per thread.
__global__ void __launch_bounds__(256) gemm_fp8_sum_kernel(const float* __restrict__ part, int64_t prows, int splits,
                                                           int64_t N, int64_t total, bf16* __restrict__ out,
                                                           int* status) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= total || !dev_check(splits > 1 && i + 8 <= total && total <= prows * N, status)) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4* p = reinterpret_cast<const float4*>(part + s * prows * N + i);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
cudaError_t launch_gemm_fp8_sum(const float* part, int64_t prows, int splits, int64_t M, int64_t N, bf16* out,
                                int* status, cudaStream_t st) {
  return launch_pdl(gemm_fp8_sum_kernel, dim3(static_cast<unsigned>((M * N / 8 + 255) / 256)), dim3(256), 0, st, part,
                    prows, splits, N, M * N, out, status);
}

// bn: output columns per tile (256 or 128); the tensor maps' boxes follow it.
cudaError_t launch_gemm_fp8(bool bwd, int bn, const Gemm8Maps& maps, const Gemm8Args& args, cudaStream_t stream) {
  if (bn == 256) return bwd ? launch_one8<true, 256>(maps, args, stream) : launch_one8<false, 256>(maps, args, stream);
  if (bn == 128) return bwd ? launch_one8<true, 128>(maps, args, stream) : launch_one8<false, 128>(maps, args, stream);
  return cudaErrorInvalidValue;
}

}  // namespace ql
