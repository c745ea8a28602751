// The passes of an e4m3 LoRA projection around its products, over T [M, C]:
//   forward   q(X), XA = X A                       (PASS_FWD, any M)
//   backward  q(dY), G = dY B^T, dB = s XA^T dY    (PASS_DY, M <= 64)
//             dA = X^T (s G)                       (PASS_DA, M <= 64)
// each in one launch that reads T once, for the row counts that launches bound: the
// general path runs a quantiser, one or two passes with fp32 partials and a reduction
// for each of them (64 rows, rank 64, 4096 -> 1024: 12 launches a step, 44 us; here 5,
// 32 us).  s X A and s G leave as pairs of bf16 numbers (the rounded sum and what the
// rounding leaves, 16 bits together) for the products that go on from them.
//
// A cluster takes 64 rows.  T comes in blocks of 128 columns, staged in shared
// memory together with the low-rank factor's block (the next blocks' copies are on
// their way meanwhile).  From there a block is quantised (fp8.cuh), multiplied into
// the low-rank sums and used for the outer product, all with warp-level MMAs.  The
// blocks are dealt to the cluster's CTAs, whose low-rank sums meet through
// distributed shared memory and are added in rank order: no partials in memory, no
// reduction launch, and nothing depends on timing.
#include "fp8.cuh"

namespace ql {

constexpr int FW_ROWS = 64, FW_R = 64, FW_THREADS = 256;
constexpr int FW_TP = 128 + 8;                 // row pitch of a staged block (elements): no bank conflicts
constexpr int FW_T_BYTES = FW_ROWS * FW_TP * 2;
constexpr int FW_STAGES = 4;
enum PassMode : int { PASS_FWD = 0, PASS_DY = 1, PASS_DA = 2 };
// Bytes of a stage (a block of T and of the factor: [128][r + 8] forward, [r][128 + 8] backward), of U
// ([64][r + 8], the pair [64][2 r + 8] for dA), and of the low-rank sums [64][r + 8] of the four reduction
// shares, which take the stages' place once these are done with.
__host__ __device__ constexpr int fw_stage_bytes(int mode, int r) {
  return FW_T_BYTES + (mode == PASS_FWD ? 128 * (r + 8) * 2 : (mode == PASS_DA ? 0 : r * FW_TP * 2));
}
__host__ __device__ constexpr int fw_u_bytes(int mode, int r) {
  return mode == PASS_FWD ? 0 : FW_ROWS * ((mode == PASS_DA ? 2 * r : r) + 8) * 2;
}
__host__ __device__ constexpr int fw_smem(int mode, int r) {
  return FW_STAGES * fw_stage_bytes(mode, r) + fw_u_bytes(mode, r);
}
static_assert(4 * FW_ROWS * (FW_R + 8) * 4 <= FW_STAGES * fw_stage_bytes(PASS_DY, FW_R) &&
                  4 * FW_ROWS * (16 + 8) * 4 <= FW_STAGES * FW_T_BYTES && fw_smem(PASS_DY, FW_R) <= 232448,
              "the shares fit over the stages, and everything into shared memory");

struct RankPass {
  const bf16* T;     // [M, C]
  int M, C, r;
  uint8_t* codes;    // q(T): [M, C]; null: not wanted
  float* tscale;     // [ceil(C / 128), M]
  const bf16* V;     // low-rank factor: A [C, r] (forward) or B [r, C] (backward)
  bf16 *low, *lows;  // T V [M, r] and scale * T V [M, 2 r] (the pair); either may be null
  const bf16* U;     // [M, r]: XA, or [M, 2 r]: the pair of s G
  bf16* outer;       // dB [r, C] (scaled) or dA [C, r]
  float scale;
  int cluster;       // CTAs per 64 rows
  int* status;       // device status word (the checked build's checks report there)
};

QL_DEV void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

template <int MODE>
__global__ void __launch_bounds__(FW_THREADS) fp8_rank_pass_kernel(const RankPass a) {
  extern __shared__ __align__(16) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int mi = lane >> 3, mr = lane & 7;  // matrix and row that this lane addresses in an ldmatrix
  const int m0 = static_cast<int>(blockIdx.x / a.cluster) * FW_ROWS;  // the cluster's rows
  const int M = min(FW_ROWS, a.M - m0);
  const int mt = (M + 15) / 16;             // row tiles
  const int nb = (a.C + 127) / 128;
  const int first = blockIdx.x % a.cluster, step = a.cluster;
  const int r = a.r, lr = __ffs(r) - 1, lc = lr - 3;  // r is 16, 32 or 64: chunks of 8 by shifts
  const int stage_bytes = fw_stage_bytes(MODE, r);
  const bf16* T = a.T + static_cast<size_t>(m0) * a.C;
  grid_dep_wait();
  grid_dep_launch();
  if (!dev_check(M > 0 && a.C > 0 && (r == 16 || r == 32 || r == 64) && (MODE == PASS_FWD || a.M <= FW_ROWS) &&
                     (MODE == PASS_DA || a.cluster <= 16) &&
                     static_cast<int>(gridDim.x) == (a.M + FW_ROWS - 1) / FW_ROWS * a.cluster,
                 a.status))
    return;

  // block kb of T (rows past M and columns past C as zeros) and of V into buffer b
  auto stage = [&](int kb, int b) {
    const int c0 = kb * 128;
    for (int i = tid; i < mt * 16 * 16; i += FW_THREADS) {
      const int m = i >> 4, c = (i & 15) * 8;
      const bool in = m < M && c0 + c < a.C;
      cp_async16(sb + b * stage_bytes + (m * FW_TP + c) * 2, T + (in ? static_cast<size_t>(m) * a.C + c0 + c : 0), in);
    }
    const uint32_t v = sb + b * stage_bytes + FW_T_BYTES;
    if constexpr (MODE == PASS_FWD) {  // [128][r + 8]
      for (int i = tid; i < 128 << lc; i += FW_THREADS) {
        const int k = i >> lc, c = (i - (k << lc)) * 8;
        const bool in = c0 + k < a.C;
        cp_async16(v + (k * (r + 8) + c) * 2, a.V + (in ? static_cast<size_t>(c0 + k) * r + c : 0), in);
      }
    } else if constexpr (MODE != PASS_DA) {  // [r][128 + 8]
      for (int i = tid; i < r * 16; i += FW_THREADS) {
        const int j = i >> 4, c = (i & 15) * 8;
        const bool in = c0 + c < a.C;
        cp_async16(v + (j * FW_TP + c) * 2, a.V + (in ? static_cast<size_t>(j) * a.C + c0 + c : 0), in);
      }
    }
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

  const uint32_t us = sb + FW_STAGES * stage_bytes;
  const int ur = MODE == PASS_DA ? 2 * r : r, ulc = MODE == PASS_DA ? lc + 1 : lc;  // U's columns
  if constexpr (MODE != PASS_FWD) {
    for (int i = tid; i < (mt * 16) << ulc; i += FW_THREADS) {
      const int m = i >> ulc, c = (i - (m << ulc)) * 8;
      cp_async16(us + (m * (ur + 8) + c) * 2, a.U + (m < M ? static_cast<size_t>(m) * ur + c : 0), m < M);
    }
  }
  for (int s = 0; s < FW_STAGES - 1; ++s) {  // a group per stage, empty past the last block
    if (first + s * step < nb) stage(first + s * step, s);
    commit();
  }

  // low-rank sums: warps split a block's 8 reduction steps (two each, by warp & 3) and the factor's columns in two
  const int kq = warp & 3, jh = warp >> 2, jt = r / 16;  // jt tiles of 8 columns per half
  float acc[4][4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][j][i] = 0.f;

  int b = 0;
  for (int kb = first; kb < nb; kb += step, b = (b + 1) % FW_STAGES) {
    const int ahead = kb + (FW_STAGES - 1) * step;
    if (ahead < nb) stage(ahead, (b + FW_STAGES - 1) % FW_STAGES);
    commit();
    asm volatile("cp.async.wait_group %0;" ::"n"(FW_STAGES - 1) : "memory");  // this block's copies have landed
    __syncthreads();
    const uint32_t ts = sb + b * stage_bytes, vs = ts + FW_T_BYTES;

    if constexpr (MODE != PASS_DA) {
      // 8-bit rows (unless the caller has them): half a warp per row of the block, four rows in flight
      if (a.codes) {
        const int h = lane >> 4, c = (lane & 15) * 8, col = kb * 128 + c;
        uint4 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // rows past the staged ones hold stale bytes that nothing below uses
          u[i] = *reinterpret_cast<const uint4*>(sm + b * stage_bytes + ((i * 16 + warp * 2 + h) * FW_TP + c) * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = i * 16 + warp * 2 + h;
          float f[8], s, inv;
          unpack_bf16x8(u[i], f);
          fp8_scale(half_warp_max(absmax8(f)), s, inv);
          if (m < M) {
            if (col < a.C) *reinterpret_cast<uint2*>(a.codes + static_cast<size_t>(m0 + m) * a.C + col) = e4m3x8(f, inv);
            if (c == 0) a.tscale[static_cast<size_t>(kb) * a.M + m0 + m] = s;
          }
        }
      }
      // T V
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k0 = (kq * 2 + s) * 16;
        uint32_t bf[4][2];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          if (j >= jt) break;
          const int n0 = (jh * jt + j) * 8;
          if (jt == 1) {  // rank 16: one tile per half
            if constexpr (MODE == PASS_FWD)
              ldsm_x2_t(vs + ((k0 + (mi & 1) * 8 + mr) * (r + 8) + n0) * 2, bf[0][0], bf[0][1]);
            else
              ldsm_x2(vs + ((n0 + mr) * FW_TP + k0 + (mi & 1) * 8) * 2, bf[0][0], bf[0][1]);
          } else {
            if constexpr (MODE == PASS_FWD)
              ldsm_x4_t(vs + ((k0 + (mi & 1) * 8 + mr) * (r + 8) + n0 + (mi >> 1) * 8) * 2, bf[j][0], bf[j][1],
                        bf[j + 1][0], bf[j + 1][1]);
            else
              ldsm_x4(vs + ((n0 + (mi >> 1) * 8 + mr) * FW_TP + k0 + (mi & 1) * 8) * 2, bf[j][0], bf[j][1],
                      bf[j + 1][0], bf[j + 1][1]);
          }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if (t >= mt) break;
          uint32_t a0, a1, a2, a3;
          ldsm_x4(ts + ((t * 16 + (lane & 15)) * FW_TP + k0 + (lane >> 4) * 8) * 2, a0, a1, a2, a3);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < jt) mma_bf16_16816(acc[t][j], a0, a1, a2, a3, bf[j][0], bf[j][1]);
        }
      }
    }
    const int g = lane >> 2, q = lane & 3;
    if constexpr (MODE == PASS_DY) {
      // dB = scale U^T T: r rows x this warp's 16 columns of the block, reduction over T's rows
      float o[4][2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][0][i] = o[j][1][i] = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t >= mt) break;
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(ts + ((t * 16 + (mi & 1) * 8 + mr) * FW_TP + warp * 16 + (mi >> 1) * 8) * 2, b0, b1, b2, b3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j * 16 >= r) break;
          uint32_t a0, a1, a2, a3;
          ldsm_x4_t(us + ((t * 16 + (mi >> 1) * 8 + mr) * (r + 8) + j * 16 + (mi & 1) * 8) * 2, a0, a1, a2, a3);
          mma_bf16_16816(o[j][0], a0, a1, a2, a3, b0, b1);
          mma_bf16_16816(o[j][1], a0, a1, a2, a3, b2, b3);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j * 16 >= r) break;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int col = kb * 128 + warp * 16 + n * 8 + q * 2;
          if (col >= a.C) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint32_t*>(a.outer + static_cast<size_t>(j * 16 + h * 8 + g) * a.C + col) =
                pack_bf16x2(o[j][n][2 * h] * a.scale, o[j][n][2 * h + 1] * a.scale);
        }
      }
    }
    if constexpr (MODE == PASS_DA) {
      // dA = T^T U: this warp's 16 columns of the block x r
      float o[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t >= mt) break;
        uint32_t a0, a1, a2, a3;
        ldsm_x4_t(ts + ((t * 16 + (mi >> 1) * 8 + mr) * FW_TP + warp * 16 + (mi & 1) * 8) * 2, a0, a1, a2, a3);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          if (j * 8 >= r) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the pair's halves
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(us + ((t * 16 + (mi & 1) * 8 + mr) * (ur + 8) + h * r + j * 8 + (mi >> 1) * 8) * 2, b0, b1, b2, b3);
            mma_bf16_16816(o[j], a0, a1, a2, a3, b0, b1);
            mma_bf16_16816(o[j + 1], a0, a1, a2, a3, b2, b3);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j * 8 >= r) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = kb * 128 + warp * 16 + h * 8 + g;
          if (n < a.C)
            *reinterpret_cast<uint32_t*>(a.outer + static_cast<size_t>(n) * r + j * 8 + q * 2) =
                pack_bf16x2(o[j][2 * h], o[j][2 * h + 1]);
        }
      }
    }
    __syncthreads();  // the buffer may be staged again
  }

  if constexpr (MODE != PASS_DA) {
    float* part = reinterpret_cast<float*>(sm);  // [share][row][pp]
    const int pp = r + 8;
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t >= mt) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= jt) break;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(part + kq * (FW_ROWS * pp) + (t * 16 + h * 8 + g) * pp + (jh * jt + j) * 8 + q * 2) =
              make_float2(acc[t][j][2 * h], acc[t][j][2 * h + 1]);
      }
    }
    __syncthreads();
    // this CTA's sum, in share 0
    const int quads = M << (lr - 2);
    for (int e = tid; e < quads; e += FW_THREADS) {
      const int m = e >> (lr - 2), c = (e - (m << (lr - 2))) * 4;
      float4* p = reinterpret_cast<float4*>(part + m * pp + c);
      float4 v = *p;
#pragma unroll
      for (int k = 1; k < 4; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(part + k * (FW_ROWS * pp) + m * pp + c);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      *p = v;
    }
    cluster_sync();
    const int ranks = a.cluster;
    for (int e = tid + FW_THREADS * first; e < quads; e += FW_THREADS * ranks) {
      const int m = e >> (lr - 2), c = (e - (m << (lr - 2))) * 4;
      const uint32_t at = sb + (m * pp + c) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c0 = 0; c0 < ranks; c0 += 8) {  // eight ranks' loads in flight, added in rank order
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = c0 + i < ranks ? ld_cluster_f32x4(mapa_shared(at, static_cast<uint32_t>(c0 + i)))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v.x += x[i].x, v.y += x[i].y, v.z += x[i].z, v.w += x[i].w;
      }
      if (a.low)
        *reinterpret_cast<uint2*>(a.low + static_cast<size_t>(m0 + m) * r + c) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      if (a.lows) {
        bf16* o = a.lows + static_cast<size_t>(m0 + m) * 2 * r + c;
        v.x *= a.scale, v.y *= a.scale, v.z *= a.scale, v.w *= a.scale;
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        *reinterpret_cast<uint2*>(o + r) = make_uint2(pack_bf16x2(bf16_rest(v.x), bf16_rest(v.y)),
                                                      pack_bf16x2(bf16_rest(v.z), bf16_rest(v.w)));
      }
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
  }
}

template <int MODE>
static cudaError_t launch_pass(RankPass a, int sms, cudaStream_t st) {
  auto kern = fp8_rank_pass_kernel<MODE>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(FW_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  static int widest[64] = {0};  // CTAs of the widest cluster this device takes: 16 (opt-in) or 8
  if (!widest[dev]) {
    cfg.dynamicSmemBytes = fw_smem(MODE, FW_R);
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes));
    if (e != cudaSuccess) return e;
    int n = 0;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(16);
    attr[0].val.clusterDim.x = 16;
    const bool wide = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
    cudaGetLastError();
    widest[dev] = wide ? 16 : 8;
  }
  // CTAs per 64 rows: enough to fill the device, at most one per block of columns
  const int nb = (a.C + 127) / 128, groups = (a.M + FW_ROWS - 1) / FW_ROWS;
  a.cluster = 1;
  if (MODE == PASS_DA) a.cluster = nb;  // no sums to share: plain CTAs
  else
    while (a.cluster * 2 <= nb && a.cluster * 2 <= widest[dev] && groups * a.cluster < sms) a.cluster *= 2;
  attr[0].val.clusterDim.x = MODE == PASS_DA ? 1 : a.cluster;
  cfg.numAttrs = 2;
  cfg.dynamicSmemBytes = fw_smem(MODE, a.r);
  cfg.gridDim = dim3(static_cast<unsigned>(groups) * a.cluster);
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// q(X) and XA (low), the pair of s XA (lows)
cudaError_t launch_pass_fwd(const bf16* X, int M, int K, const bf16* A, int r, float scale, uint8_t* codes, float* tscale,
                            bf16* low, bf16* lows, int sms, int* status, cudaStream_t st) {
  return launch_pass<PASS_FWD>({X, M, K, r, codes, tscale, A, low, lows, nullptr, nullptr, scale, 1, status}, sms, st);
}
// q(dY), the pair of s G (lows) and dB = s XA^T dY, M <= 64
cudaError_t launch_pass_dy(const bf16* dY, int M, int N, const bf16* B, int r, float scale, uint8_t* codes, float* tscale,
                           bf16* lows, const bf16* XA, bf16* dB, int sms, int* status, cudaStream_t st) {
  if (M > FW_ROWS) return cudaErrorInvalidValue;
  return launch_pass<PASS_DY>({dY, M, N, r, codes, tscale, B, nullptr, lows, XA, dB, scale, 1, status}, sms, st);
}
// dA = X^T (s G) from the pair of s G, M <= 64
cudaError_t launch_pass_da(const bf16* X, int M, int K, const bf16* sG, int r, bf16* dA, int sms, int* status,
                           cudaStream_t st) {
  if (M > FW_ROWS) return cudaErrorInvalidValue;
  return launch_pass<PASS_DA>({X, M, K, r, nullptr, nullptr, nullptr, nullptr, nullptr, sG, dA, 1.f, 1, status}, sms, st);
}

}  // namespace ql
