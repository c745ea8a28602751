// Residual addition and RMS norm in one pass, forward and backward:
//   h = bf16(x + r),  rstd = 1 / sqrt(mean_j h_j^2 + eps),  y = bf16(h * rstd * g),  g = w or 1 + w,
//   codes, scale = the 8-bit row format of y (fp8.cuh),
//   dx_j = dh_j + rstd * (g_j dy_j - n_j * mean_i(n_i g_i dy_i)),  n = h * rstd  (the norm weight is frozen).
// dx is the gradient of x and of r alike; dh is the gradient that reaches h past
// the norm (the residual stream's own).
//
// HBM-bound row kernels.  T threads hold one row in registers (16-byte loads,
// all in flight at once), so every tensor is read or written once; 16
// neighbouring threads hold one block of 128 columns, whose largest magnitude is
// a half-warp shuffle.  Squares and their sum are in binary64: a finite row keeps its
// norm whatever its size (binary32 squares end at 2^64 and 2^-75), and rstd is the
// correctly rounded value in nearly every row whatever the order of the sum, so y
// and the 8-bit codes next to a rounding border do not depend on T (49 million
// rows of 8 to 1024 columns against torch's binary64 mean: no rstd differed).  eps
// is the binary32 number that the call takes: computing with a binary64 1e-5
// instead changes the last bit of rstd in one row of a million.
#include "fp8.cuh"

namespace ql {

QL_DEV double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
QL_DEV float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the T threads of a row, in a fixed order.
template <int T, typename V>
QL_DEV V row_sum(V v, V* red) {
  if constexpr (sizeof(V) == 8) v = warp_sum_d(v); else v = warp_sum_f(v);
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < T / 32; ++i) v += red[i];
  }
  return v;
}
QL_DEV void norm_gain8(const bf16* w, int c, int plus_one, float (&g)[8]) {
  unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(w + c)), g);
  if (plus_one) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] += 1.0f;
  }
}
// x + r rounded to bf16 (h), eight elements.
QL_DEV uint4 add_bf16x8(const uint4& a, const uint4& b) {
  float x[8], r[8];
  unpack_bf16x8(a, x);
  unpack_bf16x8(b, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] += r[i];
  return pack_bf16x8(x);
}
QL_DEV void add_squares(const uint4& v, double& ss) {
  float f[8];
  unpack_bf16x8(v, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double x = f[i];
    ss = fma(x, x, ss);
  }
}
// h -> y for eight elements; returns y as bf16, and as floats for the 8-bit output.
QL_DEV uint4 norm8(const uint4& h, float rstd, const float (&g)[8], float (&y)[8]) {
  unpack_bf16x8(h, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * g[i];
  const uint4 u = pack_bf16x8(y);
  unpack_bf16x8(u, y);  // the codes are those of the rounded row
  return u;
}

struct AddNormFwd {
  const bf16 *X, *R, *w;  // R may be null: h = x
  int M, d, plus_one;
  float eps;
  bf16 *H, *Y;      // either may be null (H is, where R is)
  uint8_t* codes;   // null: no 8-bit output
  float *scale, *rstd;  // scale [ceil(d / 128), M]
};

// One row per T threads, at most NCH 16-byte chunks per thread (d <= 8 * T * NCH).
// x and r are read with plain loads, all of them before the row's first store:
// H may be X or R.
template <int T, int NCH>
__global__ void __launch_bounds__(T < 128 ? 128 : T) add_rmsnorm_fwd_kernel(const AddNormFwd a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int ROWS = T < 128 ? 128 / T : 1;
  __shared__ double red[T / 32];
  const int t = threadIdx.x % T;
  const int row = blockIdx.x * ROWS + threadIdx.x / T;
  if (row >= a.M) return;  // only where T = 32: whole warps
  const size_t off = static_cast<size_t>(row) * a.d;
  uint4 v[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * T + t) * 8;
    v[i] = c < a.d ? *reinterpret_cast<const uint4*>(a.X + off + c) : make_uint4(0, 0, 0, 0);
  }
  if (a.R) {
    uint4 r[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * T + t) * 8;
      r[i] = c < a.d ? *reinterpret_cast<const uint4*>(a.R + off + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * T + t) * 8;
      v[i] = add_bf16x8(v[i], r[i]);
      if (a.H && c < a.d) *reinterpret_cast<uint4*>(a.H + off + c) = v[i];
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NCH; ++i) add_squares(v[i], ss);
  ss = row_sum<T>(ss, red);
  const float rstd = static_cast<float>(1.0 / sqrt(ss / a.d + static_cast<double>(a.eps)));
  if (t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * T + t) * 8;
    const bool in = c < a.d;
    float g[8], y[8];
    if (in) {
      norm_gain8(a.w, c, a.plus_one, g);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = 0.f;
    }
    const uint4 u = norm8(v[i], rstd, g, y);
    if (a.Y && in) *reinterpret_cast<uint4*>(a.Y + off + c) = u;
    if (a.codes) {
      float s, inv;
      fp8_scale(half_warp_max(in ? absmax8(y) : 0.f), s, inv);
      if (in) {
        *reinterpret_cast<uint2*>(a.codes + off + c) = e4m3x8(y, inv);
        if ((c & (kFp8Block - 1)) == 0) a.scale[static_cast<size_t>(c / kFp8Block) * a.M + row] = s;
      }
    }
  }
}

// Rows too wide for registers: one CTA per row, two passes; the second reads h
// back (or x, where there is no r) from the cache.
constexpr int AN_WIDE = 512;
__global__ void __launch_bounds__(AN_WIDE) add_rmsnorm_fwd_wide_kernel(const AddNormFwd a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ double red[AN_WIDE / 32];
  const int row = blockIdx.x;
  const size_t off = static_cast<size_t>(row) * a.d;
  auto h_at = [&](int c) {
    const uint4 x = *reinterpret_cast<const uint4*>(a.X + off + c);
    return a.R ? add_bf16x8(x, *reinterpret_cast<const uint4*>(a.R + off + c)) : x;
  };
  double ss = 0.0;
#pragma unroll 2
  for (int c = threadIdx.x * 8; c < a.d; c += AN_WIDE * 8) {
    const uint4 h = h_at(c);
    if (a.H) *reinterpret_cast<uint4*>(a.H + off + c) = h;
    add_squares(h, ss);
  }
  ss = row_sum<AN_WIDE>(ss, red);
  const float rstd = static_cast<float>(1.0 / sqrt(ss / a.d + static_cast<double>(a.eps)));
  if (threadIdx.x == 0) a.rstd[row] = rstd;
  for (int c0 = 0; c0 < a.d; c0 += AN_WIDE * 8) {  // every lane takes each step: the block maximum is a shuffle
    const int c = c0 + threadIdx.x * 8;
    const bool in = c < a.d;
    float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, y[8];
    uint4 h = make_uint4(0, 0, 0, 0);
    if (in) {
      norm_gain8(a.w, c, a.plus_one, g);
      h = a.H ? *reinterpret_cast<const uint4*>(a.H + off + c) : h_at(c);
    }
    const uint4 u = norm8(h, rstd, g, y);
    if (a.Y && in) *reinterpret_cast<uint4*>(a.Y + off + c) = u;
    if (a.codes) {
      float s, inv;
      fp8_scale(half_warp_max(in ? absmax8(y) : 0.f), s, inv);
      if (in) {
        *reinterpret_cast<uint2*>(a.codes + off + c) = e4m3x8(y, inv);
        if ((c & (kFp8Block - 1)) == 0) a.scale[static_cast<size_t>(c / kFp8Block) * a.M + row] = s;
      }
    }
  }
}

struct AddNormBwd {
  const bf16 *H, *w;
  const float* rstd;
  const bf16 *dY, *dH;  // dH may be null: nothing reaches h past the norm
  int M, d, plus_one;
  bf16* dX;             // may be dY or dH
};

// n = h * rstd comes first: it is of the order of 1 where h, rstd or rstd^2 may leave binary32
QL_DEV float dot_ngdy(const uint4& h, const uint4& dy, const float (&g)[8], float rstd, float acc) {
  float f[8], e[8];
  unpack_bf16x8(h, f);
  unpack_bf16x8(dy, e);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc = fmaf(f[i] * rstd, g[i] * e[i], acc);
  return acc;
}
// dh + rstd * (g dy - h * cm), cm = rstd * mean(n g dy)
QL_DEV uint4 norm_bwd8(const uint4& h, const uint4& dy, const uint4& dh, const float (&g)[8], float rstd, float cm) {
  float f[8], e[8], o[8];
  unpack_bf16x8(h, f);
  unpack_bf16x8(dy, e);
  unpack_bf16x8(dh, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] += rstd * (g[i] * e[i] - f[i] * cm);
  return pack_bf16x8(o);
}

template <int T, int NCH>
__global__ void __launch_bounds__(T < 128 ? 128 : T) add_rmsnorm_bwd_kernel(const AddNormBwd a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int ROWS = T < 128 ? 128 / T : 1;
  __shared__ float red[T / 32];
  const int t = threadIdx.x % T;
  const int row = blockIdx.x * ROWS + threadIdx.x / T;
  if (row >= a.M) return;  // only where T = 32: whole warps
  const size_t off = static_cast<size_t>(row) * a.d;
  const float rstd = a.rstd[row];
  uint4 h[NCH], dy[NCH], dh[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * T + t) * 8;
    const bool in = c < a.d;
    const uint4 z = make_uint4(0, 0, 0, 0);
    h[i] = in ? *reinterpret_cast<const uint4*>(a.H + off + c) : z;
    dy[i] = in ? *reinterpret_cast<const uint4*>(a.dY + off + c) : z;
    dh[i] = in && a.dH ? *reinterpret_cast<const uint4*>(a.dH + off + c) : z;
  }
  float acc = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * T + t) * 8;
    if (c >= a.d) break;
    float g[8];
    norm_gain8(a.w, c, a.plus_one, g);
    acc = dot_ngdy(h[i], dy[i], g, rstd, acc);
  }
  acc = row_sum<T>(acc, red);
  const float cm = rstd * __fdiv_rn(acc, static_cast<float>(a.d));
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * T + t) * 8;
    if (c >= a.d) break;
    float g[8];
    norm_gain8(a.w, c, a.plus_one, g);
    *reinterpret_cast<uint4*>(a.dX + off + c) = norm_bwd8(h[i], dy[i], dh[i], g, rstd, cm);
  }
}

__global__ void __launch_bounds__(AN_WIDE) add_rmsnorm_bwd_wide_kernel(const AddNormBwd a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ float red[AN_WIDE / 32];
  const int row = blockIdx.x;
  const size_t off = static_cast<size_t>(row) * a.d;
  const float rstd = a.rstd[row];
  float acc = 0.f;
#pragma unroll 2
  for (int c = threadIdx.x * 8; c < a.d; c += AN_WIDE * 8) {
    float g[8];
    norm_gain8(a.w, c, a.plus_one, g);
    acc = dot_ngdy(*reinterpret_cast<const uint4*>(a.H + off + c), *reinterpret_cast<const uint4*>(a.dY + off + c), g,
                   rstd, acc);
  }
  acc = row_sum<AN_WIDE>(acc, red);
  const float cm = rstd * __fdiv_rn(acc, static_cast<float>(a.d));
#pragma unroll 2
  for (int c = threadIdx.x * 8; c < a.d; c += AN_WIDE * 8) {
    float g[8];
    norm_gain8(a.w, c, a.plus_one, g);
    const uint4 dh = a.dH ? *reinterpret_cast<const uint4*>(a.dH + off + c) : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(a.dX + off + c) =
        norm_bwd8(*reinterpret_cast<const uint4*>(a.H + off + c), *reinterpret_cast<const uint4*>(a.dY + off + c), dh,
                  g, rstd, cm);
  }
}

// Threads per row by width: a warp for narrow rows (several rows per CTA), then
// as many threads as keep at most four 16-byte chunks of each tensor per thread.
#define QL_ROW_CASES(KERN, ARGS)                                                                          \
  if (ARGS.d <= 512) return launch_pdl(KERN<32, 2>, dim3((ARGS.M + 3) / 4), dim3(128), 0, st, ARGS);      \
  if (ARGS.d <= 1024) return launch_pdl(KERN<32, 4>, dim3((ARGS.M + 3) / 4), dim3(128), 0, st, ARGS);     \
  if (ARGS.d <= 2048) return launch_pdl(KERN<128, 2>, dim3(ARGS.M), dim3(128), 0, st, ARGS);              \
  if (ARGS.d <= 4096) return launch_pdl(KERN<128, 4>, dim3(ARGS.M), dim3(128), 0, st, ARGS);              \
  if (ARGS.d <= 8192) return launch_pdl(KERN<256, 4>, dim3(ARGS.M), dim3(256), 0, st, ARGS);              \
  if (ARGS.d <= 16384) return launch_pdl(KERN<512, 4>, dim3(ARGS.M), dim3(512), 0, st, ARGS);

cudaError_t launch_add_rmsnorm_fwd(const bf16* X, const bf16* R, const bf16* w, int M, int d, float eps, int plus_one,
                                   bf16* H, bf16* Y, uint8_t* codes, float* scale, float* rstd, cudaStream_t st) {
  const AddNormFwd a = {X, R, w, M, d, plus_one, eps, H, Y, codes, scale, rstd};
  QL_ROW_CASES(add_rmsnorm_fwd_kernel, a)
  return launch_pdl(add_rmsnorm_fwd_wide_kernel, dim3(M), dim3(AN_WIDE), 0, st, a);
}

cudaError_t launch_add_rmsnorm_bwd(const bf16* H, const bf16* w, const float* rstd, const bf16* dY, const bf16* dH,
                                   int M, int d, int plus_one, bf16* dX, cudaStream_t st) {
  const AddNormBwd a = {H, w, rstd, dY, dH, M, d, plus_one, dX};
  QL_ROW_CASES(add_rmsnorm_bwd_kernel, a)
  return launch_pdl(add_rmsnorm_bwd_wide_kernel, dim3(M), dim3(AN_WIDE), 0, st, a);
}
#undef QL_ROW_CASES

}  // namespace ql
