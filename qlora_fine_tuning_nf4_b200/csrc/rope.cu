// Rotary positions on the heads of a row-strided matrix, forward and backward.
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * theta_i,
// for the pairs (2i, 2i + 1) of a head (interleaved) or (i, i + rot / 2) (halves);
// the backward is the transposed rotation, t -> -t.  Elements from rot on pass.
//
// Angles are fixed-point turns: theta_i / 2 pi is a 64-bit fraction, and position
// times it modulo 2^64 is one integer multiply whose wrap-around drops the whole
// turns exactly.  The 32 upper bits become a binary32 number: 2^-32 turns dropped and
// 2^-26 rounded at most (half a turn has 24 bits), the same at every position, where
// a binary32 product would be off by whole radians at far ones.  An entry of the
// table counts p times: p 2^-65 turns where it is the nearest fraction.  No 64-bit
// floating point and no table of cosines per position is needed.
//
// HBM-bound.  A CTA takes one or two tokens: its threads find each token's cosines
// and sines once (shared memory) while their first loads are on the way, then
// stream the heads.  Many small CTAs with 32 registers a thread (16 of 128 threads
// per SM) keep more bytes in flight than longer batches per thread: 8192 tokens of
// 40 heads of 128 in rows of 6144, 168 MB, take 30.6 us (5.5 TB/s); with 256
// threads, four tokens and two heads in flight per thread (72 registers) 36.5 us,
// with the loads of a head after the previous head's store 45 us.
#include "fp8.cuh"

namespace ql {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_TOK = 2;       // tokens per CTA at most
constexpr int ROPE_MAX_D = 512;   // widest head

struct RopeArgs {
  const bf16* X;
  bf16* out;            // may be X with the same row stride
  const uint64_t* turns;  // [rot / 2], theta_i / 2 pi in units of 2^-64 turns
  const int64_t* pos;   // [M], or null: row (modulo seq_len if that is positive)
  int64_t ldx, ldo, seq_len;
  int M, heads, D, rot;
  int tok;              // tokens per CTA
  float factor, sign;   // cos and sin are multiplied by factor; sign -1: transposed
};

template <int VEC>
struct RopeVec;
template <> struct RopeVec<8> { using T = uint4; };
template <> struct RopeVec<4> { using T = uint2; };
template <> struct RopeVec<2> { using T = uint32_t; };
template <> struct RopeVec<1> { using T = uint16_t; };

template <int VEC>
QL_DEV void rope_unpack(const typename RopeVec<VEC>::T& u, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = __uint_as_float(static_cast<uint32_t>(u) << 16);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}
template <int VEC>
QL_DEV typename RopeVec<VEC>::T rope_pack(const float (&f)[VEC]) {
  typename RopeVec<VEC>::T u;
  if constexpr (VEC == 1) {
    u = static_cast<uint16_t>(pack_bf16x2(f[0], 0.f));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
  return u;
}

// One head is `np` rotated items and then D - rot untouched elements in items of
// VEC (copied where out is not X).  A rotated item is VEC pairs read as two
// vectors (halves), or VEC / 2 pairs in one (interleaved).
template <bool INTER, int VEC>
__global__ void __launch_bounds__(ROPE_THREADS, 16) rope_kernel(const RopeArgs a) {
  using V = typename RopeVec<VEC>::T;
  constexpr int NP = INTER ? VEC / 2 : VEC;  // pairs per item
  constexpr int HB = INTER ? 2 : 1;          // items in flight per thread
  __shared__ float2 cs[ROPE_TOK * ROPE_MAX_D / 2];
  grid_dep_wait();
  grid_dep_launch();
  const int half = a.rot / 2;
  const int row0 = static_cast<int>(blockIdx.x) * a.tok;
  const int ntok = min(a.tok, a.M - row0);
  const int np = half / NP;
  const int items = np + (a.out == a.X ? 0 : (a.D - a.rot) / VEC);
  const int lanes = min(items, ROPE_THREADS);
  const int hl = threadIdx.x / lanes, nh = ROPE_THREADS / lanes;  // nh heads (of any tokens) side by side
  const int v0 = threadIdx.x % lanes;
  const int total = hl < nh ? ntok * a.heads : 0;
  const bf16* X = a.X + static_cast<size_t>(row0) * a.ldx;
  bf16* O = a.out + static_cast<size_t>(row0) * a.ldo;
  V p[HB], q[HB];
  int tk[HB], hd[HB];
  // HB (token, head) items' loads are in flight before the first store: X and out may be the same
  // memory, so the compiler cannot move a later load up
  auto load = [&](int v, int i0) {
    const int e = v >= np ? a.rot + (v - np) * VEC : v * VEC;
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      const int i = i0 + j * nh;
      tk[j] = i / a.heads;
      hd[j] = i - tk[j] * a.heads;
      if (i < total) {
        const bf16* x = X + tk[j] * a.ldx + hd[j] * a.D + e;
        p[j] = *reinterpret_cast<const V*>(x);
        if (!INTER && v < np) q[j] = *reinterpret_cast<const V*>(x + half);
      }
    }
  };
  load(v0, hl);  // on its way while the angles are found
  for (int i = threadIdx.x; i < ntok * half; i += ROPE_THREADS) {
    const int64_t row = row0 + i / half;
    const int64_t pos = a.pos ? a.pos[row] : (a.seq_len > 0 ? row % a.seq_len : row);
    const uint64_t t = static_cast<uint64_t>(pos) * a.turns[i % half];
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cs[i] = make_float2(c * a.factor, s * a.factor * a.sign);
  }
  __syncthreads();
  for (int v = v0; v < items; v += lanes) {
    const bool tail = v >= np;
    const int e = tail ? a.rot + (v - np) * VEC : v * VEC;
    if (v != v0) load(v, hl);
    for (int i0 = hl; i0 < total; i0 += HB * nh) {
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        if (i0 + j * nh >= total) break;
        bf16* o = O + tk[j] * a.ldo + hd[j] * a.D + e;
        if (!tail) {
          const float2* f = cs + tk[j] * half + v * NP;
          float r[VEC], t[VEC];
          rope_unpack<VEC>(p[j], r);
          if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const float u = r[2 * i], w = r[2 * i + 1];
              r[2 * i] = u * f[i].x - w * f[i].y;
              r[2 * i + 1] = w * f[i].x + u * f[i].y;
            }
          } else {
            rope_unpack<VEC>(q[j], t);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float u = r[i] * f[i].x - t[i] * f[i].y;
              t[i] = t[i] * f[i].x + r[i] * f[i].y;
              r[i] = u;
            }
            *reinterpret_cast<V*>(o + half) = rope_pack<VEC>(t);
          }
          p[j] = rope_pack<VEC>(r);
        }
        *reinterpret_cast<V*>(o) = p[j];
      }
      if (i0 + HB * nh < total) load(v, i0 + HB * nh);
    }
  }
}

cudaError_t launch_rope(const bf16* X, int64_t M, int64_t ldx, int heads, int D, const uint64_t* turns, int rot,
                        bool interleaved, float factor, bool transpose, const int64_t* pos, int64_t seq_len, bf16* out,
                        int64_t ldo, int sms, cudaStream_t st) {
  RopeArgs a = {X, out, turns, pos, ldx, ldo, seq_len, (int)M, heads, D, rot, 1, factor, transpose ? -1.f : 1.f};
  // Tokens per CTA, one against two (us, 148 SMs): 40 heads of 128, 148 rows 3.2 / 4.3, 592 4.2 / 4.9, 1776 8.9 / 7.6,
  // 8192 29.0 / 30.0; 12 interleaved heads of 96 with 64 rotated, 592 rows 2.5 / 2.8, 1776 4.3 / 3.5, 8192 11.9 / 9.6; 6
  // heads of 64, 592 rows 2.1 / 2.0, 8192 9.0 / 6.0.  With few rows one token spreads the heads over more CTAs; from
  // eight rows per SM on two halve the CTAs to set up, which narrow rows gain from and wide ones hardly notice.
  a.tok = M >= int64_t{8} * sms ? ROPE_TOK : 1;
  const unsigned grid = static_cast<unsigned>((M + a.tok - 1) / a.tok);
#define QL_ROPE(I_, V_) launch_pdl(rope_kernel<I_, V_>, dim3(grid), dim3(ROPE_THREADS), 0, st, a)
  // the widest vector that divides the rotated part: heads start on 16 bytes (D % 8 == 0)
  if (interleaved) {
    if (rot % 8 == 0) return QL_ROPE(true, 8);
    if (rot % 4 == 0) return QL_ROPE(true, 4);
    return QL_ROPE(true, 2);
  }
  if (rot % 16 == 0) return QL_ROPE(false, 8);
  if (rot % 8 == 0) return QL_ROPE(false, 4);
  if (rot % 4 == 0) return QL_ROPE(false, 2);
  return QL_ROPE(false, 1);
#undef QL_ROPE
}

}  // namespace ql
