// 8-bit activation checkpoints: the block format and its use (gfx950).
//
// A row is cut into blocks of 64 columns (the last may be short).  A block
// with largest magnitude A keeps the FP32 scale s = A / 127 and one signed
// byte a value, q = rint(x * (127 / A)), in [-127, 127]; it reads back as
// q s, off by at most s / 2.  A block below 2^-119 (its 127 / A would near
// FP32's limit) keeps s = 0 and reads back as zeros; a block that holds an
// infinity or a NaN keeps s = NaN, so that it reads back as NaN throughout
// rather than as finite numbers.
#pragma once

#include "dgf_device.hpp"
#include "dgf_kernels.hpp"
#include "dgf_rows.hpp"

namespace dgf {

constexpr int kQ8Block = 64;

// Scale of a block and the factor that takes its values to codes, from the
// largest FP32 magnitude bits in it (as integers, NaN above infinity above
// the finite values).
__device__ __forceinline__ void q8_scale(uint32_t top, float &s, float &inv) {
  const float a = __uint_as_float(top);
  s = a / 127.0f;
  inv = 127.0f / a;
  if (a < 0x1p-119f) s = inv = 0.0f;
  if (top >= 0x7f800000u) {
    s = __uint_as_float(0x7fc00000u);
    inv = 0.0f;
  }
}

// The 8 lanes of a block (8 columns each): codes of this lane's columns and
// the block's scale.  All 64 lanes of the wave take part.
__device__ __forceinline__ uint2 q8_pack(const float (&x)[8], float &s) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const uint32_t b = (uint32_t)__shfl_xor((int)top, o);
    top = b > top ? b : top;
  }
  float inv;
  q8_scale(top, s, inv);
  uint32_t q[2] = {0, 0};
  if (inv != 0.0f)
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e >> 2] |= (uint32_t)((int)rintf(x[e] * inv) & 0xff) << (8 * (e & 3));
  return make_uint2(q[0], q[1]);
}

// 8 codes to values.
__device__ __forceinline__ void q8_values(const uint2 &q, float s, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3))) * s;
}

typedef uint64_t u64_any __attribute__((aligned(1)));

// 8 codes of a row from column c (zeros past N; ragged ends as in row_ld), and back.
__device__ __forceinline__ uint2 q8_ld(const uint8_t *row, int64_t c, int64_t N) {
  if (c + 8 <= N) return *reinterpret_cast<const uint2 *>(row + c);
  if (N >= 8) {
    const uint64_t v = *reinterpret_cast<const u64_any *>(row + N - 8) >> (int)(c + 8 - N) * 8;
    return make_uint2((uint32_t)v, (uint32_t)(v >> 32));
  }
  uint32_t q[2] = {0, 0};
  for (int e = 0; c + e < N; ++e) q[e >> 2] |= (uint32_t)row[c + e] << (8 * (e & 3));
  return make_uint2(q[0], q[1]);
}
__device__ __forceinline__ void q8_st(uint8_t *row, int64_t c, int64_t N, const uint2 &q) {
  if (c + 8 <= N) {
    *reinterpret_cast<uint2 *>(row + c) = q;
    return;
  }
  for (int e = 0; c + e < N; ++e) row[c + e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
}

// The activation's backward at 8 columns, g and u as read back in FP32 (never
// rounded to the stored type): dU = rnd(dA silu(g)), dG = rnd((dA u) silu'(g)),
// a = rnd(silu(g) u), the FP32 operations of the 16-bit form.
template <class T>
__device__ __forceinline__ void q8_dsilu(const float (&da)[8], const float (&g)[8], const float (&u)[8], uint4 &dg,
                                         uint4 &du, uint4 &a) {
  float fg[8], fu[8], fa[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float sg = sigma_f(g[e]);
    const float s = g[e] * sg;
    const float ds = sg * (1.0f + g[e] * (1.0f - sg));
    fu[e] = da[e] * s;
    fg[e] = (da[e] * u[e]) * ds;
    fa[e] = s * u[e];
  }
  dg = row_narrow<T>(fg);
  du = row_narrow<T>(fu);
  a = row_narrow<T>(fa);
}

// A saved matrix in 8 bits: codes [M, N] (ldq bytes a row), scales [M, ceil(N/64)].
struct Q8Mat {
  uint8_t *q;
  float *s;
  int64_t ldq, lds;
};

hipError_t launch_pack8(int fmt, const uint16_t *x, int64_t ldx, Q8Mat o, int64_t M, int64_t N, hipStream_t s);
hipError_t launch_pack8_pair(int fmt, const uint16_t *g, const uint16_t *u, int64_t ld, Q8Mat g8, Q8Mat u8, int64_t M,
                             int64_t N, hipStream_t s);
hipError_t launch_unpack8(int fmt, Q8Mat x, uint16_t *o, int64_t ldo, int64_t M, int64_t N, hipStream_t s);
struct ActQ8Params {
  const uint16_t *da;
  Q8Mat g, u;
  uint16_t *dg, *du, *a;  // a may be null
  int64_t ldda, ldo;
  int64_t M, N;
};
hipError_t launch_act_bwd_q8(int fmt, const ActQ8Params &p, hipStream_t s);

// The FFN's two joins that touch g and u, with the checkpoint in 8 bits: the
// gate/up join writes a and the codes (p as for EPI_ACT, C[0], C[1] unused),
// the dA join reads them (p as for EPI_DSILU, sg, su unused).
hipError_t launch_join_act_q8(const GemmParams &p, Q8Mat g, Q8Mat u, hipStream_t s);
hipError_t launch_join_dsilu_q8(const GemmParams &p, Q8Mat g, Q8Mat u, hipStream_t s);

}  // namespace dgf
