// Eight-element chunks of rows of stored values, with ragged ends (gfx950).
#pragma once

#include "dgf_device.hpp"

namespace dgf {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// 8 stored values of a row from column c (zeros past N), and back.  A ragged
// end is read as the row's last 8 values, shifted down, so that one lane's end
// is one load like the others' (element by element only where N < 8).
__device__ __forceinline__ uint4 row_ld(const uint16_t *row, int64_t c, int64_t N) {
  if (c + 8 <= N) return *reinterpret_cast<const uint4 *>(row + c);
  if (N >= 8) {
    const u32x4_any v = *reinterpret_cast<const u32x4_any *>(row + N - 8);
    const int drop = (int)(c + 8 - N) * 16;  // bits of the columns before c: 16 to 112
    uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
    lo = drop < 64 ? lo >> drop | hi << (64 - drop) : hi >> (drop - 64);
    hi = drop < 64 ? hi >> drop : 0;
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
  }
  uint32_t r[4] = {0, 0, 0, 0};
  for (int e = 0; c + e < N; ++e) r[e >> 1] |= (uint32_t)row[c + e] << (16 * (e & 1));
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void row_st(uint16_t *row, int64_t c, int64_t N, const uint4 &v) {
  if (c + 8 <= N) {
    *reinterpret_cast<uint4 *>(row + c) = v;
    return;
  }
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  for (int e = 0; c + e < N; ++e) row[c + e] = (uint16_t)(r[e >> 1] >> (16 * (e & 1)));
}
// row_st around the caches: for outputs larger than they are.
__device__ __forceinline__ void row_st_nt(uint16_t *row, int64_t c, int64_t N, const uint4 &v) {
  if (c + 8 <= N) {
    const f32x4 f = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
    __builtin_nontemporal_store(f, reinterpret_cast<f32x4 *>(row + c));
    return;
  }
  row_st(row, c, N, v);
}
template <class T>
__device__ __forceinline__ void row_widen(const uint4 &v, float (&f)[8]) {
  f[0] = T::lo(v.x); f[1] = T::hi(v.x); f[2] = T::lo(v.y); f[3] = T::hi(v.y);
  f[4] = T::lo(v.z); f[5] = T::hi(v.z); f[6] = T::lo(v.w); f[7] = T::hi(v.w);
}
template <class T>
__device__ __forceinline__ uint4 row_narrow(const float (&f)[8]) {
  return make_uint4(T::pack_prod(f[0], f[1]), T::pack_prod(f[2], f[3]), T::pack_prod(f[4], f[5]),
                    T::pack_prod(f[6], f[7]));
}

// Elements of an output from which it is stored around the caches: 8 MB, of 32
// MB of L2 that a call's outputs share.
constexpr int64_t kStreamElements = (int64_t)1 << 22;

// The sum of v over the wave, in lane 63 (only): shifts within rows of 16
// lanes, then row ends broadcast (data-parallel moves, no trip through LDS).
__device__ __forceinline__ float wave_sum_last(float v) {
#define DGF_SUM_STEP(ctrl, rows) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, false));
  DGF_SUM_STEP(0x111, 0xf)  // row_shr:1
  DGF_SUM_STEP(0x112, 0xf)  // row_shr:2
  DGF_SUM_STEP(0x114, 0xf)  // row_shr:4
  DGF_SUM_STEP(0x118, 0xf)  // row_shr:8
  DGF_SUM_STEP(0x142, 0xa)  // row_bcast:15
  DGF_SUM_STEP(0x143, 0xc)  // row_bcast:31
#undef DGF_SUM_STEP
  return v;
}

}  // namespace dgf
