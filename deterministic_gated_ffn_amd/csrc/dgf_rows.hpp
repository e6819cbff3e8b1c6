// Eight-element chunks of rows of stored values, with ragged ends (gfx950).
#pragma once

#include "dgf_device.hpp"

namespace dgf {

// 8 stored values of a row from column c (zeros past N), and back.
__device__ __forceinline__ uint4 row_ld(const uint16_t *row, int64_t c, int64_t N) {
  if (c + 8 <= N) return *reinterpret_cast<const uint4 *>(row + c);
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

}  // namespace dgf
