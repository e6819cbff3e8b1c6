// Dropout from a counter-based generator, with the residual (gfx950).
//
//   z = alpha res + (draw >= cut ? x / (1 - cut / 65536) : 0)
//
// The mask is a function of the seed, the step and the value's place, so that it is neither
// written nor read: a call moves x, res and z only, which bounds it.  A thread takes 8 columns
// of a row and draws 16 bits for each of them, all from one block of the generator: a
// probability is a multiple of 2^-16 (0.1 is off by 6e-6), and half the 32-bit products
// that a draw of 32 bits would take.  x / (1 - p) and the sum are FP32, rounded once.
// Measured, BF16: 4096 x 4096 with the residual 16.1 us (100 MB, 6.2 TB/s: part of it comes
// from cache, at the rate of a copy 19.5); 1003 x 5125 without 6.5 us.
#include "dgf_experts.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

// Philox-4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw: Parallel random numbers:
// as easy as 1, 2, 3; 2011): 128 bits from a 128-bit counter and a 64-bit key.
__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
    c[0] = (uint32_t)(b >> 32) ^ c[1] ^ k0;
    c[1] = (uint32_t)b;
    c[2] = (uint32_t)(a >> 32) ^ c[3] ^ k1;
    c[3] = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

template <class T, bool RES>
__global__ __launch_bounds__(256) void k_dropout(DropoutParams p) {
  const int64_t per = (p.H + 7) / 8, i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.M * per) return;
  const int64_t m = i / per, col = 8 * (i - m * per);
  const uint64_t seed = (uint64_t)p.rng[0], step = (uint64_t)p.rng[1];
  const uint4 xv = row_ld(p.x + m * p.ld_x, col, p.H);
  uint4 rv;
  if constexpr (RES) rv = row_ld(p.res + m * p.ld_res, col, p.H);
  uint32_t c[4] = {(uint32_t)i, (uint32_t)(i >> 32), (uint32_t)step, (uint32_t)(step >> 32)};
  philox(c, (uint32_t)seed, (uint32_t)(seed >> 32));
  float x[8], z[8];
  row_widen<T>(xv, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t d = c[e >> 1] >> (16 * (e & 1)) & 0xffffu;
    z[e] = d >= p.cut ? x[e] * p.scale : 0.0f;
  }
  if constexpr (RES) {
    float r[8];
    row_widen<T>(rv, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = p.alpha * r[e] + z[e];
  }
  row_st(p.z + m * p.ld_z, col, p.H, row_narrow<T>(z));
}

template <class T>
hipError_t dropout_t(const DropoutParams &p, hipStream_t s) {
  // (2^32 threads are more than one dimension of a grid takes)
  constexpr int64_t kX = (int64_t)1 << 23;
  const int64_t blocks = (p.M * ((p.H + 7) / 8) + 255) / 256;
  const dim3 g((uint32_t)(blocks < kX ? blocks : kX), (uint32_t)((blocks + kX - 1) / kX)), b(256);
  if (p.res) dgf_launch((k_dropout<T, true>), g, b, 0, s, p);
  else dgf_launch((k_dropout<T, false>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? dropout_t<F16>(p, s) : dropout_t<Bf16>(p, s);
}

}  // namespace dgf
