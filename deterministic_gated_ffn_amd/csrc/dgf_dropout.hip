// Dropout from a counter-based generator, with the residual (gfx950).
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
  const int64_t per = (p.H + 7) / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
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
  const dim3 g((uint32_t)((p.M * ((p.H + 7) / 8) + 255) / 256)), b(256);
  if (p.res) dgf_launch((k_dropout<T, true>), g, b, 0, s, p);
  else dgf_launch((k_dropout<T, false>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? dropout_t<F16>(p, s) : dropout_t<Bf16>(p, s);
}

}  // namespace dgf
