// Kernels of the 8-bit activation checkpoints (format: dgf_q8.hpp).
//
// All are one pass over rows of N columns, bound by HBM: 3.06 bytes an element
// to write or read a checkpoint, 10.1 for the activation's backward (da and
// both codes in, dG, dU and a out).  At 4096 x 12288, BF16: written in 27.6 us
// (5.6 TB/s), read back in 24.0 (6.4), the activation's backward in 98 (5.2).
// A thread takes 8 columns (16 bytes in,
// 8 bytes of codes), so the 8 lanes of a block are neighbours and find its
// largest magnitude with three lane exchanges.
#include "dgf_join.hpp"
#include "dgf_q8.hpp"

namespace dgf {
namespace {

constexpr int kThreads = 256;

// A row's blocks padded to whole ones, 8 lanes each: `lanes` (a power of two,
// 8 to 256) of a workgroup's threads share a row, and grid.y workgroups its
// columns, `span` of them each: a few chunks of 8 a thread where that still
// makes 2048 workgroups, one where it does not (32 x 12288 written: 5.8 us with
// whole rows, 3.0 so; 777 x 5461 in the activation's backward: 15.8 and 13.8).
struct RowMap {
  int lanes, span;
  dim3 grid;
};
RowMap row_map(int64_t M, int64_t N) {
  const int64_t chunks = (N + kQ8Block - 1) / kQ8Block * 8;
  int lanes = 8;
  while (lanes < kThreads && lanes < chunks) lanes <<= 1;
  const int64_t rows = kThreads / lanes, groups = (M + rows - 1) / rows;
  int64_t per = (chunks + lanes - 1) / lanes;  // chunks a thread for whole rows
  while (per > 1 && groups * ((chunks + lanes * per - 1) / (lanes * per)) < 2048) per = (per + 1) / 2;
  while ((chunks + lanes * per - 1) / (lanes * per) > 65535) per *= 2;  // grid.y
  return RowMap{lanes, (int)(lanes * per * 8), dim3((unsigned)groups, (unsigned)((chunks + lanes * per - 1) / (lanes * per)))};
}

// Rows past M keep their lanes in the loop (the lane exchanges need whole
// blocks) but touch no memory.
#define DGF_ROWS(M_, N_)                                                                    \
  const int64_t m = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;         \
  const bool row_ok = m < (M_);                                                             \
  const int64_t padded = ((N_) + kQ8Block - 1) / kQ8Block * kQ8Block;                       \
  const int64_t first = (int64_t)blockIdx.y * span, last = first + span < padded ? first + span : padded; \
  for (int64_t c = first + (threadIdx.x & (lanes - 1)) * 8; c < last; c += 8 * lanes)

// One matrix, or two of one shape (grid.z).
template <class T>
__global__ __launch_bounds__(kThreads) void k_pack8(const uint16_t *x0, const uint16_t *x1, int64_t ldx, Q8Mat o0,
                                                    Q8Mat o1, int64_t M, int64_t N, int lanes, int span) {
  const uint16_t *x = blockIdx.z ? x1 : x0;
  const Q8Mat o = blockIdx.z ? o1 : o0;
  DGF_ROWS(M, N) {
    const bool in = row_ok && c < N;
    float f[8], s;
    row_widen<T>(in ? row_ld(x + m * ldx, c, N) : make_uint4(0, 0, 0, 0), f);
    const uint2 q = q8_pack(f, s);
    if (in) {
      q8_st(o.q + m * o.ldq, c, N, q);
      if ((c & (kQ8Block - 1)) == 0) o.s[m * o.lds + c / kQ8Block] = s;
    }
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_unpack8(Q8Mat x, uint16_t *o, int64_t ldo, int64_t M, int64_t N,
                                                      int lanes, int span) {
  DGF_ROWS(M, N) {
    if (!row_ok || c >= N) continue;
    float f[8];
    q8_values(q8_ld(x.q + m * x.ldq, c, N), x.s[m * x.lds + c / kQ8Block], f);
    row_st(o + m * ldo, c, N, row_narrow<T>(f));
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_act_bwd_q8(ActQ8Params p, int lanes, int span) {
  DGF_ROWS(p.M, p.N) {
    if (!row_ok || c >= p.N) continue;
    float da[8], g[8], u[8];
    row_widen<T>(row_ld(p.da + m * p.ldda, c, p.N), da);
    q8_values(q8_ld(p.g.q + m * p.g.ldq, c, p.N), p.g.s[m * p.g.lds + c / kQ8Block], g);
    q8_values(q8_ld(p.u.q + m * p.u.ldq, c, p.N), p.u.s[m * p.u.lds + c / kQ8Block], u);
    uint4 dg, du, a;
    q8_dsilu<T>(da, g, u, dg, du, a);
    if (p.M * p.N >= kStreamElements) {  // 4096 x 12288: 98.6 us against 101
      row_st_nt(p.dg + m * p.ldo, c, p.N, dg);
      row_st_nt(p.du + m * p.ldo, c, p.N, du);
      if (p.a) row_st_nt(p.a + m * p.ldo, c, p.N, a);
    } else {
      row_st(p.dg + m * p.ldo, c, p.N, dg);
      row_st(p.du + m * p.ldo, c, p.N, du);
      if (p.a) row_st(p.a + m * p.ldo, c, p.N, a);
    }
  }
}

// The gate/up join with the activation and the checkpoint: a from the rounded
// roots g and u (the bits of the 16-bit form), their codes in place of g and u.
template <class T, int S>
__global__ __launch_bounds__(kThreads) void k_join_act_q8(GemmParams p, Q8Mat g8, Q8Mat u8, int lanes, int span) {
  DGF_ROWS(p.M, p.N) {
    const bool in = row_ok && c < p.N;
    uint32_t r0[4] = {0, 0, 0, 0}, r1[4] = {0, 0, 0, 0}, a[4];
    if (in) {
      join8<T, S>(p, 0, m, c, r0);
      join8<T, S>(p, 1, m, c, r1);
      // the padding columns of the partial roots (past N) are not part of a block
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e >= p.N) {
          r0[e >> 1] &= 0xffffu << (16 * ((e & 1) ^ 1));
          r1[e >> 1] &= 0xffffu << (16 * ((e & 1) ^ 1));
        }
    }
    float g[8], u[8], sg, su;
    row_widen<T>(make_uint4(r0[0], r0[1], r0[2], r0[3]), g);
    row_widen<T>(make_uint4(r1[0], r1[1], r1[2], r1[3]), u);
    const uint2 qg = q8_pack(g, sg), qu = q8_pack(u, su);
    if (!in) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float s0 = g[2 * q] * sigma_f(g[2 * q]), s1 = g[2 * q + 1] * sigma_f(g[2 * q + 1]);
      a[q] = T::pack_prod(s0 * u[2 * q], s1 * u[2 * q + 1]);
    }
    store8(p.act_out + m * p.ld_act + c, c, p.N, a);
    q8_st(g8.q + m * g8.ldq, c, p.N, qg);
    q8_st(u8.q + m * u8.ldq, c, p.N, qu);
    if ((c & (kQ8Block - 1)) == 0) {
      g8.s[m * g8.lds + c / kQ8Block] = sg;
      u8.s[m * u8.lds + c / kQ8Block] = su;
    }
  }
}

// The dA join with the activation's backward from the checkpoint.
template <class T, int S>
__global__ __launch_bounds__(kThreads) void k_join_dsilu_q8(GemmParams p, Q8Mat g8, Q8Mat u8, int lanes, int span) {
  DGF_ROWS(p.M, p.N) {
    if (!row_ok || c >= p.N) continue;
    uint32_t r[4];
    join8<T, S>(p, 0, m, c, r);
    float da[8], g[8], u[8];
    row_widen<T>(make_uint4(r[0], r[1], r[2], r[3]), da);
    q8_values(q8_ld(g8.q + m * g8.ldq, c, p.N), g8.s[m * g8.lds + c / kQ8Block], g);
    q8_values(q8_ld(u8.q + m * u8.ldq, c, p.N), u8.s[m * u8.lds + c / kQ8Block], u);
    uint4 dg, du, a;
    q8_dsilu<T>(da, g, u, dg, du, a);
    row_st(p.dG + m * p.ld_d, c, p.N, dg);
    row_st(p.dU + m * p.ld_d, c, p.N, du);
    row_st(p.a_rm + m * p.ld_d, c, p.N, a);
  }
}

#undef DGF_ROWS

}  // namespace

#define DGF_BY_TYPE(fmt, kernel, grid, ...)                                                             \
  do {                                                                                                  \
    if ((fmt) == FMT_F16) dgf_launch((kernel<F16>), dim3(grid), dim3(kThreads), 0, s, __VA_ARGS__);     \
    else dgf_launch((kernel<Bf16>), dim3(grid), dim3(kThreads), 0, s, __VA_ARGS__);                     \
    return hipGetLastError();                                                                           \
  } while (0)

hipError_t launch_pack8(int fmt, const uint16_t *x, int64_t ldx, Q8Mat o, int64_t M, int64_t N, hipStream_t s) {
  const RowMap r = row_map(M, N);
  DGF_BY_TYPE(fmt, k_pack8, r.grid, x, x, ldx, o, o, M, N, r.lanes, r.span);
}

hipError_t launch_pack8_pair(int fmt, const uint16_t *g, const uint16_t *u, int64_t ld, Q8Mat g8, Q8Mat u8, int64_t M,
                             int64_t N, hipStream_t s) {
  RowMap r = row_map(M, N);
  r.grid.z = 2;
  DGF_BY_TYPE(fmt, k_pack8, r.grid, g, u, ld, g8, u8, M, N, r.lanes, r.span);
}

hipError_t launch_unpack8(int fmt, Q8Mat x, uint16_t *o, int64_t ldo, int64_t M, int64_t N, hipStream_t s) {
  const RowMap r = row_map(M, N);
  DGF_BY_TYPE(fmt, k_unpack8, r.grid, x, o, ldo, M, N, r.lanes, r.span);
}

hipError_t launch_act_bwd_q8(int fmt, const ActQ8Params &p, hipStream_t s) {
  const RowMap r = row_map(p.M, p.N);
  DGF_BY_TYPE(fmt, k_act_bwd_q8, r.grid, p, r.lanes, r.span);
}

// The joins' K pieces, 2^ksplit_depth of them, are a template argument.
#define DGF_JOIN(kernel, S_)                                                                                      \
  case S_:                                                                                                        \
    if (p.fmt == FMT_F16) dgf_launch((kernel<F16, S_>), dim3(r.grid), dim3(kThreads), 0, s, p, g, u, r.lanes, r.span);    \
    else dgf_launch((kernel<Bf16, S_>), dim3(r.grid), dim3(kThreads), 0, s, p, g, u, r.lanes, r.span);                    \
    break;
#define DGF_JOINS(kernel)                                                                                         \
  const RowMap r = row_map(p.M, p.N);                                                                             \
  switch (1 << p.ksplit_depth) {                                                                                  \
    DGF_JOIN(kernel, 1) DGF_JOIN(kernel, 2) DGF_JOIN(kernel, 4) DGF_JOIN(kernel, 8) DGF_JOIN(kernel, 16)          \
    DGF_JOIN(kernel, 32)                                                                                          \
    default: return hipErrorInvalidValue;                                                                         \
  }                                                                                                               \
  return hipGetLastError();

hipError_t launch_join_act_q8(const GemmParams &p, Q8Mat g, Q8Mat u, hipStream_t s) { DGF_JOINS(k_join_act_q8) }
hipError_t launch_join_dsilu_q8(const GemmParams &p, Q8Mat g, Q8Mat u, hipStream_t s) { DGF_JOINS(k_join_dsilu_q8) }

}  // namespace dgf
