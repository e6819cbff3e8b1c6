// The norms before and after a block, with its gate and residual (gfx950).
//
//   t = y r_y w_post,  r_y = 1/sqrt(mean(y^2) + eps)     (t = y without w_post)
//   z = alpha res + gate t                               (the new residual stream)
//   h = z r_z w_next,  r_z = 1/sqrt(mean(z^2) + eps)     (the next block's input)
//
// One workgroup per row, the row in its registers: y and res are read once,
// z and h written once, 8 bytes an element against about 12 operations, so
// the kernels are bound by HBM.  Everything between the loads and the stores
// is FP32; z and h are each rounded once, h from the unrounded z.
#include "dgf_block.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

// Sums of N values over the workgroup, the same bits in every thread: a
// butterfly within each wave, then the waves in order.  red holds 16 N floats
// that no other reduction of this row uses.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 16 + (threadIdx.x >> 6)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = red[i * 16];
    for (int w = 1; w < waves; ++w) t += red[i * 16 + w];
    v[i] = t;
  }
}

template <class T, int V>
__global__ __launch_bounds__(1024) void k_norm_fwd(NormFwdParams p) {
  __shared__ float red[2][16];
  const int64_t m = blockIdx.x;
  const int H = (int)p.H;
  const float inv_h = 1.0f / (float)H;
  uint4 yv[V], rv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (threadIdx.x + v * blockDim.x) * 8;
    rv[v] = yv[v] = make_uint4(0, 0, 0, 0);
    if (c < H) {
      rv[v] = row_ld(p.res + m * p.ld_res, c, H);
      if (p.y) yv[v] = row_ld(p.y + m * p.ld_y, c, H);
    }
  }
  float r_y = 1.0f;
  if (p.w_post) {
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float y[8];
      row_widen<T>(yv[v], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = fmaf(y[e], y[e], s[0]);
    }
    row_sums(s, red[0]);
    r_y = 1.0f / sqrtf(fmaf(s[0], inv_h, p.eps));
  }
  float z[V][8];
  float s[1] = {0.0f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (threadIdx.x + v * blockDim.x) * 8;
    row_widen<T>(rv[v], z[v]);
    if (p.y && c < H) {
      float t[8], f[8];
      row_widen<T>(yv[v], t);
      if (p.w_post) {
        row_widen<T>(row_ld(p.w_post, c, H), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = t[e] * r_y * f[e];
      }
      if (p.gate) {
        row_widen<T>(row_ld(p.gate + m * p.ld_gate, c, H), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] *= f[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) z[v][e] = fmaf(p.alpha, z[v][e], t[e]);
      row_st(p.z + m * p.ld_z, c, H, row_narrow<T>(z[v]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = fmaf(z[v][e], z[v][e], s[0]);
  }
  float r_z = 1.0f;
  if (p.w_next) {
    row_sums(s, red[1]);
    r_z = 1.0f / sqrtf(fmaf(s[0], inv_h, p.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= H) continue;
      float f[8];
      row_widen<T>(row_ld(p.w_next, c, H), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= z[v][e] * r_z;
      row_st(p.h + m * p.ld_h, c, H, row_narrow<T>(f));
    }
  }
  if (p.rstd && threadIdx.x == 0) {
    p.rstd[2 * m] = r_y;
    p.rstd[2 * m + 1] = r_z;
  }
}

// The backward, each workgroup over its own rows m = blockIdx.x, + groups, ...
//
//   G  = dz + r_z (dn - z r_z^2 mean(dn z)),  dn = dh w_next
//   dres = alpha G,  dgate = G t,  dq = G gate w_post,
//   dy = r_y (dq - y r_y^2 mean(dq y))
//
// mean(dq y) is linear in G, so it follows from two sums that need no other
// sum first: with q = gate w_post y, sum(G q) = sum((dz + r_z dn) q) - c sum(z q),
// c = r_z^3 mean(dn z).  All three sums of a row take one reduction.  The
// column sums dw_post, dw_next and a broadcast dgate stay in registers over
// the workgroup's rows and go to `part` once (FP32, added up by k_norm_wgrad
// in the order of the workgroups, so results do not change from run to run).
template <class T, int V>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormBwdParams p) {
  __shared__ float red[2][3][16];
  const int H = (int)p.H;
  const float inv_h = 1.0f / (float)H;
  float ap[V][8] = {}, an[V][8] = {}, ag[V][8] = {};
  int turn = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, turn ^= 1) {
    uint4 gv[V], dv[V], zv[V], yv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      gv[v] = dv[v] = zv[v] = yv[v] = make_uint4(0, 0, 0, 0);
      if (c < H) {
        if (p.dz) gv[v] = row_ld(p.dz + m * p.ld_dz, c, H);
        if (p.dh) dv[v] = row_ld(p.dh + m * p.ld_dh, c, H), zv[v] = row_ld(p.z + m * p.ld_z, c, H);
        if (p.y) yv[v] = row_ld(p.y + m * p.ld_y, c, H);
      }
    }
    const float r_y = p.rstd[2 * m], r_z = p.rstd[2 * m + 1];
    float g0[V][8], s[3] = {0.0f, 0.0f, 0.0f};  // g0 = dz + r_z dn
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      float z[8], q[8], f[8];
      row_widen<T>(gv[v], g0[v]);
      row_widen<T>(zv[v], z);
      if (p.dh && c < H) {
        float dh[8];
        row_widen<T>(dv[v], dh);
        row_widen<T>(row_ld(p.w_next, c, H), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          an[v][e] = fmaf(dh[e], z[e] * r_z, an[v][e]);
          const float dn = dh[e] * f[e];
          s[0] = fmaf(dn, z[e], s[0]);
          g0[v][e] = fmaf(r_z, dn, g0[v][e]);
        }
      }
      if (p.w_post && c < H) {
        row_widen<T>(yv[v], q);
        row_widen<T>(row_ld(p.w_post, c, H), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] *= f[e];
        if (p.gate) {
          row_widen<T>(row_ld(p.gate + m * p.ld_gate, c, H), f);
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] *= f[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[1] = fmaf(g0[v][e], q[e], s[1]);
          s[2] = fmaf(z[e], q[e], s[2]);
        }
      }
    }
    row_sums(s, red[turn][0]);  // two sets in turn: no barrier between a row's reads and the next row's writes
    const float cz = p.dh ? r_z * r_z * r_z * (s[0] * inv_h) : 0.0f;
    const float cy = p.w_post ? r_y * r_y * r_y * ((s[1] - cz * s[2]) * inv_h) : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= H) continue;
      float z[8], o[8];
      row_widen<T>(zv[v], z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g0[v][e] = fmaf(-cz, z[e], g0[v][e]);
        o[e] = p.alpha * g0[v][e];
      }
      row_st(p.dres + m * p.ld_dres, c, H, row_narrow<T>(o));
      if (!p.y) continue;
      float y[8], w[8], f[8];
      row_widen<T>(yv[v], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      if (p.w_post) row_widen<T>(row_ld(p.w_post, c, H), w);
      if (p.gate) {  // dgate = G t, t = y r_y w_post
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = g0[v][e] * (y[e] * r_y * w[e]);
        if (p.ld_gate == 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) ag[v][e] += o[e];
        } else if (p.dgate) {
          row_st(p.dgate + m * p.ld_dgate, c, H, row_narrow<T>(o));
        }
        row_widen<T>(row_ld(p.gate + m * p.ld_gate, c, H), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) g0[v][e] *= f[e];
      }
      if (p.w_post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ap[v][e] = fmaf(g0[v][e], y[e] * r_y, ap[v][e]);
          g0[v][e] = fmaf(r_y * w[e], g0[v][e], -cy * y[e]);
        }
      }
      row_st(p.dy + m * p.ld_dy, c, H, row_narrow<T>(g0[v]));
    }
  }
  const int64_t ldp = (p.H + 7) & ~(int64_t)7;
  float *out = p.part + (int64_t)blockIdx.x * ldp;
  const int64_t stride = (int64_t)gridDim.x * ldp;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (threadIdx.x + v * blockDim.x) * 8;
    if (c >= H) continue;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      if (p.dw_post) *reinterpret_cast<f32x4 *>(out + c + e) = f32x4{ap[v][e], ap[v][e + 1], ap[v][e + 2], ap[v][e + 3]};
      if (p.dw_next) *reinterpret_cast<f32x4 *>(out + stride + c + e) = f32x4{an[v][e], an[v][e + 1], an[v][e + 2], an[v][e + 3]};
      if (p.dgate && p.ld_gate == 0)
        *reinterpret_cast<f32x4 *>(out + 2 * stride + c + e) = f32x4{ag[v][e], ag[v][e + 1], ag[v][e + 2], ag[v][e + 3]};
    }
  }
}

// Column sums over the workgroups' parts: 64 columns per workgroup, 4 waves
// each over a contiguous quarter of the parts, the quarters added in order.
template <class T>
__global__ __launch_bounds__(256) void k_norm_wgrad(NormBwdParams p) {
  __shared__ float red[4][64];
  const int which = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint16_t *out = which == 0 ? p.dw_post : which == 1 ? p.dw_next : p.ld_gate == 0 ? p.dgate : nullptr;
  if (!out) return;
  const int64_t ldp = (p.H + 7) & ~(int64_t)7, c = (int64_t)blockIdx.x * 64 + lane;
  const int lo = p.groups * wave / 4, hi = p.groups * (wave + 1) / 4;
  float t = 0.0f;
  if (c < p.H)
    for (int g = lo; g < hi; ++g) t += p.part[((int64_t)which * p.groups + g) * ldp + c];
  red[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && c < p.H) out[c] = T::r(((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane]);
}

// Threads of a row: 8 elements each while 1024 threads hold the row, else 16.
int row_threads(int64_t H) {
  const int64_t chunks = (H + 7) / 8;
  if (chunks > 1024) return 1024;
  return (int)((chunks + 63) / 64 * 64);
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwdParams &p, hipStream_t s) {
  const dim3 g((unsigned)p.M), b(row_threads(p.H));
  if (p.H <= 8192) {
    if (p.fmt == FMT_F16) dgf_launch((k_norm_fwd<F16, 1>), g, b, 0, s, p);
    else dgf_launch((k_norm_fwd<Bf16, 1>), g, b, 0, s, p);
  } else {
    if (p.fmt == FMT_F16) dgf_launch((k_norm_fwd<F16, 2>), g, b, 0, s, p);
    else dgf_launch((k_norm_fwd<Bf16, 2>), g, b, 0, s, p);
  }
  return hipGetLastError();
}

int norm_bwd_groups(int64_t M, int64_t H) { return (int)(M < 512 ? M : 512); }

hipError_t launch_norm_bwd(const NormBwdParams &p, hipStream_t s) {
  const dim3 g((unsigned)p.groups), b(row_threads(p.H));
  if (p.H <= 8192) {
    if (p.fmt == FMT_F16) dgf_launch((k_norm_bwd<F16, 1>), g, b, 0, s, p);
    else dgf_launch((k_norm_bwd<Bf16, 1>), g, b, 0, s, p);
  } else {
    if (p.fmt == FMT_F16) dgf_launch((k_norm_bwd<F16, 2>), g, b, 0, s, p);
    else dgf_launch((k_norm_bwd<Bf16, 2>), g, b, 0, s, p);
  }
  return hipGetLastError();
}

hipError_t launch_norm_wgrad(const NormBwdParams &p, hipStream_t s) {
  const dim3 g((unsigned)((p.H + 63) / 64), 3);
  if (p.fmt == FMT_F16) dgf_launch(k_norm_wgrad<F16>, g, dim3(256), 0, s, p);
  else dgf_launch(k_norm_wgrad<Bf16>, g, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace dgf
