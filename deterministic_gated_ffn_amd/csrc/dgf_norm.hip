// The norms before and after a block, with its gate and residual (gfx950).
//
//   t = y r_y w_post,  r_y = 1/sqrt(mean(y^2) + eps)     (t = y without w_post)
//   z = alpha res + gate t                               (the new residual stream)
//   h = z r_z w_next,  r_z = 1/sqrt(mean(z^2) + eps)     (the next block's input)
//
// A row lives in the registers of its threads: y and res are read once, z and h
// written once, 8 bytes an element against about 12 operations, so the kernels
// are bound by HBM.  Everything between the loads and the stores is FP32; z and
// h are each rounded once, h from the unrounded z.
// Measured at 4096 x 4096, BF16, with a gate for each channel: forward 21.8 us,
// 6.2 TB/s; backward 36.9 us, 5.5 TB/s, and 4.2 us for its column sums (a copy
// of 2 GiB reaches 5.0 TB/s on the same card, one of 256 MiB 5.5).
#include "dgf_block.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

constexpr int kBwdThreads = 512;

// Sums of N <= 4 values over the waves [w0, w0 + waves) of the workgroup that
// share a row, the same bits in all their threads: within each wave, then the
// waves in order.  red: one float4 a wave, not used by the row before or after.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float4 *red, int w0, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum_last(v[i]);
  if ((threadIdx.x & 63) == 63) {
    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = v[i];
    red[threadIdx.x >> 6] = make_float4(f[0], f[1], f[2], f[3]);
  }
  __syncthreads();
  float4 t = red[w0];
#pragma unroll 4
  for (int w = 1; w < waves; ++w) {
    const float4 q = red[w0 + w];
    t.x += q.x; t.y += q.y; t.z += q.z; t.w += q.w;
  }
  const float f[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = f[i];
}

// One workgroup per row; everything it reads is asked for before the first sum.
// Large outputs are stored around the caches (4096 x 4096: 21.8 us against
// 23.2, 1024 x 16384: 20.8 against 26.0; the backward, which waits for its
// stores' slots sooner, loses by it: 41 against 37).
template <class T, int V, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(1024) void k_norm_fwd(NormFwdParams p) {
  __shared__ float4 red[2][16];
  const int64_t m = blockIdx.x;
  const int H = (int)p.H, waves = blockDim.x >> 6;
  const float inv_h = 1.0f / (float)H;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto ld = [&](const uint16_t *row, int c) {
    return WHOLE ? *reinterpret_cast<const uint4 *>(row + c) : row_ld(row, c, H);
  };
  auto st = [&](uint16_t *row, int c, const uint4 &v) {
    if constexpr (STREAM) row_st_nt(row, c, WHOLE ? c + 8 : H, v);
    else row_st(row, c, WHOLE ? c + 8 : H, v);
  };
  uint4 yv[V], rv[V], wp[V], wg[V], wn[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (threadIdx.x + v * blockDim.x) * 8;
    rv[v] = yv[v] = wp[v] = wg[v] = wn[v] = zero;
    if (c >= H) continue;
    if (p.y) yv[v] = ld(p.y + m * p.ld_y, c);
    rv[v] = ld(p.res + m * p.ld_res, c);
    if (p.w_post) wp[v] = ld(p.w_post, c);
    if (p.gate) wg[v] = ld(p.gate + m * p.ld_gate, c);
    if (p.w_next) wn[v] = ld(p.w_next, c);
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
    row_sums(s, red[0], 0, waves);
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
        row_widen<T>(wp[v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = t[e] * r_y * f[e];
      }
      if (p.gate) {
        row_widen<T>(wg[v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] *= f[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) z[v][e] = fmaf(p.alpha, z[v][e], t[e]);
      st(p.z + m * p.ld_z, c, row_narrow<T>(z[v]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = fmaf(z[v][e], z[v][e], s[0]);
  }
  float r_z = 1.0f;
  if (p.w_next) {
    row_sums(s, red[1], 0, waves);
    r_z = 1.0f / sqrtf(fmaf(s[0], inv_h, p.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (threadIdx.x + v * blockDim.x) * 8;
      if (c >= H) continue;
      float f[8];
      row_widen<T>(wn[v], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= z[v][e] * r_z;
      st(p.h + m * p.ld_h, c, row_narrow<T>(f));
    }
  }
  if (p.rstd && threadIdx.x == 0) {
    p.rstd[2 * m] = r_y;
    p.rstd[2 * m + 1] = r_z;
  }
}

// The backward.  A workgroup holds blockDim / row_threads rows at a time, and
// goes over its own rows in steps of the whole grid's.
//
//   G  = dz + r_z (dn - z r_z^2 mean(dn z)),  dn = dh w_next
//   dres = alpha G,  dgate = G t,  dq = G gate w_post,
//   dy = r_y (dq - y r_y^2 mean(dq y))
//
// mean(dq y) is linear in G, so it follows from two sums that need no other
// sum first: with n = z r_z and q = gate w_post y, sum(G q) = sum((dz + r_z dn) q)
// - c sum(n q), c = r_z mean(dn n).  All three sums of a row take one reduction.
// The normed row n, and y r_y below, take one factor r each: r^3 alone leaves
// FP32's range for rows that do not (1e-45 at a root mean square of 1e15).  The
// column sums dw_post, dw_next and a broadcast dgate stay in registers over
// the workgroup's rows, then its row slots add up through LDS, in order, and
// go to `part` once (FP32, added up by k_norm_wgrad in the order of the
// workgroups, so results do not change from run to run).
//
// PARTS: what is given, where that is known here (no test of it in the loop;
// y without w_post, and dh and y without dz, keep the tests: 48 us at 4096 x 4096
// with a gate for each channel, against 37 with every part).
// The next row is then loaded before this one's reduction, for rows of up to
// 8192 (V <= 2): with dz and dh alone 4096 x 6000 takes 35 us against 55 with the
// tests, with dh alone 26 against 48.  Wider rows leave no registers for a second one
// and keep the weights in LDS (1548 x 9819, no gate: 63 us against 80 read from
// L2 again for every row).  Up to 12288 (V = 3) the next row's dz and dh are
// loaded where this row's are used up, before the reduction, and the rest chunk
// by chunk as the outputs leave (the same: 58; 1500 x 8320: 36 against 46); with
// V <= 2 that is slower than the tests alone (4096 x 6000, inputs in the
// last-level cache: 52 against 47), with V = 4 it spills.  WHOLE: H is a multiple of 8.  Otherwise each load and store has a branch
// for the row's end, and the kernel spills scalar registers: 1003 x 5125 with a
// gate for each element takes 30.5 us, 1003 x 5128 18.5.
enum { GATE_NONE = 0, GATE_ROW = 1, GATE_FULL = 2 };
// dz, dh, y and w_post; dz and dh; dz, y and w_post; dh alone (the last norm of a network)
enum { PARTS_ANY = 0, PARTS_ALL = 1, PARTS_NEXT = 2, PARTS_POST = 3, PARTS_LAST = 4 };

template <int V, int GATE>
struct NormRow {
  uint4 dz[V], dh[V], z[V], y[V], gate[GATE == GATE_FULL ? V : 1];
  float r_y, r_z;
};

template <class T, int V, int GATE, int PARTS, bool WHOLE>
__global__ __launch_bounds__(kBwdThreads, V == 1 ? 4 : 2) void k_norm_bwd(NormBwdParams p, int row_threads) {
  __shared__ float4 red[2][kBwdThreads / 64];
  // round8(H) column sums, when a workgroup holds several rows; with V > 2 the
  // weights, [w_post, w_next, gate][V][thread] chunks of 8
  extern __shared__ __attribute__((aligned(16))) float cols[];
  constexpr bool AHEAD = PARTS != PARTS_ANY && V <= 2, IN_PLACE = V == 3, WIDE = V > 2;
  const int H = (int)p.H;
  const float inv_h = 1.0f / (float)H;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr bool any = PARTS == PARTS_ANY, block = PARTS == PARTS_ALL || PARTS == PARTS_POST;
  const bool has_dz = any ? p.dz != nullptr : PARTS != PARTS_LAST, has_dh = any ? p.dh != nullptr : PARTS != PARTS_POST;
  const bool has_y = any ? p.y != nullptr : block, has_post = any ? p.w_post != nullptr : block;
  const int slots = blockDim.x / row_threads, slot = __builtin_amdgcn_readfirstlane(threadIdx.x / row_threads);
  const int tid = threadIdx.x - slot * row_threads;
  const int w0 = slot * (row_threads >> 6), waves = row_threads >> 6;
  auto ld = [&](const uint16_t *row, int c) {
    return WHOLE ? *reinterpret_cast<const uint4 *>(row + c) : row_ld(row, c, H);
  };
  auto st = [&](uint16_t *row, int c, const uint4 &v) {
    if constexpr (WHOLE) *reinterpret_cast<uint4 *>(row + c) = v;
    else row_st(row, c, H, v);
  };
  auto col = [&](int v) { return (tid + v * row_threads) * 8; };
  float ap[V][8] = {}, an[V][8] = {}, ag[V][8] = {};
  uint4 wp[V], wn[V], wg[V];  // w_post, w_next and a broadcast gate
  // a chunk's parts that the row's sums alone need, and those its outputs need too
  auto load_sums = [&](int64_t m, NormRow<V, GATE> &r, int v) {
    const int c = col(v);
    r.dz[v] = r.dh[v] = zero;
    if (c >= H) return;
    if (has_dz) r.dz[v] = ld(p.dz + m * p.ld_dz, c);
    if (has_dh) r.dh[v] = ld(p.dh + m * p.ld_dh, c);
  };
  auto load_both = [&](int64_t m, NormRow<V, GATE> &r, int v) {
    const int c = col(v);
    r.z[v] = r.y[v] = zero;
    if constexpr (GATE == GATE_FULL) r.gate[v] = zero;
    if (c >= H) return;
    if (has_dh) r.z[v] = ld(p.z + m * p.ld_z, c);
    if (has_y) r.y[v] = ld(p.y + m * p.ld_y, c);
    if constexpr (GATE == GATE_FULL) r.gate[v] = ld(p.gate + m * p.ld_gate, c);
  };
  auto load_r = [&](int64_t m, NormRow<V, GATE> &r) {
    r.r_y = p.rstd[2 * m];
    r.r_z = p.rstd[2 * m + 1];
  };
  auto load = [&](int64_t m, NormRow<V, GATE> &r) {
    load_r(m, r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      load_sums(m, r, v);
      load_both(m, r, v);
    }
  };
  auto fetch = [&](int v) {
    const int c = col(v);
    wp[v] = wn[v] = wg[v] = zero;
    if (c >= H) return;
    if (has_post) wp[v] = ld(p.w_post, c);
    if (has_dh) wn[v] = ld(p.w_next, c);
    if constexpr (GATE == GATE_ROW) wg[v] = ld(p.gate, c);
  };
  uint4 *kept = reinterpret_cast<uint4 *>(cols) + threadIdx.x;  // each thread its own
  auto weights = [&](int v) {
    if constexpr (WIDE) {
      wp[v] = kept[v * blockDim.x];
      wn[v] = kept[(V + v) * blockDim.x];
      if constexpr (GATE == GATE_ROW) wg[v] = kept[(2 * V + v) * blockDim.x];
    } else if constexpr (!AHEAD) {
      fetch(v);
    }
  };
  if constexpr (AHEAD || WIDE)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      fetch(v);
      if constexpr (WIDE) {
        kept[v * blockDim.x] = wp[v];
        kept[(V + v) * blockDim.x] = wn[v];
        if constexpr (GATE == GATE_ROW) kept[(2 * V + v) * blockDim.x] = wg[v];
      }
    }
  NormRow<V, GATE> cur, next;
  const int64_t step = (int64_t)gridDim.x * slots;
  // a slot past the last row repeats it and keeps nothing (its waves still meet the others at the barrier)
  int64_t m = (int64_t)blockIdx.x * slots + slot;
  load(m < p.M ? m : p.M - 1, cur);
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * slots; base < p.M; base += step, m += step, turn ^= 1) {
    const bool live = m < p.M;
    const int64_t after = m + step < p.M ? m + step : p.M - 1;
    if constexpr (AHEAD) load(after, next);
    const float r_y = cur.r_y, r_z = cur.r_z;
    float g0[V][8], s[3] = {0.0f, 0.0f, 0.0f};  // g0 = dz + r_z dn
#pragma unroll
    for (int v = 0; v < V; ++v) {
      weights(v);
      float z[8], f[8];
      row_widen<T>(cur.dz[v], g0[v]);
      row_widen<T>(cur.z[v], z);
      if (has_dh) {
        float dh[8];
        row_widen<T>(cur.dh[v], dh);
        row_widen<T>(wn[v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] *= r_z;
        if (live)  // not by a factor of 0: the row repeated may hold infinities
#pragma unroll
          for (int e = 0; e < 8; ++e) an[v][e] = fmaf(dh[e], z[e], an[v][e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float dn = dh[e] * f[e];
          s[0] = fmaf(dn, z[e], s[0]);
          g0[v][e] = fmaf(r_z, dn, g0[v][e]);
        }
      }
      if (has_post) {
        float q[8];
        row_widen<T>(cur.y[v], q);
        row_widen<T>(wp[v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] *= f[e];
        if constexpr (GATE != GATE_NONE) {
          row_widen<T>(GATE == GATE_FULL ? cur.gate[v] : wg[v], f);
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
    if constexpr (IN_PLACE) {  // the next row's, where this one's are used up
      load_r(after, cur);
#pragma unroll
      for (int v = 0; v < V; ++v) load_sums(after, cur, v);
    }
    row_sums(s, red[turn], w0, waves);  // two sets in turn: no barrier between a row's reads and the next row's writes
    const float cz = has_dh ? r_z * (s[0] * inv_h) : 0.0f;
    const float cy = has_post ? r_y * (r_y * ((s[1] - cz * s[2]) * inv_h)) : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = col(v);
      if (c >= H || !live) continue;
      weights(v);
      float z[8], o[8];
      row_widen<T>(cur.z[v], z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g0[v][e] = fmaf(-cz, z[e] * r_z, g0[v][e]);
        o[e] = p.alpha * g0[v][e];
      }
      st(p.dres + m * p.ld_dres, c, row_narrow<T>(o));
      if (!has_y) {
        if constexpr (IN_PLACE) load_both(after, cur, v);
        continue;
      }
      float y[8], w[8], f[8];
      row_widen<T>(cur.y[v], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      if (has_post) row_widen<T>(wp[v], w);
      if constexpr (GATE != GATE_NONE) {  // dgate = G t, t = y r_y w_post
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = g0[v][e] * (y[e] * r_y * w[e]);
        if constexpr (GATE == GATE_ROW) {
#pragma unroll
          for (int e = 0; e < 8; ++e) ag[v][e] += o[e];
        } else if (p.dgate) {
          st(p.dgate + m * p.ld_dgate, c, row_narrow<T>(o));
        }
        row_widen<T>(GATE == GATE_FULL ? cur.gate[v] : wg[v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) g0[v][e] *= f[e];
      }
      if (has_post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = y[e] * r_y;
          ap[v][e] = fmaf(g0[v][e], n, ap[v][e]);
          g0[v][e] = fmaf(r_y * w[e], g0[v][e], -cy * n);
        }
      }
      if constexpr (IN_PLACE) load_both(after, cur, v);
      st(p.dy + m * p.ld_dy, c, row_narrow<T>(g0[v]));
    }
    if constexpr (AHEAD) cur = next;
    else if constexpr (!IN_PLACE) load(after, cur);
  }
  const int64_t ldp = (p.H + 7) & ~(int64_t)7;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k == 0 ? !p.dw_post : k == 1 ? !p.dw_next : GATE != GATE_ROW || !p.dgate) continue;
    auto &sum = k == 0 ? ap : k == 1 ? an : ag;
    // the row slots one after the other; the last writes the workgroup's part
    for (int t = 0; t < slots; ++t) {
      if (slots > 1) __syncthreads();
      if (slot != t) continue;
      float *out = t == slots - 1 ? p.part + ((int64_t)k * gridDim.x + blockIdx.x) * ldp : cols;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = col(v);
        if (c >= H) continue;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          f32x4 a = {sum[v][e], sum[v][e + 1], sum[v][e + 2], sum[v][e + 3]};
          if (t > 0) a = *reinterpret_cast<const f32x4 *>(cols + c + e) + a;
          *reinterpret_cast<f32x4 *>(out + c + e) = a;
        }
      }
    }
    if (slots > 1) __syncthreads();
  }
}

// Column sums over the workgroups' parts: 64 columns per workgroup, 16 waves
// each over a contiguous sixteenth of the parts, the sixteenths added in order.
constexpr int kSumWaves = 16;

template <class T>
__global__ __launch_bounds__(64 * kSumWaves) void k_norm_wgrad(NormBwdParams p) {
  __shared__ float red[kSumWaves][64];
  const int which = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint16_t *out = which == 0 ? p.dw_post : which == 1 ? p.dw_next : p.ld_gate == 0 ? p.dgate : nullptr;
  if (!out) return;
  const int64_t ldp = (p.H + 7) & ~(int64_t)7, c = (int64_t)blockIdx.x * 64 + lane;
  const int lo = p.groups * wave / kSumWaves, hi = p.groups * (wave + 1) / kSumWaves;
  const float *part = p.part + (int64_t)which * p.groups * ldp + c;
  float t = 0.0f;
  if (c < p.H) {
#pragma unroll 8
    for (int g = lo; g < hi; ++g) t += part[g * ldp];
  }
  red[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && c < p.H) {
#pragma unroll
    for (int w = 1; w < kSumWaves; ++w) t += red[w][lane];
    out[c] = T::r(t);
  }
}

// Threads of a row that take V chunks of 8 each, in whole waves.
int row_threads(int64_t H, int V) {
  const int64_t chunks = (H + 7) / 8, threads = (chunks + V - 1) / V;
  return (int)((threads + 63) / 64 * 64);
}

// Chunks of 8 a backward thread: with two, half the reductions and no spilled
// registers (4096 x 4096: 37 us against 49, 16384 x 1024: 40 against 45); below
// 1024 a wave would be left half empty (3000 x 700: 24 us against 17).  Past 8192
// as many as 512 threads need (1024 threads of two chunks spill: 113 us against
// 80 at 1548 x 9819).
int bwd_chunks(int64_t H) { return H < 1024 ? 1 : H <= 16 * kBwdThreads ? 2 : H <= 24 * kBwdThreads ? 3 : 4; }

// Workgroups that fit the card at once: two a CU with V = 1, else one.
int64_t bwd_most_groups(int64_t H) { return bwd_chunks(H) == 1 ? 512 : 256; }

// Rows a workgroup holds at a time: as many as its threads take, but no more
// than keep all CUs at work.
int bwd_slots(int64_t M, int64_t H) {
  const int64_t fit = kBwdThreads / row_threads(H, bwd_chunks(H)), want = (M + bwd_most_groups(H) - 1) / bwd_most_groups(H);
  return (int)(want < fit ? want : fit);
}

}  // namespace

template <class T, int V, bool WHOLE>
static void norm_fwd_t(const NormFwdParams &p, hipStream_t s) {
  const dim3 g((unsigned)p.M), b(row_threads(p.H, V));
  if (p.M * p.H >= kStreamElements) dgf_launch((k_norm_fwd<T, V, WHOLE, true>), g, b, 0, s, p);
  else dgf_launch((k_norm_fwd<T, V, WHOLE, false>), g, b, 0, s, p);
}

hipError_t launch_norm_fwd(const NormFwdParams &p, hipStream_t s) {
  switch (4 * (p.fmt == FMT_F16) + 2 * (p.H > 8192) + (p.H % 8 == 0)) {
    case 0: norm_fwd_t<Bf16, 1, false>(p, s); break;
    case 1: norm_fwd_t<Bf16, 1, true>(p, s); break;
    case 2: norm_fwd_t<Bf16, 2, false>(p, s); break;
    case 3: norm_fwd_t<Bf16, 2, true>(p, s); break;
    case 4: norm_fwd_t<F16, 1, false>(p, s); break;
    case 5: norm_fwd_t<F16, 1, true>(p, s); break;
    case 6: norm_fwd_t<F16, 2, false>(p, s); break;
    default: norm_fwd_t<F16, 2, true>(p, s); break;
  }
  return hipGetLastError();
}

int norm_bwd_groups(int64_t M, int64_t H) {
  const int64_t most = bwd_most_groups(H), slots = bwd_slots(M, H), need = (M + slots - 1) / slots;
  return (int)(need < most ? need : most);
}

template <class T, int V, int GATE>
static void norm_bwd_v(const NormBwdParams &p, hipStream_t s) {
  const int rt = row_threads(p.H, V), slots = bwd_slots(p.M, p.H);
  const dim3 g((unsigned)p.groups), b(rt * slots);
  const size_t lds = V > 2 ? (size_t)(GATE == GATE_ROW ? 3 : 2) * V * rt * 16
                   : slots > 1 ? (size_t)((p.H + 7) & ~(int64_t)7) * 4 : 0;
  const bool whole = p.H % 8 == 0;
  int parts = PARTS_ANY;
  if (p.dz && p.dh && p.y && p.w_post) parts = PARTS_ALL;
  else if (p.dh && !p.y) parts = p.dz ? PARTS_NEXT : PARTS_LAST;
  else if (p.dz && !p.dh && p.y && p.w_post) parts = PARTS_POST;
#define DGF_BWD(parts_, whole_) dgf_launch((k_norm_bwd<T, V, GATE, parts_, whole_>), g, b, lds, s, p, rt)
  if constexpr (V <= 2) {
    if constexpr (GATE == GATE_NONE) {
      if (parts == PARTS_NEXT) return whole ? DGF_BWD(PARTS_NEXT, true) : DGF_BWD(PARTS_NEXT, false);
      if (parts == PARTS_LAST) return whole ? DGF_BWD(PARTS_LAST, true) : DGF_BWD(PARTS_LAST, false);
    }
    if (parts == PARTS_ALL) return whole ? DGF_BWD(PARTS_ALL, true) : DGF_BWD(PARTS_ALL, false);
    if (parts == PARTS_POST) return whole ? DGF_BWD(PARTS_POST, true) : DGF_BWD(PARTS_POST, false);
    return DGF_BWD(PARTS_ANY, false);
  } else {
    // the tests cost less than the registers that the compiler spends without them, but for this
    if constexpr (V == 3 && GATE != GATE_ROW)
      if (parts == PARTS_ALL && whole) return DGF_BWD(PARTS_ALL, true);
    return whole ? DGF_BWD(PARTS_ANY, true) : DGF_BWD(PARTS_ANY, false);
  }
#undef DGF_BWD
}

template <class T, int GATE>
static void norm_bwd_t(const NormBwdParams &p, hipStream_t s) {
  switch (bwd_chunks(p.H)) {
    case 1: norm_bwd_v<T, 1, GATE>(p, s); break;
    case 2: norm_bwd_v<T, 2, GATE>(p, s); break;
    case 3: norm_bwd_v<T, 3, GATE>(p, s); break;
    default: norm_bwd_v<T, 4, GATE>(p, s); break;
  }
}

hipError_t launch_norm_bwd(const NormBwdParams &p, hipStream_t s) {
  const int gate = !p.gate ? GATE_NONE : p.ld_gate == 0 ? GATE_ROW : GATE_FULL;
  switch (gate * 2 + (p.fmt == FMT_F16)) {
    case 0: norm_bwd_t<Bf16, GATE_NONE>(p, s); break;
    case 1: norm_bwd_t<F16, GATE_NONE>(p, s); break;
    case 2: norm_bwd_t<Bf16, GATE_ROW>(p, s); break;
    case 3: norm_bwd_t<F16, GATE_ROW>(p, s); break;
    case 4: norm_bwd_t<Bf16, GATE_FULL>(p, s); break;
    default: norm_bwd_t<F16, GATE_FULL>(p, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_norm_wgrad(const NormBwdParams &p, hipStream_t s) {
  const dim3 g((unsigned)((p.H + 63) / 64), 3);
  if (p.fmt == FMT_F16) dgf_launch(k_norm_wgrad<F16>, g, dim3(64 * kSumWaves), 0, s, p);
  else dgf_launch(k_norm_wgrad<Bf16>, g, dim3(64 * kSumWaves), 0, s, p);
  return hipGetLastError();
}

}  // namespace dgf
