// A mixture-of-experts layer for a few tokens (gfx950), every expert the gated FFN:
//
//   l = x W_r^T;  the k largest l of a token choose its experts (ties: lowest index)
//   p = softmax of l over all E experts, or over the k chosen (renorm)
//   a_j = silu(W_gate[e_j] x) (W_up[e_j] x);  y = sum_j p_j W_down[e_j] a_j
//
// Every chosen expert's weights are read once, whatever number of tokens chose
// it: 3 H I 16-bit values for 6 H I operations a token, so up to about a
// hundred tokens an expert the layer is bound by the weights' way from HBM.
// Four launches: the router's products, the choice and the experts' token
// lists (one workgroup), the gate/up products with the activation, and the
// down products with the weighted sum over a token's experts.
//
// Products run on the matrix cores with FP32 accumulators, 8 weight rows and 8
// tokens per 16 x 16 x 32 instruction: rows 0-7 and 8-15 of the first operand
// are the same weight rows at K and K + 32, columns 0-7 and 8-15 of the second
// the same tokens at K and K + 32, so the two diagonal 8 x 8 blocks of the
// result add up to the product over 64 K (the other two are unused).  One load
// instruction then takes whole 128-byte lines, and a weight row's tile is
// narrow enough to give every CU work at one token.
//
// A token's result depends on that token alone: the K split is a function of
// H, I and k only, sums run in a fixed order, and nothing is atomic.
#include "dgf_block.hpp"
#include "dgf_device.hpp"

namespace dgf {
namespace {

constexpr int kWaves = 8;  // of the gate/up and down workgroups

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Router products, on the vector unit in FP32 (the matrix core truncates, and
// a logit's last bits decide ties): a wave per expert and kLogitTokens tokens.
constexpr int kLogitTokens = 4;

template <class T>
__global__ __launch_bounds__(256) void k_moe_logits(MoeParams p) {
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (e >= p.E) return;
  const int m0 = blockIdx.y * kLogitTokens;
  const uint16_t *w = p.w_router + (int64_t)e * p.ld_wr;
  float acc[kLogitTokens] = {};
  for (int c = lane * 8; c < p.H; c += 512) {
    const u16x8 wv = __builtin_bit_cast(u16x8, load_frag_tail<T>(w, c, p.H));
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t) {
      if (m0 + t >= p.M) break;
      const u16x8 xv = __builtin_bit_cast(u16x8, load_frag_tail<T>(p.x + (m0 + t) * p.ldx, c, p.H));
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fmaf(T::f(wv[i]), T::f(xv[i]), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t) {
    const float l = wave_sum(acc[t]);
    if (lane == 0 && m0 + t < p.M) p.logits[(int64_t)(m0 + t) * p.E + e] = l;
  }
}

// Order of logits as integers: larger float, larger integer; NaN lowest; never 0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 1u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One workgroup: each wave chooses for its tokens, then lists for its experts.
constexpr int kRouteThreads = 1024;

__global__ __launch_bounds__(kRouteThreads) void k_moe_route(MoeParams p) {
  __shared__ int ids[kMoeMaxM * kMoeMaxK];
  __shared__ int cnt[kMoeMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = kRouteThreads / 64;
  for (int m = wave; m < p.M; m += waves) {
    const float *l = p.logits + (int64_t)m * p.E;
    float v[kMoeMaxE / 64];
    uint32_t key[kMoeMaxE / 64];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMoeMaxE / 64; ++i) {
      const int e = lane + 64 * i;
      v[i] = e < p.E ? l[e] : -INFINITY;
      key[i] = e < p.E ? logit_key(v[i]) : 0u;
      top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    float mine = -INFINITY;
    int chosen = 0;
    for (int j = 0; j < p.k; ++j) {
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < kMoeMaxE / 64; ++i) {
        const uint64_t b = (uint64_t)key[i] << 32 | (uint32_t)~(lane + 64 * i);
        if (key[i] && b > best) best = b;
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        const uint64_t b = (uint64_t)__shfl_xor((unsigned long long)best, o);
        best = b > best ? b : best;
      }
      const int e = (int)~(uint32_t)best;
#pragma unroll
      for (int i = 0; i < kMoeMaxE / 64; ++i)
        if (e == lane + 64 * i) key[i] = 0u;
      if (lane == j) {
        chosen = e;
        mine = l[e];
      }
    }
    float part = 0.0f;
    if (p.renorm) {
      part = lane < p.k ? expf(mine - top) : 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < kMoeMaxE / 64; ++i)
        if (lane + 64 * i < p.E) part += expf(v[i] - top);
    }
    const float sum = wave_sum(part);
    if (lane < p.k) {
      const float w = expf(mine - top) / sum;
      const int at = m * p.k + lane;
      ids[at] = chosen;
      p.ids[at] = chosen;
      p.p[at] = w;
      if (p.ids_out) p.ids_out[at] = chosen;
      if (p.p_out) p.p_out[at] = w;
    }
  }
  __syncthreads();
  const int n = p.M * p.k;
  for (int e = wave; e < p.El; e += waves) {
    int c = 0;
    for (int b = 0; b < n; b += 64) {
      const bool hit = b + lane < n && ids[b + lane] == p.e0 + e;
      const uint64_t mask = __ballot(hit);
      if (hit) p.pairs[(int64_t)e * p.M + c + __popcll(mask & ((1ull << lane) - 1))] = b + lane;
      c += __popcll(mask);
    }
    if (lane == 0) cnt[e] = p.count[e] = c;
  }
  __syncthreads();
  if (wave == 0) {
    int c = 0;
    for (int b = 0; b < p.El; b += 64) {
      const bool hit = b + lane < p.El && cnt[b + lane] > 0;
      const uint64_t mask = __ballot(hit);
      if (hit) p.active[1 + c + __popcll(mask & ((1ull << lane) - 1))] = b + lane;
      c += __popcll(mask);
    }
    if (lane == 0) p.active[0] = c;
  }
}

// The two diagonal 8 x 8 blocks of an accumulator added: rows 4 q + i (q < 2)
// and column lane & 7 in the lanes with bit 3 clear below lane 32.
__device__ __forceinline__ f32x4 diagonal(const f32x4 &acc) {
  f32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = acc[i] + __shfl(acc[i], (threadIdx.x + 40) & 63);
  return v;
}

template <class T>
__device__ __forceinline__ typename T::frag zero_frag() {
  return __builtin_bit_cast(typename T::frag, u16x8{0, 0, 0, 0, 0, 0, 0, 0});
}

// A workgroup: 8 rows of an active expert's W_gate and W_up against all its
// tokens, 8 at a time; each wave an eighth of K.  The activation a leaves in
// two stored parts whose sum keeps twice the stored type's bits, so that
// rounding it adds nothing to the output's own rounding.
template <class T>
__global__ __launch_bounds__(64 * kWaves) void k_moe_gate_up(MoeParams p) {
  __shared__ float red[kWaves][2][8][8];
  if ((int)blockIdx.y >= p.active[0]) return;
  const int e = p.active[1 + blockIdx.y], cnt = p.count[e];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 7, q = lane >> 4, at = ((lane >> 3) & 1) * 32 + q * 8;
  const int i0 = blockIdx.x * 8;
  const int row = i0 + c < p.I ? i0 + c : p.I - 1;
  const uint16_t *wg = p.w_gate + e * p.st_wg + row * p.ld_wg;
  const uint16_t *wu = p.w_up + e * p.st_wu + row * p.ld_wu;
  const int steps = (p.H + 63) / 64, lo = steps * wave / kWaves, hi = steps * (wave + 1) / kWaves;
  const int *pairs = p.pairs + (int64_t)e * p.M;
  for (int t0 = 0; t0 < cnt; t0 += 8) {
    const bool has = t0 + c < cnt;
    const uint16_t *x = p.x + (has ? pairs[t0 + c] / p.k : 0) * p.ldx;
    f32x4 ag = {0.f, 0.f, 0.f, 0.f}, au = ag;
    for (int s = lo; s < hi; ++s) {
      const int k = s * 64 + at;
      const typename T::frag fg = load_frag_tail<T>(wg, k, p.H), fu = load_frag_tail<T>(wu, k, p.H);
      const typename T::frag fx = has ? load_frag_tail<T>(x, k, p.H) : zero_frag<T>();
      ag = T::mfma(fg, fx, ag);
      au = T::mfma(fu, fx, au);
    }
    const f32x4 g = diagonal(ag), u = diagonal(au);
    if (lane < 32 && (lane & 8) == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        red[wave][0][c][q * 4 + i] = g[i];
        red[wave][1][c][q * 4 + i] = u[i];
      }
    __syncthreads();
    if (threadIdx.x < 64) {
      const int tok = threadIdx.x >> 3, r = threadIdx.x & 7;
      float gs = 0.0f, us = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        gs += red[w][0][tok][r];
        us += red[w][1][tok][r];
      }
      if (t0 + tok < cnt && i0 + r < p.I) {
        const float a = gs * sigma_f(gs) * us;
        const uint16_t h = T::r(a);
        const int64_t o = pairs[t0 + tok] * p.lda + i0 + r;
        p.a_hi[o] = h;
        p.a_lo[o] = T::r(a - T::f(h));
      }
    }
    __syncthreads();
  }
}

// A workgroup: 8 rows of y.  Its waves work in groups of `wps`, a group on one
// active expert at a time, each wave of it a share of K = I; wps is 8 / k
// (down to a power of two), so that the experts of a single token keep all
// waves busy.  Each (token, choice) pair's partial products are kept in LDS
// and added up in order at the end: the waves' shares, then the choices by p.
template <class T>
__global__ __launch_bounds__(64 * kWaves) void k_moe_down(MoeParams p, int wps) {
  extern __shared__ float part[];  // [M k][wps][8 rows]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 7, q = lane >> 4, at = ((lane >> 3) & 1) * 32 + q * 8;
  const int h0 = blockIdx.x * 8;
  const int row = h0 + c < p.H ? h0 + c : p.H - 1;
  const int sub = wave & (wps - 1), groups = kWaves / wps;
  const int steps = (p.I + 63) / 64, lo = steps * sub / wps, hi = steps * (sub + 1) / wps;
  const int n = p.active[0];
  for (int s0 = wave / wps; s0 < n; s0 += groups) {
    const int e = p.active[1 + s0], cnt = p.count[e];
    const uint16_t *w = p.w_down + e * p.st_wd + row * p.ld_wd;
    const int *pairs = p.pairs + (int64_t)e * p.M;
    for (int t0 = 0; t0 < cnt; t0 += 8) {
      const bool has = t0 + c < cnt;
      const int pair = has ? pairs[t0 + c] : 0;
      const uint16_t *ah = p.a_hi + pair * p.lda, *al = p.a_lo + pair * p.lda;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f}, acl = acc;
      for (int s = lo; s < hi; ++s) {
        const int k = s * 64 + at;
        const typename T::frag fw = load_frag_tail<T>(w, k, p.I);
        acc = T::mfma(fw, has ? load_frag_tail<T>(ah, k, p.I) : zero_frag<T>(), acc);
        acl = T::mfma(fw, has ? load_frag_tail<T>(al, k, p.I) : zero_frag<T>(), acl);
      }
      const f32x4 v = diagonal(acc + acl);
      if (lane < 32 && (lane & 8) == 0 && has)
        *reinterpret_cast<f32x4 *>(&part[(pair * wps + sub) * 8 + q * 4]) = v;
    }
  }
  __syncthreads();
  for (int o = threadIdx.x; o < p.M * 8; o += 64 * kWaves) {
    const int m = o >> 3, r = o & 7;
    if (h0 + r >= p.H) continue;
    float y = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const int e = p.ids[m * p.k + j] - p.e0;
      if (e < 0 || e >= p.El) continue;
      float t = 0.0f;
      for (int w = 0; w < wps; ++w) t += part[((m * p.k + j) * wps + w) * 8 + r];
      y = fmaf(p.p[m * p.k + j], t, y);
    }
    p.y[m * p.ldy + h0 + r] = T::r(y);
  }
}

}  // namespace

hipError_t launch_moe_logits(const MoeParams &p, hipStream_t s) {
  const dim3 g((p.E + 3) / 4, (p.M + kLogitTokens - 1) / kLogitTokens);
  if (p.fmt == FMT_F16) dgf_launch(k_moe_logits<F16>, g, dim3(256), 0, s, p);
  else dgf_launch(k_moe_logits<Bf16>, g, dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_moe_route(const MoeParams &p, hipStream_t s) {
  dgf_launch(k_moe_route, dim3(1), dim3(kRouteThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_moe_gate_up(const MoeParams &p, hipStream_t s) {
  const int slots = p.M * p.k < p.El ? p.M * p.k : p.El;  // at most this many experts have tokens
  const dim3 g((p.I + 7) / 8, slots);
  if (p.fmt == FMT_F16) dgf_launch(k_moe_gate_up<F16>, g, dim3(64 * kWaves), 0, s, p);
  else dgf_launch(k_moe_gate_up<Bf16>, g, dim3(64 * kWaves), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_moe_down(const MoeParams &p, hipStream_t s) {
  int wps = 1;
  while (wps * 2 * p.k <= kWaves) wps *= 2;
  const dim3 g((p.H + 7) / 8);
  const size_t lds = (size_t)p.M * p.k * wps * 8 * 4;  // at most 64 KB: M k wps <= 2048
  if (p.fmt == FMT_F16) dgf_launch(k_moe_down<F16>, g, dim3(64 * kWaves), lds, s, p, wps);
  else dgf_launch(k_moe_down<Bf16>, g, dim3(64 * kWaves), lds, s, p, wps);
  return hipGetLastError();
}

}  // namespace dgf
