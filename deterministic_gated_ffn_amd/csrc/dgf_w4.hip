// Products with 4-bit weights and group scales for a few tokens (gfx950).
#include "dgf_experts.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

constexpr int kW4Rows = 16, kW4K = 128;  // weights of a tile: 1 KB of codes, 16 bytes a lane
constexpr int kW4Waves = 8;

__host__ __device__ inline int w4_tiles_k(int K) { return (K + kW4K - 1) / kW4K; }

// A tile's lane l holds row l % 16 and, in dword i, the eight columns from
// 32 i + 8 (l / 16): column 2 d in bits 4 d.., column 2 d + 1 in bits 16 + 4 d.. .
__device__ __forceinline__ int code_shift(int c) { return 4 * (c >> 1) + 16 * (c & 1); }

// ---------------------------------------------------------------- packing

template <class T>
__global__ __launch_bounds__(256) void k_pack4(const uint16_t *w, int64_t ldw, uint8_t *q, uint16_t *s, int N, int K, int group) {
  const int tiles_k = w4_tiles_k(K), lane = threadIdx.x & 63;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= (int64_t)((N + kW4Rows - 1) / kW4Rows) * tiles_k) return;
  const int n = (int)(tile / tiles_k) * kW4Rows + (lane & 15), k0 = (int)(tile % tiles_k) * kW4K + 8 * (lane >> 4);
  float f[4][8];
  float top[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = k0 + 32 * i;
    row_widen<T>(n < N && k < K ? row_ld(w + (int64_t)n * ldw, k, K) : make_uint4(0, 0, 0, 0), f[i]);
    // largest magnitude of 32 columns, as bits (NaN above infinity above the finite)
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(f[i][e]) & 0x7fffffffu;
      m = b > m ? b : m;
    }
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) {
      const uint32_t b = (uint32_t)__shfl_xor((int)m, o);
      m = b > m ? b : m;
    }
    top[i] = __uint_as_float(m);
  }
  const int per = group / 32;  // 32-column parts of a group
  uint32_t word[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = 0.0f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j / per == i / per) {
        bad |= !(top[j] < __builtin_inff());
        a = fmaxf(a, top[j]);
      }
    uint16_t sb = bad ? (T::code ? 0x7e00 : 0x7fc0) : T::r(a / 7.0f);
    // the next lower scale where the largest code would read back as infinity
    if (!bad && !(T::f(T::r(7.0f * T::f(sb))) < __builtin_inff())) --sb;
    const float sf = T::f(sb);
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = sf > 0.0f ? fminf(fmaxf(rintf(f[i][e] / sf), -7.0f), 7.0f) : 0.0f;
      c |= (uint32_t)((int)v + 8) << code_shift(e);
    }
    word[i] = c;
    if (lane < 16 && i % per == 0) s[(tile * 16 + lane) * (kW4K / group) + i / per] = sb;
  }
  *reinterpret_cast<uint4 *>(q + (tile * 64 + lane) * 16) = make_uint4(word[0], word[1], word[2], word[3]);
}

template <class T>
__global__ __launch_bounds__(256) void k_unpack4(W4Mat m, uint16_t *w, int64_t ldw, int N, int K, int group) {
  const int tiles_k = w4_tiles_k(K), lane = threadIdx.x & 63;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= (int64_t)((N + kW4Rows - 1) / kW4Rows) * tiles_k) return;
  const int n = (int)(tile / tiles_k) * kW4Rows + (lane & 15), k0 = (int)(tile % tiles_k) * kW4K + 8 * (lane >> 4);
  if (n >= N) return;
  const uint4 c = *reinterpret_cast<const uint4 *>(m.q + (tile * 64 + lane) * 16);
  const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = k0 + 32 * i;
    if (k >= K) continue;
    const float sf = T::f(m.s[(tile * 16 + (lane & 15)) * (kW4K / group) + 32 * i / group]);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)((int)(word[i] >> code_shift(e) & 15) - 8) * sf;
    row_st(w + (int64_t)n * ldw, k, K, row_narrow<T>(f));
  }
}

// ---------------------------------------------------------------- products

// Eight codes as an MFMA operand, each as 16 + code (= 24 + c for the signed c):
// the code's four bits go under the leading one of 16.0.
template <class T>
__device__ __forceinline__ typename T::frag code_frag(uint32_t w) {
  uint4 v;
  if constexpr (T::code == 0) {
    v = make_uint4((w << 3 & 0x00780078u) | 0x41804180u, (w >> 1 & 0x00780078u) | 0x41804180u,
                   (w >> 5 & 0x00780078u) | 0x41804180u, (w >> 9 & 0x00780078u) | 0x41804180u);
  } else {
    v = make_uint4((w << 6 & 0x03c003c0u) | 0x4c004c00u, (w << 2 & 0x03c003c0u) | 0x4c004c00u,
                   (w >> 2 & 0x03c003c0u) | 0x4c004c00u, (w >> 6 & 0x03c003c0u) | 0x4c004c00u);
  }
  return __builtin_bit_cast(typename T::frag, v);
}
template <class T>
__device__ __forceinline__ typename T::frag bias_frag() {  // -24 throughout
  const uint32_t b = T::code == 0 ? 0xc1c0c1c0u : 0xce00ce00u;
  return __builtin_bit_cast(typename T::frag, make_uint4(b, b, b, b));
}

// The activation a of a gate/up pair, as two BF16 values whose sum is a to 2^-17.
__device__ __forceinline__ void split2(float a, uint16_t &hi, uint16_t &lo) {
  hi = f2bf(a);
  const float h = bf2f(hi);
  lo = h - h == 0.0f ? f2bf(a - h) : 0;
}

// X: the activations' MFMA type.  S: the scales' (and the output's) type.
// NT row tiles of the weights a workgroup (PAIR: NT of gate and NT of up), MT
// tiles of 16 tokens, XP parts the activations come in.
template <class X, class S, int MT, int NT, int XP, bool PAIR>
__global__ __launch_bounds__(64 * kW4Waves) void k_w4(W4Params p) {
  constexpr int W = PAIR ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) float red[];  // [waves][W NT MT][4][64]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int tiles_k = w4_tiles_k(p.K), tiles_n = (p.N + kW4Rows - 1) / kW4Rows;
  const int nt0 = blockIdx.x * NT;
  const int64_t m0 = (int64_t)blockIdx.y * 16 * MT;
  const int gs = kW4K / p.group;  // scales a row and tile

  f32x4 acc[W][NT][MT];
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[w][n][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  const typename X::frag bias = bias_frag<X>();
  for (int kt = wave; kt < tiles_k; kt += kW4Waves) {
    uint4 code[W][NT];
    float sc[W][NT][4];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int nt = nt0 + n < tiles_n ? nt0 + n : tiles_n - 1;
        const int64_t t = (int64_t)nt * tiles_k + kt;
        code[w][n] = *reinterpret_cast<const uint4 *>(p.w[w].q + (t * 64 + lane) * 16);
#pragma unroll
        for (int q = 0; q < 4; ++q) sc[w][n][q] = q < gs ? S::f(p.w[w].s[(t * 16 + i16) * gs + q]) : 0.0f;
      }
    uint4 x[XP][MT][4];
#pragma unroll
    for (int xp = 0; xp < XP; ++xp)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t row = m0 + 16 * m + i16;
          const int k = kt * kW4K + 32 * i + 8 * g;
          x[xp][m][i] = make_uint4(0, 0, 0, 0);
          if (row < p.M && k < p.K) x[xp][m][i] = row_ld((xp ? p.x2 : p.x) + row * p.ldx, k, p.K);
        }
    const int per = 4 / gs;  // 32-column parts of a group
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q >= gs) break;
      f32x4 c0[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        c0[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i / per == q)
#pragma unroll
            for (int xp = 0; xp < XP; ++xp) c0[m] = X::mfma(__builtin_bit_cast(typename X::frag, x[xp][m][i]), bias, c0[m]);
      }
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f32x4 part[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m] = c0[m];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i / per == q) {
              const uint32_t word = i == 0 ? code[w][n].x : i == 1 ? code[w][n].y : i == 2 ? code[w][n].z : code[w][n].w;
              const typename X::frag f = code_frag<X>(word);
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int xp = 0; xp < XP; ++xp) part[m] = X::mfma(__builtin_bit_cast(typename X::frag, x[xp][m][i]), f, part[m]);
            }
          const float s = sc[w][n][q];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[w][n][m][e] = __builtin_fmaf(s, part[m][e], acc[w][n][m][e]);
        }
    }
  }
  // the waves' shares of K, added in the waves' order
  constexpr int kOut = W * NT * MT;
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[((wave * kOut + (w * NT + n) * MT + m) * 4 + e) * 64 + lane] = acc[w][n][m][e];
  __syncthreads();
  // thread t: value t % 64 of (tile, element) t / 64; its lane's column and row
  for (int o = wave; o < NT * MT * 4; o += kW4Waves) {
    float v[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      v[w] = 0.0f;
#pragma unroll
      for (int z = 0; z < kW4Waves; ++z) v[w] += red[(z * kOut * 4 + w * NT * MT * 4 + o) * 64 + lane];
    }
    const int e = o & 3, m = (o >> 2) % MT, n = (o >> 2) / MT;
    const int64_t row = m0 + 16 * m + 4 * g + e;
    const int col = (nt0 + n) * kW4Rows + i16;
    if (row >= p.M || col >= p.N) continue;
    if constexpr (PAIR) {
      const float sg = 1.0f / (1.0f + expf(-v[0]));
      split2(v[0] * sg * v[1], p.y[row * p.ldy + col], p.y2[row * p.ldy + col]);
    } else {
      p.y[row * p.ldy + col] = S::r(v[0]);
    }
  }
}

template <class X, class S, int MT, int NT, int XP, bool PAIR>
hipError_t w4_launch(const W4Params &p, hipStream_t s) {
  const int tiles_n = (p.N + kW4Rows - 1) / kW4Rows;
  const dim3 g((tiles_n + NT - 1) / NT, (uint32_t)((p.M + 16 * MT - 1) / (16 * MT))), b(64 * kW4Waves);
  const size_t lds = (size_t)kW4Waves * (PAIR ? 2 : 1) * NT * MT * 4 * 64 * 4;
  dgf_launch((k_w4<X, S, MT, NT, XP, PAIR>), g, b, lds, s, p);
  return hipGetLastError();
}

template <class X, class S, int XP, bool PAIR>
hipError_t w4_m(const W4Params &p, hipStream_t s) {
  if (p.M <= 16) return w4_launch<X, S, 1, 1, XP, PAIR>(p, s);
  return w4_launch<X, S, 2, PAIR ? 1 : 2, XP, PAIR>(p, s);
}

}  // namespace

hipError_t launch_pack4(const uint16_t *w, int64_t ldw, uint8_t *q, uint16_t *s, int N, int K, int group, int fmt, hipStream_t st) {
  const int64_t tiles = (int64_t)((N + kW4Rows - 1) / kW4Rows) * w4_tiles_k(K);
  const dim3 g((uint32_t)((tiles + 3) / 4)), b(256);
  if (fmt == FMT_F16) dgf_launch(k_pack4<F16>, g, b, 0, st, w, ldw, q, s, N, K, group);
  else dgf_launch(k_pack4<Bf16>, g, b, 0, st, w, ldw, q, s, N, K, group);
  return hipGetLastError();
}

hipError_t launch_unpack4(W4Mat m, uint16_t *w, int64_t ldw, int N, int K, int group, int fmt, hipStream_t st) {
  const int64_t tiles = (int64_t)((N + kW4Rows - 1) / kW4Rows) * w4_tiles_k(K);
  const dim3 g((uint32_t)((tiles + 3) / 4)), b(256);
  if (fmt == FMT_F16) dgf_launch(k_unpack4<F16>, g, b, 0, st, m, w, ldw, N, K, group);
  else dgf_launch(k_unpack4<Bf16>, g, b, 0, st, m, w, ldw, N, K, group);
  return hipGetLastError();
}

hipError_t launch_w4(const W4Params &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? w4_m<F16, F16, 1, false>(p, s) : w4_m<Bf16, Bf16, 1, false>(p, s);
}
hipError_t launch_w4_gate_up(const W4Params &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? w4_m<F16, F16, 1, true>(p, s) : w4_m<Bf16, Bf16, 1, true>(p, s);
}
hipError_t launch_w4_down(const W4Params &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? w4_m<Bf16, F16, 2, false>(p, s) : w4_m<Bf16, Bf16, 2, false>(p, s);
}

}  // namespace dgf
