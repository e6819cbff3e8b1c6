// Products with 4-bit weights and group scales for a few tokens (gfx950).
//
//   y[m][n] = sum over groups G of s[n][G] sum over k in G of x[m][k] c[n][k],  |c| <= 7
//
// A weight is read once for every 32 tokens, so the codes' bytes are the bound: 4.25 bits a
// weight with groups of 64.  They are laid out so that a wave reads a tile of 16 rows x 128
// columns as 1 KB in one piece and has each lane's dwords as it feeds them to the matrix core:
// c itself as an FP16 operand, c / 16 as a BF16 one, both exact, so that a code of 0 adds
// nothing however large its activation is, and an infinite activation stays what it is in the
// formula.  The group's sum, the scaled sums and those over the waves that share K are FP32.
// The activations pass from gate/up to down in three BF16 parts, which add up to the FP32 value:
// 30 of 131072 outputs then round otherwise than the exact sum does, against 180 of a product
// in FP32 and 330 with two parts, 17 bits (12288 activations, 32 tokens).
// Measured at 4096 x 12288, groups of 64, BF16, medians: gate/up 13.0 us for one token (53 MB,
// 4.1 TB/s), 18.8 for 32; down 12.8 and 26.4.  What is left over the copy rate (10 and 5 us) is one
// start-up of loads and one reduction a workgroup, and past 16 tokens the activations: each of the
// down product's 256 workgroups reads all 2.4 MB of them from L2, 600 MB (two parts: 20.8 us; two
// row tiles a workgroup, on half the CUs: 31).
#include "dgf_experts.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

constexpr int kW4Rows = 16, kW4K = 128;  // weights of a tile: 1 KB of codes, 16 bytes a lane
constexpr int kW4Waves = 8;               // that share K

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

// Eight codes as an MFMA operand, each c / code_unit, exact.
//  FP16: the code's four bits under the leading one of 16.0 are 24 + c, less 24: three
//  operations for two codes.
//  BF16, which has no packed sum: with its highest bit turned, the code is c in four bits of
//  two's complement, which v_cvt_off_f32_i4 takes from the lowest bits of a byte to c / 16;
//  the upper halves of two of them are the operands: 14 operations for eight codes.
template <class T>
__device__ __forceinline__ typename T::frag code_frag(uint32_t w) {
  uint4 v;
  if constexpr (T::code == 0) {
    const uint32_t even = w ^ 0x88888888u;
    uint32_t odd = even >> 4;
    asm("" : "+v"(odd));  // (else each of its bytes gets a shift of its own; bytes are free to pick)
    auto pair = [](uint32_t u, int lo, int hi) {  // the codes at bits lo and hi
      return __builtin_amdgcn_perm(__float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)(u >> hi & 0xff))),
                                   __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)(u >> lo & 0xff))), 0x07060302u);
    };
    v = make_uint4(pair(even, 0, 16), pair(odd, 0, 16), pair(even, 8, 24), pair(odd, 8, 24));
  } else {
    const f16x2 bias = {(_Float16)24.0f, (_Float16)24.0f};
    auto pair = [&](uint32_t u) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (u & 0x03c003c0u) | 0x4c004c00u) - bias); };
    v = make_uint4(pair(w << 6), pair(w << 2), pair(w >> 2), pair(w >> 6));
  }
  return __builtin_bit_cast(typename T::frag, v);
}
template <class T>
constexpr float code_unit = T::code == 0 ? 16.0f : 1.0f;

// An activation passes between the FFN's two kernels as kParts BF16 values whose sum it is.
constexpr int kParts = 3;

// Place of part xp of the activation (token m, column c): in the order of the down product's
// fragments, so that each load takes its tokens' lines whole (row by row, rows of 24 KB all start
// on one L2 channel: the down product took 46 us against 18 at 32 tokens).  Pieces of 8 tokens x
// 32 columns, the tokens' fastest: a few tokens take half of what a fragment holds.
__host__ __device__ inline int64_t act_octets(int64_t M) { return (M + 7) / 8; }
__host__ __device__ inline int64_t act_place(int64_t m, int c, int xp, int64_t octets) {
  const int64_t piece = ((int64_t)(c / kW4K * kParts + xp) * 4 + c % kW4K / 32) * octets + m / 8;
  return piece * 256 + ((m & 7) + 8 * (c % 32 / 8)) * 8 + c % 8;
}

// The activation a of a gate/up pair in parts: its upper 8 bits, the next 8 and the last 8, cut
// off, so that each remainder is exact and so is the sum (but for what lies below BF16's
// smallest subnormal).  An infinity or NaN is its first part.
__device__ __forceinline__ void split(float a, uint16_t (&part)[kParts]) {
  const bool finite = a - a == 0.0f;
  float rest = finite ? a : 0.0f;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    part[i] = (uint16_t)(__float_as_uint(rest) >> 16);
    rest -= bf2f(part[i]);
  }
  if (!finite) part[0] = f2bf(a);
}

__device__ const uint4 kZeros[1] = {};

// The GS scales of a tile's row, as one load.
template <class S, int GS>
struct Scales;
template <class S>
struct Scales<S, 1> {
  uint16_t v;
  __device__ __forceinline__ float get(int) const { return S::f(v); }
};
template <class S>
struct Scales<S, 2> {
  uint32_t v;
  __device__ __forceinline__ float get(int q) const { return q ? S::hi(v) : S::lo(v); }
};
template <class S>
struct Scales<S, 4> {
  uint2 v;
  __device__ __forceinline__ float get(int q) const { return q & 1 ? S::hi(q & 2 ? v.y : v.x) : S::lo(q & 2 ? v.y : v.x); }
};

// X: the activations' MFMA type.  S: the scales' (and the output's) type.  MT tiles of 16
// tokens, NT row tiles of the weights a workgroup (PAIR: NT of gate and NT of up), XP parts
// the activations come in (kParts: as act_place puts them), GS groups a tile, TAIL: K is no
// multiple of 8, kW4Waves share K: wave z takes the tiles [z n / kW4Waves, (z + 1) n / kW4Waves) of
// each row, from one that goes by the row tiles: workgroups in step do not all read the same
// columns of x, which lie on one L2 channel.
template <class X, class S, int MT, int NT, int XP, bool PAIR, int GS, bool TAIL>
__global__ __launch_bounds__(64 * kW4Waves) void k_w4(W4Params p) {
  constexpr int W = PAIR ? 2 : 1;
  // Tiles in a ring of registers: each is loaded anew as soon as it has been used, so that all
  // but one are on their way.  At 4096 x 12288 (codes then took two operations a pair) against
  // activations one tile ahead and codes two or four: gate/up 12.4 us against 14.4 for one token
  // and 16.4 against 23.1 for 32.  (Gate/up, one token, 4: 15.5 us, fewer waves fit.  TAIL's loads
  // take more registers, and activations in parts too: the whole FFN takes 24.3 us with two
  // tiles of down in flight, 25.3 with four, and at 32 tokens 42.3 with one, 42.2 with two.)
  constexpr int R = XP > 1 ? (MT > 1 ? 1 : 2) : MT > 1 ? (TAIL ? 1 : 2) : PAIR || TAIL ? 2 : 4;
  extern __shared__ __attribute__((aligned(16))) float red[];  // [waves][W NT MT][4][64]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int tiles_k = w4_tiles_k(p.K), tiles_n = (p.N + kW4Rows - 1) / kW4Rows;
  const int nt0 = blockIdx.x * NT;
  const int64_t m0 = (int64_t)blockIdx.y * 16 * MT;
  const int kt0 = (int)((int64_t)tiles_k * wave / kW4Waves), kt1 = (int)((int64_t)tiles_k * (wave + 1) / kW4Waves);

  f32x4 acc[W][NT][MT];
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[w][n][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Codes {
    uint4 q[W][NT];
    Scales<S, GS> s[W][NT];
  };
  struct Acts {  // of half a tile
    uint4 v[XP][MT][2];
  };
  const int share = kt1 - kt0, turn = share > 0 ? nt0 / 6 % share : 0;
  auto tile = [&](int j) {  // past the wave's last tile: that one again (loaded, not multiplied)
    j = (j < share ? j : share - 1) + turn;
    return kt0 + (j < share ? j : j - share);
  };
  auto codes = [&](int j, Codes &c) {
    const int kt = tile(j);
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t t = (int64_t)(nt0 + n < tiles_n ? nt0 + n : tiles_n - 1) * tiles_k + kt;
        c.q[w][n] = *reinterpret_cast<const uint4 *>(p.w[w].q + (t * 64 + lane) * 16);
        c.s[w][n] = *reinterpret_cast<const Scales<S, GS> *>(p.w[w].s + (t * 16 + i16) * GS);
      }
  };
  auto acts = [&](int j, int h, Acts &x) {
    const int kt = tile(j);
#pragma unroll
    for (int xp = 0; xp < XP; ++xp)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t row = m0 + 16 * m + i16;
          const int k = kt * kW4K + 64 * h + 32 * i + 8 * g;
          if constexpr (XP > 1) {  // (tokens past the last piece: that one again)
            const int64_t octets = act_octets(p.M), o = row / 8 < octets ? row / 8 : octets - 1;
            x.v[xp][m][i] = *reinterpret_cast<const uint4 *>(p.x + ((((int64_t)kt * kParts + xp) * 4 + 2 * h + i) * octets + o) * 256 + ((i16 & 7) + 8 * g) * 8);
          } else if constexpr (TAIL) {
            x.v[xp][m][i] = row < p.M && k < p.K ? row_ld(p.x + row * p.ldx, k, p.K) : make_uint4(0, 0, 0, 0);
          } else {
            x.v[xp][m][i] = *(row < p.M && k < p.K ? reinterpret_cast<const uint4 *>(p.x + row * p.ldx + k) : kZeros);
          }
        }
  };
  // Half h of a tile.  (A group of 128 columns is scaled in two halves.)
  auto multiply = [&](const Codes &c, const Acts &x, int h) {
    constexpr int kPer = GS == 4 ? 1 : 2;  // 32-column parts with one scale
#pragma unroll
    for (int q = 0; q < 2; q += kPer) {
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f32x4 part[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = q; i < q + kPer; ++i) {
            const uint4 &v = c.q[w][n];
            const typename X::frag f = code_frag<X>(h ? (i ? v.w : v.z) : i ? v.y : v.x);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int xp = 0; xp < XP; ++xp) part[m] = X::mfma(__builtin_bit_cast(typename X::frag, x.v[xp][m][i]), f, part[m]);
          }
          const float s = c.s[w][n].get((2 * h + q) * GS / 4);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[w][n][m][e] = __builtin_fmaf(s, part[m][e], acc[w][n][m][e]);
        }
    }
  };

  if (share > 0) {
    Codes c[R];
    Acts x[R][2];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      codes(u, c[u]);
      acts(u, 0, x[u][0]);
      acts(u, 1, x[u][1]);
    }
    int j = 0;
    for (; j + R < share; j += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        // (the barriers keep every load where it is: moved up, they cost spilled registers)
        multiply(c[u], x[u][0], 0);
        __builtin_amdgcn_sched_barrier(0);
        acts(j + R + u, 0, x[u][0]);
        __builtin_amdgcn_sched_barrier(0);
        multiply(c[u], x[u][1], 1);
        __builtin_amdgcn_sched_barrier(0);
        acts(j + R + u, 1, x[u][1]);
        __builtin_amdgcn_sched_barrier(0);
        codes(j + R + u, c[u]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int u = 0; u < R; ++u)
      if (j + u < share) {
        multiply(c[u], x[u][0], 0);
        multiply(c[u], x[u][1], 1);
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
  // (tile, element) o of every lane
  for (int o = wave; o < NT * MT * 4; o += kW4Waves) {
    float v[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      v[w] = 0.0f;
#pragma unroll
      for (int z = 0; z < kW4Waves; ++z) v[w] += red[(z * kOut * 4 + w * NT * MT * 4 + o) * 64 + lane];
      v[w] *= code_unit<X>;
    }
    const int e = o & 3, m = (o >> 2) % MT, n = (o >> 2) / MT;
    const int64_t row = m0 + 16 * m + 4 * g + e;
    const int col = (nt0 + n) * kW4Rows + i16;
    if (row >= p.M || (!PAIR && col >= p.N)) continue;
    if constexpr (PAIR) {
      const int64_t octets = act_octets(p.M);
      if (nt0 + n < tiles_n) {
        const float sg = 1.0f / (1.0f + expf(-v[0]));
        uint16_t part[kParts];
        split(col < p.N ? v[0] * sg * v[1] : 0.0f, part);
#pragma unroll
        for (int xp = 0; xp < kParts; ++xp) p.y[act_place(row, col, xp, octets)] = part[xp];
      }
      // the columns that fill up the last tile of the down product are zeros
      if (nt0 + n == tiles_n - 1)
        for (int c = col + kW4Rows; c < (tiles_n * kW4Rows + kW4K - 1) / kW4K * kW4K; c += kW4Rows)
#pragma unroll
          for (int xp = 0; xp < kParts; ++xp) p.y[act_place(row, c, xp, octets)] = 0;
    } else {
      p.y[row * p.ldy + col] = S::r(v[0]);
    }
  }
}

// Row tiles a workgroup may take.  (Three pairs with ragged rows and groups of 32 need more
// registers than there are: with 100 of them spilled the FFN took 92 us at 32 tokens, 4099 x
// 12288, against 76 with two, but 28 against 31 at 1003 x 8200.)
constexpr int w4_most(int MT, bool PAIR, int GS, bool tail) { return MT == 1 ? 1 : PAIR && GS == 4 && tail ? 2 : 3; }

template <class X, class S, int MT, int NT, int XP, bool PAIR, int GS>
hipError_t w4_launch(const W4Params &p, hipStream_t s) {
  const int tiles_n = (p.N + kW4Rows - 1) / kW4Rows;
  const dim3 g((tiles_n + NT - 1) / NT, (uint32_t)((p.M + 16 * MT - 1) / (16 * MT))), b(64 * kW4Waves);
  const size_t lds = (size_t)kW4Waves * (PAIR ? 2 : 1) * NT * MT * 4 * 64 * 4;
  if constexpr (XP == 1 && NT <= w4_most(MT, PAIR, GS, true)) {
    if (p.K % 8) {
      dgf_launch((k_w4<X, S, MT, NT, XP, PAIR, GS, true>), g, b, lds, s, p);
      return hipGetLastError();
    }
  }
  dgf_launch((k_w4<X, S, MT, NT, XP, PAIR, GS, false>), g, b, lds, s, p);
  return hipGetLastError();
}

template <class X, class S, int MT, bool DOWN, bool PAIR, int GS>
hipError_t w4_n(const W4Params &p, hipStream_t s) {
  constexpr int XP = DOWN ? kParts : 1;
  // Up to 16 tokens one row tile a workgroup (gate/up 12288 x 4096, one token, with less in
  // flight than now: 14.3 us, two tiles 18.1, three 15.6).  Past that as many as make the least
  // of what its waves read of the weights and, from L2, of the activations, over the rounds of
  // workgroups, those of every token tile counted (gate/up, 32 tokens, likewise: 31.5 us, 26.7,
  // 23.2; the FFN of 4096 x 12288 at 64 tokens with one row tile of down 83.6 us, with two 69.9).
  const int64_t tiles = (p.N + kW4Rows - 1) / kW4Rows, token_tiles = (p.M + 16 * MT - 1) / (16 * MT);
  int64_t best = 1, cost = 0;
  for (int n = 1; n <= w4_most(MT, PAIR, GS, !DOWN && p.K % 8); ++n) {
    const int64_t c = ((tiles + n - 1) / n * token_tiles + 255) / 256 * ((PAIR ? 2 : 1) * n + XP * MT);
    if (n == 1 || c < cost) best = n, cost = c;
  }
  if constexpr (MT > 1) {
    if (best == 3) return w4_launch<X, S, MT, 3, XP, PAIR, GS>(p, s);
    if (best == 2) return w4_launch<X, S, MT, 2, XP, PAIR, GS>(p, s);
  }
  return w4_launch<X, S, MT, 1, XP, PAIR, GS>(p, s);
}
// DOWN: the FFN's second product, whose activations are in parts.
template <class X, class S, bool DOWN, bool PAIR, int GS>
hipError_t w4_m(const W4Params &p, hipStream_t s) {
  return p.M <= 16 ? w4_n<X, S, 1, DOWN, PAIR, GS>(p, s) : w4_n<X, S, 2, DOWN, PAIR, GS>(p, s);
}
template <class X, class S, bool DOWN, bool PAIR>
hipError_t w4_g(const W4Params &p, hipStream_t s) {
  switch (p.group) {
    case 32: return w4_m<X, S, DOWN, PAIR, 4>(p, s);
    case 64: return w4_m<X, S, DOWN, PAIR, 2>(p, s);
    default: return w4_m<X, S, DOWN, PAIR, 1>(p, s);
  }
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

// (in whole pages of 4 KB)
size_t w4_act_bytes(int64_t M, int I) { return ((size_t)w4_tiles_k(I) * kParts * 4 * act_octets(M) * 512 + 4095) / 4096 * 4096; }

hipError_t launch_w4(const W4Params &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? w4_g<F16, F16, false, false>(p, s) : w4_g<Bf16, Bf16, false, false>(p, s);
}
hipError_t launch_w4_gate_up(const W4Params &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? w4_g<F16, F16, false, true>(p, s) : w4_g<Bf16, Bf16, false, true>(p, s);
}
hipError_t launch_w4_down(const W4Params &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? w4_g<Bf16, F16, true, false>(p, s) : w4_g<Bf16, Bf16, true, false>(p, s);
}

}  // namespace dgf
