// A mixture-of-experts layer for a few tokens (gfx950), every expert the gated FFN:
//
//   l = x W_r^T;  the k largest l of a token choose its experts (ties: lowest index)
//   p = softmax of l over all E experts, or over the k chosen (renorm)
//   a_j = silu(W_gate[e_j] x) (W_up[e_j] x);  y = sum_j p_j W_down[e_j] a_j
//
// Each chosen expert takes 3 H I 16-bit weights for 6 H I operations a token, so
// the layer is bound by the weights' way from HBM up to about 4 tokens an expert;
// with more, by the tokens' own lines and by reading weights again: one pass over
// an expert's weights takes 8, 16 or 32 tokens (by the mean number that an expert
// gets, token_tiles), and an expert that more tokens chose is passed over again.
// With 8 of 128 experts of 768 x 2048 that costs 115 + 61 us in the products at 32
// tokens and 181 + 105 at 128; all of 128 tokens on one expert 80 + 45 in 16
// passes, 8 of them on it 7.6 + 7.3.
// Launches: the router's products; the choice and the experts' token lists (one
// workgroup; for one token part of the next launch, past 32 tokens two); the
// gate/up products with the activation; the down products with the weighted sum
// over a token's experts (a launch of its own where workgroups share a row).
// Measured, BF16: 32 tokens over 8 of 128 experts of 768 x 2048 take 4.6 + 8.8 +
// 116 + 62 + 4.6 us, the products 5.9 and 5.7 TB/s of weights; one token of them
// 3.0 + 13.2 + 10.8 us, three launches long enough to start and drain.
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
#include <math.h>

#include "dgf_block.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

constexpr int kWaves = 8;  // of the gate/up and down workgroups

}  // namespace

bool moe_one(const MoeParams &p) { return p.M == 1 && p.E <= 256 && p.H >= 8; }

namespace {

// Router products, on the vector unit in FP32 (the matrix core truncates, and
// a logit's last bits decide ties): a workgroup per expert and kLogitTokens
// tokens, a lane 8 of every 2048 K.
constexpr int kLogitTokens = 4;

template <class T>
__global__ __launch_bounds__(256) void k_moe_logits(MoeParams p) {
  __shared__ float red[4][kLogitTokens];
  const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m0 = blockIdx.y * kLogitTokens;
  const uint16_t *w = p.w_router + e * p.ld_wr;
  const uint16_t *x[kLogitTokens];
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t) x[t] = p.x + (m0 + t < p.M ? m0 + t : m0) * p.ldx;
  float acc[kLogitTokens] = {};
#pragma unroll 2
  for (int c = threadIdx.x * 8; c < p.H; c += 2048) {
    const u16x8 wv = __builtin_bit_cast(u16x8, load_frag_tail<T>(w, c, p.H));
    u16x8 xv[kLogitTokens];
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t) xv[t] = __builtin_bit_cast(u16x8, load_frag_tail<T>(x[t], c, p.H));
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fmaf(T::f(wv[i]), T::f(xv[t][i]), acc[t]);
  }
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t) {
    const float l = wave_sum_last(acc[t]);
    if (lane == 63) red[wave][t] = l;
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < kLogitTokens && m0 + t < p.M)
    p.logits[(int64_t)(m0 + t) * p.E + e] = ((red[0][t] + red[1][t]) + red[2][t]) + red[3][t];
}

// Order of logits as integers: larger float, larger integer, equal floats (-0
// and +0 too) equal; NaN lowest; never 0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = l == 0.0f ? 0u : __float_as_uint(l);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 1u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The largest 32-bit value of the wave, uniform: shifts within rows of 16
// lanes, then row ends broadcast (data-parallel moves, no trip through LDS).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  uint32_t b;
#define DGF_MAX_STEP(ctrl, rows)                                                       \
  b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false);        \
  v = b > v ? b : v;
  DGF_MAX_STEP(0x111, 0xf)  // row_shr:1
  DGF_MAX_STEP(0x112, 0xf)  // row_shr:2
  DGF_MAX_STEP(0x114, 0xf)  // row_shr:4
  DGF_MAX_STEP(0x118, 0xf)  // row_shr:8
  DGF_MAX_STEP(0x142, 0xa)  // row_bcast:15
  DGF_MAX_STEP(0x143, 0xc)  // row_bcast:31
#undef DGF_MAX_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// A wave chooses the experts of one token from its logits v (NL a lane, E <= 64
// NL): lane j < k gets choice j and its routing weight.
template <int NL>
__device__ __forceinline__ void choose_token(const MoeParams &p, const float (&v)[NL], int lane, int &chosen,
                                             float &weight) {
  uint32_t key[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) key[i] = lane + 64 * i < p.E ? logit_key(v[i]) : 0u;
  float mine = -INFINITY, top = 0.0f;  // top: the first chosen, the largest
  chosen = 0;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) best = key[i] > best ? key[i] : best;
    best = wave_max(best);
    // the lowest index that has it, and its logit
    int e = -1;
    float le = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint64_t at = __ballot(key[i] == best);
      if (e < 0 && at) {
        const int src = __ffsll((unsigned long long)at) - 1;
        e = 64 * i + src;
        le = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v[i]), src));
        if (lane == src) key[i] = 0u;
      }
    }
    if (j == 0) top = le;
    if (lane == j) {
      chosen = e;
      mine = le;
    }
  }
  float part = 0.0f;
  if (p.renorm) {
    part = lane < p.k ? expf(mine - top) : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (lane + 64 * i < p.E) part += expf(v[i] - top);
  }
  const float sum = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_last(part)), 63));
  weight = expf(mine - top) / sum;
}

template <int NL>
__device__ __forceinline__ void fetch_logits(const MoeParams &p, int m, int lane, float (&v)[NL]) {
#pragma unroll
  for (int i = 0; i < NL; ++i) v[i] = m < p.M && lane + 64 * i < p.E ? p.logits[m * p.E + lane + 64 * i] : -INFINITY;
}

// Choice `lane` of token m, where the later kernels and the caller look for it.
__device__ __forceinline__ void store_choice(const MoeParams &p, int m, int lane, int chosen, float weight) {
  const int at = m * p.k + lane;
  p.ids[at] = chosen;
  p.p[at] = weight;
  if (p.ids_out) p.ids_out[at] = chosen;
  if (p.p_out) p.p_out[at] = weight;
}

// A wave chooses for tokens first, first + step, ...; ids: a copy in LDS, or null.
template <int NL>
__device__ __forceinline__ void choose(const MoeParams &p, int first, int step, int lane, int *ids) {
  float next[NL];
  fetch_logits(p, first, lane, next);
  for (int m = first; m < p.M; m += step) {
    float v[NL], weight;
    int chosen;
#pragma unroll
    for (int i = 0; i < NL; ++i) v[i] = next[i];
    fetch_logits(p, m + step, lane, next);  // the next token's logits arrive during this one's choice
    choose_token<NL>(p, v, lane, chosen, weight);
    if (lane < p.k) {
      if (ids) ids[m * p.k + lane] = chosen;
      store_choice(p, m, lane, chosen, weight);
    }
  }
}

// One workgroup orders all pairs by expert from ids in LDS: a thread per pair,
// one per expert.
constexpr int kRouteThreads = 1024;
static_assert(kRouteThreads >= kMoeMaxE && kMoeMaxE == 1 << 10, "a thread per expert, 10 bits of index");

__device__ __forceinline__ void order(const MoeParams &p, const int *ids, int *cnt, int *sums) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = p.M * p.k;
  constexpr int waves = kRouteThreads / 64;
  cnt[threadIdx.x] = 0;
  __syncthreads();
  // thread i: how many pairs before pair i (and i + 1024) have its expert.
  // Within a wave by matching the index bit by bit, then the waves in turn
  // (ascending pairs) through each expert's running count.
  constexpr int PER = kMoeMaxM * kMoeMaxK / kRouteThreads;
  int mine[PER], rank[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = threadIdx.x + u * kRouteThreads;
    mine[u] = i < n ? ids[i] - p.e0 : -1;
    if (mine[u] >= p.El) mine[u] = -1;
    uint64_t same = __ballot(mine[u] >= 0);
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const uint64_t set = __ballot(mine[u] >> b & 1);
      same &= mine[u] >> b & 1 ? set : ~set;
    }
    const int lead = mine[u] >= 0 ? __ffsll((unsigned long long)same) - 1 : lane;
    for (int w = 0; w < waves && u * kRouteThreads + w * 64 < n; ++w) {
      if (wave == w) {
        int base = 0;
        if (mine[u] >= 0 && lane == lead) {
          base = cnt[mine[u]];
          cnt[mine[u]] = base + __popcll(same);
        }
        rank[u] = __shfl(base, lead) + __popcll(same & ((1ull << lane) - 1));
      }
      __syncthreads();
    }
  }
  // thread e: local expert e's slot and first pair, (slots << 16 | pairs) before it by a scan
  const int have = (int)threadIdx.x < p.El ? cnt[threadIdx.x] : 0;
  const int own = have | (have > 0) << 16;
  int scan = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int b = __shfl_up(scan, o);
    if (lane >= o) scan += b;
  }
  if (lane == 63) sums[wave] = scan;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < waves; ++w) {
    before += w < wave ? sums[w] : 0;
    total += sums[w];
  }
  before += scan - own;
  if (threadIdx.x == 0) p.slots[0] = total >> 16;
  if (have > 0) {
    int *slot = p.slots + 1 + 3 * (before >> 16);
    slot[0] = threadIdx.x;
    slot[1] = before & 0xffff;
    slot[2] = have;
  }
  cnt[threadIdx.x] = before & 0xffff;  // each thread its own entry, read above
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u)
    if (mine[u] >= 0) p.pairs[cnt[mine[u]] + rank[u]] = threadIdx.x + u * kRouteThreads;
}

template <int NL>
__global__ __launch_bounds__(kRouteThreads) void k_moe_route(MoeParams p) {
  __shared__ __attribute__((aligned(16))) int ids[kMoeMaxM * kMoeMaxK];
  __shared__ int cnt[kMoeMaxE], sums[kRouteThreads / 64];
  choose<NL>(p, threadIdx.x >> 6, kRouteThreads / 64, threadIdx.x & 63, ids);
  order(p, ids, cnt, sums);
}

// The same in two launches for more tokens, whose choices keep one CU busy for
// longer than a launch takes.
template <int NL>
__global__ __launch_bounds__(256) void k_moe_choose(MoeParams p) {
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  choose<NL>(p, m, p.M, threadIdx.x & 63, nullptr);
}

__global__ __launch_bounds__(kRouteThreads) void k_moe_order(MoeParams p) {
  __shared__ __attribute__((aligned(16))) int ids[kMoeMaxM * kMoeMaxK];
  __shared__ int cnt[kMoeMaxE], sums[kRouteThreads / 64];
  for (int i = threadIdx.x; i < p.M * p.k; i += kRouteThreads) ids[i] = p.ids[i];
  order(p, ids, cnt, sums);
}

// The two diagonal 8 x 8 blocks of an accumulator added: rows 4 q + i (q < 2)
// and column lane & 7 in the lanes with bit 3 clear below lane 32.
__device__ __forceinline__ f32x4 diagonal(const f32x4 &acc) {
  f32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = acc[i] + __shfl(acc[i], (threadIdx.x + 40) & 63);
  return v;
}

typedef u16x8 u16x8_any __attribute__((aligned(2)));

// 8 weights, any alignment.  ONCE: their line is not asked for again, so they
// are loaded non-temporally.  That holds where rows start on 128-byte lines
// (the gate/up kernel at 8 of 8 experts of 12288 x 4096: 237 us against 271
// with plain loads); elsewhere the next step needs the line's other end (20
// experts of 1411 x 1003: 26 us against 23).
template <class T, bool ONCE>
__device__ __forceinline__ typename T::frag load_weights(const uint16_t *p) {
  const u16x8_any *q = reinterpret_cast<const u16x8_any *>(p);
  return __builtin_bit_cast(typename T::frag, ONCE ? (u16x8)__builtin_nontemporal_load(q) : (u16x8)*q);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 8 stored values with the first n zero (n <= 0: none, n >= 8: all).
template <class F>
__device__ __forceinline__ F drop_first(const F &v, int n) {
  u32x4 b = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] &= n <= 2 * j ? 0xffffffffu : n == 2 * j + 1 ? 0xffff0000u : 0u;
  return __builtin_bit_cast(F, b);
}

// Rows of the token operand through a buffer descriptor: a lane whose column
// has no token gives an offset past its range and costs no memory request.
// Leading dimensions are below 2^23, so 128 rows of x stay below 2^31 bytes.
constexpr uint32_t kNoColumn = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t column_rsrc(const uint16_t *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)p, (short)0, (int)bytes, 0x00020000);
}
template <class T>
__device__ __forceinline__ typename T::frag load_column(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(typename T::frag,
                            __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0)));
}

// A workgroup: tiles of 8 rows of an active expert's W_gate and W_up against
// its tokens, 8 NT at a time.  `share` waves split a tile's K (whole steps of
// 64, kChunk of them loaded together; the last of them also takes the ragged
// rest), so that a wave has about 4 steps or more; 8 / share tiles a workgroup.
//
// The activation a leaves in 32 bits, two lines for every 64 columns of a pair,
// so that a step of the down kernel takes both whole.  BF16: two stored parts
// whose sum is a to 2^-16 of it, so that rounding it adds nothing to the
// output's own rounding ([64 of the first, 64 of the second]).  FP16: the FP32
// value itself ([4 of every 8, the other 4]), since parts in FP16 would lose a
// past 2 x 65504 and, their second part a subnormal, below about 2^-3.  K of
// the down products is padded to lda with zeros, and a ragged last chunk of 8
// holds its values at the end, for weights read from I - 8 (see k_moe_down).
//
// Bound by HBM where weight rows start on 128-byte lines: 6.2 TB/s at 8 experts
// of 12288 x 4096 and 8 tokens, 5.9 at 128 of 768 x 2048 and 32.  Off the lines
// every line of a row is asked for twice (1.8 times the requests, 1.1 times the
// bytes from HBM) and it reaches 4.2 to 5.3; past about 4 tokens an expert the
// tokens' own lines take as many of a CU's misses as the weights' (4.2 at 8,
// 3.5 at 16 tokens an expert).
constexpr int kChunk = 2;

// Whether a passes between the kernels as FP32 values instead of two stored parts.
template <class T>
constexpr bool kWholeA = T::code == F16::code;

// First row of the tile at i0: a ragged last tile takes the last 8 rows (the
// first of them a second time).
__device__ __forceinline__ int tile_row(int i0, int I) { return i0 + 8 <= I || I < 8 ? i0 : I - 8; }

// Column i of the chunk of 8 from column k, of a pair's row of a.
template <class T>
__device__ __forceinline__ void put_a(uint16_t *row, int k, int i, float a) {
  if constexpr (kWholeA<T>) {
    asm volatile("" : "+v"(i));  // computed here, not kept over the caller's loop
    reinterpret_cast<float *>(row)[k - (k & 63) / 2 + i + 7 * (i & 4)] = a;
  } else {
    uint16_t h = T::r(a);
    // past the stored type's range the first part stays at its largest value:
    // as an infinity it would cancel against the second's into a NaN
    if ((h & 0x7fffu) == 0x7f80u) h -= 1;
    uint16_t *out = row + (k >> 6) * 128 + (k & 63) + i;
    out[0] = h;
    out[64] = T::r(a - T::f(h));
  }
}

// Sums of products of 8 weights a lane and the 8 columns of a beside them (a0,
// a1: a chunk as its two lines hold it).  FP16 weights are exact in FP32, and so
// are their products with FP32 a, four K an instruction: a sixteenth of the rate
// of FP16 products, which costs the down kernel 70 us against 62 at 32 tokens
// over 8 of 128 experts of 768 x 2048, 54 against 43 at 64 over 8 of 16 of 1024 x
// 1024.  BF16: a sum for each part, so that where an infinite weight makes the
// first an infinity, its product with the second (0, or of the other sign) is
// left out.
template <class T>
struct SumA {
  f32x4 first, second;  // second: unused with FP32 a
  __device__ __forceinline__ void clear() { first = second = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void add(const typename T::frag &w, const typename T::frag &a0, const typename T::frag &a1) {
    if constexpr (kWholeA<T>) {
      const f32x4 lo = __builtin_bit_cast(f32x4, a0), hi = __builtin_bit_cast(f32x4, a1);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        first = __builtin_amdgcn_mfma_f32_16x16x4f32((float)w[i], i < 4 ? lo[i] : hi[i - 4], first, 0, 0, 0);
    } else {
      first = T::mfma(w, a0, first);
      second = T::mfma(w, a1, second);
    }
  }
  __device__ __forceinline__ f32x4 sum() const {
    f32x4 v = first;
    if constexpr (!kWholeA<T>)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fabsf(v[i]) == INFINITY ? v[i] : v[i] + second[i];
    return v;
  }
};

//
// ONE > 0: a single token, whose choice (E <= 64 ONE) every workgroup makes for
// itself from the logits instead of waiting for a launch of its own; slot j is
// then the token's j-th local choice, and the first workgroup leaves the lists
// for the down kernel (8 of 128 experts: 5.1 us of routing and 12.1 of products
// become 13.4 us).
template <class T, int NT, int share, bool ONCE, bool SMALL, int ONE>
__global__ __launch_bounds__(64 * kWaves, NT == 1 ? 6 : 4) void k_moe_gate_up(MoeParams p) {
  __shared__ __attribute__((aligned(16))) float red[kWaves][2][8 * NT][8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int e, start, cnt, pair = 0;  // pair: the only one, with ONE
  if constexpr (ONE > 0) {
    float v[ONE], weight;
    int chosen;
    fetch_logits(p, 0, lane, v);
    choose_token<ONE>(p, v, lane, chosen, weight);
    const int le = chosen - p.e0;
    const uint64_t local = __ballot(lane < p.k && le >= 0 && le < p.El);
    const int n = __popcll(local), slot = __popcll(local & ((1ull << lane) - 1));
    if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) {
      if (lane < p.k) store_choice(p, 0, lane, chosen, weight);
      if (lane == 0) p.slots[0] = n;
      if (local >> lane & 1) {
        int *s = p.slots + 1 + 3 * slot;
        s[0] = le;
        s[1] = slot;
        s[2] = 1;
        p.pairs[slot] = lane;
      }
    }
    if ((int)blockIdx.y >= n) return;
    pair = __ffsll((unsigned long long)__ballot((local >> lane & 1) && slot == (int)blockIdx.y)) - 1;
    e = __builtin_amdgcn_readlane(le, pair);
    start = 0;
    cnt = 1;
  } else {
    const int n = p.slots[0];
    e = p.slots[1 + 3 * blockIdx.y];
    start = p.slots[2 + 3 * blockIdx.y];
    cnt = p.slots[3 + 3 * blockIdx.y];
    if ((int)blockIdx.y >= n) return;
  }
  const int c = lane & 7, q = lane >> 4, at = ((lane >> 3) & 1) * 32 + q * 8;
  const int i0 = (blockIdx.x * kWaves + wave) / share * 8, sub = wave & (share - 1);
  const int row = tile_row(i0, p.I) + c < p.I ? tile_row(i0, p.I) + c : p.I - 1;
  const uint16_t *wg = p.w_gate + e * p.st_wg + row * p.ld_wg;
  const uint16_t *wu = p.w_up + e * p.st_wu + row * p.ld_wu;
  const int steps = p.H / 64, lo = steps * sub / share, hi = steps * (sub + 1) / share;
  const bool rest = sub == share - 1 && steps * 64 < p.H;
  const __amdgpu_buffer_rsrc_t xr = column_rsrc(p.x, ((int64_t)(p.M - 1) * p.ldx + p.H) * 2);
  for (int t0 = 0; t0 < cnt; t0 += 8 * NT) {
    uint32_t x[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = t0 + 8 * t + c;
      const int token = ONE > 0 ? 0 : i < cnt ? p.pairs[start + i] / p.k : 0;
      x[t] = i < cnt ? (uint32_t)(token * (int)p.ldx + at) * 2 : kNoColumn;
    }
    f32x4 ag[NT] = {}, au[NT] = {};
    int s = lo;
    for (; s + kChunk <= hi; s += kChunk) {
      typename T::frag fg[kChunk], fu[kChunk], fx[kChunk][NT];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        fg[i] = load_weights<T, ONCE>(wg + (s + i) * 64 + at);
        fu[i] = load_weights<T, ONCE>(wu + (s + i) * 64 + at);
#pragma unroll
        for (int t = 0; t < NT; ++t) fx[i][t] = load_column<T>(xr, x[t] + (s + i) * 128);
      }
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          ag[t] = T::mfma(fg[i], fx[i][t], ag[t]);
          au[t] = T::mfma(fu[i], fx[i][t], au[t]);
        }
    }
    for (; s < hi; ++s) {
      const typename T::frag fg = load_weights<T, ONCE>(wg + s * 64 + at), fu = load_weights<T, ONCE>(wu + s * 64 + at);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const typename T::frag fx = load_column<T>(xr, x[t] + s * 128);
        ag[t] = T::mfma(fg, fx, ag[t]);
        au[t] = T::mfma(fu, fx, au[t]);
      }
    }
    if (rest) {
      // a chunk of 8 that would pass H is read from H - 8, with zeros for what
      // belongs to an earlier chunk (in both operands: either may be infinite)
      const int k = steps * 64 + at, from = k < p.H - 8 ? k : p.H - 8;
      int drop = k - from;
      asm volatile("" : "+v"(drop));  // its masks stay here: kept over the loop they cost 4 registers
      typename T::frag fg, fu;
      if constexpr (SMALL) {
        fg = load_frag_tail<T>(wg, k, p.H), fu = load_frag_tail<T>(wu, k, p.H);
      } else {
        fg = drop_first(load_weights<T, ONCE>(wg + from), drop);
        fu = drop_first(load_weights<T, ONCE>(wu + from), drop);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint16_t *row = p.x + (x[t] < kNoColumn ? x[t] / 2 - at : 0);
        typename T::frag fx;
        if constexpr (SMALL) fx = load_frag_tail<T>(row, k, p.H);
        else fx = drop_first(load_weights<T, false>(row + from), drop);
        ag[t] = T::mfma(fg, fx, ag[t]);
        au[t] = T::mfma(fu, fx, au[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 g = diagonal(ag[t]), u = diagonal(au[t]);
      if (lane < 32 && (lane & 8) == 0) {
        *reinterpret_cast<f32x4 *>(&red[wave][0][8 * t + c][q * 4]) = g;
        *reinterpret_cast<f32x4 *>(&red[wave][1][8 * t + c][q * 4]) = u;
      }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < kWaves / share * 64 * NT; o += 64 * kWaves) {
      const int w0 = o / (64 * NT) * share, tok = o / 8 % (8 * NT), r = o & 7;
      const int ti = (blockIdx.x * kWaves + w0) / share * 8;
      if (t0 + tok >= cnt || ti >= p.I) continue;
      float gs = 0.0f, us = 0.0f;
      for (int w = w0; w < w0 + share; ++w) {
        gs += red[w][0][tok][r];
        us += red[w][1][tok][r];
      }
      const int i = tile_row(ti, p.I) + r;
      const float a = i >= ti && i < p.I ? gs * sigma_f(gs) * us : 0.0f;  // zero in a repeated row's place
      uint16_t *out = p.a + (ONE > 0 ? pair : p.pairs[start + t0 + tok]) * p.lda * 2;
      put_a<T>(out, ti, r, a);
      if (ti + 8 >= p.I)  // the last tile: zeros up to lda
        for (int k = ti + 8; k < p.lda; k += 8) put_a<T>(out, k, r, 0.0f);
    }
    __syncthreads();
  }
}

// A workgroup: 8 RT rows of y over all active experts.  Its waves work in groups
// of `wps`, a group on one expert at a time, each wave of it a share of K = I;
// wps is 8 / k (down to a power of two), so that the experts of a single token
// keep all waves busy.  A wave's steps (64 K of an expert's rows against 8 NT
// of its tokens) form one stream over all its experts, and the loads run R
// steps ahead of the products through it: 8 R RT KB of weights in flight per
// workgroup (R 6 to 18 measure the same: what bounds it are the lines a CU can
// wait for, a's among them; without a's loads 128 experts of 2048 x 768 took 52
// us, with them 72 at 8 rows a workgroup and 62 at 16).  Loads past the end of
// the stream read one fixed line.  5.75 TB/s at 8 experts of 4096 x 12288.
//
// The weights' last ragged chunk of 8 is read from I - 8, against a's last
// chunk with its values at the end and zeros before, and later chunks again
// from there against zeros: no load passes a row's end.  The weights that meet
// those zeros are made zeros too (an infinity would make a NaN).  (SMALL: I < 8,
// where there is no such 8; element by element.)
//
// Each (token, choice) pair's partial products stay in LDS and are added up in
// order at the end: the waves' shares, then the choices by p.  Where the rows
// of y alone make too few workgroups, grid.y workgroups share the experts of a
// row tile: the products of a pair then go to `prod` and k_moe_combine weighs
// and adds them, the same operations in the same order.
struct MoeSlot {
  int e, start, cnt;
};
constexpr float kNotHere = -1.0f;  // in place of a routing weight (never negative): another call has that expert

template <class T, int RT, int NT, int R, bool ONCE, bool SMALL>
__global__ __launch_bounds__(64 * kWaves) void k_moe_down(MoeParams p, int wps) {
  constexpr int ROWS = 8 * RT;
  extern __shared__ __attribute__((aligned(16))) float part[];  // [M k][wps][ROWS]
  const int np = p.M * p.k, ns = np < p.El ? np : p.El;
  int *pairs = reinterpret_cast<int *>(part + np * wps * ROWS);
  MoeSlot *slots = reinterpret_cast<MoeSlot *>(pairs + np);
  for (int i = threadIdx.x; i < np; i += 64 * kWaves) pairs[i] = p.pairs[i];
  float *weight = reinterpret_cast<float *>(slots + ns);  // p, or kNotHere
  for (int i = threadIdx.x; i < 3 * ns; i += 64 * kWaves) reinterpret_cast<int *>(slots)[i] = p.slots[1 + i];
  if (!p.prod)
    for (int i = threadIdx.x; i < np; i += 64 * kWaves) {
      const int e = p.ids[i] - p.e0;
      const float w = p.p[i];
      weight[i] = e >= 0 && e < p.El ? w : kNotHere;
    }
  const int n = p.slots[0];
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 7, q = lane >> 4, at = ((lane >> 3) & 1) * 32 + q * 8;
  const int h0 = blockIdx.x * ROWS;
  const int sub = wave & (wps - 1), groups = kWaves / wps * (int)gridDim.y;
  const int len = (int)(p.lda / (64 * wps)), k0 = sub * len * 64 + at;  // this wave's steps of an expert, its first column
  const uint16_t *wrow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) wrow[i] = p.w_down + (h0 + 8 * i + c < p.H ? h0 + 8 * i + c : p.H - 1) * p.ld_wd;

  struct Step {
    typename T::frag w[RT], a0[NT], a1[NT];
  };
  struct Cursor {
    int slot, t0, step, cnt, start, e;
  };
  auto open = [&](Cursor &u) {
    const MoeSlot v = slots[u.slot < n ? u.slot : 0];
    u.e = __builtin_amdgcn_readfirstlane(v.e);
    u.start = __builtin_amdgcn_readfirstlane(v.start);
    u.cnt = __builtin_amdgcn_readfirstlane(v.cnt);
  };
  Cursor ld = {wave / wps * (int)gridDim.y + (int)blockIdx.y, 0, 0, 0, 0, 0};
  const uint16_t *w[RT];
  uint32_t a[NT];
  int go = 1;  // steps that a load advances: 0 past the end of the stream
  const __amdgpu_buffer_rsrc_t ar = column_rsrc(p.a, np * p.lda * 4);
  auto point = [&] {  // the cursor's expert and tokens
#pragma unroll
    for (int i = 0; i < RT; ++i) w[i] = wrow[i] + ld.e * p.st_wd;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = ld.t0 + 8 * t + c;
      a[t] = i < ld.cnt ? (uint32_t)((pairs[ld.start + i] * (int)p.lda + k0 - at) * 2 + at) * 2 : kNoColumn;
    }
  };
  auto load = [&](Step &v) {  // no branch around the loads: the compiler then counts them exactly
    const int k = k0 + ld.step * 64;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if constexpr (SMALL) v.w[i] = load_frag_tail<T>(w[i], k, p.I);
      else v.w[i] = load_weights<T, ONCE>(w[i] + (k < p.I - 8 ? k : p.I - 8));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      v.a0[t] = load_column<T>(ar, a[t] + ld.step * 256);
      v.a1[t] = load_column<T>(ar, a[t] + ld.step * 256 + 128);
    }
    ld.step += go;
    if (ld.step < len) return;
    ld.step = 0;
    ld.t0 += 8 * NT;
    if (ld.t0 >= ld.cnt) {
      ld.t0 = 0;
      ld.slot += groups;
      open(ld);
    }
    if (ld.slot < n) {
      point();
    } else {
      go = 0;
#pragma unroll
      for (int i = 0; i < RT; ++i) w[i] = p.w_down;
#pragma unroll
      for (int t = 0; t < NT; ++t) a[t] = kNoColumn;
    }
  };

  if (ld.slot < n) {
    Cursor cu = ld;
    open(ld);
    open(cu);
    point();
    Step ring[R];
#pragma unroll
    for (int r = 0; r < R; ++r) load(ring[r]);
    SumA<T> acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[i][t].clear();
    while (cu.slot < n) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (cu.slot < n) {
          if (!SMALL && (sub * len + cu.step + 1) * 64 > p.I) {
            // columns past I, and those of the last chunk that were read twice: as 0 x 0
            const int past = k0 + cu.step * 64 - (p.I - 8);
#pragma unroll
            for (int i = 0; i < RT; ++i) ring[r].w[i] = drop_first(ring[r].w[i], past);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[i][t].add(ring[r].w[i], ring[r].a0[t], ring[r].a1[t]);
          if (++cu.step == len) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const int at_ = cu.t0 + 8 * t + c;
#pragma unroll
              for (int i = 0; i < RT; ++i) {
                const f32x4 v = diagonal(acc[i][t].sum());
                if (lane < 32 && (lane & 8) == 0 && at_ < cu.cnt)
                  *reinterpret_cast<f32x4 *>(&part[(pairs[cu.start + at_] * wps + sub) * ROWS + 8 * i + q * 4]) = v;
                acc[i][t].clear();
              }
            }
            cu.step = 0;
            cu.t0 += 8 * NT;
            if (cu.t0 >= cu.cnt) {
              cu.t0 = 0;
              cu.slot += groups;
              open(cu);
            }
          }
        }
        load(ring[r]);
      }
    }
  }
  __syncthreads();
  if (p.prod) {
    for (int s = wave * (int)gridDim.y + (int)blockIdx.y; s < n; s += kWaves * (int)gridDim.y)
      for (int o = lane; o < slots[s].cnt * ROWS; o += 64) {
        const int pair = pairs[slots[s].start + o / ROWS], r = o % ROWS;
        float t = 0.0f;
        for (int i = 0; i < wps; ++i) t += part[(pair * wps + i) * ROWS + r];
        if (h0 + r < p.H) p.prod[(int64_t)pair * p.H + h0 + r] = t;
      }
    return;
  }
  for (int o = threadIdx.x; o < p.M * ROWS; o += 64 * kWaves) {
    const int m = o / ROWS, r = o % ROWS;
    if (h0 + r >= p.H) continue;
    float y = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const float w = weight[m * p.k + j];
      if (w == kNotHere) continue;
      float t = 0.0f;
      for (int i = 0; i < wps; ++i) t += part[((m * p.k + j) * wps + i) * ROWS + r];
      y = fmaf(w, t, y);
    }
    p.y[m * p.ldy + h0 + r] = T::r(y);
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_moe_combine(MoeParams p) {
  const int h = blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
  if (h >= p.H) return;
  float y = 0.0f;
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    float t[8], w[8];
    bool here[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // all loads first; prod holds nothing for experts of other calls
      const int at = m * p.k + (j0 + j < p.k ? j0 + j : p.k - 1), e = p.ids[at] - p.e0;
      t[j] = p.prod[(int64_t)at * p.H + h];
      w[j] = p.p[at];
      here[j] = j0 + j < p.k && e >= 0 && e < p.El;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y = here[j] ? fmaf(w[j], t[j], y) : y;
  }
  p.y[m * p.ldy + h] = T::r(y);
}

// Waves that share an expert in the down kernel.
int waves_per_slot(int k) {
  int wps = 1;
  while (wps * 2 * k <= kWaves) wps *= 2;
  return wps;
}

// What a CU reads (about 27 GB/s of it) in the time that the combining launch
// takes, and in a workgroup's start and end.
constexpr double kCombineBytes = 100e3, kStartBytes = 60e3;

// Token tiles of 8 that one pass over an expert's weights takes, from the
// mean number of tokens an expert gets.  Both products with 1 / 2 / 4 tiles, us:
// 4 of 32 experts (1024 x 2048) at a mean of 4: 80 / 92 / 121, 8: 120 / 103 / 130,
// 12: 157 / 118 / 140, 16: 206 / 163 / 151; 2 of 8 (4096 x 4096) at 4: 135 / 156 /
// 212, 8: 189 / 177 / 230, 12: 295 / 231 / 248, 16: 381 / 278 / 265.
int token_tiles(const MoeParams &p) {
  const int64_t pairs = (int64_t)p.M * p.k;
  return pairs <= 4 * (int64_t)p.E ? 1 : pairs <= 12 * (int64_t)p.E ? 2 : 4;
}

// Whether every row of an expert matrix starts on a 128-byte line.
bool line_rows(const uint16_t *w, int64_t ld, int64_t stride) {
  return ((uintptr_t)w & 127) == 0 && ld % 64 == 0 && stride % 64 == 0;
}

template <class T, int SHARE>
hipError_t gate_up_s(const MoeParams &p, hipStream_t s) {
  constexpr int rows = 8 * (kWaves / SHARE);
  const int slots = p.M * p.k < p.El ? p.M * p.k : p.El;  // at most this many experts have tokens
  const dim3 g((p.I + rows - 1) / rows, slots), b(64 * kWaves);
  const bool once = line_rows(p.w_gate, p.ld_wg, p.st_wg) && line_rows(p.w_up, p.ld_wu, p.st_wu);
  if (moe_one(p)) {
    if (p.E <= 128 && once) dgf_launch((k_moe_gate_up<T, 1, SHARE, true, false, 2>), g, b, 0, s, p);
    else if (p.E <= 128) dgf_launch((k_moe_gate_up<T, 1, SHARE, false, false, 2>), g, b, 0, s, p);
    else if (once) dgf_launch((k_moe_gate_up<T, 1, SHARE, true, false, 4>), g, b, 0, s, p);
    else dgf_launch((k_moe_gate_up<T, 1, SHARE, false, false, 4>), g, b, 0, s, p);
    return hipGetLastError();
  }
  switch (token_tiles(p) * 2 + once) {
    case 2: dgf_launch((k_moe_gate_up<T, 1, SHARE, false, false, 0>), g, b, 0, s, p); break;
    case 3: dgf_launch((k_moe_gate_up<T, 1, SHARE, true, false, 0>), g, b, 0, s, p); break;
    case 4: dgf_launch((k_moe_gate_up<T, 2, SHARE, false, false, 0>), g, b, 0, s, p); break;
    case 5: dgf_launch((k_moe_gate_up<T, 2, SHARE, true, false, 0>), g, b, 0, s, p); break;
    case 8: dgf_launch((k_moe_gate_up<T, 4, SHARE, false, false, 0>), g, b, 0, s, p); break;
    default: dgf_launch((k_moe_gate_up<T, 4, SHARE, true, false, 0>), g, b, 0, s, p); break;
  }
  return hipGetLastError();
}

// Waves that split a tile's K: 4 steps of 64 or more each.
template <class T>
hipError_t gate_up_t(const MoeParams &p, hipStream_t s) {
  if (p.H < 8) {
    const dim3 g((p.I + 63) / 64, p.M * p.k < p.El ? p.M * p.k : p.El);
    dgf_launch((k_moe_gate_up<T, 1, 1, false, true, 0>), g, dim3(64 * kWaves), 0, s, p);
    return hipGetLastError();
  }
  const int steps = p.H / 64;
  return steps >= 32 ? gate_up_s<T, 8>(p, s) : steps >= 16 ? gate_up_s<T, 4>(p, s) : steps >= 8 ? gate_up_s<T, 2>(p, s) : gate_up_s<T, 1>(p, s);
}

template <class T, int RT>
hipError_t down_rt(const MoeParams &p, hipStream_t s) {
  const int wps = waves_per_slot(p.k), np = p.M * p.k, slots = np < p.El ? np : p.El;
  const dim3 g((p.H + 8 * RT - 1) / (8 * RT), p.split), b(64 * kWaves);
  // at most 64 RT KB of partial products (M k wps <= 2048), 16 of pairs and their weights, 12 of slots: 156 of 160
  const size_t lds = (size_t)np * wps * 8 * RT * 4 + (size_t)np * 8 + (size_t)slots * sizeof(MoeSlot);
  if (p.I < 8) dgf_launch((k_moe_down<T, RT, 1, 2, false, true>), g, b, lds, s, p, wps);
  else switch (token_tiles(p) * 2 + line_rows(p.w_down, p.ld_wd, p.st_wd)) {
    case 2: dgf_launch((k_moe_down<T, RT, 1, 8, false, false>), g, b, lds, s, p, wps); break;
    case 3: dgf_launch((k_moe_down<T, RT, 1, 8, true, false>), g, b, lds, s, p, wps); break;
    case 4: dgf_launch((k_moe_down<T, RT, 2, 6, false, false>), g, b, lds, s, p, wps); break;
    case 5: dgf_launch((k_moe_down<T, RT, 2, 6, true, false>), g, b, lds, s, p, wps); break;
    case 8: dgf_launch((k_moe_down<T, RT, 4, 4, false, false>), g, b, lds, s, p, wps); break;
    default: dgf_launch((k_moe_down<T, RT, 4, 4, true, false>), g, b, lds, s, p, wps); break;
  }
  return hipGetLastError();
}

template <class T>
hipError_t down_t(const MoeParams &p, hipStream_t s) {
  return p.row_tiles == 2 ? down_rt<T, 2>(p, s) : down_rt<T, 1>(p, s);
}

}  // namespace

// Row tiles a workgroup and workgroups a row tile, by the bytes that pass
// through the busiest CU: its waves' weights, in whole rounds of experts, and
// its pairs' activations (from L2, at three quarters of the cost), for every
// round of workgroups; sharing out the experts costs the combining launch.
void moe_plan(MoeParams &p) {
  const int wps = waves_per_slot(p.k), groups = kWaves / wps;
  const double pairs = (double)p.M * p.k * p.El / p.E;
  const double slots = p.El * (1.0 - pow(1.0 - (double)p.k / p.E, p.M));  // experts with tokens, on average
  double best = 0.0;
  for (int rt = 1; rt <= 2; ++rt) {
    const int tiles = (p.H + 8 * rt - 1) / (8 * rt);
    for (int z = 1; z <= 32 && (z == 1 || (z - 1) * groups < slots); ++z) {
      // a last round that only some waves have leaves the others' bandwidth to them: count it half
      const double exact = slots / (z * groups), rounds = 0.5 * (exact + ceil(exact));
      const double wg = rounds * kWaves * 8.0 * rt * 2.0 * p.I / wps + 0.75 * pairs / z * p.I * 4.0;
      const double cost = ceil(tiles * z / 256.0) * (wg + kStartBytes) + (z > 1 ? kCombineBytes : 0.0);
      if (best == 0.0 || cost < best) {
        best = cost;
        p.row_tiles = rt;
        p.split = z;
      }
    }
  }
}

// Tokens that one workgroup both chooses for and orders (8 of 128 experts: 8.3
// us at 32 tokens, as much as the two launches; 13.2 at 64 against 8.9).
constexpr int kRouteOnce = 32;

int64_t moe_down_ld(int I, int k) {
  const int step = 64 * waves_per_slot(k);
  return (int64_t)(I + step - 1) / step * step;
}

hipError_t launch_moe_logits(const MoeParams &p, hipStream_t s) {
  const dim3 g(p.E, (p.M + kLogitTokens - 1) / kLogitTokens);
  if (p.fmt == FMT_F16) dgf_launch(k_moe_logits<F16>, g, dim3(256), 0, s, p);
  else dgf_launch(k_moe_logits<Bf16>, g, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int NL>
static hipError_t route_nl(const MoeParams &p, hipStream_t s) {
  if (p.M <= kRouteOnce) {
    dgf_launch(k_moe_route<NL>, dim3(1), dim3(kRouteThreads), 0, s, p);
    return hipGetLastError();
  }
  dgf_launch(k_moe_choose<NL>, dim3((p.M + 3) / 4), dim3(256), 0, s, p);
  dgf_launch(k_moe_order, dim3(1), dim3(kRouteThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_moe_route(const MoeParams &p, hipStream_t s) {
  if (p.E <= 128) return route_nl<2>(p, s);
  if (p.E <= 256) return route_nl<4>(p, s);
  return route_nl<kMoeMaxE / 64>(p, s);
}

hipError_t launch_moe_gate_up(const MoeParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? gate_up_t<F16>(p, s) : gate_up_t<Bf16>(p, s);
}

hipError_t launch_moe_down(const MoeParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? down_t<F16>(p, s) : down_t<Bf16>(p, s);
}

hipError_t launch_moe_combine(const MoeParams &p, hipStream_t s) {
  const dim3 g((p.H + 255) / 256, p.M);
  if (p.fmt == FMT_F16) dgf_launch(k_moe_combine<F16>, g, dim3(256), 0, s, p);
  else dgf_launch(k_moe_combine<Bf16>, g, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace dgf
