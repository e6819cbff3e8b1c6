// Routing of tokens to experts, and the experts' outputs back to tokens (gfx950).
//
// Routing: a token's k largest logits, one wave a token.  A logit becomes an integer that
// keeps its order; k times the wave's largest is found by lane moves, its lowest index by a
// ballot, and it is struck out.  Each workgroup counts its choices by expert (integer adds in
// LDS: their order does not matter) and leaves the counts; a second launch, the same tokens
// to the same workgroups, adds up those of all of them, and every pair's row follows from its
// expert's first, the earlier workgroups', waves' and lanes' pairs: a stable sort without
// another pass over anything.  The bound is the two launches and the chain of k reductions,
// not the 2.6 MB it moves: 5.8 and 6.9 us for 4096 tokens, 8 of 128 experts.  Up to 64 tokens
// one workgroup does both.
// Combination: k rows of H gathered to one, 8 columns a thread, all rows under way at once:
// bound by HBM (4096 x 2048, 8 rows each: 29.5 us, 5.1 TB/s; backward, with the k dot
// products of a token kept in registers and reduced once, 53.3 us, 5.3 TB/s).
#include "dgf_experts.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
constexpr int kRouteBlocks = 256;  // at most: one for each CU (4096 x 128, 8 choices: 5.4 and 6.4 us; half as many 8.2 and 5.8)
constexpr uint32_t kClosed = 0x007fffffu;  // key of -infinity: an expert no token may take

// A logit as the router takes it: NaN is -infinity (never chosen), +infinity the
// largest finite value (so that weights stay numbers), -0 is +0.
__device__ __forceinline__ float clean(float l) {
  if (!(l == l)) return -__builtin_inff();
  return fminf(l, 3.402823466e+38f) + 0.0f;
}
__device__ __forceinline__ float logit_at(const void *row, int lt, int64_t e) {
  if (lt == 2) return clean(static_cast<const float *>(row)[e]);
  const uint16_t h = static_cast<const uint16_t *>(row)[e];
  return clean(lt == FMT_F16 ? F16::f(h) : Bf16::f(h));
}
__device__ __forceinline__ const void *logit_row(const RouteParams &p, int64_t m) {
  return static_cast<const char *>(p.logits) + m * p.ld * (p.lt == 2 ? 4 : 2);
}
// Order-preserving bits of a cleaned logit (0 stays free: taken).
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t u = __float_as_uint(l);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define DGF_MAX_STEP(ctrl, rows)                                                                    \
  {                                                                                                 \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false);    \
    v = o > v ? o : v;                                                                              \
  }
  DGF_MAX_STEP(0x111, 0xf)
  DGF_MAX_STEP(0x112, 0xf)
  DGF_MAX_STEP(0x114, 0xf)
  DGF_MAX_STEP(0x118, 0xf)
  DGF_MAX_STEP(0x142, 0xa)
  DGF_MAX_STEP(0x143, 0xc)
#undef DGF_MAX_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_last(v)), 63));
}

// One wave chooses for token m: lane j < k ends with choice j's expert (-1: no
// open expert left), which it also counts.
template <int NL>
__device__ __forceinline__ void choose(const RouteParams &p, int64_t m, int lane, int *hist) {
  const void *row = logit_row(p, m);
  uint32_t key[NL];
  float all = 0.0f;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < p.E ? order_key(logit_at(row, p.lt, e)) : 0;
  }
  float top = 0.0f, mine = 0.0f;
  int id = -1;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NL; ++i) best = key[i] > best ? key[i] : best;
    best = wave_max(best);
    if (best <= kClosed) break;
    int at = -1;  // the lowest index that has it
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint64_t has = __ballot(key[i] == best);
      if (at < 0 && has) at = 64 * i + __builtin_ctzll(has);
    }
    const float v = key_value(best);
    if (j == 0) {
      top = v;
      if (!p.renorm) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if (key[i] > kClosed) all += expf(key_value(key[i]) - top);
      }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (lane + 64 * i == at) key[i] = 0;
    if (lane == j) {
      id = at;
      mine = expf(v - top);
    }
  }
  const float sum = wave_sum(p.renorm ? mine : all);
  if (lane < p.k) {
    p.ids[m * p.k + lane] = id;
    p.probs[m * p.k + lane] = id < 0 ? 0.0f : mine / sum;
    if (id >= 0) atomicAdd(&hist[id], 1);
  }
}

// Tokens of block b: [first, last).
__device__ __forceinline__ void block_tokens(const RouteParams &p, int b, int64_t &first, int64_t &last) {
  const int64_t per = (p.M + p.blocks - 1) / p.blocks;
  first = per * b < p.M ? per * b : p.M;
  last = first + per < p.M ? first + per : p.M;
}

struct RouteLds {
  int hist[kExpertsMaxE];
  int base[kExpertsMaxE];                 // first sorted row of the block's pairs, by expert
  int wave_sums[kRouteWaves];
  int wave_base[kRouteWaves][kExpertsMaxE];
};

template <int NL>
__device__ __forceinline__ void choose_block(const RouteParams &p, int b, int *hist) {
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  int64_t first, last;
  block_tokens(p, b, first, last);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t m = first + wave; m < last; m += kRouteWaves) choose<NL>(p, m, lane, hist);
  __syncthreads();
}

// Sorted rows of block b's pairs.  lds.base holds, by expert, how many pairs the
// blocks before this one have of it, lds.hist how many there are in all.
__device__ __forceinline__ void place_block(const RouteParams &p, int b, RouteLds &lds) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  // exclusive prefix over experts of the totals
  const int own = tid < p.E ? lds.hist[tid] : 0;
  int sum = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(sum, d);
    if (lane >= d) sum += v;
  }
  if (lane == 63) lds.wave_sums[wave] = sum;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kRouteWaves; ++w) {
    if (w < wave) before += lds.wave_sums[w];
    total += lds.wave_sums[w];
  }
  if (tid < p.E) {
    lds.base[tid] += before + sum - own;
    if (b == 0) p.off[tid + 1] = before + sum;
  }
  if (b == 0 && tid == 0) p.off[0] = 0;
  // each wave counts its run of the block's pairs, then takes its first rows
  int64_t first, last;
  block_tokens(p, b, first, last);
  const int64_t p0 = first * p.k, np = (last - first) * p.k;
  const int64_t run = (np + 64 * kRouteWaves - 1) / (64 * kRouteWaves) * 64;
  const int64_t w0 = run * wave < np ? run * wave : np, w1 = w0 + run < np ? w0 + run : np;
  const int waves = run ? (int)((np + run - 1) / run) : 0;
  if (waves > 1) {
    for (int e = lane; e < p.E; e += 64) lds.wave_base[wave][e] = 0;
    for (int64_t i = w0 + lane; i < w1; i += 64) {
      const int id = p.ids[p0 + i];
      if (id >= 0) atomicAdd(&lds.wave_base[wave][id], 1);
    }
  }
  __syncthreads();
  if (tid < p.E) {
    int at = lds.base[tid];
    lds.wave_base[0][tid] = waves > 1 ? lds.wave_base[0][tid] : 0;
    for (int w = 0; w < waves; ++w) {
      const int n = lds.wave_base[w][tid];
      lds.wave_base[w][tid] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t i0 = w0; i0 < w1; i0 += 64) {
    const int64_t i = i0 + lane;
    const int id = i < w1 ? p.ids[p0 + i] : -1;
    // the lanes with this lane's expert: their order is the pairs' own
    uint64_t same = __ballot(id >= 0);
    for (int bit = 1; bit < p.E; bit <<= 1) {
      const uint64_t set = __ballot((id & bit) != 0);
      same &= id & bit ? set : ~set;
    }
    if (id >= 0) {
      const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
      const int row = lds.wave_base[wave][id] + rank;
      p.rows[row] = (int)((p0 + i) / p.k);
      p.pos[p0 + i] = row;
      wave_lds_sync();
      if (same >> lane == 1) lds.wave_base[wave][id] = row + 1;  // the last of them
    } else if (i < w1) {
      p.pos[p0 + i] = -1;
    }
    wave_lds_sync();
  }
  // no pair behind the last sorted row
  for (int64_t r = total + (int64_t)b * kRouteThreads + tid; r < p.M * p.k; r += (int64_t)p.blocks * kRouteThreads) p.rows[r] = -1;
}

template <int NL>
__global__ __launch_bounds__(kRouteThreads) void k_route_choose(RouteParams p) {
  __shared__ int hist[kExpertsMaxE];
  choose_block<NL>(p, blockIdx.x, hist);
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) p.counts[(int64_t)blockIdx.x * p.E + e] = (uint16_t)hist[e];
}

__global__ __launch_bounds__(kRouteThreads) void k_route_place(RouteParams p) {
  __shared__ RouteLds lds;
  const int tid = threadIdx.x, b = blockIdx.x;
  // `parts` threads an expert add up the blocks' counts, those before this one apart
  int parts = kRouteThreads;
  while (parts * p.E > kRouteThreads) parts >>= 1;
  parts = parts < 1 ? 1 : parts;
  for (int e = tid; e < p.E; e += kRouteThreads) lds.hist[e] = lds.base[e] = 0;
  __syncthreads();
  if (tid < parts * p.E) {
    const int e = tid % p.E, part = tid / p.E;
    const int per = (p.blocks + parts - 1) / parts;
    const int q1 = (part + 1) * per < p.blocks ? (part + 1) * per : p.blocks;
    int all = 0, before = 0;
#pragma unroll 8
    for (int q = part * per; q < q1; ++q) {
      const int n = p.counts[(int64_t)q * p.E + e];
      all += n;
      before += q < b ? n : 0;
    }
    atomicAdd(&lds.hist[e], all);
    atomicAdd(&lds.base[e], before);
  }
  __syncthreads();
  place_block(p, b, lds);
}

// Choice and order in one workgroup.
template <int NL>
__global__ __launch_bounds__(kRouteThreads) void k_route_one(RouteParams p) {
  __shared__ RouteLds lds;
  choose_block<NL>(p, 0, lds.hist);
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) lds.base[e] = 0;
  __threadfence_block();
  __syncthreads();
  place_block(p, 0, lds);
}

// dl_e = P_e (dp_e - sum over the choices of dp p), P the softmax that the weights
// came from (over the choices: P = probs; over all experts: from the logits).
template <int NL>
__global__ __launch_bounds__(256) void k_route_bwd(RouteParams p) {
  const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (m >= p.M) return;
  int id = -1;
  float pr = 0.0f, dp = 0.0f;
  if (lane < p.k) {
    id = p.ids[m * p.k + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      pr = p.probs[m * p.k + lane];
      dp = p.dprobs[m * p.k + lane];
    }
  }
  const float s = wave_sum(dp * pr);
  float d[NL];
  if (p.renorm) {
#pragma unroll
    for (int i = 0; i < NL; ++i) d[i] = 0.0f;
  } else {
    const void *row = logit_row(p, m);
    float l[NL], sum = 0.0f;
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < p.E ? logit_at(row, p.lt, e) : -__builtin_inff();
      const uint32_t k = order_key(l[i]);
      best = k > best ? k : best;
    }
    const float top = key_value(wave_max(best));
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      d[i] = l[i] > -__builtin_inff() ? expf(l[i] - top) : 0.0f;
      sum += d[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < NL; ++i) d[i] = d[i] > 0.0f ? -s * (d[i] / sum) : 0.0f;
  }
  const float own = p.renorm ? pr * (dp - s) : pr * dp;
  for (int j = 0; j < p.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(own), j));
    if (e < 0) continue;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (lane + 64 * i == e) d[i] += v;
  }
  char *out = static_cast<char *>(p.dlogits) + m * p.ld_d * (p.lt == 2 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.E) continue;
    if (p.lt == 2) reinterpret_cast<float *>(out)[e] = d[i];
    else reinterpret_cast<uint16_t *>(out)[e] = p.lt == FMT_F16 ? F16::r(d[i]) : Bf16::r(d[i]);
  }
}

// ------------------------------------------------------------------ combine

// Threads a token of H columns: a wave at least, 8 columns a thread and step.
__host__ __device__ inline int combine_threads(int H) {
  const int want = (H + 7) / 8;
  return want <= 64 ? 64 : want <= 128 ? 128 : 256;
}

template <class T, int KK>
__global__ __launch_bounds__(256) void k_combine(CombineParams p) {
  const int per = combine_threads(p.H);
  const int64_t m = (int64_t)blockIdx.x * (256 / per) + threadIdx.x / per;
  if (m >= p.M) return;
  const int k = KK > 0 ? KK : p.k;
  for (int c = 8 * (threadIdx.x % per); c < p.H; c += 8 * per) {
    float acc[8] = {};
    constexpr int kStep = KK > 0 ? KK : 4;
    for (int j0 = 0; j0 < k; j0 += kStep) {
      uint4 v[kStep];
      float w[kStep];
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        int pos = -1;
        w[j] = 0.0f;
        if (j0 + j < k) pos = p.pos[m * p.k + j0 + j];
        v[j] = make_uint4(0, 0, 0, 0);
        if (pos >= 0 && pos < p.R) {
          w[j] = p.probs ? p.probs[m * p.k + j0 + j] : 1.0f;
          v[j] = row_ld(p.o + pos * p.ld_o, c, p.H);
        }
      }
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        float f[8];
        row_widen<T>(v[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(w[j], f[e], acc[e]);
      }
    }
    row_st(p.y + m * p.ld_y, c, p.H, row_narrow<T>(acc));
  }
}

template <class T, int KK>
__global__ __launch_bounds__(256) void k_combine_bwd(CombineParams p) {
  const int per = combine_threads(p.H), slot = threadIdx.x / per;
  const int64_t m = (int64_t)blockIdx.x * (256 / per) + slot;
  __shared__ float red[4][kExpertsMaxK];
  const int k = KK > 0 ? KK : p.k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kStep = KK > 0 ? KK : 4;
  for (int j0 = 0; j0 < k; j0 += kStep) {
    float dot[kStep];
    int pos[kStep];
    float w[kStep];
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      dot[j] = 0.0f;
      pos[j] = m < p.M && j0 + j < k ? p.pos[m * p.k + j0 + j] : -1;
      if (pos[j] >= p.R) pos[j] = -1;
      w[j] = pos[j] >= 0 && p.probs ? p.probs[m * p.k + j0 + j] : 1.0f;
    }
    if (m < p.M)
      for (int c = 8 * (threadIdx.x % per); c < p.H; c += 8 * per) {
        float d[8];
        row_widen<T>(row_ld(p.y + m * p.ld_y, c, p.H), d);
        uint4 v[kStep];
        if (p.dprobs) {
#pragma unroll
          for (int j = 0; j < kStep; ++j) v[j] = pos[j] >= 0 ? row_ld(p.o + pos[j] * p.ld_o, c, p.H) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
          if (pos[j] < 0) continue;
          float f[8], g[8];
          if (p.dprobs) {
            row_widen<T>(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[j] = __builtin_fmaf(d[e], f[e], dot[j]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = w[j] * d[e];
          row_st(p.d_o + pos[j] * p.ld_do, c, p.H, row_narrow<T>(g));
        }
      }
    if (p.dprobs) {
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const float s = wave_sum_last(dot[j]);
        if (lane == 63) red[wave][(j0 + j) & (kExpertsMaxK - 1)] = s;
      }
    }
  }
  if (!p.dprobs) return;
  __syncthreads();
  const int j = threadIdx.x % per;
  if (m < p.M && j < k) {
    float s = 0.0f;
    for (int w = 0; w < per / 64; ++w) s += red[slot * (per / 64) + w][j];
    p.dprobs[m * p.k + j] = s;
  }
}

template <class T>
hipError_t combine_t(const CombineParams &p, bool back, hipStream_t s) {
  const int tokens = 256 / combine_threads(p.H);
  const dim3 g((uint32_t)((p.M + tokens - 1) / tokens)), b(256);
#define DGF_COMBINE(KK)                                        \
  if (back) dgf_launch((k_combine_bwd<T, KK>), g, b, 0, s, p); \
  else dgf_launch((k_combine<T, KK>), g, b, 0, s, p)
  switch (p.k) {
    case 1: DGF_COMBINE(1); break;
    case 2: DGF_COMBINE(2); break;
    case 4: DGF_COMBINE(4); break;
    case 8: DGF_COMBINE(8); break;
    default: DGF_COMBINE(0); break;
  }
#undef DGF_COMBINE
  return hipGetLastError();
}

}  // namespace

int64_t route_once() { return 64; }

// Workgroups that choose and place: 16 tokens each, one a wave, as long as every
// CU has at most one.
int route_blocks(int64_t M) {
  const int64_t want = (M + kRouteWaves - 1) / kRouteWaves;
  return (int)(want < kRouteBlocks ? want : kRouteBlocks);
}

#define DGF_ROUTE(KERNEL, GRID, THREADS)                                                          \
  if (p.E <= 64) dgf_launch(KERNEL<1>, dim3(GRID), dim3(THREADS), 0, s, p);                       \
  else if (p.E <= 128) dgf_launch(KERNEL<2>, dim3(GRID), dim3(THREADS), 0, s, p);                 \
  else if (p.E <= 256) dgf_launch(KERNEL<4>, dim3(GRID), dim3(THREADS), 0, s, p);                 \
  else if (p.E <= 512) dgf_launch(KERNEL<8>, dim3(GRID), dim3(THREADS), 0, s, p);                 \
  else dgf_launch(KERNEL<kExpertsMaxE / 64>, dim3(GRID), dim3(THREADS), 0, s, p);                 \
  return hipGetLastError()

hipError_t launch_route_choose(const RouteParams &p, hipStream_t s) { DGF_ROUTE(k_route_choose, (uint32_t)p.blocks, kRouteThreads); }
hipError_t launch_route_one(const RouteParams &p, hipStream_t s) { DGF_ROUTE(k_route_one, 1, kRouteThreads); }
hipError_t launch_route_place(const RouteParams &p, hipStream_t s) {
  dgf_launch(k_route_place, dim3((uint32_t)p.blocks), dim3(kRouteThreads), 0, s, p);
  return hipGetLastError();
}
hipError_t launch_route_bwd(const RouteParams &p, hipStream_t s) { DGF_ROUTE(k_route_bwd, (uint32_t)((p.M + 3) / 4), 256); }

hipError_t launch_combine(const CombineParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? combine_t<F16>(p, false, s) : combine_t<Bf16>(p, false, s);
}
hipError_t launch_combine_bwd(const CombineParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? combine_t<F16>(p, true, s) : combine_t<Bf16>(p, true, s);
}

}  // namespace dgf
