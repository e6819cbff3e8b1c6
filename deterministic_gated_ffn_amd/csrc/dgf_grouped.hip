// Matrix products grouped by expert over ragged rows (gfx950).
#include "dgf_device.hpp"
#include "dgf_experts.hpp"

namespace dgf {
namespace {

constexpr int kBK = 64;          // contraction elements of a stage
constexpr int kGroupedWaves = 8;  // 2 over the tile's rows x 4 over its columns

typedef __attribute__((address_space(3))) uint16_t lds_u16;
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ const uint4 kZeros[1] = {};

// 16 bytes from `src` to the wave's 1024 bytes of LDS at `dst` (byte offset,
// uniform), lane l's at dst + 16 l, without passing through registers.  The
// compiler does not count the load: stage_wait() below does.
__device__ __forceinline__ void lds_load(const char *src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "memory");
}
__device__ __forceinline__ void stage_wait() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Where 16 bytes of an operand's tile of BX rows (or columns) x kBK go in LDS.
//  - contraction contiguous (TR false): row r takes 128 bytes, its 16-byte piece
//    c sits at c ^ (r & 7): the 16 rows of a fragment read take all banks.
//  - contraction across rows (TR): row k takes 2 BX bytes and is read in
//    transposed blocks of 4 k x 16 columns (32 bytes of 4 rows each), whose
//    rows sw(k) moves to different banks.
template <int BX>
__device__ __forceinline__ int tr_swizzle(int k) {
  const int s = (k & 3) | ((((k >> 2) ^ (k >> 3)) & 1) << 2);
  return BX >= 128 ? s << 1 : (s & 3) << 1;
}

// One operand's loader: the thread's pieces of a stage and their addresses.
template <bool TR, int BX>
struct Loader {
  static constexpr int NL = BX / 64;  // wave loads of 1 KB a stage and wave
  static constexpr int kPieces = BX / 8;  // 16-byte pieces of a k row (TR)
  const char *p[NL];
  uint32_t step[NL];  // bytes to the next stage; 0 where the piece is none of the tile's
  int koff[NL];       // TR: k row of the piece; else: first k of the piece

  // TR false: row i of the tile at base(i) (null: none)
  template <class F>
  __device__ __forceinline__ void start_rows(int wave, int lane, F &&base) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = 8 * (wave + kGroupedWaves * i) + (lane >> 3);
      const char *b = base(row);
      koff[i] = 8 * ((lane & 7) ^ (lane >> 3));
      p[i] = b ? b + 2 * koff[i] : reinterpret_cast<const char *>(kZeros);
      step[i] = b ? 2 * kBK : 0;
    }
  }
  // TR: k row k, columns c.. of the tile
  static __device__ __forceinline__ int k_row(int wave, int lane, int i) {
    return (wave + kGroupedWaves * i) * (64 / kPieces) + lane / kPieces;
  }
  static __device__ __forceinline__ int col(int lane, int k) { return 8 * ((lane % kPieces) ^ tr_swizzle<BX>(k)); }
};

template <class T, bool TR, int BX>
__device__ __forceinline__ typename T::frag frag_at(const uint16_t *tile, int x0, int kk, int lane) {
  const int i = lane & 15, g = lane >> 4;
  if constexpr (!TR) {
    return *reinterpret_cast<const typename T::frag *>(tile + (x0 + i) * kBK + 8 * ((4 * kk + g) ^ (i & 7)));
  } else {
    union { s16x4 h[2]; typename T::frag f; } u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 32 * kk + 8 * g + 4 * h + (i >> 2);
      const int piece = ((x0 >> 3) + ((i & 3) >> 1)) ^ tr_swizzle<BX>(k);
      const uint16_t *a = tile + k * BX + 8 * piece + 4 * (i & 1);
      u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(a));
    }
    return u.f;
  }
}

// Zeros from contraction element kv on, in a stage of rows x kBK (TR false).
__device__ __forceinline__ void zero_tail(uint16_t *tile, int rows, int kv) {
  const int c0 = kv >> 3;  // the piece that ends the row; those behind it were loaded as zeros
  if (kv & 7)
    for (int r = threadIdx.x; r < rows; r += 64 * kGroupedWaves) {
      uint16_t *q = tile + r * kBK + 8 * (c0 ^ (r & 7));
      for (int e = kv & 7; e < 8; ++e) q[e] = 0;
    }
}

// One tile of 32 FM rows x 64 FN columns at (row0, n0) of expert e, whose rows
// (TN: contraction) are [lo, hi).
template <class T, int LAYOUT, int FM, int FN>
__device__ __forceinline__ void tile(const GroupedParams &p, char *lds, int e, int64_t lo, int64_t hi, int64_t row0, int n0) {
  constexpr bool ATR = LAYOUT == DGF_LAYOUT_TN, BTR = LAYOUT != DGF_LAYOUT_NT;
  constexpr int BM = 32 * FM, BN = 64 * FN, kStage = (BM + BN) * kBK * 2;
  typedef Loader<ATR, BM> LA;
  typedef Loader<BTR, BN> LB;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t klen = ATR ? hi - lo : p.K;
  const int nb = (int)((klen + kBK - 1) / kBK), total = nb * p.terms;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;

  LA la;
  LB lb;
  int idx[LB::NL];  // TN with a row list: the rows of the stage to load next
  auto open = [&](int term) {
    const GroupedTerm &t = p.t[term];
    if constexpr (!ATR) {
      la.start_rows(wave, lane, [&](int row) -> const char * {
        const int64_t r = row0 + row;
        if (r >= hi) return nullptr;
        const int64_t a = p.rows ? p.rows[r] : r;
        if (a < 0 || a >= p.T) return nullptr;
        return reinterpret_cast<const char *>(t.A + a * t.lda);
      });
    } else {
#pragma unroll
      for (int i = 0; i < LA::NL; ++i) {
        const int k = LA::k_row(wave, lane, i);
        const int64_t c = row0 + LA::col(lane, k);
        la.koff[i] = c < p.M ? k : 1 << 30;
        la.p[i] = reinterpret_cast<const char *>(t.A + (lo + k) * t.lda + c);
      }
    }
    if constexpr (!BTR) {
      lb.start_rows(wave, lane, [&](int row) -> const char * {
        return n0 + row < p.N ? reinterpret_cast<const char *>(t.B + e * t.stride_b + (int64_t)(n0 + row) * t.ldb) : nullptr;
      });
    } else {
#pragma unroll
      for (int i = 0; i < LB::NL; ++i) {
        const int k = LB::k_row(wave, lane, i);
        const int c = n0 + LB::col(lane, k);
        lb.koff[i] = c < p.N ? k : 1 << 30;
        if (!ATR) lb.p[i] = reinterpret_cast<const char *>(t.B + e * t.stride_b + (int64_t)k * t.ldb + c);
        else if (!p.rows) lb.p[i] = reinterpret_cast<const char *>(t.B + (lo + k) * t.ldb + c);
        else lb.p[i] = reinterpret_cast<const char *>(t.B + c);
      }
    }
  };
  // the row list's entries for the stage that starts at k0
  auto list = [&](int64_t k0) {
    if constexpr (ATR) {
      if (p.rows)
#pragma unroll
        for (int i = 0; i < LB::NL; ++i) {
          const int64_t k = k0 + LB::k_row(wave, lane, i);
          idx[i] = k < klen ? p.rows[lo + k] : -1;
        }
    }
  };
  const char *const zeros = reinterpret_cast<const char *>(kZeros);
  auto load = [&](int j) {
    const int term = j >= nb;
    const int64_t k0 = (int64_t)(j - term * nb) * kBK;
    const bool tail = k0 + kBK > klen;
    const uint32_t dst = lds0 + (j & 1) * kStage + wave * 1024;
    const int64_t a_step = p.t[term].lda * (2 * kBK), b_step = p.t[term].ldb * (2 * kBK);
#pragma unroll
    for (int i = 0; i < LA::NL; ++i) {
      const char *q = la.p[i];
      if constexpr (ATR) {
        if (la.koff[i] >= klen - k0) q = zeros;
        la.p[i] += a_step;
      } else {
        if (tail && k0 + la.koff[i] >= klen) q = zeros;
        la.p[i] += la.step[i];
      }
      lds_load(q, dst + i * 1024 * kGroupedWaves);
    }
#pragma unroll
    for (int i = 0; i < LB::NL; ++i) {
      const char *q = lb.p[i];
      if constexpr (!BTR) {
        if (tail && k0 + lb.koff[i] >= klen) q = zeros;
        lb.p[i] += lb.step[i];
      } else if (ATR && p.rows) {
        q = (uint32_t)idx[i] < (uint32_t)p.T && lb.koff[i] < (1 << 30) ? q + (int64_t)idx[i] * p.t[0].ldb * 2 : zeros;
      } else {
        if (lb.koff[i] >= klen - k0) q = zeros;
        lb.p[i] += b_step;
      }
      lds_load(q, dst + BM * kBK * 2 + i * 1024 * kGroupedWaves);
    }
    if (j + 1 == nb && p.terms == 2) open(1);
    list(k0 + kBK);
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (total > 0) {
    open(0);
    list(0);
    load(0);
  }
  for (int j = 0; j < total; ++j) {
    stage_wait();  // stage j has landed in every wave; stage j - 1 is read out
    uint16_t *sa = reinterpret_cast<uint16_t *>(lds + (j & 1) * kStage), *sb = sa + BM * kBK;
    if (j + 1 < total) load(j + 1);
    if ((j + 1 == nb || j + 1 == total) && (klen & 7) && !(ATR && BTR)) {
      const int kv = (int)(klen - (int64_t)(nb - 1) * kBK);
      if (!ATR) zero_tail(sa, BM, kv);
      if (!BTR) zero_tail(sb, BN, kv);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      typename T::frag a[FM], b[FN];
#pragma unroll
      for (int n = 0; n < FN; ++n) b[n] = frag_at<T, BTR, BN>(sb, (wn * FN + n) * 16, kk, lane);
#pragma unroll
      for (int m = 0; m < FM; ++m) a[m] = frag_at<T, ATR, BM>(sa, (wm * FM + m) * 16, kk, lane);
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[m][n] = T::mfma(b[n], a[m], acc[m][n]);
    }
  }

  // lane l holds columns 4 (l / 16) .. + 3 of row l % 16 of each 16 x 16 block
  const int i = lane & 15, g = lane >> 4;
  const int64_t rend = ATR ? p.M : hi;
  uint16_t *C = ATR ? p.C + e * p.stride_c : p.C;
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int64_t r = row0 + (wm * FM + m) * 16 + i;
    if (r >= rend) continue;
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      const int c = n0 + (wn * FN + n) * 16 + 4 * g;
      uint16_t *o = C + r * p.ldc + c;
      const uint2 v = make_uint2(T::pack(acc[m][n][0], acc[m][n][1]), T::pack(acc[m][n][2], acc[m][n][3]));
      if (c + 4 <= p.N) {
        *reinterpret_cast<uint2 *>(o) = v;
      } else {
        const uint32_t w[2] = {v.x, v.y};
        for (int q = 0; c + q < p.N && q < 4; ++q) o[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
      }
    }
  }
}

// The rows [lo, hi) of expert e, within the R there are whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const GroupedParams &p, int e, int64_t &lo, int64_t &hi) {
  lo = p.off[e];
  hi = p.off[e + 1];
  lo = lo < 0 ? 0 : lo > p.R ? p.R : lo;
  hi = hi < lo ? lo : hi > p.R ? p.R : hi;
}

// NT, NN: finds the tile's expert by the prefix sum of the experts' row tiles.
template <class T, int LAYOUT, int FM, int FN>
__global__ __launch_bounds__(64 * kGroupedWaves) void k_grouped_rows(GroupedParams p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int BM = 32 * FM;
  const int lane = threadIdx.x & 63;
  int t = xcd_tile(blockIdx.x, p.tiles);
  int found = -1, local = 0, mt = 0;
  int64_t lo = 0, hi = 0;
  for (int e0 = 0; e0 < p.E && found < 0; e0 += 64) {
    int64_t l = 0, h = 0;
    if (e0 + lane < p.E) expert_rows(p, e0 + lane, l, h);
    const int m = (int)((h - l + BM - 1) / BM);
    int sum = m * p.tiles_n;
    const int own = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    const uint64_t past = __ballot(sum > t);
    if (past) {
      const int w = __builtin_ctzll(past);
      found = e0 + w;
      local = t - (__shfl(sum, w) - __shfl(own, w));
      mt = __shfl(m, w);
      lo = __shfl((int)l, w);
      hi = __shfl((int)h, w);
    } else {
      t -= __shfl(sum, 63);
    }
  }
  // (offsets that are not ascending can make the sums wrap: no tile then)
  if (found < 0 || (uint32_t)local >= (uint32_t)(mt * p.tiles_n)) return;
  found = __builtin_amdgcn_readfirstlane(found);
  local = __builtin_amdgcn_readfirstlane(local);
  mt = __builtin_amdgcn_readfirstlane(mt);
  lo = __builtin_amdgcn_readfirstlane((int)lo);
  hi = __builtin_amdgcn_readfirstlane((int)hi);
  // up to 8 row tiles in turn for each column tile
  const int group = 8 * p.tiles_n, first = local / group * 8, rows = mt - first < 8 ? mt - first : 8;
  const int in = local % group;
  const int64_t row0 = lo + (int64_t)BM * (first + in % rows);
  const int n0 = in / rows * 64 * FN;
  const int left = (int)((hi - row0 < BM ? hi - row0 : BM) + 63) / 64;
  if (FM >= 8 && left == 4) tile<T, LAYOUT, FM < 8 ? FM : 8, FN>(p, lds, found, lo, hi, row0, n0);
  else if (FM >= 6 && left == 3) tile<T, LAYOUT, FM < 6 ? FM : 6, FN>(p, lds, found, lo, hi, row0, n0);
  else if (FM >= 4 && left == 2) tile<T, LAYOUT, FM < 4 ? FM : 4, FN>(p, lds, found, lo, hi, row0, n0);
  else tile<T, LAYOUT, 2, FN>(p, lds, found, lo, hi, row0, n0);
}

template <class T, int FM, int FN>
__global__ __launch_bounds__(64 * kGroupedWaves) void k_grouped_tn(GroupedParams p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int t = xcd_tile(blockIdx.x, p.tiles);
  const int per = p.tiles_m * p.tiles_n, e = t / per, in = t % per;
  int64_t lo, hi;
  expert_rows(p, e, lo, hi);
  const int group = 8 * p.tiles_n, first = in / group * 8, rows = p.tiles_m - first < 8 ? p.tiles_m - first : 8;
  const int at = in % group;
  tile<T, DGF_LAYOUT_TN, FM, FN>(p, lds, e, lo, hi, (int64_t)(first + at % rows) * 32 * FM, at / rows * 64 * FN);
}

template <int FM, int FN>
constexpr size_t lds_bytes() { return (size_t)2 * (32 * FM + 64 * FN) * kBK * 2; }

template <class T, int FM, int FN>
hipError_t rows_launch(GroupedParams p, hipStream_t s) {
  p.tiles_n = (p.N + 64 * FN - 1) / (64 * FN);
  const int64_t most = p.R / (32 * FM) + (p.R < p.E ? p.R : p.E);  // row tiles, at most
  p.tiles = (int)(most * p.tiles_n);
  const dim3 g((uint32_t)p.tiles), b(64 * kGroupedWaves);
  if (p.layout == DGF_LAYOUT_NT) dgf_launch((k_grouped_rows<T, DGF_LAYOUT_NT, FM, FN>), g, b, lds_bytes<FM, FN>(), s, p);
  else dgf_launch((k_grouped_rows<T, DGF_LAYOUT_NN, FM, FN>), g, b, lds_bytes<FM, FN>(), s, p);
  return hipGetLastError();
}

template <class T, int FM, int FN>
hipError_t tn_launch(GroupedParams p, hipStream_t s) {
  p.tiles_m = (p.M + 32 * FM - 1) / (32 * FM);
  p.tiles_n = (p.N + 64 * FN - 1) / (64 * FN);
  p.tiles = p.tiles_m * p.tiles_n * p.E;
  dgf_launch((k_grouped_tn<T, FM, FN>), dim3((uint32_t)p.tiles), dim3(64 * kGroupedWaves), lds_bytes<FM, FN>(), s, p);
  return hipGetLastError();
}

template <class T>
hipError_t grouped_t(const GroupedParams &p, hipStream_t s) {
  if (p.layout == DGF_LAYOUT_TN) {
    const int64_t big = (int64_t)((p.M + 255) / 256) * ((p.N + 255) / 256) * p.E;
    return big >= 256 ? tn_launch<T, 8, 4>(p, s) : tn_launch<T, 4, 2>(p, s);
  }
  const int64_t rows = p.R / p.E;
  if (rows > 64) {
    const int64_t big = (p.R + 255) / 256 * ((p.N + 255) / 256);
    return big >= 192 ? rows_launch<T, 8, 4>(p, s) : rows_launch<T, 4, 2>(p, s);
  }
  return rows_launch<T, 2, 2>(p, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? grouped_t<F16>(p, s) : grouped_t<Bf16>(p, s);
}

}  // namespace dgf
