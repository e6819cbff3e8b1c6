// Matrix products grouped by expert over ragged rows (gfx950).
//
//   NT, NN: C[r] = A[rows[r]] B_e^T, A[rows[r]] B_e  for e's rows r (NN: two such terms)
//   TN:     C_e = sum over e's rows r of A[r]^T B[rows[r]]
//
// Large experts are bound by the matrix cores, many small ones by their weights (TN: their
// outputs) in HBM.  A workgroup of 8 waves owns tiles of 256 x 256 (or smaller ones, see
// grouped_l), 128 x 64 a wave, and multiplies stages of 32 contraction elements with 16 x 16 x
// 32 products, ascending, in FP32.  Stages go from memory to LDS without passing through
// registers, four of them in 128 KB, so that two are on their way while one is multiplied;
// one barrier a stage publishes the one that has landed, and the fragments of A are read a
// few products ahead of their use.  Operands whose contraction runs across rows are read back
// transposed, four rows at a time.  With a row list every lane has its row's address, which NT and
// NN look up once a tile (32768 rows over 128 experts, rows in order: 175 us with a list and
// without) and TN at every stage (213 against 194).
//
// The grid is one workgroup a CU (two of the smaller tiles) for the whole call; each takes its
// share of all tiles as one stream of stages, the next tile's loads under way while the last
// is multiplied and stored.  Row tiles are as even as their expert allows, in units of 64.
// Everything that is the same for a whole wave is kept in scalar registers: state that the
// compiler moved to vector registers cost the accumulators theirs.
//
// Measured, BF16, calls among others on several cards: 8192^3 NT / NN / TN 886-901 / 845-890 /
// 950-990 us (1220-1300 TFLOP/s, TN 1110-1160; a library's plain product 750).  32768 rows over
// 128 experts, 2048 -> 768: 161-170 us (under a profiler, median 190) against 91 for its bytes at
// the rate of a copy; their weights' gradients 206-217 (220), 91 likewise (402 MB of outputs,
// whose stores overlap little with the products); 8192 rows over 8 experts, two terms, 12288 ->
// 4096: 1710-1790 us (1810), 920-960 TFLOP/s; 1390 with equal experts: the rest is what uneven ones
// leave idle.  Tiles are dealt by their number, whatever their height: the heaviest workgroup of
// these three has 1.1 to 1.35 times the mean.
#include "dgf_device.hpp"
#include "dgf_experts.hpp"
#include "dgf_rows.hpp"

namespace dgf {
namespace {

constexpr int kU = 32;  // contraction elements of a stage

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ const uint4 kZeros[1] = {};

// 16 bytes from `src` to the wave's 1024 bytes of LDS at `dst` (byte offset,
// uniform), lane l's at dst + 16 l, without passing through registers.  The
// compiler does not count the load: stage_wait() below does.
__device__ __forceinline__ void lds_load(const char *src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(__builtin_amdgcn_readfirstlane(dst))
               : "memory");
}
// All but the N youngest of this wave's loads have landed; then every wave's.
template <int N>
__device__ __forceinline__ void stage_wait() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Where 16 bytes of an operand's tile of BX rows (or columns) x kU go in LDS.
//  - contraction contiguous (TR false): row r takes 64 bytes, its 16-byte piece
//    c sits at c ^ (r / 2 & 3): the rows of a fragment read take all banks.
//  - contraction across rows (TR): row k takes 2 BX bytes and is read in
//    transposed blocks of 4 k x 16 columns (32 bytes of 4 rows each), whose
//    rows sw(k) moves to different banks.
template <int BX>
__device__ __forceinline__ int tr_swizzle(int k) {
  const int s = (k & 3) | ((((k >> 2) ^ (k >> 3)) & 1) << 2);
  return BX >= 128 ? s << 1 : (s & 3) << 1;
}

// A wave's pieces of a stage: 1 KB loads `wave`, `wave + waves`, ... of the BX / 8
// that the operand's tile takes; 16 bytes a lane.
template <bool TR, int BX, int WAVES>
struct Pieces {
  // (a wave past the last load repeats another's: every wave counts the same loads)
  static constexpr int kAll = BX / 16, NL = (kAll + WAVES - 1) / WAVES;
  static __device__ __forceinline__ int load(int wave, int i) { return kAll % WAVES ? (wave + WAVES * i) % kAll : wave + WAVES * i; }
  static constexpr int kRow = BX / 8;  // pieces of a k row (TR)
  // TR false: row of the tile and first k of the lane's piece
  static __device__ __forceinline__ int row(int wave, int lane, int i) { return 16 * load(wave, i) + (lane >> 2); }
  static __device__ __forceinline__ int k_of(int lane) { return 8 * ((lane & 3) ^ (lane >> 3 & 3)); }
  // TR: its k row and first column
  static __device__ __forceinline__ int k_row(int wave, int lane, int i) { return load(wave, i) * (64 / kRow) + lane / kRow; }
  // (the next load's k row is kMore further, at the same column: the swizzle repeats after 16)
  static constexpr int kMore = WAVES * (64 / kRow);
  static_assert(!TR || NL == 1 || (kAll % WAVES == 0 && kMore % 16 == 0), "one address for all of a wave's loads");
  static __device__ __forceinline__ int col(int lane, int k) { return 8 * ((lane % kRow) ^ tr_swizzle<BX>(k)); }
};

template <class T, bool TR, int BX>
__device__ __forceinline__ typename T::frag frag_at(const uint16_t *tile, int x0, int lane) {
  const int i = lane & 15, g = lane >> 4;
  if constexpr (!TR) {
    return *reinterpret_cast<const typename T::frag *>(tile + (x0 + i) * kU + 8 * (g ^ (i >> 1 & 3)));
  } else {
    union { s16x4 h[2]; typename T::frag f; } u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 8 * g + 4 * h + (i >> 2);
      const int piece = ((x0 >> 3) + ((i & 3) >> 1)) ^ tr_swizzle<BX>(k);
      const uint16_t *a = tile + k * BX + 8 * piece + 4 * (i & 1);
      u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(a));
    }
    return u.f;
  }
}

// The lane number, as a value the compiler does not carry addresses made of it along
// for (they would take the registers of the accumulators).
__device__ __forceinline__ int fresh(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// Zeros behind contraction element kv of a stage's rows (TR false), in the piece that
// holds it: those behind that piece were loaded as zeros.
template <int THREADS>
__device__ __forceinline__ void zero_tail(uint16_t *tile, int rows, int kv) {
  for (int r = fresh(threadIdx.x); r < rows; r += THREADS) {
    uint16_t *q = tile + r * kU + 8 * ((kv >> 3) ^ (r >> 1 & 3));
    for (int e = kv & 7; e < 8; ++e) q[e] = 0;
  }
}

// The rows [lo, hi) of expert e, within the R there are whatever the offsets hold.
// (Read as constants: by the scalar unit, beside the counted vector loads.)  ALL: one expert has
// all rows, without offsets.
template <bool ALL>
__device__ __forceinline__ void expert_rows(const GroupedParams &p, int e, int &lo, int &hi) {
  if constexpr (ALL) {
    lo = 0;
    hi = (int)p.R;
    return;
  }
  const auto *off = (const __attribute__((address_space(4))) int *)(uintptr_t)p.off;
  const int R = (int)p.R, l = off[e], h = off[e + 1];
  lo = l < 0 ? 0 : l > R ? R : l;
  hi = h < lo ? lo : h > R ? R : h;
}

template <class V>
__device__ __forceinline__ V uniform(V v) {
  static_assert(sizeof(V) == 4, "one register");
  return __builtin_bit_cast(V, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// One output tile of expert e: columns [n0, n0 + 64 w) and, NT and NN, the sorted rows
// [lo, hi); TN: rows of C from row0, summed over the sorted rows [lo, hi).
struct Tile {
  int e, lo, hi, row0, n0, w;
};
constexpr int kNoTile = -1;  // its e: there is none

// A workgroup's tiles.  Each expert's output is cut into tiles (NT, NN: of up to BM rows,
// as even as they come in units of 64; BN columns), those of up to 8 row tiles for a column
// tile in turn.  Each XCD takes a run of all tiles, equal by what they cost, and deals it
// out to its workgroups in turn: those that share rows or weights run at one time.  What is
// left for less than half of a last round is cut into tiles of fewer columns, one for each
// workgroup.
//   cost of a tile: NT, NN: its height h in units of 64 rows, and 1 (the products, and the
//   weights' columns that it reads); TN: its stages, and kTileCost (its own store)
// The tiles of a run are looked up 32 at a time, one a lane, and kept in LDS: their numbers
// by expert, summed up (every wave writes the same values), and the next 64 of them.
constexpr int kTileCost = 8;

template <int LAYOUT, int BM, int BN, bool ALL>
struct Tiles {
  static constexpr bool TN = LAYOUT == DGF_LAYOUT_TN;
  static constexpr int HM = BM / 64, CW = BN / 64;
  const GroupedParams &p;
  int *next;   // LDS: 64 tiles of 4 values
  int *sums;   // LDS: [E + 1] tiles of the experts before
  int first, count, place, step;  // the XCD's run; this workgroup's place among the `step` that share it

  static constexpr int bytes(int E) { return 64 * 16 + (E + 4) / 4 * 16; }

  __device__ __forceinline__ int tiles_of(int rows) const {
    return (TN ? p.tiles_m : ((rows + 63) / 64 + HM - 1) / HM) * p.tiles_n;
  }
  __device__ __forceinline__ int64_t cost_of(int rows) const {
    if (TN) return ((int64_t)(rows + 2 * kU - 1) / (2 * kU) * 2 + kTileCost) * p.tiles_m * p.tiles_n;
    const int u = (rows + 63) / 64;
    return (int64_t)(u + (u + HM - 1) / HM) * p.tiles_n;
  }
  template <class V>
  static __device__ __forceinline__ V wave_scan(V v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const V o = __shfl_up(v, d);
      if (lane >= d) v += o;
    }
    return v;
  }
  // Sums up the tiles and finds the XCD's run: from the first tile that begins at its share of
  // the cost or later (within an expert, all cost the same).
  __device__ __forceinline__ void start(int b, int n, int lane) {
    int64_t all = 0;
    int tiles = 0;
    if (lane == 0) sums[0] = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      int l = 0, h = 0;
      if (e0 + lane < p.E) expert_rows<ALL>(p, e0 + lane, l, h);
      const bool in = e0 + lane < p.E;
      all += __shfl(wave_scan(in ? cost_of(h - l) : 0, lane), 63);
      const int t = wave_scan(in ? tiles_of(h - l) : 0, lane) + tiles;
      if (in) sums[e0 + lane + 1] = t;
      tiles = __shfl(t, 63);
    }
    all = uniform64(all);
    const int xcd = b & 7;
    const int64_t from = uniform64(all * xcd / 8), to = uniform64(all * (xcd + 1) / 8);
    int begin = tiles, end = tiles;
    bool open = true;
    int64_t base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      int l = 0, h = 0;
      if (e0 + lane < p.E) expert_rows<ALL>(p, e0 + lane, l, h);
      const int64_t cost = e0 + lane < p.E ? cost_of(h - l) : 0, sum = wave_scan(cost, lane) + base;
      const uint64_t a = __ballot(sum > from), z = __ballot(sum > to);
      const int t = tiles_of(h - l);
      if (open && a) {
        const int x = __builtin_ctzll(a);
        const int64_t c = __shfl(cost, x);
        begin = sums[e0 + x] + (int)(((from - (__shfl(sum, x) - c)) * __shfl(t, x) + c - 1) / c);
        open = false;
      }
      if (z) {
        const int x = __builtin_ctzll(z);
        const int64_t c = __shfl(cost, x);
        end = sums[e0 + x] + (int)(((to - (__shfl(sum, x) - c)) * __shfl(t, x) + c - 1) / c);
        break;
      }
      base = __shfl(sum, 63);
    }
    first = uniform(begin);
    count = uniform(end - begin);
    place = b >> 3;
    step = n >> 3;
  }
  // Tiles i0 .. i0 + 31 of this workgroup, into their half of `next`.
  __device__ __forceinline__ void fill(int i0, int lane) const {
    if (lane >= 32) return;
    const int i = i0 + lane, rounds = count / step, rest = count % step;
    // The last round: its tiles are cut in `split`, if that still leaves one for each.
    const int split = CW >= 4 && rest * 4 <= step ? 4 : CW >= 2 && rest * 2 <= step ? 2 : 1;
    int w = CW, part = 0, at = i * step + place;
    if (i >= rounds) {
      at = rounds * step + place / split;
      w = CW / split;
      part = place % split;
    }
    int4 v = make_int4(kNoTile, 0, 0, 0);
    if (i < rounds || (i == rounds && place < rest * split)) {
      at += first;
      int e = 0, past = p.E;  // the last expert whose tiles start at or before it
      while (past - e > 1) {
        const int mid = (e + past) / 2;
        if (sums[mid] <= at) e = mid;
        else past = mid;
      }
      int lo, hi;
      expert_rows<ALL>(p, e, lo, hi);
      const int units = (hi - lo + 63) / 64, rows = TN ? p.tiles_m : (units + HM - 1) / HM;
      const int c = at - sums[e];
      // (offsets that are not ascending can make the sums wrap: no tile then)
      if ((uint32_t)c < (uint32_t)tiles_of(hi - lo)) {
        const int group = c / (8 * p.tiles_n) * 8, of = rows - group < 8 ? rows - group : 8, in = c - group * p.tiles_n;
        const int column = in / of, row = group + in % of;
        if constexpr (!TN) {
          const int even = units / rows, more = units % rows, h = 64 * (even + (row < more));
          lo += 64 * (row * even + (row < more ? row : more));
          hi = hi - lo < h ? hi : lo + h;
        }
        // a part behind the last column is of width 0: nothing to do
        v = make_int4(e | (column * BN + part * w * 64 < p.N ? w : 0) << 10 | part << 13 | column << 15, lo, hi, row);
      }
    }
    reinterpret_cast<int4 *>(next)[i & 63] = v;
  }
  __device__ __forceinline__ Tile get(int i) const {
    const int4 v = reinterpret_cast<const int4 *>(next)[i & 63];
    const int x = uniform(v.x), w = x >> 10 & 7;
    return Tile{x < 0 ? kNoTile : x & 1023, uniform(v.y), uniform(v.z), TN ? uniform(v.w) * BM : 0, (x >> 15) * BN + (x >> 13 & 3) * w * 64, w};
  }
};

// A workgroup's tiles as one stream of stages: while a stage is multiplied, the loads of
// the next ones, of this tile or the ones after it, are under way.
// OUT32: the sums are stored as they are, in FP32 (C, of any alignment, is of floats), and one
// expert has all rows.
template <class T, int LAYOUT, int WN, int FMAX, int FNMAX, int NS, bool OUT32>
struct Stream {
  static constexpr bool ATR = LAYOUT == DGF_LAYOUT_TN, BTR = LAYOUT != DGF_LAYOUT_NT;
  static constexpr int WAVES = 2 * WN, BM = 32 * FMAX, BN = 16 * WN * FNMAX, kStage = (BM + BN) * kU * 2;
  static constexpr int kNone = 1 << 30;
  static_assert(NS % 2 == 0, "stages come in pairs");
  typedef Pieces<ATR, BM, WAVES> PA;
  typedef Pieces<BTR, BN, WAVES> PB;
  static constexpr int kLoads = PA::NL + PB::NL;
  static constexpr int kPerRow = 64 / PB::kRow;  // k rows of a 1 KB load (TR)

  const GroupedParams &p;
  char *lds;
  int lane, wave, wm, wn;
  uint32_t lds0;
  // the loader: its tile, what is left of it and the addresses of the next stage's pieces
  Tiles<LAYOUT, BM, BN, OUT32> tiles;
  int ahead, next_number;  // its number in the run (kNoTile: no more), and the one to look at next
  int end;         // TN: its last sorted row, and 1
  int left, term;  // contraction elements left of the term
  int slot;        // place of the next stage to load
  // (TR: of the first, the others a fixed number of k rows further)
  static constexpr int NA = ATR ? 1 : PA::NL, NB = BTR ? 1 : PB::NL;
  const char *pa[NA], *pb[NB];
  int ka[NA], kb[NB];  // first k of the piece (kNone: zeros)
  int idx[PB::NL * kPerRow];  // TN with a row list: the next stage's rows
  int at;          // place of the next stage to enter
  // waits to come that may leave a whole tile's stores (of every wave) under way
  static constexpr int kStores = FMAX * FNMAX / 2;
  int stored;

  __device__ __forceinline__ Stream(const GroupedParams &p_, char *lds_)
      : p(p_), lds(lds_), tiles{p_, reinterpret_cast<int *>(lds_ + NS * kStage), reinterpret_cast<int *>(lds_ + NS * kStage + 64 * 16)} {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    slot = at = 0;
    left = term = stored = 0;
  }
  __device__ __forceinline__ int contraction(const Tile &t) const { return ATR ? t.hi - t.lo : p.K; }
  // Stages of a term, a whole number of pairs (of zeros where there is nothing to sum).
  static __device__ __forceinline__ int stages(int klen) { return klen > 0 ? (klen + 2 * kU - 1) / (2 * kU) * 2 : 2; }

  __device__ __forceinline__ void open(const Tile &lt) {
    const GroupedTerm t = uniform(term) == 0 ? p.t[0] : p.t[1];
    const int lane = fresh(this->lane);
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      if constexpr (!ATR) {
        int64_t r = lt.lo + PA::row(wave, lane, i);
        const bool in = r < lt.hi;
        if (p.rows) r = p.rows[in ? r : lt.lo];
        ka[i] = in && r >= 0 && r < p.T ? PA::k_of(lane) : kNone;
        pa[i] = reinterpret_cast<const char *>(t.A + r * t.lda + PA::k_of(lane));
      } else {
        const int k = PA::k_row(wave, lane, i), c = lt.row0 + PA::col(lane, k);
        ka[i] = c < p.M ? k : kNone;
        pa[i] = reinterpret_cast<const char *>(t.A + (int64_t)(lt.lo + k) * t.lda + c);
      }
    }
    // (rows and columns that are not the tile's are multiplied as zeros and not stored)
    const int end = p.N - lt.n0 < 64 * lt.w ? p.N : lt.n0 + 64 * lt.w;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint16_t *b = t.B + lt.e * t.stride_b;
      if constexpr (!BTR) {
        const int n = lt.n0 + PB::row(wave, lane, i);
        kb[i] = n < end ? PB::k_of(lane) : kNone;
        pb[i] = reinterpret_cast<const char *>(b + (int64_t)n * t.ldb + PB::k_of(lane));
      } else {
        const int k = PB::k_row(wave, lane, i);
        const int c = lt.n0 + PB::col(lane, k);
        kb[i] = c < end ? k : kNone;
        const int64_t row = !ATR ? k : p.rows ? 0 : lt.lo + k;
        pb[i] = reinterpret_cast<const char *>(b + row * t.ldb + c);
      }
    }
  }
  // TN with a row list: the rows of the next stage (scalar loads: they do not hold up
  // the vector loads, and each 1 KB load takes few rows).
  __device__ __forceinline__ void list() {
    if constexpr (ATR) {
      if (!p.rows || left <= 0) return;
      const auto *rows = (const __attribute__((address_space(4))) int *)(uintptr_t)p.rows;
#pragma unroll
      for (int i = 0; i < PB::NL; ++i)
#pragma unroll
        for (int q = 0; q < kPerRow; ++q) {
          const int r = end - left + PB::load(wave, i) * kPerRow + q;
          idx[i * kPerRow + q] = rows[r < end ? r : end - 1];
        }
    }
  }
  __device__ __forceinline__ void next_tile() {
    term = 0;
    left = 0;
    if (uniform(ahead) == kNoTile) return;
    Tile t;
    int n = uniform(next_number);
    do t = tiles.get(n++);
    while (t.e != kNoTile && t.w == 0);  // (the last one at most)
    next_number = n;
    ahead = t.e == kNoTile ? kNoTile : n - 1;
    if (t.e == kNoTile) return;
    end = t.hi;
    left = contraction(t);
    open(t);
  }
  // The loader's state kept in scalar registers, with the branches made of it.
  __device__ __forceinline__ void scalar_state() {
    left = uniform(left);
    term = uniform(term);
    ahead = uniform(ahead);
    next_number = uniform(next_number);
    end = uniform(end);
    slot = uniform(slot);
    at = uniform(at);
    if (ATR) stored = uniform(stored);
  }
  // Load n of the next stage (of none: zeros, so that every wave always counts the same).
  __device__ __forceinline__ void load(int n) {
    const uint32_t dst = lds0 + slot * kStage;
    const char *const zeros = reinterpret_cast<const char *>(kZeros);
#pragma unroll
    for (int i = 0; i < PA::NL; ++i) {
      if (i != n) continue;
      const int j = ATR ? 0 : i;
      const char *q = ATR ? pa[j] + i * PA::kMore * 2 * p.t[0].lda : pa[j];
      if (ka[j] + (ATR ? i * PA::kMore : 0) >= left) q = zeros;
      lds_load(q, dst + PA::load(wave, i) * 1024);
      if (i + 1 == PA::NL || !ATR) pa[j] += ATR ? p.t[0].lda * (2 * kU) : 2 * kU;
    }
#pragma unroll
    for (int i = 0; i < PB::NL; ++i) {
      if (i + PA::NL != n) continue;
      const int j = BTR ? 0 : i;
      const char *q = pb[j];
      if (ATR && p.rows) {
        int r = idx[i * kPerRow];
#pragma unroll
        for (int z = 1; z < kPerRow; ++z) r = lane >= z * PB::kRow ? idx[i * kPerRow + z] : r;
        q = (uint32_t)r < (uint32_t)p.T ? q + (int64_t)r * p.t[0].ldb * 2 : zeros;
      } else {
        const int64_t ldb = ATR || uniform(term) == 0 ? p.t[0].ldb : p.t[1].ldb;
        if (BTR) q += i * PB::kMore * 2 * ldb;
        if (i + 1 == PB::NL || !BTR) pb[j] += BTR ? ldb * (2 * kU) : 2 * kU;
      }
      if (kb[j] + (BTR ? i * PB::kMore : 0) >= left) q = zeros;
      lds_load(q, dst + BM * kU * 2 + PB::load(wave, i) * 1024);
    }
    if (n + 1 < kLoads) return;
    slot = uniform(slot + 1 == NS ? 0 : slot + 1);
    left = uniform(left - kU);
    if (left <= 0 && slot % 2 == 0) {  // a term is a whole number of pairs of stages, and so is NS
      if (!ATR && uniform(term) + 1 < p.terms && uniform(ahead) != kNoTile) {
        term = 1;
        left = p.K;
        open(tiles.get(ahead));
      } else {
        next_tile();
      }
      scalar_state();
    }
    list();
  }

  // The next stage has landed in every wave, and every wave has used what it read of
  // the stage before the last, whose place takes the loads that follow.  klen: what the
  // stage holds of its term's contraction (whole, or the odd end).
  __device__ __forceinline__ uint16_t *enter(int klen) {
    // Stores count with the loads, in order: those of the last tile, issued after the
    // loads of the NS - 2 stages that follow it, need not be done for these to be there.
    // (TN only, whose tiles are short and whose outputs are large: 32768 rows over 128 experts,
    // 768 x 2048, then with 8-byte stores: 240 us, 254 when every store was waited for.)
    if (ATR && stored > 0) {
      stage_wait<(NS - 3) * kLoads + kStores>();
      stored = uniform(stored - 1);
    } else {
      stage_wait<(NS - 3) * kLoads>();
    }
    uint16_t *st = reinterpret_cast<uint16_t *>(lds + at * kStage);
    at = uniform(at + 1 == NS ? 0 : at + 1);
    if (!(ATR && BTR) && (klen & 7) && klen > 0 && klen < kU) {
      if (!ATR) zero_tail<64 * WAVES>(st, BM, klen);
      if (!BTR) zero_tail<64 * WAVES>(st + BM * kU, BN, klen);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    return st;
  }

  template <int FM, int FN>
  __device__ __forceinline__ void store32(const Tile &t, const f32x4 (&acc)[FM][FN]) {
    const int lane = fresh(this->lane), r0 = t.lo + wm * FM * 16 + (lane & 15), c0 = t.n0 + wn * FN * 16 + 4 * (lane >> 4);
    float *o = reinterpret_cast<float *>(p.C) + (int64_t)r0 * p.ldc + c0;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      if (r0 + 16 * m < t.hi) {
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if (c0 + 16 * n + z < p.N) o[16 * n + z] = acc[m][n][z];
      }
      o += 16 * p.ldc;
    }
  }

  // Multiplies out tile number n of the run, of 32 FM rows (or fewer) x 64 FN columns, with
  // contraction klen, and stores it.
  template <int FM, int FN>
  __device__ __forceinline__ void run(int number, int klen) {
    constexpr int D = FM < 4 ? FM : 4;  // fragments of A held
    const int lane = fresh(this->lane);
    f32x4 acc[FM][FN];
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    typename T::frag a[D], b[2][FN];
    const uint16_t *sa, *sb;
    auto read_a = [&](int m) { return frag_at<T, ATR, BM>(sa, (wm * FM + m) * 16, lane); };
    auto read_b = [&](int n) { return frag_at<T, BTR, BN>(sb, (wn * FN + n) * 16, lane); };
    const int total = stages(klen) * p.terms;
    {
      sa = enter(klen);
      sb = sa + BM * kU;
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(n);
#pragma unroll
      for (int n = 0; n < FN; ++n) b[0][n] = read_b(n);
#pragma unroll
      for (int m = 0; m < D; ++m) a[m] = read_a(m);
      int kleft = klen;  // of the stage being multiplied and what follows it in its term
      for (int j = 0; j < total; j += 2) {
        const bool more = j + 2 < total;
#pragma unroll
        for (int g = 0; g < 2 * FM; ++g) {
          const int kk = g / FM, m = g % FM;
          const bool go = kk == 0 || more;  // the tile has a stage after this one
          if (m == FM - D && go) {
            kleft -= kU;
            if (kk == 1 && kleft <= 0) kleft = klen;
            sa = enter(kleft);
            sb = sa + BM * kU;
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int n = 0; n < FN; ++n) acc[m][n] = T::mfma(b[kk][n], a[g % D], acc[m][n]);
          __builtin_amdgcn_sched_barrier(0);
          if (m + D < FM || go) a[g % D] = read_a((m + D) % FM);
          if (m >= FM - D && go) {
#pragma unroll
            for (int n = 0; n < FN; ++n)
              if (n * D / FN == m - (FM - D)) b[kk ^ 1][n] = read_b(n);
#pragma unroll
            for (int n = 0; n < kLoads; ++n)
              if (n * D / kLoads == m - (FM - D)) load(n);
          }
        }
      }
    }
    // Lane l holds columns 4 (l / 16) .. + 3 of row l % 16 of each 16 x 16 block.  Two blocks
    // side by side trade halves, so that a lane has 8 columns and a store 64 bytes of each
    // row: half the requests (TN, 32768 rows over 128 experts, 768 x 2048: 209 us against
    // 240 with 8-byte stores).
    const Tile t = tiles.get(number);
    if constexpr (OUT32) {
      store32<FM, FN>(t, acc);
      return;
    }
    const int out_lane = fresh(lane), i = out_lane & 15, q4 = out_lane >> 4;
    const int row0 = ATR ? t.row0 : t.lo, rend = ATR ? p.M : t.hi;
    const int r0 = row0 + wm * FM * 16 + i, c0 = t.n0 + wn * FN * 16;
    uint16_t *o = (ATR ? p.C + t.e * p.stride_c : p.C) + (int64_t)r0 * p.ldc + c0;
    const bool whole = ATR && FM == FMAX && FN == FNMAX && row0 + 32 * FM <= rend && t.n0 + 64 * FN <= p.N;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      if (whole || r0 + 16 * m < rend) {
        if constexpr (FN % 2 == 0) {
#pragma unroll
          for (int n = 0; n < FN; n += 2) {
            const uint32_t x[2] = {T::pack(acc[m][n][0], acc[m][n][1]), T::pack(acc[m][n][2], acc[m][n][3])};
            const uint32_t y[2] = {T::pack(acc[m][n + 1][0], acc[m][n + 1][1]), T::pack(acc[m][n + 1][2], acc[m][n + 1][3])};
            const u32x2 lo = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
            const u32x2 hi = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
            const uint4 v = make_uint4(lo.x, hi.x, lo.y, hi.y);
            const int c = n * 16 + 16 * (q4 & 1) + 8 * (q4 >> 1);
            if (whole) *reinterpret_cast<uint4 *>(o + c) = v;
            else if (c0 + c < p.N) row_st(o, c, p.N - c0, v);
          }
        } else {
          const int c = 4 * q4;
          const uint32_t w[2] = {T::pack(acc[m][0][0], acc[m][0][1]), T::pack(acc[m][0][2], acc[m][0][3])};
          if (c0 + c + 4 <= p.N) {
            *reinterpret_cast<uint2 *>(o + c) = make_uint2(w[0], w[1]);
          } else {
            for (int z = 0; c0 + c + z < p.N && z < 4; ++z) o[c + z] = (uint16_t)(w[z >> 1] >> (16 * (z & 1)));
          }
        }
      }
      o += 16 * p.ldc;
    }
    stored = whole ? NS - 2 : 0;
  }

  // The body for a tile of h x w units of 64.
  template <int H, int WC>
  __device__ __forceinline__ bool one_of(int h, int w, int number, int klen) {
    if constexpr (2 * H <= FMAX && WC <= FNMAX) {
      if (uniform(h * 8 + w) == H * 8 + WC) {
        run<2 * H, WC>(number, klen);
        return true;
      }
    }
    return false;
  }
  template <int H>
  __device__ __forceinline__ void of_height(int h, int w, int number, int klen) {
    if (!one_of<H, 4>(h, w, number, klen) && !one_of<H, 2>(h, w, number, klen)) one_of<H, 1>(h, w, number, klen);
  }

  __device__ __forceinline__ void go() {
    tiles.start(blockIdx.x, gridDim.x, lane);
    tiles.fill(0, lane);
    tiles.fill(32, lane);
    ahead = next_number = end = 0;
    next_tile();
    if (ahead == kNoTile) return;  // (the same for every wave: nothing is waited for yet)
    list();
#pragma unroll
    for (int i = 0; i < NS - 2; ++i)
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(n);
    for (int i = 0;; ++i) {
      // The half behind takes the tiles after it.  Waves are at most one tile apart (a barrier
      // a stage) and the loader a few ahead: after 8 tiles none looks at that half any more,
      // and none yet at the next.
      if (i >= 40 && i % 32 == 8) tiles.fill(i + 24, lane);
      const Tile t = tiles.get(i);
      if (t.e == kNoTile) break;
      scalar_state();
      const int h = ATR ? FMAX / 2 : uniform((t.hi - t.lo + 63) / 64), w = t.w, klen = contraction(t);
      if (ATR) of_height<FMAX / 2>(h, w, i, klen);
      else if (h == 4) of_height<4>(h, w, i, klen);
      else if (h == 3) of_height<3>(h, w, i, klen);
      else if (h == 2) of_height<2>(h, w, i, klen);
      else of_height<1>(h, w, i, klen);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // none may land in LDS that is another workgroup's by then
  }
};

template <class T, int LAYOUT, int WN, int FM, int FN, int NS, bool OUT32>
__global__ __launch_bounds__(128 * WN) void k_grouped(GroupedParams p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Stream<T, LAYOUT, WN, FM, FN, NS, OUT32> s(p, lds);
  s.go();
}

template <class T, int LAYOUT, int WN, int FM, int FN, int NS, bool OUT32>
hipError_t grouped_launch(GroupedParams p, int groups, hipStream_t s) {
  constexpr int BM = 32 * FM, BN = 16 * WN * FN;
  p.tiles_m = (p.M + BM - 1) / BM;
  p.tiles_n = (p.N + BN - 1) / BN;
  dgf_launch((k_grouped<T, LAYOUT, WN, FM, FN, NS, OUT32>), dim3(groups), dim3(128 * WN), (size_t)NS * (BM + BN) * kU * 2 + Tiles<LAYOUT, BM, BN, OUT32>::bytes(p.E), s, p);
  return hipGetLastError();
}

// 256 x 256 tiles where they are enough for every CU; else 128 x 128, two workgroups a CU
// (8192^3: 1268 us against 901); 64 x 128 with more stages in flight where an expert has 64
// rows or fewer on average, whose products are bound by reading the weights (128 experts of 64
// rows, 2048 -> 1024: 137 us).
template <class T, int LAYOUT, bool OUT32 = false>
hipError_t grouped_l(const GroupedParams &p, hipStream_t s) {
  const int64_t strips = (p.N + 255) / 256;
  if constexpr (LAYOUT == DGF_LAYOUT_TN) {
    if ((int64_t)((p.M + 255) / 256) * strips * p.E >= 256) return grouped_launch<T, LAYOUT, 4, 8, 4, 4, OUT32>(p, 256, s);
    return grouped_launch<T, LAYOUT, 4, 4, 2, 4, OUT32>(p, 512, s);
  } else {
    if (p.R / p.E <= 64) return grouped_launch<T, LAYOUT, 4, 2, 2, 6, OUT32>(p, 512, s);
    if (p.R / 256 * strips >= 192) return grouped_launch<T, LAYOUT, 4, 8, 4, 4, OUT32>(p, 256, s);
    return grouped_launch<T, LAYOUT, 4, 4, 2, 4, OUT32>(p, 512, s);
  }
}

template <class T>
hipError_t grouped_t(const GroupedParams &p, hipStream_t s) {
  switch (p.layout) {
    case DGF_LAYOUT_NT: return grouped_l<T, DGF_LAYOUT_NT>(p, s);
    case DGF_LAYOUT_NN: return grouped_l<T, DGF_LAYOUT_NN>(p, s);
    default: return grouped_l<T, DGF_LAYOUT_TN>(p, s);
  }
}

}  // namespace

hipError_t launch_router(const GroupedParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? grouped_l<F16, DGF_LAYOUT_NT, true>(p, s) : grouped_l<Bf16, DGF_LAYOUT_NT, true>(p, s);
}

hipError_t launch_grouped(const GroupedParams &p, hipStream_t s) {
  return p.fmt == FMT_F16 ? grouped_t<F16>(p, s) : grouped_t<Bf16>(p, s);
}

}  // namespace dgf
