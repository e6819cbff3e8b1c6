// Kernel interfaces of the mixture of experts over many tokens (internal; the
// public ABI is include/dgf.h): products grouped by expert, the routing of
// tokens, the weighted sum of the experts' outputs, and dropout.
#pragma once

#include "dgf_kernels.hpp"

namespace dgf {

constexpr int kExpertsMaxE = 1024, kExpertsMaxK = 16;

// Products grouped by expert (dgf_grouped.hip).  Rows [off[e], off[e+1]) of the
// R sorted rows belong to expert e.  NT, NN: C[r] = sum over the terms of
// A[rows[r]] B_e; TN: C_e = sum over e's rows of A[r]^T B[rows[r]].
struct GroupedTerm {
  const uint16_t *A, *B;
  int64_t lda, ldb, stride_b;  // stride_b: elements from one expert's matrix to the next
};
struct GroupedParams {
  GroupedTerm t[2];
  int terms;            // 2: NN and NT only
  const int *rows;      // [R] or null: r itself
  int64_t T;            // rows of the operand that `rows` points into (R without it)
  const int *off;       // [E + 1]; not read by launch_router
  uint16_t *C;
  int64_t ldc, stride_c;
  int64_t R;
  int M, N, K, E;       // TN: M x N outputs an expert; NT, NN: N columns, K the contraction
  int layout, fmt;
  int tiles_m, tiles_n;  // of one expert's matrix (NT, NN: columns only), set by the launch
};
hipError_t launch_grouped(const GroupedParams &p, hipStream_t s);
// One NT product of all rows (no offsets, one expert) whose sums are stored in FP32: C and ldc are of floats.
hipError_t launch_router(const GroupedParams &p, hipStream_t s);

// Routing (dgf_route.hip): each token's k largest logits, their weights, and
// the (token, choice) pairs sorted by expert.
struct RouteParams {
  const void *logits;   // [M, E] of type lt (the public dtype codes)
  int64_t ld;
  int lt;
  int *ids;             // [M, k] chosen experts, -1: none left
  float *probs;         // [M, k]
  int *off;             // [E + 1]
  int *rows;            // [M k] token of each sorted row, -1 behind the last
  int *pos;             // [M, k] sorted row of each pair, -1: none
  int64_t M;
  int E, k, renorm;
  uint16_t *counts;     // [blocks][E] workspace
  int blocks;
  // backward
  const float *dprobs;
  void *dlogits;
  int64_t ld_d;
};
int route_blocks(int64_t M);
int64_t route_once();  // tokens that one workgroup both chooses for and orders
hipError_t launch_route_choose(const RouteParams &p, hipStream_t s);
hipError_t launch_route_place(const RouteParams &p, hipStream_t s);
hipError_t launch_route_one(const RouteParams &p, hipStream_t s);
hipError_t launch_route_bwd(const RouteParams &p, hipStream_t s);

struct CombineParams {
  const uint16_t *o;    // [R, H] the experts' outputs, sorted rows
  int64_t ld_o, R;
  const int *pos;       // [M, k]
  const float *probs;   // [M, k] or null: 1
  uint16_t *y;          // [M, H]; backward: dy (read)
  int64_t ld_y;
  uint16_t *d_o;        // backward: [R, H]
  int64_t ld_do;
  float *dprobs;        // backward: [M, k] or null
  int64_t M;
  int H, k, fmt;
};
hipError_t launch_combine(const CombineParams &p, hipStream_t s);
hipError_t launch_combine_bwd(const CombineParams &p, hipStream_t s);

// Dropout (dgf_dropout.hip): z = alpha res + x keep / (1 - cut / 65536).
struct DropoutParams {
  const uint16_t *x, *res;  // res may be null
  uint16_t *z;
  int64_t ld_x, ld_res, ld_z;
  const int64_t *rng;       // {seed, step} in device memory
  uint32_t cut;             // a draw of 16 bits below it drops the value
  float scale, alpha;
  int64_t M, H;
  int fmt;
};
hipError_t launch_dropout(const DropoutParams &p, hipStream_t s);

// 4-bit weights (dgf_w4.hip): codes [ceil(N/16)][ceil(K/128)][64 lanes][16 bytes],
// scales [ceil(N/16)][ceil(K/128)][16][128/group].
struct W4Mat {
  const uint8_t *q;
  const uint16_t *s;
};
struct W4Params {
  const uint16_t *x;    // [M, K] stored type; the down product: the activations of launch_w4_gate_up
  int64_t ldx;
  W4Mat w[2];           // one weight, or gate and up
  uint16_t *y;          // [M, N]; gate/up: the activations, w4_act_bytes(M, N)
  int64_t ldy;
  int64_t M;
  int N, K, group, fmt;
};
// Bytes of the activations between the FFN's two kernels.
size_t w4_act_bytes(int64_t M, int I);
hipError_t launch_pack4(const uint16_t *w, int64_t ldw, uint8_t *q, uint16_t *s, int N, int K, int group, int fmt, hipStream_t st);
hipError_t launch_unpack4(W4Mat m, uint16_t *w, int64_t ldw, int N, int K, int group, int fmt, hipStream_t st);
hipError_t launch_w4(const W4Params &p, hipStream_t s);          // y = x w^T
hipError_t launch_w4_gate_up(const W4Params &p, hipStream_t s);  // a = silu(x w0^T) (x w1^T)
hipError_t launch_w4_down(const W4Params &p, hipStream_t s);     // y = a w^T

}  // namespace dgf
