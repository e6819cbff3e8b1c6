// Kernel interfaces of the operators around the FFN (internal; the public ABI
// is include/dgf.h): the norms before and after a block, and the
// mixture-of-experts layer for a few tokens.
#pragma once

#include "dgf_kernels.hpp"

namespace dgf {

// Widest row of the norm kernels: a row lives in the registers of one
// workgroup, 16 elements a thread of 1024.
constexpr int64_t kNormMaxH = 16384;

struct NormFwdParams {
  const uint16_t *res, *y;              // [M, H]; y null: z = res, only h is written
  const uint16_t *w_post, *gate, *w_next;  // [H]; gate [M, H] with ld_gate > 0; any may be null
  int64_t ld_res, ld_y, ld_gate;
  uint16_t *z, *h;                      // [M, H]
  int64_t ld_z, ld_h;
  float *rstd;                          // [M, 2]: post, next; or null
  float alpha, eps;
  int64_t M, H;
  int fmt;
};
hipError_t launch_norm_fwd(const NormFwdParams &p, hipStream_t s);

struct NormBwdParams {
  const uint16_t *dz, *dh, *z, *y;      // [M, H]; dz or dh may be null, y null as in the forward
  const uint16_t *w_post, *gate, *w_next;
  int64_t ld_dz, ld_dh, ld_z, ld_y, ld_gate;
  const float *rstd;                    // [M, 2]
  uint16_t *dres, *dy;                  // [M, H]
  int64_t ld_dres, ld_dy;
  uint16_t *dgate;                      // [M, H] when ld_gate > 0 (ld_dgate), else [H]; or null
  int64_t ld_dgate;
  uint16_t *dw_post, *dw_next;          // [H] or null
  float *part;                          // [3][groups][round8(H)]: dw_post, dw_next, dgate
  int groups;
  float alpha;
  int64_t M, H;
  int fmt;
};
// Workgroups of the backward, each adding up its own rows' part of the column sums.
int norm_bwd_groups(int64_t M, int64_t H);
hipError_t launch_norm_bwd(const NormBwdParams &p, hipStream_t s);
hipError_t launch_norm_wgrad(const NormBwdParams &p, hipStream_t s);

// Mixture of experts (dgf_moe.hip): E experts in all, of which this call holds
// the weights of [e0, e0 + El).  Limits: M tokens, k experts a token, E, I (the
// activations of all pairs, 4 M k I bytes, stay below 2^31).
constexpr int kMoeMaxM = 128, kMoeMaxK = 16, kMoeMaxE = 1024, kMoeMaxI = 1 << 17;
struct MoeParams {
  const uint16_t *x, *w_router;              // [M, H], [E, H]
  const uint16_t *w_gate, *w_up, *w_down;    // [El, I, H], [El, I, H], [El, H, I]
  int64_t ldx, ld_wr, ld_wg, ld_wu, ld_wd;
  int64_t st_wg, st_wu, st_wd;               // elements from one expert to the next
  uint16_t *y;                               // [M, H]
  int64_t ldy;
  int *ids_out;                              // [M, k] or null
  float *p_out;                              // [M, k] or null
  int M, H, I, E, e0, El, k, renorm, fmt;
  // workspace
  float *logits;                             // [M, E]
  float *p;                                  // [M k] routing weights
  int *ids;                                  // [M k] chosen experts
  int *slots;                                // [1 + 3 min(El, M k)]: how many local experts have tokens, then of
                                             // each its index, its first entry in `pairs` and how many it has
  int *pairs;                                // [M k] (token, choice) pairs m k + j by slot, ascending within one
  uint16_t *a;                               // [M k, lda] the experts' activations, 32 bits each (dgf_moe.hip: put_a)
  int64_t lda;
  float *prod;                               // [M k, H] each pair's down product when split > 1, else null
  int row_tiles, split;                      // of the down kernel: 8 rows each per workgroup, workgroups per row tile
};
// Sets row_tiles and split from the sizes.
void moe_plan(MoeParams &p);
// Columns of a row of `a`: I rounded up to whole steps of the down kernel.
int64_t moe_down_ld(int I, int k);
// Whether the gate/up kernel chooses the experts itself (no route launch).
bool moe_one(const MoeParams &p);
hipError_t launch_moe_logits(const MoeParams &p, hipStream_t s);
hipError_t launch_moe_route(const MoeParams &p, hipStream_t s);
hipError_t launch_moe_gate_up(const MoeParams &p, hipStream_t s);
hipError_t launch_moe_down(const MoeParams &p, hipStream_t s);
hipError_t launch_moe_combine(const MoeParams &p, hipStream_t s);

}  // namespace dgf
