// C ABI of the operators around the FFN: the norms before and after a block,
// the 8-bit activation checkpoints and the mixture of experts (declarations in include/dgf.h).
#include "dgf_block.hpp"
#include "dgf_host.hpp"
#include "dgf_q8.hpp"

using namespace dgf;

namespace {

dgf_status check_vec(const char *name, const void *p, bool wanted) {
  if (wanted && !p) return fail(DGF_EINVAL, "%s is NULL", name);
  if (!aligned16(p)) return fail(DGF_EINVAL, "%s is not 16-byte aligned", name);
  return DGF_OK;
}

// Rows and columns of the norm operators, and of the parts that go together.
dgf_status check_norm(const void *y, const void *w_post, const void *gate, int64_t ld_gate, float alpha, int64_t M,
                      int64_t H) {
  DGF_TRY(check_dims(M, H, 0));
  if (H == 0) return fail(DGF_EINVAL, "H must be positive");
  if (H > kNormMaxH) return fail(DGF_EUNSUPPORTED, "H=%lld beyond the norm kernels' limit (<= %lld)", (long long)H, (long long)kNormMaxH);
  if (!(alpha - alpha == 0.0f)) return fail(DGF_EINVAL, "alpha is not finite");
  if (M > 0 && !y && (w_post || gate || alpha != 1.0f)) return fail(DGF_EINVAL, "w_post, gate and alpha need a block output y");
  DGF_TRY(check_vec("w_post", w_post, false));
  if (gate && ld_gate != 0 && M > 0) DGF_TRY(check_mat("gate", gate, ld_gate, M, H));
  return check_vec("gate", gate, false);
}

// Workspace of the mixture of experts, laid out from ws (null: size only).
size_t carve_moe(MoeParams &p, void *ws) {
  Carve cv{(char *)ws, 0};
  const size_t pairs = (size_t)p.M * p.k;
  const size_t slots = pairs < (size_t)p.El ? pairs : (size_t)p.El;
  p.lda = moe_down_ld(p.I, p.k);
  p.logits = (float *)cv.take((size_t)p.M * p.E * 2);
  p.p = (float *)cv.take(pairs * 2);
  p.ids = (int *)cv.take(pairs * 2);
  p.slots = (int *)cv.take((1 + 3 * slots) * 2);
  p.pairs = (int *)cv.take(pairs * 2);
  p.a = cv.take(pairs * p.lda * 2);
  moe_plan(p);
  p.prod = p.split > 1 ? (float *)cv.take(pairs * p.H * 2) : nullptr;
  return cv.used;
}

dgf_status check_moe(int64_t M, int64_t H, int64_t I, int64_t E, int64_t e0, int64_t El, int64_t k) {
  DGF_TRY(check_dims(M, H, I));
  if (H == 0 || I == 0 || E <= 0) return fail(DGF_EINVAL, "H, I and E must be positive (H=%lld I=%lld E=%lld)", (long long)H, (long long)I, (long long)E);
  if (k < 1 || k > E) return fail(DGF_EINVAL, "k=%lld experts a token: need 1 to E=%lld", (long long)k, (long long)E);
  if (e0 < 0 || El < 1 || El > E || e0 > E - El)
    return fail(DGF_EINVAL, "experts [%lld, %lld + %lld) are not within the %lld of the router", (long long)e0, (long long)e0, (long long)El, (long long)E);
  if (M > kMoeMaxM || k > kMoeMaxK || E > kMoeMaxE || I > kMoeMaxI)
    return fail(DGF_EUNSUPPORTED, "mixture of experts for a few tokens: M <= %d, k <= %d, E <= %d, I <= %d (M=%lld k=%lld E=%lld I=%lld)",
                kMoeMaxM, kMoeMaxK, kMoeMaxE, kMoeMaxI, (long long)M, (long long)k, (long long)E, (long long)I);
  return DGF_OK;
}

// The experts' matrices, `stride` elements apart.
dgf_status check_experts(const char *name, const void *w, int64_t ld, int64_t stride, int64_t El, int64_t rows,
                         int64_t cols) {
  DGF_TRY(check_mat(name, w, ld, rows, cols));
  if (El > 1 && (stride < (rows - 1) * ld + cols || stride % 8 != 0))
    return fail(DGF_EINVAL, "%s: expert stride %lld: need a multiple of 8 past the %lld rows", name, (long long)stride, (long long)rows);
  return DGF_OK;
}

}  // namespace

extern "C" {

dgf_status dgf_norm_fwd(const void *res, int64_t ld_res, const void *y, int64_t ld_y, const void *w_post,
                        const void *gate, int64_t ld_gate, float alpha, const void *w_next, float eps, void *z,
                        int64_t ld_z, void *h, int64_t ld_h, float *rstd, int64_t M, int64_t H, int dtype,
                        void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_norm(y, w_post, gate, ld_gate, alpha, M, H));
  if (!(eps > 0.0f) || !(eps - eps == 0.0f)) return fail(DGF_EINVAL, "eps must be positive and finite");
  if (M == 0) return ok();
  if (!y && !w_next) return fail(DGF_EINVAL, "nothing to compute: neither y nor w_next is given");
  if ((w_next == nullptr) != (h == nullptr)) return fail(DGF_EINVAL, "w_next and h must both be given or both be NULL");
  DGF_TRY(check_mat("res", res, ld_res, M, H));
  if (y) {
    DGF_TRY(check_mat("y", y, ld_y, M, H));
    DGF_TRY(check_mat("z", z, ld_z, M, H));
  }
  if (h) {
    DGF_TRY(check_mat("h", h, ld_h, M, H));
    DGF_TRY(check_vec("w_next", w_next, true));
  }
  if ((uintptr_t)rstd & 3) return fail(DGF_EINVAL, "rstd is not 4-byte aligned");
  NormFwdParams p{};
  p.res = (const uint16_t *)res; p.ld_res = ld_res;
  p.y = (const uint16_t *)y; p.ld_y = ld_y;
  p.w_post = (const uint16_t *)w_post;
  p.gate = (const uint16_t *)gate; p.ld_gate = ld_gate;
  p.w_next = (const uint16_t *)w_next;
  p.z = (uint16_t *)z; p.ld_z = ld_z;
  p.h = (uint16_t *)h; p.ld_h = ld_h;
  p.rstd = rstd; p.alpha = alpha; p.eps = eps;
  p.M = M; p.H = H; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "norm forward", [&] { return launch_norm_fwd(p, s); }), "norm forward"));
  return ok();
}

size_t dgf_norm_bwd_workspace(int64_t M, int64_t H) {
  if (M <= 0 || H <= 0 || H > kNormMaxH) return 0;
  return (size_t)3 * norm_bwd_groups(M, H) * round8(H) * 4;
}

dgf_status dgf_norm_bwd(const void *dz, int64_t ld_dz, const void *dh, int64_t ld_dh, const void *z, int64_t ld_z,
                        const void *y, int64_t ld_y, const void *w_post, const void *gate, int64_t ld_gate,
                        float alpha, const void *w_next, const float *rstd, void *dres, int64_t ld_dres, void *dy,
                        int64_t ld_dy, void *dw_post, void *dgate, int64_t ld_dgate, void *dw_next, int64_t M,
                        int64_t H, void *ws, size_t ws_bytes, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_norm(y, w_post, gate, ld_gate, alpha, M, H));
  if ((w_next == nullptr) != (dh == nullptr) && M > 0)
    return fail(DGF_EINVAL, "dh and w_next must both be given or both be NULL");
  if (!dz && !dh && M > 0) return fail(DGF_EINVAL, "no gradient comes in: dz and dh are both NULL");
  if (dw_next && !w_next) return fail(DGF_EINVAL, "dw_next without w_next");
  if (dw_post && !w_post) return fail(DGF_EINVAL, "dw_post without w_post");
  if (dgate && !gate) return fail(DGF_EINVAL, "dgate without gate");
  DGF_TRY(check_vec("w_next", w_next, false));
  if (((uintptr_t)dw_post | (uintptr_t)dw_next) & 1) return fail(DGF_EINVAL, "dw_post and dw_next must be 2-byte aligned");
  const bool full_gate = gate && ld_gate != 0;
  if (dgate && !full_gate && ((uintptr_t)dgate & 1)) return fail(DGF_EINVAL, "dgate must be 2-byte aligned");
  NormBwdParams p{};
  p.dw_post = (uint16_t *)dw_post; p.dw_next = (uint16_t *)dw_next;
  p.dgate = (uint16_t *)dgate; p.ld_dgate = ld_dgate; p.ld_gate = ld_gate;
  p.M = M; p.H = H; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  const bool sums = dw_post || dw_next || (dgate && !full_gate);
  if (M > 0) {
    if (dz) DGF_TRY(check_mat("dz", dz, ld_dz, M, H));
    if (dh) {
      DGF_TRY(check_mat("dh", dh, ld_dh, M, H));
      DGF_TRY(check_mat("z", z, ld_z, M, H));
    }
    if (y) {
      DGF_TRY(check_mat("y", y, ld_y, M, H));
      DGF_TRY(check_mat("dy", dy, ld_dy, M, H));
    }
    DGF_TRY(check_mat("dres", dres, ld_dres, M, H));
    if (dgate && full_gate) DGF_TRY(check_mat("dgate", dgate, ld_dgate, M, H));
    if (!rstd || ((uintptr_t)rstd & 3)) return fail(DGF_EINVAL, "rstd is NULL or not 4-byte aligned");
    const size_t need = dgf_norm_bwd_workspace(M, H);
    if (!ws || ws_bytes < need || !aligned16(ws))
      return fail(DGF_EWORKSPACE, "norm backward workspace: need %zu bytes (16-byte aligned), got %zu", need, ws ? ws_bytes : 0);
    p.dz = (const uint16_t *)dz; p.ld_dz = ld_dz;
    p.dh = (const uint16_t *)dh; p.ld_dh = ld_dh;
    p.z = (const uint16_t *)z; p.ld_z = ld_z;
    p.y = (const uint16_t *)y; p.ld_y = ld_y;
    p.w_post = (const uint16_t *)w_post; p.gate = (const uint16_t *)gate; p.w_next = (const uint16_t *)w_next;
    p.rstd = rstd; p.alpha = alpha;
    p.dres = (uint16_t *)dres; p.ld_dres = ld_dres;
    p.dy = (uint16_t *)dy; p.ld_dy = ld_dy;
    p.part = (float *)ws;
    p.groups = norm_bwd_groups(M, H);
    DGF_TRY(hip_check(timed(s, "norm backward", [&] { return launch_norm_bwd(p, s); }), "norm backward"));
  }
  // no rows: each column sum is the empty sum, +0
  if (sums)
    DGF_TRY(hip_check(timed(s, "norm weight gradients", [&] { return launch_norm_wgrad(p, s); }), "norm weight gradients"));
  return ok();
}

dgf_status dgf_pack8(const void *x, int64_t ldx, void *q, int64_t ld_q, float *scales, int64_t ld_s, int64_t M,
                     int64_t N, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_dims(M, N, 0));
  if (M == 0 || N == 0) return ok();
  const Q8Mat o{(uint8_t *)q, scales, ld_q, ld_s};
  DGF_TRY(check_mat("x", x, ldx, M, N));
  DGF_TRY(check_q8("q", o, M, N));
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "pack8", [&] { return launch_pack8(fmt, (const uint16_t *)x, ldx, o, M, N, s); }), "pack8"));
  return ok();
}

dgf_status dgf_unpack8(const void *q, int64_t ld_q, const float *scales, int64_t ld_s, void *x, int64_t ldx, int64_t M,
                       int64_t N, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_dims(M, N, 0));
  if (M == 0 || N == 0) return ok();
  const Q8Mat t{(uint8_t *)q, (float *)scales, ld_q, ld_s};
  DGF_TRY(check_q8("q", t, M, N));
  DGF_TRY(check_mat("x", x, ldx, M, N));
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "unpack8", [&] { return launch_unpack8(fmt, t, (uint16_t *)x, ldx, M, N, s); }), "unpack8"));
  return ok();
}

dgf_status dgf_act_bwd_q8(const void *da, int64_t ldda, const void *g_q, const float *g_s, const void *u_q,
                          const float *u_s, int64_t ld_q, int64_t ld_s, void *dg, void *du, void *a, int64_t ld_out,
                          int64_t M, int64_t N, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_dims(M, N, 0));
  if (M == 0 || N == 0) return ok();
  ActQ8Params p{};
  p.g = Q8Mat{(uint8_t *)g_q, (float *)g_s, ld_q, ld_s};
  p.u = Q8Mat{(uint8_t *)u_q, (float *)u_s, ld_q, ld_s};
  DGF_TRY(check_mat("da", da, ldda, M, N));
  DGF_TRY(check_q8("g", p.g, M, N));
  DGF_TRY(check_q8("u", p.u, M, N));
  DGF_TRY(check_mat("dg", dg, ld_out, M, N));
  DGF_TRY(check_mat("du", du, ld_out, M, N));
  if (a) DGF_TRY(check_mat("a", a, ld_out, M, N));
  p.da = (const uint16_t *)da; p.ldda = ldda;
  p.dg = (uint16_t *)dg; p.du = (uint16_t *)du; p.a = (uint16_t *)a;
  p.ldo = ld_out; p.M = M; p.N = N;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "act_bwd_q8", [&] { return launch_act_bwd_q8(fmt, p, s); }), "act_bwd_q8"));
  return ok();
}

size_t dgf_moe_fwd_workspace(int64_t M, int64_t H, int64_t I, int64_t E, int64_t El, int64_t k) {
  if (M <= 0 || H <= 0 || I <= 0 || E <= 0 || El <= 0 || k <= 0 || M > kMoeMaxM || E > kMoeMaxE || k > kMoeMaxK ||
      El > E || I > kMoeMaxI)
    return 0;
  MoeParams p{};
  p.M = (int)M; p.H = (int)H; p.I = (int)I; p.E = (int)E; p.El = (int)El; p.k = (int)k;
  return carve_moe(p, nullptr);
}

dgf_status dgf_moe_fwd(const void *x, int64_t ldx, const void *w_router, int64_t ld_wr, const void *w_gate,
                       int64_t ld_wg, int64_t stride_wg, const void *w_up, int64_t ld_wu, int64_t stride_wu,
                       const void *w_down, int64_t ld_wd, int64_t stride_wd, void *y, int64_t ldy, int32_t *ids,
                       float *probs, int64_t M, int64_t H, int64_t I, int64_t E, int64_t e0, int64_t El, int64_t k,
                       int renorm, void *ws, size_t ws_bytes, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_moe(M, H, I, E, e0, El, k));
  if (M == 0) return ok();
  DGF_TRY(check_mat("x", x, ldx, M, H));
  DGF_TRY(check_mat("w_router", w_router, ld_wr, E, H));
  DGF_TRY(check_experts("w_gate", w_gate, ld_wg, stride_wg, El, I, H));
  DGF_TRY(check_experts("w_up", w_up, ld_wu, stride_wu, El, I, H));
  DGF_TRY(check_experts("w_down", w_down, ld_wd, stride_wd, El, H, I));
  DGF_TRY(check_mat("y", y, ldy, M, H));
  if (((uintptr_t)ids | (uintptr_t)probs) & 3) return fail(DGF_EINVAL, "ids and probs must be 4-byte aligned");
  const size_t need = dgf_moe_fwd_workspace(M, H, I, E, El, k);
  if (!ws || ws_bytes < need || !aligned16(ws))
    return fail(DGF_EWORKSPACE, "mixture of experts workspace: need %zu bytes (16-byte aligned), got %zu", need, ws ? ws_bytes : 0);
  MoeParams p{};
  p.x = (const uint16_t *)x; p.ldx = ldx;
  p.w_router = (const uint16_t *)w_router; p.ld_wr = ld_wr;
  p.w_gate = (const uint16_t *)w_gate; p.ld_wg = ld_wg; p.st_wg = stride_wg;
  p.w_up = (const uint16_t *)w_up; p.ld_wu = ld_wu; p.st_wu = stride_wu;
  p.w_down = (const uint16_t *)w_down; p.ld_wd = ld_wd; p.st_wd = stride_wd;
  p.y = (uint16_t *)y; p.ldy = ldy;
  p.ids_out = ids; p.p_out = probs;
  p.M = (int)M; p.H = (int)H; p.I = (int)I; p.E = (int)E; p.e0 = (int)e0; p.El = (int)El; p.k = (int)k;
  p.renorm = renorm != 0; p.fmt = fmt;
  carve_moe(p, ws);
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "moe logits", [&] { return launch_moe_logits(p, s); }), "moe logits"));
  if (!moe_one(p)) DGF_TRY(hip_check(timed(s, "moe route", [&] { return launch_moe_route(p, s); }), "moe route"));
  DGF_TRY(hip_check(timed(s, "moe gate/up", [&] { return launch_moe_gate_up(p, s); }), "moe gate/up"));
  DGF_TRY(hip_check(timed(s, "moe down", [&] { return launch_moe_down(p, s); }), "moe down"));
  if (p.split > 1) DGF_TRY(hip_check(timed(s, "moe combine", [&] { return launch_moe_combine(p, s); }), "moe combine"));
  return ok();
}

}  // extern "C"
