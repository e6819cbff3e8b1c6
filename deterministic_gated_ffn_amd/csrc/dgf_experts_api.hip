// C ABI of the mixture of experts over many tokens, dropout and the 4-bit
// weights (declarations in include/dgf.h).
#include <math.h>

#include "dgf_experts.hpp"
#include "dgf_host.hpp"

using namespace dgf;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 21, kMaxRows = (int64_t)1 << 25;
constexpr int64_t kW4MaxM = (int64_t)1 << 16;

dgf_status check_int32(const char *name, const void *p) {
  if (!p) return fail(DGF_EINVAL, "%s is NULL", name);
  if ((uintptr_t)p & 3) return fail(DGF_EINVAL, "%s is not 4-byte aligned", name);
  return DGF_OK;
}

dgf_status check_choices(int64_t M, int64_t E, int64_t k) {
  if (M < 0) return fail(DGF_EINVAL, "negative dimension (M=%lld)", (long long)M);
  if (E < 1 || k < 1 || k > E) return fail(DGF_EINVAL, "k=%lld experts a token of E=%lld: need 1 to E", (long long)k, (long long)E);
  if (M > kMaxTokens || E > kExpertsMaxE || k > kExpertsMaxK)
    return fail(DGF_EUNSUPPORTED, "routing: M <= 2^21, E <= %d, k <= %d (M=%lld E=%lld k=%lld)", kExpertsMaxE, kExpertsMaxK,
                (long long)M, (long long)E, (long long)k);
  return DGF_OK;
}

// Logits or their gradient: any row stride of at least E elements.
dgf_status check_logits(const char *name, const void *p, int64_t ld, int dtype, int64_t M, int64_t E) {
  if (dtype != DGF_BF16 && dtype != DGF_FP16 && dtype != DGF_FP32) return fail(DGF_EINVAL, "unknown dtype %d", dtype);
  if (M == 0) return DGF_OK;
  if (!p) return fail(DGF_EINVAL, "%s is NULL", name);
  if ((uintptr_t)p & (dtype == DGF_FP32 ? 3 : 1)) return fail(DGF_EINVAL, "%s is not aligned to its elements", name);
  if (ld < E) return fail(DGF_EINVAL, "%s: leading dimension %lld < %lld experts", name, (long long)ld, (long long)E);
  return DGF_OK;
}

dgf_status check_combine(const void *o, int64_t ld_o, int64_t R, const int32_t *pos, const float *probs, int64_t M, int64_t H,
                         int64_t k) {
  if (M < 0 || H < 0 || R < 0) return fail(DGF_EINVAL, "negative dimension (M=%lld H=%lld R=%lld)", (long long)M, (long long)H, (long long)R);
  if (k < 1) return fail(DGF_EINVAL, "k=%lld experts a token: need at least 1", (long long)k);
  if (M > kMaxTokens || R > kMaxRows || k > kExpertsMaxK)
    return fail(DGF_EUNSUPPORTED, "combination: M <= 2^21, R <= 2^25, k <= %d (M=%lld R=%lld k=%lld)", kExpertsMaxK,
                (long long)M, (long long)R, (long long)k);
  if (M == 0 || H == 0) return DGF_OK;
  if (o) DGF_TRY(check_mat("o", o, ld_o, R, H));
  DGF_TRY(check_int32("pos", pos));
  if ((uintptr_t)probs & 3) return fail(DGF_EINVAL, "probs is not 4-byte aligned");
  return DGF_OK;
}

dgf_status check_w4_dims(int64_t M, int64_t N, int64_t K, int64_t group) {
  DGF_TRY(check_dims(M, N, K));
  if (group != 32 && group != 64 && group != 128)
    return fail(DGF_EINVAL, "group=%lld: 32, 64 or 128 columns share a scale", (long long)group);
  if (N == 0 || K == 0) return fail(DGF_EINVAL, "a 4-bit matrix needs rows and columns (N=%lld K=%lld)", (long long)N, (long long)K);
  if (M > kW4MaxM || N >= kMaxLd || K >= kMaxLd)
    return fail(DGF_EUNSUPPORTED, "4-bit weights: M <= 65536, N and K below 2^23 (M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
  return DGF_OK;
}

// Packing has a wave for each tile of 16 x 128, one grid for all of them.
dgf_status check_tiles4(int64_t N, int64_t K) {
  if ((N + 15) / 16 * ((K + 127) / 128) > ((int64_t)1 << 26) - 4)
    return fail(DGF_EUNSUPPORTED, "4-bit weights: more than 2^26 tiles of 16 x 128 (N=%lld K=%lld)", (long long)N, (long long)K);
  return DGF_OK;
}

dgf_status check_w4(const char *name, const void *codes, const void *scales) {
  if (!codes || !scales) return fail(DGF_EINVAL, "%s: the %s are NULL", name, codes ? "scales" : "codes");
  if (!aligned16(codes)) return fail(DGF_EINVAL, "%s: the codes are not 16-byte aligned", name);
  if ((uintptr_t)scales & 7) return fail(DGF_EINVAL, "%s: the scales are not 8-byte aligned", name);
  return DGF_OK;
}

W4Mat w4_mat(const void *codes, const void *scales) { return W4Mat{(const uint8_t *)codes, (const uint16_t *)scales}; }

}  // namespace

extern "C" {

dgf_status dgf_gemm_grouped(int layout, const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b,
                            const void *A2, int64_t lda2, const void *B2, int64_t ldb2, int64_t stride_b2,
                            const int32_t *rows, int64_t T, const int32_t *offsets, void *C, int64_t ldc,
                            int64_t stride_c, int64_t M, int64_t N, int64_t K, int64_t E, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  if (layout != DGF_NT && layout != DGF_NN && layout != DGF_TN) return fail(DGF_EINVAL, "unknown layout %d", layout);
  const bool tn = layout == DGF_TN;
  if (M < 0 || N < 0 || K < 0) return fail(DGF_EINVAL, "negative dimension (M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
  if (E < 1) return fail(DGF_EINVAL, "E=%lld experts: need at least 1", (long long)E);
  const int64_t R = tn ? K : M;
  if (E > kExpertsMaxE || R > kMaxRows || N >= kMaxLd || (tn ? M : K) >= kMaxLd)
    return fail(DGF_EUNSUPPORTED, "grouped products: E <= %d, at most 2^25 sorted rows, the other dimensions below 2^23 (E=%lld M=%lld N=%lld K=%lld)",
                kExpertsMaxE, (long long)E, (long long)M, (long long)N, (long long)K);
  // workgroups of the smallest tile
  const int64_t cols = (N + 127) / 128, tiles = tn ? (M + 127) / 128 * cols * E : (R / 64 + (R < E ? R : E)) * cols;
  if (tiles > INT32_MAX) return fail(DGF_EUNSUPPORTED, "grouped products: more than 2^31 output tiles");
  const bool two = A2 || B2;
  // (a matrix without rows or columns may be NULL)
  if (two && (!A2 || !B2) && (tn || (K > 0 && (rows ? T : R) > 0 && N > 0)))
    return fail(DGF_EINVAL, "A2 and B2 must both be given or both be NULL");
  if (tn && two) return fail(DGF_EINVAL, "DGF_TN takes one pair of operands");
  if (rows && T < 0) return fail(DGF_EINVAL, "T=%lld rows to choose from", (long long)T);
  if (rows && T > kMaxRows) return fail(DGF_EUNSUPPORTED, "T=%lld beyond the limit (2^25 rows)", (long long)T);
  if (M == 0 || N == 0) return ok();
  if (rows) DGF_TRY(check_int32("rows", rows));
  DGF_TRY(check_int32("offsets", offsets));
  const int64_t listed = rows ? T : R;
  if (tn) {
    DGF_TRY(check_mat("A", A, lda, R, M));
    DGF_TRY(check_mat("B", B, ldb, R == 0 ? 0 : listed, N));
    DGF_TRY(check_experts("C", C, ldc, stride_c, E, M, N));
  } else {
    const int64_t b_rows = layout == DGF_NT ? N : K, b_cols = layout == DGF_NT ? K : N;
    DGF_TRY(check_mat("A", A, lda, listed, K));
    if (K > 0) DGF_TRY(check_experts("B", B, ldb, stride_b, E, b_rows, b_cols));
    if (two) {
      DGF_TRY(check_mat("A2", A2, lda2, listed, K));
      if (K > 0) DGF_TRY(check_experts("B2", B2, ldb2, stride_b2, E, b_rows, b_cols));
    }
    DGF_TRY(check_mat("C", C, ldc, R, N));
  }
  GroupedParams p{};
  p.t[0] = GroupedTerm{(const uint16_t *)A, (const uint16_t *)B, lda, ldb, stride_b};
  p.t[1] = GroupedTerm{(const uint16_t *)A2, (const uint16_t *)B2, lda2, ldb2, stride_b2};
  p.terms = two ? 2 : 1;
  p.rows = rows;
  p.T = listed;
  p.off = offsets;
  p.C = (uint16_t *)C; p.ldc = ldc; p.stride_c = stride_c;
  p.R = R;
  p.M = tn ? (int)M : 0; p.N = (int)N; p.K = tn ? 0 : (int)K; p.E = (int)E;
  p.layout = layout; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "grouped product", [&] { return launch_grouped(p, s); }), "grouped product"));
  return ok();
}

dgf_status dgf_moe_logits(const void *x, int64_t ldx, const void *w_router, int64_t ld_wr, float *logits, int64_t ld, int64_t M,
                          int64_t H, int64_t E, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  if (M < 0 || H < 0) return fail(DGF_EINVAL, "negative dimension (M=%lld H=%lld)", (long long)M, (long long)H);
  if (E < 1) return fail(DGF_EINVAL, "E=%lld experts: need at least 1", (long long)E);
  if (M > kMaxTokens || E > kExpertsMaxE || H >= kMaxLd)
    return fail(DGF_EUNSUPPORTED, "router: M <= 2^21, E <= %d, H below 2^23 (M=%lld H=%lld E=%lld)", kExpertsMaxE, (long long)M,
                (long long)H, (long long)E);
  if (M == 0) return ok();
  DGF_TRY(check_mat("x", x, ldx, M, H));
  DGF_TRY(check_mat("w_router", w_router, ld_wr, E, H));
  DGF_TRY(check_logits("logits", logits, ld, DGF_FP32, M, E));
  GroupedParams p{};
  p.t[0] = GroupedTerm{(const uint16_t *)x, (const uint16_t *)w_router, ldx, ld_wr, 0};
  p.terms = 1;
  p.T = p.R = M;
  p.C = reinterpret_cast<uint16_t *>(logits); p.ldc = ld;
  p.N = (int)E; p.K = (int)H; p.E = 1;
  p.layout = DGF_NT; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "router", [&] { return launch_router(p, s); }), "router"));
  return ok();
}

size_t dgf_moe_route_workspace(int64_t M, int64_t E, int64_t k) {
  if (M <= route_once() || M > kMaxTokens || E < 1 || E > kExpertsMaxE || k < 1 || k > kExpertsMaxK || k > E) return 0;
  return round256((size_t)route_blocks(M) * E * 2);
}

dgf_status dgf_moe_route(const void *logits, int64_t ld, int32_t *ids, float *probs, int32_t *offsets, int32_t *rows,
                         int32_t *pos, int64_t M, int64_t E, int64_t k, int renorm, void *ws, size_t ws_bytes, int dtype,
                         void *stream) {
  DGF_TRY(check_choices(M, E, k));
  DGF_TRY(check_logits("logits", logits, ld, dtype, M, E));
  DGF_TRY(check_int32("offsets", offsets));
  if (M > 0) {
    DGF_TRY(check_int32("ids", ids));
    DGF_TRY(check_int32("probs", probs));
    DGF_TRY(check_int32("rows", rows));
    DGF_TRY(check_int32("pos", pos));
  }
  const size_t need = dgf_moe_route_workspace(M, E, k);
  if (need && (!ws || ws_bytes < need || !aligned16(ws)))
    return fail(DGF_EWORKSPACE, "routing workspace: need %zu bytes (16-byte aligned), got %zu", need, ws ? ws_bytes : 0);
  RouteParams p{};
  p.logits = logits; p.ld = ld; p.lt = dtype;
  p.ids = ids; p.probs = probs; p.off = offsets; p.rows = rows; p.pos = pos;
  p.M = M; p.E = (int)E; p.k = (int)k; p.renorm = renorm != 0;
  p.counts = (uint16_t *)ws;
  p.blocks = need ? route_blocks(M) : 1;
  hipStream_t s = (hipStream_t)stream;
  if (!need) {
    DGF_TRY(hip_check(timed(s, "routing", [&] { return launch_route_one(p, s); }), "routing"));
    return ok();
  }
  DGF_TRY(hip_check(timed(s, "routing: choice", [&] { return launch_route_choose(p, s); }), "routing: choice"));
  DGF_TRY(hip_check(timed(s, "routing: order", [&] { return launch_route_place(p, s); }), "routing: order"));
  return ok();
}

dgf_status dgf_moe_route_bwd(const float *dprobs, const void *logits, int64_t ld, const int32_t *ids, const float *probs,
                             void *dlogits, int64_t ld_d, int64_t M, int64_t E, int64_t k, int renorm, int dtype,
                             void *stream) {
  DGF_TRY(check_choices(M, E, k));
  if (!renorm) DGF_TRY(check_logits("logits", logits, ld, dtype, M, E));
  DGF_TRY(check_logits("dlogits", dlogits, ld_d, dtype, M, E));
  if (M == 0) return ok();
  DGF_TRY(check_int32("dprobs", dprobs));
  DGF_TRY(check_int32("ids", ids));
  DGF_TRY(check_int32("probs", probs));
  RouteParams p{};
  p.logits = logits; p.ld = ld; p.lt = dtype;
  p.ids = const_cast<int32_t *>(ids); p.probs = const_cast<float *>(probs); p.dprobs = dprobs;
  p.dlogits = dlogits; p.ld_d = ld_d;
  p.M = M; p.E = (int)E; p.k = (int)k; p.renorm = renorm != 0;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "routing backward", [&] { return launch_route_bwd(p, s); }), "routing backward"));
  return ok();
}

dgf_status dgf_moe_combine(const void *o, int64_t ld_o, int64_t R, const int32_t *pos, const float *probs, void *y,
                           int64_t ldy, int64_t M, int64_t H, int64_t k, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_combine(o, ld_o, R, pos, probs, M, H, k));
  if (M == 0 || H == 0) return ok();
  if (!o && R > 0) return fail(DGF_EINVAL, "o is NULL");
  DGF_TRY(check_mat("y", y, ldy, M, H));
  CombineParams p{};
  p.o = (const uint16_t *)o; p.ld_o = ld_o; p.R = R;
  p.pos = pos; p.probs = probs;
  p.y = (uint16_t *)y; p.ld_y = ldy;
  p.M = M; p.H = (int)H; p.k = (int)k; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "combination", [&] { return launch_combine(p, s); }), "combination"));
  return ok();
}

dgf_status dgf_moe_combine_bwd(const void *dy, int64_t lddy, const void *o, int64_t ld_o, int64_t R, const int32_t *pos,
                               const float *probs, void *d_o, int64_t ld_do, float *dprobs, int64_t M, int64_t H,
                               int64_t k, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_combine(dprobs ? o : nullptr, ld_o, R, pos, probs, M, H, k));
  if (dprobs && !probs) return fail(DGF_EINVAL, "dprobs without probs");
  if ((uintptr_t)dprobs & 3) return fail(DGF_EINVAL, "dprobs is not 4-byte aligned");
  if (M == 0 || (H == 0 && !dprobs)) return ok();
  if (H == 0) return fail(DGF_EINVAL, "H must be positive");
  if (dprobs && !o && R > 0) return fail(DGF_EINVAL, "o is NULL");
  DGF_TRY(check_mat("dy", dy, lddy, M, H));
  DGF_TRY(check_mat("d_o", d_o, ld_do, R, H));
  CombineParams p{};
  p.o = (const uint16_t *)o; p.ld_o = ld_o; p.R = R;
  p.pos = pos; p.probs = probs;
  p.y = (uint16_t *)const_cast<void *>(dy); p.ld_y = lddy;
  p.d_o = (uint16_t *)d_o; p.ld_do = ld_do;
  p.dprobs = dprobs;
  p.M = M; p.H = (int)H; p.k = (int)k; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "combination backward", [&] { return launch_combine_bwd(p, s); }), "combination backward"));
  return ok();
}

dgf_status dgf_dropout(const void *x, int64_t ldx, const void *res, int64_t ld_res, float alpha, double p_drop,
                       const int64_t *rng, void *z, int64_t ldz, int64_t M, int64_t H, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_dims(M, H, 0));
  if (H >= kMaxLd) return fail(DGF_EUNSUPPORTED, "H=%lld beyond the limit (< 2^23)", (long long)H);
  const double cut = p_drop >= 0.0 && p_drop <= 1.0 ? rint(p_drop * 65536.0) : 65536.0;
  if (cut > 65535.0) return fail(DGF_EINVAL, "p=%g: a probability from 0 to below 1 - 2^-17", p_drop);
  if (!(alpha - alpha == 0.0f)) return fail(DGF_EINVAL, "alpha is not finite");
  if (M == 0 || H == 0) return ok();
  DGF_TRY(check_mat("x", x, ldx, M, H));
  if (res) DGF_TRY(check_mat("res", res, ld_res, M, H));
  DGF_TRY(check_mat("z", z, ldz, M, H));
  if (!rng || ((uintptr_t)rng & 7)) return fail(DGF_EINVAL, "rng is NULL or not 8-byte aligned");
  DropoutParams p{};
  p.x = (const uint16_t *)x; p.ld_x = ldx;
  p.res = (const uint16_t *)res; p.ld_res = ld_res;
  p.z = (uint16_t *)z; p.ld_z = ldz;
  p.rng = rng;
  p.cut = (uint32_t)cut;
  p.scale = (float)(65536.0 / (65536.0 - cut));
  p.alpha = alpha;
  p.M = M; p.H = H; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "dropout", [&] { return launch_dropout(p, s); }), "dropout"));
  return ok();
}

dgf_status dgf_pack4(const void *w, int64_t ldw, void *codes, void *scales, int64_t N, int64_t K, int64_t group, int dtype,
                     void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_w4_dims(0, N, K, group));
  DGF_TRY(check_tiles4(N, K));
  DGF_TRY(check_mat("w", w, ldw, N, K));
  DGF_TRY(check_w4("w4", codes, scales));
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "pack4", [&] {
    return launch_pack4((const uint16_t *)w, ldw, (uint8_t *)codes, (uint16_t *)scales, (int)N, (int)K, (int)group, fmt, s);
  }), "pack4"));
  return ok();
}

dgf_status dgf_unpack4(const void *codes, const void *scales, void *w, int64_t ldw, int64_t N, int64_t K, int64_t group,
                       int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_w4_dims(0, N, K, group));
  DGF_TRY(check_tiles4(N, K));
  DGF_TRY(check_w4("w4", codes, scales));
  DGF_TRY(check_mat("w", w, ldw, N, K));
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "unpack4", [&] {
    return launch_unpack4(w4_mat(codes, scales), (uint16_t *)w, ldw, (int)N, (int)K, (int)group, fmt, s);
  }), "unpack4"));
  return ok();
}

dgf_status dgf_gemm_w4(const void *x, int64_t ldx, const void *codes, const void *scales, void *y, int64_t ldy, int64_t M,
                       int64_t N, int64_t K, int64_t group, int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_w4_dims(M, N, K, group));
  if (M == 0) return ok();
  DGF_TRY(check_mat("x", x, ldx, M, K));
  DGF_TRY(check_w4("w4", codes, scales));
  DGF_TRY(check_mat("y", y, ldy, M, N));
  W4Params p{};
  p.x = (const uint16_t *)x; p.ldx = ldx;
  p.w[0] = w4_mat(codes, scales);
  p.y = (uint16_t *)y; p.ldy = ldy;
  p.M = M; p.N = (int)N; p.K = (int)K; p.group = (int)group; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "4-bit product", [&] { return launch_w4(p, s); }), "4-bit product"));
  return ok();
}

size_t dgf_ffn_fwd_w4_workspace(int64_t M, int64_t H, int64_t I) {
  if (M <= 0 || H <= 0 || I <= 0 || M > kW4MaxM || H >= kMaxLd || I >= kMaxLd) return 0;
  return w4_act_bytes(M, (int)I);
}

dgf_status dgf_ffn_fwd_w4(const void *x, int64_t ldx, const void *gate_codes, const void *gate_scales,
                          const void *up_codes, const void *up_scales, const void *down_codes, const void *down_scales,
                          void *y, int64_t ldy, int64_t M, int64_t H, int64_t I, int64_t group, void *ws, size_t ws_bytes,
                          int dtype, void *stream) {
  int fmt = 0;
  DGF_TRY(stored_type(dtype, &fmt));
  DGF_TRY(check_w4_dims(M, I, H, group));
  if (M == 0) return ok();
  DGF_TRY(check_mat("x", x, ldx, M, H));
  DGF_TRY(check_w4("gate", gate_codes, gate_scales));
  DGF_TRY(check_w4("up", up_codes, up_scales));
  DGF_TRY(check_w4("down", down_codes, down_scales));
  DGF_TRY(check_mat("y", y, ldy, M, H));
  const size_t need = dgf_ffn_fwd_w4_workspace(M, H, I);
  if (!ws || ws_bytes < need || !aligned16(ws))
    return fail(DGF_EWORKSPACE, "4-bit forward workspace: need %zu bytes (16-byte aligned), got %zu", need, ws ? ws_bytes : 0);
  W4Params p{};
  p.x = (const uint16_t *)x; p.ldx = ldx;
  p.w[0] = w4_mat(gate_codes, gate_scales);
  p.w[1] = w4_mat(up_codes, up_scales);
  p.y = (uint16_t *)ws;  // the activations
  p.M = M; p.N = (int)I; p.K = (int)H; p.group = (int)group; p.fmt = fmt;
  hipStream_t s = (hipStream_t)stream;
  DGF_TRY(hip_check(timed(s, "4-bit gate/up", [&] { return launch_w4_gate_up(p, s); }), "4-bit gate/up"));
  p.x = (const uint16_t *)ws;
  p.w[0] = w4_mat(down_codes, down_scales);
  p.y = (uint16_t *)y; p.ldy = ldy;
  p.N = (int)H; p.K = (int)I;
  DGF_TRY(hip_check(timed(s, "4-bit down", [&] { return launch_w4_down(p, s); }), "4-bit down"));
  return ok();
}

}  // extern "C"
