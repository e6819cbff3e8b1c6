// Host helpers shared by the C ABI's entry points: error reporting, the kernel
// timing hook, argument checks and workspace carving.
#pragma once

#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <string>

#include "dgf.h"
#include "dgf_kernels.hpp"
#include "dgf_q8.hpp"

namespace dgf {

// Message of the calling thread's last non-OK status.
extern thread_local std::string g_err;

inline dgf_status fail(dgf_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

inline dgf_status ok() {
  g_err.clear();
  return DGF_OK;
}

inline dgf_status hip_check(hipError_t e, const char *what) {
  if (e != hipSuccess) return fail(DGF_EHIP, "%s: %s", what, hipGetErrorString(e));
  return DGF_OK;
}

// Kernel timing hook: caller-created events, one pair per launch step (one
// kernel, or a vector body and its scalar tail), recorded as the kernels' own
// start and end timestamps.
struct Prof {
  hipEvent_t *ev = nullptr;
  int pairs = 0;
  int used = 0;
  const char *names[4096] = {};
};
extern thread_local Prof g_prof;

template <class F>
inline hipError_t timed(hipStream_t s, const char *name, F &&launch) {
  const int k = g_prof.used;
  const bool rec = g_prof.ev && k < g_prof.pairs;
  if (rec) {  // the launches record them as their kernels' start and end
    g_launch_events[0] = g_prof.ev[2 * k];
    g_launch_events[1] = g_prof.ev[2 * k + 1];
  }
  hipError_t e = launch();
  if (rec) {
    const bool none = g_launch_events[0] != nullptr;  // no kernel took them: an empty interval
    g_launch_events[0] = g_launch_events[1] = nullptr;
    if (none && e == hipSuccess) e = hipEventRecord(g_prof.ev[2 * k], s);
    if (none && e == hipSuccess) e = hipEventRecord(g_prof.ev[2 * k + 1], s);
  }
  if (g_prof.ev) {
    if (k < 4096) g_prof.names[k] = name;
    g_prof.used = k + 1;
  }
  return e;
}

#define DGF_TRY(expr)                  \
  do {                                 \
    dgf_status st_ = (expr);           \
    if (st_ != DGF_OK) return st_;     \
  } while (0)

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// A row-major BF16 matrix operand: non-null, 16-byte aligned, ld >= cols, ld % 8 == 0.
constexpr int64_t kMaxLd = (int64_t)1 << 23;

inline dgf_status check_mat(const char *name, const void *p, int64_t ld, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return DGF_OK;
  if (!p) return fail(DGF_EINVAL, "%s is NULL", name);
  if (!aligned16(p)) return fail(DGF_EINVAL, "%s is not 16-byte aligned", name);
  if (ld < cols) return fail(DGF_EINVAL, "%s: leading dimension %lld < row width %lld", name, (long long)ld, (long long)cols);
  if (ld % 8 != 0) return fail(DGF_EINVAL, "%s: leading dimension %lld is not a multiple of 8", name, (long long)ld);
  // a 128-row tile's byte offsets from its first row stay below 2^31
  if (ld >= kMaxLd) return fail(DGF_EUNSUPPORTED, "%s: leading dimension %lld beyond the library's limit (< 2^23)", name, (long long)ld);
  return DGF_OK;
}

inline dgf_status check_dims(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return fail(DGF_EINVAL, "negative dimension (M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
  if (M > ((int64_t)1 << 21) || N > ((int64_t)1 << 30) || K > ((int64_t)1 << 23))
    return fail(DGF_EUNSUPPORTED, "dimensions beyond the library's limits (M<=2^21, N<=2^30, K<=2^23)");
  return DGF_OK;
}

inline int64_t round8(int64_t v) { return (v + 7) & ~(int64_t)7; }
inline size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

// A matrix saved in 8 bits: codes [rows, cols] and one FP32 scale for every 64 columns.
inline dgf_status check_q8(const char *name, const Q8Mat &t, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return DGF_OK;
  const int64_t nb = (cols + kQ8Block - 1) / kQ8Block;
  if (!t.q || !t.s) return fail(DGF_EINVAL, "%s: %s is NULL", name, t.q ? "the scales" : "the codes");
  if (!aligned16(t.q)) return fail(DGF_EINVAL, "%s: the codes are not 16-byte aligned", name);
  if ((uintptr_t)t.s & 3) return fail(DGF_EINVAL, "%s: the scales are not 4-byte aligned", name);
  if (t.ldq < cols || t.ldq % 8 != 0)
    return fail(DGF_EINVAL, "%s: leading dimension %lld of the codes: need a multiple of 8, at least %lld", name, (long long)t.ldq, (long long)cols);
  if (t.lds < nb)
    return fail(DGF_EINVAL, "%s: leading dimension %lld of the scales < %lld blocks", name, (long long)t.lds, (long long)nb);
  if (t.ldq >= kMaxLd) return fail(DGF_EUNSUPPORTED, "%s: leading dimension %lld beyond the library's limit (< 2^23)", name, (long long)t.ldq);
  return DGF_OK;
}

// Public dtype code -> stored type of the kernels: BF16 and FP16 share the
// tree; an FP32 FFN has no declared leaf rule (its MFMA differs), so it is
// rejected as unsupported.
inline dgf_status stored_type(int dtype, int *fmt) {
  if (dtype == DGF_BF16) { *fmt = FMT_BF16; return DGF_OK; }
  if (dtype == DGF_FP16) { *fmt = FMT_F16; return DGF_OK; }
  if (dtype == DGF_FP32) return fail(DGF_EUNSUPPORTED, "dtype FP32: only BF16 and FP16 storage is implemented here");
  return fail(DGF_EINVAL, "unknown dtype %d", dtype);
}

// Workspace pieces, 256-byte aligned.
struct Carve {
  char *base;
  size_t used;
  uint16_t *take(size_t elems) {
    uint16_t *p = (uint16_t *)(base + used);
    used += round256(elems * 2);
    return p;
  }
};

}  // namespace dgf
