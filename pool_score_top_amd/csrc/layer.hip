// C ABI of libkpool, the layer around the selection: argument validation and launches of the layer
// norm and the attention.
//
// One translation unit with api.hip, whose error text, checks and profile records these entry
// points share and which keep to that file.
#include <initializer_list>

#include "api.hip"
#include "layer_internal.h"

namespace {

// The timing records of these entry points, apart from the selection's: a caller that knows only the
// selection's kinds collects into arrays of that many.
enum { kNorm, kAttend };
thread_local std::vector<ProfRec> g_layer_prof;

template <class F>
hipError_t timed_layer(int kind, hipStream_t stream, F &&launch) {
  const size_t before = g_prof.size();
  const hipError_t e = timed(kind, stream, launch);
  if (g_prof.size() > before) {
    g_layer_prof.push_back(g_prof.back());
    g_prof.pop_back();
  }
  return e;
}

// What a call reads or writes at p: `rows` rows of `len` bytes, `pitch` bytes apart (pitch >= len);
// one row for what is contiguous.
struct Operand {
  const char *name;
  const void *p;
  int64_t len, rows = 1, pitch = 0;
};

// Whether a contiguous operand meets one of the other's rows.
bool meets(const Operand &out, const Operand &in) {
  if (!out.p || !in.p || out.len <= 0 || in.rows <= 0 || in.len <= 0) return false;
  const int64_t from = (int64_t)((uintptr_t)out.p - (uintptr_t)in.p);
  if (from + out.len <= 0 || from >= (in.rows - 1) * in.pitch + in.len) return false;
  // the first row that ends behind `out`'s start, if that one starts before its end
  const int64_t r = from < in.len ? 0 : (from - in.len) / in.pitch + 1;
  return r < in.rows && r * in.pitch < from + out.len;
}

// What is written (contiguous, the workspace among it) apart from what is read and from one another.
int check_apart(const char *fn, std::initializer_list<Operand> written, std::initializer_list<Operand> read) {
  for (const Operand *w = written.begin(); w != written.end(); ++w) {
    for (const Operand &r : read)
      if (meets(*w, r)) return fail(KPOOL_EINVAL, "%s: %s overlaps %s", fn, w->name, r.name);
    for (const Operand *x = w + 1; x != written.end(); ++x)
      if (meets(*w, *x)) return fail(KPOOL_EINVAL, "%s: %s overlaps %s", fn, w->name, x->name);
  }
  return KPOOL_OK;
}

int check_norm(const char *fn, int64_t rows, int32_t N, int64_t x_stride, int32_t dtype) {
  if (dtype != KPOOL_DTYPE_BF16 && dtype != KPOOL_DTYPE_F32)
    return fail(KPOOL_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (rows < 0) return fail(KPOOL_EINVAL, "%s: rows must be >= 0", fn);
  if (N < 1 || N > (1 << 26)) return fail(KPOOL_EINVAL, "%s: N must be in [1, 2^26] (got %d)", fn, N);
  if (x_stride < N) return fail(KPOOL_EINVAL, "%s: x_stride must be >= N", fn);
  return KPOOL_OK;
}

// A launch's threads are counted in 32 bits.
constexpr int64_t kLaunchThreads = int64_t(1) << 32;

// Arguments that the attention entry points share.
int check_heads(const char *fn, int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv)
    return fail(KPOOL_EINVAL, "%s: Hq must be a positive multiple of Hkv (Hq=%d Hkv=%d)", fn, Hq, Hkv);
  if (Hq > 65536) return fail(KPOOL_EUNSUPPORTED, "%s: more than 65536 heads (got %d)", fn, Hq);
  if (D < 8 || D % 8) return fail(KPOOL_EINVAL, "%s: D must be a positive multiple of 8 (got %d)", fn, D);
  if (D > 128) return fail(KPOOL_EUNSUPPORTED, "%s: D up to 128 is compiled in (got %d)", fn, D);
  return KPOOL_OK;
}

int check_lengths(const char *fn, const int32_t *cu_q, const int32_t *cu_k, int32_t nseq, int32_t G) {
  int rc = check_cu(cu_q, nseq, fn);
  if (!rc) rc = check_cu(cu_k, nseq, fn);
  if (rc) return rc;
  for (int32_t s = 0; s < nseq; ++s)  // (a tile's rows are numbered in 32 bits)
    if ((int64_t)(cu_q[s + 1] - cu_q[s]) * G > 0x7FFFFF00 || cu_k[s + 1] - cu_k[s] > 0x7FFFFF00)
      return fail(KPOOL_EUNSUPPORTED, "%s: sequence %d has too many query rows or keys", fn, s);
  return KPOOL_OK;
}

// Fills in Tq and Tk.  Tq = 0 needs no pointers.
int check_attend(const char *fn, kpool::AttendCall &c, const int32_t *cu_q_host, const int32_t *cu_k_host) {
  int rc = check_heads(fn, c.Hq, c.Hkv, c.D);
  if (!rc) rc = check_lengths(fn, cu_q_host, cu_k_host, c.nseq, c.Hq / c.Hkv);
  if (rc) return rc;
  if (!(c.scale > 0.0f) || !isfinite(c.scale)) return fail(KPOOL_EINVAL, "%s: scale must be finite and > 0", fn);
  const struct { int64_t stride, least; } st[3] = {{c.q_stride, (int64_t)c.Hq * c.D},
                                                   {c.k_stride, (int64_t)c.Hkv * c.D},
                                                   {c.v_stride, (int64_t)c.Hkv * c.D}};
  for (const auto &x : st)
    if (x.stride < x.least || x.stride % 8 || x.stride > (1 << 24))
      return fail(KPOOL_EINVAL, "%s: a token stride must be a multiple of 8 in [%lld, 2^24] (got %lld)", fn,
                  (long long)x.least, (long long)x.stride);
  if (((uintptr_t)c.cu_q | (uintptr_t)c.cu_k) & 3)
    return fail(KPOOL_EINVAL, "%s: cu_q or cu_k is not aligned to its elements", fn);
  c.Tq = cu_q_host[c.nseq];
  c.Tk = cu_k_host[c.nseq];
  if (c.Tq == 0) return ok();
  if (!c.q || !c.o || !c.cu_q || !c.cu_k || (c.Tk > 0 && (!c.k || !c.v)))
    return fail(KPOOL_EINVAL, "%s: null pointer", fn);
  if (!aligned16(c.q) || !aligned16(c.k) || !aligned16(c.v) || !aligned16(c.o))
    return fail(KPOOL_EINVAL, "%s: q, k, v and o must be 16-byte aligned", fn);
  if ((uintptr_t)c.lse & 3) return fail(KPOOL_EINVAL, "%s: lse is not aligned to its elements", fn);
  return KPOOL_OK;
}

Operand q_of(const kpool::AttendCall &c) { return {"q", c.q, (int64_t)c.Hq * c.D * 2, c.Tq, c.q_stride * 2}; }
Operand k_of(const kpool::AttendCall &c) { return {"k", c.k, (int64_t)c.Hkv * c.D * 2, c.Tk, c.k_stride * 2}; }
Operand v_of(const kpool::AttendCall &c) { return {"v", c.v, (int64_t)c.Hkv * c.D * 2, c.Tk, c.v_stride * 2}; }
Operand cu_q_of(const kpool::AttendCall &c) { return {"cu_q", c.cu_q, ((int64_t)c.nseq + 1) * 4}; }
Operand cu_k_of(const kpool::AttendCall &c) { return {"cu_k", c.cu_k, ((int64_t)c.nseq + 1) * 4}; }

// The forward calls' plan, workspace and outputs; ids: the lists, if there are any.
int check_attend_plan(const char *fn, const kpool::AttendCall &c, const kpool::AttendPlan &p, const void *workspace,
                      size_t workspace_bytes, const Operand &ids) {
  if (kpool::attend_threads(p, c.Hq, c.Hkv) >= kLaunchThreads)
    return fail(KPOOL_EUNSUPPORTED, "%s: too many query rows or sequences for one launch", fn);
  const size_t need = kpool::attend_workspace(p, c.Tq * c.Hq, c.D);
  if (need && (!workspace || workspace_bytes < need))
    return fail(KPOOL_EWORKSPACE, "%s: needs %zu bytes of workspace, got %zu", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (need && !aligned16(workspace)) return fail(KPOOL_EINVAL, "%s: workspace must be 16-byte aligned", fn);
  const int64_t rows = c.Tq * c.Hq;
  return check_apart(fn, {{"o", c.o, rows * c.D * 2}, {"lse", c.lse, rows * 4}, {"workspace", workspace, (int64_t)need}},
                     {q_of(c), k_of(c), v_of(c), cu_q_of(c), cu_k_of(c), ids});
}

}  // namespace

extern "C" {

size_t kpool_attend_workspace_bytes(const int32_t *cu_q_host, const int32_t *cu_k_host, int32_t nseq,
                                    int32_t Hq, int32_t Hkv, int32_t D) {
  const char *fn = "kpool_attend_workspace_bytes";
  if (check_heads(fn, Hq, Hkv, D) || check_lengths(fn, cu_q_host, cu_k_host, nseq, Hq / Hkv)) return 0;
  ok();
  return kpool::attend_workspace(kpool::plan_attend(cu_q_host, cu_k_host, nseq, Hq, Hkv),
                                 (int64_t)cu_q_host[nseq] * Hq, D);
}

int kpool_attend(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                 const uint16_t *v, int64_t v_stride, const int32_t *cu_q_host,
                 const int32_t *cu_q_dev, const int32_t *cu_k_host, const int32_t *cu_k_dev,
                 int32_t nseq, int32_t Hq, int32_t Hkv, int32_t D, float scale, void *workspace,
                 size_t workspace_bytes, uint16_t *o, float *lse, void *stream) {
  const char *fn = "kpool_attend";
  kpool::AttendCall c{q, k, v, q_stride, k_stride, v_stride, cu_q_dev, cu_k_dev, cu_q_host,
                      cu_k_host, nseq, Hq, Hkv, D,
                      0, 0, scale, o, lse};
  int rc = check_attend(fn, c, cu_q_host, cu_k_host);
  if (rc || c.Tq == 0) return rc;
  const kpool::AttendPlan p = kpool::plan_attend(cu_q_host, cu_k_host, nseq, Hq, Hkv);
  rc = check_attend_plan(fn, c, p, workspace, workspace_bytes, {});
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = timed_layer(kAttend, st, [&] { return kpool::launch_attend(c, p, workspace, st); });
  if (e != hipSuccess) return hip_fail(fn, e);
  return ok();
}

size_t kpool_attend_backward_workspace_bytes(const int32_t *cu_q_host, const int32_t *cu_k_host,
                                             int32_t nseq, int32_t Hq, int32_t Hkv, int32_t D) {
  const char *fn = "kpool_attend_backward_workspace_bytes";
  if (check_heads(fn, Hq, Hkv, D) || check_lengths(fn, cu_q_host, cu_k_host, nseq, Hq / Hkv)) return 0;
  ok();
  return kpool::attend_bwd_workspace(kpool::plan_attend_bwd(cu_q_host, cu_k_host, nseq, Hq, Hkv),
                                     cu_q_host[nseq], cu_k_host[nseq], Hq, Hkv, D);
}

int kpool_attend_backward(const uint16_t *d_o, const uint16_t *q, int64_t q_stride, const uint16_t *k,
                          int64_t k_stride, const uint16_t *v, int64_t v_stride, const uint16_t *o,
                          const float *lse, const int32_t *cu_q_host, const int32_t *cu_q_dev,
                          const int32_t *cu_k_host, const int32_t *cu_k_dev, int32_t nseq, int32_t Hq,
                          int32_t Hkv, int32_t D, float scale, void *workspace,
                          size_t workspace_bytes, uint16_t *dq, uint16_t *dk, uint16_t *dv,
                          void *stream) {
  const char *fn = "kpool_attend_backward";
  kpool::AttendCall c{q, k, v, q_stride, k_stride, v_stride, cu_q_dev, cu_k_dev, cu_q_host,
                      cu_k_host, nseq, Hq, Hkv, D,
                      0, 0, scale, const_cast<uint16_t *>(o), const_cast<float *>(lse)};
  int rc = check_attend(fn, c, cu_q_host, cu_k_host);
  if (rc) return rc;
  if (c.Tq == 0 && c.Tk == 0) return ok();
  if (!cu_q_dev || !cu_k_dev || (c.Tq > 0 && (!d_o || !lse || !dq)) || (c.Tk > 0 && (!k || !v || !dk || !dv)))
    return fail(KPOOL_EINVAL, "%s: null pointer", fn);
  if (!aligned16(k) || !aligned16(v) || !aligned16(d_o) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(KPOOL_EINVAL, "%s: k, v, d_o, dq, dk and dv must be 16-byte aligned", fn);
  const kpool::BwdPlan p = kpool::plan_attend_bwd(cu_q_host, cu_k_host, nseq, Hq, Hkv);
  if (kpool::attend_bwd_threads(p, Hkv) >= kLaunchThreads)
    return fail(KPOOL_EUNSUPPORTED, "%s: too many rows or sequences for one launch", fn);
  const size_t need = kpool::attend_bwd_workspace(p, c.Tq, c.Tk, Hq, Hkv, D);
  if (need && (!workspace || workspace_bytes < need))
    return fail(KPOOL_EWORKSPACE, "%s: needs %zu bytes of workspace, got %zu", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned16(workspace)) return fail(KPOOL_EINVAL, "%s: workspace must be 16-byte aligned", fn);
  const int64_t qbytes = c.Tq * Hq * D * 2, kbytes = c.Tk * Hkv * D * 2, lbytes = c.Tq * Hq * 4;
  rc = check_apart(fn, {{"dq", dq, qbytes}, {"dk", dk, kbytes}, {"dv", dv, kbytes}, {"workspace", workspace, (int64_t)need}},
                   {q_of(c), k_of(c), v_of(c), cu_q_of(c), cu_k_of(c), {"d_o", d_o, qbytes}, {"o", o, qbytes},
                    {"lse", lse, lbytes}});
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = timed_layer(kAttend, st, [&] {
    return kpool::launch_attend_bwd(c, d_o, p, workspace, dq, dk, dv, st);
  });
  if (e != hipSuccess) return hip_fail(fn, e);
  return ok();
}

size_t kpool_attend_selected_workspace_bytes(int64_t Tq, int32_t nseq, int32_t width, int32_t Hq,
                                             int32_t Hkv, int32_t D) {
  const char *fn = "kpool_attend_selected_workspace_bytes";
  if (check_heads(fn, Hq, Hkv, D)) return 0;
  if (Tq < 0 || nseq < 1 || width < 0) {
    fail(KPOOL_EINVAL, "%s: need Tq >= 0, nseq >= 1, width >= 0", fn);
    return 0;
  }
  ok();
  return kpool::attend_workspace(kpool::plan_list(Tq, nseq, width, Hq, Hkv), Tq * Hq, D);
}

int kpool_attend_selected(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                          const uint16_t *v, int64_t v_stride, const int32_t *token_ids,
                          int32_t width, const int32_t *cu_q_host, const int32_t *cu_q_dev,
                          const int32_t *cu_k_host, const int32_t *cu_k_dev, int32_t nseq, int32_t Hq,
                          int32_t Hkv, int32_t D, float scale, void *workspace,
                          size_t workspace_bytes, uint16_t *o, float *lse, void *stream) {
  const char *fn = "kpool_attend_selected";
  if (width < 0 || width > (1 << 30)) return fail(KPOOL_EINVAL, "%s: width must be in [0, 2^30] (got %d)", fn, width);
  kpool::AttendCall c{q, k, v, q_stride, k_stride, v_stride, cu_q_dev, cu_k_dev, cu_q_host,
                      cu_k_host, nseq, Hq, Hkv, D,
                      0, 0, scale, o, lse};
  int rc = check_attend(fn, c, cu_q_host, cu_k_host);
  if (rc || c.Tq == 0) return rc;
  if (width > 0 && !token_ids) return fail(KPOOL_EINVAL, "%s: null pointer", fn);
  if ((uintptr_t)token_ids & 3) return fail(KPOOL_EINVAL, "%s: token_ids is not aligned to its elements", fn);
  const kpool::AttendPlan p = kpool::plan_list(c.Tq, nseq, width, Hq, Hkv);
  rc = check_attend_plan(fn, c, p, workspace, workspace_bytes, {"token_ids", token_ids, c.Tq * width * 4});
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = timed_layer(kAttend, st, [&] {
    return kpool::launch_attend_list(c, p, token_ids, width, workspace, st);
  });
  if (e != hipSuccess) return hip_fail(fn, e);
  return ok();
}

int kpool_layer_norm(const void *x, int64_t x_stride, const float *weight, const float *bias,
                     int64_t rows, int32_t N, float eps, int32_t dtype, void *y, float *mean,
                     float *rstd, void *stream) {
  const char *fn = "kpool_layer_norm";
  int rc = check_norm(fn, rows, N, x_stride, dtype);
  if (rc) return rc;
  if (!(eps >= 0.0f) || !isfinite(eps)) return fail(KPOOL_EINVAL, "%s: eps must be finite and >= 0", fn);
  if (rows == 0) return ok();
  if (!x || !y) return fail(KPOOL_EINVAL, "%s: null pointer", fn);
  const int64_t size = dtype == KPOOL_DTYPE_F32 ? 4 : 2;
  const uintptr_t mask = size - 1;
  if ((((uintptr_t)x | (uintptr_t)y) & mask) ||
      (((uintptr_t)weight | (uintptr_t)bias | (uintptr_t)mean | (uintptr_t)rstd) & 3))
    return fail(KPOOL_EINVAL, "%s: a pointer is not aligned to its elements", fn);
  rc = check_apart(fn, {{"y", y, rows * N * size}, {"mean", mean, rows * 4}, {"rstd", rstd, rows * 4}},
                   {{"x", x, N * size, rows, x_stride * size}, {"weight", weight, N * 4LL}, {"bias", bias, N * 4LL}});
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = timed_layer(kNorm, st, [&] {
    return kpool::launch_norm(dtype == KPOOL_DTYPE_F32, x, x_stride, weight, bias, rows, N, eps, y, mean,
                              rstd, st);
  });
  if (e != hipSuccess) return hip_fail(fn, e);
  return ok();
}

size_t kpool_layer_norm_backward_workspace_bytes(int64_t rows, int32_t N) {
  if (rows < 0 || N < 1) return 0;
  return (size_t)kpool::norm_bwd_blocks(std::max<int64_t>(rows, 1), N) * 2 * (size_t)N * sizeof(float);
}

int kpool_layer_norm_backward(const void *dy, const void *x, int64_t x_stride, const float *weight,
                              const float *mean, const float *rstd, int64_t rows, int32_t N,
                              int32_t dtype, void *workspace, size_t workspace_bytes, void *dx,
                              float *dweight, float *dbias, void *stream) {
  const char *fn = "kpool_layer_norm_backward";
  int rc = check_norm(fn, rows, N, x_stride, dtype);
  if (rc) return rc;
  const bool sums = dweight || dbias;
  if (!dx && !sums) return fail(KPOOL_EINVAL, "%s: no output given", fn);
  if (rows == 0 && !sums) return ok();
  if (rows > 0 && (!dy || !x || !mean || !rstd)) return fail(KPOOL_EINVAL, "%s: null pointer", fn);
  const int64_t size = dtype == KPOOL_DTYPE_F32 ? 4 : 2, row_bytes = N * size;
  const uintptr_t mask = size - 1;
  if ((((uintptr_t)x | (uintptr_t)dy | (uintptr_t)dx) & mask) ||
      (((uintptr_t)weight | (uintptr_t)mean | (uintptr_t)rstd | (uintptr_t)dweight | (uintptr_t)dbias) & 3))
    return fail(KPOOL_EINVAL, "%s: a pointer is not aligned to its elements", fn);
  size_t need = 0;
  if (sums) {
    need = kpool_layer_norm_backward_workspace_bytes(rows, N);
    if (!workspace || workspace_bytes < need)
      return fail(KPOOL_EWORKSPACE, "%s: needs %zu bytes of workspace, got %zu", fn, need,
                  workspace ? workspace_bytes : (size_t)0);
    if (!aligned16(workspace)) return fail(KPOOL_EINVAL, "%s: workspace must be 16-byte aligned", fn);
  }
  rc = check_apart(fn,
                   {{"dx", dx, rows * row_bytes}, {"dweight", dweight, N * 4LL}, {"dbias", dbias, N * 4LL},
                    {"workspace", workspace, (int64_t)need}},
                   {{"dy", dy, rows * row_bytes}, {"x", x, row_bytes, rows, x_stride * size},
                    {"weight", weight, N * 4LL}, {"mean", mean, rows * 4}, {"rstd", rstd, rows * 4}});
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = timed_layer(kNorm, st, [&] {
    return kpool::launch_norm_bwd(dtype == KPOOL_DTYPE_F32, dy, x, x_stride, weight, mean, rstd, rows, N,
                                  dx, dweight, dbias, (float *)workspace, st);
  });
  if (e != hipSuccess) return hip_fail(fn, e);
  return ok();
}

int kpool_layer_profile_collect(double *ms, int64_t *launches) {
  std::swap(g_prof, g_layer_prof);
  const int rc = kpool_profile_collect(ms, launches);
  std::swap(g_prof, g_layer_prof);
  return rc;
}

}  // extern "C"
