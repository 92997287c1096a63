// Declarations of the layer around the selection (norm.hip, attend.hip, attend_bwd.hip), apart from
// the selection's in kpool_internal.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kpool {

// Layer norm of rows (norm.hip); f32: x, y, dy and dx are fp32, else bf16 bits.  Null
// pointers among w, b, mean, rstd (forward), dx, dw, db stand for what is not there or not
// wanted.  part: norm_bwd_blocks(rows, N) * 2 * N floats where dw or db is wanted.
hipError_t launch_norm(bool f32, const void *x, int64_t x_stride, const float *w, const float *b,
                       int64_t rows, int32_t N, float eps, void *y, float *mean, float *rstd,
                       hipStream_t stream);
int norm_bwd_blocks(int64_t rows, int32_t N);
hipError_t launch_norm_bwd(bool f32, const void *dy, const void *x, int64_t x_stride, const float *w,
                           const float *mean, const float *rstd, int64_t rows, int32_t N, void *dx,
                           float *dw, float *db, float *part, hipStream_t stream);

// Attention (attend.hip).  A call's operands, its plan by the sizes alone, its workspace.
struct AttendCall {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t *cu_q, *cu_k;            // device
  const int32_t *cu_q_host, *cu_k_host;
  int32_t nseq, Hq, Hkv, D;
  int64_t Tq, Tk;
  float scale;
  uint16_t *o;
  float *lse;
};
// What a unit costs, in steps: `fixed` for each part of it, then its steps.
struct UnitCost {
  int64_t fixed, steps;
};
struct TotalCost {
  int64_t units = 0, total = 0, longest = 0, most_steps = 0;
  void add(const UnitCost &c, int64_t times) {
    units += times, total += (c.fixed + c.steps) * times;
    if (longest < c.fixed + c.steps) longest = c.fixed + c.steps;
    if (most_steps < c.steps) most_steps = c.steps;
  }
};
struct AttendPlan {
  enum Form { kRows, kTiles, kList } form;
  int64_t ntiles;  // tiles of query rows, or more
  int nsplit;      // parts of the key axis, joined by a second kernel where there are more than one
  int chunk;       // keys of a part
  bool by_place;   // lists: ordered by place in the sequence first
  bool wave_rows;  // lists: a wave a row instead of four
};
AttendPlan plan_attend(const int32_t *cu_q, const int32_t *cu_k, int nseq, int Hq, int Hkv);
AttendPlan plan_list(int64_t Tq, int nseq, int width, int Hq, int Hkv);
size_t attend_workspace(const AttendPlan &p, int64_t rows, int D);
int64_t attend_threads(const AttendPlan &p, int Hq, int Hkv);  // of its largest launch, or more
hipError_t launch_attend(const AttendCall &c, const AttendPlan &p, void *workspace, hipStream_t st);
hipError_t launch_attend_list(const AttendCall &c, const AttendPlan &p, const int32_t *ids, int width,
                              void *workspace, hipStream_t st);

// Its gradients (attend_bwd.hip); c.o and c.lse are the forward pass's.
struct BwdPlan {
  int64_t ktiles, qtiles;  // tiles of keys, of query rows, or more
  TotalCost kcost;         // dK's and dV's work
  int kshares;             // its equal shares (0: a workgroup per tile and key head)
  int qsplit, qchunk;      // parts of the keys (dQ)
};
BwdPlan plan_attend_bwd(const int32_t *cu_q, const int32_t *cu_k, int nseq, int Hq, int Hkv);
size_t attend_bwd_workspace(const BwdPlan &p, int64_t Tq, int64_t Tk, int Hq, int Hkv, int D);
int64_t attend_bwd_threads(const BwdPlan &p, int Hkv);  // of its largest launch, or more
hipError_t launch_attend_bwd(const AttendCall &c, const uint16_t *d_o, const BwdPlan &p, void *workspace,
                             uint16_t *dq, uint16_t *dk, uint16_t *dv, hipStream_t st);

#if defined(__HIPCC__)

// Two fp32 values rounded to bf16 (to nearest, ties to even) as one word, lo in the low half.
__device__ inline uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

#endif

}  // namespace kpool
