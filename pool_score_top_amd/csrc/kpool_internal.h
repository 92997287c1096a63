// Internal declarations shared by the HIP translation units of libkpool.
// Device helpers live here; each kernel is launched from the file that
// defines it through a host launcher declared below.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kpool {

// ----------------------------------------------------------------------------
// Launch planning data for the score kernel.  A "segment" is the part of one
// sequence that falls in the current row chunk; it is cut into row tiles of
// kTileRows rows that never straddle a sequence (each tile shares one set of
// pooled keys).  Segments travel by value in the kernel arguments.
// ----------------------------------------------------------------------------
constexpr int kMaxSegs = 32;

struct SegList {
  int32_t nseg;
  int32_t tile_start[kMaxSegs + 1];  // prefix of row tiles per segment
  int32_t row_lo[kMaxSegs];          // first global row of the segment
  int32_t row_hi[kMaxSegs];          // one past the last global row
  int32_t seq_start[kMaxSegs];       // global row of the sequence's token 0
  int32_t pool_base[kMaxSegs];       // first pooled-key row of the sequence
  int32_t pool_count[kMaxSegs];      // pools of the sequence (caps every row's visible count)
};

// ----------------------------------------------------------------------------
// Host launchers (each returns hipGetLastError() after the launch).
// ----------------------------------------------------------------------------
hipError_t launch_pool_keys(const uint16_t *k, const int32_t *cu_seqlens, const int32_t *cu_pools,
                            int32_t nseq, int32_t D, int32_t kpool, int64_t P_tot, uint16_t *kp,
                            hipStream_t stream);

hipError_t launch_pool_keys_gated(const uint16_t *k, const uint16_t *g, const float *ape,
                                  const int32_t *cu_seqlens, const int32_t *cu_pools, int32_t nseq,
                                  int32_t D, int32_t kpool, int64_t P_tot, uint16_t *kp,
                                  hipStream_t stream);

// true if (H, D) has a compiled score kernel
bool score_supported(int H, int D);
int score_tile_rows();
// Score workgroups the device runs at once (CUs x workgroups per CU), 0 if unknown.
int score_slots(int H, int D, int device);
// Scores of the chunk's rows go to out[(row - chunk_row0) * ld + pool]; the max of each
// 16-pool group of a row (over its visible pools) to gmax[(row - chunk_row0) * ldg + pool/16].
constexpr int kGroup = 16;
hipError_t launch_score(int H, int D, const uint16_t *q, const uint16_t *kp, const float *w,
                        float scale, int32_t kpool, const SegList &segs, int32_t ntiles,
                        int32_t npseg, int32_t pseg_pools, int64_t chunk_row0, int64_t ld,
                        float *out, int64_t ldg, float *gmax, hipStream_t stream);

constexpr int kTopkMaxBudget = 2048;
// Rows [row0, row0 + nrows) of `scores` (row r at scores + r*ld).  The number
// of ranked entries of row r is n_valid[r] if n_valid is not null, else
// (t / kpool + 1) for the row's sequence-local position t (global row
// grow0 + r looked up in cu_seqlens), capped at L / kpool for a sequence of L
// tokens in tail mode (full pools only).
// With gmax (the score kernel's 16-pool group maxima, row pitch ldg) the selection reads
// the group maxima first and then only the groups that can hold a winner; without it
// every row is read in full.
hipError_t launch_topk(const float *scores, int64_t ld, int64_t nrows, const int32_t *n_valid,
                       const int32_t *cu_seqlens, int32_t nseq, int64_t grow0, int32_t kpool,
                       bool tail, int32_t budget, int32_t *out, const float *gmax, int64_t ldg,
                       hipStream_t stream);

hipError_t launch_scores_copy(const float *ws, int64_t ld, int64_t nrows, const int32_t *cu_seqlens,
                              int32_t nseq, int64_t grow0, int32_t kpool, bool tail, float *dst,
                              int64_t dst_ld, hipStream_t stream);

// tail: full pools only, and kpool - 1 tail slots after a row's budget*kpool expanded ones
hipError_t launch_expand(const int32_t *pool_ids, const int32_t *cu_seqlens, int32_t nseq,
                         int32_t kpool, bool tail, int64_t q_lo, int64_t nrows, int32_t budget,
                         int32_t *token_ids, hipStream_t stream);

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

// ----------------------------------------------------------------------------
// Device helpers
// ----------------------------------------------------------------------------
#if defined(__HIPCC__)

// Pools visible to the row at sequence-local position t of a sequence of L tokens:
// p*kpool <= t, and in tail mode (full pools only) p < L / kpool.
__device__ inline int64_t visible_count(int64_t t, int64_t L, int kpool, bool tail) {
  const int64_t n = t / kpool + 1;
  return tail ? min(n, L / kpool) : n;
}

// Two fp32 values rounded to bf16 (to nearest, ties to even) as one word, lo in the low half.
__device__ inline uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// Index of the sequence holding global row `row`: the largest s < nseq with
// cu[s] <= row (empty sequences are skipped because their start repeats).
__device__ inline int find_seq(const int32_t *__restrict__ cu, int nseq, int64_t row) {
  int lo = 0, hi = nseq;  // answer in [lo, hi)
  while (hi - lo > 1) {
    int mid = (lo + hi) >> 1;
    if (cu[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}

// fp32 -> order-preserving uint32: larger key = larger value.  -0.0 is folded
// onto +0.0 first, and every NaN maps to 0, below -inf (whose key is
// 0x007FFFFF), so NaN is never ranked above a number.
__device__ inline uint32_t order_key(float f) {
  uint32_t u = __float_as_uint(f);
  if (u == 0x80000000u) u = 0u;
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

#endif

}  // namespace kpool
