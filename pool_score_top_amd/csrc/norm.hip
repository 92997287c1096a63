// Layer norm of rows, forward and backward, with the weight's and bias's gradients.
//
//   mean = sum_j x_j / N,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / N + eps)
//   y_j  = (x_j - mean) * rstd * w_j + b_j
//   with xh_j = (x_j - mean) * rstd and g_j = dy_j * w_j:
//   dx_j = rstd * (g_j - sum(g) / N - xh_j * sum(g xh) / N)
//   dw_j = sum over rows of dy_j * xh_j,   db_j = sum over rows of dy_j
//
// Pages: Atlas inference glm5next_dsa/tp.rs, indexer tensors of the shard plan: the
// indexer's keys pass a layer norm with weight and bias before they are pooled.
//
// HBM-bound: about 8 (forward) and 21 (step) flops an element against 4 to 16 bytes.  So
// each element is read once: a row lives in the registers of TPR threads (R vectors of VEC
// elements each) between the statistics and the output.  Everything between load and store
// is fp32; the one rounding is the output's to its type.
//   TPR 16 for rows of up to 16 vectors (a head dim of 128 in bf16): a wave holds 4 rows,
//          so no lane idles, and sums take 4 lane exchanges.
//   TPR 64 up to 256 vectors: a wave per row, no barrier.
//   TPR 256 up to 1024 vectors, 2048 of one or four elements: a workgroup per row.
//   Longer rows are read again for each pass (the second and third reads hit the caches).
// VEC is 16 bytes where pointers and pitches allow it, one element otherwise.
// Measured (the card copies at 4.75 TB/s, reads and writes counted): 524288 x 128 in bf16,
// forward, 46 us (5.8 TB/s); 8192 x 4096 in bf16, forward 24 us (5.6 TB/s), backward 45 us (4.5
// TB/s) and 4 us to join the sums; 5003 x 1237 in fp32 at a pitch of 1328, by single elements,
// forward 12.5 us (4.0 TB/s), backward 16 us (4.6 TB/s).
//
// The weight's gradient sums over rows in a fixed order: every workgroup takes a
// contiguous run of rows and keeps its columns' sums in registers, the workgroups'
// partial sums go to the workspace, and a second kernel adds them.  No atomics, so the
// result does not change from run to run; the split depends on the sizes alone.
#include <type_traits>

#include "kpool_internal.h"

namespace kpool {
namespace {

constexpr int kNormThreads = 256;

// VEC elements as they lie in memory, and as floats.
template <class T, int VEC>
struct Io {
  static_assert(VEC == 1, "one element");
  typedef T Raw;
  static __device__ inline Raw fetch(const T *p) { return *p; }
  static __device__ inline void unpack(Raw a, float (&v)[1]) {
    v[0] = sizeof(T) == 4 ? (float)a : __uint_as_float((uint32_t)a << 16);
  }
  static __device__ inline void store(T *p, const float (&v)[1]) {
    if constexpr (sizeof(T) == 4) *p = v[0];
    else *p = (T)pack_bf16(v[0], 0.0f);
  }
};
template <>
struct Io<float, 4> {
  typedef float4 Raw;
  static __device__ inline Raw fetch(const float *p) { return *reinterpret_cast<const float4 *>(p); }
  static __device__ inline void unpack(const Raw &a, float (&v)[4]) {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  }
  static __device__ inline void store(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Io<uint16_t, 8> {
  typedef uint4 Raw;
  static __device__ inline Raw fetch(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }
  static __device__ inline void unpack(const Raw &a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ inline void store(uint16_t *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                               pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};
template <class T, int VEC>
__device__ inline void load(const T *p, float (&v)[VEC]) {
  Io<T, VEC>::unpack(Io<T, VEC>::fetch(p), v);
}

template <int VEC>
__device__ inline void load_f32(const float *p, float (&v)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(p + i);
      v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
    }
  } else {
    v[0] = p[0];
  }
}

// Sums of K values over the TPR threads of a row, the same bits in every one of them.
// TPR 256 goes through `red` (two sets, used in turn, so that one barrier a sum is enough:
// a set is written again only behind the barrier of the sum between).
template <int TPR, int K>
__device__ inline void row_sum(float (&s)[K], float (*red)[4][K], int &phase) {
#pragma unroll
  for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] += __shfl_xor(s[i], d);
  if constexpr (TPR == 256) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < K; ++i) red[phase][threadIdx.x >> 6][i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i)
      s[i] = (red[phase][0][i] + red[phase][1][i]) + (red[phase][2][i] + red[phase][3][i]);
    phase ^= 1;
  }
}

// Rows in registers.  ROWS rows of a thread group are loaded before the first is worked on.
template <class T, int VEC, int TPR, int R, int ROWS>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(
    const T *__restrict__ x, int64_t x_stride, const float *__restrict__ w,
    const float *__restrict__ b, int64_t rows, int N, float eps, T *__restrict__ y,
    float *__restrict__ mean_out, float *__restrict__ rstd_out) {
  __shared__ float red[2][4][1];
  int phase = 0;
  constexpr int GROUPS = kNormThreads / TPR;
  const int col = (threadIdx.x % TPR) * VEC;
  const int64_t row0 = ((int64_t)blockIdx.x * GROUPS + threadIdx.x / TPR) * ROWS;
  float v[ROWS][R][VEC], wv[R][VEC], bv[R][VEC];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = col + r * TPR * VEC;
      if (row0 + i < rows && c < N) {
        load<T, VEC>(x + (row0 + i) * x_stride + c, v[i][r]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][r][e] = 0.0f;
      }
    }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = col + r * TPR * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) wv[r][e] = 1.0f, bv[r][e] = 0.0f;
    if (c < N) {
      if (w) load_f32<VEC>(w + c, wv[r]);
      if (b) load_f32<VEC>(b + c, bv[r]);
    }
  }
  const float inv_n = 1.0f / (float)N;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    // (a group past the last row still takes part in the workgroup's barriers)
    float s[1] = {0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += v[i][r][e];
    row_sum<TPR, 1>(s, red, phase);
    const float mean = s[0] * inv_n;
    s[0] = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (col + r * TPR * VEC < N)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          v[i][r][e] -= mean;
          s[0] = fmaf(v[i][r][e], v[i][r][e], s[0]);
        }
    row_sum<TPR, 1>(s, red, phase);
    const float rstd = 1.0f / sqrtf(fmaf(s[0], inv_n, eps));
    if (row0 + i >= rows) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = col + r * TPR * VEC;
      if (c < N) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(v[i][r][e] * rstd, wv[r][e], bv[r][e]);
        Io<T, VEC>::store(y + (row0 + i) * N + c, o);
      }
    }
    if (threadIdx.x % TPR == 0) {
      if (mean_out) mean_out[row0 + i] = mean;
      if (rstd_out) rstd_out[row0 + i] = rstd;
    }
  }
}

// Rows too long for the registers: a workgroup per row, which is read once a pass.
template <class T, int VEC>
__global__ __launch_bounds__(kNormThreads) void norm_long_kernel(
    const T *__restrict__ x, int64_t x_stride, const float *__restrict__ w,
    const float *__restrict__ b, int N, float eps, T *__restrict__ y,
    float *__restrict__ mean_out, float *__restrict__ rstd_out) {
  __shared__ float red[2][4][1];
  int phase = 0;
  const int64_t row = blockIdx.x;
  const T *xr = x + row * x_stride;
  float v[VEC], wv[VEC], bv[VEC], s[1] = {0.0f};
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    load<T, VEC>(xr + c, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] += v[e];
  }
  row_sum<256, 1>(s, red, phase);
  const float inv_n = 1.0f / (float)N, mean = s[0] * inv_n;
  s[0] = 0.0f;
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    load<T, VEC>(xr + c, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] = fmaf(v[e] - mean, v[e] - mean, s[0]);
  }
  row_sum<256, 1>(s, red, phase);
  const float rstd = 1.0f / sqrtf(fmaf(s[0], inv_n, eps));
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    load<T, VEC>(xr + c, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) wv[e] = 1.0f, bv[e] = 0.0f;
    if (w) load_f32<VEC>(w + c, wv);
    if (b) load_f32<VEC>(b + c, bv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = fmaf((v[e] - mean) * rstd, wv[e], bv[e]);
    Io<T, VEC>::store(y + row * N + c, v);
  }
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
}

// Backward, rows in registers: a workgroup takes rows_per rows, GROUPS at a time, writes
// their dx and keeps its columns' dw and db sums, which end in part[block][0 | 1][N].
template <class T, int VEC, int TPR, int R>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, int64_t x_stride,
    const float *__restrict__ w, const float *__restrict__ mean, const float *__restrict__ rstd,
    int64_t rows, int64_t rows_per, int N, T *__restrict__ dx, float *__restrict__ part) {
  __shared__ float red[2][4][2];
  int phase = 0;
  constexpr int GROUPS = kNormThreads / TPR;
  const int col = (threadIdx.x % TPR) * VEC, group = threadIdx.x / TPR;
  const int64_t lo = (int64_t)blockIdx.x * rows_per, hi = min(rows, lo + rows_per);
  const float inv_n = 1.0f / (float)N;
  float wv[R][VEC], dw[R][VEC], db[R][VEC];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) wv[r][e] = 1.0f, dw[r][e] = db[r][e] = 0.0f;
    if (w && col + r * TPR * VEC < N) load_f32<VEC>(w + col + r * TPR * VEC, wv[r]);
  }
  // Rows are fetched AHEAD of the one that is worked on: their loads and this row's exchanges
  // and barrier then run side by side (a step of 8192 x 4096 in bf16: 77 us with two, 79.5 with
  // one; more vectors a thread leave no registers for a second).
  constexpr int AHEAD = R <= 2 ? 2 : 1;
  typename Io<T, VEC>::Raw xn[AHEAD][R] = {}, gn[AHEAD][R] = {};
  float mun[AHEAD] = {}, rsn[AHEAD] = {};
  auto fetch = [&](int64_t row, auto slot) {
    constexpr int I = decltype(slot)::value;
    if (row >= hi) return;
    mun[I] = mean[row], rsn[I] = rstd[row];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = col + r * TPR * VEC;
      if (c < N)
        xn[I][r] = Io<T, VEC>::fetch(x + row * x_stride + c), gn[I][r] = Io<T, VEC>::fetch(dy + row * N + c);
    }
  };
  auto step = [&](int64_t row, auto slot) {
    constexpr int I = decltype(slot)::value;
    const bool ok = row < hi;
    const float mu = mun[I], rs = rsn[I];
    float xh[R][VEC], g[R][VEC], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Io<T, VEC>::unpack(xn[I][r], xh[r]);
      Io<T, VEC>::unpack(gn[I][r], g[r]);
      if (!ok || col + r * TPR * VEC >= N)
#pragma unroll
        for (int e = 0; e < VEC; ++e) xh[r][e] = mu, g[r][e] = 0.0f;
    }
    fetch(row + AHEAD * GROUPS, slot);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        xh[r][e] = (xh[r][e] - mu) * rs;
        db[r][e] += g[r][e];
        dw[r][e] = fmaf(g[r][e], xh[r][e], dw[r][e]);
        g[r][e] *= wv[r][e];
        s[0] += g[r][e];
        s[1] = fmaf(g[r][e], xh[r][e], s[1]);
      }
    row_sum<TPR, 2>(s, red, phase);
    const float c2 = s[0] * inv_n, c1 = s[1] * inv_n;
    if (dx && ok) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int c = col + r * TPR * VEC;
        if (c < N) {
          float o[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[e] = rs * (g[r][e] - c2 - xh[r][e] * c1);
          Io<T, VEC>::store(dx + row * N + c, o);
        }
      }
    }
  };
  std::integral_constant<int, 0> first;
  std::integral_constant<int, AHEAD - 1> second;
  fetch(lo + group, first);
  if (AHEAD > 1) fetch(lo + group + GROUPS, second);
  for (int64_t base = lo; base < hi; base += AHEAD * GROUPS) {  // the same trips for all groups
    step(base + group, first);
    if (AHEAD > 1 && base + GROUPS < hi) step(base + group + GROUPS, second);
  }
  if (!part) return;
  float *pw = part + (int64_t)blockIdx.x * 2 * N;
  if constexpr (GROUPS > 1) {
    // the groups' sums join through LDS in group order
    __shared__ float join[GROUPS][TPR * VEC];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) join[group][col + e] = half ? db[r][e] : dw[r][e];
        __syncthreads();
        for (int c = threadIdx.x; c < TPR * VEC; c += kNormThreads) {
          float t = 0.0f;
#pragma unroll
          for (int k = 0; k < GROUPS; ++k) t += join[k][c];
          if (r * TPR * VEC + c < N) pw[half * N + r * TPR * VEC + c] = t;
        }
      }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = col + r * TPR * VEC;
      if (c < N)
#pragma unroll
        for (int e = 0; e < VEC; ++e) pw[c + e] = dw[r][e], pw[N + c + e] = db[r][e];
    }
  }
}

// Backward of rows too long for the registers: dx, a workgroup per row.
template <class T, int VEC>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_long_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, int64_t x_stride,
    const float *__restrict__ w, const float *__restrict__ mean, const float *__restrict__ rstd,
    int N, T *__restrict__ dx) {
  __shared__ float red[2][4][2];
  int phase = 0;
  const int64_t row = blockIdx.x;
  const float mu = mean[row], rs = rstd[row], inv_n = 1.0f / (float)N;
  float xv[VEC], g[VEC], wv[VEC], s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < VEC; ++e) wv[e] = 1.0f;
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    load<T, VEC>(x + row * x_stride + c, xv);
    load<T, VEC>(dy + row * N + c, g);
    if (w) load_f32<VEC>(w + c, wv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      s[0] = fmaf(g[e], wv[e], s[0]);
      s[1] = fmaf(g[e] * wv[e], (xv[e] - mu) * rs, s[1]);
    }
  }
  row_sum<256, 2>(s, red, phase);
  const float c2 = s[0] * inv_n, c1 = s[1] * inv_n;
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    load<T, VEC>(x + row * x_stride + c, xv);
    load<T, VEC>(dy + row * N + c, g);
    if (w) load_f32<VEC>(w + c, wv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = rs * (g[e] * wv[e] - c2 - (xv[e] - mu) * rs * c1);
    Io<T, VEC>::store(dx + row * N + c, g);
  }
}

// and its columns' partial sums: block (column block, row run)
template <class T>
__global__ __launch_bounds__(kNormThreads) void norm_cols_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, int64_t x_stride,
    const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows, int64_t rows_per,
    int N, float *__restrict__ part) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= N) return;
  const int64_t lo = (int64_t)blockIdx.y * rows_per, hi = min(rows, lo + rows_per);
  float dw = 0.0f, db = 0.0f;
  for (int64_t r = lo; r < hi; ++r) {
    float g[1], xv[1];
    load<T, 1>(dy + r * N + c, g);
    load<T, 1>(x + r * x_stride + c, xv);
    db += g[0];
    dw = fmaf(g[0], (xv[0] - mean[r]) * rstd[r], dw);
  }
  part[(int64_t)blockIdx.y * 2 * N + c] = dw;
  part[(int64_t)blockIdx.y * 2 * N + N + c] = db;
}

// Adds the workgroups' partial sums of 16 columns a workgroup: thread (slice, column), 16
// slices, each a fixed run of every 16th partial.
__global__ __launch_bounds__(kNormThreads) void norm_join_kernel(const float *__restrict__ part,
                                                                 int nblk, int N,
                                                                 float *__restrict__ dw,
                                                                 float *__restrict__ db) {
  __shared__ float join[16][17];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;  // of the 2 N columns
  float t = 0.0f;
  if (col < 2 * (int64_t)N)
#pragma unroll 8
    for (int k = slice; k < nblk; k += 16) t += part[(int64_t)k * 2 * N + col];
  join[slice][c] = t;
  __syncthreads();
  if (slice != 0 || col >= 2 * (int64_t)N) return;
  t = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) t += join[k][c];
  if (col < N) {
    if (dw) dw[col] = t;
  } else if (db) {
    db[col - N] = t;
  }
}

// Rows of one launch: a workgroup per row of 256 threads keeps the launch's threads below
// 2^32.
constexpr int64_t kNormLaunchRows = int64_t(1) << 23;

template <class T>
constexpr int kVec = 16 / sizeof(T);

// whether 6 and 8 vectors of a row fit a thread's registers beside the sums (with 8 bf16 a
// vector they would take over 256 and leave a wave a SIMD)
template <int VEC>
constexpr bool kWide = VEC <= 4;

// (the pitch counts only where there is a second row)
template <class T>
bool vector_ok(const void *x, int64_t x_stride, int N, const void *w, const void *b, const void *y,
               const void *dy) {
  const uintptr_t bits = (uintptr_t)x | (uintptr_t)w | (uintptr_t)b | (uintptr_t)y | (uintptr_t)dy;
  return bits % 16 == 0 && N % kVec<T> == 0 && (x_stride * sizeof(T)) % 16 == 0;
}

template <class T, int VEC, int TPR, int R, int ROWS>
void norm_go(const void *x, int64_t xs, const float *w, const float *b, int64_t rows, int N,
             float eps, void *y, float *mean, float *rstd, hipStream_t st) {
  const int64_t per = (int64_t)(kNormThreads / TPR) * ROWS;
  hipLaunchKernelGGL((norm_kernel<T, VEC, TPR, R, ROWS>), dim3((unsigned)((rows + per - 1) / per)),
                     dim3(kNormThreads), 0, st, (const T *)x, xs, w, b, rows, N, eps, (T *)y, mean,
                     rstd);
}

template <class T, int VEC>
void norm_pick(const void *x, int64_t xs, const float *w, const float *b, int64_t rows, int N,
               float eps, void *y, float *mean, float *rstd, hipStream_t st) {
  const int nv = (N + VEC - 1) / VEC;
#define KPOOL_NORM(TPR, R, ROWS) norm_go<T, VEC, TPR, R, ROWS>(x, xs, w, b, rows, N, eps, y, mean, rstd, st)
  if (nv <= 16) {
    if (rows >= 65536) KPOOL_NORM(16, 1, 4); else KPOOL_NORM(16, 1, 1);
  }
  else if (nv <= 64) KPOOL_NORM(64, 1, 1);
  else if (nv <= 128) KPOOL_NORM(64, 2, 1);
  else if (nv <= 256) KPOOL_NORM(64, 4, 1);
  else if (nv <= 512) KPOOL_NORM(256, 2, 1);
  else if (nv <= 768) KPOOL_NORM(256, 3, 1);
  else if (nv <= 1024) KPOOL_NORM(256, 4, 1);
  else if (kWide<VEC> && nv <= 1536) KPOOL_NORM(256, kWide<VEC> ? 6 : 1, 1);
  else if (kWide<VEC> && nv <= 2048) KPOOL_NORM(256, kWide<VEC> ? 8 : 1, 1);
  else
    hipLaunchKernelGGL((norm_long_kernel<T, VEC>), dim3((unsigned)rows), dim3(kNormThreads), 0, st,
                       (const T *)x, xs, w, b, N, eps, (T *)y, mean, rstd);
#undef KPOOL_NORM
}

template <class T, int VEC>
void norm_bwd_pick(const void *dy, const void *x, int64_t xs, const float *w, const float *mean,
                   const float *rstd, int64_t rows, int N, void *dx, float *part, int nblk,
                   int64_t rows_per, hipStream_t st) {
  const int nv = (N + VEC - 1) / VEC;
#define KPOOL_NORM(TPR, R)                                                                        \
  hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, TPR, R>), dim3((unsigned)nblk), dim3(kNormThreads), \
                     0, st, (const T *)dy, (const T *)x, xs, w, mean, rstd, rows, rows_per, N,    \
                     (T *)dx, part)
  if (nv <= 16) KPOOL_NORM(16, 1);
  else if (nv <= 64) KPOOL_NORM(64, 1);
  else if (nv <= 128) KPOOL_NORM(64, 2);
  else if (nv <= 256) KPOOL_NORM(256, 1);
  else if (nv <= 512) KPOOL_NORM(256, 2);
  else if (nv <= 768) KPOOL_NORM(256, 3);
  else if (nv <= 1024) KPOOL_NORM(256, 4);
  else if (kWide<VEC> && nv <= 1536) KPOOL_NORM(256, kWide<VEC> ? 6 : 1);
  else if (kWide<VEC> && nv <= 2048) KPOOL_NORM(256, kWide<VEC> ? 8 : 1);
  else {
    for (int64_t r = 0; dx && r < rows; r += kNormLaunchRows) {
      const int64_t n = rows - r < kNormLaunchRows ? rows - r : kNormLaunchRows;
      hipLaunchKernelGGL((norm_bwd_long_kernel<T, VEC>), dim3((unsigned)n), dim3(kNormThreads), 0, st,
                         (const T *)dy + r * N, (const T *)x + r * xs, xs, w, mean + r, rstd + r, N,
                         (T *)dx + r * N);
    }
    if (part)
      hipLaunchKernelGGL((norm_cols_kernel<T>), dim3((N + kNormThreads - 1) / kNormThreads, nblk),
                         dim3(kNormThreads), 0, st, (const T *)dy, (const T *)x, xs, mean, rstd, rows,
                         rows_per, N, part);
  }
#undef KPOOL_NORM
}

}  // namespace

hipError_t launch_norm(bool f32, const void *x, int64_t x_stride, const float *w, const float *b,
                       int64_t rows, int32_t N, float eps, void *y, float *mean, float *rstd,
                       hipStream_t st) {
  const int64_t size = f32 ? 4 : 2;
  const bool vec = f32 ? vector_ok<float>(x, x_stride, N, w, b, y, nullptr)
                       : vector_ok<uint16_t>(x, x_stride, N, w, b, y, nullptr);
  for (int64_t r = 0; r < rows; r += kNormLaunchRows) {
    const int64_t n = rows - r < kNormLaunchRows ? rows - r : kNormLaunchRows;
    const char *xr = (const char *)x + r * x_stride * size;
    char *yr = (char *)y + r * N * size;
    float *mr = mean ? mean + r : nullptr, *rr = rstd ? rstd + r : nullptr;
    if (f32 && vec) norm_pick<float, 4>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    else if (f32) norm_pick<float, 1>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    else if (vec) norm_pick<uint16_t, 8>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    else norm_pick<uint16_t, 1>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Row runs of the backward pass, by the sizes alone: at most 1024 workgroups, runs of 8 rows
// or more, and partial sums of at most 8 MiB, unless that leaves fewer than 128 workgroups
// (8192 x 4096 in bf16: 256 workgroups 80 us a step, 512 the same, 1024 95 us).
int norm_bwd_blocks(int64_t rows, int32_t N) {
  int64_t most = (int64_t(1) << 20) / N;
  if (most > 1024) most = 1024;
  if (most < 128) most = 128;
  const int64_t want = rows > 8 ? (rows + 7) / 8 : 1;
  return (int)(want < most ? want : most);
}

hipError_t launch_norm_bwd(bool f32, const void *dy, const void *x, int64_t x_stride, const float *w,
                           const float *mean, const float *rstd, int64_t rows, int32_t N, void *dx,
                           float *dw, float *db, float *part, hipStream_t st) {
  const int nblk = norm_bwd_blocks(rows, N);
  const int64_t rows_per = (rows + nblk - 1) / nblk;
  if (!dw && !db) part = nullptr;
  if (f32) {
    if (vector_ok<float>(x, x_stride, N, w, nullptr, dx, dy))
      norm_bwd_pick<float, 4>(dy, x, x_stride, w, mean, rstd, rows, N, dx, part, nblk, rows_per, st);
    else
      norm_bwd_pick<float, 1>(dy, x, x_stride, w, mean, rstd, rows, N, dx, part, nblk, rows_per, st);
  } else {
    if (vector_ok<uint16_t>(x, x_stride, N, w, nullptr, dx, dy))
      norm_bwd_pick<uint16_t, 8>(dy, x, x_stride, w, mean, rstd, rows, N, dx, part, nblk, rows_per, st);
    else
      norm_bwd_pick<uint16_t, 1>(dy, x, x_stride, w, mean, rstd, rows, N, dx, part, nblk, rows_per, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part) return e;
  hipLaunchKernelGGL(norm_join_kernel, dim3((2 * N + 15) / 16), dim3(kNormThreads), 0, st, part, nblk, N,
                     dw, db);
  return hipGetLastError();
}

}  // namespace kpool
