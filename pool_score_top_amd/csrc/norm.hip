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
// elements each) between the statistics and the output.  Between load and store everything but
// the mean is fp32; the one rounding below that is the output's to its type.
//   The mean's error counts against the row's spread, which may be far below the mean itself: in
//   fp32 a row of 41 times 1000 gets 999.99994, off by more than its spread.  So the sum over a
//   row and the mean are in 64 bits, and x - mean is taken as (x - high) - low of the mean's two
//   fp32 parts: a constant row gives 0 exactly.
//   TPR 16 for rows of up to 16 vectors (a head dim of 128 in bf16): a wave holds 4 rows,
//          so no lane idles, and sums take 4 lane exchanges.
//   TPR 64 up to 256 vectors (backward 128): a wave per row, no barrier.
//   TPR 256 and 512 up to 2048 vectors (backward in bf16 1536): a workgroup per row.
//   Longer rows are read again for each pass (the second and third reads hit the caches).
// Measured (the card copies at 4.75 TB/s, reads and writes counted): 524288 x 128 in bf16,
// forward, 46 us (5.8 TB/s); 8192 x 4096 in bf16, forward 25 us (5.4 TB/s), backward 44 us (4.6
// TB/s) and 4 us to join the sums; 5003 x 1237 in fp32 at a pitch of 1328, forward 13.7 us (3.6
// TB/s), backward 16.5 us (4.5 TB/s) and 6 to join, which is latency, not bytes.  Long rows in bf16:
// 4096 x 16384 (forward in registers) 55 us, backward, which reads x and dy three times, once of
// them by single elements, 199 us; 3277 x 20480 forward 76, backward 204.
//
// The weight's gradient sums over rows in a fixed order: every workgroup takes a
// contiguous run of rows and keeps its columns' sums in registers, the workgroups'
// partial sums go to the workspace, and a second kernel adds them.  No atomics, so the
// result does not change from run to run; the split depends on the sizes alone.
#include <type_traits>

#include "layer_internal.h"

// (an element that two threads hold comes out the same in both: fused operations are written out)
#pragma clang fp contract(off)

namespace kpool {
namespace {

constexpr int kNormThreads = 256;

// VEC elements of a row, 16 bytes as they lie in memory, and as floats.  ALIGNED: rows start at
// 16-byte bounds and end at a whole vector.  Otherwise vectors are read and written where they are
// (the card takes 16 bytes at any element), and the one that crosses the row's end is moved back
// to end there: it shares elements with the vector before, which both hold and write alike and
// only that one counts.  (Loading single elements for the last vector instead makes the thread
// wait for them where they are put together, a row ahead of their use: 27131 x 1237 in bf16
// backward takes 102 us so, 52 this way.)
// VEC = 1, single elements, for unaligned rows of fp32 where that is faster (kSingle).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
template <class T>
constexpr int kVec = 16 / sizeof(T);

// where column c's vector starts in a row of N
template <bool ALIGNED, int VEC>
__device__ inline int start_of(int c, int N) {
  return ALIGNED ? c : max(min(c, N - VEC), 0);
}
// which of its elements count
template <bool ALIGNED, int VEC>
struct Part {
  int lo;
  uint32_t len;
  __device__ inline Part(int c, int N) {
    const int at = start_of<ALIGNED, VEC>(c, N);
    lo = c - at, len = (uint32_t)max(min(VEC, N - at) - lo, 0);
  }
  __device__ inline bool has(int e) const { return ALIGNED || (uint32_t)(e - lo) < len; }
};

template <class T, int VEC, bool ALIGNED>
struct Io {
  static_assert(VEC == kVec<T>, "whole vectors");
  typedef u32x4 Raw;
  static __device__ inline uint32_t bits(float x) { return __float_as_uint(x); }
  static __device__ inline uint32_t bits(uint16_t x) { return x; }
  static __device__ inline Raw fetch(const T *row, int c, int N) {
    if constexpr (ALIGNED) {
      return *reinterpret_cast<const u32x4 *>(row + c);
    } else {
      if (N >= VEC) return load_any(row + start_of<ALIGNED, VEC>(c, N));
      Raw a = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < VEC - 1; ++i)
        if (i < N) a[i * sizeof(T) / 4] |= bits(row[i]) << (i * sizeof(T) % 4 * 8);
      return a;
    }
  }
  static __device__ inline Raw load_any(const T *p) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const u32x4_at4 *>(p);
    else return *reinterpret_cast<const u32x4_at2 *>(p);
  }
  static __device__ inline void unpack(Raw a, float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(a[i]);
      else v[2 * i] = __uint_as_float(a[i] << 16), v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
  static __device__ inline void store(T *row, int c, int N, const float (&v)[VEC]) {
    Raw a;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) a[i] = __float_as_uint(v[i]);
      else a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
    T *p = row + start_of<ALIGNED, VEC>(c, N);
    if constexpr (ALIGNED) {
      *reinterpret_cast<u32x4 *>(p) = a;
    } else if (N >= VEC) {
      if constexpr (sizeof(T) == 4) *reinterpret_cast<u32x4_at4 *>(p) = a;
      else *reinterpret_cast<u32x4_at2 *>(p) = a;
    } else {
#pragma unroll
      for (int i = 0; i < VEC - 1; ++i)
        if (i < N) {
          if constexpr (sizeof(T) == 4) p[i] = v[i];
          else p[i] = (T)(a[i / 2] >> (i % 2 * 16));
        }
    }
  }
};
template <>
struct Io<float, 1, true> {
  typedef float Raw;
  static __device__ inline float fetch(const float *row, int c, int) { return row[c]; }
  static __device__ inline void unpack(float a, float (&v)[1]) { v[0] = a; }
  static __device__ inline void store(float *row, int c, int, const float (&v)[1]) { row[c] = v[0]; }
};
template <class T, bool ALIGNED, int VEC>
__device__ inline void load(const T *row, int c, int N, float (&v)[VEC]) {
  Io<T, VEC, ALIGNED>::unpack(Io<T, VEC, ALIGNED>::fetch(row, c, N), v);
}

// the same columns of a weight or bias
template <bool ALIGNED, int VEC>
__device__ inline void load_f32(const float *w, int c, int N, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = w[c];
    return;
  }
  const int at = start_of<ALIGNED, VEC>(c, N);
#pragma unroll
  for (int i = 0; i + 3 < VEC; i += 4) {
    if (ALIGNED || N >= VEC) {
      const u32x4 x = ALIGNED ? *reinterpret_cast<const u32x4 *>(w + at + i)
                              : (u32x4)*reinterpret_cast<const u32x4_at4 *>(w + at + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i + e] = __uint_as_float(x[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i + e] = i + e < N ? w[i + e] : 0.0f;
    }
  }
}

// Sums of K values over the TPR threads of a row, the same bits in every one of them.
// TPR 256 and 512 go through `red` (two sets, used in turn, so that one barrier a sum is enough:
// a set is written again only behind the barrier of the sum between).
template <int TPR, int K, class S>
__device__ inline void row_sum(S (&s)[K], S (*red)[8][K], int &phase) {
#pragma unroll
  for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] += __shfl_xor(s[i], d);
  if constexpr (TPR >= 256) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < K; ++i) red[phase][threadIdx.x >> 6][i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if constexpr (sizeof(S) == 8) {
        // (a wave's sum a lane: all 8 in every lane take the registers of a third workgroup a CU,
        // 8187 x 4098 in fp32 forward 55 us, so 48)
        s[i] = red[phase][threadIdx.x & (TPR / 64 - 1)][i];
#pragma unroll
        for (int d = 1; d < TPR / 64; d <<= 1) s[i] += __shfl_xor(s[i], d);
        continue;
      }
      s[i] = (red[phase][0][i] + red[phase][1][i]) + (red[phase][2][i] + red[phase][3][i]);
      if constexpr (TPR == 512)
        s[i] += (red[phase][4][i] + red[phase][5][i]) + (red[phase][6][i] + red[phase][7][i]);
    }
    phase ^= 1;
  }
}

// A row's mean as high + low in fp32.  sum / n, rounded once: where the quotient is a number (a
// constant row's), that number.
struct Mean {
  float high, low;
  __device__ inline Mean(double sum, double n, double inv_n) {
    double m = sum * inv_n;
    m = __builtin_fma(__builtin_fma(-m, n, sum), inv_n, m);
    high = (float)m, low = (float)(m - high);
  }
  __device__ inline float below(float x) const { return (x - high) - low; }
};
// What a thread adds up of a row: in bf16 at most 32 values of 8 bits each, which fp32 holds (those
// of one size exactly; beside larger ones, what it loses of a small one is far below their spread).
template <class T>
using Acc = std::conditional_t<sizeof(T) == 4, double, float>;

// Rows in registers.  ROWS rows of a thread group are loaded before the first is worked on.
template <int TPR>
constexpr int kThreads = TPR > kNormThreads ? TPR : kNormThreads;
template <class T, int VEC, bool ALIGNED, int TPR, int R, int ROWS>
__global__ __launch_bounds__(kThreads<TPR>) void norm_kernel(
    const T *__restrict__ x, int64_t x_stride, const float *__restrict__ w,
    const float *__restrict__ b, int64_t rows, int N, double inv, float eps, T *__restrict__ y,
    float *__restrict__ mean_out, float *__restrict__ rstd_out) {
  __shared__ float red[2][8][1];
  __shared__ double red_sum[2][8][1];
  int phase = 0, phase_sum = 0;
  constexpr int GROUPS = kThreads<TPR> / TPR;
  const int col = (threadIdx.x % TPR) * VEC;
  const int64_t row0 = ((int64_t)blockIdx.x * GROUPS + threadIdx.x / TPR) * ROWS;
  float v[ROWS][R][VEC], wv[R][VEC], bv[R][VEC];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = col + r * TPR * VEC;
      if (row0 + i < rows && c < N) {
        load<T, ALIGNED>(x + (row0 + i) * x_stride, c, N, v[i][r]);
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
      if (w) load_f32<ALIGNED>(w, c, N, wv[r]);
      if (b) load_f32<ALIGNED>(b, c, N, bv[r]);
    }
  }
  const float inv_n = (float)inv;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    // (a group past the last row still takes part in the workgroup's barriers)
    Acc<T> own_sum = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Part<ALIGNED, VEC> own(col + r * TPR * VEC, N);
#pragma unroll
      for (int e = 0; e < VEC; ++e) own_sum += own.has(e) ? v[i][r][e] : 0.0f;
    }
    double sum[1] = {own_sum};
    row_sum<TPR, 1>(sum, red_sum, phase_sum);
    const Mean mean(sum[0], N, inv);
    float s[1] = {0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Part<ALIGNED, VEC> own(col + r * TPR * VEC, N);
      if (col + r * TPR * VEC < N)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          v[i][r][e] = mean.below(v[i][r][e]);
          s[0] = own.has(e) ? fmaf(v[i][r][e], v[i][r][e], s[0]) : s[0];
        }
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
        Io<T, VEC, ALIGNED>::store(y + (row0 + i) * N, c, N, o);
      }
    }
    if (threadIdx.x % TPR == 0) {
      if (mean_out) mean_out[row0 + i] = mean.high;
      if (rstd_out) rstd_out[row0 + i] = rstd;
    }
  }
}

// Rows too long for the registers: a workgroup per row, which is read once a pass.
template <class T, bool ALIGNED>
__global__ __launch_bounds__(kNormThreads) void norm_long_kernel(
    const T *__restrict__ x, int64_t x_stride, const float *__restrict__ w,
    const float *__restrict__ b, int N, double inv, float eps, T *__restrict__ y,
    float *__restrict__ mean_out, float *__restrict__ rstd_out) {
  __shared__ float red[2][8][1];
  __shared__ double red_sum[2][8][1];
  int phase = 0, phase_sum = 0;
  constexpr int VEC = kVec<T>;
  const int64_t row = blockIdx.x;
  const T *xr = x + row * x_stride;
  float v[VEC], wv[VEC], bv[VEC], s[1] = {0.0f};
  double sum[1] = {0.0};
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    const Part<ALIGNED, VEC> own(c, N);
    load<T, ALIGNED>(xr, c, N, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[0] += own.has(e) ? v[e] : 0.0f;
  }
  row_sum<256, 1>(sum, red_sum, phase_sum);
  const float inv_n = (float)inv;
  const Mean mean(sum[0], N, inv);
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    const Part<ALIGNED, VEC> own(c, N);
    load<T, ALIGNED>(xr, c, N, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (own.has(e)) s[0] = fmaf(mean.below(v[e]), mean.below(v[e]), s[0]);
  }
  row_sum<256, 1>(s, red, phase);
  const float rstd = 1.0f / sqrtf(fmaf(s[0], inv_n, eps));
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    load<T, ALIGNED>(xr, c, N, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) wv[e] = 1.0f, bv[e] = 0.0f;
    if (w) load_f32<ALIGNED>(w, c, N, wv);
    if (b) load_f32<ALIGNED>(b, c, N, bv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = fmaf(mean.below(v[e]) * rstd, wv[e], bv[e]);
    Io<T, VEC, ALIGNED>::store(y + row * N, c, N, v);
  }
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[row] = mean.high;
    if (rstd_out) rstd_out[row] = rstd;
  }
}

// Backward, rows in registers: a workgroup takes rows_per rows, GROUPS at a time, writes
// their dx and keeps its columns' dw and db sums, which end in part[block][0 | 1][N].
template <class T, int VEC, bool ALIGNED, int TPR, int R>
__global__ __launch_bounds__(kThreads<TPR>) void norm_bwd_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, int64_t x_stride,
    const float *__restrict__ w, const float *__restrict__ mean, const float *__restrict__ rstd,
    int64_t rows, int64_t rows_per, int N, T *__restrict__ dx, float *__restrict__ part) {
  __shared__ float red[2][8][2];
  int phase = 0;
  constexpr int GROUPS = kThreads<TPR> / TPR;
  const int col = (threadIdx.x % TPR) * VEC, group = threadIdx.x / TPR;
  const int64_t lo = (int64_t)blockIdx.x * rows_per, hi = min(rows, lo + rows_per);
  const float inv_n = 1.0f / (float)N;
  float wv[R][VEC], dw[R][VEC], db[R][VEC];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) wv[r][e] = 1.0f, dw[r][e] = db[r][e] = 0.0f;
    const int c = col + r * TPR * VEC;
    if (w && c < N) load_f32<ALIGNED>(w, c, N, wv[r]);
  }
  // Rows are fetched AHEAD of the one that is worked on: their loads and this row's exchanges
  // and barrier then run side by side (a step of 8192 x 4096 in bf16: 77 us with two, 79.5 with
  // one; more vectors a thread leave no registers for a second).
  constexpr int AHEAD = R <= 2 ? 2 : 1;
  using IO = Io<T, VEC, ALIGNED>;
  typename IO::Raw xn[AHEAD][R] = {}, gn[AHEAD][R] = {};
  float mun[AHEAD] = {}, rsn[AHEAD] = {};
  auto fetch = [&](int64_t row, auto slot) {
    constexpr int I = decltype(slot)::value;
    if (row >= hi) return;
    mun[I] = mean[row], rsn[I] = rstd[row];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = col + r * TPR * VEC;
      if (c < N) xn[I][r] = IO::fetch(x + row * x_stride, c, N), gn[I][r] = IO::fetch(dy + row * N, c, N);
    }
  };
  auto step = [&](int64_t row, auto slot) {
    constexpr int I = decltype(slot)::value;
    const bool ok = row < hi;
    const float mu = mun[I], rs = rsn[I];
    float xh[R][VEC], g[R][VEC], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      IO::unpack(xn[I][r], xh[r]);
      IO::unpack(gn[I][r], g[r]);
      if (!ok || col + r * TPR * VEC >= N)
#pragma unroll
        for (int e = 0; e < VEC; ++e) xh[r][e] = mu, g[r][e] = 0.0f;
    }
    fetch(row + AHEAD * GROUPS, slot);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Part<ALIGNED, VEC> own(col + r * TPR * VEC, N);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        xh[r][e] = (xh[r][e] - mu) * rs;
        const float k = own.has(e) ? g[r][e] : 0.0f, kw = k * wv[r][e];
        db[r][e] += k;
        dw[r][e] = fmaf(k, xh[r][e], dw[r][e]);
        g[r][e] *= wv[r][e];
        s[0] += kw;
        s[1] = fmaf(kw, xh[r][e], s[1]);
      }
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
          for (int e = 0; e < VEC; ++e) o[e] = rs * fmaf(-xh[r][e], c1, g[r][e] - c2);
          IO::store(dx + row * N, c, N, o);
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
    for (int r = 0; r < R; ++r) {
      const int c0 = r * TPR * VEC, at = start_of<ALIGNED, VEC>(col + c0, N) - c0;
      const Part<ALIGNED, VEC> own(col + c0, N);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (own.has(e)) join[group][at + e] = half ? db[r][e] : dw[r][e];
        __syncthreads();
        for (int c = threadIdx.x; c < TPR * VEC; c += kNormThreads) {
          float t = 0.0f;
#pragma unroll
          for (int k = 0; k < GROUPS; ++k) t += join[k][c];
          if (c0 + c < N) pw[half * N + c0 + c] = t;
        }
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = col + r * TPR * VEC, at = start_of<ALIGNED, VEC>(c, N);
      const Part<ALIGNED, VEC> own(c, N);
      if (c < N)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (own.has(e)) pw[at + e] = dw[r][e], pw[N + at + e] = db[r][e];
    }
  }
}

// Backward of rows too long for the registers: dx, a workgroup per row.
template <class T, bool ALIGNED>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_long_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, int64_t x_stride,
    const float *__restrict__ w, const float *__restrict__ mean, const float *__restrict__ rstd,
    int N, T *__restrict__ dx) {
  __shared__ float red[2][8][2];
  int phase = 0;
  constexpr int VEC = kVec<T>;
  const int64_t row = blockIdx.x;
  const float mu = mean[row], rs = rstd[row], inv_n = 1.0f / (float)N;
  float xv[VEC], g[VEC], wv[VEC], s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < VEC; ++e) wv[e] = 1.0f;
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    const Part<ALIGNED, VEC> own(c, N);
    load<T, ALIGNED>(x + row * x_stride, c, N, xv);
    load<T, ALIGNED>(dy + row * N, c, N, g);
    if (w) load_f32<ALIGNED>(w, c, N, wv);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (own.has(e)) {
        s[0] = fmaf(g[e], wv[e], s[0]);
        s[1] = fmaf(g[e] * wv[e], (xv[e] - mu) * rs, s[1]);
      }
  }
  row_sum<256, 2>(s, red, phase);
  const float c2 = s[0] * inv_n, c1 = s[1] * inv_n;
  for (int c = threadIdx.x * VEC; c < N; c += kNormThreads * VEC) {
    load<T, ALIGNED>(x + row * x_stride, c, N, xv);
    load<T, ALIGNED>(dy + row * N, c, N, g);
    if (w) load_f32<ALIGNED>(w, c, N, wv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = rs * fmaf(-((xv[e] - mu) * rs), c1, fmaf(g[e], wv[e], -c2));
    Io<T, VEC, ALIGNED>::store(dx + row * N, c, N, g);
  }
}

__device__ inline float value(float x) { return x; }
__device__ inline float value(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

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
    const float g = value(dy[r * N + c]);
    db += g;
    dw = fmaf(g, (value(x[r * x_stride + c]) - mean[r]) * rstd[r], dw);
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

// Rows of one launch: a workgroup per row of 256 or 512 threads keeps the launch's threads below
// 2^32.
constexpr int64_t kNormLaunchRows = int64_t(1) << 22;

// Unaligned rows of fp32 up to these go by single elements, forward and backward (us for 32 Mi
// elements, single and by vectors: forward N = 65 139 159, 127 72 82, 253 47 48, 501 83 42, 1237 78
// 50; backward 65 115 196, 501 90 124, 1237 99 189, 2047 89 119, 4098 174 137; in bf16 vectors
// always win: forward 65 120 35, 1237 57 35, 8191 70 31).
constexpr int kSingle = 256, kSingleBwd = 2048;
static_assert(kSingle <= 256 && kSingleBwd <= 2048, "what the kernels of single elements take");

// (the pitch counts only where there is a second row)
template <class T>
bool aligned_rows(const void *x, int64_t x_stride, int64_t rows, int N, const void *w, const void *b,
                  const void *y, const void *dy) {
  const uintptr_t bits = (uintptr_t)x | (uintptr_t)w | (uintptr_t)b | (uintptr_t)y | (uintptr_t)dy;
  return bits % 16 == 0 && N % kVec<T> == 0 && (rows <= 1 || (x_stride * sizeof(T)) % 16 == 0);
}

template <class T, int VEC, bool ALIGNED, int TPR, int R, int ROWS>
void norm_go(const void *x, int64_t xs, const float *w, const float *b, int64_t rows, int N,
             float eps, void *y, float *mean, float *rstd, hipStream_t st) {
  const int64_t per = (int64_t)(kThreads<TPR> / TPR) * ROWS;
  hipLaunchKernelGGL((norm_kernel<T, VEC, ALIGNED, TPR, R, ROWS>), dim3((unsigned)((rows + per - 1) / per)),
                     dim3(kThreads<TPR>), 0, st, (const T *)x, xs, w, b, rows, N, 1.0 / N, eps, (T *)y, mean,
                     rstd);
}

template <class T, int VEC, bool ALIGNED>
void norm_pick(const void *x, int64_t xs, const float *w, const float *b, int64_t rows, int N,
               float eps, void *y, float *mean, float *rstd, hipStream_t st) {
  const int nv = (N + VEC - 1) / VEC;
#define KPOOL_NORM(TPR, R, ROWS) norm_go<T, VEC, ALIGNED, TPR, R, ROWS>(x, xs, w, b, rows, N, eps, y, mean, rstd, st)
  if (nv <= 16) {
    if (rows >= 65536) KPOOL_NORM(16, 1, 4); else KPOOL_NORM(16, 1, 1);
  }
  else if (nv <= 64) KPOOL_NORM(64, 1, 1);
  else if (nv <= 128) KPOOL_NORM(64, 2, 1);
  else if (VEC == 1 || nv <= 256) KPOOL_NORM(64, 4, 1);  // (single elements: up to kSingle of them)
  else if constexpr (VEC > 1) {
    if (nv <= 512) KPOOL_NORM(256, 2, 1);
    else if (nv <= 768) KPOOL_NORM(256, 3, 1);
    else if (nv <= 1024) KPOOL_NORM(256, 4, 1);
    else if (nv <= 2048) KPOOL_NORM(512, 4, 1);
    else
      hipLaunchKernelGGL((norm_long_kernel<T, ALIGNED>), dim3((unsigned)rows), dim3(kNormThreads), 0, st,
                         (const T *)x, xs, w, b, N, 1.0 / N, eps, (T *)y, mean, rstd);
  }
#undef KPOOL_NORM
}

template <class T, int VEC, bool ALIGNED>
void norm_bwd_pick(const void *dy, const void *x, int64_t xs, const float *w, const float *mean,
                   const float *rstd, int64_t rows, int N, void *dx, float *part, int nblk,
                   int64_t rows_per, hipStream_t st) {
  const int nv = (N + VEC - 1) / VEC;
#define KPOOL_NORM(TPR, R)                                                                            \
  hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, ALIGNED, TPR, R>), dim3((unsigned)nblk), dim3(kThreads<TPR>), \
                     0, st, (const T *)dy, (const T *)x, xs, w, mean, rstd, rows, rows_per, N,        \
                     (T *)dx, part)
  if (nv <= 16) KPOOL_NORM(16, 1);
  else if (nv <= 64) KPOOL_NORM(64, 1);
  else if (nv <= 128) KPOOL_NORM(64, 2);
  else if (nv <= 256) KPOOL_NORM(256, 1);
  else if (nv <= 512) KPOOL_NORM(256, 2);
  else if constexpr (VEC == 1) {  // (more, smaller loads a thread; 512 threads: 1237 of fp32 123 us, so 99)
    if (nv <= 1024) KPOOL_NORM(256, 4);
    else if (nv <= 1536) KPOOL_NORM(256, 6);
    else KPOOL_NORM(256, 8);
  }
  else if (nv <= 1024) KPOOL_NORM(512, 2);
  else if (nv <= 1536) KPOOL_NORM(512, 3);
  else if (VEC <= 4 && nv <= 2048) {  // (bf16: too many registers)
    if constexpr (VEC <= 4) KPOOL_NORM(512, 4);
  } else {
    for (int64_t r = 0; dx && r < rows; r += kNormLaunchRows) {
      const int64_t n = rows - r < kNormLaunchRows ? rows - r : kNormLaunchRows;
      hipLaunchKernelGGL((norm_bwd_long_kernel<T, ALIGNED>), dim3((unsigned)n), dim3(kNormThreads), 0, st,
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
  const bool vec = f32 ? aligned_rows<float>(x, x_stride, rows, N, w, b, y, nullptr)
                       : aligned_rows<uint16_t>(x, x_stride, rows, N, w, b, y, nullptr);
  for (int64_t r = 0; r < rows; r += kNormLaunchRows) {
    const int64_t n = rows - r < kNormLaunchRows ? rows - r : kNormLaunchRows;
    const char *xr = (const char *)x + r * x_stride * size;
    char *yr = (char *)y + r * N * size;
    float *mr = mean ? mean + r : nullptr, *rr = rstd ? rstd + r : nullptr;
    if (f32 && vec) norm_pick<float, 4, true>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    else if (f32 && N <= kSingle) norm_pick<float, 1, true>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    else if (f32) norm_pick<float, 4, false>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    else if (vec) norm_pick<uint16_t, 8, true>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    else norm_pick<uint16_t, 8, false>(xr, x_stride, w, b, n, N, eps, yr, mr, rr, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Row runs of the backward pass, by the sizes alone: at most 1024 workgroups, runs of 8 rows
// or more, and partial sums of at most 8 MiB, unless that leaves fewer than 256 workgroups, one a
// CU (8192 x 4096 in bf16: 256 workgroups 80 us a step, 512 the same, 1024 95 us).
int norm_bwd_blocks(int64_t rows, int32_t N) {
  int64_t most = (int64_t(1) << 20) / N;
  if (most > 1024) most = 1024;
  if (most < 256) most = 256;
  const int64_t want = rows > 8 ? (rows + 7) / 8 : 1;
  return (int)(want < most ? want : most);
}

hipError_t launch_norm_bwd(bool f32, const void *dy, const void *x, int64_t x_stride, const float *w,
                           const float *mean, const float *rstd, int64_t rows, int32_t N, void *dx,
                           float *dw, float *db, float *part, hipStream_t st) {
  const int nblk = norm_bwd_blocks(rows, N);
  const int64_t rows_per = (rows + nblk - 1) / nblk;
  if (!dw && !db) part = nullptr;
  const bool vec = f32 ? aligned_rows<float>(x, x_stride, rows, N, w, nullptr, dx, dy)
                       : aligned_rows<uint16_t>(x, x_stride, rows, N, w, nullptr, dx, dy);
#define KPOOL_NORM(T, VEC, ALIGNED) \
  norm_bwd_pick<T, VEC, ALIGNED>(dy, x, x_stride, w, mean, rstd, rows, N, dx, part, nblk, rows_per, st)
  if (f32 && vec) KPOOL_NORM(float, 4, true);
  else if (f32 && N <= kSingleBwd) KPOOL_NORM(float, 1, true);
  else if (f32) KPOOL_NORM(float, 4, false);
  else if (vec) KPOOL_NORM(uint16_t, 8, true);
  else KPOOL_NORM(uint16_t, 8, false);
#undef KPOOL_NORM
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part) return e;
  hipLaunchKernelGGL(norm_join_kernel, dim3((2 * N + 15) / 16), dim3(kNormThreads), 0, st, part, nblk, N,
                     dw, db);
  return hipGetLastError();
}

}  // namespace kpool
