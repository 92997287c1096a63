// Rotary positions: pairs of each head's values turned by an angle that grows with the token's
// position, theta = position * freq[j] for pair j,
//   (a, b) -> factor * (a cos(theta) - b sin(theta), a sin(theta) + b cos(theta)),
// the rest of the head copied.  The transpose of a rotation is the rotation back, so the backward
// pass is the same with -theta.
//
// Pages: Atlas inference glm5next_dsa/tp.rs, shard plan: q_b_proj and kv_a_proj_with_mqa carry the
// positional part of queries and keys; the indexer's own queries and keys take positions too.
//
// Angles.  position * freq in fp32 is off by half a radian at a position of 2^23; here it is taken
// in 64 bits as turns (theta / 2 pi), of which the whole ones are dropped, and sine and cosine are
// then fp32's of what is left.  A token's angles are shared by its heads: a workgroup finds
// those of its rows once and keeps cosine and sine, times factor, in LDS.
//
// HBM-bound: 6 flops a rotated value against 2 to 8 bytes.  32768 rows of 32 heads of 128 in bf16, half of each
// turned: 97.5 us, 5.5 TB/s (a copy of as many bytes 99 us, 5.4; last-level cache holds part of both, a copy of
// 2 GiB moves 4.8 to 5.0); 16 heads of 128 in fp32 97; 8192 rows of 16 heads of 192, 64 of them turned, both
// ways: 42.8 us, 4.7 TB/s; 8 rows of 32 heads: 8.3 us, which is the host's call (the kernel takes 3.5).
// A thread turns vectors of V elements, the widest up to 16 bytes that divides every offset: a vector of
// each half, or, where pairs are neighbours, one vector of whole pairs.  The copied part goes by the same width, so
// that what no vector divides is slow throughout.  The first shape with rows a few elements further apart: 8
// more 104 us, 4 more 123, 2 more 194, 5 more 296; with 9 pairs 327; in fp32 with 5 more 176.
#include <algorithm>

#include "layer_internal.h"

// (both elements of a pair take the same rounding steps whichever kernel turns them)
#pragma clang fp contract(off)

namespace kpool {
namespace {

constexpr int kRotaryThreads = 256, kRotaryAngles = 2048;  // of a workgroup

// n / d for n < 2^16 and d <= 2^16: mul = ceil(2^32 / d) (0 for d = 1)
struct Divide {
  uint32_t d, mul;
};
Divide divide_by(int d) { return {(uint32_t)d, d > 1 ? (uint32_t)(((uint64_t(1) << 32) + d - 1) / d) : 0}; }
__device__ inline uint32_t quotient(uint32_t n, const Divide &d) { return d.mul ? __umulhi(n, d.mul) : n; }

struct RotaryArgs {
  const void *x;
  void *y;
  const int32_t *positions;
  const double *freqs;
  int64_t xs, ys, rows;
  int heads, D, begin, pairs;
  float factor, sine;   // (sine: factor, with the direction's sign)
  int nrows, nheads, hblocks;  // of a workgroup; workgroups that share a row
  Divide units_row, units_head;
  int turned, before;   // units of a head: the rotated ones come first; copied vectors before `begin`
};

__device__ inline float to_float(float x) { return x; }
__device__ inline float to_float(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ inline void from_float(float &y, float x) { y = x; }
__device__ inline void from_float(uint16_t &y, float x) { y = (uint16_t)pack_bf16(x, 0.0f); }

template <class T, int V>
struct alignas(sizeof(T) * V) Vector {
  T v[V];
};

// T: float, or uint16_t for bf16's bits.  NEAR: a unit is a vector of V / 2 pairs of neighbours; else
// two vectors, `apart` elements from one another, whose elements pair up.
template <class T, int V, bool NEAR>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(RotaryArgs a, int apart, int step) {
  extern __shared__ float2 turn[];  // [nrows][pairs]: cosine and sine
  const int64_t row0 = (int64_t)(blockIdx.x / a.hblocks) * a.nrows;
  const int head0 = (int)(blockIdx.x % a.hblocks) * a.nheads;
  const int nrows = (int)(a.rows - row0 < a.nrows ? a.rows - row0 : a.nrows);
  const int nheads = min(a.nheads, a.heads - head0);
  for (int i = threadIdx.x; i < nrows * a.pairs; i += kRotaryThreads) {
    const int r = i / a.pairs, j = i - r * a.pairs;
    double t = (double)a.positions[row0 + r] * (a.freqs[j] * 0.15915494309189533577);  // 1 / (2 pi)
    t -= rint(t);
    float s, c;
    sincospif(2.0f * (float)t, &s, &c);
    turn[i] = make_float2(a.factor * c, a.sine * s);
  }
  __syncthreads();
  using Vec = Vector<T, V>;
  const uint32_t units = (uint32_t)nrows * a.units_row.d;
  for (uint32_t u = threadIdx.x; u < units; u += kRotaryThreads) {
    const uint32_t r = quotient(u, a.units_row), in_row = u - r * a.units_row.d;
    const uint32_t h = quotient(in_row, a.units_head), unit = in_row - h * a.units_head.d;
    if ((int)h >= nheads) continue;
    const int64_t head = (int64_t)(head0 + h) * a.D;
    const T *x = (const T *)a.x + (row0 + r) * a.xs + head;
    T *y = (T *)a.y + (row0 + r) * a.ys + head;
    const int c = (int)unit - a.turned;  // (from 0 on: copied)
    const float2 *t = turn + r * a.pairs + unit * (NEAR ? V / 2 : V);
    int at = c < a.before ? c * V : a.begin + 2 * a.pairs + (c - a.before) * V;
    if constexpr (NEAR) {
      // (one load for turned and copied units alike: a wave holds both, and would wait for two in turn; 8192
      // rows of 16 heads of 192, 64 of them turned, both ways: 62.8 us, so 47.7)
      if (c < 0) at = a.begin + (int)unit * V;
      Vec v = *(const Vec *)(x + at);
      if (c < 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 cs = t[i / 2];
          const float p = to_float(v.v[i]), q = to_float(v.v[i + 1]);
          from_float(v.v[i], p * cs.x - q * cs.y);
          from_float(v.v[i + 1], p * cs.y + q * cs.x);
        }
      }
      *(Vec *)(y + at) = v;
    } else if (c < 0) {
      at = a.begin + (int)unit * step;
      const Vec v0 = *(const Vec *)(x + at), v1 = *(const Vec *)(x + at + apart);
      Vec w0, w1;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 cs = t[i];
        const float p = to_float(v0.v[i]), q = to_float(v1.v[i]);
        from_float(w0.v[i], p * cs.x - q * cs.y);
        from_float(w1.v[i], p * cs.y + q * cs.x);
      }
      *(Vec *)(y + at) = w0;
      *(Vec *)(y + at + apart) = w1;
    } else {
      *(Vec *)(y + at) = *(const Vec *)(x + at);
    }
  }
}

template <class T, int V, bool NEAR>
hipError_t launch_rotary_v(RotaryArgs a, bool interleaved, bool in_place, int64_t *threads, hipStream_t st) {
  // a rotated unit: V / 2 pairs of neighbours, or V pairs `apart` from their partners
  const int step = NEAR ? V : interleaved ? 2 : V, apart = interleaved ? 1 : a.pairs;
  a.turned = NEAR ? 2 * a.pairs / V : a.pairs / V;
  a.before = a.begin / V;
  const int copied = in_place ? 0 : (a.D - 2 * a.pairs) / V;
  const int units_head = a.turned + copied;
  // heads of a workgroup, evened out over the workgroups of a row, then rows: 4 units a thread.  (8192 rows of 16
  // heads of 192, 64 of them turned, both ways, and 32768 rows of 32 heads of 128: 16 units a thread 45.5 and
  // 115 us, 8 43.0 and 110, 4 40.3 and 99.1, 2 40.7 and 97.4, 1 50.0 and 109.)
  constexpr int kUnits = 4 * kRotaryThreads;
  const int nheads = std::max(1, std::min(a.heads, kUnits / units_head));
  a.hblocks = (a.heads + nheads - 1) / nheads;
  a.nheads = (a.heads + a.hblocks - 1) / a.hblocks;
  const int units_row = a.nheads * units_head;
  a.nrows = std::max(1, std::min({64, kUnits / units_row, kRotaryAngles / a.pairs}));
  a.units_row = divide_by(units_row), a.units_head = divide_by(units_head);
  const int64_t blocks = (a.rows + a.nrows - 1) / a.nrows * a.hblocks;
  if (threads) {
    *threads = blocks * kRotaryThreads;
    return hipSuccess;
  }
  hipLaunchKernelGGL((rotary_kernel<T, V, NEAR>), dim3((unsigned)blocks), dim3(kRotaryThreads),
                     (size_t)a.nrows * a.pairs * sizeof(float2), st, a, apart, step);
  return hipGetLastError();
}

template <class T>
hipError_t launch_rotary_t(const RotaryArgs &a, bool interleaved, bool in_place, int64_t *threads, hipStream_t st) {
  // what every vector's offset is a multiple of
  const uint64_t parts = (uint64_t)a.D | (uint64_t)a.begin | (uint64_t)(interleaved ? 2 * a.pairs : a.pairs) |
                         (a.rows > 1 ? (uint64_t)a.xs | (uint64_t)a.ys : 0) |
                         ((uintptr_t)a.x | (uintptr_t)a.y) / sizeof(T);
  constexpr int kMost = 16 / sizeof(T);
  int v = kMost;
  while (parts & (v - 1)) v /= 2;
  if constexpr (kMost == 8)
    if (v == 8)
      return interleaved ? launch_rotary_v<T, 8, true>(a, true, in_place, threads, st)
                         : launch_rotary_v<T, 8, false>(a, false, in_place, threads, st);
  if (v == 4)
    return interleaved ? launch_rotary_v<T, 4, true>(a, true, in_place, threads, st)
                       : launch_rotary_v<T, 4, false>(a, false, in_place, threads, st);
  if (v == 2)
    return interleaved ? launch_rotary_v<T, 2, true>(a, true, in_place, threads, st)
                       : launch_rotary_v<T, 2, false>(a, false, in_place, threads, st);
  return launch_rotary_v<T, 1, false>(a, interleaved, in_place, threads, st);
}

}  // namespace

namespace {

// Launches, or counts the launch's threads.
hipError_t rotary_call(const RotaryCall &c, int64_t *threads, hipStream_t st) {
  RotaryArgs a{};
  a.x = c.x, a.y = c.y, a.positions = c.positions, a.freqs = c.freqs;
  a.xs = c.x_stride, a.ys = c.y_stride, a.rows = c.rows;
  a.heads = c.heads, a.D = c.D, a.begin = c.begin, a.pairs = c.pairs;
  a.factor = c.factor, a.sine = c.inverse ? -c.factor : c.factor;
  const bool in_place = c.x == c.y;
  return c.f32 ? launch_rotary_t<float>(a, c.interleaved, in_place, threads, st)
               : launch_rotary_t<uint16_t>(a, c.interleaved, in_place, threads, st);
}

}  // namespace

// (a head of at most 1024 values keeps a workgroup's units below 2^16 and its angles within 16 KiB)
int64_t rotary_threads(const RotaryCall &c) {
  int64_t n = 0;
  (void)rotary_call(c, &n, nullptr);
  return n;
}

hipError_t launch_rotary(const RotaryCall &c, hipStream_t st) { return rotary_call(c, nullptr, st); }

}  // namespace kpool
