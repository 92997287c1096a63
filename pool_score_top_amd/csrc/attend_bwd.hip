// Gradients of the attention over whole keys (attend.hip).  With P_ij = exp(scale q_i k_j -
// lse_i) over what row i sees and delta_i = sum_d do_id o_id (= sum_j P_ij (do_i v_j)):
//   dV_j = sum_i P_ij do_i          dP_ij = do_i v_j      dS_ij = P_ij (dP_ij - delta_i)
//   dK_j = scale sum_i dS_ij q_i    dQ_i = scale sum_j dS_ij k_j
//
// Three kernels: the rows' lse (base 2) and delta laid out along the virtual rows; dK and dV
// with the keys in registers and the rows walked; dQ with the rows in registers and the keys
// walked.  S and dP are thus computed twice (7 matrix products instead of 5), and in return
// no sum crosses workgroups through atomics: the same call gives the same bits, and the
// gradients of shared key heads add up over their G query heads in registers, because the
// walked axis is the virtual rows.  P and dS are rounded to bf16 for their products (as the
// outputs are); P, dP, dS and all sums are fp32.
//
// Each kernel orients S so that its result registers are the next product's B operand: S^T
// [keys, rows] where rows stay (dQ^T = K^T dS^T), S [rows, keys] where keys stay (dV^T =
// dO^T P, dK^T = Q^T dS).
//
// Where the staying axis gives too few workgroups, the walked axis is split; the parts are
// summed in fp32 in a fixed order by a fourth kernel.
#include <type_traits>

#include "attend_tile.h"

namespace kpool {
namespace {

struct BwdArgs {
  const uint16_t *q, *k, *v, *d_o, *o;
  int64_t qs, ks, vs;
  const float *lse;
  const int32_t *cu_q, *cu_k;
  int nseq, Hq, Hkv, D;
  int64_t Tq, Tk;
  float scale, scale_log2;
  float *lse2, *delta;  // [Hkv][Tq * G]: lse log2 e (+inf for a row without keys), delta
  int64_t ktiles, qtiles;
  int ksplit, qsplit;   // parts of the walked axis: rows (for dK, dV), keys (for dQ)
  int kchunk, qchunk;   // their sizes: virtual rows (multiple of 32), keys (multiple of 64)
  uint16_t *dq, *dk, *dv;
  float *part;          // fp32 parts, used by one kernel and its sum at a time
};

// One (row, head) per 16 lanes.
__global__ __launch_bounds__(256) void bwd_stat_kernel(BwdArgs a) {
  const int64_t at = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (at >= a.Tq * a.Hq) return;  // (16 lanes together)
  const int c = (threadIdx.x & 15) * 8;
  float s = 0.0f;
  if (c < a.D) {
    const uint4 x = *reinterpret_cast<const uint4 *>(a.o + at * a.D + c);
    const uint4 y = *reinterpret_cast<const uint4 *>(a.d_o + at * a.D + c);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(w[i] << 16), s);
      s = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(w[i] & 0xFFFF0000u), s);
    }
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 15) == 0) {
    const int G = a.Hq / a.Hkv;
    const int64_t row = at / a.Hq;
    const int head = (int)(at - row * a.Hq);
    const int64_t to = (int64_t)(head / G) * a.Tq * G + row * G + head % G;
    const float l = a.lse[at];
    a.lse2[to] = l > -__builtin_inff() ? l * kLog2e : __builtin_inff();
    a.delta[to] = s;
  }
}

// Writes a lane's column of a transposed result x^T [DP, 32]: row `row` of out (bf16, D
// wide), or of a part (fp32).
template <int DP>
__device__ inline void write_cols(const f32x16 (&x)[DP / 32], float mul, uint16_t *out, float *part,
                                  int64_t row, int D, int lane) {
  const int h = lane >> 5;
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int d = dt * 32 + 2 * i + 4 * h;
      if (d >= D) continue;
      if (part)
        *reinterpret_cast<float4 *>(part + row * D + d) =
            make_float4(x[dt][i] * mul, x[dt][i + 1] * mul, x[dt][i + 2] * mul, x[dt][i + 3] * mul);
      else
        *reinterpret_cast<uint2 *>(out + row * D + d) =
            make_uint2(pack_bf16(x[dt][i] * mul, x[dt][i + 1] * mul),
                       pack_bf16(x[dt][i + 2] * mul, x[dt][i + 3] * mul));
    }
}

template <int DP>
__device__ inline void load_frag(bf16x8 (&f)[DP / 16], const uint16_t *row, int D, int lane) {
#pragma unroll
  for (int ks = 0; ks < DP / 16; ++ks) {
    const int d = ks * 16 + (lane >> 5) * 8;
    uint4 z = make_uint4(0, 0, 0, 0);
    if (row && d < D) z = *reinterpret_cast<const uint4 *>(row + d);
    f[ks] = __builtin_bit_cast(bf16x8, z);
  }
}

// dK and dV: 4 waves of 32 keys; tiles of 32 virtual rows (q, do and their statistics) pass
// through LDS.
template <int DP>
__global__ __launch_bounds__(256, 1) void bwd_keys_kernel(BwdArgs a) {
  using S = Keys<DP>;
  constexpr int BR = 32, NW = 4, TILE = BR * S::ROWB, BUFB = 2 * TILE + 256;
  constexpr int PER = BR / S::REGION_ROWS / NW > 0 ? BR / S::REGION_ROWS / NW : 1;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  int64_t idx = blockIdx.x;
  const int kvh = (int)(idx % a.Hkv);
  idx /= a.Hkv;
  const int split = (int)(idx % a.ksplit);
  // (tiles of keys: the roles of the two length arrays are exchanged)
  const TileAt at = find_tile(a.cu_k, a.cu_q, a.nseq, 1, NW * 32, idx / a.ksplit, lane);
  if (at.seq < 0) return;
  const int k_start = at.q_start, Lk = at.Lq, q_start = at.k_start, Lq = at.Lk;
  const int key = at.n0 + wave * 32 + (lane & 31);  // this lane's key, of the sequence
  const bool live = key < Lk;
  bf16x8 kf[S::KS], vf[S::KS];
  load_frag<DP>(kf, live ? a.k + ((int64_t)k_start + key) * a.ks + (int64_t)kvh * a.D : nullptr, a.D, lane);
  load_frag<DP>(vf, live ? a.v + ((int64_t)k_start + key) * a.vs + (int64_t)kvh * a.D : nullptr, a.D, lane);
  f32x16 dk[S::DT], dv[S::DT];
#pragma unroll
  for (int dt = 0; dt < S::DT; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) dk[dt][i] = dv[dt][i] = 0.0f;

  // virtual rows that see the first key of the workgroup, cut to this part
  const int nvirt = Lq * G, off = Lk - Lq;
  const int first = (int)min<int64_t>(nvirt, (int64_t)max(0, at.n0 - off) * G);
  const int n_lo = max(first / 32 * 32, split * a.kchunk);
  const int n_hi = (int)min<int64_t>(nvirt, (int64_t)split * a.kchunk + a.kchunk);
  const int ntile = n_hi > n_lo ? (n_hi - n_lo + BR - 1) / BR : 0;
  // this lane's key is seen from virtual row `from` on; every key of the wave from `all` on
  const int from = live ? (int)min<int64_t>(nvirt, (int64_t)max(0, key - off) * G) : nvirt;
  const int wave_first = at.n0 + wave * 32;
  const int none = wave_first < Lk ? (int)min<int64_t>(nvirt, (int64_t)max(0, wave_first - off) * G) : nvirt;
  const int all = wave_first + 31 < Lk ? (int)min<int64_t>(nvirt, (int64_t)max(0, wave_first + 31 - off) * G)
                                       : nvirt;

  const uint16_t *qb = a.q + (int64_t)q_start * a.qs + (int64_t)kvh * G * a.D;
  const int64_t dos = (int64_t)a.Hq * a.D;
  const uint16_t *dob = a.d_o + (int64_t)q_start * dos + (int64_t)kvh * G * a.D;
  const float *stat = (lane < 32 ? a.lse2 : a.delta) + (int64_t)kvh * a.Tq * G + (int64_t)q_start * G;
  // rows of this lane's loads: token and head of the group, moved on by 32 virtual rows a tile
  int tok[PER], g[PER];
  const int sub = lane * 16 / S::ROWB;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int n = n_lo + (wave + i * NW) * S::REGION_ROWS + sub;
    tok[i] = n / G;
    g[i] = n - tok[i] * G;
  }
  const int step_tok = BR / G, step_g = BR - step_tok * G;
  auto load = [&](int tile, int buf) {
#if defined(__HIP_DEVICE_COMPILE__)
    unsigned char *at_lds = lds + buf * BUFB;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int region = wave + i * NW;
      const int row = region * S::REGION_ROWS + sub;
      const int chunk = min((lane & (DP / 8 - 1)) ^ S::swz(row), a.D / 8 - 1);
      // (rows past the last one take it again; they count for nothing)
      const bool in = tok[i] < Lq;
      const int64_t t = in ? tok[i] : Lq - 1, hd = (in ? g[i] : G - 1) * a.D + chunk * 8;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(qb + t * a.qs + hd),
                                       (KPOOL_LDS void *)(at_lds + region * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(dob + t * dos + hd),
                                       (KPOOL_LDS void *)(at_lds + TILE + region * 1024), 16, 0, 0);
      tok[i] += step_tok, g[i] += step_g;
      if (g[i] >= G) g[i] -= G, ++tok[i];
    }
    if (wave == 0) {
      const int n = min(n_lo + tile * BR + (lane & 31), nvirt - 1);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(stat + n),
                                       (KPOOL_LDS void *)(at_lds + 2 * TILE), 4, 0, 0);
    }
#endif
  };
  Frag<DP> f;
  f.init(lds_offset(lds), lane);
  const uint32_t st0 = lds_offset(lds) + 2 * TILE + (lane >> 5) * 16;
  auto step = [&](int j, auto buf_c) {
    constexpr int BUF = decltype(buf_c)::value;
    constexpr uint32_t SQ = BUF * BUFB, SO = SQ + TILE;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    if (j + 1 < ntile) load(j + 1, BUF ^ 1);
    const int n0 = n_lo + j * BR;
    if (n0 + BR <= none) return;  // (the whole wave) no row of the tile sees a key of the wave
    f32x16 s = {}, dp = {};
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) s = mfma(f.rows(SQ, ks), kf[ks], s);
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) dp = mfma(f.rows(SO, ks), vf[ks], dp);
    float lse[16], delta[16];
    typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f32x4 x = *(KPOOL_LDS const f32x4 *)(uintptr_t)(st0 + SQ + b * 32);
      const f32x4 y = *(KPOOL_LDS const f32x4 *)(uintptr_t)(st0 + SQ + 128 + b * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) lse[4 * b + i] = x[i], delta[4 * b + i] = y[i];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = exp2f_fast(fmaf(s[i], a.scale_log2, -lse[i]));
    if (n0 < all || n0 + BR > n_hi) {
      const int lo = from - n0 - 4 * (lane >> 5), hi = n_hi - n0 - 4 * (lane >> 5);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 8 * (i / 4) + i % 4;
        if (r < lo || r >= hi) s[i] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) dp[i] = s[i] * (dp[i] - delta[i]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const bf16x8 p = as_operand(s, c), ds = as_operand(dp, c);
#pragma unroll
      for (int dt = 0; dt < S::DT; ++dt) dv[dt] = mfma(f.cols(SO + c * 16 * S::ROWB, dt), p, dv[dt]);
#pragma unroll
      for (int dt = 0; dt < S::DT; ++dt) dk[dt] = mfma(f.cols(SQ + c * 16 * S::ROWB, dt), ds, dk[dt]);
    }
  };
  if (ntile > 0) load(0, 0);
  for (int j = 0; j < ntile; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < ntile) step(j + 1, std::integral_constant<int, 1>{});
  }
  if (!live) return;
  const int64_t row = ((int64_t)k_start + key) * a.Hkv + kvh, rows = a.Tk * a.Hkv;
  float *part = a.ksplit > 1 ? a.part + (int64_t)split * 2 * rows * a.D : nullptr;
  write_cols<DP>(dk, a.scale, a.dk, part, row, a.D, lane);
  write_cols<DP>(dv, 1.0f, a.dv, part ? part + rows * a.D : nullptr, row, a.D, lane);
}

// dQ: NW waves of 32 virtual rows; key tiles of 64 pass through LDS, as in the forward pass.
template <int DP, int NW>
__global__ __launch_bounds__(NW * 64) void bwd_rows_kernel(BwdArgs a) {
  using S = Keys<DP>;
  constexpr int BK = 64, BQ = NW * 32, TILE = BK * S::ROWB;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  int64_t idx = blockIdx.x;
  const int kvh = (int)(idx % a.Hkv);
  idx /= a.Hkv;
  const int split = (int)(idx % a.qsplit);
  const TileAt at = find_tile(a.cu_q, a.cu_k, a.nseq, G, BQ, a.qtiles - 1 - idx / a.qsplit, lane);
  if (at.seq < 0) return;
  const int nrows = min(BQ, at.Lq * G - at.n0);
  const int t1 = (at.n0 + nrows - 1) / G + at.Lk - at.Lq;
  const int k_lo = split * a.qchunk, k_hi = (int)min<int64_t>(t1 + 1, (int64_t)k_lo + a.qchunk);
  const uint16_t *kb = (const uint16_t *)uniform_ptr(a.k + (int64_t)at.k_start * a.ks + (int64_t)kvh * a.D);
  const uint16_t *vb = (const uint16_t *)uniform_ptr(a.v + (int64_t)at.k_start * a.vs + (int64_t)kvh * a.D);
  const int n = at.n0 + wave * 32 + (lane & 31);
  const bool live = wave * 32 + (lane & 31) < nrows;
  const int tok = n / G, head = kvh * G + (n - tok * G);
  const int t = tok + at.Lk - at.Lq;
  const int wave_rows = min(32, nrows - wave * 32);
  const int w0 = (at.n0 + wave * 32) / G + at.Lk - at.Lq;
  const int w1 = wave_rows > 0 ? (at.n0 + wave * 32 + wave_rows - 1) / G + at.Lk - at.Lq : -1;
  const int64_t row = ((int64_t)at.q_start + tok) * a.Hq + head;
  bf16x8 qf[S::KS], dof[S::KS];
  load_frag<DP>(qf, live ? a.q + ((int64_t)at.q_start + tok) * a.qs + (int64_t)head * a.D : nullptr, a.D, lane);
  load_frag<DP>(dof, live ? a.d_o + row * a.D : nullptr, a.D, lane);
  const int64_t stat = (int64_t)kvh * a.Tq * G + (int64_t)at.q_start * G + n;
  const float lse = live ? a.lse2[stat] : __builtin_inff(), delta = live ? a.delta[stat] : 0.0f;
  f32x16 dq[S::DT];
#pragma unroll
  for (int dt = 0; dt < S::DT; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) dq[dt][i] = 0.0f;

  Frag<DP> f;
  f.init(lds_offset(lds), lane);
  KeyLoader<DP, BK, NW> keys;
  keys.init(wave, lane, a.D);
  const int ntile = k_hi > k_lo ? (k_hi - k_lo + BK - 1) / BK : 0;
  auto load = [&](int tile, int buf) {
    const int k0 = k_lo + tile * BK;
    keys.load(kb + (int64_t)k0 * a.ks, a.ks, at.Lk - 1 - k0, lds + buf * 2 * TILE);
    keys.load(vb + (int64_t)k0 * a.vs, a.vs, at.Lk - 1 - k0, lds + buf * 2 * TILE + TILE);
  };
  auto step = [&](int j, auto buf_c) {
    constexpr int BUF = decltype(buf_c)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    if (j + 1 < ntile) load(j + 1, BUF ^ 1);
    const int k0 = k_lo + j * BK;
    if (k0 > w1) return;
    const bool masked = k0 + BK - 1 > w0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      constexpr uint32_t SK = BUF * 2 * TILE, SV = SK + TILE;
      const uint32_t down = half * 32 * S::ROWB;
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) s = mfma(f.rows(SK + down, ks), qf[ks], s);
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) dp = mfma(f.rows(SV + down, ks), dof[ks], dp);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = exp2f_fast(fmaf(s[i], a.scale_log2, -lse));
      if (masked) {
        const int hi = t - k0 - half * 32 - 4 * (lane >> 5);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (8 * (i / 4) + i % 4 > hi) s[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] *= dp[i] - delta;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bf16x8 ds = as_operand(s, c);
#pragma unroll
        for (int dt = 0; dt < S::DT; ++dt) dq[dt] = mfma(f.cols(SK + down + c * 16 * S::ROWB, dt), ds, dq[dt]);
      }
    }
  };
  if (ntile > 0) load(0, 0);
  for (int j = 0; j < ntile; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < ntile) step(j + 1, std::integral_constant<int, 1>{});
  }
  if (!live) return;
  float *part = a.qsplit > 1 ? a.part + (int64_t)split * a.Tq * a.Hq * a.D : nullptr;
  write_cols<DP>(dq, a.scale, a.dq, part, row, a.D, lane);
}

// out[e] = sum over parts s of part[s * pitch + e], in order; 4 elements a thread.
__global__ __launch_bounds__(256) void bwd_sum_kernel(const float *__restrict__ part, int64_t pitch,
                                                      int nsplit, int64_t count,
                                                      uint16_t *__restrict__ out) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= count) return;
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < nsplit; ++s) {
    const float4 x = *reinterpret_cast<const float4 *>(part + s * pitch + e);
    t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
  }
  *reinterpret_cast<uint2 *>(out + e) = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
}

hipError_t launch_sum(const float *part, int64_t pitch, int nsplit, int64_t count, uint16_t *out,
                      hipStream_t st) {
  if (count == 0) return hipSuccess;
  hipLaunchKernelGGL(bwd_sum_kernel, dim3((unsigned)((count / 4 + 255) / 256)), dim3(256), 0, st, part,
                     pitch, nsplit, count, out);
  return hipGetLastError();
}

constexpr int kBwdWaves = 8;

template <int DP>
hipError_t launch_bwd_t(const BwdArgs &a, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (a.Tq > 0) {
    hipLaunchKernelGGL(bwd_stat_kernel, dim3((unsigned)((a.Tq * a.Hq + 15) / 16)), dim3(256), 0, st, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.Tk > 0) {
    hipLaunchKernelGGL(bwd_keys_kernel<DP>, dim3((unsigned)(a.ktiles * a.ksplit * a.Hkv)), dim3(256),
                       2 * (2 * 32 * DP * 2 + 256), st, a);
    e = hipGetLastError();
    const int64_t count = a.Tk * a.Hkv * a.D;
    if (e == hipSuccess && a.ksplit > 1) e = launch_sum(a.part, 2 * count, a.ksplit, count, a.dk, st);
    if (e == hipSuccess && a.ksplit > 1) e = launch_sum(a.part + count, 2 * count, a.ksplit, count, a.dv, st);
    if (e != hipSuccess) return e;
  }
  if (a.Tq > 0) {
    const size_t lds = 4 * 64 * DP * 2;
    hipLaunchKernelGGL((bwd_rows_kernel<DP, kBwdWaves>), dim3((unsigned)(a.qtiles * a.qsplit * a.Hkv)),
                       dim3(kBwdWaves * 64), lds, st, a);
    e = hipGetLastError();
    const int64_t count = a.Tq * a.Hq * a.D;
    if (e == hipSuccess && a.qsplit > 1) e = launch_sum(a.part, count, a.qsplit, count, a.dq, st);
  }
  return e;
}

int64_t up_to(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Parts of a walked axis of at most `longest`, for tiles that walk `walked` in all: enough
// for two workgroups a CU, each part `least` long or more.
void split_walk(int64_t walked, int64_t longest, int64_t least, int *split, int *chunk) {
  const int64_t c = up_to(walked / 512 > least ? walked / 512 : least, 64);
  const int64_t n = (longest + c - 1) / c;
  *split = n > 1 ? (int)n : 1;
  *chunk = n > 1 ? (int)c : 0x7FFFFF00;
}

}  // namespace

BwdPlan plan_attend_bwd(const int32_t *cu_q, const int32_t *cu_k, int nseq, int Hq, int Hkv) {
  const int G = Hq / Hkv;
  BwdPlan p;
  p.ktiles = tile_start(cu_k[nseq], nseq, 1, 128);
  p.qtiles = tile_start(cu_q[nseq], nseq, G, kBwdWaves * 32);
  int64_t rows = 0, keys = 0, most_rows = 0, most_keys = 0, kt = 0, qt = 0;
  for (int s = 0; s < nseq; ++s) {
    const int64_t lq = (int64_t)(cu_q[s + 1] - cu_q[s]) * G, lk = cu_k[s + 1] - cu_k[s];
    const int64_t nk = (lk + 127) / 128, nq = (lq + kBwdWaves * 32 - 1) / (kBwdWaves * 32);
    rows += nk * lq, keys += nq * lk, kt += nk, qt += nq;
    if (lk > 0 && most_rows < lq) most_rows = lq;
    if (lq > 0 && most_keys < lk) most_keys = lk;
  }
  p.ksplit = p.qsplit = 1;
  p.kchunk = p.qchunk = 0x7FFFFF00;
  if (kt * Hkv < 256) split_walk(rows * Hkv, most_rows, 512, &p.ksplit, &p.kchunk);
  if (qt * Hkv < 256) split_walk(keys * Hkv, most_keys, 512, &p.qsplit, &p.qchunk);
  return p;
}

size_t attend_bwd_workspace(const BwdPlan &p, int64_t Tq, int64_t Tk, int Hq, int Hkv, int D) {
  const int64_t stat = up_to(Tq * Hq * 8, 16);
  const int64_t kpart = p.ksplit > 1 ? (int64_t)p.ksplit * 2 * Tk * Hkv * D * 4 : 0;
  const int64_t qpart = p.qsplit > 1 ? (int64_t)p.qsplit * Tq * Hq * D * 4 : 0;
  return (size_t)(stat + (kpart > qpart ? kpart : qpart));
}

hipError_t launch_attend_bwd(const AttendCall &c, const uint16_t *d_o, const BwdPlan &p, void *workspace,
                             uint16_t *dq, uint16_t *dk, uint16_t *dv, hipStream_t st) {
  BwdArgs a{};
  a.q = c.q, a.k = c.k, a.v = c.v, a.d_o = d_o, a.o = c.o, a.lse = c.lse;
  a.qs = c.q_stride, a.ks = c.k_stride, a.vs = c.v_stride;
  a.cu_q = c.cu_q, a.cu_k = c.cu_k, a.nseq = c.nseq, a.Hq = c.Hq, a.Hkv = c.Hkv, a.D = c.D;
  a.Tq = c.Tq, a.Tk = c.Tk;
  a.scale = c.scale, a.scale_log2 = c.scale * kLog2e;
  a.lse2 = (float *)workspace;
  a.delta = a.lse2 + c.Tq * c.Hq;
  a.part = (float *)((char *)workspace + up_to(c.Tq * c.Hq * 8, 16));
  a.ktiles = p.ktiles, a.qtiles = p.qtiles, a.ksplit = p.ksplit, a.qsplit = p.qsplit;
  a.kchunk = p.kchunk, a.qchunk = p.qchunk;
  a.dq = dq, a.dk = dk, a.dv = dv;
  return c.D <= 64 ? launch_bwd_t<64>(a, st) : launch_bwd_t<128>(a, st);
}

}  // namespace kpool
