// Attention of query rows over the keys they see: o = softmax(scale q k^T) v per head, and
// lse = log sum exp(scale q k^T), forward.
//
// Pages: Megatron-LM PR #8299 and SkyRL PR #2422 describe the selection as the step before
// sparse attention: each row then attends to the tokens selected for it.  The list kernel
// below reads such lists of token ids; the tile kernel (many rows) and the rows kernel (few)
// are the attention over everything before a row (dense layers, prompts no longer than the
// selection's width).
//
// One pass over the keys with the running maximum m and sum l of the softmax:
//   m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),
//   O' = O e^(m - m') + sum_j e^(s_j - m') v_j,   o = O / l,  lse = m + ln l
// kept in fp32 in base 2 (s = q k^T scale log2 e).  e^(s - m) is rounded to bf16 for the
// matrix product with v (relative 2^-9 on average, as the output's own rounding; it averages
// over the keys); l sums the unrounded values.  m follows the maximum only when that rises by
// more than 8 (a factor of 256 in base 2): the exact shift cancels in O / l, values up to
// 2^8 lose nothing in bf16 or fp32, and most tiles then leave O alone.
//
// S^T = K Q^T and O^T = V^T P^T: a lane owns one query row, so the softmax needs one
// exchange between the wave's halves and P feeds the second product from registers.
#include <type_traits>

#include "attend_tile.h"

namespace kpool {
namespace {

// Waves of the tile kernel, 32 rows each.  With 4, two workgroups fit a CU, but each loads its
// own key tiles: a 16384-token prompt then takes 1345 us instead of 1028.
constexpr int kTileWaves = 8;

struct AttendArgs {
  const uint16_t *q, *k, *v;
  int64_t qs, ks, vs;  // elements between tokens
  const int32_t *cu_q, *cu_k;
  int nseq, Hq, Hkv, D;
  float scale_log2;
  int64_t ntiles;
  int nsplit;
  int chunk;  // keys (or list entries) of a split, a multiple of 128
  const int32_t *ids;
  int width;
  bool by_place;
  uint16_t *o;
  float *lse;
  float *part_o, *part_lse;  // [nsplit][Tq * Hq][D], [nsplit][Tq * Hq]
  int64_t rows;              // Tq * Hq
  TileTable table;
  // expanded latent attention: the keys' positional part, the heads' strides, a query head's values
  const uint16_t *pe;
  int64_t pes, kh, vh;
  int P, QD;
};

// One wave's 32 query rows: fragments, running softmax and output.  PP: values of the keys' and queries'
// positional part, which has no values beside it (0 for none).
template <int DP, int PP = 0>
struct Rows {
  using S = Keys<DP>;
  static constexpr int PS = PP / 16;  // contraction steps over it
  static constexpr int ROWS = 32, VALUES = 16;  // of a fragment of o: its rows, a lane's values
  bf16x8 q[S::KS + PS];
  f32x16 o[S::DT];
  float m, l;  // base 2; l is this lane half's part

  // where value i of o[dt] lies in the head dim
  static __device__ inline int place(int dt, int i, int lane) {
    return dt * 32 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
  }
  // the row's sum over its lanes
  __device__ inline float sum() const { return l + other_half(l); }

  // row: this lane's query (l % 32), null for none; P: its positional values, behind the D others
  __device__ inline void init(const uint16_t *row, int D, int lane, int P = 0) {
#pragma unroll
    for (int ks = 0; ks < PS; ++ks) {
      const int d = ks * 16 + (lane >> 5) * 8;
      uint4 z = make_uint4(0, 0, 0, 0);
      if (row && d < P) z = *reinterpret_cast<const uint4 *>(row + D + d);
      q[S::KS + ks] = __builtin_bit_cast(bf16x8, z);
    }
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) {
      const int d = ks * 16 + (lane >> 5) * 8;
      uint4 z = make_uint4(0, 0, 0, 0);
      if (row && d < D) z = *reinterpret_cast<const uint4 *>(row + d);
      q[ks] = __builtin_bit_cast(bf16x8, z);
    }
#pragma unroll
    for (int dt = 0; dt < S::DT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[dt][i] = 0.0f;
    m = -__builtin_inff();
    l = 0.0f;
  }

  // S of the BK keys of a tile at LDS offset sk past the addresses of `f`
  template <int BK>
  using KeyFrag = bf16x8[BK / 32][S::KS];
  template <int BK>
  static __device__ inline void read_keys(const Frag<DP> &f, uint32_t sk, KeyFrag<BK> &kr) {
#pragma unroll
    for (int sub = 0; sub < BK / 32; ++sub)
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) kr[sub][ks] = f.rows(sk + sub * 32 * S::ROWB, ks);
  }
  template <int BK>
  __device__ inline void scores(const KeyFrag<BK> &kr, f32x16 (&s)[BK / 32]) const {
#pragma unroll
    for (int sub = 0; sub < BK / 32; ++sub) {
      f32x16 t = {};
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) t = mfma(kr[sub][ks], q[ks], t);
      s[sub] = t;
    }
  }

  // S to P, with the running maximum and sum.  Where `masked` (the same for the wave), key
  // sub * 32 + r counts only if visible(sub, r).
  template <int SUBS, class F>
  __device__ inline void weights(f32x16 (&s)[SUBS], float c, int lane, bool masked, F &&visible) {
    if (masked) {
#pragma unroll
      for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!visible(sub, 8 * (i / 4) + 4 * (lane >> 5) + i % 4)) s[sub][i] = -__builtin_inff();
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[sub][i]);
    top = fmaxf(top, other_half(top)) * c;
    if (__any(top > m + 8.0f)) {  // (m = -inf: any visible key)
      const float up = fmaxf(top, m);
      const float a = up > m ? exp2f_fast(m - up) : 1.0f;  // m = -inf gives 0
      m = up;
      l *= a;
#pragma unroll
      for (int dt = 0; dt < S::DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] *= a;
    }
    const float shift = m > -__builtin_inff() ? m : 0.0f;
#pragma unroll
    for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[sub][i] = exp2f_fast(fmaf(s[sub][i], c, -shift));
        l += s[sub][i];
      }
  }

  // O of the tile whose values lie at LDS offset sv
  template <int SUBS>
  __device__ inline void values(const Frag<DP> &f, uint32_t sv, const f32x16 (&p)[SUBS]) {
#pragma unroll
    for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
      for (int kc = 0; kc < 2; ++kc) {
        const bf16x8 w = as_operand(p[sub], kc);
#pragma unroll
        for (int dt = 0; dt < S::DT; ++dt)
          o[dt] = mfma(f.cols(sv + (sub * 32 + kc * 16) * S::ROWB, dt), w, o[dt]);
      }
  }
  // and of 32 keys whose values have been read
  using ValueFrag = bf16x8[2][S::DT];
  static __device__ inline void read_values(const Frag<DP> &f, uint32_t sv, ValueFrag &vr) {
#pragma unroll
    for (int kc = 0; kc < 2; ++kc)
#pragma unroll
      for (int dt = 0; dt < S::DT; ++dt) vr[kc][dt] = f.cols(sv + kc * 16 * S::ROWB, dt);
  }
  __device__ inline void values(const ValueFrag &vr, const f32x16 (&p)[1]) {
#pragma unroll
    for (int kc = 0; kc < 2; ++kc) {
      const bf16x8 w = as_operand(p[0], kc);
#pragma unroll
      for (int dt = 0; dt < S::DT; ++dt) o[dt] = mfma(vr[kc][dt], w, o[dt]);
    }
  }

  // The same with the positional part, whose tile lies at sp past the addresses of `fp`.  Its products come
  // first, and the keys' fragments are read beside them.
  template <int BK, class F>
  __device__ inline void add(const Frag<DP> &f, const Frag<PP> &fp, uint32_t sk, uint32_t sp, uint32_t sv, float c,
                             int lane, bool masked, F &&visible) {
    f32x16 s[BK / 32];
    bf16x8 pr[BK / 32][PS];
#pragma unroll
    for (int sub = 0; sub < BK / 32; ++sub)
#pragma unroll
      for (int ks = 0; ks < PS; ++ks) pr[sub][ks] = fp.rows(sp + sub * 32 * Keys<PP>::ROWB, ks);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int sub = 0; sub < BK / 32; ++sub) {
      bf16x8 kr[S::KS];
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) kr[ks] = f.rows(sk + sub * 32 * S::ROWB, ks);
      f32x16 t = {};
#pragma unroll
      for (int ks = 0; ks < PS; ++ks) t = mfma(pr[sub][ks], q[S::KS + ks], t);
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) t = mfma(kr[ks], q[ks], t);
      s[sub] = t;
    }
    weights(s, c, lane, masked, visible);
    values(f, sv, s);
  }

  template <int BK, class F>
  __device__ inline void add(const Frag<DP> &f, uint32_t sk, uint32_t sv, float c, int lane, bool masked,
                             F &&visible) {
    f32x16 s[BK / 32];
    KeyFrag<BK> kr;
    read_keys<BK>(f, sk, kr);
    __builtin_amdgcn_sched_barrier(0);  // (the reads go out together, ahead of what needs them)
    scores<BK>(kr, s);
    weights(s, c, lane, masked, visible);
    values(f, sv, s);
  }
};

// The same for up to 16 query rows, by products of 16 rows: 32 rows would be half empty.  o and
// S have a column l % 16 a lane, the keys of S and the head dim of o go over its four groups.
template <int DP>
struct Rows16 {
  using S = Keys16<DP>;
  static constexpr int ROWS = 16, VALUES = 4;
  bf16x8 q[S::KS];
  f32x4 o[S::DT];
  float m, l;

  static __device__ inline int place(int dt, int i, int lane) { return dt * 16 + 4 * (lane >> 4) + i; }
  __device__ inline float sum() const {
    const Pair t = row_pair(l);
    const float x = t.a + t.b;
    return x + other_half(x);
  }
  __device__ inline void init(const uint16_t *row, int D, int lane) {
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) {
      const int d = ks * 32 + (lane >> 4) * 8;
      uint4 z = make_uint4(0, 0, 0, 0);
      if (row && d < D) z = *reinterpret_cast<const uint4 *>(row + d);
      q[ks] = __builtin_bit_cast(bf16x8, z);
    }
#pragma unroll
    for (int dt = 0; dt < S::DT; ++dt) o[dt] = f32x4{};
    m = -__builtin_inff();
    l = 0.0f;
  }
  template <int BK>
  using KeyFrag = bf16x8[2][S::KS];
  template <int BK>
  static __device__ inline void read_keys(const Frag16<DP> &f, uint32_t sk, KeyFrag<BK> &kr) {
    static_assert(BK == 32, "one contraction of the second product");
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) kr[b][ks] = f.rows(sk + b * 16 * S::ROWB, ks);
  }
  template <int BK>
  __device__ inline void scores(const KeyFrag<BK> &kr, f32x4 (&s)[2]) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      s[b] = f32x4{};
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) s[b] = mfma(kr[b][ks], q[ks], s[b]);
    }
  }
  template <class F>
  __device__ inline void weights(f32x4 (&s)[2], float c, int lane, bool masked, F &&visible) {
    if (masked) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!visible(0, b * 16 + 4 * (lane >> 4) + i)) s[b][i] = -__builtin_inff();
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[b][i]);
    const Pair t = row_pair(top);
    top = fmaxf(t.a, t.b);
    top = fmaxf(top, other_half(top)) * c;
    if (__any(top > m + 8.0f)) {
      const float up = fmaxf(top, m);
      const float a = up > m ? exp2f_fast(m - up) : 1.0f;
      m = up;
      l *= a;
#pragma unroll
      for (int dt = 0; dt < S::DT; ++dt) o[dt] *= a;
    }
    const float shift = m > -__builtin_inff() ? m : 0.0f;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[b][i] = exp2f_fast(fmaf(s[b][i], c, -shift));
        l += s[b][i];
      }
  }
  using ValueFrag = bf16x8[S::DT];
  static __device__ inline void read_values(const Frag16<DP> &f, uint32_t sv, ValueFrag &vr) {
#pragma unroll
    for (int dt = 0; dt < S::DT; ++dt) vr[dt] = f.cols(sv, dt);
  }
  __device__ inline void values(const ValueFrag &vr, const f32x4 (&p)[2]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 w = {pack_bf16(p[0][0], p[0][1]), pack_bf16(p[0][2], p[0][3]), pack_bf16(p[1][0], p[1][1]),
                     pack_bf16(p[1][2], p[1][3])};
#pragma unroll
    for (int dt = 0; dt < S::DT; ++dt) o[dt] = mfma(vr[dt], __builtin_bit_cast(bf16x8, w), o[dt]);
  }
};

// Writes a row's output: the final one, or a split's part (in fp32, normalised by its own l).
template <class R>
__device__ inline void write_row(const AttendArgs &a, bool live, int64_t row, bool whole, int split, const R &r,
                                 int lane) {
  const float l = r.sum();  // (all lanes)
  if (!live) return;
  // (l is 0 where the row saw nothing; NaN goes through)
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const float lse = l == 0.0f ? -__builtin_inff() : (r.m + log2f(l)) * kLn2;
  float *part = a.part_o + ((int64_t)split * a.rows + row) * a.D;
  uint16_t *out = a.o + row * a.D;
#pragma unroll
  for (int dt = 0; dt < R::S::DT; ++dt)
#pragma unroll
    for (int i = 0; i < R::VALUES; i += 4) {
      const int d = R::place(dt, i, lane);
      if (d >= a.D) continue;
      const float x[4] = {r.o[dt][i] * inv, r.o[dt][i + 1] * inv, r.o[dt][i + 2] * inv, r.o[dt][i + 3] * inv};
      if (!whole) *reinterpret_cast<float4 *>(part + d) = make_float4(x[0], x[1], x[2], x[3]);
      else *reinterpret_cast<uint2 *>(out + d) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    }
  if (lane >= R::ROWS) return;
  if (!whole) a.part_lse[(int64_t)split * a.rows + row] = lse;
  else if (a.lse) a.lse[row] = lse;
}

// Many rows: NW waves of 32 virtual rows each share key tiles of 64.  8 waves and 64 KiB of
// tiles: one workgroup a CU, two waves a SIMD, so that one's softmax runs beside the other's
// matrix instructions.  A prompt of 16384 tokens, 16 heads over 2 of 128, 1.1 TFLOP, takes 983 to
// 1035 us (1.06 to 1.12 PFLOP/s; a 16384 library product reaches 1.3): bound by the matrix
// instructions at the clock that the card's power leaves, since with the softmax and the LDS reads
// left out it still takes 915 us (CUs busy 91% of the time, the pipe 58% of that).  A packed batch
// of 4097 to 1 tokens, 32 heads over 4: CUs 84%, the pipe 49%: shorter tiles, so a larger share goes
// to their starts and ends, beside which a CU has nothing else to run.
// Head dims above 64 run as 128: the blocks past D multiply zeros (8192 tokens, 16 heads over 2: D
// = 64 192 us, 80 258, 96 263, 128 272).
// With the positional part of expanded latent attention (PP = 64): its tile of 8 KiB stands behind the
// values', so that the heads' keys are not written out with it beside each.  8192 tokens, 16 heads of 128 + 64:
// 344 GFLOP in 347 to 366 us by box, 0.94 to 0.99 PFLOP/s (CUs busy 81% of the time, the pipe 57% of that); 4096,
// 2001, 511 and 1 tokens 143 us, 67% and 49%, as the longest tiles' 64 steps stand against 43 a CU on average.
// Every P runs as 64, its blocks past P multiplying zeros: 8192 tokens with 64, 32 and 8 of them 362, 354 and
// 348 us; 96 + 40, as 128 + 64, 345.
template <int DP, int NW, int PP>
__global__ __launch_bounds__(NW * 64) void attend_tile_kernel(AttendArgs a) {
  using S = Keys<DP>;
  constexpr int BK = 64, BQ = NW * 32, TILE = BK * S::ROWB, BUFB = 2 * TILE + BK * PP * 2;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  int64_t idx = blockIdx.x;
  const int kvh = (int)(idx % a.Hkv);
  idx = spread(idx / a.Hkv, a.ntiles * a.nsplit);
  const int split = (int)(idx / a.ntiles);
  const TileAt at = find_tile(a.table, a.cu_q, a.cu_k, a.nseq, G, BQ, idx - split * a.ntiles, a.ntiles, lane);
  if (at.seq < 0) return;
  const int nrows = min(BQ, at.Lq * G - at.n0);
  const int t1 = (at.n0 + nrows - 1) / G + at.Lk - at.Lq;  // the last row's position
  const int k_lo = split * a.chunk, k_hi = (int)min64(t1 + 1, (int64_t)k_lo + a.chunk);
  if (split > 0 && k_lo >= k_hi) return;  // (the join does not read this part)
  const uint16_t *kb = (const uint16_t *)uniform_ptr(a.k + (int64_t)at.k_start * a.ks + (int64_t)kvh * (PP ? a.kh : a.D));
  const uint16_t *vb = (const uint16_t *)uniform_ptr(a.v + (int64_t)at.k_start * a.vs + (int64_t)kvh * (PP ? a.vh : a.D));

  const int n = at.n0 + wave * 32 + (lane & 31);
  const bool live = wave * 32 + (lane & 31) < nrows;
  const int tok = n / G;
  const int head = kvh * G + (n - tok * G);
  const int t = tok + at.Lk - at.Lq;
  // this wave's first and last position
  const int wave_rows = min(32, nrows - wave * 32);
  const int w0 = (at.n0 + wave * 32) / G + at.Lk - at.Lq;
  const int w1 = wave_rows > 0 ? (at.n0 + wave * 32 + wave_rows - 1) / G + at.Lk - at.Lq : -1;
  Rows<DP, PP> r;
  r.init(live ? a.q + ((int64_t)at.q_start + tok) * a.qs + (int64_t)head * (PP ? a.QD : a.D) : nullptr, a.D, lane, a.P);

  const uint32_t lds0 = lds_offset(lds);
  Frag<DP> f;
  f.init(lds0, lane);
  KeyLoader<DP, BK, NW> keys;
  keys.init(wave, lane, a.D);
  constexpr int PW = PP ? PP : 64;
  Frag<PW> fp;
  KeyLoader<PW, BK, NW> pes;
  const uint16_t *pb = nullptr;
  if constexpr (PP > 0) {
    fp.init(lds0, lane);
    pes.init(wave, lane, a.P);
    pb = (const uint16_t *)uniform_ptr(a.pe + (int64_t)at.k_start * a.pes);
  }
  const int ntile = k_hi > k_lo ? (k_hi - k_lo + BK - 1) / BK : 0;
  auto load = [&](int tile, int buf) {
    const int k0 = k_lo + tile * BK;
    keys.load(kb + (int64_t)k0 * a.ks, a.ks, at.Lk - 1 - k0, lds0 + buf * BUFB);
    keys.load(vb + (int64_t)k0 * a.vs, a.vs, at.Lk - 1 - k0, lds0 + buf * BUFB + TILE);
    if constexpr (PP > 0) pes.load(pb + (int64_t)k0 * a.pes, a.pes, at.Lk - 1 - k0, lds0 + buf * BUFB + 2 * TILE);
  };
  auto step = [&](int j, auto buf_c) {
    constexpr int BUF = decltype(buf_c)::value;
    // this wave's part of tile j has landed; behind the barrier everyone's has, and everyone
    // is done with the buffer that tile j + 1 goes to
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    barrier_only();
    if (j + 1 < ntile) load(j + 1, BUF ^ 1);
    const int k0 = k_lo + j * BK;
    const auto visible = [&](int sub, int i) { return k0 + sub * 32 + i <= t; };
    if (k0 <= w1) {  // (the whole wave; not where it sees none of the tile, or has no rows)
      if constexpr (PP > 0)
        r.template add<BK>(f, fp, BUF * BUFB, BUF * BUFB + 2 * TILE, BUF * BUFB + TILE, a.scale_log2, lane,
                           k0 + BK - 1 > w0, visible);
      else
        r.template add<BK>(f, BUF * BUFB, BUF * BUFB + TILE, a.scale_log2, lane, k0 + BK - 1 > w0, visible);
    }
  };
  wait_loads();
  if (ntile > 0) load(0, 0);
  for (int j = 0; j < ntile; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < ntile) step(j + 1, std::integral_constant<int, 1>{});
  }
  // (a tile with one part writes the outputs themselves)
  write_row(a, live, ((int64_t)at.q_start + tok) * a.Hq + head, t1 < a.chunk, split, r, lane);
}

// The NW waves of a workgroup, each with its keys' part of the same 32 rows, join: O of every
// wave scaled to the common maximum, summed in wave order.  `lds` is free for it.  Row r of the
// workgroup is row out_row(r) of the output, r < nrows.
template <int DP, int NW>
struct Join {
  static constexpr int STAT = NW * 64;                  // m and l, [NW][2][32]
  static constexpr int LDS = (STAT + NW * DP * 33) * 4;  // and O^T, [NW][DP][33]
};
template <int DP, int NW, class R, class F>
__device__ inline void join_waves(const AttendArgs &a, const R &r, unsigned char *lds, int wave, int lane,
                                  int split, int nrows, F &&out_row) {
  const int mine = lane & (R::ROWS - 1);
  const float l = r.sum();
  __syncthreads();  // (all waves are done with their tiles)
  float *stat = reinterpret_cast<float *>(lds);
  float *acc = stat + Join<DP, NW>::STAT;
  if (lane < R::ROWS) stat[wave * 64 + lane] = r.m, stat[wave * 64 + 32 + lane] = l;
  __syncthreads();
  float m = -__builtin_inff();
#pragma unroll
  for (int w = 0; w < NW; ++w) m = fmaxf(m, stat[w * 64 + mine]);
  const float shift = m > -__builtin_inff() ? m : 0.0f;
  const float mul = exp2f_fast(r.m - shift);
#pragma unroll
  for (int dt = 0; dt < R::S::DT; ++dt)
#pragma unroll
    for (int i = 0; i < R::VALUES; ++i) acc[(wave * DP + R::place(dt, i, lane)) * 33 + mine] = r.o[dt][i] * mul;
  __syncthreads();
  // 8 columns of a row a thread at a time
  for (int e = threadIdx.x; e < R::ROWS * (DP / 8); e += NW * 64) {
    const int row = e / (DP / 8), d0 = e % (DP / 8) * 8;
    if (row >= nrows || d0 >= a.D) continue;
    float rm = -__builtin_inff(), rl = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) rm = fmaxf(rm, stat[w * 64 + row]);
    const float sh = rm > -__builtin_inff() ? rm : 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) rl += stat[w * 64 + 32 + row] * exp2f_fast(stat[w * 64 + row] - sh);
    const int64_t to = out_row(row);
    const float inv = rl == 0.0f ? 0.0f : 1.0f / rl;
    const float lse = rl == 0.0f ? -__builtin_inff() : (rm + log2f(rl)) * kLn2;
    float out[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) t += acc[(w * DP + d0 + d) * 33 + row];
      out[d] = t * inv;
    }
    if (a.nsplit > 1) {
      float *dst = a.part_o + ((int64_t)split * a.rows + to) * a.D + d0;
      *reinterpret_cast<float4 *>(dst) = make_float4(out[0], out[1], out[2], out[3]);
      *reinterpret_cast<float4 *>(dst + 4) = make_float4(out[4], out[5], out[6], out[7]);
      if (d0 == 0) a.part_lse[(int64_t)split * a.rows + to] = lse;
    } else {
      *reinterpret_cast<uint4 *>(a.o + to * a.D + d0) =
          make_uint4(pack_bf16(out[0], out[1]), pack_bf16(out[2], out[3]), pack_bf16(out[4], out[5]),
                     pack_bf16(out[6], out[7]));
      if (d0 == 0 && a.lse) a.lse[to] = lse;
    }
  }
}

// Few rows: a workgroup's 4 waves share 32 virtual rows and take key tiles of 32 in turn,
// each through its own double-buffered LDS without a barrier, and join at the end.  Bound by
// the keys' and values' bytes, each read once: 191 MB of a batch of 8 single tokens in 43 us
// (4.4 TB/s).
template <int DP>
struct FewRows {
  static constexpr int NW = 4, BK = 32, TILE = BK * Keys<DP>::ROWB;
  static constexpr int LDS = NW * 4 * TILE > Join<DP, NW>::LDS ? NW * 4 * TILE : Join<DP, NW>::LDS;
};
template <int DP>
__global__ __launch_bounds__(256) void attend_rows_kernel(AttendArgs a) {
  using S = Keys<DP>;
  constexpr int BK = FewRows<DP>::BK, NW = FewRows<DP>::NW, TILE = FewRows<DP>::TILE;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  int64_t idx = blockIdx.x;
  const int kvh = (int)(idx % a.Hkv);
  idx = spread(idx / a.Hkv, a.ntiles * a.nsplit);
  const int split = (int)(idx / a.ntiles);
  const TileAt at = find_tile(a.table, a.cu_q, a.cu_k, a.nseq, G, 32, idx - split * a.ntiles, a.ntiles, lane);
  if (at.seq < 0) return;
  const int n = at.n0 + (lane & 31), tok = n / G, head = kvh * G + n - tok * G;
  const int nrows = min(32, at.Lq * G - at.n0);
  const int t = tok + at.Lk - at.Lq;
  Rows<DP> r;
  r.init((lane & 31) < nrows ? a.q + ((int64_t)at.q_start + tok) * a.qs + (int64_t)head * a.D : nullptr, a.D,
         lane);
  const uint16_t *kb = (const uint16_t *)uniform_ptr(a.k + (int64_t)at.k_start * a.ks + (int64_t)kvh * a.D);
  const uint16_t *vb = (const uint16_t *)uniform_ptr(a.v + (int64_t)at.k_start * a.vs + (int64_t)kvh * a.D);
  const uint32_t mine = lds_offset(lds) + wave * 4 * TILE;
  Frag<DP> f;
  f.init(mine, lane);
  KeyLoader<DP, BK, 1> keys;
  keys.init(0, lane, a.D);
  // the first row's position and the last one's
  const int t0 = at.n0 / G + at.Lk - at.Lq, t1 = (at.n0 + nrows - 1) / G + at.Lk - at.Lq;
  const int k_lo = split * a.chunk, k_hi = (int)min64(t1 + 1, (int64_t)k_lo + a.chunk);
  auto load = [&](int k0, int buf) {
    keys.load(kb + (int64_t)k0 * a.ks, a.ks, at.Lk - 1 - k0, mine + buf * 2 * TILE);
    keys.load(vb + (int64_t)k0 * a.vs, a.vs, at.Lk - 1 - k0, mine + buf * 2 * TILE + TILE);
  };
  wait_loads();
  int k0 = k_lo + wave * BK, buf = 0;
  if (k0 < k_hi) load(k0, 0);
  for (; k0 < k_hi; k0 += NW * BK, buf ^= 1) {
    const bool more = k0 + NW * BK < k_hi;
    wait_reads();
    if (more) load(k0 + NW * BK, buf ^ 1);
    // the tile's own loads are the older ones: wait until only the next tile's are out
    constexpr int LOADS = 2 * BK / S::REGION_ROWS;
    static_assert(LOADS == 16 || LOADS == 8, "loads of a tile");
    if (!more) wait_loads();
    else if (LOADS == 16) __builtin_amdgcn_s_waitcnt(0x4F70);  // vmcnt(16)
    else __builtin_amdgcn_s_waitcnt(0x0F78);                   // vmcnt(8)
    asm volatile("" ::: "memory");
    r.template add<BK>(f, buf * 2 * TILE, buf * 2 * TILE + TILE, a.scale_log2, lane, k0 + BK - 1 > t0,
                       [&](int, int i) { return k0 + i <= t; });
    asm volatile("" ::: "memory");
  }
  join_waves<DP, NW>(a, r, lds, wave, lane, split, nrows, [&](int row) {
    const int m = at.n0 + row, tk = m / G;
    return ((int64_t)at.q_start + tk) * a.Hq + kvh * G + (m - tk * G);
  });
}

// Rows with lists of tokens.  A unit of work is up to 32 heads of one token and key head (and
// one part of its list); WR waves share it, each taking list tiles of 32 in turn, and join at
// the end.  The keys come from all over memory, so what counts is how many bytes are on their
// way, and how many of them from the L2.
//   Each wave has one LDS buffer for keys and one for values and asks for the next tile's as
//   soon as this one's are in registers.  Two workgroups of 4 waves fit a CU.
//   The list is taken in blocks, which first drop the entries outside 0 .. t and, where
//   a.by_place, are put into 16 groups by their place in the sequence (a counting sort whose
//   order is the same every time, and so the sums').  Workgroups of one XCD (every 8th) take
//   consecutive tokens of one key head and walk the sequence in the same direction at about
//   the same time, so what several of them selected is read from memory once.
//   WR = 1, where there are rows enough: the 256 rows that an XCD then works on at a time
//   pass a sixteenth of the sequence together and share more of it than 64 rows that each go
//   by four times as fast, and no waves have to join.
//   ROWS = 16 for up to 16 heads a key head: half the matrix and vector work of 32.
// 2048 rows of 2048 of 65536 tokens, 32 heads over 2: 274 us, 65% of the keys from the L2 (WR = 4:
// 396 us; lists in their own order: 549 us, 12%).  Bound by the loads into the LDS: with all
// keys in the L2 it takes 219 us, and without any of the products and the softmax 212.
// The last tile of a block may be short: its absent entries read the tile's first key, so that
// no other key is read, and count for nothing.
template <int DP, int WR>
struct Lists {
  static constexpr int NW = 4, BK = 32, TILE = BK * Keys<DP>::ROWB;
  static constexpr int UNITS = NW / WR;                           // of a workgroup
  static constexpr int BLOCK = 2048, EACH = BLOCK / (WR * 64), GROUPS = 16;
  // A wave a row and 128 wide: the LDS that the tiles leave holds a block's ids in 16 bits, or
  // half a block's (which then walks the sequence once more) where sequences are longer
  static constexpr bool HALF = WR == 1 && DP == 128;
  static constexpr int IDS = NW * 2 * TILE, USE = IDS + UNITS * BLOCK * (HALF ? 2 : 4);
  // (a wave's counts, [GROUPS][64], and behind them, at a unit's first wave, the unit's,
  // [GROUPS][WR] and their total, lie in its tile buffers: a block is sorted when no tile is in use
  // or on its way)
  static constexpr int COUNTS = GROUPS * 64 * 4;
  static_assert(COUNTS + (GROUPS * WR + 1) * 4 <= 2 * TILE, "counts in a tile buffer");
  static constexpr int LDS = WR > 1 && Join<DP, NW>::LDS > USE ? Join<DP, NW>::LDS : USE;
};
template <int DP, int WR, int ROWS>
__global__ __launch_bounds__(256, 2) void attend_list_kernel(AttendArgs a) {
  using S = std::conditional_t<ROWS == 16, Keys16<DP>, Keys<DP>>;
  using C = Lists<DP, WR>;
  constexpr int BK = C::BK, NW = C::NW, TILE = C::TILE;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv, per = (G + 31) / 32;
  const int64_t each = a.ntiles * per * a.nsplit, total = each * a.Hkv;  // units: of a key head, all
  const int64_t wgs = (total + C::UNITS - 1) / C::UNITS;
  int64_t idx = ((blockIdx.x & 7) * ((wgs + 7) / 8) + (blockIdx.x >> 3)) * C::UNITS + wave / WR;
  if (idx >= total) return;
  const int kvh = (int)(idx / each);
  idx -= kvh * each;
  const int split = (int)(idx % a.nsplit);
  idx /= a.nsplit;
  const int first = (int)(idx % per) * 32;  // the workgroup's first head of the group
  const TileAt at = find_tile(a.table, a.cu_q, a.cu_k, a.nseq, 1, 1, idx / per, a.ntiles, lane);
  if (at.seq < 0) return;
  const int tok = at.n0, t = tok + at.Lk - at.Lq;
  const int nrows = min(32, G - first), head = kvh * G + first;
  const int64_t token = (int64_t)at.q_start + tok;
  const int col_row = lane & (ROWS - 1);  // the lane's row
  using R = std::conditional_t<ROWS == 16, Rows16<DP>, Rows<DP>>;
  R r;
  r.init(col_row < nrows ? a.q + token * a.qs + (int64_t)(head + col_row) * a.D : nullptr, a.D, lane);
  const uint16_t *kb = (const uint16_t *)uniform_ptr(a.k + (int64_t)at.k_start * a.ks + (int64_t)kvh * a.D);
  const uint16_t *vb = (const uint16_t *)uniform_ptr(a.v + (int64_t)at.k_start * a.vs + (int64_t)kvh * a.D);
  const int32_t *list = a.ids + token * a.width;
  const uint32_t mine = lds_offset(lds) + wave * 2 * TILE;
  std::conditional_t<ROWS == 16, Frag16<DP>, Frag<DP>> f;
  f.init(mine, lane);
  const int part = wave % WR;  // of the unit's waves
  const bool narrow = C::HALF && at.Lk <= 65536;
  const int block_ids = C::HALF && !narrow ? C::BLOCK / 2 : C::BLOCK;
  int *ids = reinterpret_cast<int *>(lds + C::IDS + wave / WR * C::BLOCK * (C::HALF ? 2 : 4));
  uint16_t *ids16 = reinterpret_cast<uint16_t *>(ids);
  KPOOL_LDS int *mine_count = (KPOOL_LDS int *)(uintptr_t)mine + lane;                 // [GROUPS][64]
  int *count = reinterpret_cast<int *>(lds + (wave - part) * 2 * TILE + C::COUNTS);  // [GROUPS][WR], the total
  auto sync = [&] {  // of the unit's waves
    if (WR > 1) __syncthreads();
    else wait_reads();  // (a wave's own LDS accesses go in order)
  };
  const int e_lo = split * a.chunk, e_hi = (int)min64(a.width, (int64_t)e_lo + a.chunk);
  // group of an id: by_place the top 4 bits of the sequence's positions, else one for all
  const int shift = a.by_place ? max(0, 28 - __clz(max(at.Lk - 1, 1))) : 31;

  constexpr int REGIONS = BK / S::REGION_ROWS;  // loads of a tile's keys, and of its values
  constexpr int PATTERNS = 16 / S::REGION_ROWS;  // regions after which the swizzle repeats
  int col[PATTERNS];
#pragma unroll
  for (int i = 0; i < PATTERNS; ++i)
    col[i] = min((lane & (DP / 8 - 1)) ^ S::swz(i * S::REGION_ROWS + lane * 16 / S::ROWB), a.D / 8 - 1) * 8;
  auto load = [&](const uint16_t *base, int64_t stride, int id, uint32_t to) {
#pragma unroll
    for (int i = 0; i < REGIONS; ++i) {
      const int64_t key = __shfl(id, i * S::REGION_ROWS + lane * 16 / S::ROWB);
      load_lds_16(base + key * stride + col[i % PATTERNS], to + i * 1024);
    }
  };
  // waits until at most the loads of one side (keys or values) of a tile are out
  auto wait_side = [&](bool out) {
    static_assert(REGIONS == 8 || REGIONS == 4, "loads of a side");
    if (!out) wait_loads();
    else if (REGIONS == 8) __builtin_amdgcn_s_waitcnt(0x0F78);  // vmcnt(8)
    else __builtin_amdgcn_s_waitcnt(0x0F74);                    // vmcnt(4)
    asm volatile("" ::: "memory");
  };
  const int ngroups = a.by_place ? C::GROUPS : 1;
  for (int block = e_lo; block < e_hi; block += block_ids) {
    // the block's ids, up to EACH a lane, by group, lane and place in the list: each lane counts
    // its own, the counts are summed, and each lane takes places from its starts on
    int id[C::EACH];
    const int end = min(e_hi, block + block_ids);
#pragma unroll
    for (int i = 0; i < C::EACH; ++i) {
      const int e = block + i * WR * 64 + part * 64 + lane;
      id[i] = e < end ? list[e] : -1;
    }
    for (int g = 0; g < ngroups + 1; ++g) mine_count[(g & (C::GROUPS - 1)) * 64] = 0;  // (pairs are summed)
#pragma unroll
    for (int i = 0; i < C::EACH; ++i) {
      if (id[i] > t) id[i] = -1;
      if (id[i] >= 0)
        __hip_atomic_fetch_add(mine_count + (id[i] >> shift) * 64, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
    }
    for (int g = 0; g < ngroups; g += 2) {  // two groups' counts of 16 bits at a time
      const uint32_t c = mine_count[g * 64] | mine_count[g * 64 + 64] << 16;
      uint32_t sum = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(sum, d);
        if (lane >= d) sum += up;
      }
      mine_count[g * 64] = (sum - c) & 0xFFFF, mine_count[g * 64 + 64] = (sum - c) >> 16;
      if (lane == 63) count[g * WR + part] = sum & 0xFFFF, count[(g + 1) * WR + part] = sum >> 16;
    }
    sync();
    if (part == 0) {  // counts to starts
      static_assert(C::GROUPS * WR <= 64, "a count a lane");
      const int c = lane < ngroups * WR ? count[lane] : 0;
      int sum = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(sum, d);
        if (lane >= d) sum += up;
      }
      if (lane < C::GROUPS * WR) count[lane] = sum - c;
      if (lane == 63) count[C::GROUPS * WR] = sum;
    }
    sync();
    for (int g = 0; g < ngroups; ++g) mine_count[g * 64] += count[g * WR + part];
#pragma unroll
    for (int i = 0; i < C::EACH; ++i)
      if (id[i] >= 0) {
        const int at = __hip_atomic_fetch_add(mine_count + (id[i] >> shift) * 64, 1, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_WAVEFRONT);
        if (narrow) ids16[at] = (uint16_t)id[i];
        else ids[at] = id[i];
      }
    const int present = count[C::GROUPS * WR];
    wait_reads();  // (the tiles' loads overwrite the counts)
    sync();

    // this wave's tiles: part, part + WR, ..
    const int ntile = (present + BK - 1) / BK;
    auto entry = [&](int tile) {
      int e = tile * BK + (lane & 31);
      e = e < present ? e : tile * BK;
      return narrow ? (int)ids16[e] : ids[e];
    };
    int j = part;
    if (j < ntile) {
      const int e = entry(j);
      load(kb, a.ks, e, mine), load(vb, a.vs, e, mine + TILE);
    }
    for (; j < ntile; j += WR) {
      const bool more = j + WR < ntile;
      const int next = more ? entry(j + WR) : 0;
      std::conditional_t<ROWS == 16, f32x4[2], f32x16[1]> s;
      // (a side's next tile is asked for once this one's fragments are in registers)
      wait_side(true);  // the keys; the values may still be out
      typename R::template KeyFrag<BK> kr;
      R::template read_keys<BK>(f, 0, kr);
      wait_reads();
      if (more) load(kb, a.ks, next, mine);
      __builtin_amdgcn_sched_barrier(0);
      r.template scores<BK>(kr, s);
      r.weights(s, a.scale_log2, lane, j * BK + BK > present,
                [&](int, int i) { return j * BK + i < present; });
      wait_side(more);  // the values; the next keys may still be out
      typename R::ValueFrag vr;
      R::read_values(f, TILE, vr);
      wait_reads();
      if (more) load(vb, a.vs, next, mine + TILE);
      __builtin_amdgcn_sched_barrier(0);
      r.values(vr, s);
    }
    sync();  // (the next block's ids go where these were)
  }
  if constexpr (WR > 1)
    join_waves<DP, NW>(a, r, lds, wave, lane, split, nrows,
                       [&](int row) { return token * a.Hq + head + row; });
  else
    write_row(a, col_row < nrows, token * a.Hq + head + col_row, a.nsplit == 1, split, r, lane);
}

// Joins the splits of a row: o = sum_s 2^(lse_s - lse) o_s, 4 columns a lane, 64 / (D / 4) rows
// a workgroup, whose 4 waves take every fourth split each.  A split that saw nothing has lse
// -inf: its weight is 0 and its o is not read.  The loads do not wait for one another.
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
  __shared__ float part[4][64][5];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = a.D / 4, rows = 64 / per;  // (lanes past rows * per repeat the last row's)
  const int r = min(lane / per, rows - 1), d = min(lane - r * per, per - 1) * 4;
  const int64_t row = min64((int64_t)blockIdx.x * rows + r, a.rows - 1);
  const float none = -__builtin_inff();
  const float *lse = a.part_lse + row;
  float m = none;
#pragma unroll 8
  for (int s = 0; s < a.nsplit; ++s) m = fmaxf(m, lse[(int64_t)s * a.rows]);
  const float shift = m > none ? m : 0.0f;
  float total = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = wave; s < a.nsplit; s += 4) {
    const float x = lse[(int64_t)s * a.rows];
    const float w = exp2f_fast((x - shift) * kLog2e);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (x != none) v = *reinterpret_cast<const float4 *>(a.part_o + ((int64_t)s * a.rows + row) * a.D + d);
    total += w;
    o[0] = fmaf(w, v.x, o[0]), o[1] = fmaf(w, v.y, o[1]), o[2] = fmaf(w, v.z, o[2]), o[3] = fmaf(w, v.w, o[3]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][lane][i] = o[i];
  part[wave][lane][4] = total;
  __syncthreads();
  if (wave != 0 || lane >= rows * per || (int64_t)blockIdx.x * rows + r >= a.rows) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    total += part[w][lane][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += part[w][lane][i];
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  *reinterpret_cast<uint2 *>(a.o + row * a.D + d) =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  if (d == 0 && a.lse) a.lse[row] = total == 0.0f ? none : shift + log2f(total) * kLn2;
}

// The same for the tiles of the tile kernel that have more than one part; 8 workgroups a tile.
__global__ __launch_bounds__(256) void attend_tile_join_kernel(AttendArgs a) {
  constexpr int BQ = kTileWaves * 32, ROWS = BQ / 8;
  const int row0 = (blockIdx.x & 7) * ROWS, lane = threadIdx.x & 63, G = a.Hq / a.Hkv;
  const int unit = blockIdx.x >> 3, kvh = unit % a.Hkv;
  const TileAt at = find_tile(a.table, a.cu_q, a.cu_k, a.nseq, G, BQ, unit / a.Hkv, a.ntiles, lane);
  if (at.seq < 0) return;
  const int nrows = min(BQ, at.Lq * G - at.n0);
  const int parts = ((at.n0 + nrows - 1) / G + at.Lk - at.Lq) / a.chunk + 1;
  if (parts <= 1) return;
  const int per = a.D / 4;
  const float none = -__builtin_inff();
  for (int e = threadIdx.x; e < ROWS * per; e += 256) {
    const int n = at.n0 + row0 + e / per, d = e % per * 4;
    if (n >= at.Lq * G) break;
    const int64_t row = ((int64_t)at.q_start + n / G) * a.Hq + kvh * G + n % G;
    float m = none, total = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < parts; ++s) m = fmaxf(m, a.part_lse[(int64_t)s * a.rows + row]);
    const float shift = m > none ? m : 0.0f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float w = exp2f_fast((a.part_lse[(int64_t)s * a.rows + row] - shift) * kLog2e);
      const float4 v = *reinterpret_cast<const float4 *>(a.part_o + ((int64_t)s * a.rows + row) * a.D + d);
      total += w;
      o[0] = fmaf(w, v.x, o[0]), o[1] = fmaf(w, v.y, o[1]), o[2] = fmaf(w, v.z, o[2]), o[3] = fmaf(w, v.w, o[3]);
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    *reinterpret_cast<uint2 *>(a.o + row * a.D + d) =
        make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    if (d == 0 && a.lse) a.lse[row] = total == 0.0f ? none : shift + log2f(total) * kLn2;
  }
}

hipError_t launch_join(const AttendArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(attend_join_kernel, dim3((unsigned)((a.rows + 256 / a.D - 1) / (256 / a.D))), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_attend_t(const AttendPlan &p, const AttendArgs &a, hipStream_t st) {
  const unsigned grid = (unsigned)(a.ntiles * a.nsplit * a.Hkv);
  const bool few = p.form == AttendPlan::kRows;
  if (few) {
    constexpr size_t lds = FewRows<DP>::LDS;
    hipLaunchKernelGGL(attend_rows_kernel<DP>, dim3(grid), dim3(256), lds, st, a);
  } else {
    constexpr size_t lds = 4 * 64 * DP * 2;
    hipLaunchKernelGGL((attend_tile_kernel<DP, kTileWaves, 0>), dim3(grid), dim3(kTileWaves * 64), lds, st, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nsplit == 1) return e;
  if (few) return launch_join(a, st);
  hipLaunchKernelGGL(attend_tile_join_kernel, dim3((unsigned)(a.ntiles * a.Hkv * 8)), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int DP>
hipError_t launch_expanded_t(const AttendArgs &a, hipStream_t st) {
  constexpr size_t lds = 2 * 64 * (2 * DP + 64) * 2;
  hipLaunchKernelGGL((attend_tile_kernel<DP, kTileWaves, 64>), dim3((unsigned)(a.ntiles * a.nsplit * a.Hkv)),
                     dim3(kTileWaves * 64), lds, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nsplit == 1) return e;
  hipLaunchKernelGGL(attend_tile_join_kernel, dim3((unsigned)(a.ntiles * a.Hkv * 8)), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int DP, int WR, int ROWS>
void launch_list_dp(const AttendArgs &a, hipStream_t st) {
  using C = Lists<DP, WR>;
  const int64_t units = a.ntiles * ((a.Hq / a.Hkv + 31) / 32) * a.nsplit * a.Hkv;
  const int64_t wgs = (units + C::UNITS - 1) / C::UNITS;
  hipLaunchKernelGGL((attend_list_kernel<DP, WR, ROWS>), dim3((unsigned)((wgs + 7) / 8 * 8)), dim3(C::NW * 64),
                     C::LDS, st, a);
}
template <int WR, int ROWS>
hipError_t launch_list_t(const AttendArgs &a, hipStream_t st) {
  a.D <= 64 ? launch_list_dp<64, WR, ROWS>(a, st) : launch_list_dp<128, WR, ROWS>(a, st);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.nsplit > 1) e = launch_join(a, st);
  return e;
}

AttendArgs make_args(const AttendCall &c, const AttendPlan &p, void *workspace) {
  AttendArgs a{};
  a.q = c.q, a.k = c.k, a.v = c.v;
  a.qs = c.q_stride, a.ks = c.k_stride, a.vs = c.v_stride;
  a.cu_q = c.cu_q, a.cu_k = c.cu_k;
  a.nseq = c.nseq, a.Hq = c.Hq, a.Hkv = c.Hkv, a.D = c.D;
  a.scale_log2 = c.scale * kLog2e;
  const int BQ = p.form == AttendPlan::kList ? 1 : p.form == AttendPlan::kRows ? 32 : kTileWaves * 32;
  a.ntiles = make_table(a.table, c.cu_q_host, c.cu_k_host, c.nseq, p.form == AttendPlan::kList ? 1 : c.Hq / c.Hkv,
                        BQ, true);
  a.nsplit = p.nsplit, a.chunk = p.chunk;
  a.o = c.o, a.lse = c.lse;
  a.rows = c.Tq * c.Hq;
  if (p.nsplit > 1) {
    a.part_o = (float *)workspace;
    a.part_lse = a.part_o + (int64_t)p.nsplit * a.rows * c.D;
  }
  return a;
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

}  // namespace

size_t attend_workspace(const AttendPlan &p, int64_t rows, int D) {
  return p.nsplit > 1 ? (size_t)p.nsplit * rows * (D + 1) * sizeof(float) : 0;
}

int64_t attend_threads(const AttendPlan &p, int Hq, int Hkv) {
  const int64_t units = p.ntiles * p.nsplit * Hkv;
  if (p.form == AttendPlan::kRows) return units * 256;
  if (p.form == AttendPlan::kList) {
    const int64_t n = units * ((Hq / Hkv + 31) / 32);  // (workgroups by eights, one for each XCD)
    return round_up(p.wave_rows ? round_up(n, 4) / 4 : n, 8) * 256;
  }
  const int64_t join = p.nsplit > 1 ? p.ntiles * Hkv * 8 * 256 : 0;
  return std::max(units * kTileWaves * 64, join);
}

AttendPlan plan_attend(const int32_t *cu_q, const int32_t *cu_k, int nseq, int Hq, int Hkv, bool tiles) {
  const int64_t G = Hq / Hkv;
  int64_t most_rows = 0, most_keys = 0;
  for (int s = 0; s < nseq; ++s) {
    const int64_t lq = cu_q[s + 1] - cu_q[s], lk = cu_k[s + 1] - cu_k[s];
    if (lq > 0) most_rows = most_rows > lq * G ? most_rows : lq * G, most_keys = most_keys > lk ? most_keys : lk;
  }
  AttendPlan p;
  // 32 virtual rows fill one wave's tile; from there on sharing key tiles among waves is as good
  // (us by the rows kernel and the tile kernel, D = 128, 4 key heads: 8 sequences of 8192 keys, 32
  // rows 27 35, 64 rows 43 38, 128 rows 56 48; one of 16384 keys, 32 rows 24 24, 64 rows 26 25)
  // (expanded latent attention has the tile kernel alone: its single tokens take the absorbed form)
  p.form = most_rows <= 32 && !tiles ? AttendPlan::kRows : AttendPlan::kTiles;
  const int BQ = p.form == AttendPlan::kRows ? 32 : kTileWaves * 32;
  p.ntiles = tile_start(cu_q[nseq], nseq, (int)G, BQ);
  // workgroups, and the keys that all of them walk, without a split
  int64_t wgs = 0, walked = 0;
  for (int s = 0; s < nseq; ++s) {
    const int64_t lq = cu_q[s + 1] - cu_q[s], lk = cu_k[s + 1] - cu_k[s];
    wgs += (lq * G + BQ - 1) / BQ * Hkv;
    walked += (lq * G + BQ - 1) / BQ * lk * Hkv;
  }
  p.nsplit = 1, p.chunk = 0x7FFFFF00;
  // From 256 workgroups on, one a CU, no parts: right for sequences of like lengths (requests of
  // 8192 keys, 32 heads over 4: 63 of them, 252 workgroups, 233 us with parts, 64 270 without).
  // It does not look at the lengths: where one sequence is far longer than the others, one
  // workgroup a key head walks all of it (one request of 60000 keys, the others of 500: 63 of them
  // 244 us, 64 439 us).
  if (wgs >= 256) return p;
  const int64_t least = p.form == AttendPlan::kRows ? 1024 : 512;
  const int64_t chunk = round_up(walked / 512 > least ? walked / 512 : least, 256);
  if (most_keys > chunk) p.nsplit = (int)((most_keys + chunk - 1) / chunk), p.chunk = (int)chunk;
  return p;
}

AttendPlan plan_list(int64_t Tq, int nseq, int width, int Hq, int Hkv) {
  AttendPlan p;
  p.form = AttendPlan::kList;
  p.ntiles = tile_start(Tq, nseq, 1, 1);
  const int64_t wgs = Tq * Hkv * ((Hq / Hkv + 31) / 32);
  const int64_t want = wgs > 0 ? (256 + wgs - 1) / wgs : 1;
  // (128: 32 entries a wave; 8 tokens of 2048 entries 13.0 us captured, 13.3 with parts of 256)
  p.chunk = width > 0 ? (int)round_up((width + want - 1) / want, 128) : 128;
  p.nsplit = (int)((width + p.chunk - 1) / p.chunk);
  if (p.nsplit <= 1) p.nsplit = 1, p.chunk = 0x7FFFFF00;
  // sharing takes several workgroups an XCD at a time
  p.by_place = wgs >= 256;
  // a wave per row where that puts one on each SIMD (lists of 2048, units and us by four waves and
  // by one: 512 54 90, 1024 107 93, 1536 157 141, 2048 205 129, 4096 398 265, 8192 796 530)
  p.wave_rows = wgs >= 1024;
  return p;
}

hipError_t launch_attend(const AttendCall &c, const AttendPlan &p, void *workspace, hipStream_t st) {
  const AttendArgs a = make_args(c, p, workspace);
  return c.D <= 64 ? launch_attend_t<64>(p, a, st) : launch_attend_t<128>(p, a, st);
}

hipError_t launch_attend_expanded(const AttendCall &c, const ExpandedKeys &x, const AttendPlan &p, void *workspace,
                                  hipStream_t st) {
  AttendArgs a = make_args(c, p, workspace);
  a.pe = x.k_pe, a.pes = x.pe_stride, a.kh = x.k_head, a.vh = x.v_head, a.P = x.P, a.QD = c.D + x.P;
  return c.D <= 64 ? launch_expanded_t<64>(a, st) : launch_expanded_t<128>(a, st);
}

hipError_t launch_attend_list(const AttendCall &c, const AttendPlan &p, const int32_t *ids, int width,
                              void *workspace, hipStream_t st) {
  AttendArgs a = make_args(c, p, workspace);
  a.ids = ids, a.width = width;
  a.by_place = p.by_place;
  // (with four waves a row the loads bound it, and products of 16 rows take the same time)
  if (!p.wave_rows) return launch_list_t<4, 32>(a, st);
  return c.Hq / c.Hkv <= 16 ? launch_list_t<1, 16>(a, st) : launch_list_t<1, 32>(a, st);
}

}  // namespace kpool
