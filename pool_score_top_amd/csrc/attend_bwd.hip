// Gradients of the attention over whole keys (attend.hip).  With P_ij = exp(scale q_i k_j -
// lse_i) over what row i sees and delta_i = sum_d do_id o_id (= sum_j P_ij (do_i v_j)):
//   dV_j = sum_i P_ij do_i          dP_ij = do_i v_j      dS_ij = P_ij (dP_ij - delta_i)
//   dK_j = scale sum_i dS_ij q_i    dQ_i = scale sum_j dS_ij k_j
//
// Two kernels: dQ with the rows in registers and the keys walked, which also lays the rows' lse
// (base 2) and delta out along the virtual rows; dK and dV with the keys in registers and the
// rows walked.  S and dP are thus computed twice (7 matrix products instead of 5), and in return
// no sum crosses workgroups through atomics: the same call gives the same bits, and the
// gradients of shared key heads add up over their G query heads in registers, because the
// walked axis is the virtual rows.  P and dS are rounded to bf16 for their products (as the
// outputs are; where few keys are seen, dS to two bf16 numbers for dQ); P, dP, dS and all sums are
// fp32.
//
// Each kernel orients S so that its result registers are the next product's B operand: S^T
// [keys, rows] where rows stay (dQ^T = K^T dS^T), S [rows, keys] where keys stay (dV^T =
// dO^T P, dK^T = Q^T dS).
//
// dK and dV go by equal shares of the walked rows, dQ by tiles, whose keys are walked in parts
// where there are fewer tiles than CUs; parts are summed in fp32 in a fixed order by further
// kernels.
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
  int qsplit, qchunk;  // parts of the walked keys (for dQ), their size (a multiple of 64)
  uint16_t *dq, *dk, *dv;
  float *part;          // fp32 parts, used by one kernel and its sum at a time
  TileTable table;      // of keys, or of query rows
  // expanded latent attention: as AttendArgs has it; the keys' positional gradient by key heads in fp32,
  // [Hkv][Tk][P], and their sum
  const uint16_t *pe;
  int64_t pes, kh, vh;
  int P, QD;
  float *pe_part;
  uint16_t *dpe;
};

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

// The same for the DT blocks from column `col` on of rows of `width` columns, `end` of them in this part.
template <int DT>
__device__ inline void write_part(const f32x16 *x, float mul, uint16_t *out, float *part, int64_t row, int width, int col,
                                  int end, int lane) {
  const int h = lane >> 5;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int d = dt * 32 + 2 * i + 4 * h;
      if (d >= end) continue;
      const int64_t at = row * width + col + d;
      if (part)
        *reinterpret_cast<float4 *>(part + at) =
            make_float4(x[dt][i] * mul, x[dt][i + 1] * mul, x[dt][i + 2] * mul, x[dt][i + 3] * mul);
      else
        *reinterpret_cast<uint2 *>(out + at) =
            make_uint2(pack_bf16(x[dt][i] * mul, x[dt][i + 1] * mul), pack_bf16(x[dt][i + 2] * mul, x[dt][i + 3] * mul));
    }
}

// A lane's fragments of a row of PP values in LDS rather than in registers, for itself to read again:
// 4 KiB a wave.
template <int PP>
__device__ inline uint32_t stash(uint32_t lds0, const uint16_t *row, int P, int lane) {
  const uint32_t at = lds0 + Keys<PP>::row_base(lane);
#pragma unroll
  for (int ks = 0; ks < PP / 16; ++ks) {
    const int d = ks * 16 + (lane >> 5) * 8;
    uint4 z = make_uint4(0, 0, 0, 0);
    if (row && d < P) z = *reinterpret_cast<const uint4 *>(row + d);
    *(KPOOL_LDS bf16x8 *)(uintptr_t)(at ^ (ks << 5)) = __builtin_bit_cast(bf16x8, z);
  }
  return at;
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

// dK and dV: a workgroup's 128 keys in 4 groups of 32, two waves a group on one SIMD: the
// first computes S and P and sums dV, the second computes dP and dS one tile behind it and
// sums dK.  P passes from one to the other through LDS in fp32, lane for lane.  One wave for
// both would need over 256 registers (128 of sums, 64 of keys and values) and have the SIMD to
// itself, with nothing to fill its waits; in this form each needs under 256 and one's vector
// work runs beside the other's matrix instructions (16 a tile each).
// Tiles of 32 virtual rows (q, do, lse, delta) pass through four LDS buffers: the first
// wave's tile, the second's, and two on their way.  The steps are unrolled by four so that
// every LDS address is a register computed once plus a constant.
// Work goes by equal shares: the first key's rows are all the rows, the last one's few, and with
// parts of at most the CUs' average the CUs had work 66% of the time (the same tokens as at dQ's
// kernel: 330 us; by shares 254 and 13 to join, 210 GFLOP at 0.83 PFLOP/s; CUs busy 85% of the
// time, the matrix pipe 45% of that).
// PP = 64: with the positional part of expanded latent attention, whose 32 rows lie behind the others in
// rows as wide as theirs, so that they share their lanes' addresses.  Its products go to both waves, 4 a tile
// each: the first reads the keys' part from LDS (its registers are full), the second sums the gradient.
// 4096, 2001, 511 and 1 tokens, 16 heads of 128 + 64, 215 GFLOP: 274 us (the median of 40 calls, the least 262) and
// 19 to join, 0.78 PFLOP/s; a step takes 2210 cycles, 1280 of them products of the SIMD's two waves, a unit 22
// thousand cycles besides its steps, ten steps' time in which the pipe stands idle.
template <int DP, int PP = 0>
struct BwdKeys {
  static constexpr int BR = 32, NG = 4, KEYS = NG * 32;
  static constexpr int TILE = BR * Keys<DP>::ROWB, BUFB = (PP ? 3 : 2) * TILE;
  static constexpr int AHEAD = 2, NBUF = 4;
  static constexpr int STAT = NBUF * BUFB, STATB = 256;   // lse and delta of the buffers
  static constexpr int PBUF = 32 * 32 * 4, P = STAT + NBUF * STATB;
  static constexpr int KEYS_PE = P + 2 * NG * PBUF;  // the keys' positional parts
  static constexpr int LDS = KEYS_PE + KEYS * PP * 2;
};

// The first row of the first 32 virtual rows in which one sees a key of the tile from n0 on.
__host__ __device__ inline int64_t first_row(int64_t nvirt, int64_t Lk, int64_t Lq, int64_t n0, int64_t G) {
  const int64_t off = n0 - (Lk - Lq);
  return min64(nvirt, (off > 0 ? off : 0) * G) / 32 * 32;
}

template <int DP, int PP>
__global__ __launch_bounds__(512) void bwd_keys_kernel(BwdArgs a, Shares shares) {
  using S = Keys<DP>;
  using C = BwdKeys<DP, PP>;
  constexpr int BR = C::BR, TILE = C::TILE, BUFB = C::BUFB, NW = 8;
  constexpr int REGIONS = 2 * BR / S::REGION_ROWS;  // q's, then do's
  constexpr int PER = REGIONS / NW;                 // loads a wave
  static_assert(REGIONS % NW == 0, "whole loads a wave");
  constexpr int PS = PP / 16, PT = PP / 32;  // the positional part's steps and blocks
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave & 3;
  const bool second = wave >= 4;
  const int G = a.Hq / a.Hkv;
  const uint32_t lds0 = lds_offset(lds);
  Frag<DP> f;
  f.init(lds0, lane);
  const int q_width = PP ? a.QD : a.D;  // of a query head
  uint32_t st0 = lds0 + C::STAT + (lane >> 5) * 16 + (second ? 128 : 0);
  uint32_t pb = lds0 + C::P + group * C::PBUF + lane * 16;
  opaque(st0), opaque(pb);
  const Span span = span_of(shares, blockIdx.x);
  for (int u = span.u0; u <= span.u1; ++u) {
    const int step0 = u == span.u0 ? span.s0 : 0;
    if (u == span.u1 && span.s1 == 0) break;
    const int kvh = u % a.Hkv;
    // (tiles of keys: the roles of the two length arrays are exchanged)
    const TileAt at = find_tile(a.table, a.cu_k, a.cu_q, a.nseq, 1, C::KEYS, u / a.Hkv, a.ktiles, lane);
    if (at.seq < 0) continue;
    const int k_start = at.q_start, Lk = at.Lq, q_start = at.k_start, Lq = at.Lk;
    const int key = at.n0 + group * 32 + (lane & 31);  // this lane's key, of the sequence
    const bool live = key < Lk;

    // virtual rows that see the first key of the workgroup, cut to this share
    const int nvirt = Lq * G, off = Lk - Lq;
    auto seen_from = [&](int k) {
      return k < Lk ? (int)min64(nvirt, (int64_t)max(0, k - off) * G) : nvirt;
    };
    const int n_first = (int)first_row(nvirt, Lk, Lq, at.n0, G), nsteps = (nvirt - n_first + BR - 1) / BR;
    const int step1 = u == span.u1 ? span.s1 : nsteps;
    const int n_lo = n_first + step0 * BR, n_hi = min(nvirt, n_first + step1 * BR);
    const int ntile = step1 - step0;
    // this lane's key is seen from virtual row `from` on, the group's first key from `some` on
    // and all of them from `all` on
    const int from = live ? seen_from(key) : nvirt;
    const int some = seen_from(at.n0 + group * 32), all = seen_from(at.n0 + group * 32 + 31);
    wait_reads();
    barrier_only();  // (everyone is done with the last unit's tiles)

    bf16x8 kv[S::KS];  // the first wave's keys, the second's values
    uint32_t kp = 0;  // (and the first's positional ones)
    {
      const uint16_t *row = second ? a.v + ((int64_t)k_start + key) * a.vs : a.k + ((int64_t)k_start + key) * a.ks;
      if constexpr (PP > 0) row += (int64_t)kvh * (second ? a.vh : a.kh);
      else row += (int64_t)kvh * a.D;
      load_frag<DP>(kv, live ? row : nullptr, a.D, lane);
      if constexpr (PP > 0)
        if (!second)
          kp = stash<PP>(lds0 + C::KEYS_PE + group * 32 * PP * 2, live ? a.pe + ((int64_t)k_start + key) * a.pes : nullptr,
                         a.P, lane);
    }
    f32x16 sum[S::DT];  // dV^T of the first, dK^T of the second
    f32x16 sum_pe[PT + 1];  // (and its positional part)
  #pragma unroll
    for (int dt = 0; dt < S::DT; ++dt)
  #pragma unroll
      for (int i = 0; i < 16; ++i) sum[dt][i] = 0.0f;

    // Loads: regions wave, wave + 8, ..; for each the address of the lane's row and its head of
    // the group, moved on by 32 virtual rows a tile.
    const int sub = lane * 16 / S::ROWB;
    int g[PER];
    const uint16_t *src[PER];
    const int step_tok = BR / G, step_g = BR - step_tok * G;
    auto row_of = [&](int i) { return (wave + i * NW) % (REGIONS / 2) * S::REGION_ROWS + sub; };
    auto pitch_of = [&](int i) { return wave + i * NW >= REGIONS / 2 ? (int64_t)a.Hq * a.D : a.qs; };
    int64_t move[PER], move_over[PER];  // 32 virtual rows on, without and with a new token
  #pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int width = wave + i * NW >= REGIONS / 2 ? a.D : q_width;
      move[i] = step_tok * pitch_of(i) + step_g * width;
      move_over[i] = move[i] + pitch_of(i) - (int64_t)G * width;
    }
    auto address = [&](int i, int n) {  // of the lane's 16 bytes of virtual row n
      const int row = row_of(i);
      const int chunk = min((lane & (DP / 8 - 1)) ^ S::swz(row), a.D / 8 - 1);
      const uint16_t *p = wave + i * NW >= REGIONS / 2 ? a.d_o : a.q;
      const int tok = n / G;
      const int width = wave + i * NW >= REGIONS / 2 ? a.D : q_width;
      return p + (q_start + tok) * pitch_of(i) + (int64_t)(kvh * G + n - tok * G) * width + chunk * 8;
    };
    // the positional part's load goes with the wave's first one, of the same row (a wave whose loads are
    // all do's repeats one of them, so that all waves' loads count the same)
    int pe_off = 0;
    if (PP && wave < REGIONS / 2) {
      const int chunk = (lane & (DP / 8 - 1)) ^ S::swz(row_of(0));
      pe_off = a.D + (min(chunk, a.P / 8 - 1) - min(chunk, a.D / 8 - 1)) * 8;
    }
    auto load_pe = [&](const uint16_t *first, int buf) {
      load_lds_16(first + pe_off, lds0 + buf * BUFB + (wave < REGIONS / 2 ? 2 * TILE : 0) + wave * 1024);
    };
  #pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int n = min(n_lo + row_of(i), max(nvirt - 1, 0));
      src[i] = address(i, n);
      g[i] = n - n / G * G;
    }
    const float *stat = (lane < 32 ? a.lse2 : a.delta) + (int64_t)kvh * a.Tq * G + (int64_t)q_start * G;
    auto load = [&](int tile, int buf) {
      const uint32_t to = lds0 + buf * BUFB + wave * 1024;
      const int n0 = n_lo + tile * BR;
      if (n0 + BR <= nvirt) {
        if constexpr (PP > 0) load_pe(src[0], buf);
  #pragma unroll
        for (int i = 0; i < PER; ++i) {
          load_lds_16(src[i], to + i * NW * 1024);
          g[i] += step_g;
          const bool over = g[i] >= G;
          g[i] -= over ? G : 0;
          src[i] += over ? move_over[i] : move[i];
        }
      } else {  // the last rows: those past the end are the last one again and count for nothing
  #pragma unroll
        for (int i = 0; i < PER; ++i)
          load_lds_16(address(i, min(n0 + row_of(i), nvirt - 1)), to + i * NW * 1024);
        if constexpr (PP > 0) load_pe(address(0, min(n0 + row_of(0), nvirt - 1)), buf);
      }
      // (every wave loads the statistics, the same to the same place: its loads then count alike)
      load_lds_4(stat + min(n0 + (lane & 31), nvirt - 1), lds0 + C::STAT + buf * C::STATB);
    };
    // The reads of a phase go out together ahead of the matrix instructions that need them; the
    // compiler left to itself reads one fragment and waits for it, eight times over.
    auto product = [&](uint32_t buf, f32x4 (&st)[4], uint32_t st_at) {  // rows of the tile with kv
      bf16x8 r[S::KS];
  #pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) r[ks] = f.rows(buf, ks);
  #pragma unroll
      for (int b = 0; b < 4; ++b) st[b] = *(KPOOL_LDS const f32x4 *)(uintptr_t)(st_at + b * 32);
      __builtin_amdgcn_sched_barrier(0);
      f32x16 t = {};
  #pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) t = mfma(r[ks], kv[ks], t);
      return t;
    };
    auto positional = [&](uint32_t buf, f32x16 t) {  // what the first wave's product has besides
  #pragma unroll
      for (int ks = 0; ks < PS; ++ks) t = mfma(f.rows(buf, ks), lds_read(kp ^ (ks << 5)), t);
      return t;
    };
    auto columns = [&](uint32_t buf, int c, bf16x8 (&w)[S::DT]) {
  #pragma unroll
      for (int dt = 0; dt < S::DT; ++dt) w[dt] = f.cols(buf + c * 16 * S::ROWB, dt);
    };
    auto gather = [&](const bf16x8 (&w)[S::DT], const bf16x8 &x) {
  #pragma unroll
      for (int dt = 0; dt < S::DT; ++dt) sum[dt] = mfma(w[dt], x, sum[dt]);
    };
    auto gather_positional = [&](uint32_t buf, int c, const bf16x8 &x) {
  #pragma unroll
      for (int dt = 0; dt < PT; ++dt) sum_pe[dt] = mfma(f.cols(buf + c * 16 * S::ROWB, dt), x, sum_pe[dt]);
    };
    wait_loads();
  #pragma unroll
    for (int i = 0; i < C::AHEAD; ++i)
      if (i < ntile) load(i, i);
    auto enter = [&](int j) {
      // tile j has landed and P of tile j - 1 is written (everyone's, behind the barrier), and
      // nobody reads the buffer of tile j - 2 any more, where tile j + 2 goes
      static_assert(C::AHEAD == 2 && C::NBUF == 4 && (PER == 1 || PER == 2), "one tile's loads stay out");
      if (j + 1 >= ntile) __builtin_amdgcn_s_waitcnt(0x0070);    // vmcnt(0), lgkmcnt(0)
      else if (PP && PER == 2) __builtin_amdgcn_s_waitcnt(0x0074);  // vmcnt(4)
      else if (PP) __builtin_amdgcn_s_waitcnt(0x0073);           // vmcnt(3)
      else if (PER == 2) __builtin_amdgcn_s_waitcnt(0x0073);     // vmcnt(3)
      else __builtin_amdgcn_s_waitcnt(0x0072);                   // vmcnt(2)
      barrier_only();
      if (j + C::AHEAD < ntile) load(j + C::AHEAD, (j + C::AHEAD) & 3);
    };
    // Both waves pass ntile + 1 barriers: the first works on tiles 0 .. ntile - 1, the second
    // one step later; neither on the tiles before `skip`, which see no key of the group.
    const int skip = min(ntile, max(0, some - n_lo) / BR);
    auto first_wave = [&](int j, auto buf) {
      constexpr int BUF = decltype(buf)::value;
      enter(j);
      const int n0 = n_lo + j * BR;
      f32x4 lse[4];
      f32x16 p = product(BUF * BUFB, lse, st0 + BUF * C::STATB);
      if constexpr (PP > 0) p = positional(BUF * BUFB + 2 * TILE, p);
      bf16x8 w0[S::DT], w1[S::DT];
      columns(BUF * BUFB + TILE, 0, w0);
      __builtin_amdgcn_sched_barrier(0);
  #pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = exp2f_fast(fmaf(p[i], a.scale_log2, -lse[i / 4][i % 4]));
      if (n0 < all || n0 + BR > n_hi) {
        const int lo = from - n0 - 4 * (lane >> 5), hi = n_hi - n0 - 4 * (lane >> 5);
  #pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = 8 * (i / 4) + i % 4;
          if (r < lo || r >= hi) p[i] = 0.0f;
        }
      }
  #pragma unroll
      for (int b = 0; b < 4; ++b)
        *(KPOOL_LDS f32x4 *)(uintptr_t)(pb + (BUF & 1) * C::NG * C::PBUF + b * 1024) =
            f32x4{p[4 * b], p[4 * b + 1], p[4 * b + 2], p[4 * b + 3]};
      columns(BUF * BUFB + TILE, 1, w1);
      gather(w0, as_operand(p, 0));
      gather(w1, as_operand(p, 1));
    };
    auto second_wave = [&](int j, auto buf) {  // tile j - 1
      constexpr int BUF = (decltype(buf)::value + 3) & 3;
      enter(j);
      f32x4 delta[4], p[4];
      auto read_p = [&] {
  #pragma unroll
        for (int b = 0; b < 4; ++b)
          p[b] = *(KPOOL_LDS const f32x4 *)(uintptr_t)(pb + (BUF & 1) * C::NG * C::PBUF + b * 1024);
      };
      if constexpr (PP > 0) {
        // (P once the product's fragments are used up: beside them it would not fit the registers)
        f32x16 ds = product(BUF * BUFB + TILE, delta, st0 + BUF * C::STATB);
        __builtin_amdgcn_sched_barrier(0);
        read_p();
        bf16x8 w[S::DT];
        columns(BUF * BUFB, 0, w);
        __builtin_amdgcn_sched_barrier(0);
  #pragma unroll
        for (int i = 0; i < 16; ++i) ds[i] = p[i / 4][i % 4] * (ds[i] - delta[i / 4][i % 4]);
        const bf16x8 x0 = as_operand(ds, 0), x1 = as_operand(ds, 1);
        gather(w, x0);
        gather_positional(BUF * BUFB + 2 * TILE, 0, x0);
        columns(BUF * BUFB, 1, w);
        gather(w, x1);
        gather_positional(BUF * BUFB + 2 * TILE, 1, x1);
        return;
      }
      read_p();
      f32x16 ds = product(BUF * BUFB + TILE, delta, st0 + BUF * C::STATB);
      bf16x8 w0[S::DT], w1[S::DT];
      columns(BUF * BUFB, 0, w0);
      __builtin_amdgcn_sched_barrier(0);
  #pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] = p[i / 4][i % 4] * (ds[i] - delta[i / 4][i % 4]);
      columns(BUF * BUFB, 1, w1);
      gather(w0, as_operand(ds, 0));
      gather(w1, as_operand(ds, 1));
    };
    // steps [j, end), in rounds of four from a multiple of four on
    auto steps = [&](int j, int end, auto &&step) {
      using B0 = std::integral_constant<int, 0>;
      using B1 = std::integral_constant<int, 1>;
      using B2 = std::integral_constant<int, 2>;
      using B3 = std::integral_constant<int, 3>;
      if (j < end && (j & 3) == 1) step(j++, B1{});
      if (j < end && (j & 3) == 2) step(j++, B2{});
      if (j < end && (j & 3) == 3) step(j++, B3{});
      for (; j + 4 <= end; j += 4) step(j, B0{}), step(j + 1, B1{}), step(j + 2, B2{}), step(j + 3, B3{});
      if (j < end) step(j++, B0{});
      if (j < end) step(j++, B1{});
      if (j < end) step(j++, B2{});
    };
    if (!second) {
      for (int j = 0; j < skip; ++j) enter(j);
      steps(skip, ntile, first_wave);
      enter(ntile);
    } else {
  #pragma unroll
      for (int dt = 0; dt < PT; ++dt)
  #pragma unroll
        for (int i = 0; i < 16; ++i) sum_pe[dt][i] = 0.0f;
      for (int j = 0; j <= skip; ++j) enter(j);
      steps(skip + 1, ntile + 1, second_wave);
      if constexpr (PP > 0) {
        // (a part's rows are D + P wide; a whole unit's positional columns go to their head's sums)
        const bool whole = ntile == nsteps;
        float *part = a.part + ((2 * span.share + (step0 == 0)) * 2 + 1) * (int64_t)(C::KEYS * q_width);
        if (live)
          write_part<PT>(sum_pe, a.scale, nullptr, whole ? a.pe_part : part,
                         whole ? kvh * a.Tk + k_start + key : group * 32 + (lane & 31), whole ? a.P : q_width,
                         whole ? 0 : a.D, a.P, lane);
      }
    }
    const bool whole = ntile == nsteps;
    if constexpr (PP == 0) {
      float *part = a.part + ((2 * span.share + (step0 == 0)) * 2 + second) * (int64_t)(C::KEYS * a.D);
      if (live)
        write_cols<DP>(sum, second ? a.scale : 1.0f, second ? a.dk : a.dv, whole ? nullptr : part,
                       whole ? ((int64_t)k_start + key) * a.Hkv + kvh : group * 32 + (lane & 31), a.D, lane);
    } else if (live) {
      float *part = a.part + ((2 * span.share + (step0 == 0)) * 2 + second) * (int64_t)(C::KEYS * q_width);
      write_part<S::DT>(sum, second ? a.scale : 1.0f, second ? a.dk : a.dv, whole ? nullptr : part,
                        whole ? ((int64_t)k_start + key) * a.Hkv + kvh : group * 32 + (lane & 31),
                        whole ? a.D : q_width, 0, a.D, lane);
    }
  }
}

// Adds the parts of the units that lie across shares, in order: 16 workgroups a share, for 8 keys
// each of the unit that it begins and does not end.
__global__ __launch_bounds__(256) void bwd_keys_sum_kernel(BwdArgs a, Shares shares) {
  constexpr int KEYS = 128;
  const int share = blockIdx.x >> 4, key0 = (blockIdx.x & 15) * 8, lane = threadIdx.x & 63;
  int u, end;
  if (!begins_cut(shares, share, lane, u, end)) return;
  const int kvh = u % a.Hkv;
  const TileAt at = find_tile(a.table, a.cu_k, a.cu_q, a.nseq, 1, KEYS, u / a.Hkv, a.ktiles, lane);
  const int per = a.D / 4;
  const int64_t pitch = (int64_t)KEYS * a.D;
  for (int e = threadIdx.x; e < 2 * 8 * per; e += 256) {
    const int which = e >= 8 * per, r = key0 + (e - which * 8 * per) / per, d = e % per * 4;
    if (at.n0 + r >= at.Lq) continue;
    const float *part = a.part + which * pitch + r * a.D + d;
    float4 t = *reinterpret_cast<const float4 *>(part + (2 * share + 1) * 2 * pitch);
#pragma unroll 4
    for (int s = share + 1; s < end; ++s) {
      const float4 x = *reinterpret_cast<const float4 *>(part + 2 * s * 2 * pitch);
      t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    *reinterpret_cast<uint2 *>((which ? a.dk : a.dv) +
                               (((int64_t)at.q_start + at.n0 + r) * a.Hkv + kvh) * a.D + d) =
        make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
  }
}

// Rows that see few keys have the largest gradients, and their roundings show in the whole's.
// Tiles whose rows see no more than kFewKeys take delta from the keys instead of from o; up to
// kFineKeys dS is held in two bf16 numbers for dQ (a fourth product, of operands that are there).
// (Both limits were set at the shape below; others differ with their lengths and head counts.)
// The errors against 64 bits, in units of what rounding the exact gradient to bf16 gives (one
// rounding of dS beside it gives 1.41), for 2048 tokens, 8 heads over 1 of 64, and the time of a
// step there and of 8192 packed tokens with 16 heads over 4 of 128:
//   few, fine      dQ    dK    us
//   1024, none     1.49  1.43  94.5  574
//   512, none      1.53  1.45  87    561
//   512, 512       1.36  1.45  89    565
//   512, 1024      1.26  1.45  89    566
//   512, 2048      1.12  1.45  89    576
constexpr int kFewKeys = 512, kFineKeys = 1024;

// The same with rows of D + P columns, whose positional ones go to their head's sums.
__global__ __launch_bounds__(256) void bwd_expanded_sum_kernel(BwdArgs a, Shares shares) {
  constexpr int KEYS = 128;
  const int share = blockIdx.x >> 4, key0 = (blockIdx.x & 15) * 8, lane = threadIdx.x & 63;
  int u, end;
  if (!begins_cut(shares, share, lane, u, end)) return;
  const int kvh = u % a.Hkv;
  const TileAt at = find_tile(a.table, a.cu_k, a.cu_q, a.nseq, 1, KEYS, u / a.Hkv, a.ktiles, lane);
  const int per = (a.D + a.QD) / 4, per_v = a.D / 4;  // of a key: dv, then dk and its positional part
  const int64_t pitch = (int64_t)KEYS * a.QD;
  for (int e = threadIdx.x; e < 8 * per; e += 256) {
    const int r = key0 + e / per, c = e % per, which = c >= per_v, d = (c - which * per_v) * 4;
    if (at.n0 + r >= at.Lq) continue;
    const float *part = a.part + which * pitch + r * a.QD + d;
    float4 t = *reinterpret_cast<const float4 *>(part + (2 * share + 1) * 2 * pitch);
#pragma unroll 4
    for (int s = share + 1; s < end; ++s) {
      const float4 x = *reinterpret_cast<const float4 *>(part + 2 * s * 2 * pitch);
      t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    const int64_t token = (int64_t)at.q_start + at.n0 + r;
    if (d >= a.D)
      *reinterpret_cast<float4 *>(a.pe_part + (kvh * a.Tk + token) * a.P + d - a.D) = t;
    else
      *reinterpret_cast<uint2 *>((which ? a.dk : a.dv) + (token * a.Hkv + kvh) * a.D + d) =
          make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
  }
}

// The positional gradient, of a row that all key heads share: their sums, each head's in fp32 by the kernel
// above or by dK's, added in the heads' order.  (6609 tokens, 16 heads: 27 MB in 5.5 us.)
__global__ __launch_bounds__(256) void bwd_positional_kernel(BwdArgs a) {
  const int64_t n = a.Tk * a.P, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int h = 0; h < a.Hkv; ++h) {
    const float4 x = *reinterpret_cast<const float4 *>(a.pe_part + h * n + i);
    t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
  }
  *reinterpret_cast<uint2 *>(a.dpe + i) = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
}

// dQ: NW waves of 32 virtual rows; key tiles of 64 pass through LDS, as in the forward pass.
// 8192 packed tokens (4096, 2777, 1000, 319), 16 heads over 4 of 128: 157 GFLOP in 193 us, 0.81
// PFLOP/s.  CUs are busy 75% of the time, the matrix pipe 54% of that: within a wave a half tile's
// exponentials wait for its products and the next half's products for them (the scheduling
// barriers keep the phases apart), and all waves wait for a whole tile's loads together.  Cutting
// the longest tiles to the CUs' average leaves the time as it is.
// With the positional part (PP = 64) the rows' share of it lies in LDS, each lane's for itself, as the registers
// are full, and fragments are read four ahead of their products.  4096, 2001, 511 and 1 tokens, 16 heads of
// 128 + 64: 172 GFLOP in 239 us (the least 231), 0.72 PFLOP/s; a step of 64 keys takes 6700 cycles, 4100 of them
// products.
// With one of a SIMD's two waves ahead of the other (s_setprio), or with the rows read through LDS, the same.
template <int DP, int NW, int PP>
__global__ __launch_bounds__(NW * 64) void bwd_rows_kernel(BwdArgs a) {
  using S = Keys<DP>;
  constexpr int BK = 64, BQ = NW * 32, TILE = BK * S::ROWB, BUFB = 2 * TILE + BK * PP * 2;
  constexpr int PS = PP / 16, PT = PP / 32, PW = PP ? PP : 64;  // the positional part's steps, blocks, width
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.Hq / a.Hkv;
  int64_t idx = blockIdx.x;
  const int kvh = (int)(idx % a.Hkv);
  idx = spread(idx / a.Hkv, a.qtiles * a.qsplit);
  const int split = (int)(idx / a.qtiles);
  const TileAt at = find_tile(a.table, a.cu_q, a.cu_k, a.nseq, G, BQ, idx - split * a.qtiles, a.qtiles, lane);
  if (at.seq < 0) return;
  const int nrows = min(BQ, at.Lq * G - at.n0);
  const int t1 = (at.n0 + nrows - 1) / G + at.Lk - at.Lq;
  const bool whole = t1 < a.qchunk;  // (the only part, which writes dQ itself)
  const int k_lo = split * a.qchunk, k_hi = (int)min64(t1 + 1, (int64_t)k_lo + a.qchunk);
  if (split > 0 && k_lo >= k_hi) return;  // (the sum does not read this part)
  const uint16_t *kb = (const uint16_t *)uniform_ptr(a.k + (int64_t)at.k_start * a.ks + (int64_t)kvh * (PP ? a.kh : a.D));
  const uint16_t *vb = (const uint16_t *)uniform_ptr(a.v + (int64_t)at.k_start * a.vs + (int64_t)kvh * (PP ? a.vh : a.D));
  const int n = at.n0 + wave * 32 + (lane & 31);
  const bool live = wave * 32 + (lane & 31) < nrows;
  const int tok = n / G, head = kvh * G + (n - tok * G);
  const int t = tok + at.Lk - at.Lq;
  const int wave_rows = min(32, nrows - wave * 32);
  const int w0 = (at.n0 + wave * 32) / G + at.Lk - at.Lq;
  const int w1 = wave_rows > 0 ? (at.n0 + wave * 32 + wave_rows - 1) / G + at.Lk - at.Lq : -1;
  const int64_t row = ((int64_t)at.q_start + tok) * a.Hq + head;
  const uint32_t lds0 = lds_offset(lds);
  Frag<DP> f;
  f.init(lds0, lane);
  KeyLoader<DP, BK, NW> keys;
  keys.init(wave, lane, a.D);
  Frag<PW> fp;
  KeyLoader<PW, BK, NW> pes;
  const uint16_t *pb = nullptr;
  if constexpr (PP > 0) {
    fp.init(lds0, lane);
    pes.init(wave, lane, a.P);
    pb = (const uint16_t *)uniform_ptr(a.pe + (int64_t)at.k_start * a.pes);
  }
  const int ntile = k_hi > k_lo ? (k_hi - k_lo + BK - 1) / BK : 0;
  auto load = [&](int k0, int buf) {
    keys.load(kb + (int64_t)k0 * a.ks, a.ks, at.Lk - 1 - k0, lds0 + buf * BUFB);
    keys.load(vb + (int64_t)k0 * a.vs, a.vs, at.Lk - 1 - k0, lds0 + buf * BUFB + TILE);
    if constexpr (PP > 0) pes.load(pb + (int64_t)k0 * a.pes, a.pes, at.Lk - 1 - k0, lds0 + buf * BUFB + 2 * TILE);
  };
  // (the first tile is on its way while the rows' own values are)
  const bool few = t1 < kFewKeys;
  if (!few && ntile > 0) load(k_lo, 0);
  bf16x8 qf[S::KS], dof[S::KS];
  const uint16_t *q_row = a.q + ((int64_t)at.q_start + tok) * a.qs + (int64_t)head * (PP ? a.QD : a.D);
  load_frag<DP>(qf, live ? q_row : nullptr, a.D, lane);
  uint32_t qp = 0;
  if constexpr (PP > 0)
    qp = stash<PP>(lds_offset(lds) + 2 * BUFB + wave * 32 * Keys<PP>::ROWB, live ? q_row + a.D : nullptr, a.P, lane);
  load_frag<DP>(dof, live ? a.d_o + row * a.D : nullptr, a.D, lane);
  // the rows' lse and delta, which dK's and dV's kernel reads
  const int64_t stat = (int64_t)kvh * a.Tq * G + (int64_t)at.q_start * G + n;
  const float none = -__builtin_inff(), given = live ? a.lse[row] : none;
  const float lse = given != none ? given * kLog2e : -none;
  float delta = 0.0f;
  if (!few) {
    bf16x8 of[S::KS];
    load_frag<DP>(of, live ? a.o + row * a.D : nullptr, a.D, lane);
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks)
#pragma unroll
      for (int i = 0; i < 8; ++i) delta = fmaf((float)of[ks][i], (float)dof[ks][i], delta);
    delta += other_half(delta);
  }
  f32x16 dq[S::DT + PT];
#pragma unroll
  for (int dt = 0; dt < S::DT + PT; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) dq[dt][i] = 0.0f;

  // S and dP of 32 keys
  auto half_tile = [&](uint32_t sk, uint32_t sv, uint32_t sp, f32x16 &s, f32x16 &dp) {
    if constexpr (PP > 0) {  // (a few fragments ahead: more would not fit the registers)
      constexpr int N = 2 * PS + 2 * S::KS, AHEAD = 4;
      auto read = [&](int n) {  // fragments in the order of their use: positional pairs, keys, values
        return n < 2 * PS ? (n & 1 ? lds_read(qp ^ (n / 2 << 5)) : fp.rows(sp, n / 2))
                          : n < 2 * PS + S::KS ? f.rows(sk, n - 2 * PS) : f.rows(sv, n - 2 * PS - S::KS);
      };
      bf16x8 r[N];
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) r[n] = read(n);
      s = f32x16{}, dp = f32x16{};
#pragma unroll
      for (int n = 0; n < N; n += 2) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (n + AHEAD + u < N) r[n + AHEAD + u] = read(n + AHEAD + u);
        if (n < 2 * PS) s = mfma(r[n], r[n + 1], s);
        else
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int ks = n + u - 2 * PS;
            if (ks < S::KS) s = mfma(r[n + u], qf[ks < S::KS ? ks : 0], s);
            else dp = mfma(r[n + u], dof[ks < S::KS ? 0 : ks - S::KS], dp);
          }
      }
      __builtin_amdgcn_sched_barrier(0);
      return;
    }
    // (the reads of a phase go out together, ahead of what needs them)
    bf16x8 kr[S::KS], vr[S::KS];
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) kr[ks] = f.rows(sk, ks), vr[ks] = f.rows(sv, ks);
    __builtin_amdgcn_sched_barrier(0);
    s = f32x16{}, dp = f32x16{};
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) s = mfma(kr[ks], qf[ks], s);
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) dp = mfma(vr[ks], dof[ks], dp);
  };
  auto to_weights = [&](f32x16 &s, int k0, bool masked) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = exp2f_fast(fmaf(s[i], a.scale_log2, -lse));
    if (masked) {
      const int hi = t - k0 - 4 * (lane >> 5);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (8 * (i / 4) + i % 4 > hi) s[i] = 0.0f;
    }
  };
  auto enter = [&](int j, int ntile, int k_first, int buf) {
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    barrier_only();
    if (j + 1 < ntile) load(k_first + (j + 1) * BK, buf ^ 1);
  };
  wait_loads();
  if (few) {
    // delta from P and dP themselves: o was rounded to bf16, and where a few keys share the
    // weight that error reaches dS at the size of dS's own rounding
    const int n_all = t1 >= 0 ? t1 / BK + 1 : 0;
    float sum = 0.0f;
    if (n_all > 0) load(0, 0);
    for (int j = 0; j < n_all; ++j) {
      enter(j, n_all, 0, j & 1);
      const int k0 = j * BK;
      if (k0 > w1) continue;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sk = (j & 1) * BUFB + half * 32 * S::ROWB;
        f32x16 s, dp;
        half_tile(sk, sk + TILE, (j & 1) * BUFB + 2 * TILE + half * 32 * Keys<PW>::ROWB, s, dp);
        to_weights(s, k0 + half * 32, k0 + BK - 1 > w0);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(s[i], dp[i], sum);
      }
    }
    delta = sum + other_half(sum);
    __builtin_amdgcn_s_waitcnt(0x0070);
    barrier_only();
    if (ntile > 0) load(k_lo, 0);
  }
  if (split == 0 && live && lane < 32) a.lse2[stat] = lse, a.delta[stat] = delta;
  auto step = [&](int j, auto buf_c) {
    constexpr int BUF = decltype(buf_c)::value;
    enter(j, ntile, k_lo, BUF);
    const int k0 = k_lo + j * BK;
    if (k0 > w1) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      constexpr uint32_t SK = BUF * BUFB, SV = SK + TILE, SP = SK + 2 * TILE;
      const uint32_t down = half * 32 * S::ROWB, pe_down = half * 32 * Keys<PW>::ROWB;
      f32x16 s, dp;
      half_tile(SK + down, SV + down, SP + pe_down, s, dp);
      if constexpr (PP > 0) {
        to_weights(s, k0 + half * 32, k0 + BK - 1 > w0);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= dp[i] - delta;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const bf16x8 ds = as_operand(s, c), rest = as_operand_rest(s, c, ds);
#pragma unroll
          for (int dt = 0; dt < S::DT + PT; ++dt) {
            const bf16x8 w = dt < S::DT ? f.cols(SK + down + c * 16 * S::ROWB, dt < S::DT ? dt : 0)
                                        : fp.cols(SP + pe_down + c * 16 * Keys<PW>::ROWB, dt < S::DT ? 0 : dt - S::DT);
            dq[dt] = mfma(w, ds, dq[dt]);
            if (t1 < kFineKeys) dq[dt] = mfma(w, rest, dq[dt]);
          }
        }
        continue;
      }
      bf16x8 w[2][S::DT];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int dt = 0; dt < S::DT; ++dt) w[c][dt] = f.cols(SK + down + c * 16 * S::ROWB, dt);
      __builtin_amdgcn_sched_barrier(0);
      to_weights(s, k0 + half * 32, k0 + BK - 1 > w0);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] *= dp[i] - delta;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bf16x8 ds = as_operand(s, c);
#pragma unroll
        for (int dt = 0; dt < S::DT; ++dt) dq[dt] = mfma(w[c][dt], ds, dq[dt]);
        if (t1 >= kFineKeys) continue;
        const bf16x8 rest = as_operand_rest(s, c, ds);
#pragma unroll
        for (int dt = 0; dt < S::DT; ++dt) dq[dt] = mfma(w[c][dt], rest, dq[dt]);
      }
    }
  };
  for (int j = 0; j < ntile; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < ntile) step(j + 1, std::integral_constant<int, 1>{});
  }
  if (!live) return;
  if constexpr (PP > 0) {
    float *part = whole ? nullptr : a.part + (int64_t)split * a.Tq * a.Hq * a.QD;
    write_part<S::DT>(dq, a.scale, a.dq, part, row, a.QD, 0, a.D, lane);
    write_part<PT>(dq + S::DT, a.scale, a.dq, part, row, a.QD, a.D, a.P, lane);
  } else {
    float *part = whole ? nullptr : a.part + (int64_t)split * a.Tq * a.Hq * a.D;
    write_cols<DP>(dq, a.scale, a.dq, part, row, a.D, lane);
  }
}

constexpr int kBwdWaves = 8;

// Adds dQ's parts, in order, of the tiles that have more than one; 8 workgroups a tile.
__global__ __launch_bounds__(256) void bwd_rows_sum_kernel(BwdArgs a, int width) {
  constexpr int BQ = kBwdWaves * 32, ROWS = BQ / 8;
  const int row0 = (blockIdx.x & 7) * ROWS, lane = threadIdx.x & 63, G = a.Hq / a.Hkv;
  const int unit = blockIdx.x >> 3, kvh = unit % a.Hkv;
  const TileAt at = find_tile(a.table, a.cu_q, a.cu_k, a.nseq, G, BQ, unit / a.Hkv, a.qtiles, lane);
  if (at.seq < 0) return;
  const int nrows = min(BQ, at.Lq * G - at.n0);
  const int parts = ((at.n0 + nrows - 1) / G + at.Lk - at.Lq) / a.qchunk + 1;
  if (parts <= 1) return;
  const int per = width / 4;
  const int64_t pitch = a.Tq * a.Hq * width;
  for (int e = threadIdx.x; e < ROWS * per; e += 256) {
    const int n = at.n0 + row0 + e / per;
    if (n >= at.Lq * G) break;
    const int64_t to = (((int64_t)at.q_start + n / G) * a.Hq + kvh * G + n % G) * width + e % per * 4;
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float4 x = *reinterpret_cast<const float4 *>(a.part + s * pitch + to);
      t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    *reinterpret_cast<uint2 *>(a.dq + to) = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
  }
}

// Costs of a tile of keys and of a tile of rows (which may have to find delta first, two of its
// three products), and the steps that a share has at least.
// A unit of dK's and dV's kernel costs 4 steps besides its own, with the positional part 12: its first
// tiles and its sums, half as wide again, pass while nothing else runs on the CU, and where every head has
// its own keys there are many short units.  (Lengths 4096, 2001, 511 and 1, 16 heads of 128 + 64, forward and
// backward: 730 us with 4, 677 with 8, 642 with 12, 648 with 16.  Parts of 16 steps where those 12 are counted
// cut units that are better left whole: 300 and 77 tokens, 8 heads of 64 + 32, 54.3 us, with 24 50.6, which
// 32 and 48 leave as it is.  Each was set by that one batch; others were not measured for them.)
constexpr int kKeysShare = 16, kRowsShare = 6;
constexpr int kUnitCost = 4, kExpandedCost = 12, kExpandedShare = 24;
UnitCost keys_cost(int64_t lk, int64_t lq, int64_t n0, int64_t G, bool expanded = false) {
  return {expanded ? kExpandedCost : kUnitCost, (lq * G - first_row(lq * G, lk, lq, n0, G) + 31) / 32};
}
UnitCost rows_cost(int64_t lq, int64_t lk, int64_t n0, int64_t G) {
  const int64_t last = std::min<int64_t>(lq * G, n0 + kBwdWaves * 32) - 1, t1 = last / G + lk - lq;
  const int64_t steps = t1 >= 0 ? t1 / 64 + 1 : 0;
  return {2 + (t1 < kFewKeys ? steps * 2 / 3 : 0), steps};
}

template <int DP, int PP>
hipError_t launch_bwd_t(const AttendCall &c, const BwdPlan &p, BwdArgs a, hipStream_t st) {
  using C = BwdKeys<DP, PP>;
  hipError_t e = hipSuccess;
  const int G = a.Hq / a.Hkv;
  if (a.Tq > 0) {
    a.qtiles = make_table(a.table, c.cu_q_host, c.cu_k_host, a.nseq, a.Hq / a.Hkv, kBwdWaves * 32, true);
    const size_t lds = 2 * 64 * (2 * DP + PP) * 2 + kBwdWaves * 32 * PP * 2;
    hipLaunchKernelGGL((bwd_rows_kernel<DP, kBwdWaves, PP>), dim3((unsigned)(a.qtiles * a.qsplit * a.Hkv)),
                       dim3(kBwdWaves * 64), lds, st, a);
    e = hipGetLastError();
    if (e == hipSuccess && a.qsplit > 1) {
      hipLaunchKernelGGL(bwd_rows_sum_kernel, dim3((unsigned)(a.qtiles * a.Hkv * 8)), dim3(256), 0, st, a,
                         a.D + a.P);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  // (behind dQ's kernel, which lays lse and delta out for it)
  if (a.Tk > 0) {
    a.ktiles = make_table(a.table, c.cu_k_host, c.cu_q_host, a.nseq, 1, C::KEYS, false);
    Shares shares;
    const bool cut = make_shares(shares, p.kshares, p.kcost, a.Hkv, a.table, c.cu_k_host, c.cu_q_host, a.nseq, 1,
                                 C::KEYS, a.ktiles, [&](int64_t lk, int64_t lq, int64_t n0) {
                                   return keys_cost(lk, lq, n0, G, PP > 0);
                                 });
    const unsigned grid = (unsigned)(shares.n ? shares.n : a.ktiles * a.Hkv);
    hipLaunchKernelGGL((bwd_keys_kernel<DP, PP>), dim3(grid), dim3(512), C::LDS, st, a, shares);
    e = hipGetLastError();
    if (e == hipSuccess && cut) {
      if (PP) hipLaunchKernelGGL(bwd_expanded_sum_kernel, dim3(grid * 16), dim3(256), 0, st, a, shares);
      else hipLaunchKernelGGL(bwd_keys_sum_kernel, dim3(grid * 16), dim3(256), 0, st, a, shares);
      e = hipGetLastError();
    }
    if (e == hipSuccess && PP) {
      hipLaunchKernelGGL(bwd_positional_kernel, dim3((unsigned)((a.Tk * a.P / 4 + 255) / 256)), dim3(256), 0, st, a);
      e = hipGetLastError();
    }
  }
  return e;
}

int64_t up_to(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

}  // namespace

BwdPlan plan_attend_bwd(const int32_t *cu_q, const int32_t *cu_k, int nseq, int Hq, int Hkv, bool expanded) {
  const int G = Hq / Hkv;
  BwdPlan p;
  p.ktiles = tile_start(cu_k[nseq], nseq, 1, 128);
  p.qtiles = tile_start(cu_q[nseq], nseq, G, kBwdWaves * 32);
  TotalCost qcost;
  for (int s = 0; s < nseq; ++s) {
    const int64_t lq = cu_q[s + 1] - cu_q[s], lk = cu_k[s + 1] - cu_k[s];
    for (int64_t n0 = 0; n0 < lk; n0 += 128) p.kcost.add(keys_cost(lk, lq, n0, G, expanded), Hkv);
    for (int64_t n0 = 0; n0 < lq * G; n0 += kBwdWaves * 32) qcost.add(rows_cost(lq, lk, n0, G), Hkv);
  }
  p.kshares = share_count(p.kcost, expanded ? kExpandedShare : kKeysShare);
  plan_parts(qcost, kRowsShare, &p.qsplit, &p.qchunk);
  return p;
}

size_t attend_bwd_workspace(const BwdPlan &p, int64_t Tq, int64_t Tk, int Hq, int Hkv, int D, int P) {
  const int64_t stat = up_to(Tq * Hq * 8, 16), width = D + P;
  const int64_t kpart = (int64_t)p.kshares * 4 * 128 * width * 4;             // dK and dV, two slots a share
  const int64_t qpart = p.qsplit > 1 ? (int64_t)p.qsplit * Tq * Hq * width * 4 : 0;
  return (size_t)(stat + Tk * Hkv * P * 4 + (kpart > qpart ? kpart : qpart));
}

int64_t attend_bwd_threads(const BwdPlan &p, int Hkv) {
  const int64_t sum = p.qsplit > 1 ? p.qtiles * Hkv * 8 * 256 : 0;
  return std::max({p.ktiles * Hkv * 512, p.qtiles * p.qsplit * Hkv * kBwdWaves * 64, sum});
}

namespace {

BwdArgs make_bwd_args(const AttendCall &c, const uint16_t *d_o, const BwdPlan &p, void *workspace, uint16_t *dq,
                      uint16_t *dk, uint16_t *dv) {
  BwdArgs a{};
  a.q = c.q, a.k = c.k, a.v = c.v, a.d_o = d_o, a.o = c.o, a.lse = c.lse;
  a.qs = c.q_stride, a.ks = c.k_stride, a.vs = c.v_stride;
  a.cu_q = c.cu_q, a.cu_k = c.cu_k, a.nseq = c.nseq, a.Hq = c.Hq, a.Hkv = c.Hkv, a.D = c.D;
  a.Tq = c.Tq, a.Tk = c.Tk;
  a.scale = c.scale, a.scale_log2 = c.scale * kLog2e;
  a.lse2 = (float *)workspace;
  a.delta = a.lse2 + c.Tq * c.Hq;
  a.part = (float *)((char *)workspace + up_to(c.Tq * c.Hq * 8, 16));
  a.qsplit = p.qsplit, a.qchunk = p.qchunk;
  a.dq = dq, a.dk = dk, a.dv = dv;
  return a;
}

}  // namespace

hipError_t launch_attend_bwd(const AttendCall &c, const uint16_t *d_o, const BwdPlan &p, void *workspace,
                             uint16_t *dq, uint16_t *dk, uint16_t *dv, hipStream_t st) {
  const BwdArgs a = make_bwd_args(c, d_o, p, workspace, dq, dk, dv);
  return c.D <= 64 ? launch_bwd_t<64, 0>(c, p, a, st) : launch_bwd_t<128, 0>(c, p, a, st);
}

hipError_t launch_expanded_bwd(const AttendCall &c, const ExpandedKeys &x, const uint16_t *d_o, const BwdPlan &p,
                               void *workspace, uint16_t *dq, uint16_t *dk, uint16_t *dk_pe, uint16_t *dv,
                               hipStream_t st) {
  BwdArgs a = make_bwd_args(c, d_o, p, workspace, dq, dk, dv);
  a.pe = x.k_pe, a.pes = x.pe_stride, a.kh = x.k_head, a.vh = x.v_head, a.P = x.P, a.QD = c.D + x.P;
  a.pe_part = a.part, a.part += c.Tk * c.Hkv * x.P;
  a.dpe = dk_pe;
  return c.D <= 64 ? launch_bwd_t<64, 64>(c, p, a, st) : launch_bwd_t<128, 64>(c, p, a, st);
}

}  // namespace kpool
