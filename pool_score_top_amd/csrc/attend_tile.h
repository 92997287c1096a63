// Device pieces shared by the attention kernels (attend.hip, attend_bwd.hip): key tiles in
// LDS, their loads and fragments, and where a workgroup's query rows sit.
//
// Query rows.  The G = Hq / Hkv query heads of one key head see the same keys, so the G
// heads of the Lq tokens of a sequence form one axis of Lq * G "virtual" rows, row n being
// head n % G of token n / G.  A tile of virtual rows then shares every key it reads among
// the heads as well as the tokens, and one new token of a serving step fills G rows.
//
// Matrix products are v_mfma_f32_32x32x16_bf16.  Lane l holds of A row l % 32 and of B
// column l % 32, each the 8 values k = 8 (l / 32) + j; of the result column l % 32 and rows
// 8 (i / 4) + 4 (l / 32) + i % 4, i < 16.  A product whose result is the next one's B
// operand (S^T = K Q^T, then O^T = V^T P^T) needs no exchange between lanes: registers
// 8c .. 8c + 7 of the result are B for 16 of the contracted indexes, in the order
// 4 h + {0..3}, 8 + 4 h + {0..3} of lane half h, and the A operand is read in that order.
//
// Key tiles in LDS.  A row of DP bf16 values is DP / 8 slots of 16 bytes; slot s holds chunk
// s ^ swz(row).  Two kinds of reads have to be free of bank conflicts (64 banks, 256 bytes a
// phase): 16-byte reads of one chunk of 32 rows, whose phases hold rows {0-3, 12-15, 20-27}
// and {4-11, 16-19, 28-31}, and transposing 8-byte reads of 4 consecutive rows by 64 bytes.
// The first needs swz to differ over a phase's rows (row % 16 does), the second needs the 4
// rows' 64-byte blocks to differ, so the row's lowest bits go to the chunk's highest ones.
#pragma once

#include <algorithm>

#include "layer_internal.h"

namespace kpool {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

#define KPOOL_LDS __attribute__((address_space(3)))

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// (HIP's min of two integer types goes through double)
__host__ __device__ inline int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

template <int DP>
struct Keys {
  static_assert(DP == 64 || DP == 128, "padded head dims");
  static constexpr int ROWB = DP * 2;            // bytes of a row
  static constexpr int KS = DP / 16;             // contraction steps over the head dim
  static constexpr int DT = DP / 32;             // 32-wide blocks of the head dim
  static constexpr int REGION_ROWS = 1024 / ROWB;  // rows of one wave-wide 1 KiB load

  static __device__ inline int swz(int row) {
    const int r = DP == 128 ? row : row >> 1;
    return DP == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r & 1) << 2) | ((r >> 1) & 3);
  }
  // byte of chunk 0's fragment for row l % 32, half l / 32; chunk step ks is ^ (ks << 5)
  static __device__ inline uint32_t row_base(int lane) {
    const int row = lane & 31;
    return row * ROWB + (((lane >> 5) ^ swz(row)) << 4);
  }
  // byte of the transposing read of rows 4 h + {0..3} (+ 8 where second), columns 0..31;
  // column block dt is ^ (dt << 6), 16 rows further down + 16 * ROWB
  static __device__ inline uint32_t col_base(int lane, int second) {
    const int i = lane & 15, g = lane >> 4;
    const int row = 8 * second + 4 * (g >> 1) + (i >> 2);
    const int chunk = (g & 1) * 2 + ((i & 3) >> 1);
    return row * ROWB + ((chunk ^ swz(row)) << 4) + (i & 1) * 8;
  }
};

__device__ inline uint32_t lds_offset(const void *p) {
  return (uint32_t)(uintptr_t)(KPOOL_LDS const char *)p;
}
__device__ inline bf16x8 lds_read(uint32_t at) { return *(KPOOL_LDS const bf16x8 *)(uintptr_t)at; }

// A operand for 16 contracted rows, transposed out of LDS: two reads of 4 rows each half
__device__ inline bf16x8 lds_read_cols(uint32_t first, uint32_t second) {
  typedef short i16x8 __attribute__((ext_vector_type(8)));
  const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KPOOL_LDS i16x4 *)(uintptr_t)first);
  const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KPOOL_LDS i16x4 *)(uintptr_t)second);
  const i16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}

// Keeps the compiler from looking through a value.
__device__ inline void opaque(uint32_t &x) { asm volatile("" : "+v"(x)); }

// A lane's addresses of the fragments of a key tile
template <int DP>
struct Frag {
  using S = Keys<DP>;
  uint32_t row[S::KS], col0[S::DT], col1[S::DT];
  __device__ inline void init(uint32_t lds0, int lane) {
    const uint32_t rb = S::row_base(lane), c0 = S::col_base(lane, 0), c1 = S::col_base(lane, 1);
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) row[ks] = lds0 + (rb ^ (ks << 5));
#pragma unroll
    for (int dt = 0; dt < S::DT; ++dt) col0[dt] = lds0 + (c0 ^ (dt << 6)), col1[dt] = lds0 + (c1 ^ (dt << 6));
    // (opaque, so that a tile's constant offset stays apart and goes into the read itself)
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) opaque(row[ks]);
#pragma unroll
    for (int dt = 0; dt < S::DT; ++dt) opaque(col0[dt]), opaque(col1[dt]);
  }
  // rows l % 32 from `off` on, contraction step ks over the head dim
  __device__ inline bf16x8 rows(uint32_t off, int ks) const { return lds_read(row[ks] + off); }
  // columns 32 dt + l % 32, contraction over the 16 rows from `off` on
  __device__ inline bf16x8 cols(uint32_t off, int dt) const {
    return lds_read_cols(col0[dt] + off, col1[dt] + off);
  }
};

// The same for v_mfma_f32_16x16x32_bf16, whose operands are 16 rows of 32 values (lane l: row
// l % 16, values 8 (l / 16) + j) and whose result has column l % 16 and rows 4 (l / 16) + i,
// i < 4: results of 32 keys, 16 at a time, are the next product's B operand in the order
// 4 g + {0..3}, 16 + 4 g + {0..3} of lane group g = l / 16.  A phase of the 16-byte reads holds 8
// rows' chunk c and 8 other rows' chunk c ^ 1, one of the transposing reads 8 rows by 32 bytes.
template <int DP>
struct Keys16 : Keys<DP> {
  static constexpr int KS = DP / 32, DT = DP / 16;
  static __device__ inline int swz(int row) {
    if (DP == 64) return ((row >> 1) & 3) << 1;
    const int quad = (row >> 2) & 3, gray = quad ^ (quad >> 1);
    return (row & 3) << 2 | (gray & 1) << 1 | gray >> 1;
  }
};
template <int DP>
struct Frag16 {
  using S = Keys16<DP>;
  uint32_t row[S::KS], col[S::DT];
  __device__ inline void init(uint32_t lds0, int lane) {
    const int r = lane & 15, g = lane >> 4, c = 4 * g + (r >> 2);  // (the transposing read's row)
    const uint32_t rb = r * S::ROWB + ((g ^ S::swz(r)) << 4);
    const uint32_t cb = c * S::ROWB + ((((r & 3) >> 1) ^ S::swz(c)) << 4) + (r & 1) * 8;
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) row[ks] = lds0 + (rb ^ (ks << 6)), opaque(row[ks]);
#pragma unroll
    for (int dt = 0; dt < S::DT; ++dt) col[dt] = lds0 + (cb ^ (dt << 5)), opaque(col[dt]);
  }
  // rows l % 16 from `off` on, contraction step ks over the head dim
  __device__ inline bf16x8 rows(uint32_t off, int ks) const { return lds_read(row[ks] + off); }
  // columns 16 dt + l % 16, contraction over the 32 rows from `off` on
  __device__ inline bf16x8 cols(uint32_t off, int dt) const {
    return lds_read_cols(col[dt] + off, col[dt] + off + 16 * S::ROWB);
  }
};

__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// registers 8c .. 8c + 7 of a result as a B operand, each value rounded to bf16
__device__ inline bf16x8 as_operand(const f32x16 &p, int c) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = {pack_bf16(p[8 * c], p[8 * c + 1]), pack_bf16(p[8 * c + 2], p[8 * c + 3]),
                   pack_bf16(p[8 * c + 4], p[8 * c + 5]), pack_bf16(p[8 * c + 6], p[8 * c + 7])};
  return __builtin_bit_cast(bf16x8, v);
}

// and what that rounding took from them, rounded to bf16 in turn
__device__ inline bf16x8 as_operand_rest(const f32x16 &p, int c, bf16x8 rounded) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 r = __builtin_bit_cast(u32x4, rounded);
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack_bf16(p[8 * c + 2 * i] - __uint_as_float(r[i] << 16),
                     p[8 * c + 2 * i + 1] - __uint_as_float(r[i] & 0xFFFF0000u));
  return __builtin_bit_cast(bf16x8, v);
}

// the same value from the other half of the wave (lane ^ 32)
__device__ inline float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  // r[0] = [lo, lo], r[1] = [hi, hi]
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// the values of the lane and of lane ^ 16, in the same order in both
struct Pair {
  float a, b;
};
__device__ inline Pair row_pair(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// A workgroup barrier alone.  __syncthreads() also waits for all of the wave's loads, those
// that are meant to stay out among them; here the wave waits for what it needs beforehand.
// The compiler keeps LDS accesses on their side of it.
__device__ inline void barrier_only() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Waits for all of the wave's loads.  Before a loop it keeps the compiler, which would wait at
// the first use, from doing so in every round, for that round's loads as well.
__device__ inline void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// Waits for the wave's LDS reads: what it read may then be overwritten, by its own loads or, past
// a barrier, by others'.  (The values are long in use where this stands; it costs nothing and
// does not leave to the instructions' order what has to hold.)
__device__ inline void wait_reads() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
}

// 2^x by the hardware's instruction (relative error about 2^-23; -inf gives 0)
__device__ inline float exp2f_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ inline const void *uniform_ptr(const void *p) {
  const uint64_t a = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return (const void *)(((uint64_t)hi << 32) | lo);
}

// Loads from memory straight into LDS: lane i's 16 (or 4) bytes go to LDS byte `to` + 16 i
// (4 i).  Written as asm because the compiler, which knows the builtins' loads to write LDS,
// waits for all of them before each transposing LDS read and so for the tile that was just
// asked for.  The loads have no result registers; the kernels wait for them by count before
// the barrier behind which the tile is read, and the compiler's own waits, which do not count
// them, can only wait longer.  (One wait state between writing M0 and its use.)
__device__ inline void load_lds_16(const void *src, uint32_t to) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(to), "v"(src) : "memory");
#endif
}
__device__ inline void load_lds_4(const void *src, uint32_t to) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(to), "v"(src) : "memory");
#endif
}

// Reads key tiles of BK rows from memory straight into LDS, by NWAVES waves of which this is
// `wave`.  Row r of a tile comes from its base + min(r, last) * stride, so a tile that ends
// inside takes its last row again and every byte of LDS is a key's.  Chunks past D (head dims
// below DP) take the row's last chunk: they meet zeros of the query.  A wave's load covers
// REGION_ROWS rows; the rows' swizzles repeat every 16 rows, so loads 16 rows apart share
// their chunks' offsets.
template <int DP, int BK, int NWAVES>
struct KeyLoader {
  using S = Keys<DP>;
  static constexpr int REGIONS = BK / S::REGION_ROWS;
  static constexpr int PER = REGIONS / NWAVES;  // loads a wave
  static constexpr int CYCLE = 16 / S::REGION_ROWS;  // regions after which the swizzle repeats
  static constexpr int NOFF = PER < CYCLE ? PER : CYCLE;
  // (with several waves, a wave's regions are NWAVES apart, and those share one swizzle)
  static_assert(REGIONS % NWAVES == 0 && (NWAVES == 1 || NWAVES % CYCLE == 0), "regions of a wave");
  static constexpr int NCOL = NWAVES == 1 ? NOFF : 1;
  uint32_t col[NCOL];  // byte of the lane's chunk
  int wave, lane;

  __device__ inline void init(int wave_, int lane_, int D) {
    wave = wave_, lane = lane_;
#pragma unroll
    for (int i = 0; i < NCOL; ++i) {
      const int row = (wave + i) * S::REGION_ROWS + lane * 16 / S::ROWB;
      col[i] = min((lane & (DP / 8 - 1)) ^ S::swz(row), D / 8 - 1) * 16;
    }
  }
  // base and to (an LDS offset) are the same in every lane
  __device__ inline void load(const uint16_t *base, int64_t stride, int last, uint32_t to) const {
#if defined(__HIP_DEVICE_COMPILE__)
    const uint32_t pitch = (uint32_t)stride * 2;
    const uint64_t b = (uint64_t)uniform_ptr(base);
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 rs = {(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, 0xFFFFFFFFu, 0x00020000u};
    const int sub = lane * 16 / S::ROWB;  // the lane's row of a region
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int region = wave + i * NWAVES;
      const int row = min(region * S::REGION_ROWS + sub, last);
      // (load_lds_16 through a buffer resource: the lane holds a 32-bit offset)
      asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(to + region * 1024),
                   "v"(row * pitch + col[i % NCOL]), "s"(rs)
                   : "memory");
    }
#endif
  }
};

// Where a tile sits: BQ virtual rows of a sequence's queries, or 128 keys (cu_q and cu_k
// exchanged, G = 1).
struct TileAt {
  int seq;     // -1: no such tile
  int n0;      // its first virtual row
  int q_start, k_start;
  int Lq, Lk;
};

// Workgroups go to the 8 XCDs in turn, and units of work (tile, part) of one key head often
// repeat in weight with a period that divides 8 (the parts of a tile), which would give some
// XCDs all the heavy ones: unit u of n takes the place of another of its 8, a different one in
// every 8 (a packed batch of 4097, 2050, 1500, 513, 33 and 1 tokens, 32 heads over 4: 226 us
// without, 216 with it).
__device__ inline int64_t spread(int64_t u, int64_t n) {
  const int64_t b = u >> 3;
  return b * 8 + 8 <= n ? b * 8 + ((u + b) & 7) : u;
}

// Tiles of up to kTableSeqs sequences are found in a table that travels with the arguments,
// longest sequence first: workgroups start in this order, and what starts last should be
// short.  (A packed batch of 4097, 2050, .. 1 tokens takes 225 us so, and 245 with the shortest
// sequence first.)  `last_first` walks a sequence from its end, where
// causal rows see the most keys.
constexpr int kTableSeqs = 32;
struct TileTable {
  int32_t n;  // 0: more sequences than that; find_tile searches cu_q
  int32_t last_first;
  int32_t tile0[kTableSeqs + 1];
  int32_t q_start[kTableSeqs], k_start[kTableSeqs], Lq[kTableSeqs], Lk[kTableSeqs];
};

// Without a table, tiles are numbered through the batch with sequence s starting at tile
// cu_q[s] * G / BQ + s: that leaves room for ceil(Lq * G / BQ) tiles each (a sequence may leave
// its last number unused).
__host__ __device__ inline int64_t tile_start(int64_t cu, int s, int G, int BQ) {
  return cu * G / BQ + s;
}

// Fills in the table and returns the number of tiles.
inline int64_t make_table(TileTable &t, const int32_t *cu_q, const int32_t *cu_k, int nseq, int G, int BQ,
                          bool last_first) {
  t.n = 0;
  t.last_first = last_first;
  int64_t tiles = 0;
  if (nseq > kTableSeqs) return tile_start(cu_q[nseq], nseq, G, BQ);
  for (int s = 0; s < nseq; ++s) {
    const int32_t lq = cu_q[s + 1] - cu_q[s], lk = cu_k[s + 1] - cu_k[s];
    if (lq == 0) continue;
    int i = t.n++;  // insertion by the walked length, longest first
    for (; i > 0 && t.Lk[i - 1] < lk; --i)
      t.q_start[i] = t.q_start[i - 1], t.k_start[i] = t.k_start[i - 1], t.Lq[i] = t.Lq[i - 1],
      t.Lk[i] = t.Lk[i - 1];
    t.q_start[i] = cu_q[s], t.k_start[i] = cu_k[s], t.Lq[i] = lq, t.Lk[i] = lk;
  }
  for (int i = 0; i < t.n; ++i) {
    t.tile0[i] = (int32_t)tiles;
    tiles += ((int64_t)t.Lq[i] * G + BQ - 1) / BQ;
  }
  for (int i = t.n; i <= kTableSeqs; ++i) t.tile0[i] = 0x7FFFFFFF;
  return tiles;
}

// All 64 lanes call it.  Tiles past the last one (their number is below the grid's) give seq -1.
__device__ inline TileAt find_tile(const TileTable &tab, const int32_t *__restrict__ cu_q,
                                   const int32_t *__restrict__ cu_k, int nseq, int G, int BQ, int64_t tile,
                                   int64_t ntiles, int lane) {
  TileAt r;
  if (tab.n > 0) {
    const int hits = __popcll(__ballot(lane < kTableSeqs && tab.tile0[lane & (kTableSeqs - 1)] <= (int)tile));
    const int i = __builtin_amdgcn_readfirstlane(hits - 1);
    r.seq = i;
    r.q_start = tab.q_start[i], r.k_start = tab.k_start[i], r.Lq = tab.Lq[i], r.Lk = tab.Lk[i];
    int local = (int)tile - tab.tile0[i];
    if (tab.last_first) local = (int)(((int64_t)r.Lq * G + BQ - 1) / BQ) - 1 - local;
    r.n0 = local * BQ;
    return r;
  }
  if (tab.last_first) tile = ntiles - 1 - tile;
  int lo = 0, n = nseq;  // the answer is in [lo, lo + n); 64 sequences are probed at a time
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int s = lo + lane * step;
    const bool below = s < lo + n && tile_start(cu_q[min(s, nseq)], s, G, BQ) <= tile;
    const int hits = __popcll(__ballot(below));
    const int at = lo + (hits > 0 ? hits - 1 : 0) * step;
    n = min(step, lo + n - at);
    lo = at;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int q0 = cu_q[lo], q1 = cu_q[lo + 1], k0 = cu_k[lo], k1 = cu_k[lo + 1];
  r.q_start = q0, r.k_start = k0, r.Lq = q1 - q0, r.Lk = k1 - k0;
  const int64_t n0 = (tile - tile_start(q0, lo, G, BQ)) * BQ;
  r.n0 = (int)n0;
  r.seq = n0 < (int64_t)r.Lq * G ? lo : -1;  // (Lq * G fits 32 bits, checked by the host)
  return r;
}

// Equal shares of a kernel's work.  Units (tile, key head) lie one behind the other, each as
// long as the steps that it walks and a fixed cost; workgroup w takes the steps from
// (unit[w], step[w]) to (unit[w + 1], step[w + 1]).  So all CUs end together, whatever the
// lengths, and a unit that lies across workgroups leaves at most two parts a workgroup to join:
// slot 2 w for the unit that w does not begin, slot 2 w + 1 for one that it begins and does not
// end.  n = 0: a workgroup per unit.
constexpr int kMostShares = 256;  // one a CU
struct Shares {
  int32_t n;
  int32_t unit[kMostShares + 1], step[kMostShares + 1];
};

// How many shares: `least` steps or more each, but as many as there are units for the CUs.  None
// where units by themselves end about as early: where no unit is longer than a share (and the
// steps of a join), and either they all run at once or there are so many that the last of them
// end close together.
inline int share_count(const TotalCost &c, int64_t least) {
  const int64_t n = std::min<int64_t>(kMostShares, std::max<int64_t>(c.units, c.total / least));
  if (n <= 1) return 0;
  const bool even = c.longest <= std::max(c.total / n, least) + 4;
  return even && (c.units <= kMostShares || c.units >= 4 * kMostShares) ? 0 : (int)n;
}

// Parts of the walked keys (64 a step) where there are fewer tiles than CUs: no tile walks more
// than the average of the CUs, or `least` steps, in one part.  All tiles start at their first key,
// so what runs at a time reads much the same keys; equal shares, which do not, find 48% of them in
// the L2 instead of 84% (dQ of 8192 packed tokens, 516 tiles: 235 us by equal shares, 200 by
// tiles, 200 and 6 to join with the longest tiles cut to the CUs' average).
inline void plan_parts(const TotalCost &c, int64_t least, int *nsplit, int *chunk) {
  const int64_t steps = std::max(c.total / kMostShares + 1, least);
  *nsplit = 1, *chunk = 0x7FFFFF00;
  if (c.units < kMostShares && c.most_steps > steps)
    *nsplit = (int)((c.most_steps + steps - 1) / steps), *chunk = (int)steps * 64;
}

// Calls f(tile, Lq, Lk, n0) for the tiles in the order of their numbers.
template <class F>
void for_tiles(const TileTable &t, const int32_t *cu_q, const int32_t *cu_k, int nseq, int G, int BQ,
               int64_t ntiles, F &&f) {
  const int seqs = t.n > 0 ? t.n : nseq;
  for (int i = 0; i < seqs; ++i) {
    const int s = t.n > 0 || !t.last_first ? i : nseq - 1 - i;
    const int64_t lq = t.n > 0 ? t.Lq[s] : cu_q[s + 1] - cu_q[s], lk = t.n > 0 ? t.Lk[s] : cu_k[s + 1] - cu_k[s];
    const int64_t n = (lq * G + BQ - 1) / BQ;
    for (int64_t j = 0; j < n; ++j) {
      const int64_t local = t.last_first ? n - 1 - j : j;
      const int64_t number = t.n > 0 ? t.tile0[s] + j : tile_start(cu_q[s], s, G, BQ) + local;
      f(t.n > 0 || !t.last_first ? number : ntiles - 1 - number, lq, lk, local * BQ);
    }
  }
}

// Fills in n shares; cost(Lq, Lk, n0) is a tile's, c their sum.  Parts of fewer than 4 steps are
// left to the neighbour.  Returns whether any unit lies across shares.
template <class F>
bool make_shares(Shares &sh, int n, const TotalCost &c, int Hkv, const TileTable &t, const int32_t *cu_q,
                 const int32_t *cu_k, int nseq, int G, int BQ, int64_t ntiles, F &&cost) {
  sh.n = n;
  if (n == 0) return false;
  sh.unit[0] = sh.step[0] = 0;
  bool cut = false;
  int w = 1;
  int64_t at = 0, next = c.total / n;
  for_tiles(t, cu_q, cu_k, nseq, G, BQ, ntiles, [&](int64_t tile, int64_t lq, int64_t lk, int64_t n0) {
    const UnitCost u = cost(lq, lk, n0);
    for (int h = 0; h < Hkv; ++h) {
      for (; w < n && next < at + u.fixed + u.steps; ++w, next = c.total * w / n) {
        int64_t step = next - at - u.fixed, unit = tile * Hkv + h;
        if (step < 4) step = 0;
        else if (step > u.steps - 4) step = 0, ++unit;
        sh.unit[w] = (int32_t)unit, sh.step[w] = (int32_t)step;
        cut |= step > 0;
      }
      at += u.fixed + u.steps;
    }
  });
  for (; w <= n; ++w) sh.unit[w] = (int32_t)(Hkv * ntiles), sh.step[w] = 0;
  return cut;
}

// A workgroup's steps: the units u0 .. u1, from step s0 of the first to s1 of the last.
struct Span {
  int share, u0, s0, u1, s1;
};
__device__ inline Span span_of(const Shares &sh, int block) {
  if (sh.n == 0) return {0, block, 0, block + 1, 0};
  return {block, sh.unit[block], sh.step[block], sh.unit[block + 1], sh.step[block + 1]};
}

// The shares [share, end) of the unit that `share` begins and does not end, or false.  All 64
// lanes call it.
__device__ inline bool begins_cut(const Shares &sh, int share, int lane, int &unit, int &end) {
  unit = sh.unit[share + 1];
  if (sh.step[share + 1] == 0 || (sh.unit[share] == unit && sh.step[share] > 0)) return false;
  uint64_t others;
  end = share + 1 - 64;
  do {  // (the last step is 0)
    end += 64;
    const int i = min(end + lane, sh.n);
    others = __ballot(sh.unit[i] != unit || sh.step[i] == 0);
  } while (others == 0);
  end += __builtin_ctzll(others);
  return true;
}

}  // namespace kpool
