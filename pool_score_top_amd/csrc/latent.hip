// Latent attention in its absorbed form: queries over a cache that holds one row of R + P values a
// token, which is the key of every head and whose first R values are its value.  For query head h of
// token row i, over the tokens j that the row sees (all up to its position, or those of its list):
//   s_j = scale <q[i,h,:], c[j,:]>,   o[i,h,:] = sum_j softmax_j(s) c[j,:R],   lse[i,h] = log sum_j e^s_j
//
// Pages: Atlas inference glm5next_dsa/tp.rs, shard plan: kv_a_proj_with_mqa gives the row, kv_b_proj
// is what is absorbed into the queries and the outputs; Megatron-LM PR #8299 "Mechanism": the selected
// tokens are what a row attends to.
//
// All heads share one key, so the heads of a sequence's new tokens form one axis of Lq * H rows
// (row n: head n % H of token n / H).  A workgroup of 4 waves, one a CU, takes up to 64 of them and walks
// key tiles of 64 through two LDS buffers (72 KiB each at R + P = 576), each read once from memory and used
// twice, as keys and, transposed, as values:
//   S^T = C Q^T, the queries in registers, which lie in the accumulation half of the file;
//   P to LDS in bf16, where all waves read it back;
//   O^T = C^T P^T: wave w keeps columns w R / 4 .. of all rows (128 registers a lane at 64 rows).
// Statistics as in attend.hip: fp32, base 2.  The maximum is followed only when a score lies more than 8
// (a factor of 256) above it: the waves vote on that through flags in LDS, and exchange maxima only then.  P is
// rounded to bf16 for its product (as the keys that it meets are), l is summed from the unrounded values.
//
// Keys lie anywhere (pages, lists): a block of 1024 (lists: 2048) of them is first turned into a list of
// rows in LDS, without those that do not exist, and tiles are gathered by it.  The next tile's loads
// go out one by one between the matrix instructions of S.
//
// Work goes by equal shares of all the units' costs, one share a CU.  Where the shares begin depends on
// the lengths, which are on the device (a captured decoding step replays while its lengths grow), so each
// workgroup finds its share itself.  A unit (rows of one tile) that lies across shares leaves a
// part each in fp32; a second kernel joins them in order.
//
// What bounds it, at R + P = 512 + 64 (captured calls, both kernels):
//   few rows: memory.  16 requests of one token, 205k cached tokens, 16 heads: 62.5 us; the first kernel
//     takes 45 (236 MB, 5.3 TB/s, as a copy of 268 MB does), the join 7;
//   many rows: the matrix instructions and what they wait for within a tile, as there is one wave a
//     SIMD: S 1600 cycles of 4200 (1152 of products), softmax and its exchange 700, O 1530 (1024), the
//     tile's arrival 310.  8 requests of 2 tokens, 128 heads, 117k tokens: 106 us (100 and 11; 65 GFLOP; CUs busy
//     79% of the time, the matrix pipe 36% of that): a unit's start and end take 22k cycles besides, 5 tiles' time;
//   lists of many rows: the listed rows' way from beyond the L2, which holds 12% of them.  1024 rows of 2048
//     tokens, 64 heads: 358 us, 2.4 GB at 7 TB/s (CUs busy 94%, the pipe 42% of that);
//   a token or two: latencies.  One token over 1003, 16 heads: 17 us (11 and 4);
//   chunks of a prompt: 512 tokens behind 8192, 16 heads 177 us (0.85 PFLOP/s), 128 heads 1176 us (1.03).  A unit
//     counts the tiles of its whole sequence, also of keys behind its rows: 2048 tokens of a new prompt, 16
//     heads, 153 us (0.48), which the expanded form is for.
#include <type_traits>

#include "attend_tile.h"

namespace kpool {
namespace {

constexpr int kLatentKeys = 64;

struct LatentArgs {
  const uint16_t *q, *cache;
  int64_t qs, cs, nrows;  // elements between tokens, between cache rows; cache rows
  const int32_t *table, *starts, *lens, *cu_q, *ids;
  int per_seq, page, npages, max_len;
  int nseq, H, R, P, width;
  float scale_log2;
  int shares, hblocks, units;  // most shares; lists: units of a token, of the call
  uint16_t *o;
  float *lse;
  struct LatentCut *cut;     // [shares]
  float *part_o, *part_lse;  // [2 * shares][BQ][R], [2 * shares][BQ]
};

// The unit that a share begins and does not end: where its tiles end, and its rows.
struct LatentCut {
  int64_t row0;
  int32_t end, total, shares, nrows;  // (end 0: none)
};

// Shares are of the units' costs: a unit costs its tiles and, where shares are of several tiles, `fixed` more
// for its start and end (rows of queries in, outputs out, no products meanwhile).  With tiles alone a share of
// many short units took up to twice its time: 8 requests of 2 tokens, 128 heads, us of the first kernel by tiles
// 118, by cost 93; 16 requests, 16 heads, 49.6 and 43.7 (whole calls: cost 3 62.6 and 103, 4 62.5 and 102, 6 64.1
// and 101; no other batches were measured for it).  Where shares are of fewer tiles, a unit has a share and more
// to itself either way.
// A cut that would leave a part of fewer than `least` tiles moves to the unit's start or end.
constexpr int kUnitCost = 4;
struct LatentCosts {
  int fixed, least, total, shares;
  __host__ __device__ inline LatentCosts(int tiles, int units, int most) {
    shares = most < tiles ? most : tiles;
    fixed = tiles >= 4 * shares ? kUnitCost : 0, least = fixed ? 4 : 1;
    total = tiles + fixed * units;
  }
  // the tiles before position x of a unit of kt tiles that starts at `start`
  __host__ __device__ inline int cut(int x, int start, int kt) const {
    const int t = x - start - fixed;
    return t > kt - least ? kt : t < least ? 0 : t;  // (its end before its start: a unit may be shorter than `least`)
  }
};

// Where the share begins.
__host__ __device__ inline int share_start(int total, int n, int share) {
  const int each = total / n;
  return each * share + (total - each * n) * share / n;
}

// The keys [lo, hi) by blocks, counted by what is left of them: the last block may end past 2^31, so no number
// past hi is formed.
struct KeyBlocks {
  int hi, left;
  __host__ __device__ inline KeyBlocks(int lo, int hi_) : hi(hi_), left(hi_ - lo) {}
  __host__ __device__ inline bool any() const { return left > 0; }
  __host__ __device__ inline int at() const { return hi - left; }  // the block's first key
  // key i of the block, -1 where there is none
  __host__ __device__ inline int key(int i) const { return i < left ? hi - left + i : -1; }
  __host__ __device__ inline void next(int size) { left -= size; }  // (below 0 behind the last, by less than size)
};

// A workgroup's tiles and LDS, NB blocks of 128 columns wide (R padded), for BQ rows.
template <int NB, int ROWS, bool LIST>
struct Latent {
  static constexpr int BK = kLatentKeys, BQ = ROWS;
  static constexpr int BLOCKB = BK * 256;           // bytes of 128 columns of a tile
  static constexpr int PE = NB * BLOCKB;            // where the positional part lies in it
  static constexpr int TILE = PE + BK * 128;
  static constexpr int LOADS = 4 * NB + 2;          // a wave's loads of a tile
  static constexpr int EACH = LIST ? 8 : 4, BLOCK = EACH * 256;
  // P; the rows of a block's keys, and, whole keys, their places.  What is used between tiles only
  // lies in the tiles (counts, the queries on their way to registers) or in P (exchanges of
  // maxima and sums), and a tile's four flags where the first keys of the list were, which are loaded.
  static constexpr int P = 2 * TILE, KEYS = P + BQ * BK * 2, PLACES = KEYS + BLOCK * 4,
                       LDS = PLACES + (LIST ? 0 : BLOCK * 4);
  static constexpr int CHUNKS = NB * 16 + 8;    // of 16 bytes in a row of queries
  static constexpr int QROW = CHUNKS * 16 + 16;  // its bytes in LDS (16 rows over all banks)
  static_assert(LDS <= 163840 && BQ * QROW <= TILE + BQ * BK * 2 && 4 * BQ * 4 <= BQ * BK * 2, "LDS");
};

// What a wave knows of a tile in LDS
struct TileKeys {
  uint32_t at;        // its first byte
  int first, present;  // number of its first key in the block, keys of the block
  bool masked;         // whether some row does not see some key
};

// n tokens of a sequence, at most what the caller said and what its pages hold
__device__ inline int latent_len(const LatentArgs &a, int s) {
  const int len = min(max(a.lens[s], 0), a.max_len);
  return a.table ? (int)min64(len, (int64_t)a.per_seq * a.page) : len;
}
__device__ inline int tiles_of(int keys) { return max(1, (keys + kLatentKeys - 1) / kLatentKeys); }
// a sequence's units (high 32 bits) and tiles
__device__ inline int64_t seq_work(const LatentArgs &a, int s, int BQ) {
  if (s >= a.nseq) return 0;
  const int units = ((a.cu_q[s + 1] - a.cu_q[s]) * a.H + BQ - 1) / BQ;
  return (int64_t)units << 32 | (int64_t)units * tiles_of(latent_len(a, s));
}

// Keeps the compiler from looking through a value that is the same in all lanes.
__device__ inline void opaque_uniform(uint32_t &x) { asm volatile("" : "+s"(x)); }

// Moves a fragment to accumulation registers, from where matrix instructions take it as it is.
__device__ inline void to_accumulation(bf16x8 &x) { asm volatile("" : "+a"(x)); }

// inclusive sum over the workgroup's 256 threads; scratch: 4 values of LDS.  All threads call it.
template <class T>
__device__ inline T scan_256(T x, T *scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T up = __shfl_up(x, d);
    if (lane >= d) x += up;
  }
  __syncthreads();
  if (lane == 63) scratch[wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x += scratch[w];
  return x;
}

// Up to 32 rows, by products of 16 rows: wave w has keys 16 w .. 16 w + 15 of a tile and all RB blocks
// of rows for S, columns w R / 4 .. and all rows for O.
template <int NB, int RB, bool LIST>
struct Latent16 {
  using C = Latent<NB, 16 * RB, LIST>;
  using S = Keys16<128>;
  using SP = Keys16<64>;
  static constexpr int KS = NB * 4 + 2;  // contraction steps of 32: the latent part, then the positional
  static constexpr int CB = NB * 2;      // 16-column blocks of a wave
  static constexpr int VALUES = 2 * CB, AHEAD = VALUES < 4 ? VALUES : 4;
  int wave, lane, col, group;
  // addresses are kept as few registers and made where they are used: (a ^ b) + c is one instruction
  uint32_t krow, kpe, vcol;
  bf16x8 q[RB][KS];
  f32x4 o[CB][RB], s[RB];
  float m[RB], l[RB], part[RB], top[RB];
  int t[RB];  // positions of the lane's rows (whole keys)
  bf16x8 v[VALUES], p[2][RB];

  __device__ inline void init(int wave_, int lane_) {
    wave = wave_, lane = lane_, col = lane & 15, group = lane >> 4;
    const int key = 4 * group + (col >> 2);
    krow = (wave * 16 + col) * 256 + ((group ^ S::swz(col)) << 4);
    kpe = (wave * 16 + col) * 128 + ((group ^ SP::swz(col)) << 4);
    vcol = key * 256 + ((((col & 3) >> 1) ^ S::swz(key)) << 4) + (col & 1) * 8;
    opaque(krow), opaque(kpe), opaque(vcol);
  }
  // position(r): the token position of row r
  template <class F>
  __device__ inline void begin(uint32_t queries, F &&position) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = rb * 16 + col;
      t[rb] = LIST ? 0 : position(r);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        q[rb][ks] = lds_read(queries + r * C::QROW + ks * 64 + group * 16);
        to_accumulation(q[rb][ks]);
      }
      m[rb] = -__builtin_inff(), l[rb] = 0.0f;
#pragma unroll
      for (int c = 0; c < CB; ++c) o[c][rb] = f32x4{};
    }
  }
  __device__ inline bf16x8 key(const TileKeys &k, int ks) const {
    return ks < NB * 4 ? lds_read((krow ^ ((ks & 3) << 6)) + (k.at + (ks >> 2) * C::BLOCKB))
                       : lds_read((kpe ^ ((ks & 1) << 6)) + (k.at + C::PE));
  }
  __device__ inline bf16x8 value(const TileKeys &k, int i) const {  // columns i % CB of the wave's, keys 32 (i / CB) ..
    const int c = wave * CB + i % CB;
    const uint32_t at = (vcol ^ ((c & 7) << 5)) + (k.at + (c >> 3) * C::BLOCKB + i / CB * 32 * 256);
    return lds_read_cols(at, at + 16 * 256);
  }
  // S.  Keys are read a few steps ahead; the next tile's loads go out beside the products, a load's
  // address and the load itself apart (a product takes 16 cycles, of which 12 are left for others).
  template <class L>
  __device__ inline void scores(const TileKeys &k, L &&loads) {
    constexpr int KAHEAD = 4;
    bf16x8 kr[KS];
#pragma unroll
    for (int n = 0; n < KAHEAD; ++n) kr[n] = key(k, n);
#pragma unroll
    for (int n = 0; n < KS; ++n) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        __builtin_amdgcn_sched_barrier(0);
        s[rb] = mfma(kr[n], q[rb][n], n == 0 ? f32x4{} : s[rb]);
        __builtin_amdgcn_sched_barrier(0);
        if (rb == 0) loads.address(n);
        if (rb == 0 && RB > 1) __builtin_amdgcn_sched_barrier(0);
        if (rb == RB - 1) {
          loads.issue(n);
          if (n + KAHEAD < KS) kr[n + KAHEAD] = key(k, n + KAHEAD);
        }
      }
    }
    static_assert(KS == C::LOADS, "a load a step");
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ inline void mask(const TileKeys &k, const int *places) {
    if (!k.masked) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = k.first + wave * 16 + 4 * group + i;
      const bool absent = n >= k.present;
      const int place = absent || LIST ? 0 : places[n];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
        if (absent || (!LIST && place > t[rb])) s[rb][i] = -__builtin_inff();
    }
  }
  // P to LDS, with the maxima so far
  __device__ inline void weights(uint32_t to, float c) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const float shift = m[rb] > -__builtin_inff() ? m[rb] : 0.0f;
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = exp2f_fast(fmaf(s[rb][i], c, -shift));
      part[rb] = (x[0] + x[1]) + (x[2] + x[3]);
      // row r: 16-byte chunks, each with a lane group's 8 keys of a contraction of 32 in the order of
      // lds_read_cols
      const int r = rb * 16 + col, chunk = (wave >> 1) * 4 + group;
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *(KPOOL_LDS u32x2 *)(uintptr_t)(to + r * 128 + ((chunk ^ (r & 7)) << 4) + (wave & 1) * 8) =
          u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    }
  }
  // whether a score lies far above its row's maximum so far (m = -inf: any visible key)
  __device__ inline bool over(float c) {
    bool far = false;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      top[rb] = fmaxf(fmaxf(s[rb][0], s[rb][1]), fmaxf(s[rb][2], s[rb][3]));
      far |= top[rb] * c > m[rb] + 8.0f;
    }
    return far;
  }
  // a value of each row, found over the lanes that share it, to the exchange [4][BQ]
  template <class F>
  __device__ inline void give(float *exchange, const float (&x)[RB], F &&join) const {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const Pair y = row_pair(x[rb]);
      const float z = join(y.a, y.b), all = join(z, other_half(z));
      if (lane < 16) exchange[wave * C::BQ + rb * 16 + col] = all;
    }
  }
  __device__ inline void give_top(float *exchange) const {
    give(exchange, top, [](float a, float b) { return fmaxf(a, b); });
  }
  __device__ inline void raise(const float *exchange, float c) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const float *x = exchange + rb * 16 + col;
      const float most = fmaxf(fmaxf(x[0], x[C::BQ]), fmaxf(x[2 * C::BQ], x[3 * C::BQ])) * c;
      if (most > m[rb] + 8.0f) {  // (the same in every wave)
        const float f = exp2f_fast(m[rb] - most);  // m = -inf gives 0
        m[rb] = most, l[rb] *= f;
#pragma unroll
        for (int b = 0; b < CB; ++b) o[b][rb] *= f;
      }
    }
  }
  __device__ inline void read_values(const TileKeys &k) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) v[i] = value(k, i);
  }
  __device__ inline void read_p(uint32_t from, int kc) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = rb * 16 + col;
      p[kc][rb] = lds_read(from + r * 128 + (((kc * 4 + group) ^ (r & 7)) << 4));
    }
  }
  __device__ inline void first_p(uint32_t from) { read_p(from, 0); }
  // O, once read_values and first_p have begun
  __device__ inline void values(const TileKeys &k, uint32_t p_at) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) l[rb] += part[rb];
#pragma unroll
    for (int i = 0; i < VALUES; ++i) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        __builtin_amdgcn_sched_barrier(0);
        o[i % CB][rb] = mfma(v[i], p[i / CB][rb], o[i % CB][rb]);
        __builtin_amdgcn_sched_barrier(0);
        if (rb == 0 && i + AHEAD < VALUES) v[i + AHEAD] = value(k, i + AHEAD);
      }
      if (i == 1) read_p(p_at, 1);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ inline void give_sum(float *exchange) const {
    give(exchange, l, [](float a, float b) { return a + b; });
  }
  // out(r, lse) for the rows, then to8(r, column, 8 values packed) or to4(r, column, 4 values)
  template <class L, class F8, class F4>
  __device__ inline void finish(const float *exchange, bool whole, L &&out, F8 &&to8, F4 &&to4) const {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = rb * 16 + col;
      const float *x = exchange + r;
      const float sum = (x[0] + x[C::BQ]) + (x[2 * C::BQ] + x[3 * C::BQ]);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (wave == 0 && group == 0) out(r, m[rb], sum);
#pragma unroll
      for (int c = 0; c < CB; c += 2) {
        const int d = (wave * CB + c) * 16;
        const f32x4 y0 = o[c][rb] * inv, y1 = o[c + 1][rb] * inv;
        if (whole) {
          // lane groups exchange halves: groups 0 and 2 take 8 columns each of the first block, 1 and 3 of
          // the second
          const auto a = __builtin_amdgcn_permlane16_swap(pack_bf16(y0[0], y0[1]), pack_bf16(y1[0], y1[1]), false, false);
          const auto b = __builtin_amdgcn_permlane16_swap(pack_bf16(y0[2], y0[3]), pack_bf16(y1[2], y1[3]), false, false);
          to8(r, d + (group & 1) * 16 + (group >> 1) * 8, make_uint4(a[0], b[0], a[1], b[1]));
        } else {
          to4(r, d + group * 4, y0);
          to4(r, d + 16 + group * 4, y1);
        }
      }
    }
  }
};

// 64 rows, by products of 32 rows, half as many instructions for the same work (8 requests of 2 tokens, 128
// heads, 123 us by products of 16 rows, 118 so): wave w has 32 keys (w / 2)
// and 32 rows (w % 2) for S, columns w R / 4 .. and all rows for O.  Queries of 64 rows for 16 keys a
// wave would read each key once instead of twice, but take 288 registers beside O's 128: they spill.
template <int NB, bool LIST>
struct Latent32 {
  using C = Latent<NB, 64, LIST>;
  using S = Keys<128>;
  using SP = Keys<64>;
  static constexpr int KS = NB * 8 + 4;  // contraction steps of 16
  static constexpr int CB = NB;          // 32-column blocks of a wave
  static constexpr int VALUES = 4 * CB, AHEAD = VALUES < 4 ? VALUES : 4;
  int wave, lane, col, half, rows0, keys0;
  uint32_t krow, kpe, vcol0, vcol1;
  bf16x8 q[KS];
  f32x16 o[CB][2], s;
  float m[2], l, part, top;  // m: of rows l % 32 and 32 + l % 32; the others of the wave's own row
  int t;
  bf16x8 v[VALUES], p[4][2];

  __device__ inline void init(int wave_, int lane_) {
    wave = wave_, lane = lane_, col = lane & 31, half = lane >> 5;
    rows0 = (wave & 1) * 32, keys0 = (wave >> 1) * 32;
    krow = keys0 * 256 + S::row_base(lane), kpe = keys0 * 128 + SP::row_base(lane);
    vcol0 = S::col_base(lane, 0), vcol1 = S::col_base(lane, 1);
    opaque(krow), opaque(kpe), opaque(vcol0), opaque(vcol1);
  }
  template <class F>
  __device__ inline void begin(uint32_t queries, F &&position) {
    t = LIST ? 0 : position(rows0 + col);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks] = lds_read(queries + (rows0 + col) * C::QROW + ks * 32 + half * 16);
      to_accumulation(q[ks]);
    }
    l = 0.0f;
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      m[rb] = -__builtin_inff();
#pragma unroll
      for (int c = 0; c < CB; ++c) o[c][rb] = f32x16{};
    }
  }
  __device__ inline float own() const {
    const float first = m[0], second = m[1];
    return rows0 ? second : first;
  }
  __device__ inline bf16x8 key(const TileKeys &k, int ks) const {
    return ks < NB * 8 ? lds_read((krow ^ ((ks & 7) << 5)) + (k.at + (ks >> 3) * C::BLOCKB))
                       : lds_read((kpe ^ ((ks & 3) << 5)) + (k.at + C::PE));
  }
  __device__ inline bf16x8 value(const TileKeys &k, int i) const {  // columns i % CB of the wave's, keys 16 (i / CB) ..
    const int c = wave * CB + i % CB;
    const uint32_t to = k.at + (c >> 2) * C::BLOCKB + i / CB * 16 * 256;
    return lds_read_cols((vcol0 ^ ((c & 3) << 6)) + to, (vcol1 ^ ((c & 3) << 6)) + to);
  }
  // (two sums in turn: a product's result is not there yet when the next one starts)
  template <class L>
  __device__ inline void scores(const TileKeys &k, L &&loads) {
    constexpr int KAHEAD = 4;
    bf16x8 kr[KS];
    f32x16 x[2];
#pragma unroll
    for (int n = 0; n < KAHEAD; ++n) kr[n] = key(k, n);
#pragma unroll
    for (int n = 0; n < KS; ++n) {
      __builtin_amdgcn_sched_barrier(0);
      x[n & 1] = mfma(kr[n], q[n], n < 2 ? f32x16{} : x[n & 1]);
      __builtin_amdgcn_sched_barrier(0);
      if (n + KAHEAD < KS) kr[n + KAHEAD] = key(k, n + KAHEAD);
      if (n & 1) loads.issue(n / 2);
      else loads.address(n / 2);
    }
    static_assert(KS == 2 * C::LOADS, "a load for two steps");
    __builtin_amdgcn_sched_barrier(0);
    s = x[0] + x[1];
  }
  __device__ inline void mask(const TileKeys &k, const int *places) {
    if (!k.masked) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = k.first + keys0 + 8 * (i / 4) + 4 * half + i % 4;
      const bool absent = n >= k.present;
      if (absent || (!LIST && places[absent ? 0 : n] > t)) s[i] = -__builtin_inff();
    }
  }
  __device__ inline void weights(uint32_t to, float c) {
    const float most = own(), shift = most > -__builtin_inff() ? most : 0.0f;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = exp2f_fast(fmaf(s[i], c, -shift));
      sum[i % 4] += x[i];
    }
    part = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    // 16-byte chunks of row r, each with a lane half's 8 keys of 16
    const int r = rows0 + col;
#pragma unroll
    for (int kc = 0; kc < 2; ++kc)
      *(KPOOL_LDS bf16x8 *)(uintptr_t)(to + r * 128 + (((keys0 / 8 + kc * 2 + half) ^ (r & 7)) << 4)) = as_operand(x, kc);
  }
  __device__ inline bool over(float c) {
    top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    return top * c > own() + 8.0f;
  }
  __device__ inline void give_top(float *exchange) const {
    const float x = fmaxf(top, other_half(top));
    if (lane < 32) exchange[(wave >> 1) * 64 + rows0 + col] = x;
  }
  __device__ inline void raise(const float *exchange, float c) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      const float most = fmaxf(exchange[rb * 32 + col], exchange[64 + rb * 32 + col]) * c;
      if (most > m[rb] + 8.0f) {  // (the same in every wave)
        const float f = exp2f_fast(m[rb] - most);  // m = -inf gives 0
        m[rb] = most;
        if (rows0 == rb * 32) l *= f;
#pragma unroll
        for (int b = 0; b < CB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[b][rb][i] *= f;
      }
    }
  }
  __device__ inline void read_values(const TileKeys &k) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) v[i] = value(k, i);
  }
  __device__ inline void read_p(uint32_t from, int kc) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      const int r = rb * 32 + col;
      p[kc][rb] = lds_read(from + r * 128 + (((kc * 2 + half) ^ (r & 7)) << 4));
    }
  }
  __device__ inline void first_p(uint32_t from) { read_p(from, 0), read_p(from, 1); }
  __device__ inline void values(const TileKeys &k, uint32_t p_at) {
    l += part;
#pragma unroll
    for (int i = 0; i < VALUES; ++i) {
#pragma unroll
      for (int rb = 0; rb < 2; ++rb) {
        __builtin_amdgcn_sched_barrier(0);
        o[i % CB][rb] = mfma(v[i], p[i / CB][rb], o[i % CB][rb]);
        __builtin_amdgcn_sched_barrier(0);
        if (rb == 0 && i + AHEAD < VALUES) v[i + AHEAD] = value(k, i + AHEAD);
        if (rb == 1 && i < 2) read_p(p_at, 2 + i);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ inline void give_sum(float *exchange) const {
    const float x = l + other_half(l);
    if (lane < 32) exchange[(wave >> 1) * 64 + rows0 + col] = x;
  }
  template <class L, class F8, class F4>
  __device__ inline void finish(const float *exchange, bool whole, L &&out, F8 &&to8, F4 &&to4) const {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      const int r = rb * 32 + col;
      const float sum = exchange[r] + exchange[64 + r];
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (wave == 0 && half == 0) out(r, m[rb], sum);
#pragma unroll
      for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          const int d = (wave * CB + c) * 32 + 2 * i;
          f32x4 y0, y1;
#pragma unroll
          for (int u = 0; u < 4; ++u) y0[u] = o[c][rb][i + u] * inv, y1[u] = o[c][rb][i + 4 + u] * inv;
          if (whole) {
            // the halves exchange: the first takes 8 columns of the first 8, the second those of the next
            const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16(y0[0], y0[1]), pack_bf16(y1[0], y1[1]), false, false);
            const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16(y0[2], y0[3]), pack_bf16(y1[2], y1[3]), false, false);
            to8(r, d + half * 8, make_uint4(a[0], b[0], a[1], b[1]));
          } else {
            to4(r, d + half * 4, y0);
            to4(r, d + 8 + half * 4, y1);
          }
        }
    }
  }
};

template <int NB, int RB, bool LIST>
using LatentRows = std::conditional_t<RB == 4, Latent32<NB, LIST>, Latent16<NB, RB == 4 ? 1 : RB, LIST>>;

template <int NB, int RB, bool LIST>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void latent_kernel(LatentArgs a) {
  using R = LatentRows<NB, RB, LIST>;
  using C = typename R::C;
  constexpr int BK = C::BK, BQ = C::BQ, TILE = C::TILE;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = lds_offset(lds);

  // this workgroup's share of all units' costs: [pos, hi), from sequence `seq` on, whose units begin at `before`
  int before, seq, tiles, units_all;
  int64_t mine = 0, upto = 0;  // work of the thread's sequence, and up to its end
  const int list_tiles = LIST ? tiles_of(a.width) : 0;
  int64_t *scratch = reinterpret_cast<int64_t *>(lds);
  if (LIST) {
    tiles = a.units * list_tiles, units_all = a.units;
  } else {
    int64_t all = 0;
    for (int base = 0; base < a.nseq; base += 256) {
      mine = seq_work(a, base + threadIdx.x, BQ);
      upto = all + scan_256(mine, scratch);
      if (threadIdx.x == 255) scratch[4] = upto;
      __syncthreads();
      all = scratch[4];
    }
    tiles = __builtin_amdgcn_readfirstlane((int)all), units_all = __builtin_amdgcn_readfirstlane((int)(all >> 32));
  }
  const LatentCosts costs(tiles, units_all, a.shares);
  // (workgroups go to the 8 XCDs in turn: those of one take neighbouring shares)
  const int share = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (threadIdx.x == 0 && a.cut && share < a.shares) a.cut[share].end = 0;
  if (share >= costs.shares) return;
  const int pos = share_start(costs.total, costs.shares, share), hi = share_start(costs.total, costs.shares, share + 1);
  if (LIST) {
    const int token = pos / (list_tiles + costs.fixed) / a.hblocks;
    int step = a.nseq;  // (the sequence of a token: the last that starts at or before it)
    seq = 0;
    while (step > 1) {
      const int half = step / 2;
      if (a.cu_q[seq + half] <= token) seq += half;
      step -= half;
    }
    before = a.cu_q[seq] * a.hblocks * (list_tiles + costs.fixed);
  } else {
    auto cost = [&](int64_t work) { return (int)work + costs.fixed * (int)(work >> 32); };
    int64_t run = 0;
    for (int base = 0; base < a.nseq; base += 256) {
      if (a.nseq > 256) {  // (otherwise they are as they were)
        mine = seq_work(a, base + threadIdx.x, BQ);
        upto = run + scan_256(mine, scratch);
        if (threadIdx.x == 255) scratch[4] = upto;
      }
      if (cost(upto - mine) <= pos && pos < cost(upto)) scratch[5] = cost(upto - mine), scratch[6] = base + threadIdx.x;
      __syncthreads();
      run = scratch[4];
    }
    before = __builtin_amdgcn_readfirstlane((int)scratch[5]), seq = __builtin_amdgcn_readfirstlane((int)scratch[6]);
  }

  R r;
  r.init(wave, lane);
  // Loads: of the latent part 4 NB a wave, 4 rows each; of the positional one 2 a wave, 8 rows each.  A
  // lane's chunk of its row is chunk ^ swz(4 i) (i the load's place in 16 rows; 8 i), its last where the
  // row ends before it.
  constexpr int LOADS = C::LOADS;
  const uint32_t pitch = (uint32_t)a.cs * 2;
  const uint16_t *from[4], *pe_from[2];  // the lane's places in row 0
  {
    const int chunk = wave * NB / 4 * 16 + ((lane & 15) ^ R::S::swz(lane >> 4)), pe = (lane & 7) ^ R::SP::swz(lane >> 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) from[i] = a.cache + min(chunk ^ R::S::swz(4 * i), a.R / 8 - 1) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) pe_from[i] = a.cache + (a.P ? a.R + min(pe ^ R::SP::swz(8 * i), a.P / 8 - 1) * 8 : 0);
  }
  uint32_t rows_at = lds0 + C::KEYS + (wave * 4 * NB % 16 * 4 + (lane >> 4)) * 4,
           pe_rows_at = lds0 + C::KEYS + (wave * 16 + (lane >> 3)) * 4;
  opaque(rows_at), opaque(pe_rows_at);
  auto read_rows = [&](int tile, uint32_t (&at)[LOADS]) {
    const uint32_t r = rows_at + tile * BK * 4, pe = pe_rows_at + tile * BK * 4;
#pragma unroll
    for (int n = 0; n < LOADS; ++n)
      at[n] = *(KPOOL_LDS const uint32_t *)(uintptr_t)(n < 4 * NB ? r + n * 16 : pe + (n - 4 * NB) * 32);
  };
  auto address = [&](int n, uint32_t row) {
    return (const char *)(n < 4 * NB ? from[n % 4] : pe_from[n % 2]) + (uint64_t)row * pitch;
  };
  auto load_row = [&](int n, const char *from, uint32_t to) {  // to: the tile's buffer
    load_lds_16(from, to + (n < 4 * NB ? (wave * 4 * NB + n) * 1024 : C::PE + (wave * 2 + n - 4 * NB) * 1024));
  };
  int *list = reinterpret_cast<int *>(lds + C::KEYS), *places = reinterpret_cast<int *>(lds + C::PLACES);
  float *exchange = reinterpret_cast<float *>(lds + C::P);  // [4][BQ]

  int unit = -1;  // of the sequence
  for (;;) {
    const int q_start = a.cu_q[seq], Lq = a.cu_q[seq + 1] - q_start, len = latent_len(a, seq);
    const int kt = LIST ? list_tiles : tiles_of(len), cost = kt + costs.fixed;
    const int units = LIST ? Lq * a.hblocks : (Lq * a.H + BQ - 1) / BQ;
    if (unit < 0) unit = max(pos - before, 0) / cost;
    if (unit >= units) {  // (no rows, or no more)
      before += units * cost, ++seq, unit = 0;
      continue;
    }
    const int start = before + unit * cost;
    if (start >= hi) break;
    const int k0 = costs.cut(pos, start, kt), k1 = costs.cut(hi, start, kt);
    if (k0 >= k1) {
      if (start + cost >= costs.total) break;
      ++unit;
      continue;
    }
    // rows n0 .. n0 + nrows - 1 of the sequence's Lq * H
    const int tok = LIST ? unit / a.hblocks : 0, first = LIST ? (unit - tok * a.hblocks) * BQ : 0;
    const int n0 = LIST ? tok * a.H + first : unit * BQ;
    const int nrows = LIST ? min(BQ, a.H - first) : min(BQ, Lq * a.H - n0);
    const int64_t row0 = (int64_t)q_start * a.H + n0;
    const int t0 = n0 / a.H + len - Lq, t1 = (n0 + nrows - 1) / a.H + len - Lq;  // first and last position
    const int e_lo = k0 * BK;
    KeyBlocks blocks(e_lo, min(k1 * BK, LIST ? a.width : t1 + 1));

    // A block's keys.  place: of a thread's entries; found: what the page table (or the starts) say of them.
    int place[C::EACH], found[C::EACH];
    auto look_up = [&](const KeyBlocks &blocks) {
#pragma unroll
      for (int i = 0; i < C::EACH; ++i) {
        const int e = blocks.key((int)threadIdx.x * C::EACH + i);
        place[i] = -1;
        if (e >= 0) place[i] = LIST ? a.ids[((int64_t)q_start + tok) * a.width + e] : e;
      }
#pragma unroll
      for (int i = 0; i < C::EACH; ++i) {
        if (place[i] > t1) place[i] = -1;
        found[i] = -1;
        if (place[i] >= 0) found[i] = a.table ? a.table[(int64_t)seq * a.per_seq + place[i] / a.page] : a.starts[seq];
      }
    };
    // queries to LDS (behind the first tile), whole rows at a time, and from there to registers
    __syncthreads();
    {
      constexpr int CHUNKS = C::CHUNKS, THREADS = 256 / BQ, BATCH = (CHUNKS + THREADS - 1) / THREADS;  // of a row
      uint32_t tid = threadIdx.x;  // (opaque: what depends on it is not worth a register from one unit to the next)
      opaque(tid);
      const int row = tid / THREADS, c0 = tid % THREADS, at = (n0 + row) / a.H;
      const int latent = row < nrows ? a.R / 8 : 0, pe = row < nrows ? NB * 16 + a.P / 8 : 0;  // ends of its parts
      const uint16_t *src = a.q + (int64_t)(q_start + at) * a.qs + (n0 + row - at * a.H) * (a.R + a.P) + c0 * 8;
      uint4 z[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int chunk = c0 + u * THREADS;
        z[u] = make_uint4(0, 0, 0, 0);
        if (chunk < NB * 16 ? chunk < latent : chunk < pe)
          z[u] = *reinterpret_cast<const uint4 *>(src + u * THREADS * 8 + (chunk < NB * 16 ? 0 : a.R - NB * 128));
      }
      look_up(blocks);
#pragma unroll
      for (int u = 0; u < BATCH; ++u)
        if (CHUNKS % THREADS == 0 || c0 + u * THREADS < CHUNKS)
          *reinterpret_cast<uint4 *>(lds + TILE + row * C::QROW + (c0 + u * THREADS) * 16) = z[u];
    }
    __syncthreads();
    r.begin(lds0 + TILE, [&](int row) { return (n0 + row) / a.H + len - Lq; });

    for (; blocks.any(); blocks.next(C::BLOCK)) {
      // the block's keys that exist, in order: their rows (and places) in LDS
      if (blocks.at() > e_lo) look_up(blocks);
      int row[C::EACH];
#pragma unroll
      for (int i = 0; i < C::EACH; ++i) {
        const int p = place[i], id = found[i];
        row[i] = -1;
        if (a.table) {
          if (id >= 0 && id < a.npages) row[i] = id * a.page + p % a.page;
        } else if (id >= 0 && (int64_t)id + p < a.nrows) {
          row[i] = id + p;
        }
      }
      __syncthreads();  // (nobody reads the last block's list or tiles, or the queries, any more)
      int sum = 0;
#pragma unroll
      for (int i = 0; i < C::EACH; ++i) sum += row[i] >= 0;
      int *counts = reinterpret_cast<int *>(lds);
      const int upto = scan_256(sum, counts);
      if (threadIdx.x == 255) counts[4] = upto;
      int to = upto - sum;
      __syncthreads();
      const int present = __builtin_amdgcn_readfirstlane(counts[4]);
#pragma unroll
      for (int i = 0; i < C::EACH; ++i)
        if (row[i] >= 0) {
          list[to] = row[i];
          if (!LIST) places[to] = place[i];
          ++to;
        }
      __syncthreads();
      const int ntile = (present + BK - 1) / BK;
      // (the last tile's absent keys read its first one and count for nothing)
      if ((int)threadIdx.x < ntile * BK - present) list[present + threadIdx.x] = list[(ntile - 1) * BK];
      __syncthreads();

      uint32_t at[LOADS];
      if (ntile > 0) {
        read_rows(0, at);
#pragma unroll
        for (int n = 0; n < LOADS; ++n) load_row(n, address(n, at[n]), lds0);
      }
      const uint32_t p_at = lds0 + C::P;
      for (int j = 0; j < ntile; ++j) {
        const bool more = j + 1 < ntile;
        read_rows(more ? j + 1 : j, at);
        // the wave's part of tile j has landed; behind the barrier everyone's has, and everyone is done with
        // the buffer that tile j + 1 goes to
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
        barrier_only();
        uint32_t to = lds0 + ((j + 1) & 1) * TILE;
        opaque_uniform(to);
        const int last = LIST ? 0 : places[min(present, j * BK + BK) - 1];
        const TileKeys k{lds0 + (j & 1) * TILE, j * BK, present, j * BK + BK > present || (!LIST && last > t0)};
        struct Loads {  // the next tile's
          decltype(address) &make;
          decltype(load_row) &send;
          const uint32_t (&at)[LOADS];
          uint32_t to;
          const char *from;
          __device__ inline void address(int n) { from = make(n, at[n]); }
          __device__ inline void issue(int n) { send(n, from, to); }
        };
        struct NoLoads {
          __device__ inline void address(int) {}
          __device__ inline void issue(int) {}
        };
        if (more) r.scores(k, Loads{address, load_row, at, to, nullptr});
        else r.scores(k, NoLoads{});
        // the first columns of values do not wait for P
        r.read_values(k);
        __builtin_amdgcn_sched_barrier(0);
        // P, with the maximum so far.  A score far above it is rare: the waves say so, and only then find
        // the tile's maximum together and begin again.
        r.mask(k, places);
        const bool any_over = __any(r.over(a.scale_log2));
        if (lane == 0) list[wave] = any_over;
        r.weights(p_at, a.scale_log2);
        wait_reads();
        barrier_only();
        const int4 flags = *reinterpret_cast<const int4 *>(list);
        r.first_p(p_at);
        if (__builtin_amdgcn_readfirstlane(flags.x | flags.y | flags.z | flags.w)) {
          // (the maxima go where P is, which is written anew)
          wait_reads();
          barrier_only();
          r.give_top(exchange);
          wait_reads();
          barrier_only();
          r.raise(exchange, a.scale_log2);
          wait_reads();
          barrier_only();
          r.weights(p_at, a.scale_log2);
          wait_reads();
          barrier_only();
          r.first_p(p_at);
        }
        r.values(k, p_at);
      }
    }

    // l of a row over the lanes and waves
    __syncthreads();
    r.give_sum(exchange);
    __syncthreads();
    const bool whole = k1 - k0 == kt;
    const int slot = 2 * share + (k0 == 0);
    r.finish(
        exchange, whole,
        [&](int row, float m, float sum) {
          if (row >= nrows) return;
          // (0 where the row saw nothing; NaN goes through)
          const float lse = sum == 0.0f ? -__builtin_inff() : (m + log2f(sum)) * kLn2;
          if (!whole) a.part_lse[(int64_t)slot * BQ + row] = lse;
          else if (a.lse) a.lse[row0 + row] = lse;
        },
        [&](int row, int d, uint4 x) {
          if (row < nrows && d < a.R) *reinterpret_cast<uint4 *>(a.o + (row0 + row) * a.R + d) = x;
        },
        [&](int row, int d, f32x4 x) {
          if (row < nrows && d < a.R) *reinterpret_cast<f32x4 *>(a.part_o + ((int64_t)slot * BQ + row) * a.R + d) = x;
        });
    if (!whole && k0 == 0 && threadIdx.x == 0)
      a.cut[share] = {row0, start + costs.fixed + kt - costs.least + 1, costs.total, costs.shares, nrows};
    if (start + cost >= costs.total) break;
    ++unit;
  }
}

// Joins the parts of the units that lie across shares, o = sum_s e^(lse_s - lse) o_s: a workgroup for a
// row of the unit that a share begins (8 tokens of 2048 selected ones, 64 heads: 65 us with a workgroup for all
// of its rows, 10 so; 4 us, a chain of latencies, at the least).  256 / (R / 4) groups of threads take the parts in turn, each
// thread 4 columns, and add up in order.
__global__ __launch_bounds__(256) void latent_join_kernel(LatentArgs a, int BQ) {
  __shared__ float lse_of[kMostShares], weight[kMostShares];
  __shared__ f32x4 sums[256];
  const int share = blockIdx.x / BQ, r = blockIdx.x - share * BQ, tid = threadIdx.x;
  const LatentCut cut = a.cut[share];
  if (cut.end == 0 || r >= cut.nrows) return;
  const float none = -__builtin_inff();
  // part i is share `share` + i's; the unit's end lies in the last of them
  const int s = share + tid;
  const bool mine = tid == 0 || (s < cut.shares && share_start(cut.total, cut.shares, s) < cut.end);
  auto slot = [&](int i) { return (int64_t)(2 * (share + i) + (i == 0)) * BQ + r; };
  lse_of[tid] = mine ? a.part_lse[slot(tid)] : none;
  const int parts = __syncthreads_count(mine);
  float m = none;
  for (int i = 0; i < parts; ++i) m = fmaxf(m, lse_of[i]);
  const float shift = m > none ? m : 0.0f;
  if (mine) weight[tid] = exp2f_fast((lse_of[tid] - shift) * kLog2e);
  __syncthreads();
  float total = 0.0f;
  for (int i = 0; i < parts; ++i) total += weight[i];
  const int per = a.R / 4, groups = 256 / per, g = tid / per, d = (tid - g * per) * 4;
  f32x4 o = {};
  if (g < groups) {
#pragma unroll 8
    for (int i = g; i < parts; i += groups) o += weight[i] * *reinterpret_cast<const f32x4 *>(a.part_o + slot(i) * a.R + d);
  }
  sums[tid] = o;
  __syncthreads();
  if (g > 0) return;
  for (int i = 1; i < groups; ++i) o += sums[i * per + tid];
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t row = cut.row0 + r;
  *reinterpret_cast<uint2 *>(a.o + row * a.R + d) =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  if (tid == 0 && a.lse) a.lse[row] = total == 0.0f ? none : shift + log2f(total) * kLn2;
}

template <int NB, int RB, bool LIST>
hipError_t launch_latent_t(const LatentArgs &a, hipStream_t st) {
  using C = typename LatentRows<NB, RB, LIST>::C;
  hipLaunchKernelGGL((latent_kernel<NB, RB, LIST>), dim3((a.shares + 7) / 8 * 8), dim3(256), C::LDS, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.shares == 1) return e;
  hipLaunchKernelGGL(latent_join_kernel, dim3(a.shares * C::BQ), dim3(256), 0, st, a, C::BQ);
  return hipGetLastError();
}

template <int NB, int RB>
hipError_t launch_latent_l(bool list, const LatentArgs &a, hipStream_t st) {
  return list ? launch_latent_t<NB, RB, true>(a, st) : launch_latent_t<NB, RB, false>(a, st);
}
template <int NB>
hipError_t launch_latent_r(int rb, bool list, const LatentArgs &a, hipStream_t st) {
  return rb == 1   ? launch_latent_l<NB, 1>(list, a, st)
         : rb == 2 ? launch_latent_l<NB, 2>(list, a, st)
                   : launch_latent_l<NB, 4>(list, a, st);
}

int64_t cut_bytes(int shares) { return (int64_t)shares * 32; }
static_assert(sizeof(LatentCut) <= 32, "parts stay aligned");

LatentPlan shares_of(LatentPlan p, int64_t units, int64_t keys) {
  p.units = units;
  // (more units than a call may have tiles are refused as they are: their product may not fit 64 bits)
  p.tiles = units < (1 << 28) ? units * std::max<int64_t>(1, (keys + kLatentKeys - 1) / kLatentKeys) : units;
  // A share for each tile, of 64 rows for two, as their parts cost four tiles' time to begin and to join.  (By
  // the most tiles that max_len allows: a call whose lengths on the device are shorter has up to a share a tile
  // of its own.  8 requests of 2 tokens over 500, 128 heads, 31.7 us with max_len 500, 35.2 with 524288.)
  // (us with one, two and four tiles a share: 8 tokens of 2048 selected ones, 64 heads, 35, 32, 34; one token
  // over 1003, 16 heads, 16.3, 18.0, 21.8.)
  const int64_t shares = p.rb == 4 ? (p.tiles + 1) / 2 : p.tiles;
  p.shares = (int)std::min<int64_t>(kMostShares, std::max<int64_t>(1, shares));
  return p;
}

}  // namespace

// Units of 16, 32 or 64 rows: as many as share keys and no more.  (us with 16, 32 and 64 rows, 8 requests of
// one token over 64k cached tokens in all, and 256 rows of 1024 selected tokens: 16 heads 37, 41, - and 51, 54,
// -; 32 heads 46, 43, 50 and 89, 54, 62; 64 heads -, 51, 55 and -, 95, 67; 128 heads -, 66, 60 and -, 173, 114.)
// A batch takes the units of its longest sequence throughout: of 16 requests over 205k tokens, 16 heads, 62.5 us,
// one of 4 tokens instead of one makes it 68 to 69, one of 64 over 300 68.
LatentPlan plan_latent(const int32_t *cu_q, int nseq, int H, int64_t max_len) {
  int64_t most = 0, units = 0;
  for (int s = 0; s < nseq; ++s) most = std::max<int64_t>(most, (int64_t)(cu_q[s + 1] - cu_q[s]) * H);
  LatentPlan p;
  p.rb = most <= 16 ? 1 : most <= 32 ? 2 : 4;
  for (int s = 0; s < nseq; ++s) units += ((int64_t)(cu_q[s + 1] - cu_q[s]) * H + 16 * p.rb - 1) / (16 * p.rb);
  return shares_of(p, units, max_len);
}

LatentPlan plan_latent_list(int64_t Tq, int H, int width) {
  LatentPlan p;
  p.rb = H <= 16 ? 1 : H <= 32 ? 2 : 4;
  return shares_of(p, Tq * ((H + 16 * p.rb - 1) / (16 * p.rb)), width);
}

// (one share leaves no parts)
size_t latent_workspace(const LatentPlan &p, int R) {
  if (p.shares == 1) return 0;
  return (size_t)(cut_bytes(p.shares) + (int64_t)2 * p.shares * 16 * p.rb * (R + 1) * 4);
}

hipError_t launch_latent(const LatentCall &c, const LatentPlan &p, void *workspace, hipStream_t st) {
  LatentArgs a{};
  a.q = c.q, a.cache = c.cache;
  a.qs = c.q_stride, a.cs = c.cache_stride, a.nrows = c.cache_rows;
  a.table = c.page_table, a.starts = c.k_starts, a.lens = c.k_lens, a.cu_q = c.cu_q, a.ids = c.ids;
  a.per_seq = c.pages_per_seq, a.page = c.page_size, a.max_len = c.max_len;
  a.npages = c.page_table ? (int)(c.cache_rows / c.page_size) : 0;
  a.nseq = c.nseq, a.H = c.H, a.R = c.R, a.P = c.P, a.width = c.width;
  a.scale_log2 = c.scale * kLog2e;
  a.shares = p.shares, a.units = (int)p.units, a.hblocks = (c.H + 16 * p.rb - 1) / (16 * p.rb);
  a.o = c.o, a.lse = c.lse;
  if (p.shares > 1) {
    a.cut = (LatentCut *)workspace;
    a.part_o = (float *)((char *)workspace + cut_bytes(p.shares));
    a.part_lse = a.part_o + (int64_t)2 * p.shares * 16 * p.rb * c.R;
  }
  return c.R <= 256 ? launch_latent_r<2>(p.rb, c.list, a, st) : launch_latent_r<4>(p.rb, c.list, a, st);
}

}  // namespace kpool
