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
// (row n: head n % H of token n / H).  A workgroup takes up to 64 of them (16 RB) and walks key tiles
// of 64 through LDS, each read once from memory and used twice, as keys and, transposed, as values.
//   S^T = C Q^T: wave w multiplies keys 16 w .. 16 w + 15 of the tile with all rows, whose
//     fragments stay in registers (R + P = 576 and 64 rows: 288 a lane);
//   the running maximum is common to the four waves (one exchange a tile), P goes through LDS in
//     bf16, each wave sums its own keys' share of l;
//   O^T = C^T P^T: wave w keeps columns w R / 4 .. of all rows (128 registers a lane).
// So a key tile passes from LDS to registers 1 + 8 / 9 times, whatever the rows.  Statistics as in
// attend.hip: fp32, base 2, the maximum followed when it rises by more than 8; P rounded to bf16 for
// its product, l from the unrounded values.
//
// Keys lie anywhere (pages, lists): a block of 512 of them is first turned into a list of row offsets
// in LDS, without those that do not exist, and tiles are gathered by it.
//
// Work goes by equal shares of all the tiles, one share a CU.  Where the shares begin depends on
// the lengths, which are on the device (a captured decoding step replays while its lengths grow), so each
// workgroup finds its share itself.  A unit (rows of one tile) that lies across shares leaves a
// part each in fp32; a second kernel joins them in order.
#include "attend_tile.h"

namespace kpool {
namespace {

constexpr int kLatentKeys = 64, kLatentBlock = 512;

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

// The first of n equal shares' tiles.
__device__ inline int share_start(int total, int n, int share) {
  const int each = total / n;
  return each * share + (total - each * n) * share / n;
}

template <int NB, int RB>
struct Latent {
  static constexpr int BK = kLatentKeys, BQ = 16 * RB;
  static constexpr int KS = NB * 4 + 2;             // contraction steps of 32: the latent part, then the positional
  static constexpr int CB = NB * 2;                 // 16-column blocks of a wave
  static constexpr int BLOCKB = BK * 256;           // bytes of 128 columns of a tile
  static constexpr int TILE = NB * BLOCKB + BK * 128;
  static constexpr int PBUF = 2 * TILE, OFFS = PBUF + BQ * BK * 2, POS = OFFS + kLatentBlock * 8,
                       TOP = POS + kLatentBlock * 4, COUNT = TOP + 4 * BQ * 4, LDS = COUNT + 64;
  static_assert(LDS <= 163840, "LDS of a CU");
};

// n tokens of a sequence, at most what the caller said and what its pages hold
__device__ inline int latent_len(const LatentArgs &a, int s) {
  const int len = min(max(a.lens[s], 0), a.max_len);
  return a.table ? (int)min64(len, (int64_t)a.per_seq * a.page) : len;
}
__device__ inline int tiles_of(int keys) { return max(1, (keys + kLatentKeys - 1) / kLatentKeys); }
__device__ inline int seq_tiles(const LatentArgs &a, int s, int BQ) {
  if (s >= a.nseq) return 0;
  const int64_t rows = (int64_t)(a.cu_q[s + 1] - a.cu_q[s]) * a.H;
  return (int)((rows + BQ - 1) / BQ) * tiles_of(latent_len(a, s));
}

// Keeps the compiler from looking through a value that is the same in all lanes.
__device__ inline void opaque_uniform(uint32_t &x) { asm volatile("" : "+s"(x)); }

// inclusive sum over the workgroup's 256 threads; scratch: 4 values of LDS.  All threads call it.
__device__ inline int scan_256(int x, int *scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(x, d);
    if (lane >= d) x += up;
  }
  __syncthreads();
  if (lane == 63) scratch[wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x += scratch[w];
  return x;
}

template <int NB, int RB, bool LIST>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void latent_kernel(LatentArgs a) {
  using C = Latent<NB, RB>;
  constexpr int BK = C::BK, BQ = C::BQ, TILE = C::TILE;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, group = lane >> 4;
  const uint32_t lds0 = lds_offset(lds);

  // this workgroup's share of all tiles: [pos, hi), from sequence `seq` on, whose tiles begin at `before`
  int total = 0, before, seq;
  const int list_tiles = LIST ? tiles_of(a.width) : 0;
  int *scratch = reinterpret_cast<int *>(lds);
  if (LIST) {
    total = a.units * list_tiles;
  } else {
    for (int base = 0; base < a.nseq; base += 256) {
      const int x = scan_256(seq_tiles(a, base + threadIdx.x, BQ), scratch);
      if (threadIdx.x == 255) scratch[4] = x;
      __syncthreads();
      total += scratch[4];
    }
  }
  total = __builtin_amdgcn_readfirstlane(total);
  if (threadIdx.x == 0 && a.cut) a.cut[blockIdx.x].end = 0;
  const int n = min(a.shares, total), share = blockIdx.x;
  if (share >= n) return;
  int pos = share_start(total, n, share);
  const int hi = share_start(total, n, share + 1);
  if (LIST) {
    const int token = pos / list_tiles / a.hblocks;
    int step = a.nseq;  // (the sequence of a token: the last that starts at or before it)
    seq = 0;
    while (step > 1) {
      const int half = step / 2;
      if (a.cu_q[seq + half] <= token) seq += half;
      step -= half;
    }
    before = a.cu_q[seq] * a.hblocks * list_tiles;
  } else {
    int run = 0;
    for (int base = 0; base < a.nseq; base += 256) {
      const int mine = seq_tiles(a, base + threadIdx.x, BQ);
      const int x = run + scan_256(mine, scratch);
      if (x - mine <= pos && pos < x) scratch[5] = x - mine, scratch[6] = base + threadIdx.x;
      if (threadIdx.x == 255) scratch[4] = x;
      __syncthreads();
      run = scratch[4];
    }
    before = __builtin_amdgcn_readfirstlane(scratch[5]), seq = __builtin_amdgcn_readfirstlane(scratch[6]);
  }

  // Addresses are kept as few registers and made where they are used (one instruction, (a ^ b) + c):
  // fragments of a wave's 16 keys, whose step of 32 is ^ (step << 6) in the latent part; of its columns,
  // whose block of 16 is ^ (block << 5)
  uint32_t krow, kpe, vcol;
  {
    const int r = lane & 15, key = 4 * group + (r >> 2);
    krow = (wave * 16 + r) * 256 + ((group ^ Keys16<128>::swz(r)) << 4);
    kpe = (wave * 16 + r) * 128 + ((group ^ Keys16<64>::swz(r)) << 4);
    vcol = key * 256 + ((((r & 3) >> 1) ^ Keys16<128>::swz(key)) << 4) + (r & 1) * 8;
    opaque(krow), opaque(kpe), opaque(vcol);
  }
  // Loads: of the latent part 4 NB a wave, 4 rows each; of the positional one 2 a wave, 8 rows each; in
  // steps of two, whose rows are read from the list one step ahead of their use.  A lane's chunk of its
  // row is lchunk ^ swz(4 i) (i the load's place in 16 rows), its last where the row ends before it.
  constexpr int LOADS = 4 * NB + 2;
  const uint32_t last_chunk = a.R / 8 - 1;
  uint32_t lchunk = wave * NB / 4 * 16 + ((lane & 15) ^ Keys16<128>::swz(group)),
           pcol = (a.R + (a.P ? min((lane & 7) ^ Keys16<64>::swz(lane >> 3), a.P / 8 - 1) * 8 : -8)) * 2;
  opaque(lchunk), opaque(pcol);
  struct Tile {
    uint32_t rows, pe_rows, to, pe_to;  // LDS: the lane's places in the list, where the loads go
  };
  auto tile_at = [&](int tile, int buf) {
    Tile x;
    const uint32_t offs = lds0 + C::OFFS + tile * BK * 8;
    x.rows = offs + (wave * 4 * NB % 16 * 4 + group) * 8, x.pe_rows = offs + (wave * 16 + (lane >> 3)) * 8;
    x.to = lds0 + buf * TILE + wave * 4 * NB * 1024, x.pe_to = lds0 + buf * TILE + NB * C::BLOCKB + wave * 2048;
    opaque(x.rows), opaque(x.pe_rows), opaque_uniform(x.to), opaque_uniform(x.pe_to);
    return x;
  };
  auto read_rows = [&](const Tile &x, int i, uint64_t (&at)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int n = 2 * i + u;
      at[u] = *(KPOOL_LDS const uint64_t *)(uintptr_t)(n < 4 * NB ? x.rows + n * 32 : x.pe_rows + (n - 4 * NB) * 64);
    }
  };
  auto load_rows = [&](const Tile &x, int i, const uint64_t (&at)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int n = 2 * i + u;
      uint32_t off = pcol;
      if (n < 4 * NB) off = min(lchunk ^ (uint32_t)Keys16<128>::swz(n % 4 * 4), last_chunk) * 16;
      load_lds_16((const void *)(at[u] + off), n < 4 * NB ? x.to + n * 1024 : x.pe_to + (n - 4 * NB) * 1024);
    }
  };
  uint64_t *list = reinterpret_cast<uint64_t *>(lds + C::OFFS);  // the rows' addresses
  int *places = reinterpret_cast<int *>(lds + C::POS);
  float *top_of = reinterpret_cast<float *>(lds + C::TOP);  // [4][BQ]
  int *count = reinterpret_cast<int *>(lds + C::COUNT);

  while (pos < hi) {
    const int q_start = a.cu_q[seq], Lq = a.cu_q[seq + 1] - q_start, len = latent_len(a, seq);
    const int kt = LIST ? list_tiles : tiles_of(len);
    const int units = LIST ? Lq * a.hblocks : (Lq * a.H + BQ - 1) / BQ;
    const int unit = (pos - before) / kt, k0 = pos - before - unit * kt, k1 = min(kt, k0 + hi - pos);
    // rows n0 .. n0 + nrows - 1 of the sequence's Lq * H
    const int tok = LIST ? unit / a.hblocks : 0, first = LIST ? (unit - tok * a.hblocks) * BQ : 0;
    const int n0 = LIST ? tok * a.H + first : unit * BQ;
    const int nrows = LIST ? min(BQ, a.H - first) : min(BQ, Lq * a.H - n0);
    const int64_t row0 = (int64_t)q_start * a.H + n0;
    const int t0 = n0 / a.H + len - Lq, t1 = (n0 + nrows - 1) / a.H + len - Lq;  // first and last position
    const int e_lo = k0 * BK, e_hi = min(k1 * BK, LIST ? a.width : t1 + 1);

    bf16x8 q[RB][C::KS];
    int t[RB];
    int part = group * 8;  // (opaque: what depends on it is not worth a register from one unit to the next)
    asm volatile("" : "+v"(part));
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = rb * 16 + col;
      const int at = (n0 + r) / a.H;
      const uint16_t *src = a.q + (int64_t)(q_start + at) * a.qs + (n0 + r - at * a.H) * (a.R + a.P);
      t[rb] = at + len - Lq;
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        const int d = (ks < NB * 4 ? ks : ks - NB * 4) * 32 + part, most = ks < NB * 4 ? a.R : a.P;
        uint4 z = make_uint4(0, 0, 0, 0);
        if (r < nrows && d < most) z = *reinterpret_cast<const uint4 *>(src + (ks < NB * 4 ? 0 : a.R) + d);
        q[rb][ks] = __builtin_bit_cast(bf16x8, z);
      }
    }
    f32x4 o[C::CB][RB];
    float m[RB], l[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      m[rb] = -__builtin_inff(), l[rb] = 0.0f;
#pragma unroll
      for (int c = 0; c < C::CB; ++c) o[c][rb] = f32x4{};
    }
    wait_loads();

    for (int block = e_lo; block < e_hi; block += kLatentBlock) {
      // the block's keys that exist, in order: offsets of their rows, and their places
      const int end = min(e_hi, block + kLatentBlock);
      uint64_t off[2];
      int place[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = block + i * 256 + threadIdx.x;
        int p = -1;
        if (e < end) p = LIST ? a.ids[((int64_t)q_start + tok) * a.width + e] : e;
        if (p > t1) p = -1;
        int64_t row = -1;
        if (p >= 0 && a.table) {
          const int pg = p / a.page;
          const int id = a.table[(int64_t)seq * a.per_seq + pg];
          if (id >= 0 && id < a.npages) row = (int64_t)id * a.page + (p - pg * a.page);
        } else if (p >= 0) {
          const int64_t start = a.starts[seq];
          if (start >= 0 && start + p < a.nrows) row = start + p;
        }
        place[i] = row >= 0 ? p : -1;
        off[i] = (uint64_t)(a.cache + row * a.cs);
      }
      uint64_t there[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) there[i] = __ballot(place[i] >= 0);
      __syncthreads();  // (nobody reads the last block's list or tiles any more)
      if (lane == 0) count[wave] = __popcll(there[0]), count[4 + wave] = __popcll(there[1]);
      __syncthreads();
      int present = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (w == wave && place[i] >= 0) {
            const int to = present + __popcll(there[i] & ((uint64_t(1) << lane) - 1));
            list[to] = off[i], places[to] = place[i];
          }
          present += count[i * 4 + w];
        }
      __syncthreads();
      const int ntile = (present + BK - 1) / BK;
      // (the last tile's absent keys read its first one and count for nothing)
      if ((int)threadIdx.x < ntile * BK - present)
        list[present + threadIdx.x] = list[(ntile - 1) * BK];
      __syncthreads();

      if (ntile > 0) {
        const Tile x = tile_at(0, 0);
        uint64_t at[2][2];
        read_rows(x, 0, at[0]);
#pragma unroll
        for (int i = 0; i < LOADS / 2; ++i) {
          if (i + 1 < LOADS / 2) read_rows(x, i + 1, at[(i + 1) & 1]);
          load_rows(x, i, at[i & 1]);
        }
      }
      for (int j = 0; j < ntile; ++j) {
        const uint32_t buf = (j & 1) * TILE;
        f32x4 s[RB];
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
        barrier_only();
        const bool more = j + 1 < ntile;
        const Tile next = tile_at(more ? j + 1 : j, (j + 1) & 1);
        uint64_t at[2][2];
        read_rows(next, 0, at[0]);
        // S.  Fragments of keys are read a few ahead of the products that need them.
        const uint32_t tile0 = lds0 + buf;
        auto read_key = [&](int ks) {
          return ks < NB * 4 ? lds_read((krow ^ ((ks & 3) << 6)) + (tile0 + (ks >> 2) * C::BLOCKB))
                             : lds_read((kpe ^ ((ks & 1) << 6)) + (tile0 + NB * C::BLOCKB));
        };
        // (and so are the loads of the next tile issued beside them)
        constexpr int AHEAD = 4;
        static_assert(C::KS == LOADS, "two loads for two steps");
        bf16x8 k[C::KS];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) s[rb] = f32x4{};
#pragma unroll
        for (int ks = 0; ks < AHEAD; ++ks) k[ks] = read_key(ks);
#pragma unroll
        for (int ks = 0; ks < C::KS; ks += 2) {
          __builtin_amdgcn_sched_barrier(0);
          if (ks + 2 < LOADS) read_rows(next, ks / 2 + 1, at[(ks / 2 + 1) & 1]);
          if (more) load_rows(next, ks / 2, at[(ks / 2) & 1]);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (ks + AHEAD + u < C::KS) k[ks + AHEAD + u] = read_key(ks + AHEAD + u);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) s[rb] = mfma(k[ks + u], q[rb][ks + u], s[rb]);
        }
        __builtin_amdgcn_sched_barrier(0);
        // what a row does not see
        const int key = j * BK + wave * 16 + 4 * group;
        const int last = places[min(present, j * BK + BK) - 1];
        if (j * BK + BK > present || (!LIST && last > t0)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool absent = key + i >= present;
            const int p = absent || LIST ? 0 : places[key + i];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
              if (absent || (!LIST && p > t[rb])) s[rb][i] = -__builtin_inff();
          }
        }
        // the tile's maximum of a row
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const Pair x = row_pair(fmaxf(fmaxf(s[rb][0], s[rb][1]), fmaxf(s[rb][2], s[rb][3])));
          float y = fmaxf(x.a, x.b);
          y = fmaxf(y, other_half(y));
          if (lane < 16) top_of[wave * BQ + rb * 16 + col] = y;
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);
        barrier_only();
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const float *x = top_of + rb * 16 + col;
          const float top = fmaxf(fmaxf(x[0], x[BQ]), fmaxf(x[2 * BQ], x[3 * BQ])) * a.scale_log2;
          if (__any(top > m[rb] + 8.0f)) {  // (the same in every wave)
            const float up = fmaxf(top, m[rb]);
            const float f = up > m[rb] ? exp2f_fast(m[rb] - up) : 1.0f;
            m[rb] = up;
            l[rb] *= f;
#pragma unroll
            for (int c = 0; c < C::CB; ++c) o[c][rb] *= f;
          }
          const float shift = m[rb] > -__builtin_inff() ? m[rb] : 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[rb][i] = exp2f_fast(fmaf(s[rb][i], a.scale_log2, -shift));
            l[rb] += s[rb][i];
          }
          // P of row rb * 16 + col: 16-byte chunks, each with a lane group's 8 keys of a contraction of
          // 32 in the order of lds_read_cols
          const int r = rb * 16 + col, chunk = (wave >> 1) * 4 + group;
          const uint32_t at = lds0 + C::PBUF + r * 128 + ((chunk ^ (r & 7)) << 4) + (wave & 1) * 8;
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          *(KPOOL_LDS u32x2 *)(uintptr_t)at = u32x2{pack_bf16(s[rb][0], s[rb][1]), pack_bf16(s[rb][2], s[rb][3])};
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);
        barrier_only();
        // O
        auto read_value = [&](int i) {  // columns i % CB of the wave's, keys 32 (i / CB) ..
          const int c = wave * C::CB + i % C::CB;
          const uint32_t at = (vcol ^ ((c & 7) << 5)) + (tile0 + (c >> 3) * C::BLOCKB + i / C::CB * 32 * 256);
          return lds_read_cols(at, at + 16 * 256);
        };
        bf16x8 v[2 * C::CB], p[RB];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = read_value(i);
#pragma unroll
        for (int i = 0; i < 2 * C::CB; ++i) {
          if (i % 2 == 0) {
            __builtin_amdgcn_sched_barrier(0);
            if (i + 4 < 2 * C::CB) v[i + 4] = read_value(i + 4), v[i + 5] = read_value(i + 5);
          }
          if (i % C::CB == 0) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
              const int r = rb * 16 + col;
              p[rb] = lds_read(lds0 + C::PBUF + r * 128 + (((i / C::CB * 4 + group) ^ (r & 7)) << 4));
            }
          }
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) o[i % C::CB][rb] = mfma(v[i], p[rb], o[i % C::CB][rb]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    // l of a row over the lane groups and waves
    __syncthreads();
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const Pair x = row_pair(l[rb]);
      float y = x.a + x.b;
      y += other_half(y);
      if (lane < 16) top_of[wave * BQ + rb * 16 + col] = y;
    }
    __syncthreads();
    const bool whole = k1 - k0 == kt;
    const int slot = 2 * share + (k0 == 0);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = rb * 16 + col;
      if (r >= nrows) continue;
      const float *x = top_of + r;
      const float sum = (x[0] + x[BQ]) + (x[2 * BQ] + x[3 * BQ]);
      // (0 where the row saw nothing; NaN goes through)
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const float lse = sum == 0.0f ? -__builtin_inff() : (m[rb] + log2f(sum)) * kLn2;
#pragma unroll
      for (int c = 0; c < C::CB; ++c) {
        const int d = (wave * C::CB + c) * 16 + group * 4;
        if (d >= a.R) continue;
        const f32x4 y = o[c][rb] * inv;
        if (whole)
          *reinterpret_cast<uint2 *>(a.o + (row0 + r) * a.R + d) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        else
          *reinterpret_cast<f32x4 *>(a.part_o + ((int64_t)slot * BQ + r) * a.R + d) = y;
      }
      if (wave == 0 && group == 0) {
        if (!whole) a.part_lse[(int64_t)slot * BQ + r] = lse;
        else if (a.lse) a.lse[row0 + r] = lse;
      }
    }
    if (!whole && k0 == 0 && threadIdx.x == 0)
      a.cut[share] = {row0, before + (unit + 1) * kt, total, n, nrows};
    pos += k1 - k0;
    if (pos == before + units * kt) {
      before = pos;
      do ++seq;
      while (seq < a.nseq && a.cu_q[seq + 1] == a.cu_q[seq]);
    }
  }
}

// Joins the parts of the units that lie across shares, o = sum_s e^(lse_s - lse) o_s: a workgroup for a
// row of the unit that a share begins.  256 / (R / 4) groups of threads take the parts in turn, each
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
  using C = Latent<NB, RB>;
  hipLaunchKernelGGL((latent_kernel<NB, RB, LIST>), dim3(a.shares), dim3(256), C::LDS, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.shares == 1) return e;
  hipLaunchKernelGGL(latent_join_kernel, dim3(a.shares * C::BQ), dim3(256), 0, st, a, C::BQ);
  return hipGetLastError();
}

template <int NB, int RB>
hipError_t launch_latent_l(const LatentArgs &a, hipStream_t st) {
  return a.ids ? launch_latent_t<NB, RB, true>(a, st) : launch_latent_t<NB, RB, false>(a, st);
}
template <int NB>
hipError_t launch_latent_r(int rb, const LatentArgs &a, hipStream_t st) {
  return rb == 1 ? launch_latent_l<NB, 1>(a, st) : rb == 2 ? launch_latent_l<NB, 2>(a, st) : launch_latent_l<NB, 4>(a, st);
}

int64_t cut_bytes(int shares) { return (int64_t)shares * 32; }
static_assert(sizeof(LatentCut) <= 32, "parts stay aligned");

LatentPlan shares_of(LatentPlan p, int64_t units, int64_t keys) {
  p.units = units;
  p.tiles = units * std::max<int64_t>(1, (keys + kLatentKeys - 1) / kLatentKeys);
  p.shares = (int)std::min<int64_t>(kMostShares, std::max<int64_t>(1, p.tiles));
  return p;
}

}  // namespace

// 16-row blocks: as many as the rows that share keys fill.
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
  return c.R <= 256 ? launch_latent_r<2>(p.rb, a, st) : launch_latent_r<4>(p.rb, a, st);
}

}  // namespace kpool
