// qsa_select.cu -- the cheap score of every query row against the micro-blocks of its
// sequence and the choice of the row's slots.  Contract: include/qsa_layer.h
// (qsa_select_slots).
//
// Two kernels over chunks of rows: the score kernel writes a 32-bit score per (row, block)
// into the workspace, the choice kernel finds the border of each row's top_blocks best and
// writes the slots of the blocks above it.
#include "qsa_layer.cuh"
#include "qsa_probe.h"

#include <atomic>

namespace {

using namespace qsa;

constexpr int kKeyTile = 128;                 // micro-blocks per tile
constexpr int kScoreThreads = 256;
constexpr int kScoreBlocks = 2;               // of an SM
constexpr int64_t kChunkBytes = 512 << 20;    // scores of one chunk of rows, while that is kMinChunkRows
constexpr int kMinChunkRows = 64;
constexpr int32_t kLate = 1 << 30;            // of a tile's number of rows (at most 256): see SelectParams

struct SelectParams {
  const uint16_t* q;
  const float* weight;
  const int8_t* codes;
  const float* scales;
  const int32_t *table, *lens, *cu;
  int32_t *out, *width;
  float* scores;       // [chunk rows, ld]
  uint32_t* err_word;
  int64_t q_st, q_sh, w_st, code_st, table_st, out_st, pages, ld;
  int32_t c0, c1;      // the chunk's rows
  int32_t Tq, B, P, page_size, per_page, Hi, block, top, sink, local;
  int4* tiles;         // tcgen05 form: tiles of rows [chunks, max_tiles], and their codes and gains
  uint8_t* tile_q;
  int32_t* late;       // tcgen05 form: a word of the chunk's first tile, kLate set when a wait ran out
  uint32_t wait_ns;    // limit of each such wait
  int32_t first;       // the choice is the call's first kernel
  int32_t cap, queue, window;              // keys of a row, and words of its marks, in the choice's shared memory
  uint32_t page_magic, block_magic; // 2^32 / per_page (/ block), rounded up
};

// The score as it is kept: a NaN (of the codes or weights, or the scale of a block whose page
// lies outside the pool) counts as -infinity.  (Adding +0 spares most zeros their sign, but a
// negative product that underflows is -0.)
__device__ __forceinline__ float kept_score(float sum, float scale) {
  return fmaxf(__fmaf_rn(sum, scale, 0.f), -__builtin_huge_valf());
}

// The order of scores as an order of unsigned integers: both zeros the same, -infinity, and
// with it any NaN that a failed score kernel left, at kLeastKey and nothing below it; 0 is
// left for blocks that take no part.  So keys compare as the scores do, whatever their bits.
// And back.
constexpr uint32_t kLeastKey = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(uint32_t bits) {
  const uint32_t score = __float_as_uint(fmaxf(__fadd_rn(__uint_as_float(bits), 0.f), -__builtin_huge_valf()));
  return score ^ (uint32_t(int32_t(score) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t key) {
  key = max(key, kLeastKey);
  return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

// Rows of sequence b, clamped to [0, Tq].
__device__ __forceinline__ int2 rows_of(const SelectParams& p, int b, bool report) {
  if (p.cu == nullptr) return make_int2(b, b + 1);
  int lo = p.cu[b], hi = p.cu[b + 1];
  if (report && p.err_word != nullptr && (lo < 0 || lo > p.Tq || hi < lo || hi > p.Tq))
    atomicOr(p.err_word, QSA_ERRBIT_WIDTH_RANGE);
  lo = min(max(lo, 0), p.Tq);
  hi = min(max(hi, 0), p.Tq);
  return make_int2(lo, max(hi, lo));
}

__device__ __forceinline__ int length_of(const SelectParams& p, int b, bool report) {
  const int64_t most = int64_t(p.P) * p.page_size;
  const int n = p.lens[b];
  if (report && p.err_word != nullptr && (n < 0 || n > most)) atomicOr(p.err_word, QSA_ERRBIT_WIDTH_RANGE);
  return int(min(int64_t(max(n, 0)), most));
}

// Inclusive scan over the block's threads; `total` gets the sum.  `tmp`: one int per warp.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // tmp is free
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    before += w < warp ? tmp[w] : 0;
    total += tmp[w];
  }
  return v + before;
}

// ---- the score of few rows per sequence -----------------------------------------------------

// Columns of a tile of rows: 8 NT of them, a thread of quad position u holding columns 2u and
// 2u + 1 of every n8 tile: kPer = 2 NT columns, which are kPer / HP rows of HP heads each, so
// one thread holds all heads of a row (16 at a time) and adds them in order without crossing
// lanes.  Column c of an n8 tile i is (row u kPer/HP + x / HP, head x mod HP) with u = c / 2
// and x = 2 i + (c mod 2).  Heads beyond Hi, and rows beyond the tile's, have gain 0.
template <int DI, int HP, int NT>
struct Score {
  static constexpr int kPer = 2 * NT;       // columns of a thread
  static constexpr int kRx = kPer / HP;     // rows of a thread
  static constexpr int kRows = 4 * kRx;     // rows of a tile
  static constexpr int kSteps = DI / 32;    // k-steps of a product
  static_assert(kPer % HP == 0 && kRx >= 1, "a thread holds whole rows");
  // the query codes as the MMA's B fragments, and the gains
  static size_t smem(int groups) { return size_t(groups) * NT * (kSteps * 256 + 32); }
};

// The units (128 blocks of one tile of rows) of all sequences are shared out evenly over the
// thread blocks; the eight warps of one take 16 blocks of a unit each.  A lane holds, of two
// of the 16 blocks, 16 bytes of every 64 as they lie in memory: that is an A fragment of the
// 8-bit MMA up to the order of the products in the sum, which is exact, and the query codes
// are put in the same order; so the codes go from memory to the MMA without shared memory,
// the next blocks' loads in flight, and the page lookups one step further ahead.
// Bound: HBM, the codes are read once per four rows or more of a sequence.
// 64 rows over ragged caches of up to 16,384 blocks (78 MB): 29 us (128-block tiles through
// shared memory with a barrier each, split evenly by the page table's capacity: 44 us).
template <int DI, int HP, int NT>
__global__ void __launch_bounds__(kScoreThreads, kScoreBlocks)
    qsa_select_score_kernel(const SelectParams p, int groups) {
  using C = Score<DI, HP, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint2* sQ = reinterpret_cast<uint2*>(smem);  // [group, tile][k-step][lane]
  float* sGain = reinterpret_cast<float*>(smem + size_t(groups) * NT * C::kSteps * 256);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, u = lane & 3;
  begin_kernel();

  // units of sequence b's rows in this chunk: as many as if every tile saw all of its blocks
  auto rows_here = [&](int b) {
    int2 r = rows_of(p, b, false);
    r.x = max(r.x, p.c0);
    r.y = min(r.y, p.c1);
    return r;
  };
  auto units_at = [&](int b) -> int64_t {
    if (b >= p.B) return 0;
    const int2 r = rows_here(b);
    const int f = length_of(p, b, false) / p.block;
    if (r.y <= r.x || f <= p.top) return 0;
    return int64_t((r.y - r.x + C::kRows - 1) / C::kRows) * ((f + kKeyTile - 1) / kKeyTile);
  };
  int64_t total = 0;
  for (int b = lane; b < p.B; b += 32) total += units_at(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int64_t u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  if (u0 == u1) return;
  int b = 0;
  int64_t before = 0;  // units of the sequences before b
  for (;; b += 32) {   // (every warp for itself)
    const int64_t n = units_at(b + lane);
    int64_t to = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + to > u0);
    if (past != 0u) {
      const int l = __ffs(past) - 1;
      before += __shfl_sync(0xffffffffu, to - n, l);
      b += l;
      break;
    }
    before += __shfl_sync(0xffffffffu, to, 31);
  }

  for (int64_t at = u0; at < u1;) {
    // ---- a piece: key tiles of one tile of rows ------------------------------------------------
    const int2 r = rows_here(b);
    const int last = rows_of(p, b, false).y - 1, len = length_of(p, b, false);
    const int per_tile = (len / p.block + kKeyTile - 1) / kKeyTile;
    const int tile = int((at - before) / per_tile), kt = int(at - before - int64_t(tile) * per_tile);
    const int64_t end = min(u1, before + int64_t(tile + 1) * per_tile);
    const int t0 = r.x + tile * C::kRows, n = min(C::kRows, r.y - t0);
    const int f_most = max(len - (last - (t0 + n - 1)), 0) / p.block;
    const int k0 = kt * kKeyTile, k1 = min(k0 + int(end - at) * kKeyTile, f_most);
    const int subs = f_most <= p.top ? 0 : (k1 - k0 + 15) / 16;  // (0: every row takes all its blocks)
    const int32_t* table = p.table + b * p.table_st;

    // pages of blocks k0 + 16 s + g8 and + 8; then their codes
    int page[2], off[2];
    auto lookup = [&](int sub) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = k0 + sub * 16 + g8 + 8 * h;
        page[h] = -1;
        off[h] = -1;  // no such block
        if (j < k1) {
          int m = j;
          if (p.per_page > 1) {
            m = __umulhi(uint32_t(j), p.page_magic);
            if (int64_t(m) * p.per_page > j) --m;
          }
          off[h] = j - m * p.per_page;
          page[h] = table[m];
        }
      }
    };
    uint4 key[2][DI / 64], next_key[2][DI / 64];
    float scale[2], next_scale[2];
    auto fetch = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool ok = page[h] >= 0 && page[h] < p.pages;
        if (!ok && off[h] >= 0 && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
        const int64_t phys = ok ? int64_t(page[h]) * p.per_page + off[h] : 0;
        next_scale[h] = __int_as_float(0x7fffffff);
#pragma unroll
        for (int i = 0; i < DI / 64; ++i) next_key[h][i] = make_uint4(0u, 0u, 0u, 0u);
        if (ok) {
          next_scale[h] = p.scales[phys];
#pragma unroll
          for (int i = 0; i < DI / 64; ++i)
            next_key[h][i] = *reinterpret_cast<const uint4*>(p.codes + phys * p.code_st + i * 64 + u * 16);
        }
      }
    };
    if (warp < subs) {
      lookup(warp);
      fetch();
      lookup(warp + kScoreThreads / 32);
    }

    // ---- the rows' codes and gains ----------------------------------------------------------
    __syncthreads();  // (the last piece's)
    for (int x = warp; subs > 0 && x < groups * NT; x += kScoreThreads / 32) {
      const int i = x % NT, c = 2 * i + (g8 & 1), row = (g8 >> 1) * C::kRx + c / HP, head = x / NT * 16 + c % HP;
      const bool live = row < n && head < p.Hi;
      uint4 raw[DI / 64][2];
#pragma unroll
      for (int k = 0; k < DI / 64; ++k) raw[k][0] = raw[k][1] = make_uint4(0u, 0u, 0u, 0u);
      float gain = 0.f;
      if (live) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (t0 + row) * p.q_st + head * p.q_sh + u * 16);
#pragma unroll
        for (int k = 0; k < DI / 64; ++k) raw[k][0] = src[k * 8], raw[k][1] = src[k * 8 + 1];
        gain = p.weight[(t0 + row) * p.w_st + head];
      }
      float xs[DI / 64][2][8];
      uint32_t top = 0u;
#pragma unroll
      for (int k = 0; k < DI / 64; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          bf16x8_to_f32(raw[k][e], xs[k][e]);
          top = max(top, top_bits(xs[k][e]));
        }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float s = code_scale(__uint_as_float(top));
#pragma unroll
      for (int k = 0; k < DI / 64; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) sQ[(x * C::kSteps + 2 * k + e) * 32 + lane] = int8x8_codes(xs[k][e], s);
      if (u == 0) sGain[x * 8 + g8] = live ? __fmul_rn(gain, s) : 0.f;
    }
    __syncthreads();
    // in registers where there is room
    constexpr bool kHold = NT <= 2;
    uint2 q[kHold ? NT : 1][C::kSteps];
    float gain[kHold ? C::kPer : 1];
    if constexpr (kHold) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int ks = 0; ks < C::kSteps; ++ks) q[i][ks] = sQ[(i * C::kSteps + ks) * 32 + lane];
#pragma unroll
      for (int x = 0; x < C::kPer; ++x) gain[x] = sGain[(x >> 1) * 8 + 2 * u + (x & 1)];
    }

    for (int sub = warp; sub < subs; sub += kScoreThreads / 32) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        scale[h] = next_scale[h];
#pragma unroll
        for (int i = 0; i < DI / 64; ++i) key[h][i] = next_key[h][i];
      }
      fetch();
      lookup(sub + 2 * (kScoreThreads / 32));
      float sum[C::kRx][2];  // [row of the thread][block g8, block g8 + 8]
      for (int g = 0; g < groups; ++g) {
        int acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0;
#pragma unroll
        for (int ks = 0; ks < C::kSteps; ++ks) {
          const uint4 k0w = key[0][ks >> 1], k1w = key[1][ks >> 1];
          const uint32_t a[4] = {ks & 1 ? k0w.z : k0w.x, ks & 1 ? k1w.z : k1w.x, ks & 1 ? k0w.w : k0w.y,
                                 ks & 1 ? k1w.w : k1w.y};
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            uint2 c;
            if constexpr (kHold) c = q[i][ks]; else c = sQ[((g * NT + i) * C::kSteps + ks) * 32 + lane];
            mma_s8_16832(acc[i], a, c.x, c.y);
          }
        }
#pragma unroll
        for (int x = 0; x < C::kPer; ++x) {
          float gx;
          if constexpr (kHold) gx = gain[x]; else gx = sGain[(g * NT + (x >> 1)) * 8 + 2 * u + (x & 1)];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // (a dot of 128 codes is below 2^24: exact)
            const float term = __fmul_rn(gx, float(max(acc[x >> 1][h * 2 + (x & 1)], 0)));
            float& s = sum[x / HP][h];
            s = (x % HP == 0 && g == 0) ? term : __fadd_rn(s, term);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = k0 + sub * 16 + g8 + 8 * h;
#pragma unroll
        for (int i = 0; i < C::kRx; ++i) {
          const int t = t0 + u * C::kRx + i;
          if (j < k1 && t < t0 + n)
            p.scores[(t - p.c0) * p.ld + j] = kept_score(sum[i][h], scale[h]);
        }
      }
    }
    at = end;
    if (at < u1 && at == before + int64_t((r.y - r.x + C::kRows - 1) / C::kRows) * per_tile) {  // the next sequence
      before = at;
      do ++b; while (units_at(b) == 0);
    }
  }
}

// ---- the score of many rows: tcgen05 -------------------------------------------------------

// A tile is 128 micro-blocks (the rows of the accumulator) by 256 columns, which are
// 256 / HP query rows of HP heads (HP: the heads rounded up to a power of two; missing ones
// have gain 0).  Column (r / 2) 2 HP + 2 h + r mod 2 is head h of row r: a lane of the
// accumulator holds one block's dots with all rows and heads, so the heads are added in order
// within a thread, two rows per packed instruction.
constexpr int kWideCols = 256;
constexpr int kWideStages = 6;                     // key tiles in shared memory
constexpr int kWideQ = 3;                          // Q tiles in shared memory (see the producers)
constexpr int kPrepParts = 4;                      // thread blocks that make a tile's codes
constexpr int kEpilogueWarps = 16, kGroupWarps = 4, kProducerWarps = 2 * kGroupWarps;
constexpr int kWideThreads = 32 * (kEpilogueWarps + kProducerWarps + 1);

__host__ __device__ constexpr int wide_tile_bytes(int DI) { return kWideCols * (DI + 4); }  // codes, then gains

struct WideTile {
  int b, t0, n, f;  // sequence, first row, rows, blocks to score (0: every row takes all its blocks)
};
__device__ __forceinline__ int tile_units(int f) { return (f + kKeyTile - 1) / kKeyTile; }

// The tile'th tile of the chunk [c0, c1): sequences in order, each cut into tiles of `rows`
// rows.  Called by a whole thread block; b = -1 past the last one.  `sh`: 4 ints.
template <int THREADS>
__device__ WideTile find_tile(const SelectParams& p, int c0, int c1, int tile, int rows, int* tmp, int* sh) {
  const int tid = threadIdx.x;
  if (tid == 0) sh[0] = -1;
  __syncthreads();
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += THREADS) {
    int2 r = make_int2(0, 0);
    if (b0 + tid < p.B) r = rows_of(p, b0 + tid, false);
    r.x = max(r.x, c0);
    r.y = min(r.y, c1);
    const int mine = r.y > r.x ? (r.y - r.x + rows - 1) / rows : 0;
    int total;
    const int before = base + block_scan<THREADS>(mine, tmp, total) - mine;
    if (tile >= before && tile < before + mine) {
      const int t0 = r.x + (tile - before) * rows;
      sh[0] = b0 + tid, sh[1] = t0, sh[2] = min(rows, r.y - t0);
    }
    base += total;
    __syncthreads();
    if (tile < base) break;
  }
  WideTile w{sh[0], sh[1], sh[2], 0};
  if (w.b >= 0) {
    const int last = rows_of(p, w.b, false).y - 1, len = length_of(p, w.b, false);
    const int f_most = max(len - (last - (w.t0 + w.n - 1)), 0) / p.block;
    w.f = f_most <= p.top ? 0 : f_most;
  }
  return w;
}

// The codes and gains of every tile's rows, laid out as the MMA reads them (no swizzle: 8
// columns by 16 bytes contiguous), and the list of tiles: blockIdx.x is the tile and the
// quarter of its columns, blockIdx.y the chunk of rows.
template <int DI, int HP>
__global__ void __launch_bounds__(256) qsa_select_prep_kernel(const SelectParams p, int chunk_rows) {
  constexpr int kLanes = DI / 8, kVec = 32 / kLanes;
  __shared__ int sTmp[8], sFound[4];
  begin_kernel();
  const int c0 = int(min(int64_t(blockIdx.y) * chunk_rows, int64_t(p.Tq)));
  const int c1 = int(min(int64_t(c0) + chunk_rows, int64_t(p.Tq)));
  const int tile = blockIdx.x / kPrepParts, part = blockIdx.x % kPrepParts;
  const WideTile w = find_tile<256>(p, c0, c1, tile, kWideCols / HP, sTmp, sFound);
  const int64_t slot = int64_t(blockIdx.y) * (gridDim.x / kPrepParts) + tile;
  if (threadIdx.x == 0 && part == 0) p.tiles[slot] = w.b < 0 ? make_int4(-1, 0, 0, 0) : make_int4(w.b, w.t0, w.n, w.f);
  if (w.b < 0 || w.f == 0) return;
  uint8_t* dst = p.tile_q + slot * wide_tile_bytes(DI);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % kLanes;
  constexpr int kRounds = kWideCols / kPrepParts / (8 * kVec);  // vectors of a thread
  constexpr int kAhead = kRounds < 4 ? kRounds : 4;
  static_assert(kRounds % kAhead == 0, "whole rounds");
  for (int i0 = 0; i0 < kRounds; i0 += kAhead) {
    uint4 raw[kAhead];
    float gain[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int v = part * (kWideCols / kPrepParts) + ((i0 + u) * 8 + warp) * kVec + lane / kLanes;  // column
      const int row = v / (2 * HP) * 2 + (v & 1), head = (v % (2 * HP)) >> 1;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      gain[u] = 0.f;
      if (row < w.n && head < p.Hi) {
        raw[u] = *reinterpret_cast<const uint4*>(p.q + (w.t0 + row) * p.q_st + head * p.q_sh + l * 8);
        gain[u] = p.weight[(w.t0 + row) * p.w_st + head];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int v = part * (kWideCols / kPrepParts) + ((i0 + u) * 8 + warp) * kVec + lane / kLanes;
      const int row = v / (2 * HP) * 2 + (v & 1), head = (v % (2 * HP)) >> 1;
      float xs[8];
      bf16x8_to_f32(raw[u], xs);
      uint32_t top = top_bits(xs);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = code_scale(__uint_as_float(top));
      const int c = l >> 1;
      *reinterpret_cast<uint2*>(dst + (c >> 1) * (kWideCols * 32) + (v >> 3) * 256 + (c & 1) * 128 + (v & 7) * 16 +
                                (l & 1) * 8) = int8x8_codes(xs, scale);
      if (l == 0)
        reinterpret_cast<float*>(dst + kWideCols * DI)[v] =
            row < w.n && head < p.Hi ? __fmul_rn(gain[u], scale) : 0.f;
    }
  }
}

// Shared-memory matrix descriptor of a K-major tile of 8-row, 16-byte core matrices without
// swizzle: 128 bytes between the two 16-byte halves of a 32-byte K step, 256 between 8-row
// groups; instruction descriptor of kind::i8: signed A and B, 32-bit integer accumulator.
__device__ __forceinline__ uint64_t core_desc(uint32_t addr) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t(128 >> 4) << 16) | (uint64_t(256 >> 4) << 32) | (uint64_t(1) << 46);
}
constexpr uint32_t kI8Desc = (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kWideCols >> 3) << 17) |
                             (uint32_t(kKeyTile >> 4) << 24);

__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

template <int DI>
struct Wide {
  static constexpr int kKeyBytes = kKeyTile * DI;
  static constexpr int kQBytes = wide_tile_bytes(DI);
  // key stages, Q tiles, the stages' scales
  static constexpr int kSmem = kWideStages * kKeyBytes + kWideQ * kQBytes + kWideStages * kKeyTile * 4;
};

// score(j) = scales[j] sum_h g_h max(0, c_h . codes[j]), the products of codes in 8-bit MMAs.
// One thread block per SM walks an equal share of all (tile of rows, tile of keys) pairs.
// Two groups of four warps bring key tiles in (16-byte asynchronous copies through the page
// table, a step behind their page lookups), one thread issues the MMAs into two
// accumulators, sixteen warps turn dots into scores.  What bounds it is those warps'
// instructions, not the MMAs (512 cycles of a unit's 3,400): per pair of dots an
// add-with-maximum each (the integer to float conversion 2^23 + max(d, 0) and the clamp at
// once; a dot of 128 codes is below 2^21), and a packed subtraction, product and sum.
// 7,810 rows of 4 heads over 14,400 to 16,384 blocks of 128 codes: 186 us, 0.66 P op/s (the
// same through warp-level MMAs with 64 columns a thread block took 1,000 us); eight warps
// with 128 columns each were 7 % slower, and neither the stores, the gains' loads nor the
// conversion's form (int to float instructions, or the subtraction folded into the product)
// moves the time.
template <int DI, int HP>
__global__ void __launch_bounds__(kWideThreads, 1)
    qsa_select_wide_kernel(const SelectParams p, const int4* tiles, const uint8_t* tile_q, int max_tiles) {
  using C = Wide<DI>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* sQ = smem + kWideStages * C::kKeyBytes;
  float* sScale = reinterpret_cast<float*>(sQ + kWideQ * C::kQBytes);             // [stages][128]
  // key stage full / free, Q full / free, accumulator full / free
  __shared__ __align__(8) uint64_t sBar[2 * kWideStages + 2 * kWideQ + 4];
  __shared__ uint32_t sTmem;
  __shared__ int sTmp[kWideThreads / 32], sStart[2], sLoaded[kWideQ];  // the last Q tile in each place
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return smem_addr(sBar + i); };
  constexpr int kFull = 0, kFree = kWideStages, kQFull = 2 * kWideStages, kQFree = kQFull + kWideQ,
                kAccFull = kQFree + kWideQ, kAccFree = kAccFull + 2;

  begin_kernel();
  // ---- this block's share ------------------------------------------------------------------
  int64_t total_units = 0;
  for (int i0 = 0; i0 < max_tiles; i0 += kWideThreads) {
    int total;
    block_scan<kWideThreads>(i0 + tid < max_tiles ? tile_units(tiles[i0 + tid].w) : 0, sTmp, total);
    total_units += total;
  }
  const int64_t u0 = total_units * blockIdx.x / gridDim.x, u1 = total_units * (blockIdx.x + 1) / gridDim.x;
  if (u0 == u1) return;
  int64_t base = 0;
  for (int i0 = 0; i0 < max_tiles; i0 += kWideThreads) {
    const int mine = i0 + tid < max_tiles ? tile_units(tiles[i0 + tid].w) : 0;
    int total;
    const int64_t before = base + block_scan<kWideThreads>(mine, sTmp, total) - mine;
    if (u0 >= before && u0 < before + mine) sStart[0] = i0 + tid, sStart[1] = int(u0 - before);
    base += total;
    if (base > u0) break;  // (uniform)
  }
  if (tid == 0) {
    for (int i = 0; i < kWideStages; ++i) {
      mbar_init(bar(kFull + i), 32 * kGroupWarps);
      mbar_init(bar(kFree + i), 1 + kEpilogueWarps);
    }
    for (int i = 0; i < kWideQ; ++i) {
      sLoaded[i] = -1;
      mbar_init(bar(kQFull + i), 1);
      mbar_init(bar(kQFree + i), 1 + kEpilogueWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kAccFull + i), 1);
      mbar_init(bar(kAccFree + i), kEpilogueWarps);
    }
    mbar_init_fence();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sTmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sTmem;
  const int tile0 = sStart[0], first_kt = sStart[1];
  const int share = int(u1 - u0);
  bool late = false;

  if (warp >= kEpilogueWarps && warp < kEpilogueWarps + kProducerWarps) {
    // ---- producers: two groups take the key tiles in turn, one key row per thread ----------------
    // A group hands tile i over once it has issued tile i + 2.  So when it waits for the Q tile
    // three before the one it is about to load, whose last key tile is i - 3 or earlier, both
    // groups have handed over all that the wait depends on, or will without waiting for this.
    const int group = (warp - kEpilogueWarps) / kGroupWarps, r = tid - 32 * (kEpilogueWarps + group * kGroupWarps);
    int tile = tile0, kt = first_kt, qn = 0;  // qn: the Q tile's number within this block
    bool new_q = true;
    int4 w = tiles[tile];
    auto advance = [&]() {
      new_q = false;
      if (++kt == tile_units(w.w)) {
        kt = 0;
        new_q = true;
        ++qn;
        do ++tile; while (tile < max_tiles && tiles[tile].w == 0);
        if (tile < max_tiles) w = tiles[tile];
      }
    };
    // of this thread's row of key tile kt of w: the page as the table has it, the block within
    // it, and whether there is such a block (used one step later, when the load has arrived)
    int page = -1, off = 0;
    bool live = false;
    auto lookup = [&]() {
      const int j = kt * kKeyTile + r;
      live = j < w.w;
      if (!live) return;
      int m = j;
      if (p.per_page > 1) {
        m = __umulhi(uint32_t(j), p.page_magic);
        if (int64_t(m) * p.per_page > j) --m;
      }
      off = j - m * p.per_page;
      page = p.table[w.x * p.table_st + m];
    };
    if (group == 1 && share > 1) advance();
    lookup();
    const uint32_t row_s = smem_addr(smem) + (r >> 3) * 256 + (r & 7) * 16;
    int issued = 0;
    for (int i = group; i < share; i += 2, ++issued) {
      const bool ok = live && page >= 0 && page < p.pages, bad = live && !ok;
      const int64_t phys = ok ? int64_t(page) * p.per_page + off : 0;
      const bool load_q = new_q;
      const int this_tile = tile, this_q = qn;
      if (i + 1 < share) advance();
      if (i + 2 < share) {
        advance();
        lookup();
      }
      const int stage = i % kWideStages;
      if (i >= kWideStages && !wait_phase(bar(kFree + stage), (i / kWideStages - 1) & 1, p.wait_ns)) late = true;
      if (load_q && r == 0 && !late) {
        const int qb = this_q % kWideQ;
        if (this_q >= kWideQ && !wait_phase(bar(kQFree + qb), (this_q / kWideQ - 1) & 1, p.wait_ns)) late = true;
        if (!late) {
          mbar_arrive_expect_tx(bar(kQFull + qb), C::kQBytes);
          bulk_copy(smem_addr(sQ) + qb * C::kQBytes, tile_q + int64_t(this_tile) * C::kQBytes, C::kQBytes,
                    bar(kQFull + qb));
          atomicMax(&sLoaded[qb], this_q);
        }
      }
      if (late) break;
      if (bad && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      const int8_t* src = p.codes + phys * p.code_st;
      const uint32_t dst = row_s + stage * C::kKeyBytes;
#pragma unroll
      for (int c = 0; c < DI / 16; ++c)
        cp_async_16(dst + (c >> 1) * (kKeyTile * 32) + (c & 1) * 128, ok ? src + c * 16 : src, ok);
      if (ok)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem_addr(sScale + stage * kKeyTile + r)),
                     "l"(p.scales + phys)
                     : "memory");
      else
        sScale[stage * kKeyTile + r] = __int_as_float(0x7fffffff);
      cp_async_commit();
      if (issued >= 1) {  // the group's tile before has landed: hand it over
        cp_async_wait<1>();
        fence_proxy_async_smem();
        mbar_arrive(bar(kFull + (i - 2) % kWideStages));
      }
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    if (!late && issued > 0) mbar_arrive(bar(kFull + (group + 2 * (issued - 1)) % kWideStages));
  } else if (warp == kEpilogueWarps + kProducerWarps) {
    // ---- one thread issues the MMAs ------------------------------------------------------------
    if (lane == 0) {
      int kt = first_kt, tile = tile0, units = tile_units(tiles[tile0].w), qn = 0;
      bool new_q = true;
      int i = 0;
      for (; i < share; ++i) {
        const int stage = i % kWideStages, acc = i & 1;
        if (new_q) late = !wait_phase(bar(kQFull + qn % kWideQ), (qn / kWideQ) & 1, p.wait_ns);
        if (!late) late = !wait_phase(bar(kFull + stage), (i / kWideStages) & 1, p.wait_ns);
        if (!late && i >= 2) late = !wait_phase(bar(kAccFree + acc), ((i >> 1) - 1) & 1, p.wait_ns);
        if (late) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t a = smem_addr(smem) + stage * C::kKeyBytes, q = smem_addr(sQ) + (qn % kWideQ) * C::kQBytes;
#pragma unroll
        for (int k = 0; k < DI / 32; ++k)
          asm volatile(
              "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
              "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem + acc * kWideCols),
              "l"(core_desc(a + k * (kKeyTile * 32))), "l"(core_desc(q + k * (kWideCols * 32))), "r"(kI8Desc),
              "r"(uint32_t(k != 0)));
        auto commit = [&](int b) {
          asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar(b))
                       : "memory");
        };
        commit(kAccFull + acc);
        commit(kFree + stage);
        new_q = false;
        if (++kt == units) {
          commit(kQFree + qn % kWideQ);
          ++qn;
          kt = 0;
          new_q = true;
          do ++tile; while (tile < max_tiles && tiles[tile].w == 0);
          units = tile < max_tiles ? tile_units(tiles[tile].w) : 0;
        }
      }
      if (i > 0) late |= !wait_phase(bar(kAccFull + ((i - 1) & 1)), ((i - 1) >> 1) & 1);  // no MMA in flight
    }
  } else {
    // ---- dots to keys --------------------------------------------------------------------------
    constexpr int kParts = kEpilogueWarps / 4, kPartCols = kWideCols / kParts;
    static_assert(kPartCols % 32 == 0, "whole loads");
    const int quad = warp & 3, part = warp >> 2;  // lanes of the accumulator, part of its columns
    const int r = quad * 32 + lane;
    constexpr int kPartRows = kPartCols / HP;
    int tile = tile0, kt = first_kt, qn = 0;
    bool new_q = true;
    int4 w = tiles[tile];
    for (int i = 0; i < share; ++i) {
      const int stage = i % kWideStages, acc = i & 1;
      // (the key stage and the Q tile landed before their product: these waits order the reads)
      bool here = wait_phase(bar(kFull + stage), (i / kWideStages) & 1, p.wait_ns);
      if (new_q) here = here && wait_phase(bar(kQFull + qn % kWideQ), (qn / kWideQ) & 1, p.wait_ns);
      new_q = false;
      here = here && wait_phase(bar(kAccFull + acc), (i >> 1) & 1, p.wait_ns);
      if (__any_sync(0xffffffffu, !here)) {
        late = true;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const float scale = sScale[stage * kKeyTile + r];
      const int j = kt * kKeyTile + r;
      const uint64_t scale2 = pack2(scale, scale);
      const float* gains = reinterpret_cast<const float*>(sQ + (qn % kWideQ) * C::kQBytes + kWideCols * DI) + part * kPartCols;
      const int row0 = part * kPartRows;
      uint32_t at = uint32_t(w.y + row0 - p.c0) * uint32_t(p.ld) + uint32_t(j);  // (a chunk has fewer than 2^30)
      const int rows = j < p.ld ? (w.z & (kLate - 1)) - row0 : 0;  // that this lane stores
      const uint64_t minus = pack2(-8388608.f, -8388608.f), zero = pack2(0.f, 0.f);
      uint64_t sum = zero;
#pragma unroll
      for (int c = 0; c < kPartCols / 32; ++c) {
        uint32_t d[32];
        tmem_ld32(d, tmem + acc * kWideCols + part * kPartCols + c * 32 + (uint32_t(quad * 32) << 16));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (c == kPartCols / 32 - 1) {  // the accumulator has been read
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kAccFree + acc));
        }
#pragma unroll
        for (int x = 0; x < 32; x += 4) {  // two heads of a pair of rows (HP = 1: two pairs of rows)
          const float4 g = *reinterpret_cast<const float4*>(gains + c * 32 + x);
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = __int_as_float(__viaddmax_s32(int(d[x + e]), 0x4B000000, 0x4B000000));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = c * 32 + x + 2 * e, head = (col % (2 * HP)) >> 1, pair = col / (2 * HP);
            // (a product rounded by itself: written as mul2, it and the sum's add2 became one fused
            // operation, packed .rn instructions or not, and 17 % of four-head scores came out a step off)
            const uint64_t term = fma2(add2(pack2(f[2 * e], f[2 * e + 1]), minus),
                                       e == 0 ? pack2(g.x, g.y) : pack2(g.z, g.w), zero);
            sum = head == 0 ? term : add2(sum, term);
            if (head == HP - 1) {
              float s[2];
              unpack2(fma2(sum, scale2, zero), s[0], s[1]);  // (as kept_score)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if (2 * pair + k < rows) p.scores[at] = fmaxf(s[k], -__builtin_huge_valf());  // (NaN: -infinity)
                at += uint32_t(p.ld);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kFree + stage));
      if (++kt == tile_units(w.w)) {
        if (lane == 0) mbar_arrive(bar(kQFree + qn % kWideQ));
        ++qn;
        kt = 0;
        new_q = true;
        do ++tile; while (tile < max_tiles && tiles[tile].w == 0);
        if (tile < max_tiles) w = tiles[tile];
      }
    }
  }
  // A wait that ran out leaves scores unwritten: the choice gives the chunk's rows no slots.  No
  // product and no copy of a thread of its own is in flight here; the bulk copies of Q tiles have
  // landed when their product was issued, or are waited for now (one second at most).
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  if (__syncthreads_or(late)) {
    if (late) {
      atomicOr(p.late, kLate);
      if (p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_TIMEOUT);
    }
    if (tid < kWideQ && sLoaded[tid] >= 0) wait_phase(bar(kQFull + tid), (sLoaded[tid] / kWideQ) & 1);
    __syncthreads();
  }
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// ---- the choice --------------------------------------------------------------------------

constexpr int kBins = 512;     // of a histogram: 16 per lane of one warp
constexpr int kSample = 1024;  // keys that estimate the border of a long row
constexpr int kWindow = 1024;  // most words of the marks: 32,768 blocks at a time

// The border of a row: blocks of a larger key are taken, of `equal` equal ones the first `want`.
struct Border {
  uint32_t key;
  int want, equal;
};

// Blocks to slots through a sequence's pages.
struct SlotMap {
  const SelectParams& p;
  const int32_t* table;
  __device__ __forceinline__ int first_slot(int j) const {  // of block j, or -1
    int m = j;
    if (p.per_page > 1) {
      m = __umulhi(uint32_t(j), p.page_magic);  // j / per_page, or one more
      if (int64_t(m) * p.per_page > j) --m;
    }
    const int page = table[m];
    if (page < 0 || page >= p.pages) {
      if (p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      return -1;
    }
    return page * p.page_size + (j - m * p.per_page) * p.block;
  }
};

// A list of blocks becomes a list of their first slots, four page lookups of a thread at once.
template <int THREADS>
__device__ __forceinline__ void list_slots(const SlotMap& map, int* list, int n, int tid) {
  const SelectParams& p = map.p;
  bool bad = false;
  for (int i0 = tid; i0 < n; i0 += 4 * THREADS) {
    int off[4], page[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * THREADS;
      page[u] = 0;
      off[u] = 0;
      if (i >= n) continue;
      const int j = list[i];
      int m = j;
      if (p.per_page > 1) {
        m = __umulhi(uint32_t(j), p.page_magic);  // j / per_page, or one more
        if (int64_t(m) * p.per_page > j) --m;
      }
      off[u] = (j - m * p.per_page) * p.block;
      page[u] = map.table[m];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool ok = page[u] >= 0 && page[u] < p.pages;
      bad |= !ok;
      if (i0 + u * THREADS < n) list[i0 + u * THREADS] = ok ? page[u] * p.page_size + off[u] : -1;
    }
  }
  if (bad && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
}

// Whether the chunk's scores are not whole (read after the score kernel's end): the choice then
// goes on as if its rows saw nothing.
__device__ __forceinline__ bool scores_late(const SelectParams& p) { return p.late != nullptr && (*p.late & kLate) != 0; }

// Row t's output from the first slots of its taken blocks, by THREADS threads.
template <int THREADS>
__device__ __forceinline__ void write_row(const SelectParams& p, const SlotMap& map, int t, int tid, const int* sList,
                                          int f, int taken, int seen) {
  int32_t* out = p.out + t * p.out_st;
  const int W = p.top * p.block + p.block - 1, full = taken * p.block, tail = seen - f * p.block;
  if (p.block == 4) {  // (the usual micro-block: no division)
#pragma unroll 8
    for (int w = tid; w < full; w += THREADS) {
      const int s = sList[w >> 2];
      out[w] = s < 0 ? -1 : s + (w & 3);
    }
  } else {
    for (int w = tid; w < full; w += THREADS) {
      const int i = p.block == 1 ? w : int(__umulhi(uint32_t(w), p.block_magic));  // w / block (w below 2^14)
      out[w] = sList[i] < 0 ? -1 : sList[i] + (w - i * p.block);
    }
  }
  const int tail_slot = tail > 0 ? map.first_slot(f) : -1;
  for (int w = full + tid; w < W; w += THREADS)
    out[w] = w < full + tail && tail_slot >= 0 ? tail_slot + (w - full) : -1;
  if (tid == 0) p.width[t] = full + tail;
}

struct alignas(16) ChooseShared {  // (the histogram is read 16 bytes at a time)
  int hist[kBins];
  uint32_t few[32];
  uint32_t hi;
  int n_few, bin, above, count, n;
};

constexpr int kPickWarps = 4;    // rows of a thread block of the kernel for short rows
constexpr int kPickKeys = 2048;  // most blocks of such a row

// mask |= bit when x >= low: two instructions.
__device__ __forceinline__ void keep_bit(uint32_t& mask, float x, float low, uint32_t bit) {
  asm("{\n  .reg .pred q;\n  setp.ge.f32 q, %1, %2;\n  @q or.b32 %0, %0, %3;\n}\n" : "+r"(mask) : "f"(x), "f"(low), "r"(bit));
}

template <int THREADS>
__device__ __forceinline__ void sync_all() {
  if constexpr (THREADS == 32) __syncwarp(); else __syncthreads();
}

// The want-th largest (at least 1) of the keys keys_at(0 .. n - 1) of four neighbours each, the
// zeros among them not counted, by histograms of the key range that still holds it; the
// last step ranks at most 32 keys within each warp.  Without EXACT: a key at most that one
// with few keys between them (`key` alone is meant).  (The keys come four at a time because
// no load moves ahead of an atomic: key by key a warp took 10,000 to 27,000 cycles for 500 to
// 2,000 keys.)
template <int THREADS, bool EXACT, class F>
__device__ Border kth_largest(int n, int want, F keys_at, ChooseShared& sh) {
  const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x, lane = tid & 31;
  sync_all<THREADS>();  // (sh and the keys)
  if (tid == 0) sh.hi = kLeastKey, sh.n_few = 0;
  for (int i = tid; i < kBins; i += THREADS) sh.hist[i] = 0;
  uint32_t hi = 0u;
#pragma unroll 4
  for (int i = tid; i < n; i += THREADS) {
    const uint4 k = keys_at(i);
    hi = max(max(max(hi, k.x), k.y), max(k.z, k.w));
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (THREADS > 32) {
    sync_all<THREADS>();
    if (lane == 0) atomicMax(&sh.hi, hi);
    sync_all<THREADS>();
    hi = sh.hi;
  } else {
    hi = max(hi, kLeastKey);
    sync_all<THREADS>();
  }
  // The keys are floats in order: most of a row's lie in a few octaves below the largest, so
  // the first histogram takes four of them, and the whole range only if that is not enough.
  uint32_t lo = hi - kLeastKey > (4u << 23) ? hi - (4u << 23) : kLeastKey;
  for (;;) {
    const uint32_t range = hi - lo;
    const int shift = range < uint32_t(kBins) ? 0 : 32 - __clz(range) - 9;  // 2^9 = kBins
    for (int i = tid; i < n; i += 2 * THREADS) {
      const uint4 a = keys_at(i), b = i + THREADS < n ? keys_at(i + THREADS) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t k[8] = {a.x - lo, a.y - lo, a.z - lo, a.w - lo, b.x - lo, b.y - lo, b.z - lo, b.w - lo};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k[e] <= range) atomicAdd(&sh.hist[k[e] >> shift], 1);
    }
    sync_all<THREADS>();
    if (tid < 32) {  // lane i holds bins 511 - 16 i down to 496 - 16 i
      const int first = kBins - 16 * (lane + 1);
      int c[16], mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int4 x = *reinterpret_cast<const int4*>(&sh.hist[first + 4 * e]);
        c[4 * e] = x.x, c[4 * e + 1] = x.y, c[4 * e + 2] = x.z, c[4 * e + 3] = x.w;
        mine += x.x + x.y + x.z + x.w;
      }
      int above = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += y;
      }
      above -= mine;
      if (lane == 31 && above + mine < want) sh.bin = -1;
      if (above < want && above + mine >= want) {
#pragma unroll
        for (int e = 15; e >= 0; --e) {
          if (above < want && above + c[e] >= want) sh.bin = first + e, sh.above = above, sh.count = c[e];
          above += c[e];
        }
      }
    }
    sync_all<THREADS>();
    if (sh.bin < 0) {  // fewer keys than wanted above lo
      if (lo == kLeastKey) return {lo, want, want};  // (never: at least `want` keys take part)
      lo = kLeastKey;
      for (int i = tid; i < kBins; i += THREADS) sh.hist[i] = 0;
      sync_all<THREADS>();
      continue;
    }
    want -= sh.above;
    const int count = sh.count;
    lo += uint32_t(sh.bin) << shift;
    hi = lo + min(hi - lo, (1u << shift) - 1u);
    if (shift == 0) return {lo, want, count};
    if (count <= 32) {
      if constexpr (!EXACT) {
        return {lo, want, count};
      } else {
        for (int i = tid; i < n; i += 2 * THREADS) {
          const uint4 a = keys_at(i), b = i + THREADS < n ? keys_at(i + THREADS) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t k[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          bool any = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) any |= k[e] - lo <= hi - lo;
          if (!any) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (k[e] - lo <= hi - lo) sh.few[atomicAdd(&sh.n_few, 1)] = k[e];
        }
        sync_all<THREADS>();
        const uint32_t mine = sh.few[lane < count ? lane : 0];
        int more = 0, same = 0;
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
          const uint32_t k = __shfl_sync(0xffffffffu, mine, i);
          more += k > mine;
          same += k == mine;
        }
        const uint32_t at = __ballot_sync(0xffffffffu, lane < count && more < want && more + same >= want);
        const int src = __ffs(at) - 1;
        return {__shfl_sync(0xffffffffu, mine, src), want - __shfl_sync(0xffffffffu, more, src),
                __shfl_sync(0xffffffffu, same, src)};
      }
    }
    for (int i = tid; i < kBins; i += THREADS) sh.hist[i] = 0;
    sync_all<THREADS>();
  }
}

// Rows of at most kPickKeys blocks, a warp each: its keys lie in the warp's shared memory,
// nothing is shared between warps, and no barrier is waited for.  Bound: the latency of its
// steps in shared memory, with 20 warps to an SM.  16,384 rows of up to 2,048 blocks, 512
// taken: 110 us.
__global__ void __launch_bounds__(32 * kPickWarps) qsa_select_pick_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint32_t dyn[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row_at = blockIdx.x * kPickWarps + warp, t = p.c0 + row_at;
  launch_next();
  if (p.first) wait_for_last();  // (no score kernel came before)
  if (t >= p.c1) {
    wait_for_last();
    return;
  }
  __shared__ __align__(16) ChooseShared sSearch[kPickWarps];
  uint32_t* sKey = dyn + warp * p.cap;
  int* sList = reinterpret_cast<int*>(sKey);  // (a taken block's place is never behind its own key's)
  int b = -1;
  if (p.cu == nullptr) {
    if (t < p.B) b = t;
  } else {
    for (int i0 = 0; i0 < p.B; i0 += 32) {
      bool mine = false;
      if (i0 + lane < p.B) {
        const int2 r = rows_of(p, i0 + lane, row_at == 0 && p.c0 == 0);
        mine = t >= r.x && t < r.y;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, mine);
      if (m != 0u) b = i0 + 31 - __clz(m);  // (offsets that overlap: the last one)
    }
  }
  if (b < 0) {
    wait_for_last();
    return;
  }
  const int last = rows_of(p, b, false).y - 1, len = length_of(p, b, lane == 0);
  wait_for_last();  // the scores
  const int seen = scores_late(p) ? 0 : max(len - (last - t), 0), f = seen / p.block, taken = min(f, p.top);
  const SlotMap map{p, p.table + b * p.table_st};
  if (f <= p.top) {
    for (int j = lane; j < f; j += 32) sList[j] = map.first_slot(j);
  } else {
    // blocks that are taken whatever they score do not take part in the search: key 0
    const uint4* row4 = reinterpret_cast<const uint4*>(p.scores + int64_t(row_at) * p.ld) + lane;
    uint4* key4 = reinterpret_cast<uint4*>(sKey) + lane;
    auto forced = [&](int j) { return j < p.sink || j >= f - p.local; };
#pragma unroll 4
    for (int i = 0; i * 128 < f; ++i) {
      const int j = i * 128 + lane * 4;
      uint4 k = make_uint4(0u, 0u, 0u, 0u);
      if (j < f) k = load_l2(row4 + i * 32);
      k = make_uint4(order_key(k.x), order_key(k.y), order_key(k.z), order_key(k.w));
      if (i * 128 < p.sink || i * 128 + 128 > f - p.local) {
        if (forced(j)) k.x = 0u;  // (or past the end)
        if (forced(j + 1)) k.y = 0u;
        if (forced(j + 2)) k.z = 0u;
        if (forced(j + 3)) k.w = 0u;
      }
      key4[i * 32] = k;
    }
    __syncwarp();
    const int want = p.top - p.sink - p.local;
    Border border{0xffffffffu, 0, 0};
    if (want > 0) border = kth_largest<32, true>((f + 3) / 4, want, [&](int i) { return reinterpret_cast<uint4*>(sKey)[i]; }, sSearch[warp]);
    const bool all_same = border.want == border.equal;
    const uint32_t below = (1u << lane) - 1u, least = all_same ? border.key : border.key + 1u;
    int have = 0, same = 0;
    for (int i = 0; i * 128 < f; ++i) {  // a lane has four neighbours
      const uint4 k4 = key4[i * 32];
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
      const int j = i * 128 + lane * 4;
      const bool edge = i * 128 < p.sink || i * 128 + 128 > f - p.local;
      uint32_t take[4];
      int at = have, mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bool in = k[e] >= least;
        if (edge || least == 0u) in = j + e < f && ((want > 0 && in && !forced(j + e)) || forced(j + e));
        take[e] = __ballot_sync(0xffffffffu, in);
      }
      if (!all_same) {  // of equal keys the first ones
        uint32_t eq[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          eq[e] = __ballot_sync(0xffffffffu, j + e < f && k[e] == border.key && !forced(j + e));
        int before = same;
#pragma unroll
        for (int e = 0; e < 4; ++e) before += __popc(eq[e] & below);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool is_eq = (eq[e] >> lane) & 1;
          take[e] |= __ballot_sync(0xffffffffu, is_eq && before < border.want);
          before += is_eq;
          same += __popc(eq[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) at += __popc(take[e] & below);
      __syncwarp();  // (every lane has its keys of this group)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((take[e] >> lane) & 1) sList[at + mine++] = j + e;
        have += __popc(take[e]);
      }
    }
    __syncwarp();
    list_slots<32>(map, sList, p.top, lane);
  }
  __syncwarp();
  write_row<32>(p, map, t, lane, sList, f, taken, seen);
}

// One thread block per row.  A row of at most `cap` blocks has its keys in shared memory.  Of
// a longer one, the keys above a border estimated from kSample of them are collected there
// in one pass.  For about one row in 400 of random scores that is more than there is room for,
// and the row is collected again above a better border; one that still does not fit, or an
// estimate that left out too many (keys that repeat with the sample's period), has its keys
// searched in place.
// The exact border follows from what was collected; a bit per block marks the taken ones,
// and a scan over the marks gives them their places in ascending order.
// Bound: instructions and the latency of its steps, 10 rows to an SM; the scores are read
// once.  7,810 rows of 15,400 blocks, 512 taken: 244 us (radix passes over the whole row, four
// reads and a conflicting shared-memory atomic per score and pass, took 1,250).
template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? 10 : THREADS == 256 ? 4 : 1) qsa_select_choose_kernel(const SelectParams p) {
  constexpr int kBatch = THREADS == 1024 ? 4 : 2;  // 16-byte loads of keys per thread and step
  extern __shared__ __align__(16) uint32_t dyn[];
  uint32_t* sKey = dyn;  // [cap], and room for `queue` 16-bit numbers before the keys are there
  int* sIdx = reinterpret_cast<int*>(sKey + max(p.cap, p.ld > p.cap ? p.queue / 2 : 0));  // [cap], absent when every row fits
  int* sList = sIdx + (p.ld > p.cap ? p.cap : 0);             // [top] first slot of each taken block, or -1
  __shared__ __align__(16) ChooseShared sh;
  uint32_t* sOver = reinterpret_cast<uint32_t*>(sList + (p.top + 3) / 4 * 4);  // [window] each
  uint32_t* sSame = sOver + p.window;
  __shared__ int sTmp[THREADS / 32], sSeq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = p.c0 + blockIdx.x;
  launch_next();
  if (p.first) wait_for_last();  // (no score kernel came before)
  if (tid == 0) sSeq = (p.cu == nullptr && t < p.B) ? t : -1;
  __syncthreads();
  if (p.cu != nullptr) {
    for (int i = tid; i < p.B; i += THREADS) {
      const int2 r = rows_of(p, i, blockIdx.x == 0 && p.c0 == 0);
      if (t >= r.x && t < r.y) atomicMax(&sSeq, i);  // (offsets that overlap: the last one)
    }
    __syncthreads();
  }
  const int b = sSeq;
  if (b < 0) {
    wait_for_last();
    return;
  }
  const int last = rows_of(p, b, false).y - 1, len = length_of(p, b, tid == 0);
  wait_for_last();  // the scores
  const int seen = scores_late(p) ? 0 : max(len - (last - t), 0);
  const int f = seen / p.block, taken = min(f, p.top);
  const float* row = p.scores + blockIdx.x * p.ld;
  const SlotMap map{p, p.table + b * p.table_st};
  if (f <= p.top) {
    for (int j = tid; j < f; j += THREADS) sList[j] = map.first_slot(j);
  } else {
    // blocks that are taken whatever they score do not take part in the search
    const int want = p.top - p.sink - p.local;
    auto forced = [&](int j) { return j < p.sink || j >= f - p.local; };
    auto searched = [&](int j, uint32_t score) { return forced(j) ? 0u : order_key(score); };
    auto in_row = [&](int j) { return searched(j, __float_as_uint(load_l2(row + j))); };
    const uint4* row4 = reinterpret_cast<const uint4*>(row);  // (ld is a multiple of 32)
    auto four_in_row = [&](int i) {  // (past the end: not searched)
      const uint4 k = load_l2(row4 + i);
      return make_uint4(searched(4 * i, k.x), searched(4 * i + 1, k.y), searched(4 * i + 2, k.z),
                        searched(4 * i + 3, k.w));
    };
    auto four_in_list = [&](int i) { return reinterpret_cast<const uint4*>(sKey)[i]; };
    Border border{0xffffffffu, 0, 0};
    int listed = want > 0 ? -1 : 0;  // keys collected with their blocks; -1: every block of the row is searched
    if (want == 0) {
      // nothing but those
    } else if (f <= p.cap) {
      for (int i0 = tid; i0 * 4 < f; i0 += THREADS * kBatch) {
        uint4 k[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if ((i0 + u * THREADS) * 4 < f) k[u] = load_l2(row4 + i0 + u * THREADS);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = (i0 + u * THREADS) * 4;
          if (j >= f) break;
          *reinterpret_cast<uint4*>(sKey + j) = make_uint4(searched(j, k[u].x), searched(j + 1, k[u].y),
                                                           searched(j + 2, k[u].z), searched(j + 3, k[u].w));
        }
      }
      border = kth_largest<THREADS, true>((f + 3) / 4, want, four_in_list, sh);
    } else {
      {
        uint32_t k[kSample / THREADS];  // one from each of kSample equal parts of the row
#pragma unroll
        for (int u = 0; u < kSample / THREADS; ++u) {
          const uint32_t i = tid + u * THREADS;
          k[u] = in_row(int((uint64_t(i) * uint32_t(f) + __umulhi(i * 2654435769u, uint32_t(f))) / kSample));
        }
#pragma unroll
        for (int u = 0; u < kSample / THREADS; ++u) sKey[tid + u * THREADS] = k[u];
      }
      // of the row's `want` best, about `hits` are in the sample: the border lies 4 deviations lower
      const float hits = float(want) * kSample / float(f);
      int rank = min(int(hits + 4.f * sqrtf(hits)) + 4, kSample);
      uint32_t low = kth_largest<THREADS, false>(kSample / 4, rank, four_in_list, sh).key;
      // The blocks of keys from `low` up: every lane queues the ones it meets (16-bit numbers, in
      // the keys' room), a scan over the lanes then puts the queues together.  More than there
      // is room for: the want-th largest of those that had room is a better border, since as
      // many keys as wanted reach it (if it is the border they were collected by, the keys above it
      // come next).  Otherwise every block of the row is searched.
      uint16_t* queue = reinterpret_cast<uint16_t*>(sKey);
      const int longest = p.queue / THREADS;
      constexpr int kStep = THREADS * kBatch;  // 16-byte loads of a step
      bool tied = false;  // the want-th largest of some of the keys is low - 1
      bool found = false;
      for (int tries = 0; tries < 3; ++tries) {
        __syncthreads();
        if (tid == 0) sh.n = 0;
        __syncthreads();
        const float least = key_score(low);
        int have = 0, all = 0;
        for (int s0 = 0; s0 * 4 < f; s0 += kStep * (65536 / (4 * kBatch))) {
          const int s1 = int(min(int64_t(s0) + kStep * (65536 / (4 * kBatch)), int64_t(f + 3) / 4));
          uint4 raw[kBatch], next[kBatch];
          auto load = [&](int i0) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              next[u] = make_uint4(0u, 0u, 0u, 0u);
              if ((i0 + lane + u * THREADS) * 4 < f) next[u] = load_l2(row4 + i0 + lane + u * THREADS);
            }
          };
          load(s0 + warp * 32);
          int mine = 0, number = 0;
          for (int i0 = s0 + warp * 32; i0 < s1; i0 += kStep, number += 4 * kBatch) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) raw[u] = next[u];
            if (i0 + kStep < s1) load(i0 + kStep);
            float k[4 * kBatch];
            uint32_t keep = 0u;  // a bit per score of this lane
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
              k[4 * u] = __uint_as_float(raw[u].x), k[4 * u + 1] = __uint_as_float(raw[u].y),
              k[4 * u + 2] = __uint_as_float(raw[u].z), k[4 * u + 3] = __uint_as_float(raw[u].w);
            if (i0 * 4 >= p.sink && (i0 + 32 + (kBatch - 1) * THREADS) * 4 <= f - p.local) {
#pragma unroll
              for (int x = 0; x < 4 * kBatch; ++x) keep_bit(keep, k[x], least, 1u << x);
            } else {
#pragma unroll
              for (int x = 0; x < 4 * kBatch; ++x) {
                const int j = (i0 + lane + (x >> 2) * THREADS) * 4 + (x & 3);
                keep |= j < f && !forced(j) && k[x] >= least ? 1u << x : 0u;
              }
            }
            while (keep != 0u) {
              const int x = __ffs(keep) - 1;
              keep &= keep - 1;
              if (mine < longest) queue[mine * THREADS + tid] = uint16_t(number + x);
              ++mine;
            }
          }
          all += mine;
          const int kept = min(mine, longest);
          int total;
          int at = have + block_scan<THREADS>(kept, sTmp, total) - kept;
          for (int i = 0; i < kept && at < p.cap; ++i, ++at) {
            const int v = queue[i * THREADS + tid], x = v % (4 * kBatch);
            sIdx[at] = (s0 + v / (4 * kBatch) * kStep + warp * 32 + lane + (x >> 2) * THREADS) * 4 + (x & 3);
          }
          have += total;
          __syncthreads();  // (the queues)
        }
        all = int(__reduce_add_sync(0xffffffffu, unsigned(all)));
        if (lane == 0) atomicAdd(&sh.n, all);
        __syncthreads();
        const int n = sh.n, room = min(have, p.cap);
        if (room < want) {
          // above a key that more share than there is room for: that one is the border
          // (a number of equal ones that is never `want`: the first of them are counted off)
          if (tied && n < want) border = {low - 1u, want - n, INT32_MAX}, found = true;
          break;
        }
#pragma unroll 4
        for (int i = tid; i < room; i += THREADS) sKey[i] = order_key(__float_as_uint(load_l2(row + sIdx[i])));
        if (tid < 4 && room + tid < (room + 3) / 4 * 4) sKey[room + tid] = 0u;
        border = kth_largest<THREADS, true>((room + 3) / 4, want, four_in_list, sh);
        if (n == room) {
          listed = n;
          break;
        }
        tied = border.key <= low;
        low = tied ? low + 1u : border.key;
      }
      if (listed < 0 && !found) border = kth_largest<THREADS, true>((f + 3) / 4, want, four_in_row, sh);
    }
    // ---- marks and places, a window of blocks at a time ----------------------------------------
    const bool all_same = border.want == border.equal;  // no choice between equal keys
    int have = 0, same = 0;
    for (int w0 = 0; w0 * 32 < f; w0 += p.window) {
      const int words = min(p.window, (f + 31) / 32 - w0);
      auto over = [&](uint32_t k) { return k > border.key || (all_same && k == border.key); };
      if (listed >= 0) {
        __syncthreads();  // (the last window's marks)
        for (int i = tid; i < words; i += THREADS) sOver[i] = sSame[i] = 0u;
        __syncthreads();
        for (int i = tid; i < listed; i += THREADS) {
          const uint32_t k = sKey[i];
          const int j = sIdx[i], w = (j >> 5) - w0;
          if (k >= border.key && w >= 0 && w < words) atomicOr(over(k) ? &sOver[w] : &sSame[w], 1u << (j & 31));
        }
        for (int i = tid; i < p.sink + p.local; i += THREADS) {
          const int j = i < p.sink ? i : f - p.local + (i - p.sink), w = (j >> 5) - w0;
          if (w >= 0 && w < words) atomicOr(&sOver[w], 1u << (j & 31));
        }
      } else {
        __syncthreads();
        for (int w = warp * 4; w < words; w += THREADS / 8) {  // four words of a warp at once
          uint32_t k[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = (w0 + w + u) * 32 + lane;
            k[u] = w + u < words && j < f ? (f <= p.cap ? sKey[j] : in_row(j)) : 0u;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = (w0 + w + u) * 32 + lane;
            const uint32_t o = __ballot_sync(0xffffffffu, j < f && (over(k[u]) || forced(j)));
            const uint32_t s = __ballot_sync(0xffffffffu, j < f && !all_same && k[u] == border.key && !forced(j));
            if (lane == 0 && w + u < words) sOver[w + u] = o, sSame[w + u] = s;
          }
        }
      }
      __syncthreads();
      const int per = (words + THREADS - 1) / THREADS, first = tid * per, end = min(first + per, words);
      int mine = 0, mine_same = 0;
      for (int w = first; w < end; ++w) {
        mine += __popc(sOver[w]);
        mine_same += __popc(sSame[w]);
      }
      int total, total_same = 0;
      int before = have + block_scan<THREADS>(mine, sTmp, total) - mine, before_same = same;
      if (!all_same) before_same += block_scan<THREADS>(mine_same, sTmp, total_same) - mine_same;
      for (int w = first; w < end; ++w) {
        uint32_t o = sOver[w], any = o | sSame[w];
        while (any != 0u) {
          const int bit = __ffs(any) - 1;
          any &= any - 1;
          const bool is_over = (o >> bit) & 1;
          if (is_over || before_same < border.want)
            sList[before + (all_same ? 0 : min(before_same, border.want))] = (w0 + w) * 32 + bit;
          if (is_over) ++before; else ++before_same;
        }
      }
      have += total;
      same += total_same;
    }
    __syncthreads();
    list_slots<THREADS>(map, sList, p.top, tid);
  }
  __syncthreads();
  write_row<THREADS>(p, map, t, tid, sList, f, taken, seen);
}

// ---- the launch --------------------------------------------------------------------------

int64_t blocks_ld(int32_t P, int32_t page_size, int32_t block) {
  const int64_t n = int64_t(P) * (page_size / block);
  return (n + 31) / 32 * 32;
}

// Rows of a chunk: as many as kChunkBytes of scores hold, at least kMinChunkRows, and the
// chunks as equal as they can be.  (Chunks that stay in the 126 MB L2 between the kernels cost
// more in the ends of their launches than they save: 7,810 rows of 16,384 blocks took 583 us
// in chunks of 64 MB, 556 of 128, 527 of 192, 460 in one piece.)
int32_t chunk_rows(int32_t Tq, int64_t ld) {
  int64_t n = ld > 0 ? kChunkBytes / (ld * 4) : Tq;
  n = n < kMinChunkRows ? kMinChunkRows : n;
  if (ld > 0 && n * ld >= (1 << 30)) n = ((1 << 30) - 1) / ld;
  if (n < 1) return 0;
  const int64_t chunks = (int64_t(Tq) + n - 1) / n;
  return chunks > 0 ? int32_t((int64_t(Tq) + chunks - 1) / chunks) : 0;
}

template <int DI, int HP, int NT>
cudaError_t launch_score(SelectParams& p, int groups, int num_sms, cudaStream_t st) {
  using C = Score<DI, HP, NT>;
  const size_t smem = C::smem(groups);
  // (no allow_smem: with a limit that it does not need, the kernel was left less L1, and one row
  // over 65,535 blocks took 48 us in place of 28)
  static_assert((HP == 16 ? QSA_MAX_INDEX_HEADS / 16 : 1) * NT * (C::kSteps * 256 + 32) <= 48 * 1024,
                "within what every kernel may have");
  // as many blocks as the device holds, or as there are units at most
  const int rows = p.c1 - p.c0;
  const int64_t row_tiles = p.cu == nullptr ? rows : rows / C::kRows + (p.B < rows ? p.B : rows);
  const int64_t most = row_tiles * ((p.ld + kKeyTile - 1) / kKeyTile), all = int64_t(num_sms) * kScoreBlocks;
  return launch(qsa_select_score_kernel<DI, HP, NT>, unsigned(most < all ? most : all), kScoreThreads, smem, st, p,
                groups);
}

int heads_padded(int Hi) {
  int hp = 1;
  while (hp < Hi) hp *= 2;
  return hp;
}

// The tcgen05 form (a pair of rows within 64 columns: at most 32 heads) pays once a tile's 256
// columns are filled to more than a half on average.  16 sequences of 16,384 tokens, whole
// calls, the few-rows form against this one: 4 heads, 16 rows each 35 against 40 us, 32 rows
// 48 / 51, 64 rows 62 / 51, 128 rows 101 / 70; 16 heads, 8 rows 33 / 38, 16 rows 39 / 36.
// The average decides for all of a call's sequences, so the single rows among many long ones
// take a tile each; 33 to 64 heads always take the few-rows form.
bool use_wide(int32_t Tq, int32_t B, int32_t Hi, bool has_cu) {
  return has_cu && Hi <= 32 && int64_t(Tq) * heads_padded(Hi) * 2 > int64_t(B) * kWideCols;
}

int64_t wide_max_tiles(int32_t rows, int32_t B, int32_t Hi) {  // a sequence adds at most one partial tile
  return rows / (kWideCols / heads_padded(Hi)) + (B < rows ? B : rows);
}

template <int DI, int HP>
cudaError_t launch_prep(const SelectParams& p, int chunk_rows, int chunks, cudaStream_t st) {
  const dim3 grid(unsigned(wide_max_tiles(chunk_rows, p.B, p.Hi) * kPrepParts), unsigned(chunks));
  return launch(qsa_select_prep_kernel<DI, HP>, grid, 256, 0, st, p, chunk_rows);
}

std::atomic<uint32_t> g_wait_ns{kWaitLimit};  // see qsa_probe_select_wait_ns

template <int DI, int HP>
cudaError_t launch_wide(const SelectParams& p, int chunk, int chunk_rows, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> done[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(qsa_select_wide_kernel<DI, HP>), done);
  if (e != cudaSuccess) return e;
  const int64_t max_tiles = wide_max_tiles(chunk_rows, p.B, p.Hi);
  return launch(qsa_select_wide_kernel<DI, HP>, num_sms, kWideThreads, Wide<DI>::kSmem, st, p,
                static_cast<const int4*>(p.tiles + chunk * max_tiles),
                static_cast<const uint8_t*>(p.tile_q + chunk * max_tiles * wide_tile_bytes(DI)), int(max_tiles));
}

// prep: the tiles of all chunks (chunk < 0), or the scores of one chunk
template <int DI>
cudaError_t launch_wide_for(const SelectParams& p, int chunk, int chunk_rows, int chunks, int num_sms, cudaStream_t st) {
#define QSA_WIDE(HP)                                                       \
  case HP:                                                                 \
    return chunk < 0 ? launch_prep<DI, HP>(p, chunk_rows, chunks, st)      \
                     : launch_wide<DI, HP>(p, chunk, chunk_rows, num_sms, st);
  switch (heads_padded(p.Hi)) {
    QSA_WIDE(1)
    QSA_WIDE(2)
    QSA_WIDE(4)
    QSA_WIDE(8)
    QSA_WIDE(16)
    QSA_WIDE(32)
    default: return cudaErrorInvalidValue;
  }
#undef QSA_WIDE
}

// The narrowest tile that holds all heads of a row per thread: four rows (eight of one head).
template <int DI>
cudaError_t launch_score_for(SelectParams& p, int num_sms, cudaStream_t st) {
  if (p.Hi > 8) return launch_score<DI, 16, 8>(p, (p.Hi + 15) / 16, num_sms, st);
  if (p.Hi > 4) return launch_score<DI, 8, 4>(p, 1, num_sms, st);
  if (p.Hi > 2) return launch_score<DI, 4, 2>(p, 1, num_sms, st);
  if (p.Hi > 1) return launch_score<DI, 2, 1>(p, 1, num_sms, st);
  return launch_score<DI, 1, 1>(p, 1, num_sms, st);
}

template <int THREADS>
cudaError_t launch_choose_for(const SelectParams& p, size_t smem, cudaStream_t st) {
  static std::atomic<uint64_t> done[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(qsa_select_choose_kernel<THREADS>), done);
  if (e != cudaSuccess) return e;
  return launch(qsa_select_choose_kernel<THREADS>, p.c1 - p.c0, THREADS, smem, st, p);
}

cudaError_t launch_choose(SelectParams& p, int num_sms, cudaStream_t st) {
  const int rows = p.c1 - p.c0;
  // Short rows, a warp each, once there are enough of them: 600 rows of 2,048 blocks take 46 us
  // so and 41 by a block of 256 per row, 1,200 rows 47 and 47, 2,400 rows 54 and 64 (whole calls).
  if (p.ld <= kPickKeys && p.top <= kPickKeys && rows > 8 * num_sms) {
    p.cap = int((p.ld + 127) / 128 * 128);
    const size_t smem = size_t(kPickWarps) * p.cap * 4;
    static_assert(kPickWarps * (kPickKeys * 4 + sizeof(ChooseShared)) <= 48 * 1024, "within what every kernel may have");
    return launch(qsa_select_pick_kernel, (rows + kPickWarps - 1) / kPickWarps, 32 * kPickWarps, smem, st, p);
  }
  // Room for what the sample's border lets through of the longest row: the expected number and
  // five deviations (a row that does not fit is collected twice), within what a block can
  // have.
  const double share = double(p.ld) / kSample, hits = p.top / share;
  const double rank = hits + 4 * std::sqrt(hits) + 4, room = share * (rank + 5 * std::sqrt(rank));
  int want = p.top * 5 / 2 > 1536 ? p.top * 5 / 2 : 1536;
  want = room > want ? (room < 16384 ? int(room) : (want > 16384 ? want : 16384)) : want;
  p.cap = int(p.ld < want ? (p.ld < kSample ? kSample : p.ld) : want);
  p.cap = (p.cap + 127) / 128 * 128;
  p.window = p.ld / 32 < kWindow ? int(p.ld / 32) : kWindow;  // (ld is a multiple of 32)
  // Threads of a row: one row of 65,535 blocks takes 29 us with 1,024 and 73 with 256; 200 rows of
  // 8,192 blocks 87 and 76; 600 rows 183 with 256 and 191 with 128; 7,810 rows of 16,384 blocks
  // 490 and 436 (whole calls).
  const int threads = rows > 8 * num_sms ? 128 : rows > num_sms ? 256 : 1024;
  // a lane's queue: at least 24 entries (about 8 are expected of 128 lanes, fewer of more)
  p.queue = 2 * p.cap > 24 * threads ? 2 * p.cap / (2 * threads) * (2 * threads) : 24 * threads;
  const size_t keys = p.ld > p.cap ? size_t(p.cap > p.queue / 2 ? p.cap : p.queue / 2) + p.cap : size_t(p.cap);
  const size_t smem = keys * 4 + size_t(p.top + 3) / 4 * 16 + size_t(p.window) * 8;
  return threads == 128   ? launch_choose_for<128>(p, smem, st)
         : threads == 256 ? launch_choose_for<256>(p, smem, st)
                          : launch_choose_for<1024>(p, smem, st);
}

// The workspace: keys of a chunk of rows, then the tiles of all chunks.  Sized for the call
// with cu_q; one without it needs the keys alone.
struct SelectLayout {
  int64_t ld;
  int32_t rows, chunks;  // of a chunk; how many
  size_t tiles, tile_q, bytes;
};

SelectLayout select_layout(int32_t Tq, int32_t B, int32_t P, int32_t page_size, int32_t Hi, int32_t Di, int32_t block) {
  SelectLayout l{};
  l.ld = blocks_ld(P, page_size, block);
  l.rows = chunk_rows(Tq, l.ld);
  l.chunks = l.rows > 0 ? int32_t((int64_t(Tq) + l.rows - 1) / l.rows) : 0;
  l.tiles = (size_t(l.rows) * size_t(l.ld) * 4 + 255) / 256 * 256;
  l.tile_q = l.bytes = l.tiles;
  if (l.ld > 0 && use_wide(Tq, B, Hi, true)) {
    const size_t n = size_t(wide_max_tiles(l.rows, B, Hi)) * size_t(l.chunks);
    l.tile_q = l.tiles + (n * sizeof(int4) + 255) / 256 * 256;
    l.bytes = l.tile_q + n * wide_tile_bytes(Di);
  }
  return l;
}

qsa_status_t check_select_sizes(int32_t Tq, int32_t B, int32_t P, int32_t page_size, int32_t Hi, int32_t Di,
                                int32_t block) {
  if (Tq < 0 || B < 0 || P < 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "negative size: Tq=%d B=%d P=%d", Tq, B, P);
  if (block < 1 || block > kMaxBlock)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "block size %d outside 1..%d", block, kMaxBlock);
  if (page_size < 1 || page_size % block != 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "page_size=%d must be a positive multiple of block=%d", page_size, block);
  if (int64_t(P) * page_size > INT32_MAX - 4096)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "a page table of %lld tokens", (long long)(int64_t(P) * page_size));
  if (Di != 64 && Di != 128) QSA_REJECT(QSA_ERR_UNSUPPORTED, "index dimension %d (64 or 128)", Di);
  if (Hi < 1 || Hi > QSA_MAX_INDEX_HEADS)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "%d index heads (1..%d)", Hi, QSA_MAX_INDEX_HEADS);
  return QSA_OK;
}

}  // namespace

extern "C" uint32_t qsa_probe_select_wait_ns(uint32_t ns) { return g_wait_ns.exchange(ns); }

extern "C" size_t qsa_select_slots_workspace_bytes(int32_t Tq, int32_t B, int32_t P, int32_t page_size,
                                                   int32_t Hi, int32_t Di, int32_t block) {
  set_error_detail("%s", "");
  if (check_select_sizes(Tq, B, P, page_size, Hi, Di, block) != QSA_OK) return SIZE_MAX;
  return select_layout(Tq, B, P, page_size, Hi, Di, block).bytes;
}

extern "C" qsa_status_t qsa_select_slots(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const float* weight,
    int64_t weight_stride, const int8_t* codes, int64_t code_stride, const float* scales,
    const int32_t* page_table, int64_t page_stride, const int32_t* seq_lens, const int32_t* cu_q,
    int32_t Tq, int32_t B, int32_t P, int64_t pages, int32_t page_size, int32_t Hi, int32_t Di,
    int32_t block, int32_t top_blocks, int32_t sink_blocks, int32_t local_blocks, int32_t* slot_idx,
    int64_t idx_stride_t, int32_t* width, void* workspace, size_t workspace_bytes,
    uint32_t* err_word, void* stream) {
  set_error_detail("%s", "");
  const qsa_status_t sizes = check_select_sizes(Tq, B, P, page_size, Hi, Di, block);
  if (sizes != QSA_OK) return sizes;
  if (pages < 0 || pages * page_size > INT32_MAX)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "%lld pages of %d slots: slots are int32", (long long)pages, page_size);
  if (top_blocks < 1 || int64_t(top_blocks) * block > QSA_MAX_TOP_BLOCKS)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "top_blocks=%d of %d slots: 1..%d slots", top_blocks, block, QSA_MAX_TOP_BLOCKS);
  if (sink_blocks < 0 || local_blocks < 0 || int64_t(sink_blocks) + local_blocks > top_blocks)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "sink_blocks=%d + local_blocks=%d: 0..top_blocks=%d", sink_blocks,
               local_blocks, top_blocks);
  if (cu_q == nullptr && Tq != B)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "Tq=%d must be B=%d without cu_q", Tq, B);
  if (Tq == 0 || B == 0) return QSA_OK;
  if (q == nullptr || weight == nullptr || seq_lens == nullptr || slot_idx == nullptr || width == nullptr ||
      (P > 0 && (page_table == nullptr || (pages > 0 && (codes == nullptr || scales == nullptr)))))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL q, weight, codes, scales, page_table, seq_lens, slot_idx or width");
  if (!aligned_to(q, 16) || !aligned_to(codes, 16))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "q and codes must be 16-byte aligned");
  if (!aligned_to(weight, 4) || !aligned_to(scales, 4) || !aligned_to(page_table, 4) || !aligned_to(seq_lens, 4) ||
      !aligned_to(cu_q, 4) || !aligned_to(slot_idx, 4) || !aligned_to(width, 4) || !aligned_to(err_word, 4))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "4-byte tensors must be 4-byte aligned");
  if (!stride_multiple(q_stride_t, 2, 16) || !stride_multiple(q_stride_h, 2, 16) ||
      !stride_multiple(code_stride, 1, 16) || weight_stride < 0 || page_stride < 0 || idx_stride_t < 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "strides must be non-negative, of q and codes multiples of 16 bytes");
  const SelectLayout lay = select_layout(Tq, B, P, page_size, Hi, Di, block);
  const int64_t ld = lay.ld;
  const int32_t rows = lay.rows;
  const bool wide = use_wide(Tq, B, Hi, cu_q != nullptr);
  if (ld >= (1 << 30)) QSA_REJECT(QSA_ERR_UNSUPPORTED, "a page table of %lld blocks", (long long)ld);
  const size_t need = cu_q != nullptr ? lay.bytes : lay.tiles;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    QSA_REJECT(QSA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu", need,
               workspace == nullptr ? size_t(0) : workspace_bytes);
  if (!aligned_to(workspace, 256)) QSA_REJECT(QSA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  int dev = 0, num_sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return launch_status(e, "qsa_select_slots");

  SelectParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.weight = weight;
  p.codes = codes;
  p.scales = scales;
  p.table = page_table, p.lens = seq_lens, p.cu = cu_q;
  p.out = slot_idx, p.width = width;
  p.scores = static_cast<float*>(workspace);
  p.tiles = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + lay.tiles);
  p.tile_q = static_cast<uint8_t*>(workspace) + lay.tile_q;
  p.err_word = err_word;
  p.q_st = q_stride_t, p.q_sh = q_stride_h, p.w_st = weight_stride, p.code_st = code_stride;
  p.table_st = page_stride, p.out_st = idx_stride_t, p.pages = pages, p.ld = ld;
  p.Tq = Tq, p.B = B, p.P = P, p.page_size = page_size, p.per_page = page_size / block;
  p.Hi = Hi, p.block = block, p.top = top_blocks, p.sink = sink_blocks, p.local = local_blocks;
  const auto st = static_cast<cudaStream_t>(stream);
  p.page_magic = uint32_t(((uint64_t(1) << 32) + p.per_page - 1) / p.per_page);
  p.block_magic = uint32_t(((uint64_t(1) << 32) + block - 1) / block);
  p.first = ld <= top_blocks;
  const bool scored = !p.first;  // (a table of at most top_blocks blocks needs no scores)
  p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  auto wide_launch = [&](int chunk) {
    return Di == 128 ? launch_wide_for<128>(p, chunk, rows, lay.chunks, num_sms, st)
                     : launch_wide_for<64>(p, chunk, rows, lay.chunks, num_sms, st);
  };
  if (scored && wide) {
    if (lay.chunks > 65535) QSA_REJECT(QSA_ERR_UNSUPPORTED, "%d chunks of rows in one call", lay.chunks);
    if ((e = wide_launch(-1)) != cudaSuccess) return launch_status(e, "qsa_select_slots: query codes");
  }
  for (int32_t chunk = 0; chunk < lay.chunks; ++chunk) {
    const int64_t c0 = int64_t(chunk) * rows;
    p.c0 = int32_t(c0);
    p.c1 = int32_t(c0 + rows < Tq ? c0 + rows : Tq);
    if (scored && wide) p.late = &p.tiles[chunk * wide_max_tiles(rows, B, Hi)].z;
    if (scored) {
      e = wide ? wide_launch(chunk)
          : Di == 128 ? launch_score_for<128>(p, num_sms, st) : launch_score_for<64>(p, num_sms, st);
      if (e != cudaSuccess) return launch_status(e, "qsa_select_slots: score");
    }
    if ((e = launch_choose(p, num_sms, st)) != cudaSuccess) return launch_status(e, "qsa_select_slots: choice");
  }
  return QSA_OK;
}
