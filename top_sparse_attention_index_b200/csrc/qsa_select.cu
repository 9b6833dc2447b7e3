// qsa_select.cu -- the cheap score of every query row against the micro-blocks of its
// sequence and the choice of the row's slots.  Contract: include/qsa_layer.h
// (qsa_select_slots).
//
// Two kernels over chunks of rows: the score kernel writes an order-preserving 32-bit key
// per (row, block) into the workspace, the choice kernel finds each row's top_blocks-th
// largest key by radix passes and writes the slots of the blocks above it.  A chunk's keys
// are at most kChunkBytes, so they stay in the 126 MB L2 between the two kernels.
#include "qsa_layer.cuh"

namespace {

using namespace qsa;

constexpr int kKeyTile = 128;                 // micro-blocks per tile: 16 per warp
constexpr int kScoreThreads = 256;
constexpr int kChooseThreads = 512;
constexpr int64_t kChunkBytes = 64 << 20;     // keys of one chunk of rows
constexpr int kMinChunkRows = 64;

struct SelectParams {
  const uint16_t* q;
  const float* weight;
  const int8_t* codes;
  const float* scales;
  const int32_t *table, *lens, *cu;
  int32_t *out, *width;
  uint32_t* keys;      // [chunk rows, ld]
  uint32_t* err_word;
  int64_t q_st, q_sh, w_st, code_st, table_st, out_st, pages, ld;
  int32_t c0, c1;      // the chunk's rows
  int32_t Tq, B, P, page_size, per_page, Hi, block, top, sink, local;
  int32_t chunk_tiles, chunks;  // score kernel: key tiles of a thread block, blocks of a row tile
};

// The order of floats as an order of unsigned integers; NaN and -infinity share the lowest
// value a block can have, -0 equals +0.  0 is left for blocks of a page outside the pool,
// 0xffffffff for blocks that are taken whatever they score.
__device__ __forceinline__ uint32_t order_key(float s) {
  s = s != s ? -__builtin_huge_valf() : s + 0.0f;
  const uint32_t u = __float_as_uint(s);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Rows of sequence b, clamped to [0, Tq].
__device__ __forceinline__ int2 rows_of(const SelectParams& p, int b, bool report) {
  if (p.cu == nullptr) return make_int2(b, b + 1);
  int lo = p.cu[b], hi = p.cu[b + 1];
  if (report && p.err_word != nullptr && (lo < 0 || lo > p.Tq || hi < 0 || hi > p.Tq))
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

// ---- the score ---------------------------------------------------------------------------

// Columns of a tile: 8 NT of them, a thread of quad position u holding columns 2u and 2u + 1
// of every n8 tile: kPer = 2 NT columns, which are kPer / HP rows of HP heads each, so one
// thread holds all heads of a row (16 at a time) and adds them in order without crossing
// lanes.  Column c of an n8 tile i is (row u kPer/HP + x / HP, head x mod HP) with u = c / 2
// and x = 2 i + (c mod 2).  Heads beyond Hi, and rows beyond the tile's, have gain 0.
template <int DI, int HP, int NT>
struct Score {
  static constexpr int kCols = 8 * NT;
  static constexpr int kPer = 2 * NT;       // columns of a thread
  static constexpr int kRx = kPer / HP;     // rows of a thread
  static constexpr int kRows = 4 * kRx;     // rows of a tile
  static constexpr int kTileBytes = kKeyTile * DI;
  static_assert(kPer % HP == 0 && kRx >= 1, "a thread holds whole rows");
  // two key tiles, the query codes and gains, and per key tile the scales and valid marks
  static size_t smem(int groups) {
    return 2 * kTileBytes + size_t(groups) * kCols * (DI + 4) + 4 * kKeyTile * 4;
  }
};

template <int DI, int HP, int NT>
__global__ void __launch_bounds__(kScoreThreads) qsa_select_score_kernel(const SelectParams p, int groups) {
  using C = Score<DI, HP, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* sQ = smem + 2 * C::kTileBytes;
  float* sGain = reinterpret_cast<float*>(sQ + groups * C::kCols * DI);
  float* sScale = sGain + groups * C::kCols;                     // [2][kKeyTile]
  int* sValid = reinterpret_cast<int*>(sScale + 2 * kKeyTile);   // [2][kKeyTile]
  __shared__ int sTmp[kScoreThreads / 32], sFound[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- which rows -----------------------------------------------------------------------
  const int tile = blockIdx.x / p.chunks, kc = blockIdx.x % p.chunks;
  if (tid == 0) {
    sFound[0] = -1;
    if (p.cu == nullptr && p.c0 + tile < p.c1) sFound[0] = sFound[1] = p.c0 + tile, sFound[2] = 1;
  }
  __syncthreads();
  if (p.cu != nullptr) {
    int base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kScoreThreads) {
      int2 r = make_int2(0, 0);
      if (b0 + tid < p.B) r = rows_of(p, b0 + tid, false);
      r.x = max(r.x, p.c0);
      r.y = min(r.y, p.c1);
      const int mine = r.y > r.x ? (r.y - r.x + C::kRows - 1) / C::kRows : 0;
      int total;
      const int before = base + block_scan<kScoreThreads>(mine, sTmp, total) - mine;
      if (tile >= before && tile < before + mine) {
        const int t0 = r.x + (tile - before) * C::kRows;
        sFound[0] = b0 + tid, sFound[1] = t0, sFound[2] = min(C::kRows, r.y - t0);
      }
      base += total;
      __syncthreads();
      if (tile < base) break;
    }
  }
  const int b = sFound[0];
  if (b < 0) return;
  const int t0 = sFound[1], n = sFound[2];
  // row t sees len - (last - t) tokens
  const int last = rows_of(p, b, false).y - 1, len = length_of(p, b, false);
  const int f_most = max(len - (last - (t0 + n - 1)), 0) / p.block;
  if (f_most <= p.top) return;  // every row of the tile takes all its blocks
  const int k0 = kc * p.chunk_tiles * kKeyTile, k1 = min(k0 + p.chunk_tiles * kKeyTile, f_most);
  if (k0 >= k1) return;

  const uint32_t key_s = smem_addr(smem), q_s = smem_addr(sQ);
  // 16-byte chunk c of row r lies at chunk c ^ (r mod 8) of the row (64-byte rows:
  // c ^ (r / 2 mod 4)), so the 8 rows of a matrix fall into different banks.
  auto swz = [](int r, int c) { return DI == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3); };
  auto load_tile = [&](int kt, int buf) {
    const int r = tid >> 1, j = k0 + kt * kKeyTile + r;
    bool ok = false;
    int64_t phys = 0;
    if (j < k1) {
      const int m = j / p.per_page;
      const int page = __ldg(p.table + b * p.table_st + m);
      ok = page >= 0 && page < p.pages;
      if (!ok && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      phys = ok ? int64_t(page) * p.per_page + (j - m * p.per_page) : 0;
    }
    const int8_t* src = p.codes + phys * p.code_st;
#pragma unroll
    for (int i = 0; i < DI / 32; ++i) {
      const int c = (tid & 1) * (DI / 32) + i;
      cp_async_16(key_s + buf * C::kTileBytes + r * DI + (swz(r, c) << 4), ok ? src + c * 16 : p.codes, ok);
    }
    if ((tid & 1) == 0) {
      sScale[buf * kKeyTile + r] = ok ? __ldg(p.scales + phys) : 0.f;
      sValid[buf * kKeyTile + r] = ok;
    }
  };
  load_tile(0, 0);
  cp_async_commit();

  // ---- the rows' codes and gains ----------------------------------------------------------
  {
    constexpr int kLanes = DI / 8, kVec = 32 / kLanes;  // lanes of a vector, vectors of a warp
    const int l = lane % kLanes;
    for (int v0 = warp * kVec; v0 < groups * C::kCols; v0 += (kScoreThreads / 32) * kVec) {
      const int v = v0 + lane / kLanes;  // (kCols is a multiple of kVec)
      const int g = v / C::kCols, c = v % C::kCols;
      const int x = (c >> 3) * 2 + (c & 1);
      const int row = ((c & 7) >> 1) * C::kRx + x / HP, head = g * 16 + x % HP;
      const bool live = row < n && head < p.Hi;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (live)
        raw = *reinterpret_cast<const uint4*>(p.q + (t0 + row) * p.q_st + head * p.q_sh + l * 8);
      float xs[8], top = 0.f;
      bf16x8_to_f32(raw, xs);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = nan_max(top, fabsf(xs[e]));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = nan_max(top, __shfl_xor_sync(0xffffffffu, top, o));
      float scale = __fdiv_rn(top, 127.f);
      if (!(scale < __builtin_huge_valf())) scale = __int_as_float(0x7fffffff);
      *reinterpret_cast<uint2*>(sQ + v * DI + (swz(c, l >> 1) << 4) + (l & 1) * 8) = int8x8_codes(xs, scale);
      if (l == 0) sGain[v] = live ? __fmul_rn(p.weight[(t0 + row) * p.w_st + head], scale) : 0.f;
    }
  }

  const int tiles = (k1 - k0 + kKeyTile - 1) / kKeyTile;
  const int u = lane & 3;
  for (int kt = 0; kt < tiles; ++kt) {
    const int buf = kt & 1;
    cp_async_wait<0>();
    __syncthreads();  // the tile has landed, and nothing reads the other buffer any more
    if (kt + 1 < tiles) {
      load_tile(kt + 1, buf ^ 1);
      cp_async_commit();
    }
    uint32_t a[DI / 32][4];
#pragma unroll
    for (int ks = 0; ks < DI / 32; ++ks) {
      const int r = warp * 16 + (lane & 15);
      ldmatrix_x4(a[ks], key_s + buf * C::kTileBytes + r * DI + (swz(r, ks * 2 + (lane >> 4)) << 4));
    }
    float sum[C::kRx][2];  // [row of the thread][key lane / 4, key lane / 4 + 8]
    for (int g = 0; g < groups; ++g) {
      int acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0;
#pragma unroll
      for (int ks = 0; ks < DI / 32; ++ks) {
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          // four matrices: both 16-byte halves of tile i, then of tile i + 1 (NT = 1: tile 0 again)
          const int c = (NT > 1 ? i + (lane >> 4) : i) * 8 + (lane & 7);
          uint32_t bq[4];
          ldmatrix_x4(bq, q_s + (g * C::kCols + c) * DI + (swz(c, ks * 2 + ((lane >> 3) & 1)) << 4));
          mma_s8_16832(acc[i], a[ks], bq[0], bq[1]);
          if constexpr (NT > 1) mma_s8_16832(acc[i + 1], a[ks], bq[2], bq[3]);
        }
      }
#pragma unroll
      for (int x = 0; x < C::kPer; ++x) {
        const float gain = sGain[g * C::kCols + (x >> 1) * 8 + 2 * u + (x & 1)];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (a dot of 128 codes is below 2^24: exact)
          const float term = __fmul_rn(gain, float(max(acc[x >> 1][h * 2 + (x & 1)], 0)));
          float& s = sum[x / HP][h];
          s = (x % HP == 0 && g == 0) ? term : __fadd_rn(s, term);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = warp * 16 + (lane >> 2) + 8 * h, j = k0 + kt * kKeyTile + r;
      const float scale = sScale[buf * kKeyTile + r];
      const bool ok = sValid[buf * kKeyTile + r] != 0;
#pragma unroll
      for (int i = 0; i < C::kRx; ++i) {
        const int t = t0 + u * C::kRx + i;
        if (t < t0 + n && j < (len - (last - t)) / p.block)
          p.keys[(t - p.c0) * p.ld + j] = ok ? order_key(__fmul_rn(sum[i][h], scale)) : 0u;
      }
    }
  }
}

// ---- the choice --------------------------------------------------------------------------

// One thread block per row.  Three radix passes over the row's keys (11, 11 and 10 bits,
// highest first) find the key of the top-th block and how many blocks of exactly that key
// belong to it; a scan in block order then collects the taken blocks.
__global__ void __launch_bounds__(kChooseThreads) qsa_select_choose_kernel(const SelectParams p) {
  extern __shared__ int sList[];  // [min(top, blocks)] first physical slot of each taken block, or -1
  __shared__ int sHist[2048];
  __shared__ int sTmp[kChooseThreads / 32], sPick[2], sSeq;
  const int tid = threadIdx.x;
  const int t = p.c0 + blockIdx.x;
  if (tid == 0) sSeq = (p.cu == nullptr && t < p.B) ? t : -1;
  __syncthreads();
  if (p.cu != nullptr)
    for (int i = tid; i < p.B; i += kChooseThreads) {
      const int2 r = rows_of(p, i, blockIdx.x == 0 && p.c0 == 0);
      if (t >= r.x && t < r.y) atomicMax(&sSeq, i);  // (offsets that overlap: the last one)
    }
  __syncthreads();
  const int b = sSeq;
  if (b < 0) return;
  const int last = rows_of(p, b, false).y - 1, len = length_of(p, b, tid == 0);
  const int seen = max(len - (last - t), 0);
  const int f = seen / p.block, taken = min(f, p.top);
  const uint32_t* row = p.keys + blockIdx.x * p.ld;
  auto first_slot = [&](int j) {  // of block j, or -1
    const int m = j / p.per_page;
    const int page = __ldg(p.table + b * p.table_st + m);
    if (page < 0 || page >= p.pages) {
      if (p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      return -1;
    }
    return page * p.page_size + (j - m * p.per_page) * p.block;
  };
  if (f <= p.top) {
    for (int j = tid; j < f; j += kChooseThreads) sList[j] = first_slot(j);
  } else {
    auto key_of = [&](int j) { return (j < p.sink || j >= f - p.local) ? 0xffffffffu : row[j]; };
    uint32_t prefix = 0, mask = 0;
    int want = p.top;  // blocks still to be found among the keys that match the prefix
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 0x3ffu : 0x7ffu;
      for (int i = tid; i < 2048; i += kChooseThreads) sHist[i] = 0;
      __syncthreads();
      for (int j = tid; j < f; j += kChooseThreads) {
        const uint32_t k = key_of(j);
        if ((k & mask) == prefix) atomicAdd(&sHist[(k >> shift) & digit], 1);
      }
      __syncthreads();
      // thread i owns the bins 2047 - 4 i down to 2044 - 4 i: the scan runs from the top
      int c[4], mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) mine += c[e] = sHist[2047 - 4 * tid - e];
      int total;
      int above = block_scan<kChooseThreads>(mine, sTmp, total) - mine;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (above < want && above + c[e] >= want) sPick[0] = 2047 - 4 * tid - e, sPick[1] = want - above;
        above += c[e];
      }
      __syncthreads();
      prefix |= uint32_t(sPick[0]) << shift;
      mask |= digit << shift;
      want = sPick[1];
      __syncthreads();
    }
    // blocks above `prefix` are taken, and the first `want` that equal it
    int have = 0, same = 0;
    for (int j0 = 0; j0 < f; j0 += kChooseThreads) {
      const int j = j0 + tid;
      const uint32_t k = j < f ? key_of(j) : 0u;
      const bool over = j < f && k > prefix, equal = j < f && k == prefix;
      int total;
      const int incl = block_scan<kChooseThreads>((over ? 1 : 0) | (equal ? 1 << 16 : 0), sTmp, total);
      const int ties = same + (incl >> 16) - (equal ? 1 : 0);  // equal ones before this block
      if (over || (equal && ties < want)) {
        const int at = have + (incl & 0xffff) - (over ? 1 : 0) + min(ties, want);
        sList[at] = first_slot(j);
      }
      have += total & 0xffff;
      same += total >> 16;
    }
  }
  __syncthreads();
  int32_t* out = p.out + t * p.out_st;
  const int W = p.top * p.block + p.block - 1, full = taken * p.block, tail = seen - f * p.block;
  const int tail_slot = tail > 0 ? first_slot(f) : -1;
  for (int w = tid; w < W; w += kChooseThreads) {
    int s = -1;
    if (w < full) {
      const int i = w / p.block;
      s = sList[i] < 0 ? -1 : sList[i] + (w - i * p.block);
    } else if (w < full + tail) {
      s = tail_slot < 0 ? -1 : tail_slot + (w - full);
    }
    out[w] = s;
  }
  if (tid == 0) p.width[t] = full + tail;
}

// ---- the launch --------------------------------------------------------------------------

int64_t blocks_ld(int32_t P, int32_t page_size, int32_t block) {
  const int64_t n = int64_t(P) * (page_size / block);
  return (n + 31) / 32 * 32;
}

// Rows of a chunk: as many as kChunkBytes of keys hold, at least kMinChunkRows.
int32_t chunk_rows(int32_t Tq, int64_t ld) {
  int64_t n = ld > 0 ? kChunkBytes / (ld * 4) : Tq;
  n = n < kMinChunkRows ? kMinChunkRows : n;
  return int32_t(n < Tq ? n : Tq);
}

template <int DI, int HP, int NT>
cudaError_t launch_score(SelectParams& p, int groups, int num_sms, cudaStream_t st) {
  using C = Score<DI, HP, NT>;
  const size_t smem = C::smem(groups);
  cudaError_t e = cudaFuncSetAttribute(qsa_select_score_kernel<DI, HP, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int rows = p.c1 - p.c0;
  // a sequence adds at most one partial tile
  const int64_t row_tiles = p.cu == nullptr ? rows : rows / C::kRows + (p.B < rows ? p.B : rows);
  const int64_t key_tiles = (p.ld + kKeyTile - 1) / kKeyTile;
  // up to 8 key tiles to a thread block, fewer while the blocks do not fill the device twice
  int64_t per = row_tiles * key_tiles / (4 * int64_t(num_sms));
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  p.chunk_tiles = int32_t(per);
  p.chunks = int32_t((key_tiles + per - 1) / per);
  if (row_tiles * p.chunks > INT32_MAX) return cudaErrorInvalidConfiguration;
  qsa_select_score_kernel<DI, HP, NT><<<unsigned(row_tiles * p.chunks), kScoreThreads, smem, st>>>(p, groups);
  return cudaGetLastError();
}

// One row per sequence fills a tile of four rows at most: the narrowest tile that holds all
// heads.  Otherwise 64 columns.
template <int DI>
cudaError_t launch_score_for(SelectParams& p, int num_sms, cudaStream_t st) {
  const bool narrow = p.cu == nullptr || p.Tq <= 4 * p.B;
  const int groups = p.Hi > 16 ? (p.Hi + 15) / 16 : 1;
  if (p.Hi > 8) return launch_score<DI, 16, 8>(p, groups, num_sms, st);
  if (p.Hi > 4) return narrow ? launch_score<DI, 8, 4>(p, 1, num_sms, st) : launch_score<DI, 8, 8>(p, 1, num_sms, st);
  if (p.Hi > 2) return narrow ? launch_score<DI, 4, 2>(p, 1, num_sms, st) : launch_score<DI, 4, 8>(p, 1, num_sms, st);
  if (p.Hi > 1) return narrow ? launch_score<DI, 2, 1>(p, 1, num_sms, st) : launch_score<DI, 2, 8>(p, 1, num_sms, st);
  return narrow ? launch_score<DI, 1, 1>(p, 1, num_sms, st) : launch_score<DI, 1, 8>(p, 1, num_sms, st);
}

qsa_status_t check_select_sizes(int32_t Tq, int32_t B, int32_t P, int32_t page_size, int32_t block) {
  if (Tq < 0 || B < 0 || P < 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "negative size: Tq=%d B=%d P=%d", Tq, B, P);
  if (block < 1 || block > kMaxBlock)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "block size %d outside 1..%d", block, kMaxBlock);
  if (page_size < 1 || page_size % block != 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "page_size=%d must be a positive multiple of block=%d", page_size, block);
  if (int64_t(P) * page_size > INT32_MAX - 4096)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "a page table of %lld tokens", (long long)(int64_t(P) * page_size));
  return QSA_OK;
}

}  // namespace

extern "C" size_t qsa_select_slots_workspace_bytes(int32_t Tq, int32_t B, int32_t P,
                                                   int32_t page_size, int32_t block) {
  set_error_detail("%s", "");
  if (check_select_sizes(Tq, B, P, page_size, block) != QSA_OK) return SIZE_MAX;
  const int64_t ld = blocks_ld(P, page_size, block);
  return size_t(chunk_rows(Tq, ld)) * size_t(ld) * 4;
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
  const qsa_status_t sizes = check_select_sizes(Tq, B, P, page_size, block);
  if (sizes != QSA_OK) return sizes;
  if (pages < 0 || pages * page_size > INT32_MAX)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "%lld pages of %d slots: slots are int32", (long long)pages, page_size);
  if (Di != 64 && Di != 128) QSA_REJECT(QSA_ERR_UNSUPPORTED, "index dimension %d (64 or 128)", Di);
  if (Hi < 1 || Hi > QSA_MAX_INDEX_HEADS)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "%d index heads (1..%d)", Hi, QSA_MAX_INDEX_HEADS);
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
  const int64_t ld = blocks_ld(P, page_size, block);
  const int32_t rows = chunk_rows(Tq, ld);
  const size_t need = size_t(rows) * size_t(ld) * 4;
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
  p.keys = static_cast<uint32_t*>(workspace);
  p.err_word = err_word;
  p.q_st = q_stride_t, p.q_sh = q_stride_h, p.w_st = weight_stride, p.code_st = code_stride;
  p.table_st = page_stride, p.out_st = idx_stride_t, p.pages = pages, p.ld = ld;
  p.Tq = Tq, p.B = B, p.P = P, p.page_size = page_size, p.per_page = page_size / block;
  p.Hi = Hi, p.block = block, p.top = top_blocks, p.sink = sink_blocks, p.local = local_blocks;
  const auto st = static_cast<cudaStream_t>(stream);
  const size_t list = size_t(top_blocks) * 4;
  for (int64_t c0 = 0; c0 < Tq; c0 += rows) {
    p.c0 = int32_t(c0);
    p.c1 = int32_t(c0 + rows < Tq ? c0 + rows : Tq);
    if (ld > top_blocks) {  // (a table of at most top_blocks blocks needs no scores)
      e = Di == 128 ? launch_score_for<128>(p, num_sms, st) : launch_score_for<64>(p, num_sms, st);
      if (e != cudaSuccess) return launch_status(e, "qsa_select_slots: score");
    }
    qsa_select_choose_kernel<<<p.c1 - p.c0, kChooseThreads, list, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return launch_status(e, "qsa_select_slots: choice");
  }
  return QSA_OK;
}
