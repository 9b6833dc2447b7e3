// qsa_decode.cu -- attention of one new token per sequence over its whole paged cache, split
// over the cache's length and joined.  Contract: include/qsa_layer.h (qsa_paged_decode).
#include "qsa_layer.cuh"

namespace {

using namespace qsa;

constexpr int kD = kHeadDim;
constexpr int kStages = 2;
constexpr int kSub = 16;                 // slots of a warp's sub-tile (the M of one MMA)
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kRescaleLog2 = 8.0f;

struct DecodeParams {
  const uint16_t* q;
  const uint8_t *k, *v;
  const int32_t *table, *lens;
  uint16_t* out;
  float *lse, *ws_o, *ws_lse;  // ws_o [blocks, 2, G, D], ws_lse [blocks, 2, G]
  uint32_t* err_word;
  int64_t q_sb, q_sh, o_sb, o_sh, table_st, pages;
  uint32_t k_ss, v_ss;  // bytes
  int64_t k_sh, v_sh;   // bytes
  int32_t B, Hq, Hkv, G, P, page_size;
  int32_t unit, unit_log2;  // slots that the work is shared out in: a sub-tile for each warp of a block
  uint32_t page_magic;  // 2^32 / page_size, rounded up
  float scale_log2, v_scale;
};

// The larger one, or a NaN if either is one: fmaxf drops it, and where every other score of a
// piece is masked the piece then counts as empty.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float x;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(a), "f"(b));
  return x;
}

__device__ __forceinline__ int tokens_of(const DecodeParams& p, int b, bool report) {
  const int64_t most = int64_t(p.P) * p.page_size;
  const int n = p.lens[b];
  if (report && p.err_word != nullptr && (n < 0 || n > most)) atomicOr(p.err_word, QSA_ERRBIT_WIDTH_RANGE);
  return int(min(int64_t(max(n, 0)), most));
}

__device__ __forceinline__ int units_of(const DecodeParams& p, int len) { return (len + p.unit - 1) >> p.unit_log2; }

// The work: the units of all sequences in order, cut into `groups` shares whose sizes differ
// by one at most.  Group c's Hkv thread blocks take the same share of one KV head each, side
// by side in time: the heads' rows of a slot are neighbours in memory.
struct Share {
  int64_t each, longer;  // units of a share; the first `longer` shares have one more
  int32_t groups;        // shares that hold units
  __device__ int64_t begin(int64_t c) const { return c * each + (c < longer ? c : longer); }
  __device__ int32_t owner(int64_t unit) const {  // the share that has this unit
    const int64_t in_longer = longer * (each + 1);
    return int32_t(unit < in_longer ? quotient(unit, each + 1) : longer + quotient(unit - in_longer, each));
  }
  static __device__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
  }
};

__device__ __forceinline__ Share share_of(int64_t total, int groups) {
  Share s{0, 0, int32_t(total < groups ? total : groups)};
  if (s.groups > 0) {
    s.each = Share::quotient(total, s.groups);
    s.longer = total - s.each * s.groups;
  }
  return s;
}

// Units of all sequences and of those before sequence `b`; by every warp for itself.
__device__ __forceinline__ int64_t units_before(const DecodeParams& p, int b, int64_t& all, bool report) {
  int64_t mine = 0, before = 0;
  for (int i = threadIdx.x & 31; i < p.B; i += 32) {
    const int n = units_of(p, tokens_of(p, i, report));
    mine += n;
    before += i < b ? n : 0;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    mine += __shfl_xor_sync(0xffffffffu, mine, d);
    before += __shfl_xor_sync(0xffffffffu, before, d);
  }
  all = mine;
  return before;
}

// NT n8 tiles hold the G heads of a KV head.  Rows in shared memory are padded by 16 bytes,
// so the eight rows that one 8x8 matrix load touches fall into different banks.
template <bool FP8, int NT>
struct Decode {
  // Of E4M3 rows twice as many are in flight, and twice the warps work on them (4 x 262,144
  // tokens: 203 us with two warps to a block, 192 with four; with bf16 rows four warps leave
  // an SM one block instead of three: 64 ragged sequences 130 us, 118 with two).
  static constexpr int kWarps = FP8 ? 4 : 2;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRow = FP8 ? kD : 2 * kD;  // bytes of a cache row
  static constexpr int kPitch = kRow + 16;
  static constexpr int kStageBytes = 2 * kSub * kPitch;  // K rows, then V rows
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kQPitch = 2 * kD + 16;
  static constexpr int kQBytes = NT * 8 * kQPitch;
  static constexpr int kMergePitch = kD + 4;
  // What log2 of the weights is raised by: 16-bit floats have their smallest step at 2^-24, and a
  // weight of 2^-25 of the largest or less would vanish, 262,144 of which hold 2^-7 of the sum.  The
  // largest weight, 2^(kRescaleLog2 + 7) = 2^15, is still one of them (below 65,504).
  static constexpr float kRaise = FP8 ? 7.f : 0.f;
  static constexpr size_t kSmem = kRing + kQBytes;
  static constexpr int kMergeBytes = kWarps * NT * 8 * kMergePitch * 4;
  // thread blocks of an SM: 228 KB of shared memory, 1 KB of each block reserved
  static constexpr int kResident = (228 * 1024) / (int(kSmem) + 1024 + 512);
  static_assert(kMergeBytes <= int(kSmem), "the merge buffer reuses the ring and the Q rows");
};

// The units of all sequences are shared out evenly over the thread blocks that the device
// holds at once, whatever the lengths (64 ragged sequences: 111 us; split evenly by the page
// table's capacity, 157); a sequence that one block holds whole is written to the
// output, a piece of one to the block's record (its first piece to record 0, its last to
// record 1: pieces between them are whole sequences).
// Within a block each warp takes its 16-slot sub-tiles of a unit and runs a pipeline of its
// own: asynchronous copies into a stage while it works on the other, no block-wide barrier
// in the loop.  Scores are S^T = K Q^T with the slots as M and the heads as N, so the group
// shares every row that is read; the softmax is online (base 2, the reference moves only when
// the maximum rises by more than 2^8); P is rounded to 16 bits (bf16, or f16 raised by 2^7 for
// E4M3) for O^T += V^T P^T, and the denominator sums the same rounded values.  The bound is HBM: every row is read once.
// 64 sequences of up to 8,192 tokens, 24 + 2 heads: 605 MB in 111 us, 0.84 of the copy rate
// (and 8 us for the join); 4 of 262,144 tokens in E4M3: 1.07 GB in 182 us, 0.91.
template <bool FP8, int NT>
__global__ void __launch_bounds__(Decode<FP8, NT>::kThreads) qsa_paged_decode_kernel(const DecodeParams p) {
  using C = Decode<FP8, NT>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 sState[kWarps][NT * 8];  // (m, l) of each warp and head
  uint8_t* sQ = smem + C::kRing;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  begin_kernel();
  int64_t total;
  units_before(p, 0, total, blockIdx.x == 0 && warp == 0);
  // sequences without a token: zeros
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (tokens_of(p, b, false) > 0) continue;
    for (int i = tid; i < p.Hq * (kD / 8); i += kThreads)
      *reinterpret_cast<uint4*>(p.out + b * p.o_sb + (i / (kD / 8)) * p.o_sh + (i % (kD / 8)) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int h = tid; h < p.Hq; h += kThreads) p.lse[int64_t(b) * p.Hq + h] = kNegInf;
  }
  const int groups = int(gridDim.x) / p.Hkv, group = int(blockIdx.x) / p.Hkv, j = int(blockIdx.x) - group * p.Hkv;
  const Share share = share_of(total, groups);
  if (group >= share.groups) return;
  const int64_t u0 = share.begin(group), u1 = share.begin(group + 1);
  // the sequence of unit u0: every warp searches for itself, 32 sequences at a time
  int b = 0;
  int64_t seg0 = 0;  // its first unit
  for (;; b += 32) {
    const int64_t n = b + lane < p.B ? int64_t(units_of(p, tokens_of(p, b + lane, false))) : 0;
    int64_t to = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, seg0 + to > u0);
    if (past != 0u) {
      const int l = __ffs(past) - 1;
      seg0 += __shfl_sync(0xffffffffu, to - n, l);
      b += l;
      break;
    }
    seg0 += __shfl_sync(0xffffffffu, to, 31);
  }
  int len = tokens_of(p, b, false), units = units_of(p, len);

  const uint32_t ring = smem_addr(smem) + warp * kStages * C::kStageBytes;
  const uint32_t q_s = smem_addr(sQ);
  const int g8 = lane >> 2, t4 = lane & 3;
  int stage = 0;
  for (int64_t u = u0; u < u1;) {
  const int64_t seg1 = seg0 + units, end = min(seg1, u1);
  const int s0 = int(u - seg0) * p.unit, s1 = int(min(int64_t(len), (end - seg0) * p.unit));
  const int h0 = j * p.G;
  const uint8_t* kg = p.k + j * p.k_sh;
  const uint8_t* vg = p.v + j * p.v_sh;
  const int subs = (s1 - s0 + kSub - 1) / kSub;  // sub-tiles of the piece; warp w takes w, w + kWarps, ...
  uint32_t valid[kStages];                       // one bit per slot of the stage's sub-tile

  // The sub-tile's rows, 16 bytes per lane and copy: a row is kRow / 16 lanes.  Lane r looks up
  // slot r; rows past the end or in a page outside the pool are not read, and become zeros.
  // (One bulk copy per row, issued by its own lane, cost more instructions than everything
  // else here: 226 us for 1.07 GB of E4M3 rows, 203 with these copies and two warps.)
  constexpr int kRowLanes = C::kRow / 16, kRows = 32 / kRowLanes;  // lanes of a row, rows of a copy
  const uint8_t* kl = kg + (lane % kRowLanes) * 16;
  const uint8_t* vl = vg + (lane % kRowLanes) * 16;
  const uint32_t to_lane = ring + (lane / kRowLanes) * C::kPitch + (lane % kRowLanes) * 16;
  auto issue = [&](int sub, int to) -> uint32_t {
    const int i = s0 + sub * kSub + (lane & 15);
    bool ok = i < s1;
    int slot = 0;
    if (ok) {
      int m = i;
      if (p.page_size > 1) {
        m = __umulhi(uint32_t(i), p.page_magic);  // i / page_size, or one more
        if (int64_t(m) * p.page_size > i) --m;
      }
      const int page = p.table[b * p.table_st + m];
      ok = page >= 0 && page < p.pages;
      if (!ok && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      slot = ok ? page * p.page_size + (i - m * p.page_size) : 0;
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
    const uint32_t dst = to_lane + to * C::kStageBytes;
#pragma unroll
    for (int r = 0; r < kSub; r += kRows) {
      const int row = r + lane / kRowLanes;
      const uint32_t from = uint32_t(__shfl_sync(0xffffffffu, slot, row));
      const bool there = (mask >> row) & 1;
      cp_async_16(dst + r * C::kPitch, kl + uint64_t(from) * p.k_ss, there);
      cp_async_16(dst + (kSub + r) * C::kPitch, vl + uint64_t(from) * p.v_ss, there);
    }
    return mask;
  };
  valid[0] = valid[1] = 0;
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    if (warp + s * kWarps < subs) {
      const uint32_t mk = issue(warp + s * kWarps, stage ^ s);
      if ((stage ^ s) == 0) valid[0] = mk; else valid[1] = mk;
    }
    cp_async_commit();
  }

  // ---- Q: bf16 rows, or f16 for an E4M3 cache (its codes are exact in f16) -----------------
  for (int i = tid; i < NT * 8 * (kD / 8); i += kThreads) {
    const int g = i / (kD / 8), c = i % (kD / 8);
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (g < p.G) raw = *reinterpret_cast<const uint4*>(p.q + b * p.q_sb + (h0 + g) * p.q_sh + c * 8);
    if constexpr (FP8) {
      float x[8];
      bf16x8_to_f32(raw, x);
      bool big = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) big |= fabsf(x[e]) >= 65536.f;
      if (big && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_Q_RANGE);
      // K's fragments have codes 4 t .. 4 t + 3 of 16 where the MMA has k = 2 t, 2 t + 1, 2 t + 8,
      // 2 t + 9: the same order for Q (c is half of 16 dimensions)
      uint8_t* dst = sQ + g * C::kQPitch + (c >> 1) * 32 + (c & 1) * 8;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_f16x2(x[0], x[1]), pack_f16x2(x[4], x[5]));
      *reinterpret_cast<uint2*>(dst + 16) = make_uint2(pack_f16x2(x[2], x[3]), pack_f16x2(x[6], x[7]));
    } else {
      *reinterpret_cast<uint4*>(sQ + g * C::kQPitch + c * 16) = raw;
    }
  }
  __syncthreads();

  float o[NT][16][4];  // O^T: 16 m-tiles of 16 dimensions
  float l[NT][4];      // P's sums over the slots: an m-tile whose A is all ones
  float m_ref[NT][2];  // a maximum less kRaise; moves when one is more than kMove above it
  constexpr float kMove = kRescaleLog2 + C::kRaise;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m_ref[n][0] = m_ref[n][1] = kNegInf;
    l[n][0] = l[n][1] = l[n][2] = l[n][3] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
  }

  for (int sub = warp; sub < subs; sub += kWarps) {
    const uint32_t kbuf = ring + stage * C::kStageBytes, vbuf = kbuf + kSub * C::kPitch;
    const uint32_t mask = stage == 0 ? valid[0] : valid[1];
    cp_async_wait<kStages - 1>();
    __syncwarp();

    // ---- S^T = K Q^T: two accumulators per n8 tile keep two chains in flight ---------------
    float s[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) s[n][c][0] = s[n][c][1] = s[n][c][2] = s[n][c][3] = 0.f;
    const uint32_t krow = kbuf + (lane & 15) * C::kPitch + (lane >> 4) * 16;
#pragma unroll
    for (int kp = 0; kp < 8; ++kp) {  // two 16-wide k-steps
      uint32_t b[NT][2][2], a[2][4];  // Q [tile][step], K [step]
      if constexpr (NT == 1) {
        uint32_t r[4];
        ldmatrix_x4(r, q_s + (lane & 7) * C::kQPitch + kp * 64 + (lane >> 3) * 16);
        b[0][0][0] = r[0], b[0][0][1] = r[1], b[0][1][0] = r[2], b[0][1][1] = r[3];
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t r[4];
          ldmatrix_x4(r, q_s + ((lane >> 4) * 8 + (lane & 7)) * C::kQPitch + (kp * 2 + e) * 32 + ((lane >> 3) & 1) * 16);
          b[0][e][0] = r[0], b[0][e][1] = r[1], b[NT - 1][e][0] = r[2], b[NT - 1][e][1] = r[3];
        }
      }
      if constexpr (!FP8) {
        ldmatrix_x4(a[0], krow + kp * 64);
        ldmatrix_x4(a[1], krow + kp * 64 + 32);
      } else {
        uint32_t r[4];
        ldmatrix_x4(r, krow + kp * 32);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          e4m3x4_to_f16x2x2(r[2 * e], a[e][0], a[e][2]);
          e4m3x4_to_f16x2x2(r[2 * e + 1], a[e][1], a[e][3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (FP8) mma_f16_16816(s[n][e], a[e], b[n][e][0], b[n][e][1]);
          else mma_bf16_16816(s[n][e], a[e], b[n][e][0], b[n][e][1]);
        }
    }

    // ---- softmax over the sub-tile's slots (rows g8 and g8 + 8) ------------------------------
    float x[NT][4], top[NT][2];
    bool rises = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] = (s[n][0][e] + s[n][1][e]) * p.scale_log2;
      if (mask != 0xffffu) {
        if (!((mask >> g8) & 1)) x[n][0] = x[n][1] = kNegInf;
        if (!((mask >> (g8 + 8)) & 1)) x[n][2] = x[n][3] = kNegInf;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[n][c] = max_or_nan(x[n][c], x[n][c + 2]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top[n][c] = max_or_nan(top[n][c], __shfl_xor_sync(0xffffffffu, top[n][c], d));
        rises |= top[n][c] > m_ref[n][c] + kMove || m_ref[n][c] == kNegInf;
      }
    }
    if (__any_sync(0xffffffffu, rises)) {  // some head's reference moves
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (!(top[n][c] > m_ref[n][c] + kMove || m_ref[n][c] == kNegInf)) continue;
          const float m_new = top[n][c] - C::kRaise;
          if (m_ref[n][c] != kNegInf) {
            const float f = fast_exp2(m_ref[n][c] - m_new);
            l[n][c] *= f;
            l[n][c + 2] *= f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[n][i][c] *= f;
              o[n][i][c + 2] *= f;
            }
          }
          m_ref[n][c] = m_new;
        }
      }
    }
    uint32_t pb[NT][2];
    const uint32_t one = FP8 ? 0x3C003C00u : 0x3F803F80u;
    const uint32_t ones[4] = {one, one, one, one};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // (a reference of -infinity, where no slot was valid yet: the weights are 0)
      const float r0 = fmaxf(m_ref[n][0], -3.402823466e38f), r1 = fmaxf(m_ref[n][1], -3.402823466e38f);
      const float w0 = fast_exp2(x[n][0] - r0), w1 = fast_exp2(x[n][1] - r1);
      const float w2 = fast_exp2(x[n][2] - r0), w3 = fast_exp2(x[n][3] - r1);
      // slots g8 and g8 + 8, heads 2 t4 and 2 t4 + 1
      pb[n][0] = movmatrix_trans(FP8 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1));
      pb[n][1] = movmatrix_trans(FP8 ? pack_f16x2(w2, w3) : pack_bf16x2(w2, w3));
      if constexpr (FP8) mma_f16_16816(l[n], ones, pb[n][0], pb[n][1]);
      else mma_bf16_16816(l[n], ones, pb[n][0], pb[n][1]);
    }

    // ---- O^T += V^T P^T --------------------------------------------------------------------
    if constexpr (!FP8) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // matrices: slots 0-7 x dims 0-7, slots 0-7 x 8-15, slots 8-15 x 0-7, slots 8-15 x 8-15
        uint32_t a[4];
        ldmatrix_x4_trans(a, vbuf + ((lane & 7) + (lane >> 4) * 8) * C::kPitch + i * 32 + ((lane >> 3) & 1) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16_16816(o[n][i], a, pb[n][0], pb[n][1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        // matrices of 8 slots x 16 codes: slots 0-7 and 8-15 of m-tile i, then of i + 1
        uint32_t r[4];
        ldmatrix_x4_trans(r, vbuf + (lane & 15) * C::kPitch + i * 16 + (lane >> 4) * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // a register holds dims 2 g8, 2 g8 + 1 of slots 2 t4, 2 t4 + 1: rows g8 and g8 + 8 of
          // the m-tile are dims 2 g8 and 2 g8 + 1
          uint32_t a[4];
          e4m3x4_to_f16x2x2(byte_perm(r[2 * e], 0u, 0x3120u), a[0], a[1]);
          e4m3x4_to_f16x2x2(byte_perm(r[2 * e + 1], 0u, 0x3120u), a[2], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16_16816(o[n][i + e], a, pb[n][0], pb[n][1]);
        }
      }
    }

    __syncwarp();  // the stage's rows have been read: the next sub-tile may land in it
    const int next = sub + kStages * kWarps;
    if (next < subs) {
      const uint32_t mk = issue(next, stage);
      if (stage == 0) valid[0] = mk; else valid[1] = mk;
    }
    cp_async_commit();
    stage ^= 1;
  }

  // ---- merge the warps, then the piece's record or the output ------------------------------
  __syncthreads();  // all warps are done with the ring and the Q rows
  float* sO = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int g = n * 8 + 2 * t4 + c;
      if (g8 == 0) sState[warp][g] = make_float2(m_ref[n][c], l[n][c]);
      float* dst = sO + (warp * NT * 8 + g) * C::kMergePitch;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (FP8) {
          *reinterpret_cast<float2*>(dst + i * 16 + 2 * g8) = make_float2(o[n][i][c], o[n][i][c + 2]);
        } else {
          dst[i * 16 + g8] = o[n][i][c];
          dst[i * 16 + g8 + 8] = o[n][i][c + 2];
        }
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < p.G * (kD / 4); i += kThreads) {
    const int g = i / (kD / 4), d = (i % (kD / 4)) * 4;
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max_or_nan(top, sState[w][g].x);
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 st = sState[w][g];
      if (st.x == kNegInf) continue;  // this warp saw no slot
      const float f = fast_exp2(st.x - top);
      const float4 x = *reinterpret_cast<const float4*>(sO + (w * NT * 8 + g) * C::kMergePitch + d);
      sum = fmaf(st.y, f, sum);
      acc[0] = fmaf(x.x, f, acc[0]);
      acc[1] = fmaf(x.y, f, acc[1]);
      acc[2] = fmaf(x.z, f, acc[2]);
      acc[3] = fmaf(x.w, f, acc[3]);
    }
    // (no slot: every page of the split lies outside the pool)
    const float inv = top == kNegInf ? 0.f : p.v_scale / sum;
    const float lse = top == kNegInf ? kNegInf : top + fast_log2(sum);
    if (seg0 >= u0 && seg1 <= u1) {  // the whole sequence
      *reinterpret_cast<uint2*>(p.out + b * p.o_sb + (h0 + g) * p.o_sh + d) =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      if (d == 0 && p.lse != nullptr) p.lse[int64_t(b) * p.Hq + h0 + g] = lse;
    } else {
      const int64_t rec = (int64_t(blockIdx.x) * 2 + (u == u0 ? 0 : 1)) * p.G + g;
      *reinterpret_cast<float4*>(p.ws_o + rec * kD + d) =
          make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      if (d == 0) p.ws_lse[rec] = lse;
    }
  }
  u = end;
  if (u < u1) {  // the next sequence
    __syncthreads();  // (the ring held the merge)
    seg0 = seg1;
    do ++b; while (tokens_of(p, b, false) == 0);
    len = tokens_of(p, b, false);
    units = units_of(p, len);
  }
  }
}

// Joins the pieces of one (sequence, head): 64 lanes of four dimensions by THREADS / 64 parts
// of the pieces; the parts are added in a fixed order.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) qsa_paged_join_kernel(const DecodeParams p, int groups) {
  constexpr int kParts = THREADS / 64;
  __shared__ float4 sPart[kParts][64];
  __shared__ float sRed[THREADS / 32], sSum[kParts];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, j = h / p.G, g = h - j * p.G;
  launch_next();
  const int units = units_of(p, tokens_of(p, b, false));
  int64_t total;
  const int64_t seg0 = units_before(p, b, total, false), seg1 = seg0 + units;
  const Share share = share_of(total, groups);
  int first = 0, n = 0;
  if (units > 0) first = share.owner(seg0), n = share.owner(seg1 - 1) - first + 1;
  wait_for_last();
  if (n <= 1) return;  // written whole
  // the first block's piece is its last unless it begins with it; the others begin with theirs
  const int shift = share.begin(first) < seg0 ? 1 : 0;
  auto record = [&](int i) { return (((int64_t(first) + i) * p.Hkv + j) * 2 + (i == 0 ? shift : 0)) * p.G + g; };
  float top = kNegInf;
  for (int i = tid; i < n; i += THREADS) top = max_or_nan(top, load_l2(p.ws_lse + record(i)));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) sRed[warp] = top;
  __syncthreads();
  top = sRed[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) top = max_or_nan(top, sRed[w]);

  const int part = tid >> 6, l = tid & 63;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int i = part; i < n; i += kParts) {
    const int64_t rec = record(i);
    const float ls = load_l2(p.ws_lse + rec);
    const float4 x = load_l2(reinterpret_cast<const float4*>(p.ws_o + rec * kD + l * 4));
    if (ls == kNegInf) continue;  // a piece without a valid page
    const float f = fast_exp2(ls - top);
    sum += f;
    acc.x = fmaf(x.x, f, acc.x);
    acc.y = fmaf(x.y, f, acc.y);
    acc.z = fmaf(x.z, f, acc.z);
    acc.w = fmaf(x.w, f, acc.w);
  }
  sPart[part][l] = acc;
  if (l == 0) sSum[part] = sum;
  __syncthreads();
  if (tid >= 64) return;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  float l_all = 0.f;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const float4 x = sPart[i][tid];
    t.x += x.x;
    t.y += x.y;
    t.z += x.z;
    t.w += x.w;
    l_all += sSum[i];
  }
  const float inv = l_all > 0.f || l_all != l_all ? 1.f / l_all : 0.f;
  *reinterpret_cast<uint2*>(p.out + b * p.o_sb + h * p.o_sh + tid * 4) =
      make_uint2(pack_bf16x2(t.x * inv, t.y * inv), pack_bf16x2(t.z * inv, t.w * inv));
  if (tid == 0 && p.lse != nullptr)
    p.lse[int64_t(b) * p.Hq + h] = top == kNegInf ? kNegInf : top + fast_log2(l_all);
}

int decode_unit(int32_t kv_fp8) { return kSub * (kv_fp8 ? Decode<true, 1>::kWarps : Decode<false, 1>::kWarps); }

struct DecodePlan {
  int32_t blocks;
  size_t lse_offset, bytes;
};

DecodePlan decode_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t P, int32_t page_size, int32_t kv_fp8,
                       int32_t num_sms, int32_t request) {
  const int G = Hq / Hkv;
  const int resident = kv_fp8 ? (G <= 8 ? Decode<true, 1>::kResident : Decode<true, 2>::kResident)
                              : (G <= 8 ? Decode<false, 1>::kResident : Decode<false, 2>::kResident);
  // groups of a block per KV head; no more of them than there are units when every sequence
  // is as long as its pages
  const int unit = decode_unit(kv_fp8);
  const int64_t most = int64_t(B) * ((int64_t(P) * page_size + unit - 1) / unit);
  int64_t n = (request > 0 ? request : int64_t(num_sms > 0 ? num_sms : 1) * resident) / Hkv;
  n = n > most ? most : n;
  n = n < 1 ? 1 : n;
  DecodePlan pl{int32_t(n * Hkv), 0, 0};
  if (n > 1) {
    const size_t records = size_t(pl.blocks) * 2 * size_t(G);
    pl.lse_offset = records * kD * 4;
    pl.bytes = pl.lse_offset + (records * 4 + 255) / 256 * 256;
  }
  return pl;
}

qsa_status_t check_decode_sizes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t P,
                                int32_t page_size, int32_t kv_fp8, int32_t blocks) {
  if (B < 0 || P < 0) QSA_REJECT(QSA_ERR_INVALID_ARG, "negative size: B=%d P=%d", B, P);
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "Hq=%d must be a positive multiple of Hkv=%d", Hq, Hkv);
  if (D != kD) QSA_REJECT(QSA_ERR_UNSUPPORTED, "head dimension %d (only 256)", D);
  if (Hq / Hkv > kMaxGroup) QSA_REJECT(QSA_ERR_UNSUPPORTED, "group size G=%d (1..16)", Hq / Hkv);
  if (page_size < 1) QSA_REJECT(QSA_ERR_INVALID_ARG, "page_size=%d", page_size);
  if (int64_t(P) * page_size > INT32_MAX - 4096)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "a page table of %lld tokens", (long long)(int64_t(P) * page_size));
  if (blocks < 0 || blocks > (1 << 16)) QSA_REJECT(QSA_ERR_INVALID_ARG, "blocks=%d outside 0..65536", blocks);
  if (kv_fp8 != 0 && kv_fp8 != 1) QSA_REJECT(QSA_ERR_INVALID_ARG, "kv_fp8 must be 0 or 1");
  return QSA_OK;
}

template <bool FP8, int NT>
cudaError_t launch_decode(const DecodeParams& p, int blocks, cudaStream_t st) {
  using C = Decode<FP8, NT>;
  static std::atomic<uint64_t> done[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(qsa_paged_decode_kernel<FP8, NT>), done);
  if (e != cudaSuccess) return e;
  return launch(qsa_paged_decode_kernel<FP8, NT>, blocks, C::kThreads, C::kSmem, st, p);
}

template <int THREADS>
cudaError_t launch_join(const DecodeParams& p, int groups, cudaStream_t st) {
  return launch(qsa_paged_join_kernel<THREADS>, unsigned(p.B) * p.Hq, THREADS, 0, st, p, groups);
}

}  // namespace

extern "C" int32_t qsa_paged_decode_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t P,
                                         int32_t page_size, int32_t kv_fp8, int32_t num_sms,
                                         int32_t blocks_request, size_t* workspace_bytes) {
  set_error_detail("%s", "");
  const qsa_status_t st = check_decode_sizes(B, Hq, Hkv, D, P, page_size, kv_fp8, blocks_request);
  if (st != QSA_OK) return -int32_t(st);
  const DecodePlan pl = decode_plan(B, Hq, Hkv, P, page_size, kv_fp8, num_sms, blocks_request);
  if (workspace_bytes != nullptr) *workspace_bytes = pl.bytes;
  return pl.blocks;
}

extern "C" qsa_status_t qsa_paged_decode(
    const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* k_cache, int64_t k_stride_s,
    int64_t k_stride_h, const void* v_cache, int64_t v_stride_s, int64_t v_stride_h,
    const int32_t* page_table, int64_t page_stride, const int32_t* seq_lens, int32_t B, int32_t Hq,
    int32_t Hkv, int32_t D, int32_t P, int64_t pages, int32_t page_size, float scale, int32_t kv_fp8,
    float k_scale, float v_scale, void* out, int64_t out_stride_b, int64_t out_stride_h, float* lse,
    int32_t blocks, void* workspace, size_t workspace_bytes, uint32_t* err_word, void* stream) {
  set_error_detail("%s", "");
  const qsa_status_t sizes = check_decode_sizes(B, Hq, Hkv, D, P, page_size, kv_fp8, blocks);
  if (sizes != QSA_OK) return sizes;
  if (!std::isfinite(scale)) QSA_REJECT(QSA_ERR_INVALID_ARG, "scale is not finite");
  if (kv_fp8 && (!std::isfinite(k_scale) || !std::isfinite(v_scale)))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "k_scale or v_scale is not finite");
  if (pages < 0 || pages * page_size > INT32_MAX)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "%lld pages of %d slots: slots are int32", (long long)pages, page_size);
  if (k_stride_s > INT32_MAX / 2 || v_stride_s > INT32_MAX / 2)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "slot strides of 2^30 elements or more");
  if (B == 0) return QSA_OK;
  if (q == nullptr || seq_lens == nullptr || out == nullptr ||
      (P > 0 && (page_table == nullptr || (pages > 0 && (k_cache == nullptr || v_cache == nullptr)))))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL q, k_cache, v_cache, page_table, seq_lens or out");
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
  if (!aligned_to(page_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(lse, 4) || !aligned_to(err_word, 4))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "page_table, seq_lens, lse and err_word must be 4-byte aligned");
  const int64_t e = kv_fp8 ? 1 : 2;
  if (!stride_multiple(q_stride_b, 2, 16) || !stride_multiple(q_stride_h, 2, 16) ||
      !stride_multiple(out_stride_b, 2, 16) || !stride_multiple(out_stride_h, 2, 16) ||
      !stride_multiple(k_stride_s, e, 16) || !stride_multiple(k_stride_h, e, 16) ||
      !stride_multiple(v_stride_s, e, 16) || !stride_multiple(v_stride_h, e, 16) || page_stride < 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "strides must be non-negative multiples of 16 bytes");
  int dev = 0, num_sms = 0;
  if (blocks == 0) {
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (ce != cudaSuccess) return launch_status(ce, "qsa_paged_decode");
  }
  const DecodePlan pl = decode_plan(B, Hq, Hkv, P, page_size, kv_fp8, num_sms, blocks);
  if (int64_t(B) * Hq > INT32_MAX) QSA_REJECT(QSA_ERR_INVALID_ARG, "too many (sequence, head) pairs for one launch");
  if (pl.bytes > 0 && (workspace == nullptr || workspace_bytes < pl.bytes))
    QSA_REJECT(QSA_ERR_WORKSPACE, "workspace of %zu bytes needed for blocks=%d, got %zu", pl.bytes, pl.blocks,
               workspace == nullptr ? size_t(0) : workspace_bytes);
  if (!aligned_to(workspace, 16)) QSA_REJECT(QSA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");

  DecodeParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.table = page_table, p.lens = seq_lens;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = pl.bytes > 0 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.lse_offset) : nullptr;
  p.err_word = err_word;
  p.q_sb = q_stride_b, p.q_sh = q_stride_h, p.o_sb = out_stride_b, p.o_sh = out_stride_h;
  p.table_st = page_stride, p.pages = pages;
  p.k_ss = uint32_t(k_stride_s * e), p.k_sh = k_stride_h * e;
  p.v_ss = uint32_t(v_stride_s * e), p.v_sh = v_stride_h * e;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.P = P, p.page_size = page_size;
  p.unit = decode_unit(kv_fp8);
  for (p.unit_log2 = 0; (1 << p.unit_log2) < p.unit;) ++p.unit_log2;
  p.page_magic = uint32_t(((uint64_t(1) << 32) + page_size - 1) / page_size);
  // log2(e): the softmax runs in base 2
  p.scale_log2 = (kv_fp8 ? scale * k_scale : scale) * 1.4426950408889634f;
  p.v_scale = kv_fp8 ? v_scale : 1.0f;
  const auto st = static_cast<cudaStream_t>(stream);
  const int n = pl.blocks;
  cudaError_t ce = kv_fp8 ? (p.G <= 8 ? launch_decode<true, 1>(p, n, st) : launch_decode<true, 2>(p, n, st))
                          : (p.G <= 8 ? launch_decode<false, 1>(p, n, st) : launch_decode<false, 2>(p, n, st));
  if (ce != cudaSuccess) return launch_status(ce, "qsa_paged_decode");
  // 16 pieces of a sequence or more on average: more parts of them at once
  const int groups = n / Hkv;
  if (groups > 1) ce = groups >= 16 * B ? launch_join<1024>(p, groups, st) : launch_join<128>(p, groups, st);
  return launch_status(ce, "qsa_paged_decode: join");
}
