// qsa_decode.cu -- attention of one new token per sequence over its whole paged cache, split
// over the cache's length and joined.  Contract: include/qsa_layer.h (qsa_paged_decode).
#include "qsa_layer.cuh"

namespace {

using namespace qsa;

constexpr int kD = kHeadDim;
constexpr int kDecodeWarps = 2;
constexpr int kDecodeThreads = 32 * kDecodeWarps;
constexpr int kStages = 2;
constexpr int kSub = 16;                 // slots of a warp's sub-tile (the M of one MMA)
constexpr int kMinSplit = 64;            // slots: what a thread block has in flight at once
constexpr int kJoinThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kRescaleLog2 = 8.0f;

struct DecodeParams {
  const uint16_t* q;
  const uint8_t *k, *v;
  const int32_t *table, *lens;
  uint16_t* out;
  float *lse, *ws_o, *ws_lse;  // ws_o [B, Hq, nsplit, D], ws_lse [B, Hq, nsplit]
  uint32_t* err_word;
  int64_t q_sb, q_sh, o_sb, o_sh, table_st, pages;
  int64_t k_ss, k_sh, v_ss, v_sh;  // bytes
  int32_t B, Hq, Hkv, G, P, page_size, nsplit, split_len;
  float scale_log2, v_scale;
};

__device__ __forceinline__ int tokens_of(const DecodeParams& p, int b, bool report) {
  const int64_t most = int64_t(p.P) * p.page_size;
  const int n = p.lens[b];
  if (report && p.err_word != nullptr && (n < 0 || n > most)) atomicOr(p.err_word, QSA_ERRBIT_WIDTH_RANGE);
  return int(min(int64_t(max(n, 0)), most));
}

// NT n8 tiles hold the G heads of a KV head.  Rows in shared memory are padded by 16 bytes,
// so the eight rows that one 8x8 matrix load touches fall into different banks.
template <bool FP8, int NT>
struct Decode {
  static constexpr int kRow = FP8 ? kD : 2 * kD;  // bytes of a cache row
  static constexpr int kPitch = kRow + 16;
  static constexpr int kStageBytes = 2 * kSub * kPitch;  // K rows, then V rows
  static constexpr int kRing = kDecodeWarps * kStages * kStageBytes;
  static constexpr int kQPitch = 2 * kD + 16;
  static constexpr int kQBytes = NT * 8 * kQPitch;
  static constexpr int kMergePitch = kD + 4;
  static constexpr size_t kSmem = kRing + kQBytes;
  static constexpr int kMergeBytes = kDecodeWarps * NT * 8 * kMergePitch * 4;
  static_assert(kMergeBytes <= int(kSmem), "the merge buffer reuses the ring and the Q rows");
};

// One thread block per (sequence, KV head, split of the length).  Each warp takes every
// second 16-slot sub-tile of the split and runs a pipeline of its own: one bulk copy per K
// or V row and lane, an mbarrier per stage, no block-wide barrier in the loop.  Scores are
// S^T = K Q^T with the slots as M and the heads as N, so the group shares every row that is
// read; the softmax is online (base 2, the reference moves only when the maximum rises by
// more than 2^8); P is rounded to 16 bits for O^T += V^T P^T, and the denominator sums the
// same rounded values.  The bound is HBM: every row is read once.
template <bool FP8, int NT>
__global__ void __launch_bounds__(kDecodeThreads) qsa_paged_decode_kernel(const DecodeParams p) {
  using C = Decode<FP8, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t sBar[kDecodeWarps * kStages];
  __shared__ float2 sState[kDecodeWarps][NT * 8];  // (m, l) of each warp and head
  uint8_t* sQ = smem + C::kRing;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = blockIdx.x % p.nsplit;
  const int j = (blockIdx.x / p.nsplit) % p.Hkv, b = blockIdx.x / p.nsplit / p.Hkv;
  const int len = tokens_of(p, b, tid == 0);
  const int s0 = split * p.split_len, s1 = s0 + min(p.split_len, len - s0);  // (s0 is below the table's tokens)
  const int h0 = j * p.G;
  if (s0 >= s1) {  // nothing here; the only split of an empty sequence writes its zeros
    if (p.nsplit == 1) {
      for (int i = tid; i < p.G * (kD / 8); i += kDecodeThreads)
        *reinterpret_cast<uint4*>(p.out + b * p.o_sb + (h0 + i / (kD / 8)) * p.o_sh + (i % (kD / 8)) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr)
        for (int g = tid; g < p.G; g += kDecodeThreads) p.lse[int64_t(b) * p.Hq + h0 + g] = kNegInf;
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kDecodeWarps * kStages; ++i) mbar_init(smem_addr(sBar + i), 1);
    mbar_init_fence();
  }
  __syncthreads();

  const uint32_t ring = smem_addr(smem) + warp * kStages * C::kStageBytes;
  const uint32_t bars = smem_addr(sBar + warp * kStages);
  const uint8_t* kg = p.k + j * p.k_sh;
  const uint8_t* vg = p.v + j * p.v_sh;
  const int subs = (s1 - s0 + kSub - 1) / kSub;  // sub-tiles of the split; warp w takes w, w + 2, ...
  uint32_t valid[kStages];                       // one bit per slot of the stage's sub-tile

  // Lanes 0-15 copy the sub-tile's K rows, lanes 16-31 its V rows.  Slots past the end or
  // in a page outside the pool are not read.
  auto issue = [&](int sub, int stage, uint32_t& mask) {
    const int i = s0 + sub * kSub + (lane & 15);
    bool ok = i < s1;
    int64_t slot = 0;
    if (ok) {
      const int m = i / p.page_size;
      const int page = __ldg(p.table + b * p.table_st + m);
      ok = page >= 0 && page < p.pages;
      if (!ok && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      slot = int64_t(page) * p.page_size + (i - m * p.page_size);
    }
    mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
    const uint32_t bar = bars + stage * 8;
    if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(__popc(mask)) * 2 * C::kRow);
    __syncwarp();
    if (ok)
      bulk_copy(ring + stage * C::kStageBytes + lane * C::kPitch,
               lane < 16 ? kg + slot * p.k_ss : vg + slot * p.v_ss, C::kRow, bar);
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    valid[s] = 0;
    if (warp + s * kDecodeWarps < subs) issue(warp + s * kDecodeWarps, s, valid[s]);
  }

  // ---- Q: bf16 rows, or f16 for an E4M3 cache (its codes are exact in f16) -----------------
  const uint32_t q_s = smem_addr(sQ);
  for (int i = tid; i < NT * 8 * (kD / 8); i += kDecodeThreads) {
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
      raw = make_uint4(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]), pack_f16x2(x[4], x[5]),
                       pack_f16x2(x[6], x[7]));
    }
    *reinterpret_cast<uint4*>(sQ + g * C::kQPitch + c * 16) = raw;
  }
  __syncthreads();

  float o[NT][16][4];  // O^T: 16 m-tiles of 16 dimensions
  float m_ref[NT][2], l_sum[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m_ref[n][0] = m_ref[n][1] = kNegInf;
    l_sum[n][0] = l_sum[n][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
  }
  const int g8 = lane >> 2, t4 = lane & 3;
  bool late = false;

  int stage = 0;
  uint32_t phase = 0;
  for (int sub = warp; sub < subs; sub += kDecodeWarps) {
    const uint32_t kbuf = ring + stage * C::kStageBytes, vbuf = kbuf + kSub * C::kPitch;
    const uint32_t mask = stage == 0 ? valid[0] : valid[1];
    if (__any_sync(0xffffffffu, !wait_phase(bars + stage * 8, phase))) {
      late = true;
      break;
    }
    if (mask != 0xffffu) {  // V rows that were not read: zeros, so that 0 * V is 0
      if (lane >= 16 && !((mask >> (lane - 16)) & 1)) {
        uint8_t* row = smem + (kbuf - smem_addr(smem)) + lane * C::kPitch;
        for (int c = 0; c < C::kRow / 16; ++c) reinterpret_cast<uint4*>(row)[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }

    // ---- S^T = K Q^T: two accumulators per n8 tile keep two chains in flight ---------------
    float s[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) s[n][c][0] = s[n][c][1] = s[n][c][2] = s[n][c][3] = 0.f;
    if constexpr (!FP8) {
#pragma unroll
      for (int ks = 0; ks < 16; ++ks) {
        uint32_t a[4];
        ldmatrix_x4(a, kbuf + (lane & 15) * C::kPitch + ks * 32 + (lane >> 4) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t qa = q_s + (n * 8 + g8) * C::kQPitch + ks * 32 + t4 * 4;
          uint32_t b0, b1;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b0) : "r"(qa));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b1) : "r"(qa + 16));
          mma_bf16_16816(s[n][ks & 1], a, b0, b1);
        }
      }
    } else {
#pragma unroll
      for (int kp = 0; kp < 8; ++kp) {  // two 16-code k-steps per load
        uint32_t r[4];
        ldmatrix_x4(r, kbuf + (lane & 15) * C::kPitch + kp * 32 + (lane >> 4) * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // the lane's codes 4 t4 .. 4 t4 + 3 of a row stand for k = 2 t4, 2 t4 + 1, 2 t4 + 8,
          // 2 t4 + 9: a permutation of the sum's order that Q's fragments share
          uint32_t a[4];
          e4m3x4_to_f16x2x2(r[2 * e], a[0], a[2]);
          e4m3x4_to_f16x2x2(r[2 * e + 1], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t qa = q_s + (n * 8 + g8) * C::kQPitch + (kp * 2 + e) * 32 + t4 * 8;
            uint32_t b0, b1;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b0), "=r"(b1) : "r"(qa));
            mma_f16_16816(s[n][e], a, b0, b1);
          }
        }
      }
    }

    // ---- softmax over the sub-tile's slots (rows g8 and g8 + 8) ------------------------------
    const bool ok0 = (mask >> g8) & 1, ok1 = (mask >> (g8 + 8)) & 1;
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = (s[n][0][e] + s[n][1][e]) * p.scale_log2;
        x[e] = (e < 2 ? ok0 : ok1) ? y : kNegInf;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = fmaxf(x[c], x[c + 2]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (top > m_ref[n][c] + kRescaleLog2 || m_ref[n][c] == kNegInf) {
          const float f = m_ref[n][c] == kNegInf ? 0.f : fast_exp2(m_ref[n][c] - top);
          if (m_ref[n][c] != kNegInf) {
            l_sum[n][c] *= f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[n][i][c] *= f;
              o[n][i][c + 2] *= f;
            }
          }
          m_ref[n][c] = top;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m_ref[n][e & 1];
        x[e] = ref == kNegInf ? 0.f : fast_exp2(x[e] - ref);
      }
      uint32_t lo, hi;  // slots g8 and g8 + 8, heads 2 t4 and 2 t4 + 1
      if constexpr (FP8) {
        lo = pack_f16x2(x[0], x[1]);
        hi = pack_f16x2(x[2], x[3]);
        l_sum[n][0] += f16lo_to_f32(lo) + f16lo_to_f32(hi);
        l_sum[n][1] += f16hi_to_f32(lo) + f16hi_to_f32(hi);
      } else {
        lo = pack_bf16x2(x[0], x[1]);
        hi = pack_bf16x2(x[2], x[3]);
        l_sum[n][0] += bf16lo_to_f32(lo) + bf16lo_to_f32(hi);
        l_sum[n][1] += bf16hi_to_f32(lo) + bf16hi_to_f32(hi);
      }
      pb[n][0] = movmatrix_trans(lo);
      pb[n][1] = movmatrix_trans(hi);
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

    // the stage's rows have been read: the next sub-tile may land in it
    fence_proxy_async_smem();
    __syncwarp();
    const int next = sub + kStages * kDecodeWarps;
    if (next < subs) {
      uint32_t mk;
      issue(next, stage, mk);
      if (stage == 0) valid[0] = mk; else valid[1] = mk;
    }
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (late) {  // give the copies in flight a second chance to land, then leave without a result
    if (lane == 0 && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_TIMEOUT);
    wait_phase(bars + stage * 8, phase);
    wait_phase(bars + (stage ^ 1) * 8, phase ^ uint32_t(stage));
  }
  if (__syncthreads_or(late)) return;

  // ---- merge the warps, then the split's record or the output ------------------------------
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l_sum[n][c] += __shfl_xor_sync(0xffffffffu, l_sum[n][c], d);
  // (both warps are done with the ring and Q: the barrier above)
  float* sO = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int g = n * 8 + 2 * t4 + c;
      if (g8 == 0) sState[warp][g] = make_float2(m_ref[n][c], l_sum[n][c]);
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
  for (int i = tid; i < p.G * (kD / 4); i += kDecodeThreads) {
    const int g = i / (kD / 4), d = (i % (kD / 4)) * 4;
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kDecodeWarps; ++w) top = fmaxf(top, sState[w][g].x);
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
    for (int w = 0; w < kDecodeWarps; ++w) {
      const float2 st = sState[w][g];
      if (st.x == kNegInf) continue;  // this warp saw no slot
      const float f = fast_exp2(st.x - top);
      const float4 x = *reinterpret_cast<const float4*>(sO + (w * NT * 8 + g) * C::kMergePitch + d);
      l = fmaf(st.y, f, l);
      acc[0] = fmaf(x.x, f, acc[0]);
      acc[1] = fmaf(x.y, f, acc[1]);
      acc[2] = fmaf(x.z, f, acc[2]);
      acc[3] = fmaf(x.w, f, acc[3]);
    }
    // (no slot: every page of the split lies outside the pool)
    const float inv = top == kNegInf ? 0.f : p.v_scale / l;
    const float lse = top == kNegInf ? kNegInf : top + fast_log2(l);
    const int64_t row = int64_t(b) * p.Hq + h0 + g;
    if (p.nsplit == 1) {
      *reinterpret_cast<uint2*>(p.out + b * p.o_sb + (h0 + g) * p.o_sh + d) =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      if (d == 0 && p.lse != nullptr) p.lse[row] = lse;
    } else {
      *reinterpret_cast<float4*>(p.ws_o + (row * p.nsplit + split) * kD + d) =
          make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      if (d == 0) p.ws_lse[row * p.nsplit + split] = lse;
    }
  }
}

// Joins the splits of one (sequence, head): 64 dimensions per thread block, 16 lanes of four
// dimensions by 16 parts of the splits; the parts are added in a fixed order.
__global__ void __launch_bounds__(kJoinThreads) qsa_paged_join_kernel(const DecodeParams p) {
  __shared__ float4 sPart[16][16];
  __shared__ float sRed[kJoinThreads / 32], sSum[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = blockIdx.x & 3;
  const int64_t row = blockIdx.x >> 2;
  const int b = int(row / p.Hq), h = int(row % p.Hq);
  const int len = tokens_of(p, b, false);
  const int n = int((int64_t(len) + p.split_len - 1) / p.split_len);  // splits that hold tokens
  const float* lse = p.ws_lse + row * p.nsplit;
  float top = kNegInf;
  for (int s = tid; s < n; s += kJoinThreads) top = fmaxf(top, lse[s]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) sRed[warp] = top;
  __syncthreads();
  top = sRed[0];
#pragma unroll
  for (int w = 1; w < kJoinThreads / 32; ++w) top = fmaxf(top, sRed[w]);

  const int part = tid >> 4, l = tid & 15;
  const float* src = p.ws_o + row * p.nsplit * kD + quarter * 64 + l * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int s = part; s < n; s += 16) {
    const float ls = lse[s];
    const float4 x = *reinterpret_cast<const float4*>(src + int64_t(s) * kD);
    if (ls == kNegInf) continue;  // a split without a valid page
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
  if (tid >= 16) return;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  float l_all = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float4 x = sPart[i][tid];
    t.x += x.x;
    t.y += x.y;
    t.z += x.z;
    t.w += x.w;
    l_all += sSum[i];
  }
  const float inv = l_all > 0.f || l_all != l_all ? 1.f / l_all : 0.f;
  *reinterpret_cast<uint2*>(p.out + b * p.o_sb + h * p.o_sh + quarter * 64 + tid * 4) =
      make_uint2(pack_bf16x2(t.x * inv, t.y * inv), pack_bf16x2(t.z * inv, t.w * inv));
  if (quarter == 0 && tid == 0 && p.lse != nullptr)
    p.lse[row] = top == kNegInf ? kNegInf : top + fast_log2(l_all);
}

struct DecodePlan {
  int32_t nsplit, split_len;
  size_t lse_offset, bytes;
};

DecodePlan decode_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t P, int32_t page_size,
                       int32_t num_sms, int32_t request) {
  const int64_t cap = int64_t(P) * page_size;  // tokens of a sequence at most
  int64_t n;
  if (request > 0) {
    n = request;
  } else {
    // four waves of three blocks per SM, so that sequences of different lengths even out
    const int64_t units = int64_t(B) * Hkv, want = int64_t(num_sms > 0 ? num_sms : 1) * 3;
    n = units > 0 ? (want * (units * 2 > want ? 4 : 1) + units - 1) / units : 1;
  }
  const int64_t most = (cap + kMinSplit - 1) / kMinSplit;
  n = n > most ? most : n;
  n = n < 1 ? 1 : n;
  int64_t len = cap > 0 ? ((cap + n - 1) / n + kSub - 1) / kSub * kSub : kSub;
  n = cap > 0 ? (cap + len - 1) / len : 1;
  DecodePlan pl{int32_t(n), int32_t(len), 0, 0};
  if (n > 1) {
    const size_t rows = size_t(B) * size_t(Hq) * size_t(n);
    pl.lse_offset = (rows * kD * 4 + 255) / 256 * 256;
    pl.bytes = pl.lse_offset + (rows * 4 + 255) / 256 * 256;
  }
  return pl;
}

qsa_status_t check_decode_sizes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t P,
                                int32_t page_size, int32_t nsplit) {
  if (B < 0 || P < 0) QSA_REJECT(QSA_ERR_INVALID_ARG, "negative size: B=%d P=%d", B, P);
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "Hq=%d must be a positive multiple of Hkv=%d", Hq, Hkv);
  if (D != kD) QSA_REJECT(QSA_ERR_UNSUPPORTED, "head dimension %d (only 256)", D);
  if (Hq / Hkv > kMaxGroup) QSA_REJECT(QSA_ERR_UNSUPPORTED, "group size G=%d (1..16)", Hq / Hkv);
  if (page_size < 1) QSA_REJECT(QSA_ERR_INVALID_ARG, "page_size=%d", page_size);
  if (int64_t(P) * page_size > INT32_MAX - 4096)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "a page table of %lld tokens", (long long)(int64_t(P) * page_size));
  if (nsplit < 0) QSA_REJECT(QSA_ERR_INVALID_ARG, "negative nsplit");
  return QSA_OK;
}

template <bool FP8, int NT>
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t st) {
  using C = Decode<FP8, NT>;
  const cudaError_t e = cudaFuncSetAttribute(qsa_paged_decode_kernel<FP8, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  if (e != cudaSuccess) return e;
  qsa_paged_decode_kernel<FP8, NT><<<unsigned(p.B) * p.Hkv * p.nsplit, kDecodeThreads, C::kSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

extern "C" int32_t qsa_paged_decode_plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t P,
                                         int32_t page_size, int32_t num_sms,
                                         int32_t nsplit_request, size_t* workspace_bytes) {
  set_error_detail("%s", "");
  const qsa_status_t st = check_decode_sizes(B, Hq, Hkv, D, P, page_size, nsplit_request);
  if (st != QSA_OK) return -int32_t(st);
  const DecodePlan pl = decode_plan(B, Hq, Hkv, P, page_size, num_sms, nsplit_request);
  if (workspace_bytes != nullptr) *workspace_bytes = pl.bytes;
  return pl.nsplit;
}

extern "C" qsa_status_t qsa_paged_decode(
    const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* k_cache, int64_t k_stride_s,
    int64_t k_stride_h, const void* v_cache, int64_t v_stride_s, int64_t v_stride_h,
    const int32_t* page_table, int64_t page_stride, const int32_t* seq_lens, int32_t B, int32_t Hq,
    int32_t Hkv, int32_t D, int32_t P, int64_t pages, int32_t page_size, float scale, int32_t kv_fp8,
    float k_scale, float v_scale, void* out, int64_t out_stride_b, int64_t out_stride_h, float* lse,
    int32_t nsplit, void* workspace, size_t workspace_bytes, uint32_t* err_word, void* stream) {
  set_error_detail("%s", "");
  const qsa_status_t sizes = check_decode_sizes(B, Hq, Hkv, D, P, page_size, nsplit);
  if (sizes != QSA_OK) return sizes;
  if (kv_fp8 != 0 && kv_fp8 != 1) QSA_REJECT(QSA_ERR_INVALID_ARG, "kv_fp8 must be 0 or 1");
  if (!std::isfinite(scale)) QSA_REJECT(QSA_ERR_INVALID_ARG, "scale is not finite");
  if (kv_fp8 && (!std::isfinite(k_scale) || !std::isfinite(v_scale)))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "k_scale or v_scale is not finite");
  if (pages < 0) QSA_REJECT(QSA_ERR_INVALID_ARG, "negative pages");
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
  if (nsplit == 0) {
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (ce != cudaSuccess) return launch_status(ce, "qsa_paged_decode");
  }
  const DecodePlan pl = decode_plan(B, Hq, Hkv, P, page_size, num_sms, nsplit);
  if (int64_t(B) * Hkv * pl.nsplit > INT32_MAX || int64_t(B) * Hq * 4 > INT32_MAX)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "too many work units for one launch");
  if (pl.bytes > 0 && (workspace == nullptr || workspace_bytes < pl.bytes))
    QSA_REJECT(QSA_ERR_WORKSPACE, "workspace of %zu bytes needed for nsplit=%d, got %zu", pl.bytes, pl.nsplit,
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
  p.k_ss = k_stride_s * e, p.k_sh = k_stride_h * e, p.v_ss = v_stride_s * e, p.v_sh = v_stride_h * e;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.P = P, p.page_size = page_size;
  p.nsplit = pl.nsplit, p.split_len = pl.split_len;
  // log2(e): the softmax runs in base 2
  p.scale_log2 = (kv_fp8 ? scale * k_scale : scale) * 1.4426950408889634f;
  p.v_scale = kv_fp8 ? v_scale : 1.0f;
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t ce = kv_fp8 ? (p.G <= 8 ? launch_decode<true, 1>(p, st) : launch_decode<true, 2>(p, st))
                          : (p.G <= 8 ? launch_decode<false, 1>(p, st) : launch_decode<false, 2>(p, st));
  if (ce != cudaSuccess) return launch_status(ce, "qsa_paged_decode");
  if (pl.nsplit > 1) {
    qsa_paged_join_kernel<<<unsigned(B) * Hq * 4, kJoinThreads, 0, st>>>(p);
    ce = cudaGetLastError();
  }
  return launch_status(ce, "qsa_paged_decode: join");
}
