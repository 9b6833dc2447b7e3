// qsa_rope.cu -- what fills the caches: per-head norm and position rotation of queries and
// keys with the store to the cache slots, and the int8 keys of the cheap score.  Contracts:
// include/qsa_layer.h.
#include "qsa_layer.cuh"

namespace {

using namespace qsa;

constexpr int kMaxPairs = 128;  // rot / 2 at D = 256
constexpr int kRopeRows = 4;    // warp-rows in flight per warp

struct RopeParams {
  const uint16_t *q, *k, *v, *qw, *kw;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;
  const int32_t* pos;
  int64_t pos_stride;
  const float* inv_freq;
  uint16_t* q_out;
  uint8_t *k_dst, *v_dst;
  int64_t qo_st, qo_sh, kd_ss, kd_sh, vd_ss, vd_sh;  // kd, vd: bytes
  const int32_t* slots;
  int64_t rows;
  uint32_t* err_word;
  int32_t T, Hq, Hkv, half, interleaved;
  int32_t axis_end[QSA_MAX_ROPE_AXES];  // pairs below axis_end[a] (and not below a - 1's) turn by a
  float offset, eps, rope_scale, k_scale, v_scale;
  int32_t kv_fp8;
};

// One thread block per token; a row (one head of q, k or v) is D / 8 lanes of 16 bytes, so
// a warp holds 256 / D rows, and each warp keeps kRopeRows of them in flight.  Every byte
// is read and written once: the bound is HBM.  The token's sines and cosines are made once
// per block (one pair per thread) and shared by its heads: made per row they would cost
// more instructions than the row's own work.  The pair of dimension d in the halves form
// is d +- rot / 2, which another lane of the row holds at the same place of its vector
// (rot / 2 is a multiple of 8): one shuffle per element.
template <int D>
__global__ void qsa_norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;        // lanes of a row
  constexpr int kPer = 32 / kLanes;    // rows of a warp access
  __shared__ float2 sTurn[kMaxPairs];  // (cos, sin) of the token's pairs
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int sub = lane / kLanes, l = lane % kLanes;
  const int n_k = p.k != nullptr ? p.Hkv : 0, n_v = p.v != nullptr ? p.Hkv : 0;
  const int n_rows = p.Hq + n_k + n_v;

  int64_t dst = t;
  if (p.slots != nullptr) {
    const int32_t s = p.slots[t];
    if (s < -1 || s >= p.rows) {
      if (threadIdx.x == 0 && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      dst = -1;
    } else {
      dst = s;
    }
  }

  for (int r0 = warp * kPer * kRopeRows; r0 < n_rows || r0 == warp * kPer * kRopeRows;
       r0 += warps * kPer * kRopeRows) {
    uint4 raw[kRopeRows];
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      const int r = r0 + i * kPer + sub;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < n_rows) {
        const uint16_t* src = r < p.Hq ? p.q + t * p.q_st + r * p.q_sh
                              : r < p.Hq + n_k ? p.k + t * p.k_st + (r - p.Hq) * p.k_sh
                                               : p.v + t * p.v_st + (r - p.Hq - n_k) * p.v_sh;
        raw[i] = *reinterpret_cast<const uint4*>(src + l * 8);
      }
    }
    if (r0 == warp * kPer * kRopeRows) {  // the block's first round: make the turns
      for (int i = threadIdx.x; i < p.half; i += blockDim.x) {
        int a = 0;
        while (i >= p.axis_end[a]) ++a;  // axis_end[axes - 1] = half
        // the angle in whole turns, reduced in 64 bits: position * inv_freq has up to 55 bits
        const double turns = double(p.pos[a * p.pos_stride + t]) * double(p.inv_freq[i]) *
                             0.15915494309189533576888;  // 1 / (2 pi)
        float s, c;
        sincospif(2.0f * float(turns - rint(turns)), &s, &c);
        sTurn[i] = make_float2(c * p.rope_scale, s * p.rope_scale);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      const int r = r0 + i * kPer + sub;
      if (r0 + i * kPer >= n_rows) break;  // whole warp past the end
      const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + n_k;
      float x[8];
      bf16x8_to_f32(raw[i], x);
      const uint16_t* w = is_q ? p.qw : is_k ? p.kw : nullptr;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (w != nullptr) {
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
        float wf[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(w + l * 8), wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * (wf[e] + p.offset);
      }
      // the shuffles below run for every lane; rows of v and lanes past rot keep x
      const bool turn = (is_q || is_k) && l * 8 < 2 * p.half;
      if (p.interleaved) {
        if (turn) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 cs = sTurn[l * 4 + (e >> 1)];
            const float u = x[e], v = x[e + 1];
            x[e] = u * cs.x - v * cs.y;
            x[e + 1] = v * cs.x + u * cs.y;
          }
        }
      } else if (p.half > 0) {
        const int hl = p.half >> 3;  // lanes of half the rotated part
        const bool low = l < hl;
        const int other = sub * kLanes + (turn ? (low ? l + hl : l - hl) : l);
        const int pair0 = low ? l * 8 : l * 8 - p.half;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = __shfl_sync(0xffffffffu, x[e], other);
          if (turn) {
            const float2 cs = sTurn[pair0 + e];
            x[e] = low ? x[e] * cs.x - y * cs.y : x[e] * cs.x + y * cs.y;
          }
        }
      }
      if (r >= n_rows) continue;
      if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + t * p.qo_st + r * p.qo_sh + l * 8) = f32_to_bf16x8(x);
      } else if (dst >= 0) {
        const int h = is_k ? r - p.Hq : r - p.Hq - n_k;
        uint8_t* row = is_k ? p.k_dst + dst * p.kd_ss + h * p.kd_sh : p.v_dst + dst * p.vd_ss + h * p.vd_sh;
        if (p.kv_fp8) {
          const float sc = is_k ? p.k_scale : p.v_scale;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], sc);
          *reinterpret_cast<uint2*>(row + l * 8) =
              make_uint2(pack_e4m3x2(x[0], x[1]) | (pack_e4m3x2(x[2], x[3]) << 16),
                         pack_e4m3x2(x[4], x[5]) | (pack_e4m3x2(x[6], x[7]) << 16));
        } else {
          *reinterpret_cast<uint4*>(row + l * 16) = f32_to_bf16x8(x);
        }
      }
    }
  }
}

struct PackParams {
  const uint16_t* keys;
  int64_t key_stride;
  const int32_t* blocks;
  int8_t* codes;
  int64_t code_stride;
  float* scales;
  uint32_t* err_word;
  int64_t n_blocks;
  int32_t n, block;
};

// Di / 8 lanes per micro-block, each summing its eight dimensions over the block's slots
// in order; the maximum crosses the lanes by shuffles.  HBM-bound: the keys are read once.
template <int DI>
__global__ void __launch_bounds__(256) qsa_pack_index_kernel(const PackParams p) {
  constexpr int kLanes = DI / 8;
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes;
  int64_t b = -1;
  if (i < p.n) {
    b = p.blocks[i];
    if (b < -1 || b >= p.n_blocks) {
      if (l == 0 && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      b = -1;
    }
  }
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (b >= 0) {
    const uint16_t* src = p.keys + b * p.block * p.key_stride + l * 8;
    for (int e0 = 0; e0 < p.block; e0 += 4) {
      uint4 raw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e0 + e < p.block) raw[e] = *reinterpret_cast<const uint4*>(src + (e0 + e) * p.key_stride);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e0 + e >= p.block) break;
        float x[8];
        bf16x8_to_f32(raw[e], x);
#pragma unroll
        for (int d = 0; d < 8; ++d) sum[d] = e0 + e == 0 ? x[d] : __fadd_rn(sum[d], x[d]);
      }
    }
  }
  float top = 0.f;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    sum[d] = __fdiv_rn(sum[d], float(p.block));
    top = nan_max(top, fabsf(sum[d]));
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = nan_max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (b < 0) return;
  float scale = __fdiv_rn(top, 127.f);
  if (!(scale < __builtin_huge_valf())) scale = __int_as_float(0x7fffffff);
  *reinterpret_cast<uint2*>(p.codes + b * p.code_stride + l * 8) = int8x8_codes(sum, scale);
  if (l == 0) p.scales[b] = scale;
}

}  // namespace

extern "C" qsa_status_t qsa_qk_norm_rope(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k, int64_t k_stride_t,
    int64_t k_stride_h, const void* v, int64_t v_stride_t, int64_t v_stride_h, const void* q_weight,
    const void* k_weight, float weight_offset, float eps, const int32_t* positions,
    int64_t pos_stride, const float* inv_freq, int32_t rot, int32_t interleaved,
    const int32_t* sections, int32_t axes, float rope_scale, int32_t T, int32_t Hq, int32_t Hkv,
    int32_t D, void* q_out, int64_t q_out_stride_t, int64_t q_out_stride_h, void* k_dst,
    int64_t k_dst_stride_s, int64_t k_dst_stride_h, void* v_dst, int64_t v_dst_stride_s,
    int64_t v_dst_stride_h, const int32_t* slots, int64_t rows, int32_t kv_fp8, float k_scale,
    float v_scale, uint32_t* err_word, void* stream) {
  set_error_detail("%s", "");
  if (T < 0 || Hq < 0 || Hkv < 0 || rows < 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "negative size: T=%d Hq=%d Hkv=%d rows=%lld", T, Hq, Hkv, (long long)rows);
  if (D != 64 && D != 128 && D != 256)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "head dimension %d (64, 128 or 256)", D);
  if (rot < 0 || rot > D || rot % 16 != 0)
    QSA_REJECT(QSA_ERR_UNSUPPORTED, "rot=%d must be a multiple of 16 in 0..%d", rot, D);
  if (Hq > 65536 || Hkv > 65536) QSA_REJECT(QSA_ERR_UNSUPPORTED, "more than 65536 heads");
  if (axes < 1 || axes > QSA_MAX_ROPE_AXES)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "axes=%d outside 1..%d", axes, QSA_MAX_ROPE_AXES);
  if (interleaved != 0 && interleaved != 1) QSA_REJECT(QSA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (kv_fp8 != 0 && kv_fp8 != 1) QSA_REJECT(QSA_ERR_INVALID_ARG, "kv_fp8 must be 0 or 1");
  if (!std::isfinite(weight_offset) || !std::isfinite(eps) || eps < 0.f || !std::isfinite(rope_scale))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "weight_offset, eps (>= 0) and rope_scale must be finite");
  if (kv_fp8 && !(k_scale > 0.f && std::isfinite(k_scale) && v_scale > 0.f && std::isfinite(v_scale)))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  RopeParams p{};
  p.half = rot / 2;
  if (sections == nullptr) {
    if (axes != 1) QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL sections with axes=%d", axes);
    p.axis_end[0] = p.half;
  } else {
    int32_t end = 0;
    for (int a = 0; a < axes; ++a) {
      if (sections[a] < 0 || sections[a] > p.half - end)
        QSA_REJECT(QSA_ERR_INVALID_ARG, "sections must be non-negative with a sum of rot / 2 = %d", p.half);
      p.axis_end[a] = end += sections[a];
    }
    if (end != p.half)
      QSA_REJECT(QSA_ERR_INVALID_ARG, "sections sum to %d, rot / 2 is %d", end, p.half);
  }
  if (T == 0 || (Hq == 0 && Hkv == 0)) return QSA_OK;
  if (Hq > 0 && (q == nullptr || q_out == nullptr)) QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL q or q_out");
  if (Hkv > 0 && (k == nullptr || k_dst == nullptr)) QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL k or k_dst");
  if ((v == nullptr) != (v_dst == nullptr) || (v != nullptr && Hkv == 0))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "v and v_dst must come together, with k");
  if (rot > 0 && (positions == nullptr || inv_freq == nullptr))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL positions or inv_freq with rot=%d", rot);
  if (Hkv > 0 && slots == nullptr && rows < T)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "rows=%lld below T=%d without slots", (long long)rows, T);
  const uintptr_t kv_align = kv_fp8 ? 8 : 16;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(q_weight, 16) ||
      !aligned_to(k_weight, 16) || !aligned_to(q_out, 16) || !aligned_to(k_dst, kv_align) ||
      !aligned_to(v_dst, kv_align))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "q, k, v, weights and outputs must be 16-byte aligned (E4M3 destinations 8)");
  if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4) || !aligned_to(slots, 4) || !aligned_to(err_word, 4))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "positions, inv_freq, slots and err_word must be 4-byte aligned");
  const int64_t ke = kv_fp8 ? 1 : 2;
  if (!stride_multiple(q_stride_t, 2, 16) || !stride_multiple(q_stride_h, 2, 16) ||
      !stride_multiple(k_stride_t, 2, 16) || !stride_multiple(k_stride_h, 2, 16) ||
      !stride_multiple(v_stride_t, 2, 16) || !stride_multiple(v_stride_h, 2, 16) ||
      !stride_multiple(q_out_stride_t, 2, 16) || !stride_multiple(q_out_stride_h, 2, 16) ||
      !stride_multiple(k_dst_stride_s, ke, kv_align) || !stride_multiple(k_dst_stride_h, ke, kv_align) ||
      !stride_multiple(v_dst_stride_s, ke, kv_align) || !stride_multiple(v_dst_stride_h, ke, kv_align) ||
      pos_stride < 0)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "strides must be non-negative multiples of 16 bytes (E4M3 destinations 8)");
  p.q = static_cast<const uint16_t*>(q);
  p.k = Hkv > 0 ? static_cast<const uint16_t*>(k) : nullptr;
  p.v = static_cast<const uint16_t*>(v);
  p.qw = static_cast<const uint16_t*>(q_weight);
  p.kw = static_cast<const uint16_t*>(k_weight);
  p.q_st = q_stride_t, p.q_sh = q_stride_h;
  p.k_st = k_stride_t, p.k_sh = k_stride_h;
  p.v_st = v_stride_t, p.v_sh = v_stride_h;
  p.pos = positions;
  p.pos_stride = pos_stride;
  p.inv_freq = inv_freq;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_dst = static_cast<uint8_t*>(k_dst);
  p.v_dst = static_cast<uint8_t*>(v_dst);
  p.qo_st = q_out_stride_t, p.qo_sh = q_out_stride_h;
  p.kd_ss = k_dst_stride_s * ke, p.kd_sh = k_dst_stride_h * ke;
  p.vd_ss = v_dst_stride_s * ke, p.vd_sh = v_dst_stride_h * ke;
  p.slots = slots;
  p.rows = rows;
  p.err_word = err_word;
  p.T = T, p.Hq = Hq, p.Hkv = Hkv, p.interleaved = interleaved;
  p.offset = weight_offset, p.eps = eps, p.rope_scale = rope_scale;
  p.k_scale = k_scale, p.v_scale = v_scale, p.kv_fp8 = kv_fp8;
  const int n_rows = Hq + (k != nullptr ? Hkv : 0) + (v != nullptr ? Hkv : 0);
  const int per_warp = 256 / D * kRopeRows;
  int warps = (n_rows + per_warp - 1) / per_warp;
  warps = warps > 16 ? 16 : warps;
  const auto st = static_cast<cudaStream_t>(stream);
  if (D == 256) qsa_norm_rope_kernel<256><<<T, warps * 32, 0, st>>>(p);
  else if (D == 128) qsa_norm_rope_kernel<128><<<T, warps * 32, 0, st>>>(p);
  else qsa_norm_rope_kernel<64><<<T, warps * 32, 0, st>>>(p);
  return launch_status(cudaGetLastError(), "qsa_qk_norm_rope");
}

extern "C" qsa_status_t qsa_pack_index_keys(const void* keys, int64_t key_stride_s,
                                            const int32_t* blocks, int32_t n, int32_t block,
                                            int32_t Di, int64_t S, int8_t* codes,
                                            int64_t code_stride, float* scales, uint32_t* err_word,
                                            void* stream) {
  set_error_detail("%s", "");
  if (n < 0 || S < 0) QSA_REJECT(QSA_ERR_INVALID_ARG, "negative size: n=%d S=%lld", n, (long long)S);
  if (Di != 64 && Di != 128) QSA_REJECT(QSA_ERR_UNSUPPORTED, "index dimension %d (64 or 128)", Di);
  if (block < 1 || block > kMaxBlock)
    QSA_REJECT(QSA_ERR_INVALID_ARG, "block size %d outside 1..%d", block, kMaxBlock);
  if (n == 0) return QSA_OK;
  if (blocks == nullptr || (S >= block && (keys == nullptr || codes == nullptr || scales == nullptr)))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL keys, blocks, codes or scales");
  if (!aligned_to(keys, 16) || !aligned_to(codes, 16) || !aligned_to(blocks, 4) ||
      !aligned_to(scales, 4) || !aligned_to(err_word, 4))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "keys and codes must be 16-byte aligned, blocks, scales and err_word 4-byte");
  if (!stride_multiple(key_stride_s, 2, 16) || !stride_multiple(code_stride, 1, 16))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "strides of keys and codes must be non-negative multiples of 16 bytes");
  PackParams p{};
  p.keys = static_cast<const uint16_t*>(keys);
  p.key_stride = key_stride_s;
  p.blocks = blocks;
  p.codes = codes;
  p.code_stride = code_stride;
  p.scales = scales;
  p.err_word = err_word;
  p.n_blocks = S / block;
  p.n = n;
  p.block = block;
  const int per = 256 / (Di / 8);
  const int grid = int((int64_t(n) + per - 1) / per);
  const auto st = static_cast<cudaStream_t>(stream);
  if (Di == 128) qsa_pack_index_kernel<128><<<grid, 256, 0, st>>>(p);
  else qsa_pack_index_kernel<64><<<grid, 256, 0, st>>>(p);
  return launch_status(cudaGetLastError(), "qsa_pack_index_keys");
}
