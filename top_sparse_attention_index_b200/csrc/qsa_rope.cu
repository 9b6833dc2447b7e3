// qsa_rope.cu -- what fills the caches: per-head norm and position rotation of queries and
// keys with the store to the cache slots, and the int8 keys of the cheap score.  Contracts:
// include/qsa_layer.h.
#include "qsa_layer.cuh"

namespace {

using namespace qsa;

constexpr int kMaxPairs = 128;    // rot / 2 at D = 256
constexpr int kRopeWarps = 4;     // of a thread block; each works for itself

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
  int64_t rows, units;  // units: T * parts
  uint32_t* err_word;
  int32_t T, Hq, Hkv, half, interleaved;
  int32_t q_steps, k_steps, v_steps, steps, parts;  // of a token; of a warp; warps of a token
  int32_t axis_end[QSA_MAX_ROPE_AXES];  // pairs below axis_end[a] (and not below a - 1's) turn by a
  float offset, eps, rope_scale, inv_k_scale, inv_v_scale;
  int32_t kv_fp8;
};

__device__ __forceinline__ void bf16x8_to_pairs(const uint4& r, uint64_t (&x)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i]));
}

__device__ __forceinline__ uint4 pairs_to_bf16x8(const uint64_t (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(x[i], lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 pairs_to_e4m3x8(const uint64_t (&x)[4], uint64_t inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(mul2(x[i], inv), lo, hi);
    w[i] = pack_e4m3x2(lo, hi);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// A warp takes `steps` steps of one token, a step being 512 / D rows of q, of k or of v: every
// warp makes its token's sines and cosines for itself.  A row is D / 16 lanes of two 16-byte
// vectors, chosen so that both dimensions of every rotated pair are in one lane (halves:
// vectors l and l + rot / 16 for the rotated part; otherwise neighbours), so the rotation
// crosses no lanes and a lane's eight (cos, sin) and its weights stay in registers for all
// its rows; two values per arithmetic instruction; a step loads while the last is worked on.
// Bound: every byte is read and written once, HBM.  16,384 tokens of 24 + 2 + 2 heads (470 MB):
// 94 us, 0.77 of the copy rate; what is left is issue slots, 20 warps to an SM.  (A vector per
// lane, shuffles for the pairs and a thread block per token took 149 us.)
template <int D>
__global__ void __launch_bounds__(32 * kRopeWarps, 5) qsa_norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;      // lanes of a row
  constexpr int kRows = 32 / kLanes;  // rows of a step
  __shared__ float2 sTurn[kRopeWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = int64_t(blockIdx.x) * kRopeWarps + warp;
  begin_kernel();
  if (unit >= p.units) return;
  const int t = p.parts == 1 ? int(unit) : int(unit / p.parts);
  const int first = int(unit - int64_t(t) * p.parts) * p.steps;
  const int all = p.q_steps + p.k_steps + p.v_steps, end = min(first + p.steps, all);

  const int sub = lane / kLanes, l = lane % kLanes;
  const int turned = p.interleaved ? 0 : p.half >> 3;  // lanes whose vectors are a half apart
  const int va = l < turned ? l : 2 * l, vb = l < turned ? l + turned : 2 * l + 1;
  auto kind_of = [&](int step) { return step < p.q_steps ? 0 : step < p.q_steps + p.k_steps ? 1 : 2; };  // q, k, v
  auto head_of = [&](int step, int kind) {
    return (step - (kind == 0 ? 0 : kind == 1 ? p.q_steps : p.q_steps + p.k_steps)) * kRows + sub;
  };
  // the next step's rows: this lane's row of it, rows of the kind that are left from it on, and
  // the kind's pitch between steps
  uint4 raw[2], next[2];
  const uint16_t* row_in = nullptr;
  int64_t pitch_in = 0;
  int left_in = 0, kind_in = -1;
  auto load = [&](int step) {
    if (kind_of(step) != kind_in) {
      kind_in = kind_of(step);
      const int h = head_of(step, kind_in);
      const int64_t sh = kind_in == 0 ? p.q_sh : kind_in == 1 ? p.k_sh : p.v_sh;
      row_in = (kind_in == 0 ? p.q + t * p.q_st : kind_in == 1 ? p.k + t * p.k_st : p.v + t * p.v_st) + h * sh;
      pitch_in = sh * kRows;
      left_in = (kind_in == 0 ? p.Hq : p.Hkv) - h;
    }
    next[0] = next[1] = make_uint4(0u, 0u, 0u, 0u);
    if (left_in > 0) {
      next[0] = *reinterpret_cast<const uint4*>(row_in + va * 8);
      next[1] = *reinterpret_cast<const uint4*>(row_in + vb * 8);
    }
    row_in += pitch_in;
    left_in -= kRows;
  };
  load(first);

  int64_t dst = t;
  if (end > p.q_steps && p.slots != nullptr) {
    const int32_t s = p.slots[t];
    dst = s;
    if (s < -1 || s >= p.rows) {
      if (lane == 0 && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      dst = -1;
    }
  }
  if (p.half > 0 && first < p.q_steps + p.k_steps) {
    for (int i = lane; i < p.half; i += 32) {
      int a = 0;
      while (i >= p.axis_end[a]) ++a;  // axis_end[axes - 1] = half
      // the angle in whole turns, reduced in 64 bits: position * inv_freq has up to 55 bits
      const double turns = double(p.pos[a * p.pos_stride + t]) * double(p.inv_freq[i]) *
                           0.15915494309189533576888;  // 1 / (2 pi)
      float s, c;
      sincospif(2.0f * float(turns - rint(turns)), &s, &c);
      sTurn[warp][i] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    __syncwarp();
  }
  // this lane's pairs: halves, pair 8 va + e is (a[e], b[e]); neighbours, pair 4 va + e is
  // (a[2 e], a[2 e + 1]) and pair 4 vb + e is (b[2 e], b[2 e + 1])
  const bool turns_a = p.interleaved ? va * 4 < p.half : l < turned;
  const bool turns_b = p.interleaved && vb * 4 < p.half;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = !p.interleaved ? va * 8 + e : e < 4 ? va * 4 + e : vb * 4 + e - 4;
    const float2 cs = turns_a && i < p.half ? sTurn[warp][i] : make_float2(1.f, 0.f);
    c[e] = cs.x;
    s[e] = cs.y;
  }

  int kind = -1, left = 0;
  const uint16_t* w = nullptr;
  uint8_t* row = nullptr;
  int64_t pitch = 0;
  uint64_t wa[4], wb[4];
  for (int step = first; step < end; ++step) {
    raw[0] = next[0], raw[1] = next[1];
    if (step + 1 < end) load(step + 1);
    if (kind_of(step) != kind) {  // the weights and destinations of this kind of rows
      kind = kind_of(step);
      const int h = head_of(step, kind);
      const int64_t sh = kind == 0 ? p.qo_sh * 2 : kind == 1 ? p.kd_sh : p.vd_sh;
      row = (kind == 0   ? reinterpret_cast<uint8_t*>(p.q_out + t * p.qo_st)
             : kind == 1 ? p.k_dst + dst * p.kd_ss
                         : p.v_dst + dst * p.vd_ss) + h * sh;
      pitch = sh * kRows;
      left = kind == 0 ? p.Hq - h : dst >= 0 ? p.Hkv - h : 0;
      w = kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr;
      if (w != nullptr) {
        const uint64_t offset2 = pack2(p.offset, p.offset);
        bf16x8_to_pairs(*reinterpret_cast<const uint4*>(w + va * 8), wa);
        bf16x8_to_pairs(*reinterpret_cast<const uint4*>(w + vb * 8), wb);
#pragma unroll
        for (int e = 0; e < 4; ++e) wa[e] = add2(wa[e], offset2), wb[e] = add2(wb[e], offset2);
      }
    }
    uint64_t a[4], b[4];
    bf16x8_to_pairs(raw[0], a);
    bf16x8_to_pairs(raw[1], b);
    if (w != nullptr) {
      uint64_t sq = mul2(a[0], a[0]), sq2 = mul2(b[0], b[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) sq = fma2(a[e], a[e], sq), sq2 = fma2(b[e], b[e], sq2);
      float ss, hi;
      unpack2(add2(sq, sq2), ss, hi);
      ss += hi;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
      const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = mul2(mul2(a[e], inv2), wa[e]);
        b[e] = mul2(mul2(b[e], inv2), wb[e]);
      }
    }
    if (kind != 2) {
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float u, v;
          unpack2(a[e], u, v);
          if (turns_a) a[e] = pack2(u * c[e] - v * s[e], v * c[e] + u * s[e]);
          unpack2(b[e], u, v);
          if (turns_b) b[e] = pack2(u * c[4 + e] - v * s[4 + e], v * c[4 + e] + u * s[4 + e]);
        }
      } else if (turns_a) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t c2 = pack2(c[2 * e], c[2 * e + 1]), s2 = pack2(s[2 * e], s[2 * e + 1]);
          const uint64_t n2 = pack2(-s[2 * e], -s[2 * e + 1]), u = a[e];
          a[e] = fma2(u, c2, mul2(b[e], n2));
          b[e] = fma2(b[e], c2, mul2(u, s2));
        }
      }
    }
    if (left > 0) {
      if (kind != 0 && p.kv_fp8) {
        const float scale = kind == 1 ? p.inv_k_scale : p.inv_v_scale;
        const uint64_t scale2 = pack2(scale, scale);
        *reinterpret_cast<uint2*>(row + va * 8) = pairs_to_e4m3x8(a, scale2);
        *reinterpret_cast<uint2*>(row + vb * 8) = pairs_to_e4m3x8(b, scale2);
      } else {
        *reinterpret_cast<uint4*>(row + va * 16) = pairs_to_bf16x8(a);
        *reinterpret_cast<uint4*>(row + vb * 16) = pairs_to_bf16x8(b);
      }
    }
    row += pitch;
    left -= kRows;
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
// 65,536 blocks of 4 keys of 128 (76 MB): 20 us, 0.58 of the copy rate; the chain of a
// block's number, its keys and the maximum is what the rest waits for.
constexpr int kPackThreads = 128;
template <int DI>
__global__ void __launch_bounds__(kPackThreads) qsa_pack_index_kernel(const PackParams p) {
  constexpr int kLanes = DI / 8;
  begin_kernel();
  const int64_t i = (int64_t(blockIdx.x) * kPackThreads + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes;
  int64_t b = -1;
  if (i < p.n) {
    b = p.blocks[i];
    if (b < -1 || b >= p.n_blocks) {
      if (l == 0 && p.err_word != nullptr) atomicOr(p.err_word, QSA_ERRBIT_SLOT_RANGE);
      b = -1;
    }
  }
  uint64_t sum2[4] = {0u, 0u, 0u, 0u};  // two sums each
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
        uint64_t x[4];
        bf16x8_to_pairs(raw[e], x);
#pragma unroll
        for (int d = 0; d < 4; ++d) sum2[d] = e0 + e == 0 ? x[d] : add2(sum2[d], x[d]);
      }
    }
  }
  float sum[8];
  if ((p.block & (p.block - 1)) == 0) {  // the product with a power of two's reciprocal is the quotient
    const float inv = 1.0f / float(p.block);
#pragma unroll
    for (int d = 0; d < 4; ++d) unpack2(mul2(sum2[d], pack2(inv, inv)), sum[2 * d], sum[2 * d + 1]);
  } else {
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      float x[2];
      unpack2(sum2[d >> 1], x[0], x[1]);
      sum[d] = __fdiv_rn(x[d & 1], float(p.block));
    }
  }
  uint32_t top = top_bits(sum);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (b < 0) return;
  const float scale = code_scale(__uint_as_float(top));
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
  if (kv_fp8 && !(k_scale > 0.f && std::isfinite(1.0f / k_scale) && std::isfinite(k_scale) && v_scale > 0.f &&
                  std::isfinite(1.0f / v_scale) && std::isfinite(v_scale)))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite, and so their reciprocals");
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
  const bool no_pool = rows == 0 && slots != nullptr;  // of no row: every token is dropped, the pool may be NULL
  if (Hkv > 0 && (k == nullptr || (k_dst == nullptr && !no_pool)))
    QSA_REJECT(QSA_ERR_INVALID_ARG, "NULL k or k_dst");
  if (((v == nullptr) != (v_dst == nullptr) && !no_pool) || (v != nullptr && Hkv == 0))
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
  p.inv_k_scale = 1.0f / k_scale, p.inv_v_scale = 1.0f / v_scale, p.kv_fp8 = kv_fp8;
  int dev = 0, num_sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return launch_status(e, "qsa_qk_norm_rope");
  // A warp takes a whole token once that makes 32 warps for every SM (of which 20 run at a time),
  // else as many steps as do, at least two (it makes its token's sines and cosines, about the
  // work of three steps).
  const int per_step = 512 / D;
  p.q_steps = (Hq + per_step - 1) / per_step;
  p.k_steps = k != nullptr ? (Hkv + per_step - 1) / per_step : 0;
  p.v_steps = v != nullptr ? (Hkv + per_step - 1) / per_step : 0;
  const int64_t all = p.q_steps + p.k_steps + p.v_steps;
  const int64_t warps = int64_t(num_sms) * 32;
  int64_t steps = (int64_t(T) * all + warps - 1) / warps;
  steps = steps < 2 ? 2 : steps;
  p.parts = int32_t((all + steps - 1) / steps);
  p.steps = int32_t((all + p.parts - 1) / p.parts);
  p.units = int64_t(T) * p.parts;
  const int64_t grid = (p.units + kRopeWarps - 1) / kRopeWarps;
  if (grid > INT32_MAX) QSA_REJECT(QSA_ERR_UNSUPPORTED, "%lld thread blocks in one launch", (long long)grid);
  const auto st = static_cast<cudaStream_t>(stream);
  const auto kernel = D == 256   ? qsa_norm_rope_kernel<256>
                      : D == 128 ? qsa_norm_rope_kernel<128>
                                 : qsa_norm_rope_kernel<64>;
  return launch_status(launch(kernel, unsigned(grid), 32 * kRopeWarps, 0, st, p), "qsa_qk_norm_rope");
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
  const int per = kPackThreads / (Di / 8);
  const int grid = int((int64_t(n) + per - 1) / per);
  const auto st = static_cast<cudaStream_t>(stream);
  const auto kernel = Di == 128 ? qsa_pack_index_kernel<128> : qsa_pack_index_kernel<64>;
  return launch_status(launch(kernel, grid, kPackThreads, 0, st, p), "qsa_pack_index_keys");
}
