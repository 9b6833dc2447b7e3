// qsa_layer.cuh -- shared by the layer operators (qsa_rope.cu, qsa_select.cu,
// qsa_decode.cu): host-side argument helpers and small device functions.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "qsa_internal.h"
#include "qsa_layer.h"
#include "qsa_ptx.cuh"

namespace qsa {

#define QSA_REJECT(status, ...)     \
  do {                              \
    qsa::set_error_detail(__VA_ARGS__); \
    return status;                  \
  } while (0)

inline bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// a stride of `elem`-byte elements: non-negative and a multiple of `bytes`
inline bool stride_multiple(int64_t s, int64_t elem, int64_t bytes) {
  return s >= 0 && s <= INT64_MAX / 16 && (s * elem) % bytes == 0;
}

// The status of a launch sequence: reports the runtime's error and clears it.
inline qsa_status_t launch_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return QSA_OK;
  set_error_detail("%s: %s", what, cudaGetErrorString(e));
  (void)cudaGetLastError();
  return QSA_ERR_CUDA;
}

// Every kernel of these operators is launched while the one before it in its stream may still
// run, and begins by waiting for that one's end and letting the next one be launched: the
// launch and the scheduling of its thread blocks then overlap (64 blocks of index keys: 4.1 us
// a call without, 3.0 with).  Nothing in global memory is touched before the wait, except
// by the second kernel of a call (launch_next, then wait_for_last): the first one let it be
// launched after its own wait, so all that the call's inputs depend on has ended by then.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void begin_kernel() {
  wait_for_last();
  launch_next();
}

// What an earlier kernel of the stream wrote is read after that wait, by plain loads, or by
// these, which pass the L1 by; never by the read-only path (__ldg), which is defined only for
// memory that nobody writes while the kernel exists, and a kernel launched early exists while
// the one before it still writes.  The asm is volatile: it stays behind the wait.
__device__ __forceinline__ float load_l2(const float* p) {
  float x;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(x) : "l"(__cvta_generic_to_global(p)));
  return x;
}
__device__ __forceinline__ uint4 load_l2(const uint4* p) {
  uint4 x;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(__cvta_generic_to_global(p)));
  return x;
}
__device__ __forceinline__ float4 load_l2(const float4* p) {
  const uint4 x = load_l2(reinterpret_cast<const uint4*>(p));
  return make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
}

// Lets a kernel have as much dynamic shared memory as the device gives a block beside the
// kernel's own.  The limit is shared by all host threads: were it set to what one call needs, a
// smaller call of another thread would lower it between that and the launch.  Set once in each
// context (`done`: one per kernel, by device).
inline cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t> (&done)[64]) {
  int dev = 0, most = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  const uint64_t context = current_context_id();
  if (known && context != 0 && done[dev].load(std::memory_order_acquire) == context) return cudaSuccess;
  cudaFuncAttributes own{};
  if ((e = cudaFuncGetAttributes(&own, kernel)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - int(own.sharedSizeBytes));
  if (e != cudaSuccess) return e;
  const uint64_t now = current_context_id();  // (the first call made the context current)
  if (known && now != 0) done[dev].store(now, std::memory_order_release);
  return cudaSuccess;
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// D = A(16x32, row) * B(32x8, col) + D, int8 inputs, int32 accumulators.
__device__ __forceinline__ void mma_s8_16832(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight bf16 values from 16 bytes.
__device__ __forceinline__ void bf16x8_to_f32(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(w[i]);
    x[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}

// Two floats -> two E4M3 codes (round to nearest even, saturated); `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The scale of int8 codes whose largest magnitude is `top`; NaN when that is not finite.
__device__ __forceinline__ float code_scale(float top) {
  const float s = __fdiv_rn(top, 127.f);
  return s < __builtin_huge_valf() ? s : __int_as_float(0x7fffffff);
}

// Largest magnitude of eight values, as the bits of a non-negative float (in whose order a
// NaN is above infinity); combined across lanes by an unsigned maximum.
__device__ __forceinline__ uint32_t top_bits(const float (&x)[8]) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  return top;
}

// int8 codes of eight values over a scale: the 32-bit quotient rounded half to even, so every
// caller gets the same codes; zeros when the scale is not a positive finite number.  The
// product with the reciprocal is within 127 * 3 * 2^-24 of the quotient (at most 127 in
// magnitude), so it rounds to the same code unless it lies that close to a half: only then
// are the quotients themselves taken; also over a subnormal scale, whose reciprocal may overflow
// and which may be so far below a 127th of the largest value that a quotient has to be held to
// 127.  Adding 1.5 * 2^23 rounds to a whole number and leaves it in the low bits.
__device__ __forceinline__ uint2 int8x8_codes(const float (&x)[8], float scale) {
  if (!(scale > 0.f && scale < __builtin_huge_valf())) return make_uint2(0u, 0u);
  const float inv = __frcp_rn(scale);
  uint32_t c[8];
  bool close = scale < 0x1p-126f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = __fmul_rn(x[i], inv), t = __fadd_rn(q, 12582912.f);
    close |= !(fabsf(q - __fsub_rn(t, 12582912.f)) < 0.5f - 0x1p-13f);
    c[i] = __float_as_uint(t);
  }
  if (close) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float v = x[0];  // x[i], without an index into registers
#pragma unroll
      for (int k = 1; k < 8; ++k) v = i == k ? x[k] : v;
      const float ratio = fminf(fmaxf(__fdiv_rn(v, scale), -127.f), 127.f);
      const uint32_t q = __float_as_uint(__fadd_rn(ratio, 12582912.f));
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = i == k ? q : c[k];
    }
  }
  return make_uint2(byte_perm(byte_perm(c[0], c[1], 0x0040u), byte_perm(c[2], c[3], 0x0040u), 0x5410u),
                    byte_perm(byte_perm(c[4], c[5], 0x0040u), byte_perm(c[6], c[7], 0x0040u), 0x5410u));
}

__device__ __forceinline__ uint64_t clock_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  return t;
}

// Waits for a phase of an mbarrier, `limit` ns at most; false when it has not come by then.
// The hint lets the hardware hold the thread for up to 100 us, or until the phase completes,
// instead of a few cycles: waiting warps would otherwise take issue slots from working ones.
constexpr uint32_t kWaitLimit = 1000000000u;  // one second
__device__ __forceinline__ bool poll_phase(uint32_t bar, uint32_t parity, uint32_t hint) {
  uint32_t done;
  asm volatile(
      "{\n  .reg .pred p;\n  mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      "  selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(hint)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint32_t limit = kWaitLimit) {
  const uint32_t hint = min(limit, 100000u);
  if (poll_phase(bar, parity, hint)) return true;
  const uint64_t start = clock_ns();
  do {
    if (poll_phase(bar, parity, hint)) return true;
  } while (clock_ns() - start < limit);
  return false;
}

// Bulk copy from this device's memory to shared memory, completing on an mbarrier; both
// addresses 16-byte aligned, the size a multiple of 16.  No multicast.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// Two floats per instruction, each operation rounded as the scalar one; but the compiler fuses
// a mul2 and the add2 of its result, .rn or not: where a product has to be rounded by itself
// before a sum, it is an fma2 with +0.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

}  // namespace qsa
