// Codes of the 8-bit K/V cache on the device: their formats, the power-of-two
// scale of a block, and the exact conversion of codes to bf16 pairs.
//
// A code's value is its format's value times the scale of its (block of
// tokens, head).  The scale is a power of two, so v / s is exact in fp32: the
// code of a value depends on the value and the scale alone, and a row that
// stays in a block is re-scaled without loss when the block's scale falls and
// rounded once when it grows.  (With s = max / qmax every change of scale
// would round every remaining row, and the cache rewrites scattered rows in
// every step.)  The price is up to one bit of an int8 code's range.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spa_device.cuh"

namespace spa {

constexpr int kQ8Int8 = 0, kQ8E4m3 = 1;

// Smallest power of two s >= 2^-126 with a <= qmax * s (0 for a = 0; a finite).
// 127 = 1.984375 * 2^6 and 448 = 1.75 * 2^8: compare mantissas, adjust exponents.
template <int FMT> __device__ __forceinline__ float q8_scale(float a) {
  if (!(a > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23);  // biased; 0 for a subnormal, which ends at the lower bound below
  const uint32_t m = u & 0x7FFFFFu;
  constexpr uint32_t mq = FMT == kQ8Int8 ? 0x7E0000u : 0x600000u;
  constexpr int eq = FMT == kQ8Int8 ? 6 : 8;
  int t = e - eq + (m > mq ? 1 : 0);
  if (t < 1) t = 1;  // 2^-126
  return __uint_as_float((uint32_t)t << 23);
}
// 1 / s of a scale q8_scale returned (2^-126 .. 2^122): exact.
__device__ __forceinline__ float q8_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Pair of bf16 from the two codes at byte positions 0 and 2 of t (bytes 1 and
// 3: anything for int8, the codes' sign bits for e4m3, as q8_pair makes them):
// exact, since a code has at most 8 significant bits.
//   int8:  0x4300 | (c & 0x7F) is 128 + (c & 0x7F) and 0x4300 | (c & 0x80) is
//          128 or 256; their difference is the signed value.
//   e4m3:  the 7 low bits at bf16's exponent and mantissa positions read as
//          the value times 2^-120 (subnormals included).
template <int FMT> __device__ __forceinline__ uint32_t q8_to_bf162_lo(uint32_t t) {
  __nv_bfloat162 r;
  if constexpr (FMT == kQ8Int8) {
    const uint32_t lo = (t & 0x007F007Fu) | 0x43004300u, hi = (t & 0x00800080u) | 0x43004300u;
    r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&hi));
  } else {
    const uint32_t w = (t << 4) & 0x87F087F0u;  // t's codes are sign-extended to 16 bits
    const uint32_t f = 0x7B807B80u;  // 2^120
    r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&f));
  }
  return *reinterpret_cast<uint32_t*>(&r);
}
// Codes i of x and of y (i = 0..3; 4..7: of the other word) at byte positions 0 and 2.
template <int FMT> __device__ __forceinline__ uint32_t q8_pair(uint32_t x, uint32_t y, int i, int j) {
  // a selector with bit 3 set replicates the byte's sign
  const uint32_t a = (uint32_t)i, b = (uint32_t)j;
  uint32_t r;  // prmt itself: __byte_perm leaves that bit out
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(a | ((a | 8u) << 4) | (b << 8) | ((b | 8u) << 12)));
  return r;
}
// Four codes of a word -> two bf16 pairs (bytes 0, 1 and bytes 2, 3).
template <int FMT> __device__ __forceinline__ void q8_word_to_bf16(uint32_t w, uint32_t& p01, uint32_t& p23) {
  p01 = q8_to_bf162_lo<FMT>(q8_pair<FMT>(w, w, 0, 1));
  p23 = q8_to_bf162_lo<FMT>(q8_pair<FMT>(w, w, 2, 3));
}

// The same to f16 pairs, times 2^-8 for e4m3 (which q8_f16_unit puts right):
// fewer instructions than to bf16, for operands whose range is under control.
//   int8:  0x6400 | (c + 128) is 1152 + c; minus 1152.
//   e4m3:  the 7 low bits at f16's exponent and mantissa positions.
template <int FMT> __device__ __forceinline__ float q8_f16_unit() { return FMT == kQ8Int8 ? 1.f : 256.f; }
template <int FMT> __device__ __forceinline__ uint32_t q8_pair_f16(uint32_t x, uint32_t y, int i, int j) {
  if constexpr (FMT == kQ8Int8) {
    const uint32_t t = (q8_pair<FMT>(x, y, i, j) & 0x00FF00FFu) ^ 0x64806480u, c = 0x64806480u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&t), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    return (q8_pair<FMT>(x, y, i, j) << 7) & 0xBF80BF80u;
  }
}

// Four codes of a word -> two f16 pairs.
template <int FMT> __device__ __forceinline__ void q8_word_to_f16(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if constexpr (FMT == kQ8Int8) {
    const uint32_t x = w ^ 0x80808080u, k = 0x64646464u, c = 0x64806480u;
    const uint32_t a = __byte_perm(x, k, 0x4140), b = __byte_perm(x, k, 0x4342);
    const __half2 h = *reinterpret_cast<const __half2*>(&c);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), h), t = __hsub2(*reinterpret_cast<const __half2*>(&b), h);
    p01 = *reinterpret_cast<const uint32_t*>(&r);
    p23 = *reinterpret_cast<const uint32_t*>(&t);
  } else {
    p01 = q8_pair_f16<FMT>(w, w, 0, 1);
    p23 = q8_pair_f16<FMT>(w, w, 2, 3);
  }
}

// Asynchronous copies to shared memory; bytes 0: zeros, src is not read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One code as float.
template <int FMT> __device__ __forceinline__ float q8_value(uint32_t byte) {
  if constexpr (FMT == kQ8Int8) return (float)(int8_t)(uint8_t)byte;
  __nv_fp8_e4m3 v;
  v.__x = (__nv_fp8_storage_t)byte;
  return (float)v;
}

}  // namespace spa
