// The 8-bit key/value cache: page layout, codes and scales (device side).
//
// A page of 32 tokens of one head is one 32 x 32 tile of the matrix
// instructions per 32 channels, so tokens sit where the operands of
// v_mfma_f32_32x32x16 want them (lane = 32 h + i):
//   keys:   lane (h, token i) holds 16 consecutive channels of one 16-byte
//           piece: element 16 c' + j of piece c' = 2 c + h;
//   values: lane (h, channel i) holds 16 tokens of one 16-byte piece, in the
//           order in which the scores of those tokens sit in its accumulator
//           registers: byte 4 g + i of half h is token 8 g + 4 h + i.
// Every wave load of a page is then 1 KiB contiguous, and neither keys, nor
// values, nor the weights between the two products cross lanes.
#pragma once

#include "common.h"

namespace dllm {

constexpr int kPage = DLLM_KV_PAGE;
constexpr int kScaleMin = -100;     // smallest and largest scale exponents
constexpr int kScaleMax = 119;      // 448 * 2^119 is finite
constexpr float kFp8Max = 448.0f;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// The page holding tokens 32 p .. of a table row, or -1.
__device__ __forceinline__ int64_t page_of(const int32_t *row, int64_t p, int64_t num_pages) {
  const int64_t id = row[p];
  return id >= 0 && id < num_pages ? id : -1;
}

// A length cut to what the table can hold.
__device__ __forceinline__ int64_t cut_len(int64_t n, int64_t max_pages) {
  return n < 0 ? 0 : n > max_pages * kPage ? max_pages * kPage : n;
}

// Exponent of the smallest power of two s in [2^-100, 2^119] with
// amax <= 448 s (2^119 beyond that), for a finite amax >= 0: with amax = m 2^e, 1 <= m < 2, and 448 = 1.75 * 2^8, s is
// 2^(e - 8), or twice that when m > 1.75.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kScaleMin), kScaleMax);
}
// Exponent of a stored scale, whatever the bits are (an unwritten page's may
// be anything): in the range that scale_exp gives.
__device__ __forceinline__ int stored_exp(float s) {
  const int e = (int)((__float_as_uint(s) >> 23) & 0xffu) - 127;
  return min(max(e, kScaleMin), kScaleMax);
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four values, already divided by the scale, as codes: to nearest, ties to
// even, +-inf to +-448.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  a = fminf(fmaxf(a, -kFp8Max), kFp8Max);
  b = fminf(fmaxf(b, -kFp8Max), kFp8Max);
  c = fminf(fmaxf(c, -kFp8Max), kFp8Max);
  d = fminf(fmaxf(d, -kFp8Max), kFp8Max);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}
// Four codes in another scale: values times 2^shift (a zero stays zero
// whatever the shift is).
__device__ __forceinline__ uint32_t recode4(uint32_t w, int shift) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return encode4(__builtin_amdgcn_ldexpf(lo.x, shift), __builtin_amdgcn_ldexpf(lo.y, shift),
                 __builtin_amdgcn_ldexpf(hi.x, shift), __builtin_amdgcn_ldexpf(hi.y, shift));
}
// |value| of the largest of four codes (NaN codes as 0).
__device__ __forceinline__ float amax4(uint32_t w) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return fmaxf(fmaxf(fabsf(lo.x), fabsf(lo.y)), fmaxf(fabsf(hi.x), fabsf(hi.y)));
}

}  // namespace dllm
