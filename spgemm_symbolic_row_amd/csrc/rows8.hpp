// Rows kept in 8 bits: blocks of 128 columns share a power of two s = 2^e, the
// smallest with max |x| <= 448 s over the block's finite values, and hold x / s
// rounded to e4m3 (to nearest, ties to even).  s is no smaller than 2^-15 (fp16)
// or 2^-117 (bf16, fp32), and where s = 2^(top exponent of x's type - 7) the code
// ends at 240: so code * s is a normal number of x's type or zero, exact there.
// What is not finite is held as NaN.  The code depends on x's bits alone: every
// step but the one rounding is exact.
//
// Half a step of e4m3 is 2^-4 of the value down to 2^-6 s, and below that the error is
// at most 2^-10 s.  Where s is above its floor, 448 s < 2 max: the two are less than
// max / 14336 and max / 229376 of the block's maximum.
//
// A lane holds 8 neighbouring columns, so 16 lanes hold a block: its maximum is
// four DPP steps inside a row of lanes.
#pragma once
#include "expert_common.hpp"

namespace sg {

constexpr int kKeptBlock = 128;

// Row pitch of the codes, and scales to a row.
__host__ __device__ inline int64_t kept_pitch(int64_t D) { return (D + 7) / 8 * 8; }
__host__ __device__ inline int64_t kept_blocks(int64_t D) {
  return (D + kKeptBlock - 1) / kKeptBlock;
}

template <typename T>
struct KeptRange {
  static constexpr int kLow = sizeof(T) == 2 && !__is_same(T, __bf16) ? -15 : -117;
  static constexpr int kTop = sizeof(T) == 2 && !__is_same(T, __bf16) ? 8 : 120;
};

// Codes of 8 columns (zeros outside the row) and the block's e + 127.  All 16
// lanes of a block call it together.
template <typename T>
__device__ __forceinline__ uint2 kept_encode(const float v[8], uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
    m = max(m, b < 0x7f800000u ? b : 0u);
  }
  m = max(m, dpp_or_zero<0x128, 0xf>(m));  // row_ror:8
  m = max(m, dpp_or_zero<0x124, 0xf>(m));
  m = max(m, dpp_or_zero<0x122, 0xf>(m));
  m = max(m, dpp_or_zero<0x121, 0xf>(m));
  // 448 = 1.75 * 2^8.
  const int e = max((int)(m >> 23) - 135 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0),
                    KeptRange<T>::kLow);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  const float top = e == KeptRange<T>::kTop ? 240.0f : 448.0f;
  scale = (uint32_t)(e + 127);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool finite = (__float_as_uint(v[j]) & 0x7fffffffu) < 0x7f800000u;
    q[j] = finite ? fminf(fmaxf(v[j] * inv, -top), top) : __uint_as_float(0x7fc00000u);
  }
  uint32_t lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return uint2{lo, hi};
}

// 4 codes as fp32, without the scale.
__device__ __forceinline__ void decode4(uint32_t q, float v[4]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(q, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(q, true);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
}

__device__ __forceinline__ void kept_decode(uint2 q, uint32_t scale, float v[8]) {
  decode4(q.x, v);
  decode4(q.y, v + 4);
  const float s = __uint_as_float(scale << 23);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= s;
}

// 8 values from p, wherever it is aligned; those from n on are 0 and not read.
template <typename T>
__device__ __forceinline__ void load8_any(const T* p, int n, float v[8]) {
  if (n >= 8) {
    struct Pack { T v[8]; } q;
    __builtin_memcpy(&q, p, sizeof(q));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f32(q.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? to_f32(p[j]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store8_any(T* p, int n, const float v[8]) {
  if (n >= 8) {
    struct Pack { T v[8]; } q;
#pragma unroll
    for (int j = 0; j < 8; ++j) q.v[j] = from_f32<T>(v[j]);
    __builtin_memcpy(p, &q, sizeof(q));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = from_f32<T>(v[j]);
  }
}

// Rows of `ld` elements (bf16 or fp16) to rows of kept_pitch(D) codes and
// kept_blocks(D) scales, and back to rows of kept_pitch(D) elements.
void launch_rows_encode(spgemm_dtype type, int64_t rows, int64_t D, int64_t ld, const void* x,
                        uint8_t* code, uint8_t* scale, hipStream_t s);
void launch_rows_decode(spgemm_dtype type, int64_t rows, int64_t D, const uint8_t* code,
                        const uint8_t* scale, void* x, hipStream_t s);

}  // namespace sg
