// Device helpers of the microscaled 4-bit format (include/mxfp4.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "topk_wave.h"

namespace moe {

constexpr int kMxBlock = 32;    // values that share a scale
constexpr int kMxPad = 256;     // columns a row is padded to: 128 bytes of codes

__host__ __device__ inline int64_t mx_padded(int64_t cols) { return (cols + kMxPad - 1) / kMxPad * kMxPad; }

// Scale byte of a block from the bits of its largest magnitude: the exponent
// field less that of 4 (E2M1's largest power of two), at least 0 (2^-127);
// 255 for a block with an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t mag_bits) {
  const uint32_t f = mag_bits >> 23;
  return f >= 255u ? 255u : (f > 2u ? f - 2u : 0u);
}

// The power of two that a scale byte stands for (NaN for 255).  2^-127 is a
// subnormal fp32 number.
__device__ __forceinline__ float mx_scale_f32(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7fc00000u : byte << 23));
}

// Eight values of a row as they are stored: fp32, or pairs of bf16.
template <int DT>
struct Eight {
  uint32_t w[DT == kF32 ? 8 : 4];
};

// Eight values from element c of a row of `cols`; zeros past its end.  The
// row's start is aligned to the element only.
template <int DT>
__device__ __forceinline__ void mx_load8(const void* base, int64_t row, int64_t c, int64_t cols, Eight<DT>& v) {
  constexpr int kWords = DT == kF32 ? 8 : 4;
  if constexpr (DT == kF32) {
    const float* p = static_cast<const float*>(base) + row;
    if (c + 8 <= cols) __builtin_memcpy(v.w, p + c, 32);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) v.w[i] = c + i < cols ? __float_as_uint(p[c + i]) : 0u;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row;
    if (c + 8 <= cols) __builtin_memcpy(v.w, p + c, 16);
    else
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        v.w[i] = (c + 2 * i < cols ? p[c + 2 * i] : 0u) | ((c + 2 * i + 1 < cols ? p[c + 2 * i + 1] : 0u) << 16);
  }
}

// The largest magnitude's fp32 bits (as whole numbers NaN > inf > any number).
template <int DT>
__device__ __forceinline__ uint32_t mx_mag8(const Eight<DT>& v) {
  if constexpr (DT == kF32) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = v.w[i] & 0x7fffffffu;
      m = b > m ? b : m;
    }
    return m;
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v.w[i] & 0x7fff7fffu));
    return static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16;
  }
}

// Eight values over the block's power of two as eight codes, the first in the
// lowest four bits.  The conversions divide by the power exactly, round to
// nearest with ties to even and saturate at 6 (checked against the formula
// over all exponents); a block of scale byte 255 gets zero codes.
template <int DT>
__device__ __forceinline__ uint32_t mx_codes8(const Eight<DT>& v, uint32_t byte) {
  const float s = mx_scale_f32(byte);
  uint32_t c = 0;
  if constexpr (DT == kF32) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[0]), __uint_as_float(v.w[1]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[2]), __uint_as_float(v.w[3]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[4]), __uint_as_float(v.w[5]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[6]), __uint_as_float(v.w[7]), s, 3);
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[3]), s, 3);
  }
  return byte == 255u ? 0u : c;
}

// Piece p (eight values) of the padded matrix -> its row and column.
struct Piece {
  int64_t row;
  int64_t col;
};

__device__ __forceinline__ Piece piece_at(int64_t p, uint32_t per_row) {
  const int64_t r = (p >> 31) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(p) / per_row) : p / per_row;
  return {r, (p - r * per_row) * 8};
}

// One piece of a row-major matrix quantised; the four lanes of a block call it
// together.
template <int DT>
__device__ __forceinline__ void mx_quantize_piece(const void* x, int64_t stride, int64_t cols, uint32_t per_row, int64_t p,
                                                  int64_t pieces, uint32_t* codes, uint8_t* scales) {
  if (p >= pieces) return;   // pieces of a block are whole: per_row is a multiple of 32
  const int lane = threadIdx.x & (kWave - 1);
  const Piece at = piece_at(p, per_row);
  Eight<DT> v;
  mx_load8<DT>(x, at.row * stride, at.col, cols, v);
  uint32_t m = mx_mag8(v);
  uint32_t o = lane_xor<1>(m, lane);
  m = o > m ? o : m;
  o = lane_xor<2>(m, lane);
  m = o > m ? o : m;
  const uint32_t byte = mx_scale_byte(m);
  codes[p] = mx_codes8(v, byte);
  if ((lane & 3) == 0) scales[p >> 2] = static_cast<uint8_t>(byte);
}

}  // namespace moe
