// Microscaled 4-bit quantisation and its inverse (include/mxfp4.h).
//
// Bound by HBM: 2 or 4 bytes a value on one side, 17/32 byte on the other, a
// handful of instructions each.  Four lanes share a block of 32 values, eight
// values a lane, so that a wave's 16-byte loads and 4-byte stores are
// contiguous; the block's largest magnitude takes two lane exchanges.  A
// thread handles kIter such pieces, kQThr pieces apart, all requested before
// any is used.  131072 x 2048 bf16 values take 148 us to quantise (4.6 TB/s; a
// copy of 4 GiB reaches 4.7, one of 0.5 GiB 5.3) and 105 us back (6.5 TB/s,
// part of it out of and into the last-level cache); 8 x 2048 take 2.5 and 2.3
// us, an empty kernel's time.
#include <hip/hip_runtime.h>

#include <cstdio>

#include "mx_common.h"
#include "mx_internal.h"
#include "topk_wave.h"

namespace moe {
namespace {

constexpr int kQThr = 256;
constexpr int kIter = 4;

template <int DT>
__global__ __launch_bounds__(kQThr) void k_mx_quantize(const void* x, int64_t stride, int64_t cols, uint32_t per_row,
                                                       int64_t pieces, uint32_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (kQThr * kIter) + threadIdx.x;
  Eight<DT> v[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int64_t p = p0 + i * kQThr;
    const Piece at = piece_at(p < pieces ? p : 0, per_row);
    if (p < pieces) mx_load8<DT>(x, at.row * stride, at.col, cols, v[i]);
    else v[i] = Eight<DT>{};
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int64_t p = p0 + i * kQThr;
    uint32_t m = mx_mag8(v[i]);
    uint32_t o = lane_xor<1>(m, lane);
    m = o > m ? o : m;
    o = lane_xor<2>(m, lane);
    m = o > m ? o : m;
    const uint32_t byte = mx_scale_byte(m);
    if (p < pieces) {   // pieces of a block are whole: per_row is a multiple of 32
      codes[p] = mx_codes8(v[i], byte);
      if ((lane & 3) == 0) scales[p >> 2] = static_cast<uint8_t>(byte);
    }
  }
}

// The value of one code over the exact power of two: both factors are exact in
// fp32 and so is their product (subnormals included); in bf16 too, since a
// code has two significant bits.
__device__ __forceinline__ void mx_values8(uint32_t c, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    f32x2 r;
    if (i == 0) r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    else if (i == 1) r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    else if (i == 2) r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    else r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[2 * i] = r[0] * s;
    v[2 * i + 1] = r[1] * s;
  }
}

template <int DT>
__global__ __launch_bounds__(kQThr) void k_mx_dequantize(const uint32_t* codes, const uint8_t* scales, int64_t cols,
                                                         uint32_t per_row, int64_t pieces, void* out, int64_t stride) {
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (kQThr * kIter) + threadIdx.x;
  uint32_t c[kIter], b[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int64_t p = p0 + i * kQThr;
    c[i] = p < pieces ? codes[p] : 0u;
    b[i] = p < pieces ? scales[p >> 2] : 0u;
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int64_t p = p0 + i * kQThr;
    if (p >= pieces) continue;
    const Piece at = piece_at(p, per_row);
    float v[8];
    mx_values8(c[i], mx_scale_f32(b[i]), v);
    if constexpr (DT == kF32) {
      float* o = static_cast<float*>(out) + at.row * stride + at.col;
      if (at.col + 8 <= cols) {
        __builtin_memcpy(o, v, 32);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at.col + j < cols) o[j] = v[j];
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(out) + at.row * stride + at.col;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xffff0000u);
      if (at.col + 8 <= cols) {
        __builtin_memcpy(o, w, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at.col + j < cols) o[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
      }
    }
  }
}

int bad(const char* fmt, long long x = 0, long long y = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, x, y);
  return api_fail(MOE_EINVAL, buf);
}

bool at(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_matrix(int32_t dtype, int64_t rows, int64_t cols, const void* x, int64_t stride, const void* codes,
                 const void* scales) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return bad("dtype=%lld is neither MOE_F32 nor MOE_BF16", dtype);
  if (mx_codes_bytes(rows, cols) < 0) return bad("rows=%lld must be in [0, 2^31), cols=%lld in [0, 2^20]", rows, cols);
  if (rows == 0 || cols == 0) return MOE_OK;
  // the last row's place in bytes has to fit 64 bits
  if (rows > 1 && (stride < cols || stride > (int64_t(1) << 56) / (rows - 1)))
    return bad("row stride %lld is smaller than cols=%lld or too large", stride, cols);
  if (!x || !codes || !scales) return bad("NULL pointer argument");
  const int64_t sz = dtype == MOE_F32 ? 4 : 2;
  if (!at(x, sz) || !at(codes, 16) || !at(scales, 16))
    return bad("codes and scales must be 16-byte aligned, the values to their %lld bytes", sz);
  const int64_t n_x = ((rows - 1) * stride + cols) * sz, n_c = mx_codes_bytes(rows, cols), n_s = mx_scales_bytes(rows, cols);
  if (mx_overlaps(x, n_x, codes, n_c) || mx_overlaps(x, n_x, scales, n_s) || mx_overlaps(codes, n_c, scales, n_s))
    return bad("the values, codes and scales overlap");
  return MOE_OK;
}

int launched() {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return api_ok();
  char buf[256];
  snprintf(buf, sizeof(buf), "launch failed: %s", hipGetErrorString(e));
  return api_fail(MOE_EHIP, buf);
}

}  // namespace

void launch_mx_quantize(int dtype, int64_t rows, int64_t cols, const void* x, int64_t stride, void* codes,
                        void* scales, hipStream_t s) {
  const uint32_t per_row = static_cast<uint32_t>(mx_padded(cols) / 8);
  const int64_t pieces = rows * per_row;
  const dim3 grid(static_cast<uint32_t>((pieces + kQThr * kIter - 1) / (kQThr * kIter))), block(kQThr);
  if (dtype == MOE_F32)
    launch_kernel(k_mx_quantize<kF32>, grid, block, 0, s, x, stride, cols, per_row, pieces, static_cast<uint32_t*>(codes),
                  static_cast<uint8_t*>(scales));
  else
    launch_kernel(k_mx_quantize<kBF16>, grid, block, 0, s, x, stride, cols, per_row, pieces, static_cast<uint32_t*>(codes),
                  static_cast<uint8_t*>(scales));
}

}  // namespace moe

extern "C" {

int64_t mx_codes_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || rows >= (int64_t(1) << 31) || cols < 0 || cols > (1 << 20)) return -1;
  return rows * (moe::mx_padded(cols) / 2);
}

int64_t mx_scales_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || rows >= (int64_t(1) << 31) || cols < 0 || cols > (1 << 20)) return -1;
  return rows * (moe::mx_padded(cols) / moe::kMxBlock);
}

int mx_quantize(int32_t dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* codes, void* scales,
                void* stream) {
  using namespace moe;
  MarkScope marks;
  if (const int rc = check_matrix(dtype, rows, cols, x, x_stride, codes, scales)) return rc;
  if (rows == 0 || cols == 0) return api_ok();
  if (rows * (mx_padded(cols) / 8) / kIter >= (int64_t(1) << 32) - 2048) return bad("rows * cols is too large for one launch");
  launch_mx_quantize(dtype, rows, cols, x, rows > 1 ? x_stride : 0, codes, scales, static_cast<hipStream_t>(stream));
  return launched();
}

int mx_dequantize(int32_t dtype, int64_t rows, int64_t cols, const void* codes, const void* scales, void* out,
                  int64_t out_stride, void* stream) {
  using namespace moe;
  MarkScope marks;
  if (const int rc = check_matrix(dtype, rows, cols, out, out_stride, codes, scales)) return rc;
  if (rows == 0 || cols == 0) return api_ok();
  const uint32_t per_row = static_cast<uint32_t>(mx_padded(cols) / 8);
  const int64_t pieces = rows * per_row, blocks = (pieces + kQThr * kIter - 1) / (kQThr * kIter);
  if (blocks * kQThr >= int64_t(1) << 32) return bad("rows * cols is too large for one launch");
  const dim3 grid(static_cast<uint32_t>(blocks)), block(kQThr);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t st = rows > 1 ? out_stride : 0;
  if (dtype == MOE_F32)
    launch_kernel(k_mx_dequantize<kF32>, grid, block, 0, s, static_cast<const uint32_t*>(codes),
                  static_cast<const uint8_t*>(scales), cols, per_row, pieces, out, st);
  else
    launch_kernel(k_mx_dequantize<kBF16>, grid, block, 0, s, static_cast<const uint32_t*>(codes),
                  static_cast<const uint8_t*>(scales), cols, per_row, pieces, out, st);
  return launched();
}

}  // extern "C"
