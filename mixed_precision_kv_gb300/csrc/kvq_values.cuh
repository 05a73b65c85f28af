// One cached value at a time, in fp32: code * scale + zero of (slot, channel) of a page block.
#pragma once
#include <cuda_fp16.h>

#include "kvq_attend.h"

namespace kvq {
namespace {

__device__ __forceinline__ float half_at(const uint8_t* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }

__device__ float k_value(const uint8_t* b, int cls, int t, int c) {
  const int gr = c >> 5;
  if (cls == kClsInt2) {
    const int mi = i2k_meta_index(c);
    return fmaf((float)((b[i2k_byte(t, c)] >> i2k_shift(c)) & 3u), half_at(b + kI2KMeta + 2 * mi),
                half_at(b + kI2KMeta + 256 + 2 * mi));
  }
  if (cls == kClsFp4)
    return e2m1_value(((uint32_t)b[f4k_byte(t, c)] >> f4k_shift(c)) & 15u) * half_at(b + kF4KScale + 8 * t + 2 * gr);
  const uint8_t* m = b + (cls == kClsInt3 ? kI3KMeta : kI4KMeta) + 16 * t + 4 * gr;
  const uint32_t code = cls == kClsInt3 ? (((uint32_t)b[i3k_lo_byte(t, c)] >> i3k_lo_shift(c)) & 3u) |
                                              ((((uint32_t)b[i3k_hi_byte(t, c)] >> i3k_hi_shift(c)) & 1u) << 2)
                                        : ((uint32_t)b[i4k_byte(t, c)] >> i4k_shift(c)) & 15u;
  return fmaf((float)code, half_at(m), half_at(m + 2));
}
__device__ float v_value(const uint8_t* b, int cls, int t, int c) {
  const int mi = v_meta_index(t, c >> 5);
  if (cls == kClsFp4)
    return e2m1_value(((uint32_t)b[f4v_byte(t, c)] >> f4v_shift(t)) & 15u) * half_at(b + kF4VScale + 2 * mi);
  const uint8_t* m = b + (cls == kClsInt2 ? kI2VMeta : (cls == kClsInt3 ? kI3VMeta : kI4VMeta));
  const uint32_t code = cls == kClsInt2   ? ((uint32_t)b[i2v_byte(t, c)] >> i2v_shift(t)) & 3u
                        : cls == kClsInt3 ? (((uint32_t)b[i3v_lo_byte(t, c)] >> i3v_lo_shift(t)) & 3u) |
                                                ((((uint32_t)b[i3v_hi_byte(t, c)] >> i3v_hi_shift(t, c)) & 1u) << 2)
                                          : ((uint32_t)b[i4v_byte(t, c)] >> i4v_shift(t)) & 15u;
  return fmaf((float)code, half_at(m + 2 * mi), half_at(m + 256 + 2 * mi));
}

}  // namespace
}  // namespace kvq
