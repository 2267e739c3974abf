// OCP MXFP8 (E4M3 codes, an E8M0 scale per 32 elements) on the device: the
// format of the 8-bit activation checkpoints.
#pragma once
#include "device.h"

namespace nvfp4 {

// E8M0 byte (2^(byte - 127)) for a block whose largest finite magnitude has
// the bf16 bits m: the smallest power of two with magnitude <= 448 * 2^E
// (448 = 1.75 * 2^8), at least 2^-117, so that the smallest E4M3 step times
// the scale, 2^-9 * 2^-117, is still a normal bf16.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t m) {
  const int e = (int)(m >> 7) - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
  return (uint32_t)(e < 10 ? 10 : e);
}

__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 codes times their scale -> 8 bf16 values, exact (4 significant bits): one
// hardware conversion per pair, which applies the scale's power of two
__device__ __forceinline__ u32x4 mx_decode8(uint2 c, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, true))};
}

}  // namespace nvfp4
