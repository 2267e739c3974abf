// OCP MXFP4 (E2M1 codes, an E8M0 scale per 32 elements) on the device.
#pragma once
#include "device.h"

namespace nvfp4 {

constexpr uint32_t kMx4Nan = 255;   // E8M0's NaN: every value of the block is NaN

// E8M0 byte (2^(byte - 127)) for a block whose largest magnitude has the bf16
// bits m: the smallest power of two with magnitude <= 7 * 2^E (7 = 1.75 *
// 2^2), E from -125 to 125; NaN for a block with a NaN or an infinity.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t m) {
  int b = (int)(m >> 7) - 2 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
  b = b < 2 ? 2 : (b > 252 ? 252 : b);
  return m >= 0x7F80u ? kMx4Nan : (uint32_t)b;
}

// 2^-E for a byte from 2 to 252 (a normal number; any number for the NaN)
__device__ __forceinline__ float mx4_inverse(uint32_t byte) {
  return __uint_as_float(((254u - byte) & 0xFFu) << 23);
}

// 2^(byte - 127) for every byte: 2^-127 is subnormal, 255 is NaN
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

}  // namespace nvfp4
