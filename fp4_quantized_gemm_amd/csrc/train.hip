// Element-wise calls of the training step around the W4A16 expert products
// (asymmetric W4A16 QAT, gist.science technical summary §2.2 A): 8-bit
// activation checkpoints, with the forward SwiGLU from the same read, and the
// SwiGLU's backward pass with the gradient of the routing weights.
//
// A checkpoint is OCP MXFP8: E4M3 codes, one power-of-two (E8M0) scale per 32
// consecutive elements of a row.  The scale is the smallest power of two that
// keeps the block's largest magnitude at or below 448, so no code saturates
// and each rounding is half an E4M3 step (the floor(log2) rule of the format's
// description would saturate magnitudes above 1.75 times a power of two).  A
// code times its scale has 4 significant bits: exact in bf16, so the gradient
// kernels read codes as bf16 operands without another rounding.
#include <type_traits>

#include "device.h"
#include "mx.h"
#include "runtime.h"

namespace nvfp4 {

// 8 bf16 values of one lane; its block of 32 is lanes 4 i .. 4 i + 3.
// Returns the 8 codes and the block's scale byte.
__device__ __forceinline__ uint2 mx_encode8(const uint4& v, uint32_t& sbyte) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = max(m, lo < 0x7F80u ? lo : 0u);
    m = max(m, hi < 0x7F80u ? hi : 0u);
  }
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  sbyte = mx_scale_byte(m);
  uint32_t nan[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    nan[i] = ((w[i] & 0x7F80u) == 0x7F80u ? 0x7Fu : 0u) |
             ((w[i] & 0x7F800000u) == 0x7F800000u ? 0x7F00u : 0u);
  }
  if (m > 0x7F70u) {   // above 240 * 2^120: would round to 2^128, which bf16 does not hold
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = min(w[i] & 0x7FFFu, 0x7F70u), hi = min((w[i] >> 16) & 0x7FFFu, 0x7F70u);
      w[i] = (w[i] & 0x80008000u) | lo | (hi << 16);
    }
  }
  const float inv = __uint_as_float((254u - sbyte) << 23);   // 2^-E, a normal number
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = bf16_bits_to_f32(w[i] & 0xFFFFu) * inv, b = bf16_bits_to_f32(w[i] >> 16) * inv;
    const uint32_t p =
        ((uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu) | nan[i];
    c[i >> 1] |= p << (16 * (i & 1));
  }
  return make_uint2(c[0], c[1]);
}

// One lane per 8 columns (GLU: per 8 gate columns and the same up columns),
// one pass: 2 bytes read and 1.03 written per element, 1 more written with h.
// Bound by memory: with the restore behind it 73 us for 16384x4096 (5.6 TB/s of both
// together), 65 us for 32768x1536 with h; nontemporal loads and stores gained
// 4% there, and would take h and the codes past the caches of their readers.
// IT: index type of the flat chunk number (32 bits where it fits: the
// division by the chunks of a row is then a short sequence).
template <bool GLU, typename IT>
__global__ void __launch_bounds__(256)
k_checkpoint(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t ldx,
             uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
             uint16_t* __restrict__ h) {
  const IT per_row = (IT)((GLU ? K / 2 : K) / 8);
  const IT total = (IT)M * per_row;
  // whole blocks of 32 elements: total is a multiple of 4, so the lanes of a
  // block take part together
  for (IT q = (IT)blockIdx.x * 256 + threadIdx.x; q < total; q += (IT)gridDim.x * 256) {
    const IT row = q / per_row;
    const int64_t col = (int64_t)(q - row * per_row) * 8;
    const uint16_t* src = x + (int64_t)row * ldx + col;
    const uint4 a = *reinterpret_cast<const uint4*>(src);
    uint4 b = a;
    if constexpr (GLU) b = *reinterpret_cast<const uint4*>(src + K / 2);
    if (codes) {
      uint32_t sb;
      const uint2 c = mx_encode8(a, sb);
      *reinterpret_cast<uint2*>(codes + (int64_t)row * K + col) = c;
      if ((threadIdx.x & 3) == 0) scales[(int64_t)row * (K / 32) + col / 32] = (uint8_t)sb;
      if constexpr (GLU) {
        const uint2 d = mx_encode8(b, sb);
        *reinterpret_cast<uint2*>(codes + (int64_t)row * K + K / 2 + col) = d;
        if ((threadIdx.x & 3) == 0)
          scales[(int64_t)row * (K / 32) + K / 64 + col / 32] = (uint8_t)sb;
      }
    }
    if constexpr (GLU) {
      const uint4 o = make_uint4(swiglu_pair(a.x, b.x), swiglu_pair(a.y, b.y),
                                 swiglu_pair(a.z, b.z), swiglu_pair(a.w, b.w));
      *reinterpret_cast<uint4*>(h + (int64_t)row * (K / 2) + col) = o;
    }
  }
}

// one lane per 8 elements: exact products, no rounding
template <typename IT>
__global__ void __launch_bounds__(256)
k_restore(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t M,
          int64_t K, uint16_t* __restrict__ x, int64_t ldx) {
  const IT per_row = (IT)(K / 8);
  const IT total = (IT)M * per_row;
  for (IT q = (IT)blockIdx.x * 256 + threadIdx.x; q < total; q += (IT)gridDim.x * 256) {
    const IT row = q / per_row;
    const int64_t col = (int64_t)(q - row * per_row) * 8;
    const uint2 c = *reinterpret_cast<const uint2*>(codes + (int64_t)row * K + col);
    const u32x4 v = mx_decode8(c, mx_scale(scales[(int64_t)row * (K / 32) + col / 32]));
    *reinterpret_cast<uint4*>(x + (int64_t)row * ldx + col) = make_uint4(v.x, v.y, v.z, v.w);
  }
}

// Backward of h = silu(g) u with the routing weight w of the row's slot:
//   s = 1 / (1 + e^-g), dg = w dh u s (1 + g (1 - s)), du = w dh g s,
//   hw = w g s u, dw = sum_i dh_i g_i s_i u_i
// all in float32 (hardware exp2 and reciprocal, a few ulps; a reciprocal below
// 2^-126 comes out as 0, here as in the forward), one rounding to bf16 per
// output.  One wave per (token, slot), one pass: bound by memory, 265
// us for 131072 rows of 1024 from 8-bit y (5.1 TB/s, a plain copy's rate); the
// nontemporal forms of its loads and stores measured the same.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dh, float w, float& dg,
                                            float& du, float& hw, float& dot) {
  const float e = __builtin_amdgcn_exp2f(-g * 1.4426950408889634f);
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  const float gs = g * s, h = gs * u, wd = w * dh;
  // 1 - s = e s loses nothing where s is near 1; e overflows to infinity
  // only where s is 0
  const float t = s > 0.0f ? e * s : 1.0f;
  dg = wd * u * (s + gs * t);
  du = wd * gs;
  hw = w * h;
  dot += dh * h;
}

template <bool FP8>
__global__ void __launch_bounds__(256)
k_swiglu_backward(const void* __restrict__ y, const uint8_t* __restrict__ y_scales,
                  const uint16_t* __restrict__ dh, const int32_t* __restrict__ inv_perm,
                  const float* __restrict__ topk_w, int64_t P, int64_t I,
                  uint16_t* __restrict__ dy, uint16_t* __restrict__ hw,
                  float* __restrict__ d_topk_w) {
  const int lane = threadIdx.x & 63;
  for (int64_t slot = blockIdx.x * 4LL + (threadIdx.x >> 6); slot < P; slot += gridDim.x * 4LL) {
    const int64_t p = inv_perm ? (int64_t)inv_perm[slot] : slot;
    if (p < 0 || p >= P) continue;
    const float w = topk_w ? topk_w[slot] : 1.0f;
    float dot = 0.0f;
    for (int64_t c = lane * 8; c < I; c += 512) {
      u32x4 g8, u8;
      if constexpr (FP8) {
        const uint8_t* src = static_cast<const uint8_t*>(y) + p * 2 * I + c;
        const uint8_t* sc = y_scales + p * (I / 16) + c / 32;
        g8 = mx_decode8(*reinterpret_cast<const uint2*>(src), mx_scale(sc[0]));
        u8 = mx_decode8(*reinterpret_cast<const uint2*>(src + I), mx_scale(sc[I / 32]));
      } else {
        const uint16_t* src = static_cast<const uint16_t*>(y) + p * 2 * I + c;
        const uint4 a = *reinterpret_cast<const uint4*>(src);
        const uint4 b = *reinterpret_cast<const uint4*>(src + I);
        g8 = u32x4{a.x, a.y, a.z, a.w};
        u8 = u32x4{b.x, b.y, b.z, b.w};
      }
      const uint4 d = *reinterpret_cast<const uint4*>(dh + p * I + c);
      const uint32_t d4[4] = {d.x, d.y, d.z, d.w};
      uint32_t og[4], ou[4], oh[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float dg0, du0, h0, dg1, du1, h1;
        swiglu_grad(bf16_bits_to_f32(g8[i] & 0xFFFFu), bf16_bits_to_f32(u8[i] & 0xFFFFu),
                    bf16_bits_to_f32(d4[i] & 0xFFFFu), w, dg0, du0, h0, dot);
        swiglu_grad(bf16_bits_to_f32(g8[i] >> 16), bf16_bits_to_f32(u8[i] >> 16),
                    bf16_bits_to_f32(d4[i] >> 16), w, dg1, du1, h1, dot);
        og[i] = bf16x2_rne(dg0, dg1);
        ou[i] = bf16x2_rne(du0, du1);
        oh[i] = bf16x2_rne(h0, h1);
      }
      *reinterpret_cast<uint4*>(dy + p * 2 * I + c) = make_uint4(og[0], og[1], og[2], og[3]);
      *reinterpret_cast<uint4*>(dy + p * 2 * I + I + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
      if (hw) *reinterpret_cast<uint4*>(hw + p * I + c) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
    }
    if (d_topk_w) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
      if (lane == 0) d_topk_w[slot] = dot;
    }
  }
}

// workgroups of 256 lanes for n >= 1 lanes' work; the kernels stride past 2^20
static unsigned grid_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (unsigned)(b < (1 << 20) ? b : 1 << 20);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int mxfp8_checkpoint(const void* x, int64_t M, int64_t K, int64_t ldx, uint8_t* codes,
                     uint8_t* scales, void* h, void* stream) {
  NV_REQUIRE(M >= 0 && K >= 32 && K % 32 == 0 && ldx >= K && ldx % 8 == 0 &&
                 M < (1LL << 40) && K < (1LL << 22),
             NVFP4_ERR_SHAPE,
             "mxfp8_checkpoint: need 0 <= M < 2^40, K %% 32 == 0, 32 <= K < 2^22, ldx >= K, "
             "ldx %% 8 == 0 (M=%lld K=%lld ldx=%lld)",
             (long long)M, (long long)K, (long long)ldx);
  NV_REQUIRE(h == nullptr || K % 64 == 0, NVFP4_ERR_SHAPE,
             "mxfp8_checkpoint: the SwiGLU needs K %% 64 == 0 (K=%lld)", (long long)K);
  if (M == 0) return ok();
  NV_REQUIRE((codes == nullptr) == (scales == nullptr) && (codes || h), NVFP4_ERR_NULL,
             "mxfp8_checkpoint: codes and scales go together, and with neither h is needed");
  NV_REQUIRE(x, NVFP4_ERR_NULL, "mxfp8_checkpoint: missing pointer");
  NV_REQUIRE(aligned(x, 16) && aligned(codes, 8) && aligned(h, 16), NVFP4_ERR_ALIGN,
             "mxfp8_checkpoint: misaligned pointer");
  hipStream_t s = as_stream(stream);
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  uint16_t* hp = static_cast<uint16_t*>(h);
  const int64_t n = M * ((h ? K / 2 : K) / 8);
  const unsigned g = grid_for(n);
  const bool small = n < (1LL << 31);   // plus the grid's stride of 2^28, still below 2^32
  if (h && small)
    k_checkpoint<true, uint32_t><<<g, 256, 0, s>>>(xp, M, K, ldx, codes, scales, hp);
  else if (h)
    k_checkpoint<true, uint64_t><<<g, 256, 0, s>>>(xp, M, K, ldx, codes, scales, hp);
  else if (small)
    k_checkpoint<false, uint32_t><<<g, 256, 0, s>>>(xp, M, K, ldx, codes, scales, hp);
  else
    k_checkpoint<false, uint64_t><<<g, 256, 0, s>>>(xp, M, K, ldx, codes, scales, hp);
  return check_launch("mxfp8_checkpoint");
}

int mxfp8_restore(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* x,
                  int64_t ldx, void* stream) {
  NV_REQUIRE(M >= 0 && K >= 32 && K % 32 == 0 && ldx >= K && ldx % 8 == 0 &&
                 M < (1LL << 40) && K < (1LL << 22),
             NVFP4_ERR_SHAPE,
             "mxfp8_restore: need 0 <= M < 2^40, K %% 32 == 0, 32 <= K < 2^22, ldx >= K, "
             "ldx %% 8 == 0 (M=%lld K=%lld ldx=%lld)",
             (long long)M, (long long)K, (long long)ldx);
  if (M == 0) return ok();
  NV_REQUIRE(codes && scales && x, NVFP4_ERR_NULL, "mxfp8_restore: missing pointer");
  NV_REQUIRE(aligned(codes, 8) && aligned(x, 16), NVFP4_ERR_ALIGN,
             "mxfp8_restore: misaligned pointer");
  hipStream_t s = as_stream(stream);
  const int64_t n = M * (K / 8);
  const unsigned g = grid_for(n);
  if (n < (1LL << 31))
    k_restore<uint32_t><<<g, 256, 0, s>>>(codes, scales, M, K, static_cast<uint16_t*>(x), ldx);
  else
    k_restore<uint64_t><<<g, 256, 0, s>>>(codes, scales, M, K, static_cast<uint16_t*>(x), ldx);
  return check_launch("mxfp8_restore");
}

int moe_swiglu_backward(const void* y, const uint8_t* y_scales, const void* dh,
                        const int32_t* inv_perm, const float* topk_w, int64_t T, int64_t tk,
                        int64_t I, void* dy, void* hw, float* d_topk_w, void* stream) {
  NV_REQUIRE(T >= 0 && tk >= 1 && tk <= 32 && T < (1LL << 31) && T * tk < (1LL << 31) && I >= 8 &&
                 I % 8 == 0 && I < (1LL << 31) && (y_scales == nullptr || I % 32 == 0),
             NVFP4_ERR_SHAPE,
             "moe_swiglu_backward: need T >= 0, 1 <= tk <= 32, T*tk < 2^31, 8 <= I < 2^31, "
             "I %% 8 == 0 (I %% 32 == 0 for 8-bit y) (T=%lld tk=%lld I=%lld)",
             (long long)T, (long long)tk, (long long)I);
  if (T == 0) return ok();
  NV_REQUIRE(y && dh && dy, NVFP4_ERR_NULL, "moe_swiglu_backward: missing pointer");
  NV_REQUIRE(topk_w || !d_topk_w, NVFP4_ERR_NULL,
             "moe_swiglu_backward: d_topk_w without topk_w");
  NV_REQUIRE(inv_perm || tk == 1, NVFP4_ERR_NULL, "moe_swiglu_backward: tk > 1 needs inv_perm");
  NV_REQUIRE(aligned(y, y_scales ? 8 : 16) && aligned(dh, 16) && aligned(dy, 16) && aligned(hw, 16) &&
                 aligned(inv_perm, 4) && aligned(topk_w, 4) && aligned(d_topk_w, 4),
             NVFP4_ERR_ALIGN, "moe_swiglu_backward: misaligned pointer");
  hipStream_t s = as_stream(stream);
  const int64_t P = T * tk;
  const unsigned g = grid_for(P * 64);
  if (y_scales)
    k_swiglu_backward<true><<<g, 256, 0, s>>>(y, y_scales, static_cast<const uint16_t*>(dh),
                                              inv_perm, topk_w, P, I, static_cast<uint16_t*>(dy),
                                              static_cast<uint16_t*>(hw), d_topk_w);
  else
    k_swiglu_backward<false><<<g, 256, 0, s>>>(y, nullptr, static_cast<const uint16_t*>(dh),
                                               inv_perm, topk_w, P, I, static_cast<uint16_t*>(dy),
                                               static_cast<uint16_t*>(hw), d_topk_w);
  return check_launch("moe_swiglu_backward");
}

}  // extern "C"
