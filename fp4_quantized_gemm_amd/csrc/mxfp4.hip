// OCP MXFP4: E2M1 codes, two per byte, with one E8M0 byte (2^(byte - 127))
// per 32 consecutive elements; the quantiser, along the rows and of the
// transpose, and the values that codes stand for.  (The MX format is the
// 4-bit one that CDNA4's matrix cores multiply natively; the QUADS pages name
// only the E2M1 grid and "fine-grained scaling", gist.science summary §1.)
//
// Scale of a block with largest magnitude A: the smallest power of two 2^E
// with A <= 7 * 2^E.  Elements between 6 and 7 times it become 6: at most one
// 2^E off, as much as the grid's widest half step (4 to 6) is anyway.  Mean
// square error of blocks of normal values: 0.0125 of the variance, against
// 0.0133 with A <= 6 * 2^E and 0.0132 with E = floor(log2 A) - 2 (Student-t
// with 3 degrees: 0.0192, 0.0225, 0.0200).  E is kept within -125 .. 125, so
// that every value is a normal bf16 or 0.
#include "device.h"
#include "mx4.h"
#include "runtime.h"

namespace nvfp4 {

// 8 bf16 values of one lane; its block of 32 is lanes 4 i .. 4 i + 3.
// Returns the 8 codes and the block's scale byte.
__device__ __forceinline__ uint32_t mx4_encode8(const uint4& v, uint32_t& sbyte) {
  uint32_t m = absmax_bf16x8(v);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  sbyte = mx4_scale_byte(m);
  const float inv = mx4_inverse(sbyte);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c = 0;
#define NV_MX4(I)                                                                       \
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_bits_to_f32(w[I] & 0xFFFFu) * inv, \
                                               bf16_bits_to_f32(w[I] >> 16) * inv, 1.0f, I)
  NV_MX4(0); NV_MX4(1); NV_MX4(2); NV_MX4(3);
#undef NV_MX4
  return sbyte == kMx4Nan ? 0x77777777u : c;
}

// One lane per 8 columns, one pass: 2 bytes read and 0.53 written per
// element.  Bound by memory: 16384x4096 33 us = 5.2 TB/s.  IT: index type of the flat chunk number.
template <typename IT>
__global__ void __launch_bounds__(256)
k_mx4_quantize(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t ldx,
               uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const IT per_row = (IT)(K / 8);
  const IT total = (IT)M * per_row;
  // whole blocks of 32 elements: total is a multiple of 4, so the lanes of a
  // block take part together
  for (IT q = (IT)blockIdx.x * 256 + threadIdx.x; q < total; q += (IT)gridDim.x * 256) {
    const IT row = q / per_row;
    const int64_t col = (int64_t)(q - row * per_row) * 8;
    uint32_t sb;
    const uint32_t c =
        mx4_encode8(*reinterpret_cast<const uint4*>(x + (int64_t)row * ldx + col), sb);
    // (codes and scales are contiguous, and a row is whole chunks: chunk q's place)
    *reinterpret_cast<uint32_t*>(codes + 4 * (int64_t)q) = c;
    if ((threadIdx.x & 3) == 0) scales[(int64_t)q >> 2] = (uint8_t)sb;
  }
}

// Codes of the transpose: blocks of 32 rows of x, one column each.  A
// workgroup takes 256 rows x 64 columns through LDS; then each lane has two
// columns of one block of 32 rows, and the 8 lanes of a column's 8 blocks write
// 128 contiguous bytes of codes.  (A block's rows are rotated by 8 dwords more
// than those of the block before: the lanes of a read take every bank alike.)
// 128 matrices of 2048x768: 113 us = 4.5 TB/s; with a wave on two blocks of 64
// columns, 32 contiguous bytes at a time, 132.
constexpr int kTM = 256, kTK = 64;
__global__ void __launch_bounds__(256)
k_mx4_quantize_t(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t ldx,
                 uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[kTM * kTK];
  const int tid = threadIdx.x;
  const int64_t k0 = (int64_t)blockIdx.x * kTK, m0 = (int64_t)blockIdx.y * kTM;
  const int64_t e = blockIdx.z;
  const uint16_t* src = x + e * M * ldx;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 32 * i + (tid >> 3), c = (tid & 7) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (m0 + r < M && k0 + c < K)
      v = *reinterpret_cast<const uint4*>(src + (m0 + r) * ldx + k0 + c);
    *reinterpret_cast<uint4*>(tile + r * kTK + ((c + 16 * i) & (kTK - 1))) = v;
  }
  __syncthreads();
  const int blk = tid & 7, c = (tid >> 3) * 2;
  if (m0 + 32 * blk >= M) return;          // M % 32 == 0: whole blocks
  const uint32_t* col =
      reinterpret_cast<const uint32_t*>(tile + 32 * blk * kTK + ((c + 16 * blk) & (kTK - 1)));
  uint32_t w[32];
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    w[r] = col[r * (kTK / 2)];
    lo = max(lo, w[r] & 0x7FFFu);
    hi = max(hi, (w[r] >> 16) & 0x7FFFu);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (k0 + c + h >= K) break;
    const uint32_t sb = mx4_scale_byte(h ? hi : lo);
    const float inv = mx4_inverse(sb);
    uint32_t o[4] = {0, 0, 0, 0};
    auto val = [&](int r) {
      return bf16_bits_to_f32(h ? w[r] >> 16 : w[r] & 0xFFFFu) * inv;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, val(8 * i), val(8 * i + 1), 1.0f, 0);
      o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o[i], val(8 * i + 2), val(8 * i + 3), 1.0f, 1);
      o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o[i], val(8 * i + 4), val(8 * i + 5), 1.0f, 2);
      o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o[i], val(8 * i + 6), val(8 * i + 7), 1.0f, 3);
      if (sb == kMx4Nan) o[i] = 0x77777777u;
    }
    const int64_t block = ((e * K + k0 + c + h) * M + m0) / 32 + blk;
    *reinterpret_cast<uint4*>(codes + 16 * block) = make_uint4(o[0], o[1], o[2], o[3]);
    scales[block] = (uint8_t)sb;
  }
}

// one lane per 8 elements: exact products (2 significant bits), no rounding;
// 16384x4096 25 us
template <typename IT>
__global__ void __launch_bounds__(256)
k_mx4_restore(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t M,
              int64_t K, uint16_t* __restrict__ x, int64_t ldx) {
  const IT per_row = (IT)(K / 8);
  const IT total = (IT)M * per_row;
  for (IT q = (IT)blockIdx.x * 256 + threadIdx.x; q < total; q += (IT)gridDim.x * 256) {
    const IT row = q / per_row;
    const int64_t col = (int64_t)(q - row * per_row) * 8;
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + 4 * (int64_t)q);
    const u32x4 v = decode8_bf16(c, mx4_scale(scales[(int64_t)q >> 2]));
    *reinterpret_cast<uint4*>(x + (int64_t)row * ldx + col) = make_uint4(v.x, v.y, v.z, v.w);
  }
}

// workgroups of 256 lanes for n >= 1 lanes' work; the kernels stride past 2^20
static unsigned mx4_grid(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (unsigned)(b < (1 << 20) ? b : 1 << 20);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int mxfp4_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, uint8_t* codes,
                   uint8_t* scales, void* stream) {
  NV_REQUIRE(M >= 0 && M < (1LL << 40) && K >= 32 && K % 32 == 0 && K < (1LL << 22) && ldx >= K &&
                 ldx % 8 == 0 && ldx < (1LL << 22),
             NVFP4_ERR_SHAPE,
             "mxfp4_quantize: need 0 <= M < 2^40, K %% 32 == 0, 32 <= K <= ldx < 2^22, "
             "ldx %% 8 == 0 (M=%lld K=%lld ldx=%lld)",
             (long long)M, (long long)K, (long long)ldx);
  if (M == 0) return ok();
  NV_REQUIRE(x && codes && scales, NVFP4_ERR_NULL, "mxfp4_quantize: missing pointer");
  NV_REQUIRE(aligned(x, 16) && aligned(codes, 16), NVFP4_ERR_ALIGN,
             "mxfp4_quantize: misaligned pointer");
  hipStream_t s = as_stream(stream);
  const int64_t n = M * (K / 8);
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  if (n < (1LL << 31))
    k_mx4_quantize<uint32_t><<<mx4_grid(n), 256, 0, s>>>(xp, M, K, ldx, codes, scales);
  else
    k_mx4_quantize<uint64_t><<<mx4_grid(n), 256, 0, s>>>(xp, M, K, ldx, codes, scales);
  return check_launch("mxfp4_quantize");
}

int mxfp4_quantize_transposed(const void* x, int64_t E, int64_t M, int64_t K, int64_t ldx,
                              uint8_t* codes, uint8_t* scales, void* stream) {
  NV_REQUIRE(E >= 0 && E < 65536 && M >= 32 && M % 32 == 0 && M < (1LL << 22) && K >= 8 &&
                 K % 8 == 0 && K < (1LL << 22) && ldx >= K && ldx % 8 == 0 && ldx < (1LL << 22),
             NVFP4_ERR_SHAPE,
             "mxfp4_quantize_transposed: need 0 <= E < 65536, M %% 32 == 0, 32 <= M < 2^22, "
             "K %% 8 == 0, 8 <= K <= ldx < 2^22, ldx %% 8 == 0 (E=%lld M=%lld K=%lld ldx=%lld)",
             (long long)E, (long long)M, (long long)K, (long long)ldx);
  if (E == 0) return ok();
  NV_REQUIRE(x && codes && scales, NVFP4_ERR_NULL, "mxfp4_quantize_transposed: missing pointer");
  NV_REQUIRE(aligned(x, 16) && aligned(codes, 16), NVFP4_ERR_ALIGN,
             "mxfp4_quantize_transposed: misaligned pointer");
  const dim3 grid((unsigned)((K + kTK - 1) / kTK), (unsigned)((M + kTM - 1) / kTM), (unsigned)E);
  k_mx4_quantize_t<<<grid, 256, 0, as_stream(stream)>>>(static_cast<const uint16_t*>(x), M, K, ldx,
                                                        codes, scales);
  return check_launch("mxfp4_quantize_transposed");
}

int mxfp4_restore(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* x,
                  int64_t ldx, void* stream) {
  NV_REQUIRE(M >= 0 && M < (1LL << 40) && K >= 32 && K % 32 == 0 && K < (1LL << 22) && ldx >= K &&
                 ldx % 8 == 0 && ldx < (1LL << 22),
             NVFP4_ERR_SHAPE,
             "mxfp4_restore: need 0 <= M < 2^40, K %% 32 == 0, 32 <= K <= ldx < 2^22, "
             "ldx %% 8 == 0 (M=%lld K=%lld ldx=%lld)",
             (long long)M, (long long)K, (long long)ldx);
  if (M == 0) return ok();
  NV_REQUIRE(codes && scales && x, NVFP4_ERR_NULL, "mxfp4_restore: missing pointer");
  NV_REQUIRE(aligned(codes, 16) && aligned(x, 16), NVFP4_ERR_ALIGN,
             "mxfp4_restore: misaligned pointer");
  hipStream_t s = as_stream(stream);
  const int64_t n = M * (K / 8);
  uint16_t* xp = static_cast<uint16_t*>(x);
  if (n < (1LL << 31))
    k_mx4_restore<uint32_t><<<mx4_grid(n), 256, 0, s>>>(codes, scales, M, K, xp, ldx);
  else
    k_mx4_restore<uint64_t><<<mx4_grid(n), 256, 0, s>>>(codes, scales, M, K, xp, ldx);
  return check_launch("mxfp4_restore");
}

}  // extern "C"
