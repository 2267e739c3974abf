// Gradients of the W4A16 expert product y[p] = W~_e x[p] (asymmetric W4A16
// QAT: bf16 activations times the weights of the shared QDQ path, gist.science
// technical summary §2.2 A): the input gradient, a product with the same NVFP4
// weights contracted over their rows, and the weight gradient, contracted over
// each expert's own rows (the straight-through gradient of the master weight).
#include <cstring>

#include "device.h"
#include "mfma.h"
#include "mx.h"
#include "runtime.h"

namespace nvfp4 {

struct GradArgs {
  const uint16_t* dy;          // [M_dy][N] bf16
  const int32_t* dy_rows;      // [M_total] or null (identity)
  const void* x;               // wgrad: [M_x][K] bf16, or E4M3 codes
  const uint8_t* x_scales;     // wgrad: [M_x][K/32] or null
  const int32_t* x_rows;       // wgrad: [M_total] or null
  const uint8_t* w_codes;      // dgrad: packed weights
  const uint8_t* w_scales;
  const float* g_w;
  const int32_t* offsets;      // [E + 1]
  const int32_t* prefix;       // dgrad: row tiles before each expert
  uint16_t* dx;                // dgrad: [M_total][K] bf16
  void* dw;                    // wgrad: [E][N][K] f32 or bf16
  int64_t M_dy, M_x, M_total, N, K;
  int E;
  int dw_bf16, accumulate;
};

__device__ __forceinline__ void expert_rows(const GradArgs& p, int e, int64_t& lo, int64_t& hi) {
  lo = p.offsets[e];
  hi = p.offsets[e + 1];
  lo = lo < 0 ? 0 : (lo > p.M_total ? p.M_total : lo);
  hi = hi < lo ? lo : (hi > p.M_total ? p.M_total : hi);
}

__device__ __forceinline__ int64_t source_row(const int32_t* rows, int64_t p, int64_t M) {
  const int64_t t = rows ? (int64_t)rows[p] : p;
  return t < 0 ? 0 : (t >= M ? M - 1 : t);
}

// 64x64 outputs per workgroup, contraction 32 at a time; both operands in LDS
// with the contraction contiguous.  DGRAD: outputs [rows][k], contraction n;
// else outputs [n][k], contraction over the expert's rows.
template <bool DGRAD>
__global__ void __launch_bounds__(256)
k_grad_simple(GradArgs p) {
  __shared__ __attribute__((aligned(16))) uint16_t As[64][40];
  __shared__ __attribute__((aligned(16))) uint16_t Bs[64][40];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b0 = (int64_t)blockIdx.x * 64;
  int e;
  int64_t lo, hi, a0;
  if constexpr (DGRAD) {
    const int gt = blockIdx.y;
    if (gt >= p.prefix[p.E]) return;
    int l = 0, h = p.E;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (p.prefix[mid] <= gt) l = mid; else h = mid;
    }
    e = l;
    expert_rows(p, e, lo, hi);
    a0 = lo + (int64_t)(gt - p.prefix[e]) * 64;
  } else {
    e = blockIdx.z;
    expert_rows(p, e, lo, hi);
    a0 = (int64_t)blockIdx.y * 64;
  }
  f32x4_t acc[2][2] = {};
  const int wa = (wave >> 1) * 32, wb = (wave & 1) * 32;
  const int64_t c_end = DGRAD ? p.N : hi - lo;
  for (int64_t c0 = 0; c0 < c_end; c0 += 32) {
    u32x4 va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
    if constexpr (DGRAD) {
      const int r = tid >> 2;
      const int64_t pr = a0 + r, c = c0 + (tid & 3) * 8;
      if (pr < hi && c < p.N)
        va = *reinterpret_cast<const u32x4*>(p.dy + source_row(p.dy_rows, pr, p.M_dy) * p.N + c);
      *reinterpret_cast<u32x4*>(&As[r][(tid & 3) * 8]) = va;
      const int cc = tid >> 3;
      const int64_t n = c0 + cc, k = b0 + (tid & 7) * 8;
      if (n < p.N && k < p.K) {
        const uint8_t* wc = p.w_codes + e * packed_codes_per_expert(p.N, p.K);
        const uint8_t* ws = p.w_scales + e * packed_scales_per_expert(p.N, p.K);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(wc + wcode_offset(n, k, p.K));
        vb = decode8_bf16(w, e4m3_decode(ws[wscale_offset(n, k >> 4, p.K)]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        Bs[(tid & 7) * 8 + i][cc] = (uint16_t)(vb[i >> 1] >> (16 * (i & 1)));
    } else {
      const int cc = tid >> 3, j = (tid & 7) * 8;
      const int64_t pr = lo + c0 + cc, n = a0 + j, k = b0 + j;
      if (pr < hi) {
        if (n < p.N)
          va = *reinterpret_cast<const u32x4*>(p.dy + source_row(p.dy_rows, pr, p.M_dy) * p.N + n);
        if (k < p.K) {
          const int64_t t = source_row(p.x_rows, pr, p.M_x);
          if (p.x_scales)
            vb = mx_decode8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x) +
                                                            t * p.K + k),
                            mx_scale(p.x_scales[t * (p.K / 32) + k / 32]));
          else
            vb = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + t * p.K + k);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        As[j + i][cc] = (uint16_t)(va[i >> 1] >> (16 * (i & 1)));
        Bs[j + i][cc] = (uint16_t)(vb[i >> 1] >> (16 * (i & 1)));
      }
    }
    __syncthreads();
    const int r = lane & 15, g = lane >> 4;
    u32x4 fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = *reinterpret_cast<const u32x4*>(&As[wa + 16 * i + r][8 * g]);
      fb[i] = *reinterpret_cast<const u32x4*>(&Bs[wb + 16 * i + r][8 * g]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16(fa[i], fb[j], acc[i][j]);
    __syncthreads();
  }
  const float sc = DGRAD ? p.g_w[e] : 1.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t a = a0 + wa + 16 * i + 4 * (lane >> 4) + r;
        const int64_t k = b0 + wb + 16 * j + (lane & 15);
        if (k >= p.K || a >= (DGRAD ? hi : p.N)) continue;
        if constexpr (DGRAD) {
          p.dx[a * p.K + k] = (uint16_t)bf16x2_rne(acc[i][j][r] * sc, 0.f);
        } else {
          const int64_t at = ((int64_t)e * p.N + a) * p.K + k;
          if (p.dw_bf16) {
            static_cast<uint16_t*>(p.dw)[at] = (uint16_t)bf16x2_rne(acc[i][j][r], 0.f);
          } else {
            float* d = static_cast<float*>(p.dw) + at;
            *d = p.accumulate ? *d + acc[i][j][r] : acc[i][j][r];
          }
        }
      }
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t grouped_w4a16_dgrad_workspace_size(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  (void)M_total; (void)N; (void)K;
  return round_up((size_t)((E < 1 ? 1 : E) + 1) * sizeof(int32_t), 256);
}

int grouped_w4a16_dgrad(const void* dy, const int32_t* dy_rows, int64_t M_src,
                        const uint8_t* w_codes, const uint8_t* w_scales, const float* g_w,
                        const int32_t* expert_offsets, int64_t E, int64_t M_total, int64_t N,
                        int64_t K, void* dx, void* ws, size_t ws_bytes, void* stream) {
  NV_REQUIRE(E >= 1 && E <= 1024 && M_total >= 0 && M_total < (1LL << 31) && M_src >= 0 &&
                 N >= 16 && N % 16 == 0 && K >= 64 && K % 64 == 0 && N < (1LL << 31) &&
                 K < (1LL << 31),
             NVFP4_ERR_SHAPE,
             "grouped_w4a16_dgrad: need 1 <= E <= 1024, M_total < 2^31, N %% 16 == 0, K %% 64 == 0 "
             "(E=%lld M_total=%lld N=%lld K=%lld)",
             (long long)E, (long long)M_total, (long long)N, (long long)K);
  NV_REQUIRE(dy_rows != nullptr || M_src >= M_total, NVFP4_ERR_SHAPE,
             "grouped_w4a16_dgrad: without dy_rows, M_src must be >= M_total");
  NV_REQUIRE(M_total == 0 || M_src >= 1, NVFP4_ERR_SHAPE, "grouped_w4a16_dgrad: M_src == 0");
  NV_REQUIRE((uint64_t)M_src < (1ULL << 32) / (2 * (uint64_t)N) &&
                 (uint64_t)N * (uint64_t)K / 2 < (1ULL << 32),
             NVFP4_ERR_UNSUPPORTED, "grouped_w4a16_dgrad: dy or one expert's codes exceed 4 GiB");
  NV_REQUIRE(w_codes && w_scales && g_w && expert_offsets && ws && (M_total == 0 || (dy && dx)),
             NVFP4_ERR_NULL, "grouped_w4a16_dgrad: missing pointer");
  NV_REQUIRE(aligned(dy, 16) && aligned(w_codes, 16) && aligned(w_scales, 16) && aligned(ws, 16) &&
                 aligned(dx, 16),
             NVFP4_ERR_ALIGN, "grouped_w4a16_dgrad: misaligned pointer");
  NV_REQUIRE(ws_bytes >= grouped_w4a16_dgrad_workspace_size(E, M_total, N, K),
             NVFP4_ERR_WORKSPACE, "grouped_w4a16_dgrad: workspace too small");
  if (M_total == 0) return ok();
  hipStream_t s = as_stream(stream);
  GradArgs p{};
  p.dy = static_cast<const uint16_t*>(dy);
  p.dy_rows = dy_rows;
  p.w_codes = w_codes;
  p.w_scales = w_scales;
  p.g_w = g_w;
  p.offsets = expert_offsets;
  p.prefix = static_cast<int32_t*>(ws);
  p.dx = static_cast<uint16_t*>(dx);
  p.M_dy = M_src;
  p.M_total = M_total;
  p.N = N;
  p.K = K;
  p.E = (int)E;
  tile_prefix(expert_offsets, (int)E, M_total, 64, static_cast<int32_t*>(ws), s);
  const int64_t m_tiles = (M_total + 63) / 64 + E;
  k_grad_simple<true><<<dim3((unsigned)((K + 63) / 64), (unsigned)m_tiles), 256, 0, s>>>(p);
  return check_launch("grouped_w4a16_dgrad");
}

size_t grouped_wgrad_workspace_size(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  (void)E; (void)M_total; (void)N; (void)K;
  return 256;
}

int grouped_wgrad(const void* dy, const int32_t* dy_rows, int64_t M_dy, const void* x,
                  const uint8_t* x_scales, const int32_t* x_rows, int64_t M_x,
                  const int32_t* expert_offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                  void* dw, int dw_bf16, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  NV_REQUIRE(E >= 1 && E <= 1024 && M_total >= 0 && M_total < (1LL << 31) && M_dy >= 0 &&
                 M_x >= 0 && N >= 8 && N % 8 == 0 && K >= 8 && K % 8 == 0 && N < (1LL << 31) &&
                 K < (1LL << 31) && (x_scales == nullptr || K % 32 == 0),
             NVFP4_ERR_SHAPE,
             "grouped_wgrad: need 1 <= E <= 1024, M_total < 2^31, N %% 8 == 0, K %% 8 == 0 "
             "(K %% 32 == 0 for 8-bit x) (E=%lld M_total=%lld N=%lld K=%lld)",
             (long long)E, (long long)M_total, (long long)N, (long long)K);
  NV_REQUIRE((dy_rows != nullptr || M_dy >= M_total) && (x_rows != nullptr || M_x >= M_total),
             NVFP4_ERR_SHAPE, "grouped_wgrad: an operand without a row list needs M_total rows");
  NV_REQUIRE(M_total == 0 || (M_dy >= 1 && M_x >= 1), NVFP4_ERR_SHAPE,
             "grouped_wgrad: an operand has no rows");
  NV_REQUIRE((uint64_t)M_dy < (1ULL << 32) / (2 * (uint64_t)N) &&
                 (uint64_t)M_x < (1ULL << 32) / ((x_scales ? 1 : 2) * (uint64_t)K),
             NVFP4_ERR_UNSUPPORTED, "grouped_wgrad: dy or x exceeds 4 GiB");
  NV_REQUIRE(dw_bf16 == 0 || dw_bf16 == 1, NVFP4_ERR_UNSUPPORTED,
             "grouped_wgrad: dw_bf16 must be 0 or 1");
  NV_REQUIRE(!(accumulate && dw_bf16), NVFP4_ERR_UNSUPPORTED,
             "grouped_wgrad: only a float32 dw can be added to");
  NV_REQUIRE(expert_offsets && ws && dw && (M_total == 0 || (dy && x)), NVFP4_ERR_NULL,
             "grouped_wgrad: missing pointer");
  NV_REQUIRE(aligned(dy, 16) && aligned(x, 16) && aligned(dw, 16) && aligned(ws, 16),
             NVFP4_ERR_ALIGN, "grouped_wgrad: misaligned pointer");
  NV_REQUIRE(ws_bytes >= grouped_wgrad_workspace_size(E, M_total, N, K), NVFP4_ERR_WORKSPACE,
             "grouped_wgrad: workspace too small");
  hipStream_t s = as_stream(stream);
  GradArgs p{};
  p.dy = static_cast<const uint16_t*>(dy);
  p.dy_rows = dy_rows;
  p.x = x;
  p.x_scales = x_scales;
  p.x_rows = x_rows;
  p.offsets = expert_offsets;
  p.dw = dw;
  p.M_dy = M_dy;
  p.M_x = M_x;
  p.M_total = M_total;
  p.N = N;
  p.K = K;
  p.E = (int)E;
  p.dw_bf16 = dw_bf16;
  p.accumulate = accumulate != 0;
  k_grad_simple<false><<<dim3((unsigned)((K + 63) / 64), (unsigned)((N + 63) / 64), (unsigned)E),
                         256, 0, s>>>(p);
  return check_launch("grouped_wgrad");
}

}  // extern "C"
