// Expert-grouped product of MXFP4 operands (E2M1 codes, an E8M0 scale per 32
// elements along K, both row-major) on CDNA4's scaled 4-bit matrix
// instructions: for permuted row p of expert e, t = a_rows ? a_rows[p] : p,
//   y[p][n] = bf16( sum_b 2^(sa + sw) sum_{k in block b} a[t][k] w[e][n][k] ),
// every product exact, float32 accumulation.  The SwiGLU form has W = [gate |
// up] along N and writes h = bf16(silu(gate) up), both taken from the float32
// sums.
//
// The weights are the instructions' first operand and the activations the
// second, so a lane's accumulator registers are consecutive columns of one
// row of y.
#include <type_traits>

#include "device.h"
#include "mfma.h"
#include "runtime.h"

namespace nvfp4 {

struct MxGemmArgs {
  const uint8_t* a_codes;   // [M_src][K/2]
  const uint8_t* a_scales;  // [M_src][K/32]
  const int32_t* a_rows;    // [M_total] or null (identity)
  const uint8_t* w_codes;   // [E][N][K/2]
  const uint8_t* w_scales;  // [E][N][K/32]
  const int32_t* offsets;   // [E + 1]
  uint16_t* y;              // [M_total][N], SwiGLU [M_total][N/2]
  int64_t M_src, M_total, N, K;
  int E;
};

typedef int mx_i32x8 __attribute__((ext_vector_type(8)));

// D += 2^(sa - 127 + sb - 127) A B over 128 k: lane (r = l % 16, q = l / 16)
// has 32 codes of row r in 16 bytes, the low byte of sa / sb their scale
__device__ __forceinline__ f32x4_t mfma16_mx4(const u32x4& a, uint32_t sa, const u32x4& b,
                                              uint32_t sb, f32x4_t c) {
  const mx_i32x8 a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const mx_i32x8 b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// The rows of expert e, within the output.
__device__ __forceinline__ void expert_rows(const MxGemmArgs& p, int e, int64_t& lo, int64_t& hi) {
  lo = p.offsets[e];
  hi = p.offsets[e + 1];
  lo = lo < 0 ? 0 : (lo > p.M_total ? p.M_total : lo);
  hi = hi < lo ? lo : (hi > p.M_total ? p.M_total : hi);
}

__device__ __forceinline__ int64_t source_row(const MxGemmArgs& p, int64_t row) {
  const int64_t t = p.a_rows ? (int64_t)p.a_rows[row] : row;
  return t < 0 ? 0 : (t >= p.M_src ? p.M_src - 1 : t);
}

// Weight streaming, without LDS: each wave owns R groups of 16 weight rows
// and multiplies all of K with TT tiles of 16 activation rows, operands
// straight from memory to registers.  K advances in chunks of 512: lane (r,
// q) takes the 16-byte pieces 4 s + q, s = 0 .. 3, of its row's 256 bytes (64
// contiguous bytes of a row per load), and the chunk's 16 scale bytes, of
// which byte q of dword s belongs to piece s.
// GLU: half of the groups are gate columns, the other half the same up ones.
template <int R, int TT, bool GLU>
__global__ void __launch_bounds__(256, 2)
k_mx_few(MxGemmArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int e = blockIdx.y;
  int64_t lo, hi;
  expert_rows(p, e, lo, hi);
  constexpr int RO = GLU ? R / 2 : R;                  // output groups
  const int64_t NO = GLU ? p.N / 2 : p.N;              // output columns
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * 16 * RO;
  if (n0 >= NO) return;
  const int64_t KC = p.K / 2, KS = p.K / 32;
  const uint8_t* wc[R];
  const uint8_t* wsc[R];
#pragma unroll
  for (int g = 0; g < R; ++g) {
    int64_t n = n0 + 16 * (g % RO) + r16;
    n = n < NO ? n : NO - 1;
    if (GLU && g >= RO) n += NO;
    wc[g] = p.w_codes + ((int64_t)e * p.N + n) * KC + 16 * q;
    wsc[g] = p.w_scales + ((int64_t)e * p.N + n) * KS;
  }
  for (int64_t p0 = lo + (int64_t)blockIdx.z * 16 * TT; p0 < hi; p0 += (int64_t)gridDim.z * 16 * TT) {
    const uint8_t* ac[TT];
    const uint8_t* asc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int64_t row = p0 + 16 * t + r16;
      const int64_t src = source_row(p, row < hi ? row : hi - 1);
      ac[t] = p.a_codes + src * KC + 16 * q;
      asc[t] = p.a_scales + src * KS;
    }
    f32x4_t acc[R][TT];
#pragma unroll
    for (int g = 0; g < R; ++g)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[g][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int64_t k = 0; k < p.K; k += 128) {
      const uint32_t sh = 8 * q;
      u32x4 a[TT];
      uint32_t sa[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        a[t] = *reinterpret_cast<const u32x4*>(ac[t] + k / 2);
        sa[t] = *reinterpret_cast<const uint32_t*>(asc[t] + k / 32) >> sh;
      }
#pragma unroll
      for (int g = 0; g < R; ++g) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(wc[g] + k / 2);
        const uint32_t sw = *reinterpret_cast<const uint32_t*>(wsc[g] + k / 32) >> sh;
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[g][t] = mfma16_mx4(w, sw, a[t], sa[t], acc[g][t]);
      }
    }
    // lane (r, q): columns n0 + 16 g + 4 q .. + 3 of row p0 + 16 t + r
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int64_t row = p0 + 16 * t + r16;
      if (row >= hi) continue;
#pragma unroll
      for (int g = 0; g < RO; ++g) {
        const int64_t n = n0 + 16 * g + 4 * q;
        if (n >= NO) continue;
        f32x4_t v = acc[g][t];
        if constexpr (GLU) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = silu_mul(v[i], acc[g + RO][t][i]);
        }
        *reinterpret_cast<uint2*>(p.y + row * NO + n) =
            make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
      }
    }
  }
}

}  // namespace nvfp4

using namespace nvfp4;

static int mx_gemm(const char* name, bool glu, const uint8_t* a_codes, const uint8_t* a_scales,
                   const int32_t* a_rows, int64_t M_src, const uint8_t* w_codes,
                   const uint8_t* w_scales, const int32_t* expert_offsets, int64_t E,
                   int64_t M_total, int64_t N, int64_t K, void* y, void* ws, size_t ws_bytes,
                   void* stream) {
  NV_REQUIRE(E >= 1 && E <= 1024 && M_total >= 0 && M_total < (1LL << 31) && M_src >= 0 && N >= 16 &&
                 N % (glu ? 32 : 16) == 0 && N <= (1 << 20) && K >= 128 && K % 128 == 0 &&
                 K <= (1 << 20),
             NVFP4_ERR_SHAPE,
             "%s: need 1 <= E <= 1024, 0 <= M_total < 2^31, N %% %d == 0, K %% 128 == 0, N and K <= "
             "2^20 (E=%lld M_total=%lld N=%lld K=%lld)",
             name, glu ? 32 : 16, (long long)E, (long long)M_total, (long long)N, (long long)K);
  NV_REQUIRE(a_rows != nullptr || M_src >= M_total, NVFP4_ERR_SHAPE,
             "%s: without a_rows, M_src must be >= M_total", name);
  NV_REQUIRE(M_total == 0 || M_src >= 1, NVFP4_ERR_SHAPE, "%s: M_src == 0", name);
  NV_REQUIRE(M_src < (1LL << 31) && M_src * K < (1LL << 33) && N * K < (1LL << 33),
             NVFP4_ERR_UNSUPPORTED, "%s: the activation's or one expert's codes exceed 4 GiB", name);
  NV_REQUIRE(w_codes && w_scales && expert_offsets && ws &&
                 (M_total == 0 || (a_codes && a_scales && y)),
             NVFP4_ERR_NULL, "%s: missing pointer", name);
  NV_REQUIRE(aligned(a_codes, 16) && aligned(w_codes, 16) && aligned(y, 16) && aligned(ws, 16) &&
                 aligned(a_scales, 4) && aligned(w_scales, 4) && aligned(a_rows, 4) &&
                 aligned(expert_offsets, 4),
             NVFP4_ERR_ALIGN, "%s: misaligned pointer", name);
  NV_REQUIRE(ws_bytes >= grouped_mxfp4_gemm_workspace_size(E, M_total, N, K), NVFP4_ERR_WORKSPACE,
             "%s: workspace too small", name);
  if (M_total == 0) return ok();
  MxGemmArgs p{a_codes, a_scales, a_rows, w_codes, w_scales, expert_offsets,
               static_cast<uint16_t*>(y), M_src, M_total, N, K, (int)E};
  hipStream_t s = as_stream(stream);
  const int64_t NO = glu ? N / 2 : N;
  const int64_t avg = (M_total + E - 1) / E;
  int64_t z = (avg + 31) / 32;
  if (z > 1024) z = 1024;
  const dim3 grid((unsigned)((NO + (glu ? 63 : 127)) / (glu ? 64 : 128)), (unsigned)E, (unsigned)z);
  if (glu)
    k_mx_few<2, 2, true><<<grid, 256, 0, s>>>(p);
  else
    k_mx_few<2, 2, false><<<grid, 256, 0, s>>>(p);
  return check_launch(name);
}

extern "C" {

size_t grouped_mxfp4_gemm_workspace_size(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  (void)M_total, (void)N, (void)K;
  if (E < 1 || E > 1024) return 256;
  return round_up((size_t)(E + 1) * sizeof(int32_t), 256);
}

int grouped_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const int32_t* a_rows,
                       int64_t M_src, const uint8_t* w_codes, const uint8_t* w_scales,
                       const int32_t* expert_offsets, int64_t E, int64_t M_total, int64_t N,
                       int64_t K, void* y, void* ws, size_t ws_bytes, void* stream) {
  return mx_gemm("grouped_mxfp4_gemm", false, a_codes, a_scales, a_rows, M_src, w_codes, w_scales,
                 expert_offsets, E, M_total, N, K, y, ws, ws_bytes, stream);
}

int grouped_mxfp4_gemm_swiglu(const uint8_t* a_codes, const uint8_t* a_scales,
                              const int32_t* a_rows, int64_t M_src, const uint8_t* w_codes,
                              const uint8_t* w_scales, const int32_t* expert_offsets, int64_t E,
                              int64_t M_total, int64_t N, int64_t K, void* h, void* ws,
                              size_t ws_bytes, void* stream) {
  return mx_gemm("grouped_mxfp4_gemm_swiglu", true, a_codes, a_scales, a_rows, M_src, w_codes,
                 w_scales, expert_offsets, E, M_total, N, K, h, ws, ws_bytes, stream);
}

}  // extern "C"
