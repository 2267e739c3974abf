// Gradients of the routing around the expert products: of the weighted
// un-permute and combine (moe_unpermute_combine) and of the routing weights
// (moe_permute: the softmax over the tk chosen experts of logit + bias).
//
//   out[t] = sum_j w[t][j] y[inv[t][j]]:   dy[inv[t][j]] = w[t][j] d_out[t],
//                                          dw[t][j] = d_out[t] . y[inv[t][j]]
//   w[t] = softmax(l[t][ids[t]]):          dl[t][ids[t][j]] = w_j (dw_j - sum_i w_i dw_i),
//                                          0 for the experts not chosen,
//                                          dbias = sum_t dl[t]
#include <type_traits>

#include "device.h"
#include "runtime.h"

namespace nvfp4 {

// One wave per (token, slot): the row's products and their sum in one pass.
// A token's slots are neighbouring waves, so its d_out row comes from HBM
// once and from the caches tk - 1 times.  Bound by memory: 131072 rows of 4096
// 452 us, 2.28 GB at 5.05 TB/s.
template <bool DW>
__global__ void __launch_bounds__(256)
k_combine_backward(const uint16_t* __restrict__ d_out, const uint16_t* __restrict__ y,
                   const int32_t* __restrict__ inv_perm, const float* __restrict__ topk_w,
                   int64_t P, int tk, int64_t N, uint16_t* __restrict__ dy,
                   float* __restrict__ d_topk_w) {
  const int lane = threadIdx.x & 63;
  for (int64_t slot = blockIdx.x * 4LL + (threadIdx.x >> 6); slot < P; slot += gridDim.x * 4LL) {
    const int64_t p = inv_perm[slot];
    if (p < 0 || p >= P) continue;
    const float w = topk_w[slot];
    const uint16_t* d_row = d_out + slot / tk * N;
    float dot = 0.0f;
    for (int64_t c = lane * 8; c < N; c += 512) {
      const uint4 d = *reinterpret_cast<const uint4*>(d_row + c);
      const uint32_t d4[4] = {d.x, d.y, d.z, d.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = bf16x2_rne(w * bf16_bits_to_f32(d4[i] & 0xFFFFu), w * bf16_bits_to_f32(d4[i] >> 16));
      if constexpr (DW) {
        const uint4 v = *reinterpret_cast<const uint4*>(y + p * N + c);
        const uint32_t v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dot = __builtin_fmaf(bf16_bits_to_f32(d4[i] & 0xFFFFu), bf16_bits_to_f32(v4[i] & 0xFFFFu), dot);
          dot = __builtin_fmaf(bf16_bits_to_f32(d4[i] >> 16), bf16_bits_to_f32(v4[i] >> 16), dot);
        }
      }
      *reinterpret_cast<uint4*>(dy + p * N + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if constexpr (DW) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
      if (lane == 0) d_topk_w[slot] = dot;
    }
  }
}

// A wave takes `per` consecutive tokens, as many at once as have their slots in
// 64 lanes (a token's slots are 2^sh >= tk neighbours, 64 >> sh tokens), so that
// one round trip brings the ids and weights of them all; the next ones' are
// under way while these rows are written.  Lane l holds the experts l, l + 64,
// ... of a row, finds its chosen ones by comparing with the row's ids, and
// writes whole rows.  An expert chosen twice by a token gets both gradients.
// BIAS: the workgroup's sum of its rows goes to part; a wave adds up at most 64
// rows in float32 and these sums in float64, as the terms of either sign cancel.
// 16384 tokens, 8 of 128 experts: 7.7 us, and 6 us for the sum of the parts; a
// wave that waits for one token's slots after the other 26 us in all.
template <int KPER, bool BIAS>
__global__ void __launch_bounds__(512)
k_route_backward(const int32_t* __restrict__ ids, const float* __restrict__ w,
                 const float* __restrict__ dw, int64_t T, int E, int tk, int sh, int per,
                 float* __restrict__ d_logits, float* __restrict__ part) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (blockIdx.x * 8LL + wave) * per;
  const int64_t t1 = t0 + per < T ? t0 + per : T;
  const int at_once = 64 >> sh, j_own = lane & ((1 << sh) - 1);
  double total[KPER];
#pragma unroll
  for (int i = 0; i < KPER; ++i) total[i] = 0.0;
  int id = -1;
  float wj = 0.0f, dj = 0.0f;
  auto fetch = [&](int64_t t) {
    const int64_t own = t + (lane >> sh);
    const bool in = own < t1 && j_own < tk;
    id = in ? ids[own * tk + j_own] : -1;
    wj = in ? w[own * tk + j_own] : 0.0f;
    dj = in ? dw[own * tk + j_own] : 0.0f;
  };
  fetch(t0);
  for (int64_t t = t0; t < t1; t += at_once) {
    float s = wj * dj;
    for (int o = 1 << sh >> 1; o > 0; o >>= 1) s += __shfl_xor(s, o);
    const float g = wj * (dj - s);
    const int now = id;
    fetch(t + at_once);
    const int n = t1 - t < at_once ? (int)(t1 - t) : at_once;
    float sum[KPER];
#pragma unroll
    for (int i = 0; i < KPER; ++i) sum[i] = 0.0f;
    for (int r = 0; r < n; ++r) {
      float v[KPER];
#pragma unroll
      for (int i = 0; i < KPER; ++i) v[i] = 0.0f;
      for (int j = 0; j < tk; ++j) {
        const int ej = __builtin_amdgcn_readlane(now, (r << sh) + j);
        const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), (r << sh) + j));
#pragma unroll
        for (int i = 0; i < KPER; ++i) v[i] += ej == lane + 64 * i ? gj : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < KPER; ++i) {
        const int e = lane + 64 * i;
        if (e < E) d_logits[(t + r) * E + e] = v[i];
        sum[i] += v[i];
      }
    }
    if constexpr (BIAS) {
#pragma unroll
      for (int i = 0; i < KPER; ++i) total[i] += (double)sum[i];
    }
  }
  if constexpr (BIAS) {
    __shared__ float acc[8][KPER * 64];
#pragma unroll
    for (int i = 0; i < KPER; ++i) acc[wave][lane + 64 * i] = (float)total[i];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 512) {
      double s = 0.0;
#pragma unroll
      for (int q = 0; q < 8; ++q) s += (double)acc[q][e];
      part[(int64_t)blockIdx.x * E + e] = (float)s;
    }
  }
}

// d_bias[e] = sum over the workgroups' at most 256 parts, in a fixed order: wave
// q of 16 takes every 16th, all loads at once, then the sixteen are added.
__global__ void __launch_bounds__(1024)
k_route_bias(const float* __restrict__ part, int n, int E, float* __restrict__ d_bias) {
  __shared__ double acc[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int b = wave + 16 * i;
    v[i] = e < E && b < n ? part[(int64_t)b * E + e] : 0.0f;
  }
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += (double)v[i];
  acc[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && e < E) {
    for (int q = 1; q < 16; ++q) s += acc[q][lane];
    d_bias[e] = (float)s;
  }
}

// tokens of a wave: at most 256 workgroups of eight waves, so that the sum of
// their parts is one round trip
static int64_t route_per(int64_t T) { return (T + 2047) / 2048; }
static int64_t route_blocks(int64_t T) { return (T + 8 * route_per(T) - 1) / (8 * route_per(T)); }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int moe_unpermute_combine_backward(const void* d_out, const void* y, const int32_t* inv_perm,
                                   const float* topk_w, int64_t T, int64_t tk, int64_t N, void* dy,
                                   float* d_topk_w, void* stream) {
  NV_REQUIRE(T >= 0 && T < (1LL << 31) && tk >= 1 && tk <= 32 && T * tk < (1LL << 31) && N >= 8 &&
                 N % 8 == 0 && N < (1LL << 31),
             NVFP4_ERR_SHAPE,
             "moe_unpermute_combine_backward: need T >= 0, 1 <= tk <= 32, T*tk < 2^31, "
             "N %% 8 == 0, 8 <= N < 2^31 (T=%lld tk=%lld N=%lld)",
             (long long)T, (long long)tk, (long long)N);
  if (T == 0) return ok();
  NV_REQUIRE(d_out && inv_perm && topk_w && dy && (y == nullptr) == (d_topk_w == nullptr),
             NVFP4_ERR_NULL,
             "moe_unpermute_combine_backward: missing pointer (y and d_topk_w go together)");
  NV_REQUIRE(aligned(d_out, 16) && aligned(y, 16) && aligned(dy, 16) && aligned(inv_perm, 4) &&
                 aligned(topk_w, 4) && aligned(d_topk_w, 4),
             NVFP4_ERR_ALIGN, "moe_unpermute_combine_backward: misaligned pointer");
  hipStream_t s = as_stream(stream);
  const int64_t P = T * tk;
  const int64_t nb = (P + 3) / 4;
  const unsigned g = (unsigned)(nb < (1 << 20) ? nb : 1 << 20);
  const uint16_t* dp = static_cast<const uint16_t*>(d_out);
  const uint16_t* yp = static_cast<const uint16_t*>(y);
  if (y)
    k_combine_backward<true><<<g, 256, 0, s>>>(dp, yp, inv_perm, topk_w, P, (int)tk, N,
                                               static_cast<uint16_t*>(dy), d_topk_w);
  else
    k_combine_backward<false><<<g, 256, 0, s>>>(dp, yp, inv_perm, topk_w, P, (int)tk, N,
                                                static_cast<uint16_t*>(dy), d_topk_w);
  return check_launch("moe_unpermute_combine_backward");
}

size_t moe_permute_backward_workspace_size(int64_t T, int64_t E) {
  if (T < 1 || T >= (1LL << 31) || E < 1 || E > 1024) return 256;
  return round_up((size_t)route_blocks(T) * (size_t)E * sizeof(float), 256);
}

int moe_permute_backward(const int32_t* topk_ids, const float* topk_w, const float* d_topk_w,
                         int64_t T, int64_t E, int64_t tk, float* d_logits, float* d_bias, void* ws,
                         size_t ws_bytes, void* stream) {
  NV_REQUIRE(T >= 0 && T < (1LL << 31) && E >= 1 && E <= 1024 && tk >= 1 && tk <= E && tk <= 32 &&
                 T * tk < (1LL << 31),
             NVFP4_ERR_SHAPE,
             "moe_permute_backward: need T >= 0, 1 <= tk <= min(E, 32), E <= 1024, T*tk < 2^31 "
             "(T=%lld E=%lld tk=%lld)",
             (long long)T, (long long)E, (long long)tk);
  NV_REQUIRE(T == 0 || (topk_ids && topk_w && d_topk_w && d_logits), NVFP4_ERR_NULL,
             "moe_permute_backward: missing pointer");
  NV_REQUIRE(aligned(topk_ids, 4) && aligned(topk_w, 4) && aligned(d_topk_w, 4) &&
                 aligned(d_logits, 4) && aligned(d_bias, 4) && aligned(ws, 16),
             NVFP4_ERR_ALIGN, "moe_permute_backward: misaligned pointer");
  hipStream_t s = as_stream(stream);
  if (T == 0) {
    if (!d_bias) return ok();
    fill_u32(reinterpret_cast<uint32_t*>(d_bias), E, 0u, s);
    return check_launch("moe_permute_backward");
  }
  NV_REQUIRE(!d_bias || ws, NVFP4_ERR_NULL, "moe_permute_backward: d_bias needs the workspace");
  NV_REQUIRE(!d_bias || ws_bytes >= moe_permute_backward_workspace_size(T, E), NVFP4_ERR_WORKSPACE,
             "moe_permute_backward: workspace too small");
  const int per = (int)route_per(T);
  int sh = 0;
  while (1 << sh < tk) ++sh;
  const int64_t nb = route_blocks(T);
  float* part = static_cast<float*>(ws);
  auto launch = [&](auto kper) {
    constexpr int KP = decltype(kper)::value;
    if (d_bias)
      k_route_backward<KP, true><<<(unsigned)nb, 512, 0, s>>>(topk_ids, topk_w, d_topk_w, T, (int)E,
                                                              (int)tk, sh, per, d_logits, part);
    else
      k_route_backward<KP, false><<<(unsigned)nb, 512, 0, s>>>(topk_ids, topk_w, d_topk_w, T, (int)E,
                                                               (int)tk, sh, per, d_logits, nullptr);
  };
  if (E <= 64)
    launch(std::integral_constant<int, 1>{});
  else if (E <= 128)
    launch(std::integral_constant<int, 2>{});
  else
    launch(std::integral_constant<int, 16>{});
  if (d_bias)
    k_route_bias<<<(unsigned)((E + 63) / 64), 1024, 0, s>>>(part, (int)nb, (int)E, d_bias);
  return check_launch("moe_permute_backward");
}

}  // extern "C"
