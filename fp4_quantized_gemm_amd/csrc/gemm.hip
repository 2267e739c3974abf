// Expert-grouped W4A4 GEMM with Residual Activation Compensation (QUADS:
// keep the native FP4 product over all of K and add back, for the few
// channels of largest activation residual, the residual times the same FP4
// weights; gist.science technical summary §2.2 B; arXiv abstract).
//
// Mapping of NVFP4 onto CDNA4 matrix cores.  gfx950's scaled FP4 MFMA applies
// power-of-two (E8M0) scales per 32 elements; NVFP4 needs a full E4M3 scale
// per 16 elements.  An element times its block scale, q * s, has at most
// 2 + 4 significant bits, so it is exact in bf16: the kernel decodes packed
// codes and scales into bf16 operands in registers and runs the bf16 MFMA,
// which makes every product exact and leaves only float32 accumulation
// rounding.  The residual correction is a K-extension of the same
// accumulator: acc = g_x * sum_K x~ w~  +  sum_S r w~,  y = bf16(g_w * acc).
//
// Tiling: a workgroup owns one (expert, 128-row tile, 128-column tile); its
// four waves own 64x64 each.  K advances 128 at a time through LDS, one row
// of a stage being 64 bytes of codes + 8 scale bytes + 8 pad (80-byte stride:
// conflict-free 16-byte reads).  Lane l of a wave reads the 16 bytes at
// k-offset 32*(l/16) of its row and feeds four MFMA k-slices from them; the
// k order inside an MFMA is permuted identically for A and B, which leaves
// the dot products unchanged.
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "device.h"
#include "mfma.h"
#include "runtime.h"

namespace nvfp4 {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kBK = 128;
constexpr int kRowBytes = 80;

struct GemmArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const float* g_x;
  const int32_t* a_rows;
  const uint16_t* R;
  const int32_t* S;
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  const float* g_w;
  const int32_t* offsets;
  const int32_t* tile_prefix;
  uint16_t* y;
  int64_t M_src, M_total, N, K;
  int E, k;
  // per-expert compensation: expert e's channels are S[e * s_stride ..]
  // (s_stride = k; 0 = one set for all experts), and R is indexed by
  // permuted row (r_perm = 1) instead of by activation row
  int64_t s_stride;
  int r_perm;
  // fused SwiGLU (large-tile kernel): glu_i = I > 0 means the weight rows
  // are [gate (I) | up (I)], a column tile pairs gate columns with the same
  // up columns, and y receives h = bf16(silu(gate) * up), [M_total][I];
  // h_amax (nullable) receives max |h| as bf16 bits (atomic max)
  int64_t glu_i;
  uint32_t* h_amax;
  // split of K over blockIdx.y (large-tile kernel, SPLIT instantiation):
  // slice s writes its float32 partial to part[s][M_total][N]
  int ksplit;
  float* part;
};

// tile_prefix[e] = number of 128-row tiles of experts before e; [E] = total
__global__ void __launch_bounds__(1024)
k_tile_prefix(const int32_t* __restrict__ offsets, int E, int64_t M_total, int bm,
              int32_t* __restrict__ prefix) {
  __shared__ int wsum[16];
  const int tid = threadIdx.x;
  int v = 0;
  if (tid < E) {
    int64_t lo = offsets[tid], hi = offsets[tid + 1];
    lo = lo < 0 ? 0 : (lo > M_total ? M_total : lo);
    hi = hi < lo ? lo : (hi > M_total ? M_total : hi);
    v = (int)((hi - lo + bm - 1) / bm);
  }
  int incl = v;
  for (int o = 1; o < 64; o <<= 1) {
    int u = __shfl_up(incl, o);
    if ((tid & 63) >= o) incl += u;
  }
  if ((tid & 63) == 63) wsum[tid >> 6] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < (tid >> 6); ++w) base += wsum[w];
  if (tid < E) prefix[tid] = base + incl - v;
  if (tid == E - 1) prefix[E] = base + incl;
}

__global__ void __launch_bounds__(256)
k_gemm_generic(GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smA[kBM * kRowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t smB[kBN * kRowBytes];
  __shared__ int32_t rows_src[kBM];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int g = lane >> 4, r16 = lane & 15;

  // which expert / row tile
  const int gt = blockIdx.x;
  if (gt >= p.tile_prefix[p.E]) return;
  int lo = 0, hi = p.E;                       // largest e with prefix[e] <= gt
  while (hi - lo > 1) {
    int mid = (lo + hi) >> 1;
    if (p.tile_prefix[mid] <= gt) lo = mid; else hi = mid;
  }
  const int e = lo;
  int64_t e_lo = p.offsets[e], e_hi = p.offsets[e + 1];
  e_lo = e_lo < 0 ? 0 : (e_lo > p.M_total ? p.M_total : e_lo);
  e_hi = e_hi < e_lo ? e_lo : (e_hi > p.M_total ? p.M_total : e_hi);
  const int64_t p0 = e_lo + (int64_t)(gt - p.tile_prefix[e]) * kBM;
  const int64_t n0 = (int64_t)blockIdx.y * kBN;
  const int64_t Kh = p.K / 2, Ks = p.K / 16;

  if (tid < kBM) {
    int64_t pr = p0 + tid;
    if (pr >= e_hi) pr = e_hi - 1;
    int64_t t = p.a_rows ? (int64_t)p.a_rows[pr] : pr;
    t = t < 0 ? 0 : (t >= p.M_src ? p.M_src - 1 : t);
    rows_src[tid] = (int32_t)t;
  }
  __syncthreads();

  const uint8_t* wc = p.w_codes + e * packed_codes_per_expert(p.N, p.K);
  const uint8_t* wsc = p.w_scales + e * packed_scales_per_expert(p.N, p.K);

  f32x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  for (int64_t k0 = 0; k0 < p.K; k0 += kBK) {
    // global -> registers
    uint4 ga[2], gb[2];
    uint2 gsa = make_uint2(0, 0), gsb = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = tid + 256 * i;
      const int r = q >> 2, part = q & 3;
      ga[i] = *reinterpret_cast<const uint4*>(p.a_codes + (int64_t)rows_src[r] * Kh + k0 / 2 + part * 16);
      int64_t n = n0 + r;
      if (n >= p.N) n = p.N - 1;
      gb[i] = *reinterpret_cast<const uint4*>(wc + wcode_offset(n, k0 + 32 * part, p.K));
    }
    if (tid < kBM) {
      gsa = *reinterpret_cast<const uint2*>(p.a_scales + (int64_t)rows_src[tid] * Ks + k0 / 16);
    } else {
      int64_t n = n0 + (tid - kBM);
      if (n >= p.N) n = p.N - 1;
      const uint8_t* t0 = wsc + wscale_offset(n, k0 / 16, p.K);   // two 64-k tiles
      gsb = make_uint2(*reinterpret_cast<const uint32_t*>(t0), *reinterpret_cast<const uint32_t*>(t0 + 64));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = tid + 256 * i;
      const int r = q >> 2, part = q & 3;
      *reinterpret_cast<uint4*>(smA + r * kRowBytes + part * 16) = ga[i];
      *reinterpret_cast<uint4*>(smB + r * kRowBytes + part * 16) = gb[i];
    }
    if (tid < kBM) *reinterpret_cast<uint2*>(smA + tid * kRowBytes + 64) = gsa;
    else *reinterpret_cast<uint2*>(smB + (tid - kBM) * kRowBytes + 64) = gsb;
    __syncthreads();

    // LDS -> registers (packed), decode per k-slice, MFMA
    uint4 ar[4], br[4];
    uint32_t as[4], bs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ra = wm * 64 + 16 * i + r16;
      ar[i] = *reinterpret_cast<const uint4*>(smA + ra * kRowBytes + 16 * g);
      as[i] = *reinterpret_cast<const uint16_t*>(smA + ra * kRowBytes + 64 + 2 * g);
      const int rb = wn * 64 + 16 * i + r16;
      br[i] = *reinterpret_cast<const uint4*>(smB + rb * kRowBytes + 16 * g);
      bs[i] = *reinterpret_cast<const uint16_t*>(smB + rb * kRowBytes + 64 + 2 * g);
    }
#pragma unroll
    for (int sl = 0; sl < 4; ++sl) {
      u32x4 A[4], B[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t wa = sl == 0 ? ar[i].x : sl == 1 ? ar[i].y : sl == 2 ? ar[i].z : ar[i].w;
        const uint32_t wb = sl == 0 ? br[i].x : sl == 1 ? br[i].y : sl == 2 ? br[i].z : br[i].w;
        A[i] = decode8_bf16(wa, e4m3_decode((as[i] >> (8 * (sl >> 1))) & 0xFFu));
        B[i] = decode8_bf16(wb, e4m3_decode((bs[i] >> (8 * (sl >> 1))) & 0xFFu));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma_bf16(A[i], B[j], acc[i][j]);
    }
  }

  // epilogue: x g_x, residual K-extension over S, x g_w, bf16 store
  const float gx = *p.g_x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] *= gx;

  for (int kc = 0; kc < p.k; kc += 32) {
    u32x4 A[4], B[4];
    int ch[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int slot = kc + 8 * g + t;
      int c = slot < p.k ? p.S[(int64_t)e * p.s_stride + slot] : -1;
      ch[t] = c < 0 ? -1 : (c >= p.K ? (int)p.K - 1 : c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = wm * 64 + 16 * i + r16;
      int64_t t = rows_src[lr];
      if (p.r_perm) t = p0 + lr < e_hi ? p0 + lr : e_hi - 1;
      const uint16_t* rr = p.R + t * p.k + kc + 8 * g;
      uint32_t v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = (kc + 8 * g + q < p.k) ? rr[q] : 0u;
      A[i] = u32x4{v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16)};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int64_t n = n0 + wn * 64 + 16 * j + r16;
      if (n >= p.N) n = p.N - 1;
      uint32_t v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (ch[q] < 0) { v[q] = 0u; continue; }
        const uint32_t byte = wc[wcode_offset(n, ch[q], p.K)];
        const float wq = e2m1_unpack2<0>((byte >> (4 * (ch[q] & 1))) & 0xFu).x;
        const float ws = e4m3_decode(wsc[wscale_offset(n, ch[q] >> 4, p.K)]);
        v[q] = __float_as_uint(wq * ws) >> 16;
      }
      B[j] = u32x4{v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16)};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = mfma_bf16(A[i], B[j], acc[i][j]);
  }

  const float gw = p.g_w[e];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int rr = 0; rr < 4; ++rr) {
      const int64_t prow = p0 + wm * 64 + 16 * i + 4 * g + rr;
      if (prow >= e_hi) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + wn * 64 + 16 * j + r16;
        if (n < p.N) p.y[prow * p.N + n] = (uint16_t)f32_to_bf16_rne(acc[i][j][rr] * gw);
      }
    }
  }
}


// ---------------------------------------------------------------------------
// Large-tile path (two kernels).
//
// 1. k_decode_a: the activation operand, codes and E4M3 block scales, is
//    decoded once per call into an exact f16 image x~ = q * s (at most 6
//    significant bits, magnitudes 2^-10 .. 2880, so f16 holds it exactly) in
//    the workspace.  Inside every 64-wide K block the eight 16-byte chunks
//    are stored in the order the matrix-core lanes consume them.
// 2. k_gemm_big: 256x256 per workgroup, eight waves of 256x32, K in steps of
//    64 through double-buffered LDS filled by buffer loads straight into
//    LDS.  A tiles arrive as f16; weight tiles arrive packed and each wave
//    decodes its 32 columns in registers: the hardware FP4 convert applies
//    the block scale's power of two, one packed f16 multiply its significand
//    (s = 2^E * mu, mu in [1, 2)).  Products run on v_mfma_f32_32x32x16_f16.
//    The weights of the selected residual channels are decoded per tile from
//    the channel-major part of the packed weights into an LDS tile (bf16,
//    exact); after the loop the correction runs on v_mfma_f32_32x32x16_bf16
//    into the same accumulators.
//
// MFMA 32x32x16 operand layout: lane l supplies row (or column) l % 32 and
// the 8 k values of group kg = l / 32.  Within a 64-wide K step, lane group
// kg at k-slice t (0..3) covers k in [32 kg + 8 t, +8) for both operands; the
// 16 accumulators of a lane hold column l % 32, rows 8 (r/4) + 4 kg + r % 4.
// ---------------------------------------------------------------------------
namespace big {
constexpr int BM = 256, BN = 256, BK = 64;
// LDS reads of 16 bytes serve 16 lanes per pass over 64 four-byte banks, so
// 16 consecutive rows of a fragment must land in 16 distinct 16-byte bank
// groups: with 128-byte A rows two rows share a 256-byte bank line, hence the
// A swizzle on row >> 1.  B keeps the code tiles' own order, in which a
// half's 16 rows are 256 consecutive bytes.
constexpr int A_BYTES = BM * BK * 2;           // f16 [256][64]: 8 chunks/row, chunk c at c ^ ((row >> 1) & 7)
constexpr int B_CODES = BN * 32;               // [16][2][16][16 B]: the packed code tiles as stored
constexpr int B_SCALES = BN * 4;               // [256][4 B]
constexpr int STAGE = A_BYTES + B_CODES + B_SCALES;   // 41984
constexpr int KMAX = 128;                      // residual channels held in LDS
constexpr int KSTEPS_MAX = 256;                // K <= 16384
constexpr int WSROW = KMAX * 2 + 16;           // bf16 row of the W_S tile (+pad)
constexpr int OUTROW = BN * 2 + 16;            // bf16 output staging row (+pad)
constexpr int OUT_ROWS = BM / 2;               // output staged in two halves
constexpr int WS_BYTES = BN * WSROW > OUT_ROWS * OUTROW ? BN * WSROW : OUT_ROWS * OUTROW;
}  // namespace big

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

template <int SEL>
__device__ __forceinline__ uint32_t dec2_f16(uint32_t w, float sc, h2_t mu) {
  h2_t v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, SEL);
  return __builtin_bit_cast(uint32_t, v * mu);
}

// 8 codes (one dword) -> 8 exact f16 values q * s.  `sc` is the block scale
// as float32 (the convert uses only its exponent), `mu` its significand.
__device__ __forceinline__ u32x4 decode8_f16(uint32_t w, float sc, h2_t mu) {
  return u32x4{dec2_f16<0>(w, sc, mu), dec2_f16<1>(w, sc, mu), dec2_f16<2>(w, sc, mu),
               dec2_f16<3>(w, sc, mu)};
}

__device__ __forceinline__ void scale_prep(uint32_t byte, float& sc, h2_t& mu) {
  const float s = __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
  const float m = __uint_as_float((__float_as_uint(s) & 0x007FFFFFu) | 0x3F800000u);
  mu = __builtin_bit_cast(h2_t, __builtin_amdgcn_cvt_pkrtz(m, m));
  sc = s;
}

__device__ __forceinline__ f32x16_t mfma32_f16(const u32x4& a, const u32x4& b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// codes [M][K/2] + scales [M][K/16] -> f16 image [M][K]; one thread per 8
// consecutive k (one code dword, one block scale), written to the chunk slot
// 2 t + kg of its 64-wide block, where k % 64 = 32 kg + 8 t.
__global__ void __launch_bounds__(256)
k_decode_a(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t M,
           int64_t K, uint16_t* __restrict__ img) {
  const int64_t per_row = K / 8;
  const int64_t total = M * per_row;
  for (int64_t q = blockIdx.x * 256LL + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
    const int64_t m = q / per_row;
    const int64_t c8 = q - m * per_row;
    const int64_t k = c8 * 8;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + m * (K / 2) + k / 2);
    float sc;
    h2_t mu;
    scale_prep(scales[m * (K / 16) + k / 16], sc, mu);
    const u32x4 v = decode8_f16(w, sc, mu);
    const int kk = (int)(k & 63), kg = kk >> 5, t = (kk & 31) >> 3;
    uint16_t* dst = img + m * K + (k - kk) + (2 * t + kg) * 8;
    *reinterpret_cast<uint4*>(dst) = make_uint4(v.x, v.y, v.z, v.w);
  }
}

// Eight waves (two per SIMD, so one wave's waits are covered by the other's
// MFMAs): wave w owns all 256 rows and columns 32 w .. +32 of the 256x256
// tile, so each weight fragment it decodes feeds eight MFMAs (the decode's
// instructions are what limits a SIMD's issue).
//
// W16 = true is the trainer-side W4A16 product (bf16 activations times the
// same dequantized weights): A is the bf16 activation itself, staged the same
// way (the 8-element chunk the image would hold in slot c is chunk
// 4 (c & 1) + (c >> 1) of the row's 64-wide block), the weights are decoded to
// bf16 (q * s, exact), the MFMA is bf16, and there is no correction.
template <bool W16, bool SPLIT = false>
__global__ void __launch_bounds__(512, 1)
k_gemm_big(GemmArgs p, const uint8_t* __restrict__ a_img, int n_tiles, int m_tiles) {
  using namespace big;
  // The two k-step stages are separate LDS objects and the loop below is
  // unrolled by two, so every access names its stage statically: the
  // compiler can then tell the asynchronous global->LDS fill of one stage
  // from the reads of the other and does not wait for that fill before
  // computing on the current stage.
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t wsl[WS_BYTES];   // W_S tile, then output staging
  __shared__ int32_t rows_src[BM];
  __shared__ int32_t s_sel[KMAX];                      // the first W_S tile's channels

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // 0..7, wave-uniform (SGPR)
  const int wn = wave;
  const int kg = lane >> 5, r32 = lane & 31;

  // tile order: groups of 4 row tiles x all column tiles, so the workgroups
  // in flight share A and weight tiles through L2.  Workgroup b runs on XCD
  // b % 8 (each XCD has its own L2), so each XCD takes a contiguous range of
  // that order, counted over the real tiles (the grid is sized for the most
  // padding tiles the expert boundaries can add; the rest exit).
  int v;
  {
    const int real_m = p.tile_prefix[p.E];
    const int real_blocks = ((real_m + 3) / 4) * 4 * n_tiles;
    const int per_xcd = (real_blocks + 7) / 8;
    const int b = (int)blockIdx.x;
    const int loc = b >> 3;
    if (loc >= per_xcd) return;
    v = (b & 7) * per_xcd + loc;
    if (v >= real_blocks) return;
  }
  const int group = 4 * n_tiles;
  const int gi = v / group, gr = v - gi * group;
  if (4 * gi >= m_tiles) return;
  const int gm = m_tiles - 4 * gi < 4 ? m_tiles - 4 * gi : 4;
  const int gt = 4 * gi + gr % gm;                // row tile
  const int nt = gr / gm;                         // column tile
  if (gt >= p.tile_prefix[p.E] || nt >= n_tiles) return;
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    int mid = (lo + hi) >> 1;
    if (p.tile_prefix[mid] <= gt) lo = mid; else hi = mid;
  }
  const int e = lo;
  int64_t e_lo = p.offsets[e], e_hi = p.offsets[e + 1];
  e_lo = e_lo < 0 ? 0 : (e_lo > p.M_total ? p.M_total : e_lo);
  e_hi = e_hi < e_lo ? e_lo : (e_hi > p.M_total ? p.M_total : e_hi);
  const int64_t p0 = e_lo + (int64_t)(gt - p.tile_prefix[e]) * BM;
  const int64_t n0 = (int64_t)nt * BN;
  // weight row of the tile's local row r; with the fused SwiGLU the tile
  // holds gate columns 128 nt .. +127 (rows 0..127) and the same up columns
  // I + 128 nt .. (rows 128..255)
  auto wrow = [&](int r) -> int64_t {
    if (W16 || p.glu_i == 0) return n0 + r;
    int64_t c = (int64_t)nt * 128 + (r & 127);
    c = c < p.glu_i ? c : p.glu_i - 1;
    return r < 128 ? c : p.glu_i + c;
  };
  const uint32_t K2 = (uint32_t)(p.K * 2);
  // channels of the correction (K slices: all on slice 0, none on the others)
  const int kk = (W16 || (SPLIT && blockIdx.y != 0)) ? 0 : p.k;
  // The selected channels' weight columns go through LDS KMAX channels (one
  // W_S tile, bf16, zero past k) at a time; the first tile is loaded with
  // the first k-step.
  const int ws_ch = kk > KMAX ? KMAX : (int)((kk + 15) & ~15);   // channels per W_S tile
  // the residual rows by direct loads in 64-channel halves (k % 64 == 0);
  // otherwise each lane loads its own
  const bool rdma = kk > 0 && (kk & 63) == 0;

  auto sel_col = [&](int c) { return c < 0 ? 0 : (c >= p.K ? (int)p.K - 1 : c); };
  if (tid < BM) {
    int64_t pr = p0 + tid;
    if (pr >= e_hi) pr = e_hi - 1;
    int64_t t = p.a_rows ? (int64_t)p.a_rows[pr] : pr;
    rows_src[tid] = (int32_t)(t < 0 ? 0 : (t >= p.M_src ? p.M_src - 1 : t));
  } else if (tid - BM < ws_ch) {
    const int j = tid - BM;
    s_sel[j] = sel_col(p.S[(int64_t)e * p.s_stride + (j < kk ? j : kk - 1)]);
  }
  __syncthreads();
  const int nk = (int)(p.K / BK);
  // this workgroup's k-steps: all of them, or slice blockIdx.y of ksplit
  // (an even number of steps each)
  const int nks = SPLIT ? nk / p.ksplit : nk;
  const int kt_lo = SPLIT ? (int)blockIdx.y * nks : 0;
  const int kt_hi = kt_lo + nks;

  const uint8_t* wc = p.w_codes + e * packed_codes_per_expert(p.N, p.K);
  const uint8_t* wsc = p.w_scales + e * packed_scales_per_expert(p.N, p.K);

  // byte offsets of this lane's staging loads (fixed over K): A 2048 chunks
  // (4 per thread), B codes 512 chunks (1 per thread), B scales 256 dwords
  // (waves 0..3)
  uint32_t off_a[4], off_b, off_s = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = (i * 8 + wave) * 64 + lane;
    const int r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
    off_a[i] = (uint32_t)rows_src[r] * K2 + 16u * (W16 ? 4 * (c & 1) + (c >> 1) : c);
  }
  {
    // lane q of the stage's B area takes bytes 16 q .. of the tiles in their
    // stored order (16-row block q / 32, 32-column half (q / 16) % 2, row
    // q % 16), so a load instruction reads two whole 512-byte code tiles
    const int q = wave * 64 + lane;
    const int r = 16 * (q >> 5) + (q & 15), c = (q >> 4) & 1;
    int64_t n = wrow(r);
    if (n >= p.N) n = p.N - 1;
    off_b = (uint32_t)wcode_offset(n, 32 * c, p.K);   // + 8 k0: the step's tile
  }
  if (wave == 7) {
    // the step's 256 x 4 scale bytes in one instruction: lane l takes rows
    // 4 l .. 4 l + 3 (16 bytes of one scale tile: a 4-row group starting at
    // a multiple of 4 never crosses a 16-row tile, as N and the gate/up
    // split are multiples of 8)
    const int r = 4 * lane;
    int64_t n;
    if (W16 || p.glu_i == 0) {
      n = n0 + r;
      if (n + 4 > p.N) n = p.N - 4;
    } else {
      int64_t c = (int64_t)nt * 128 + (r & 127);
      if (c + 4 > p.glu_i) c = p.glu_i - 4;
      n = r < 128 ? c : p.glu_i + c;
    }
    off_s = (uint32_t)wscale_offset(n, 0, p.K);   // + k0: the step's tile
  }
  // rows of the tile inside the expert: a load instruction covers 8
  // consecutive rows, and one whose rows all lie past the expert's last row
  // is skipped (its LDS rows then hold stale values, which only reach output
  // rows that are never stored: an MFMA's output row depends only on its own
  // A row)
  const int64_t vt = e_hi - p0;
  const int v_tile = vt > BM ? BM : (int)vt;
  // Stage loads are buffer loads into LDS: the lane's byte offset (fixed
  // over K) is the VGPR offset and the step, k0 times the bytes per column,
  // the scalar offset, so no per-step address register exists (the image
  // and one expert's code tiles are below 4 GiB; a buffer's range is its
  // size, and a load past it reads zeros).
  const __amdgpu_buffer_rsrc_t rs_a =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a_img), (short)0,
                                        (int)(uint32_t)((uint64_t)p.M_src * (uint64_t)p.K * 2),
                                        kBufferRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(wc), (short)0, (int)(uint32_t)(p.N * p.K / 2), kBufferRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs_s = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(wsc), (short)0, (int)(uint32_t)(p.N * p.K / 16), kBufferRsrcWord3);
  auto issue_loads = [&](uint8_t* st, uint32_t k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((i * 8 + wave) * 8 < v_tile)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(st + (i * 8 + wave) * 1024), 16,
                                                 off_a[i], k0 * 2, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, lds_ptr(st + A_BYTES + wave * 1024), 16, off_b,
                                             k0 * 8, 0, 0);
    if (wave == 7)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_s, lds_ptr(st + A_BYTES + B_CODES), 16, off_s, k0,
                                               0, 0);
  };

  // W_S tile of channels c0 .. c0 + ws_ch into wsl, read from the channel-
  // major part of the packed weights (a selected channel is N / 2 code bytes
  // and, for its block of 16 channels, N scale bytes): wave u takes channels
  // c0 + 16 u .. +16 (u < ws_ch / 16), lane l the tile rows 8 (l % 32) .. +8
  // (eight consecutive weight rows) and channels 8 (l / 32) .. +8 of those,
  // one code dword and two scale dwords per channel (whole 128-byte lines
  // across the wave).  ws_issue loads them, ws_store decodes bf16 q * s
  // (exact; zero past k) and writes each row's 8 channels as one 16-byte
  // piece.
  const uint8_t* wcm = wc + (int64_t)p.N * p.K / 2;     // codes [K][N / 2]
  const uint8_t* wscm = wsc + (int64_t)p.N * p.K / 16;  // scales [K / 16][N]
  const int ws_r8 = 8 * (lane & 31);
  const int ws_cl = 16 * wave + 8 * (lane >> 5);         // the lane's first channel slot
  uint32_t wq[8], wsa[8], wsb[8];
  auto ws_issue = [&](int c0) __attribute__((always_inline)) {
    if (16 * wave >= ws_ch) return;
    int64_t n;                                          // first of the lane's 8 weight rows
    if (W16 || p.glu_i == 0) {
      n = n0 + ws_r8;
      if (n + 8 > p.N) n = p.N - 8;
    } else {
      int64_t c = (int64_t)nt * 128 + (ws_r8 & 127);
      if (c + 8 > p.glu_i) c = p.glu_i - 8;
      n = ws_r8 < 128 ? c : p.glu_i + c;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int slot = c0 + ws_cl + j;
      const int c = c0 == 0 ? s_sel[slot < KMAX ? slot : KMAX - 1]
                            : sel_col(p.S[(int64_t)e * p.s_stride + (slot < kk ? slot : kk - 1)]);
      wq[j] = *reinterpret_cast<const uint32_t*>(wcm + (uint32_t)c * (uint32_t)(p.N / 2) +
                                                 (uint32_t)(n >> 1));
      const uint2 sv = *reinterpret_cast<const uint2*>(wscm + (uint32_t)(c >> 4) * (uint32_t)p.N +
                                                       (uint32_t)n);
      wsa[j] = sv.x;
      wsb[j] = sv.y;
    }
  };
  auto ws_store = [&](int c0) __attribute__((always_inline)) {
    if (16 * wave >= ws_ch) return;
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = c0 + ws_cl + j < kk ? wq[j] : 0u;   // +0 past k
    // rows 2 h and 2 h + 1: code byte h of each channel, scale bytes 2 h, 2 h + 1
    auto rows2 = [&](auto h_c) __attribute__((always_inline)) {
      constexpr int H = decltype(h_c)::value;
      float v0[8], v1[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const f32x2 f = e2m1_unpack2<H>(q[j]);
        const int sw = H < 2 ? (int)wsa[j] : (int)wsb[j];
        v0[j] = f.x * __builtin_amdgcn_cvt_f32_fp8(sw, (2 * H) & 3);
        v1[j] = f.y * __builtin_amdgcn_cvt_f32_fp8(sw, (2 * H + 1) & 3);
      }
      *reinterpret_cast<uint4*>(wsl + (ws_r8 + 2 * H) * WSROW + 2 * ws_cl) =
          make_uint4(pack_hi16(v0[0], v0[1]), pack_hi16(v0[2], v0[3]), pack_hi16(v0[4], v0[5]),
                     pack_hi16(v0[6], v0[7]));
      *reinterpret_cast<uint4*>(wsl + (ws_r8 + 2 * H + 1) * WSROW + 2 * ws_cl) =
          make_uint4(pack_hi16(v1[0], v1[1]), pack_hi16(v1[2], v1[3]), pack_hi16(v1[4], v1[5]),
                     pack_hi16(v1[6], v1[7]));
    };
    rows2(std::integral_constant<int, 0>{});
    rows2(std::integral_constant<int, 1>{});
    rows2(std::integral_constant<int, 2>{});
    rows2(std::integral_constant<int, 3>{});
  };

  // residual rows for the correction, staged like the A image: 64 channels
  // of the tile's 256 rows per stage, 8-channel chunks swizzled as A's
  // (whole 64-channel halves, so only when k % 64 == 0)
  auto issue_r = [&](uint8_t* st, int cb0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = (i * 8 + wave) * 64 + lane;
      const int r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
      const int64_t rr = p.r_perm ? (p0 + r < e_hi ? p0 + r : e_hi - 1) : rows_src[r];
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.R) +
                           (uint32_t)rr * (uint32_t)(2 * p.k) + 2u * (uint32_t)(cb0 + 8 * c);
      __builtin_amdgcn_global_load_lds(src, st + (i * 8 + wave) * 1024, 16, 0, 0);
    }
  };

  f32x16_t acc[8][1];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 1; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int swa = (r32 >> 1) & 7;                  // A rows = 32 i + r32 (+ multiples of 32)
  // the lane's B fragment in the stage: row wn * 32 + r32, half kg, in the
  // code tiles' order (the empty asm keeps the sum an opaque offset from the
  // stage, so the compiler still tells the two stages apart)
  int b_off = (2 * wn + (r32 >> 4)) * 512 + kg * 256 + (r32 & 15) * 16;
  asm volatile("" : "+v"(b_off));

  // one k-step on stage `ab` while stage `nxt` fills with step kt + 1; the
  // wave computes its first NV 32-row blocks (the others lie past the
  // expert's last row)
  auto kstep = [&](const uint8_t* ab, uint8_t* nxt, int kt, auto nv_c) __attribute__((always_inline)) {
    constexpr int NV = decltype(nv_c)::value;
    if (kt + 1 < kt_hi) issue_loads(nxt, (uint32_t)(kt + 1) * BK);
    else if (rdma) issue_r(nxt, 0);
    const uint8_t* bb = ab + A_BYTES;
    const uint8_t* sb = bb + B_CODES;

    uint4 br[1];
    uint32_t bs[1];
#pragma unroll
    for (int j = 0; j < 1; ++j) {
      const int rb = wn * 32 + 32 * j + r32;
      br[j] = *reinterpret_cast<const uint4*>(bb + b_off);
      bs[j] = *reinterpret_cast<const uint16_t*>(sb + rb * 4 + 2 * kg);
    }
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
      float sbv[1];
      h2_t mb[1];
#pragma unroll
      for (int j = 0; j < 1; ++j) {
        if constexpr (W16) sbv[j] = e4m3_decode((bs[j] >> (8 * hb)) & 0xFFu);
        else scale_prep((bs[j] >> (8 * hb)) & 0xFFu, sbv[j], mb[j]);
      }
#pragma unroll
      for (int s2 = 0; s2 < 2; ++s2) {
        const int t = 2 * hb + s2;
        u32x4 A[8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int ra = 32 * i + r32;
          const uint4 v4 = *reinterpret_cast<const uint4*>(ab + ra * 128 + (((2 * t + kg) ^ swa) << 4));
          A[i] = u32x4{v4.x, v4.y, v4.z, v4.w};
        }
#pragma unroll
        for (int j = 0; j < (NV > 0 ? 1 : 0); ++j) {
          const uint32_t w = t == 0 ? br[j].x : t == 1 ? br[j].y : t == 2 ? br[j].z : br[j].w;
          if constexpr (W16) {
            const u32x4 B = decode8_bf16(w, sbv[j]);
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[i][j] = mfma32_bf16(A[i], B, acc[i][j]);
          } else {
            const u32x4 B = decode8_f16(w, sbv[j], mb[j]);
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[i][j] = mfma32_f16(A[i], B, acc[i][j]);
          }
        }
      }
    }

    wait_vmem0();
    __syncthreads();
  };

  issue_loads(st0, (uint32_t)kt_lo * BK);
  if (kk > 0) ws_issue(0);
  wait_vmem0();
  __syncthreads();
  if (kk > 0) ws_store(0);                       // (read after the k-steps' barriers)
  // the tile's valid rows: expert tail tiles run fewer MFMAs (their first NV
  // 32-row blocks; every wave still takes part in the loads and barriers).
  // nk is even (K % 128 == 0).
  auto run = [&](auto nv_c) __attribute__((always_inline)) {
    for (int kt = kt_lo; kt < kt_hi; kt += 2) {
      kstep(st0, st1, kt, nv_c);
      kstep(st1, st0, kt + 1, nv_c);
    }
  };
  if (W16 || v_tile > 128)       // (the W4A16 kernel keeps one loop: less code)
    run(std::integral_constant<int, 8>{});
  else if (v_tile > 64)
    run(std::integral_constant<int, 4>{});
  else if (v_tile > 32)
    run(std::integral_constant<int, 2>{});
  else
    run(std::integral_constant<int, 1>{});

  // epilogue: x g_x, residual K-extension (16 channels per MFMA), x g_w.
  // Residual operand loads are issued in batches of four chunks, then consumed.
  if constexpr (!W16) {
    const float gx = *p.g_x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 1; ++j) acc[i][j] *= gx;
  }

  // (the loop ends on stage st1: the first residual half is in st0)
  auto rac_half = [&](const uint8_t* rb, int cb0) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u32x4 A[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ra = 32 * i + r32;
        const uint4 v4 = *reinterpret_cast<const uint4*>(rb + ra * 128 + (((2 * c + kg) ^ swa) << 4));
        A[i] = u32x4{v4.x, v4.y, v4.z, v4.w};
      }
      const int slot = cb0 + 16 * c + 8 * kg;
#pragma unroll
      for (int j = 0; j < 1; ++j) {
        const uint4 vv = *reinterpret_cast<const uint4*>(wsl + (wn * 32 + 32 * j + r32) * WSROW + 2 * slot);
        const u32x4 B = u32x4{vv.x, vv.y, vv.z, vv.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i][j] = mfma32_bf16(A[i], B, acc[i][j]);
      }
    }
  };
  if (rdma) {
    // W_S tiles of KMAX channels; a tile's residual rows in two 64-channel
    // halves (the first tile's first half arrived with the last k-step)
#pragma unroll 1
    for (int c0 = 0; c0 < kk; c0 += KMAX) {
      const bool two = kk - c0 > 64;
      if (c0 > 0) {
        __syncthreads();                       // the last reads of wsl and the stages are done
        ws_issue(c0);
        issue_r(st0, c0);
      }
      if (two) issue_r(st1, c0 + 64);
      if (c0 > 0) {
        ws_store(c0);
        wait_vmem0();
        __syncthreads();
      }
      rac_half(st0, 0);
      if (two) {
        wait_vmem0();
        __syncthreads();
        rac_half(st1, 64);
      }
    }
  }
  // (k % 64 != 0: each lane loads its residual rows' 8-channel pieces)
#pragma unroll 1
  for (int cb = 0; !rdma && cb < kk; cb += 16) {
    const int slot = cb + 8 * kg;
    u32x4 A[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int lr = 32 * i + r32;
      int64_t t = rows_src[lr];
      if (p.r_perm) t = p0 + lr < e_hi ? p0 + lr : e_hi - 1;
      const uint16_t* rr = p.R + t * kk + slot;
      if ((kk & 7) == 0 && slot + 8 <= kk) {
        const uint4 vv = *reinterpret_cast<const uint4*>(rr);
        A[i] = u32x4{vv.x, vv.y, vv.z, vv.w};
      } else {
        uint32_t vv[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) vv[q] = (slot + q < kk) ? rr[q] : 0u;
        A[i] = u32x4{vv[0] | (vv[1] << 16), vv[2] | (vv[3] << 16), vv[4] | (vv[5] << 16),
                     vv[6] | (vv[7] << 16)};
      }
    }
    const uint4 vv = *reinterpret_cast<const uint4*>(wsl + (wn * 32 + r32) * WSROW + 2 * slot);
    const u32x4 B = u32x4{vv.x, vv.y, vv.z, vv.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = mfma32_bf16(A[i], B, acc[i][0]);
  }

  if constexpr (SPLIT) {
    // this slice's float32 partial, with g_x (and on slice 0 the
    // correction); g_w and the rounding come in the fixed-order reduction.
    // Staged through LDS a 64-row quarter of the tile at a time for 16-byte
    // row stores.
    float* dst = p.part + (int64_t)blockIdx.y * p.M_total * p.N;
    constexpr int FROW = BN * 4 + 16;            // float32 staging row (+pad)
    static_assert(64 * FROW <= WS_BYTES, "quarter staging fits the W_S tile");
#pragma unroll
    for (int qd = 0; qd < 4; ++qd) {
      __syncthreads();
#pragma unroll
      for (int ii = 0; ii < 2; ++ii)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = 32 * ii + 8 * (r >> 2) + 4 * kg + (r & 3);
          const int col = wn * 32 + r32;
          *reinterpret_cast<float*>(wsl + row * FROW + 4 * col) = acc[2 * qd + ii][0][r];
        }
      __syncthreads();
      for (int q = tid; q < 64 * (BN / 4); q += 512) {
        const int row = q / (BN / 4), ch = q % (BN / 4);
        const int64_t prow = p0 + 64 * qd + row;
        const int64_t n = n0 + ch * 4;
        if (prow < e_hi && n < p.N)
          *reinterpret_cast<float4*>(dst + prow * p.N + n) =
              *reinterpret_cast<const float4*>(wsl + row * FROW + ch * 16);
      }
    }
    return;
  }

  // y = bf16(g_w * acc), staged through LDS (one 128-row half at a time)
  // for 16-byte row stores
  const float gw = p.g_w[e];
  uint32_t hmax = 0;                             // max |h| bits (fused SwiGLU)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * i + 8 * (r >> 2) + 4 * kg + (r & 3);
        const int col = wn * 32 + r32;
        *reinterpret_cast<uint16_t*>(wsl + row * OUTROW + 2 * col) =
            (uint16_t)f32_to_bf16_rne(acc[4 * h + i][0][r] * gw);
      }
    __syncthreads();
    if (p.glu_i > 0) {
      // h = bf16(silu(gate) * up) of the staged bf16 outputs: gate columns
      // in the first 128 of the row, the matching up columns in the next 128
      for (int q = tid; q < OUT_ROWS * (BN / 16); q += 512) {
        const int row = q / (BN / 16), ch = q % (BN / 16);
        const int64_t prow = p0 + h * OUT_ROWS + row;
        const int64_t c = (int64_t)nt * 128 + ch * 8;
        if (prow < e_hi && c < p.glu_i) {
          const uint4 g4 = *reinterpret_cast<const uint4*>(wsl + row * OUTROW + ch * 16);
          const uint4 u4 = *reinterpret_cast<const uint4*>(wsl + row * OUTROW + 256 + ch * 16);
          const uint4 o = make_uint4(swiglu_pair(g4.x, u4.x), swiglu_pair(g4.y, u4.y),
                                     swiglu_pair(g4.z, u4.z), swiglu_pair(g4.w, u4.w));
          *reinterpret_cast<uint4*>(p.y + prow * p.glu_i + c) = o;
          hmax = max(hmax, absmax_bf16x8(o));
        }
      }
    } else {
      for (int q = tid; q < OUT_ROWS * (BN / 8); q += 512) {
        const int row = q / (BN / 8), ch = q % (BN / 8);
        const int64_t prow = p0 + h * OUT_ROWS + row;
        const int64_t n = n0 + ch * 8;
        if (prow < e_hi && n < p.N)
          *reinterpret_cast<uint4*>(p.y + prow * p.N + n) =
              *reinterpret_cast<const uint4*>(wsl + row * OUTROW + ch * 16);
      }
    }
  }
  if (p.glu_i > 0 && p.h_amax != nullptr) block_atomic_max<512>(hmax, p.h_amax);
}

// y[p] = bf16(g_w[e] * sum_s part[s][p]) over the K slices in order s = 0, 1,
// ..., for row p of expert e; 8 columns per thread
__global__ void __launch_bounds__(256)
k_split_reduce(const float* __restrict__ part, int ksplit, int64_t M_total, int64_t N,
               const int32_t* __restrict__ offsets, int E, const float* __restrict__ g_w,
               uint16_t* __restrict__ y) {
  const int64_t n8 = N / 8;
  for (int64_t q = blockIdx.x * 256LL + threadIdx.x; q < M_total * n8;
       q += (int64_t)gridDim.x * 256) {
    const int64_t row = q / n8, c = (q - row * n8) * 8;
    int lo = 0, hi = E;                          // last e with offsets[e] <= row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (offsets[mid] <= row) lo = mid; else hi = mid;
    }
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int sp = 0; sp < ksplit; ++sp) {
      const float4* src = reinterpret_cast<const float4*>(part + ((int64_t)sp * M_total + row) * N + c);
      const float4 a = src[0], b = src[1];
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    const float gw = g_w[lo];
    uint4 o;
    o.x = f32_to_bf16_rne(v[0] * gw) | (f32_to_bf16_rne(v[1] * gw) << 16);
    o.y = f32_to_bf16_rne(v[2] * gw) | (f32_to_bf16_rne(v[3] * gw) << 16);
    o.z = f32_to_bf16_rne(v[4] * gw) | (f32_to_bf16_rne(v[5] * gw) << 16);
    o.w = f32_to_bf16_rne(v[6] * gw) | (f32_to_bf16_rne(v[7] * gw) << 16);
    *reinterpret_cast<uint4*>(y + row * N + c) = o;
  }
}

// h [M][I] = bf16(silu(gate) * up) of y [M][2I] = [gate | up], 8 columns per
// thread (the fused SwiGLU for shapes the large-tile kernel does not take)
__global__ void __launch_bounds__(256)
k_swiglu_rows(const uint16_t* __restrict__ y, int64_t M, int64_t I, uint16_t* __restrict__ h,
              uint32_t* __restrict__ h_amax) {
  const int64_t n8 = M * (I / 8);
  uint32_t m8 = 0;
  for (int64_t q = blockIdx.x * 256LL + threadIdx.x; q < n8; q += (int64_t)gridDim.x * 256) {
    const int64_t m = q / (I / 8), c = (q - m * (I / 8)) * 8;
    const uint4 g4 = *reinterpret_cast<const uint4*>(y + m * 2 * I + c);
    const uint4 u4 = *reinterpret_cast<const uint4*>(y + m * 2 * I + I + c);
    const uint4 o = make_uint4(swiglu_pair(g4.x, u4.x), swiglu_pair(g4.y, u4.y),
                               swiglu_pair(g4.z, u4.z), swiglu_pair(g4.w, u4.w));
    *reinterpret_cast<uint4*>(h + m * I + c) = o;
    m8 = max(m8, absmax_bf16x8(o));
  }
  if (h_amax != nullptr) block_atomic_max<256>(m8, h_amax);
}

// ---------------------------------------------------------------------------
// Decode-sized grouped GEMM: a few rows per expert, so the weights dominate
// the traffic and every expert's weights should cross HBM once.  A
// workgroup takes a few consecutive blocks of 256 weight rows of one expert
// (one round of workgroups fills the chip) and streams them as one sequence
// of K chunks of 256; each of its 4 waves streams 64 weight rows (4 blocks of
// 16) with register loads one chunk ahead, and multiplies them with all of
// the expert's rows (token tiles of 16, up to TMAX per pass) on 16x16x32 f16
// MFMAs.  Both operands are
// decoded from NVFP4 codes in registers (exact in f16), so no activation
// image is needed.  Weight rows are the MFMA's M side, tokens its N side.
//
// Lane l covers weight (or token) row l % 16 and, within a chunk at k0,
// k in [k0 + 64 (l / 16), +64): 32 code bytes and four block scales, so the
// four lanes of a row read its whole 128-byte line of the chunk together (a
// line split over two chunks was evicted from L2 between its halves).  MFMA
// step s (0..7) takes the lane's code dword s, i.e. k0 + 64 (l / 16) + 8 s + i
// in the instruction's k slot 8 (l / 16) + i; both operands use this order.
// The residual correction runs after each block (bf16 MFMAs over the
// selected channels, whose weight columns are gathered into LDS from the
// channel-major part of the packed weights during the block's last chunks).
// ---------------------------------------------------------------------------
namespace dec {
constexpr int ROWS = 256;
constexpr int KC = 256;
constexpr int TMAX = 2;
constexpr int KMAX = 128;
constexpr int CHUNKS_MAX = 64;            // K <= 16384
}  // namespace dec

typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma16_f16(const u32x4& a, const u32x4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16_bf16(const u32x4& a, const u32x4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// dword s (0..7) of a lane's 32 code bytes
// (selects, not indexing: a runtime index would put the arrays in scratch)
__device__ __forceinline__ uint32_t dword_of(const uint4 (&v)[2], int s) {
  const uint32_t a = (s & 1) ? v[0].y : v[0].x, b = (s & 1) ? v[0].w : v[0].z;
  const uint32_t c = (s & 1) ? v[1].y : v[1].x, d = (s & 1) ? v[1].w : v[1].z;
  const uint32_t lo = (s & 2) ? b : a, hi = (s & 2) ? d : c;
  return (s & 4) ? hi : lo;
}

struct DecChunk {
  uint4 wc[4][2];          // weight codes, row blocks 0..3, 32 bytes each
  uint32_t ws[4];          // their four block scales
  uint2 tc[dec::TMAX];     // token codes of this wave's two MFMA steps
  uint32_t ts[dec::TMAX];  // the token rows' four block scales
};

// Dynamic LDS: token fragments [2][TMAX][8 steps][64 lanes][16 B], then the
// W_S tile [256][wsrow] (wsrow = 2 * k rounded up to 32, + 16; none for k = 0).
constexpr int kDecTokBytes = 2 * dec::TMAX * 8 * 64 * 16;
constexpr int kDecStaticLds = 4 * dec::KMAX + 16;
constexpr int kLdsPerCu = 160 * 1024;

// W16 = true is the trainer-side W4A16 product on decode-sized problems: the
// tokens are bf16 activations x [M_src][K] (p.a_codes holds their address),
// copied by global->LDS loads straight into the token-fragment slots instead
// of being decoded (so they take no registers), the weights are decoded to
// bf16 (q * s, exact), the MFMA is bf16, and there is no g_x and no
// correction.
template <bool W16>
__global__ void __launch_bounds__(256, 2)
k_gemm_decode(GemmArgs p, int n_blocks, int bpw, int wsrow, int rsrow) {
  using namespace dec;
  extern __shared__ __attribute__((aligned(16))) uint8_t dsm[];
  __shared__ int32_t s_local[KMAX];
  uint8_t* const tok = dsm;
  uint8_t* const wsl = dsm + kDecTokBytes;
  // the pass's residual rows (16 TMAX rows x the selected channels rounded
  // up to 32, zero past k, row stride rsrow bytes), for every block's epilogue
  uint8_t* const rsl = wsl + ROWS * wsrow;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, kq = lane >> 4;
  // workgroup (eo, g) takes row blocks g * bpw .. + bpw of the expert of
  // rank eo by descending row count (ties by index): the costliest experts'
  // workgroups are dispatched first and single-tile experts fill the tail.
  // The token-fragment area holds the row counts meanwhile.
  const int groups = (n_blocks + bpw - 1) / bpw;
  const int eo = (int)blockIdx.x / groups;
  const int g = (int)blockIdx.x - eo * groups;
  __shared__ int32_t e_rank_sel;
  {
    int32_t* cnt = reinterpret_cast<int32_t*>(tok);   // E <= 1024 entries, 4 KB
    for (int f = tid; f < p.E; f += 256) {
      int64_t lo = p.offsets[f], hi = p.offsets[f + 1];
      lo = lo < 0 ? 0 : (lo > p.M_total ? p.M_total : lo);
      hi = hi < lo ? lo : (hi > p.M_total ? p.M_total : hi);
      cnt[f] = (int32_t)(hi - lo);
    }
    __syncthreads();
    for (int f = tid; f < p.E; f += 256) {
      const int32_t me = cnt[f];
      int rank = 0;
      for (int h = 0; h < p.E; ++h) rank += (cnt[h] > me) || (cnt[h] == me && h < f);
      if (rank == eo) e_rank_sel = f;
    }
    __syncthreads();
  }
  const int e = e_rank_sel;
  const int blk_lo = g * bpw;
  const int nbw = n_blocks - blk_lo < bpw ? n_blocks - blk_lo : bpw;
  int64_t e_lo = p.offsets[e], e_hi = p.offsets[e + 1];
  e_lo = e_lo < 0 ? 0 : (e_lo > p.M_total ? p.M_total : e_lo);
  e_hi = e_hi < e_lo ? e_lo : (e_hi > p.M_total ? p.M_total : e_hi);
  const int64_t Me = e_hi - e_lo;
  if (Me == 0 || nbw <= 0) return;           // uniform over the workgroup
  const int64_t Kh = p.K / 2, Ks = p.K / 16;
  const int nc = (int)((p.K + KC - 1) / KC);
  const int kk = W16 ? 0 : p.k;

  if (kk > 0) {
    for (int j = tid; j < kk; j += 256) {
      const int c = p.S[(int64_t)e * p.s_stride + j];
      s_local[j] = c < 0 ? 0 : (c >= p.K ? (int)p.K - 1 : c);
    }
    const int kpad = (kk + 31) & ~31;        // zero channels k .. next multiple of 32
    for (int j = kk; j < kpad; ++j) *reinterpret_cast<uint16_t*>(wsl + tid * wsrow + 2 * j) = 0;
    __syncthreads();
  }

  const uint8_t* wc = p.w_codes + e * packed_codes_per_expert(p.N, p.K);
  const uint8_t* wsc = p.w_scales + e * packed_scales_per_expert(p.N, p.K);
  // the channel-major copies (the residual correction's weight columns)
  const uint8_t* wcm = wc + p.N * p.K / 2;
  const uint8_t* wscm = wsc + p.N * p.K / 16;
  // load addresses = a uniform offset (row block, chunk) + a per-lane
  // offset fixed over the stream: row r16 of the chunk's code tile kq, whose
  // two 16-byte halves lie 256 bytes apart (512-byte tiles of 16 rows x 64
  // columns: a row block's chunk is one contiguous 2 KB run starting at byte
  // rb / 16 * 8 K + 2048 c) and scale
  // byte 4 r16 + 64 kq of its scale tile (row block rb starts at byte
  // rb / 16 * K)
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const uint32_t lane_c0 = (uint32_t)(512 * kq + 16 * r16);
  const uint32_t lane_s0 = (uint32_t)(4 * r16 + 64 * kq);
  const bool half_last = (p.K % KC) != 0;    // the last chunk holds 128 columns
  const float gx = W16 ? 1.0f : *p.g_x;
  const float gw = p.g_w[e];

  // position in the workgroup's chunk stream: local row block, chunk
  struct Pos {
    int blk, c;
  };
  auto advance = [&](Pos q) { return q.c + 1 == nc ? Pos{q.blk + 1, 0} : Pos{q.blk, q.c + 1}; };

  for (int64_t t0 = 0; t0 < Me; t0 += 16 * TMAX) {
    // a pass's first chunk refills fragment buffer 0, which the previous
    // pass's last chunk may still be reading when its chunk count is odd
    if (t0 > 0) __syncthreads();
    const int ntile_rt = (int)((Me - t0 + 15) / 16 < TMAX ? (Me - t0 + 15) / 16 : TMAX);
    int64_t src[TMAX];
#pragma unroll
    for (int t = 0; t < TMAX; ++t) {
      int64_t q = t0 + 16 * t + r16;
      if (q >= Me) q = Me - 1;
      const int64_t pr = e_lo + q;
      int64_t sr = p.a_rows ? (int64_t)p.a_rows[pr] : pr;
      src[t] = sr < 0 ? 0 : (sr >= p.M_src ? p.M_src - 1 : sr);
    }

    // K is a multiple of 128: the lanes of a half chunk past the end (kq >= 2
    // in the last chunk when K % 256 == 128) re-read the chunk's first half
    // (offsets >= 0 since kq >= 2) and their products vanish: their token
    // fragments are zero (zeroing the loaded weight registers instead would
    // make the compiler wait for those loads).  Token codes: each wave loads
    // (and decodes for the whole workgroup) only its MFMA steps 2 wave and
    // 2 wave + 1.
    // the loads of chunk q in six parts (weight row blocks 0..3: codes and
    // scales; token tiles 0..TMAX-1), issued one per MFMA step of the chunk
    // before: issued in one burst right after the barrier, all eight waves of
    // a CU stalled for thousands of cycles at vector-memory issue
    // per-lane offsets as values of this pass (else the prologue's load
    // addresses are hoisted out of the pass loop and held in registers)
    uint32_t lane_c = lane_c0, lane_s = lane_s0;
    asm volatile("" : "+v"(lane_c), "+v"(lane_s));
    uint32_t lane_tc[TMAX], lane_ts[TMAX];
#pragma unroll
    for (int t = 0; t < TMAX; ++t) {
      // W4A16: byte offset of the lane's 16 bf16 tokens (2 * (64 kq + 16 wave))
      lane_tc[t] = W16 ? (uint32_t)(src[t] * p.K * 2) + 32 * wave + 128 * kq
                       : (uint32_t)(src[t] * Kh) + 8 * wave + 32 * kq;
      lane_ts[t] = (uint32_t)(src[t] * Ks) + 4 * kq;
    }
    // the chunk stream for ntile token tiles (a constant, so the unrolled
    // MFMA steps hold no branches)
    auto run = [&](auto ntc) __attribute__((always_inline)) {
      constexpr int ntile = decltype(ntc)::value;
      auto load_part = [&](DecChunk& d, Pos q, int part, int buf) __attribute__((always_inline)) {
        // lanes kq >= 2 of a last half chunk re-read the chunk's first half
        const bool tl = half_last && q.c == nc - 1 && kq >= 2;
        if (part < 4) {
          // a row block past N (N % 16 == 0) reads the last one instead
          int64_t rb = (int64_t)(blk_lo + q.blk) * ROWS + 64 * wave_u + 16 * part;
          if (rb >= p.N) rb = p.N - 16;
          const uint8_t* cb = wc + (uint32_t)((rb >> 4) * p.K * 8) + (uint32_t)q.c * (KC / 64) * 512;
          const uint8_t* sb = wsc + (uint32_t)((rb >> 4) * p.K) + (uint32_t)q.c * (KC / 64) * 64;
          // (nontemporal: each weight byte is read once per call, and the
          // streaming hint measured ~10% more read bandwidth on this chip)
          // (the row's two 16-byte halves of the tile, 256 bytes apart: each
          // load instruction reads whole cache lines)
          const u32x4* src4 = reinterpret_cast<const u32x4*>(cb + (lane_c - (tl ? 1024u : 0u)));
          const u32x4 c0 = __builtin_nontemporal_load(src4), c1 = __builtin_nontemporal_load(src4 + 16);
          d.wc[part][0] = make_uint4(c0.x, c0.y, c0.z, c0.w);
          d.wc[part][1] = make_uint4(c1.x, c1.y, c1.z, c1.w);
          d.ws[part] = __builtin_nontemporal_load(
              reinterpret_cast<const uint32_t*>(sb + (lane_s - (tl ? 128u : 0u))));
        } else if (part - 4 < TMAX) {
          const int t = part - 4;
          if constexpr (W16) {
            // this wave's two steps of token tile t, into the fragment slots
            // of buffer `buf` (lane i's 16 bytes land at slot base + 16 i);
            // lanes past K load nothing and are zeroed before use
            if (!tl) {
              const uint8_t* xs = p.a_codes + (uint32_t)q.c * (KC * 2) + lane_tc[t];
              __builtin_amdgcn_global_load_lds(xs, tok + (((buf * TMAX + t) * 8 + 2 * wave_u) << 10),
                                               16, 0, 0);
              __builtin_amdgcn_global_load_lds(xs + 16,
                                               tok + (((buf * TMAX + t) * 8 + 2 * wave_u + 1) << 10),
                                               16, 0, 0);
            }
          } else {
            d.tc[t] = *reinterpret_cast<const uint2*>(p.a_codes + (uint32_t)q.c * (KC / 2) +
                                                      (lane_tc[t] - (tl ? 64u : 0u)));
            d.ts[t] = *reinterpret_cast<const uint32_t*>(p.a_scales + (uint32_t)q.c * (KC / 16) +
                                                         (lane_ts[t] - (tl ? 8u : 0u)));
          }
        }
      };
      auto load = [&](DecChunk& d, Pos q, int buf) __attribute__((always_inline)) {
  #pragma unroll
        for (int part = 0; part < 4 + TMAX; ++part) load_part(d, q, part, buf);
      };

      f32x4_t acc[4][TMAX];
  #pragma unroll
      for (int b = 0; b < 4; ++b)
  #pragma unroll
        for (int t = 0; t < TMAX; ++t) acc[b][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

      // The block's W_S tile (bf16 q * s of the selected channels' weight
      // columns), gathered from the channel-major copy of the weights in
      // parts of 32 channels: each wave its own 64 rows (it alone writes and
      // later reads them); lane task i of part h covers channel
      // 32 h + (lane + 64 i) / 8 and rows 8 ((lane + 64 i) % 8) .. + 8 of the
      // wave's rows (4 code bytes, 8 scale bytes).  With enough chunks a
      // part's loads go out at the end of chunk c_first + h and are stored
      // at the start of the next chunk.  (32-bit offsets: one expert's
      // codes are below 4 GiB.)
      const int nh = (kk + 31) >> 5;
      const int c_first = nc - 1 - nh < 0 ? 0 : nc - 1 - nh;
      uint32_t gq[4];
      uint2 gs[4];
      auto gather_issue = [&](int blk, int h) __attribute__((always_inline)) {
        const uint32_t nb = (uint32_t)((blk_lo + blk) * ROWS + 64 * wave);
  #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int task = lane + 64 * i, ch = 32 * h + (task >> 3), rg = task & 7;
          uint32_t n = nb + 8 * rg;
          if (n + 8 > (uint32_t)p.N) n = (uint32_t)p.N - 8;   // rows past N: never stored
          const uint32_t col = (uint32_t)s_local[ch < kk ? ch : kk - 1];
          gq[i] = *reinterpret_cast<const uint32_t*>(wcm + (col * (uint32_t)(p.N / 2) + n / 2));
          gs[i] = *reinterpret_cast<const uint2*>(wscm + ((col >> 4) * (uint32_t)p.N + n));
        }
      };
      auto gather_store = [&](int h) __attribute__((always_inline)) {
  #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int task = lane + 64 * i, ch = 32 * h + (task >> 3), rg = task & 7;
          if (ch >= kk) continue;
          uint8_t* dst = wsl + (64 * wave + 8 * rg) * wsrow + 2 * ch;
          const uint32_t sc[2] = {gs[i].x, gs[i].y};
  #pragma unroll
          for (int m = 0; m < 4; ++m) {
            f32x2 q2;
            if (m == 0) q2 = e2m1_unpack2<0>(gq[i]);
            else if (m == 1) q2 = e2m1_unpack2<1>(gq[i]);
            else if (m == 2) q2 = e2m1_unpack2<2>(gq[i]);
            else q2 = e2m1_unpack2<3>(gq[i]);
            const float s0 = e4m3_decode((sc[m >> 1] >> (16 * (m & 1))) & 0xFFu);
            const float s1 = e4m3_decode((sc[m >> 1] >> (16 * (m & 1) + 8)) & 0xFFu);
            *reinterpret_cast<uint16_t*>(dst + (2 * m) * wsrow) =
                (uint16_t)(__float_as_uint(q2.x * s0) >> 16);
            *reinterpret_cast<uint16_t*>(dst + (2 * m + 1) * wsrow) =
                (uint16_t)(__float_as_uint(q2.y * s1) >> 16);
          }
        }
      };

      // token fragment of tile t, step s, this lane, in buffer `buf`
      auto frag = [&](int buf, int t, int s) {
        return tok + ((((buf * TMAX + t) * 8 + s) * 64 + lane) << 4);
      };

      // the block's epilogue: x g_x, residual (32 channels per MFMA), x g_w,
      // store; then the accumulators restart for the next block
      auto finish = [&](int blk) __attribute__((always_inline)) {
        const int64_t n0 = (int64_t)(blk_lo + blk) * ROWS;
  #pragma unroll
        for (int b = 0; b < 4; ++b)
  #pragma unroll
          for (int t = 0; t < TMAX; ++t) acc[b][t] *= gx;
        if (!W16 && kk > 0) {
          // (short K: parts whose loads could not go out a chunk early)
  #pragma unroll
          for (int h = 0; h < 4; ++h)
            if (h < nh && c_first + h > nc - 2) {
              gather_issue(blk, h);
              gather_store(h);
            }
          __syncthreads();                     // W_S complete
          for (int cb = 0; cb < kk; cb += 32) {
            const int slot = cb + 8 * kq;
            u32x4 rf[TMAX];
  #pragma unroll
            for (int t = 0; t < TMAX; ++t) {
              const uint4 v = *reinterpret_cast<const uint4*>(rsl + (16 * t + r16) * rsrow + 2 * slot);
              rf[t] = u32x4{v.x, v.y, v.z, v.w};
            }
  #pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint4 v = *reinterpret_cast<const uint4*>(wsl + (64 * wave + 16 * b + r16) * wsrow + 2 * slot);
              const u32x4 wf = u32x4{v.x, v.y, v.z, v.w};
  #pragma unroll
              for (int t = 0; t < TMAX; ++t)
                if (t < ntile) acc[b][t] = mfma16_bf16(wf, rf[t], acc[b][t]);
            }
          }
        }
  #pragma unroll
        for (int t = 0; t < TMAX; ++t) {
          const int64_t q = t0 + 16 * t + r16;
          if (t >= ntile || q >= Me) continue;
          uint16_t* yr = p.y + (e_lo + q) * p.N;
  #pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int64_t n = n0 + 64 * wave + 16 * b + 4 * kq;
            if (n >= p.N) continue;
            const f32x4_t v = acc[b][t];
            const uint32_t lo = f32_to_bf16_rne(v[0] * gw) | (f32_to_bf16_rne(v[1] * gw) << 16);
            const uint32_t hi = f32_to_bf16_rne(v[2] * gw) | (f32_to_bf16_rne(v[3] * gw) << 16);
            *reinterpret_cast<uint2*>(yr + n) = make_uint2(lo, hi);
          }
        }
  #pragma unroll
        for (int b = 0; b < 4; ++b)
  #pragma unroll
          for (int t = 0; t < TMAX; ++t) acc[b][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      };

      // chunk q's arithmetic (buffer parity buf); with NEXT, the parts of
      // chunk qn are loaded into dn along the way (part s before MFMA step s);
      // after a block's last chunk, its epilogue
      auto compute = [&](const DecChunk& d, Pos q, int buf, DecChunk& dn, Pos qn, auto next) __attribute__((always_inline)) {
        constexpr bool NEXT = decltype(next)::value;
        const int c = q.c;
        // decode this wave's two steps of every token tile for the workgroup;
        // the barrier also ends every wave's reads of this buffer two chunks ago
        if constexpr (W16) wait_vmem0();         // this chunk's token slots have landed
  #pragma unroll
        for (int t = 0; t < TMAX; ++t) {
          if (t >= ntile) continue;
          const bool past_k = (int64_t)c * KC + 64 * kq >= p.K;
          if constexpr (W16) {
            if (past_k) {
              *reinterpret_cast<u32x4*>(frag(buf, t, 2 * wave)) = u32x4{0u, 0u, 0u, 0u};
              *reinterpret_cast<u32x4*>(frag(buf, t, 2 * wave + 1)) = u32x4{0u, 0u, 0u, 0u};
            }
            continue;
          }
          float sc;
          h2_t mu;
          scale_prep((d.ts[t] >> (8 * wave)) & 0xFFu, sc, mu);
          u32x4 f0 = decode8_f16(d.tc[t].x, sc, mu), f1 = decode8_f16(d.tc[t].y, sc, mu);
          if (past_k) f0 = f1 = u32x4{0u, 0u, 0u, 0u};
          *reinterpret_cast<u32x4*>(frag(buf, t, 2 * wave)) = f0;
          *reinterpret_cast<u32x4*>(frag(buf, t, 2 * wave + 1)) = f1;
        }
  #pragma unroll
        for (int h = 0; h < 4; ++h)
          if (!W16 && h < nh && c_first + h <= nc - 2 && c == c_first + h + 1) gather_store(h);
        __syncthreads();
  #pragma unroll
        for (int s = 0; s < 8; ++s) {
          // token tiles first: their fragments are decoded first next chunk
          if (NEXT && s < 4 + TMAX) load_part(dn, qn, (s + 4) % (4 + TMAX), buf ^ 1);
          u32x4 tf[TMAX];
  #pragma unroll
          for (int t = 0; t < TMAX; ++t)
            if (t < ntile) tf[t] = *reinterpret_cast<const u32x4*>(frag(buf, t, s));
  #pragma unroll
          for (int b = 0; b < 4; ++b) {
            if constexpr (W16) {
              const u32x4 wf = decode8_bf16(dword_of(d.wc[b], s),
                                            e4m3_decode((d.ws[b] >> (8 * (s >> 1))) & 0xFFu));
  #pragma unroll
              for (int t = 0; t < TMAX; ++t)
                if (t < ntile) acc[b][t] = mfma16_bf16(wf, tf[t], acc[b][t]);
            } else {
              float sc;
              h2_t mu;
              scale_prep((d.ws[b] >> (8 * (s >> 1))) & 0xFFu, sc, mu);
              const u32x4 wf = decode8_f16(dword_of(d.wc[b], s), sc, mu);
  #pragma unroll
              for (int t = 0; t < TMAX; ++t)
                if (t < ntile) acc[b][t] = mfma16_f16(wf, tf[t], acc[b][t]);
            }
          }
        }
        // the block's W_S parts: loads out one chunk before their stores
  #pragma unroll
        for (int h = 0; h < 4; ++h)
          if (!W16 && h < nh && c_first + h <= nc - 2 && c == c_first + h) gather_issue(q.blk, h);
        if (c + 1 == nc) finish(q.blk);
      };

      // one stream of nbw * nc chunks: steady state loading one chunk ahead
      // (across block boundaries, so a block's epilogue overlaps the next
      // block's first loads), then the last one or two chunks (no load past
      // the end)
      using yes = std::integral_constant<bool, true>;
      using no = std::integral_constant<bool, false>;
      const int total = nbw * nc;
      DecChunk b0, b1;
      Pos qa{0, 0};
      load(b0, qa, 0);
      if (!W16 && kk > 0) {
        // residual rows of this pass into LDS (their loads overlap the first
        // chunk's; the first epilogue's barrier orders them before any read)
        const int kp32 = (kk + 31) & ~31, per_row = kp32 / 8;
        for (int q = tid; q < 16 * TMAX * per_row; q += 256) {
          const int row = q / per_row, c8 = q - row * per_row;
          int64_t tq = t0 + row;
          if (tq >= Me) tq = Me - 1;
          const int64_t pr = e_lo + tq;
          int64_t sr = p.a_rows ? (int64_t)p.a_rows[pr] : pr;
          sr = sr < 0 ? 0 : (sr >= p.M_src ? p.M_src - 1 : sr);
          const int64_t rr = p.r_perm ? pr : sr;
          const uint16_t* src = p.R + rr * kk + 8 * c8;
          uint4 o;
          if ((kk & 7) == 0 && 8 * c8 + 8 <= kk) {
            o = *reinterpret_cast<const uint4*>(src);
          } else {
            uint32_t v[8];
  #pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (8 * c8 + j < kk) ? src[j] : 0u;
            o = make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16),
                           v[6] | (v[7] << 16));
          }
          *reinterpret_cast<uint4*>(rsl + row * rsrow + 16 * c8) = o;
        }
      }
      int i = 0;
      for (; i + 2 < total; i += 2) {
        const Pos qb = advance(qa), qc = advance(qb);
        compute(b0, qa, 0, b1, qb, yes());
        compute(b1, qb, 1, b0, qc, yes());
        qa = qc;
      }
      if (i + 1 < total) {
        const Pos qb = advance(qa);
        compute(b0, qa, 0, b1, qb, yes());
        compute(b1, qb, 1, b0, qa, no());
      } else {
        compute(b0, qa, 0, b1, qa, no());
      }
    };
    if (ntile_rt >= 2)
      run(std::integral_constant<int, 2>());
    else
      run(std::integral_constant<int, 1>());
  }
}


// ---------------------------------------------------------------------------
// FP8 (E4M3) W8A8 grouped GEMM: the low-precision baseline the pages compare
// NVFP4 against (arXiv abstract; gist.science technical summary §1 and §4).
// Both operands are E4M3 bytes with one float32 scale per tensor (per expert
// for the weights): y[p, n] = bf16(g_x g_w[e] sum_k a[t, k] w_e[n, k]).
//
// The same 256x256 tile, eight waves, XCD-aware tile order and tail-row
// skipping as the large-tile NVFP4 kernel; E4M3 needs no decode, so A and B
// go from global memory to LDS as they are (128 bytes of K per row per step)
// and feed the gfx950 32x32x64 FP8 MFMA with unit block scales.
// ---------------------------------------------------------------------------
namespace f8 {
constexpr int BM = 256, BN = 256, BK = 128;     // BK in bytes (= elements)
constexpr int A_BYTES = BM * BK;               // [256][128 B]: chunk c at c ^ ((row >> 1) & 7)
constexpr int STAGE = A_BYTES + BN * BK;       // 65536
constexpr int OUTROW = BN * 2 + 16;            // bf16 output staging row (+pad)
}  // namespace f8

struct Fp8Args {
  const uint8_t* a;            // [M_src][K] E4M3
  const float* g_x;
  const int32_t* a_rows;       // [M_total] or null (identity)
  const uint8_t* w;            // [E][N][K] E4M3
  const float* g_w;            // [E]
  const int32_t* offsets;      // [E + 1]
  const int32_t* tile_prefix;  // [E + 1], 256-row tiles
  uint16_t* y;                 // [M_total][N] bf16
  int64_t M_src, M_total, N, K;
  int E;
};

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// D += A B over 64 k: A, B 32 E4M3 bytes per lane; the block scales are
// E8M0 127 = 2^0, so this is the plain product
__device__ __forceinline__ f32x16_t mfma32_fp8(const i32x8_t& a, const i32x8_t& b, f32x16_t c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
}

__global__ void __launch_bounds__(512, 1)
k_gemm_fp8(Fp8Args p, int n_tiles, int m_tiles) {
  using namespace f8;
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
  __shared__ int32_t rows_src[BM];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform, in an SGPR
  const int wm = wave >> 2, wn = wave & 3;      // rows 128 wm .., columns 64 wn ..
  const int kg = lane >> 5, r32 = lane & 31;

  // tile order as in k_gemm_big: groups of 4 row tiles x all column tiles,
  // each XCD (workgroup b runs on XCD b % 8) a contiguous range of it
  int v;
  {
    const int real_m = p.tile_prefix[p.E];
    const int real_blocks = ((real_m + 3) / 4) * 4 * n_tiles;
    const int per_xcd = (real_blocks + 7) / 8;
    const int b = (int)blockIdx.x;
    const int loc = b >> 3;
    if (loc >= per_xcd) return;
    v = (b & 7) * per_xcd + loc;
    if (v >= real_blocks) return;
  }
  const int group = 4 * n_tiles;
  const int gi = v / group, gr = v - gi * group;
  if (4 * gi >= m_tiles) return;
  const int gm = m_tiles - 4 * gi < 4 ? m_tiles - 4 * gi : 4;
  const int gt = 4 * gi + gr % gm;
  const int nt = gr / gm;
  if (gt >= p.tile_prefix[p.E] || nt >= n_tiles) return;
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    int mid = (lo + hi) >> 1;
    if (p.tile_prefix[mid] <= gt) lo = mid; else hi = mid;
  }
  const int e = lo;
  int64_t e_lo = p.offsets[e], e_hi = p.offsets[e + 1];
  e_lo = e_lo < 0 ? 0 : (e_lo > p.M_total ? p.M_total : e_lo);
  e_hi = e_hi < e_lo ? e_lo : (e_hi > p.M_total ? p.M_total : e_hi);
  const int64_t p0 = e_lo + (int64_t)(gt - p.tile_prefix[e]) * BM;
  const int64_t n0 = (int64_t)nt * BN;
  const uint32_t K = (uint32_t)p.K;

  if (tid < BM) {
    int64_t pr = p0 + tid;
    if (pr >= e_hi) pr = e_hi - 1;
    int64_t t = p.a_rows ? (int64_t)p.a_rows[pr] : pr;
    rows_src[tid] = (int32_t)(t < 0 ? 0 : (t >= p.M_src ? p.M_src - 1 : t));
  }
  __syncthreads();

  const uint8_t* wc = p.w + (int64_t)e * p.N * p.K;
  // thread q = (8 i + wave) 64 + lane stages 16 bytes of row q / 8 (A and
  // B alike): chunk c = (q % 8) ^ ((row >> 1) & 7) of the row's 128 bytes
  uint32_t off_a[4], off_b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = (i * 8 + wave) * 64 + lane;
    const int r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
    off_a[i] = (uint32_t)rows_src[r] * K + 16u * c;
    int64_t n = n0 + r;
    if (n >= p.N) n = p.N - 1;
    off_b[i] = (uint32_t)n * K + 16u * c;
  }
  const int64_t vt = e_hi - p0;
  const int v_tile = vt > BM ? BM : (int)vt;
  // stage loads as buffer loads into LDS, as in k_gemm_big: the lane's
  // offset (fixed over K) in a VGPR, the step in the scalar offset (M_src K
  // and one expert's N K are below 2^32; a load past a buffer reads zeros)
  const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.a), (short)0, (int)(uint32_t)(p.M_src * p.K), kBufferRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs_w = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(wc), (short)0, (int)(uint32_t)(p.N * p.K), kBufferRsrcWord3);
  auto issue_loads = [&](uint8_t* st, uint32_t k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(st + (i * 8 + wave) * 1024), 16, off_a[i],
                                               k0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_w, lds_ptr(st + A_BYTES + (i * 8 + wave) * 1024), 16,
                                               off_b[i], k0, 0, 0);
    }
  };

  f32x16_t acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int sw = (r32 >> 1) & 7;                 // rows 32 i + r32 (+ multiples of 32)
  const int nk = (int)(p.K / BK);
  // lane (r32, kg) of a 64-k MFMA takes k 32 kg .. +31 of its row, both
  // operands alike (chunks 2 kg, 2 kg + 1 of the 64)
  auto ld32 = [&](const uint8_t* base, int row, int c0) -> i32x8_t {
    const uint4 u = *reinterpret_cast<const uint4*>(base + row * 128 + ((c0 ^ sw) << 4));
    const uint4 w = *reinterpret_cast<const uint4*>(base + row * 128 + (((c0 + 1) ^ sw) << 4));
    return i32x8_t{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)w.x, (int)w.y, (int)w.z, (int)w.w};
  };
  auto kstep = [&](const uint8_t* ab, uint8_t* nxt, int kt, auto nv_c) {
    constexpr int NV = decltype(nv_c)::value;
    if (kt + 1 < nk) issue_loads(nxt, (uint32_t)(kt + 1) * BK);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c0 = 4 * u + 2 * kg;
      i32x8_t B[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) B[j] = ld32(ab + A_BYTES, wn * 64 + 32 * j + r32, c0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const i32x8_t A = ld32(ab, wm * 128 + 32 * i + r32, c0);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32_fp8(A, B[j], acc[i][j]);
      }
      // keep the two halves' operand reads apart (32 bytes per operand per
      // lane: hoisting both halves' reads overflows the register file)
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_vmem0();
    __syncthreads();
  };

  issue_loads(st0, 0);
  wait_vmem0();
  __syncthreads();
  // nk may be odd here (K % 128 == 0): the loop runs pairs, then one step
  const int v_wave = v_tile - wm * 128;
  using nv4 = std::integral_constant<int, 4>;
  using nv1 = std::integral_constant<int, 1>;
  using nv0 = std::integral_constant<int, 0>;
  if (v_wave > 32) {
    int kt = 0;
    for (; kt + 1 < nk; kt += 2) {
      kstep(st0, st1, kt, nv4{});
      kstep(st1, st0, kt + 1, nv4{});
    }
    if (kt < nk) kstep(st0, st1, kt, nv4{});
  } else if (v_wave > 0) {
    int kt = 0;
    for (; kt + 1 < nk; kt += 2) {
      kstep(st0, st1, kt, nv1{});
      kstep(st1, st0, kt + 1, nv1{});
    }
    if (kt < nk) kstep(st0, st1, kt, nv1{});
  } else {
    int kt = 0;
    for (; kt + 1 < nk; kt += 2) {
      kstep(st0, st1, kt, nv0{});
      kstep(st1, st0, kt + 1, nv0{});
    }
    if (kt < nk) kstep(st0, st1, kt, nv0{});
  }

  // y = bf16(acc g_x g_w), staged through LDS (a 128-row half at a time:
  // rows 0..63 in st0, 64..127 in st1) for 16-byte row stores
  const float sc = *p.g_x * p.g_w[e];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncthreads();
    if (wm == h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint8_t* half = i < 2 ? st0 : st1;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int row = 32 * (i & 1) + 8 * (r >> 2) + 4 * kg + (r & 3);
            const int col = wn * 64 + 32 * j + r32;
            *reinterpret_cast<uint16_t*>(half + row * OUTROW + 2 * col) =
                (uint16_t)f32_to_bf16_rne(acc[i][j][r] * sc);
          }
      }
    }
    __syncthreads();
    for (int q = tid; q < 128 * (BN / 8); q += 512) {
      const int row = q / (BN / 8), ch = q % (BN / 8);
      const int64_t prow = p0 + h * 128 + row;
      const int64_t n = n0 + ch * 8;
      const uint8_t* src = (row < 64 ? st0 + row * OUTROW : st1 + (row - 64) * OUTROW) + ch * 16;
      if (prow < e_hi && n < p.N)
        *reinterpret_cast<uint4*>(p.y + prow * p.N + n) = *reinterpret_cast<const uint4*>(src);
    }
  }
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

// prefix [E+1] int32, then (large-tile path) the f16 image of A [M_src][K]
static size_t img_offset(int64_t E) { return round_up((size_t)(E + 1) * sizeof(int32_t), 256); }

// large k (more than the large-tile kernel's W_S tile): the kernel takes a
// multiple of it
static bool big_streams_ws(int64_t k) { return k > big::KMAX && k % big::KMAX == 0; }
// K slices of the large-tile kernel for a problem whose tiles fill less than
// the chip (sized for 256 CUs from the fewest tiles M_total can make; each
// slice an even number of 64-k steps, at most 4 slices), or 1.
// NVFP4RAC_SPLIT overrides it (tests).  Not with the fused SwiGLU or the
// streamed correction.
static int big_ksplit(int64_t M_total, int64_t N, int64_t K, int64_t k) {
  if (big_streams_ws(k) || M_total <= 0) return 1;
  const int64_t nk = K / big::BK;
  const int64_t tiles = ((M_total + big::BM - 1) / big::BM) * ((N + big::BN - 1) / big::BN);
  int s = 1;
  if (const char* o = getenv("NVFP4RAC_SPLIT")) {
    const int want = atoi(o);
    while (s * 2 <= want && nk % (4 * s) == 0) s *= 2;
    return s;
  }
  while (s < 4 && tiles * 2 * s <= 256 && nk % (4 * s) == 0) s *= 2;
  return s;
}
static size_t split_bytes(int64_t M_total, int64_t N, int64_t K, int64_t k) {
  const int s = big_ksplit(M_total, N, K, k);
  return s > 1 ? round_up((size_t)s * (size_t)M_total * (size_t)N * 4, 256) : 0;
}

size_t grouped_w4a4_gemm_rac_workspace_size(int64_t E, int64_t M_src, int64_t M_total, int64_t N,
                                            int64_t K, int64_t k) {
  if (E < 1 || M_src < 0 || M_total < 0 || K < 0 || N < 0) return 256;
  size_t n = img_offset(E) + round_up((size_t)M_src * (size_t)K * 2, 256);
  n += split_bytes(M_total, N, K, k);
  return n;
}

// per_expert: S is [E][k] and R_S is [M_total][k] by permuted row
// glu: y receives h = bf16(silu(gate) * up) [M_total][N/2] of the [gate | up]
// product, fused into the large-tile kernel's epilogue, else formed from a
// product staged in the workspace
static int gemm_rac(bool per_expert, bool glu, uint32_t* h_amax, const uint8_t* a_codes,
                    const uint8_t* a_scales,
                    const float* g_x, const int32_t* a_rows, int64_t M_src, const void* R_S,
                    const int32_t* S, int64_t k, const uint8_t* w_codes, const uint8_t* w_scales,
                    const float* g_w, const int32_t* expert_offsets, int64_t E, int64_t M_total,
                    int64_t N, int64_t K, void* y, void* ws, size_t ws_bytes, void* stream) {
  NV_REQUIRE(E >= 1 && E <= 1024 && M_total >= 0 && N >= 16 && N % 16 == 0 && K >= kBK &&
                 K % kBK == 0 && k >= 0 && k <= K && M_src >= 0,
             NVFP4_ERR_SHAPE,
             "grouped_w4a4_gemm_rac: need 1 <= E <= 1024, N %% 16 == 0, K %% 128 == 0, "
             "0 <= k <= K (E=%lld N=%lld K=%lld k=%lld)",
             (long long)E, (long long)N, (long long)K, (long long)k);
  NV_REQUIRE(a_rows != nullptr || M_src >= M_total, NVFP4_ERR_SHAPE,
             "grouped_w4a4_gemm_rac: without a_rows, M_src must be >= M_total");
  NV_REQUIRE(M_total == 0 || M_src >= 1, NVFP4_ERR_SHAPE, "grouped_w4a4_gemm_rac: M_src == 0");
  NV_REQUIRE(g_x && w_codes && w_scales && g_w && expert_offsets && ws &&
                 (M_total == 0 || (a_codes && a_scales && y)) && (k == 0 || (R_S && S)),
             NVFP4_ERR_NULL, "grouped_w4a4_gemm_rac: missing pointer");
  NV_REQUIRE(aligned(a_codes, 16) && aligned(w_codes, 16) && aligned(a_scales, 8) &&
                 aligned(w_scales, 8) && aligned(ws, 16) && aligned(y, 16) && aligned(R_S, 16),
             NVFP4_ERR_ALIGN, "grouped_w4a4_gemm_rac: misaligned pointer");
  NV_REQUIRE(ws_bytes >= grouped_w4a4_gemm_rac_workspace_size(E, M_src, M_total, N, K, k),
             NVFP4_ERR_WORKSPACE, "grouped_w4a4_gemm_rac: workspace too small");
  if (M_total == 0) return ok();
  hipStream_t s = as_stream(stream);
  int32_t* prefix = static_cast<int32_t*>(ws);
  GemmArgs a{};
  a.a_codes = a_codes;
  a.a_scales = a_scales;
  a.g_x = g_x;
  a.a_rows = a_rows;
  a.R = static_cast<const uint16_t*>(R_S);
  a.S = S;
  a.w_codes = w_codes;
  a.w_scales = w_scales;
  a.g_w = g_w;
  a.offsets = expert_offsets;
  a.tile_prefix = prefix;
  a.y = static_cast<uint16_t*>(y);
  a.M_src = M_src;
  a.M_total = M_total;
  a.N = N;
  a.K = K;
  a.E = (int)E;
  a.k = (int)k;
  a.s_stride = per_expert ? k : 0;
  a.r_perm = per_expert ? 1 : 0;
  // the [gate | up] product for the fused SwiGLU outside the large-tile
  // kernel: after the plain GEMM's workspace
  uint16_t* glu_stage = glu ? reinterpret_cast<uint16_t*>(
      static_cast<char*>(ws) + grouped_w4a4_gemm_rac_workspace_size(E, M_src, M_total, N, K, k))
                            : nullptr;
  auto launch_swiglu = [&]() {
    const int64_t n8 = M_total * (N / 16);
    int64_t nb = (n8 + 255) / 256;
    if (nb > 16LL * num_cus()) nb = 16LL * num_cus();
    k_swiglu_rows<<<(unsigned)(nb > 0 ? nb : 1), 256, 0, s>>>(glu_stage, M_total, N / 2,
                                                             static_cast<uint16_t*>(y), h_amax);
  };
  const int64_t m_tiles = (M_total + kBM - 1) / kBM + E;
  const int64_t n_tiles = (N + kBN - 1) / kBN;
  const int64_t n_tiles_big = glu ? (N / 2 + 127) / 128 : (N + big::BN - 1) / big::BN;
  const int64_t m_tiles_big = (M_total + big::BM - 1) / big::BM + E;
  // NVFP4RAC_GEMM=generic|big forces a kernel (tests use it to cover both on
  // small shapes).  The large-tile path holds at most KMAX residual channels,
  // needs the f16 image of A in the workspace, and 32-bit offsets into the
  // image, one expert's weights and the residual rows.
  const char* force = getenv("NVFP4RAC_GEMM");
  // few rows per expert (decode): stream each expert's weights once; else
  // the large-tile kernel wherever it takes the shape (it is also the faster
  // one on small problems that fill only part of the chip: 64x512x512 and
  // 2048x1024x2048 measured 20-25% faster than the generic kernel)
  bool use_dec = M_total <= 48 * E;
  bool use_big = true;
  if (force && strcmp(force, "big") == 0) use_big = true, use_dec = false;
  if (force && strcmp(force, "generic") == 0) use_big = false, use_dec = false;
  if (force && strcmp(force, "decode") == 0) use_dec = true;
  use_dec = use_dec && k <= dec::KMAX && K / dec::KC <= dec::CHUNKS_MAX &&
            (uint64_t)N * (uint64_t)K / 2 < (1ULL << 32) &&
            (uint64_t)M_src * (uint64_t)K / 2 < (1ULL << 32);
  if (use_dec) {
    const int64_t n_blocks = (N + dec::ROWS - 1) / dec::ROWS;
    const int wsrow = k > 0 ? (int)(((k + 31) & ~31) * 2 + 16) : 0;
    const int rsrow = wsrow;                    // (the residual rows: the same channel span)
    const size_t lds = (size_t)kDecTokBytes + (size_t)dec::ROWS * wsrow +
                       (size_t)(16 * dec::TMAX) * rsrow;
    // dynamic LDS above 64 KB needs the kernel's limit raised (once per
    // device; the cache is shared by all calling threads)
    static std::mutex dec_mu;
    static int dec_lds_limit[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64)
      return fail(NVFP4_ERR_HIP, "grouped_w4a4_gemm_rac: hipGetDevice failed");
    {
      std::lock_guard<std::mutex> lock(dec_mu);
      if ((size_t)dec_lds_limit[dev] < lds) {
        const int want = (int)kDecTokBytes + (dec::ROWS + 16 * dec::TMAX) * (dec::KMAX * 2 + 16);
        if (hipFuncSetAttribute(reinterpret_cast<const void*>(&k_gemm_decode<false>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, want) != hipSuccess)
          return fail(NVFP4_ERR_HIP, "grouped_w4a4_gemm_rac: cannot raise the LDS limit");
        dec_lds_limit[dev] = want;
      }
    }
    // one round of workgroups: each takes bpw consecutive row blocks of its
    // expert (two workgroups per CU when the LDS allows it)
    const int64_t slots = (int64_t)num_cus() * (2 * (lds + kDecStaticLds) <= kLdsPerCu ? 2 : 1);
    int64_t bpw = (E * n_blocks + slots - 1) / slots;
    if (const char* o = getenv("NVFP4RAC_DEC_BPW")) bpw = atoll(o);
    bpw = bpw < 1 ? 1 : (bpw > n_blocks ? n_blocks : bpw);
    const int64_t groups = (n_blocks + bpw - 1) / bpw;
    if (glu) a.y = glu_stage;
    k_gemm_decode<false><<<(unsigned)(E * groups), 256, lds, s>>>(a, (int)n_blocks, (int)bpw, wsrow,
                                                                 rsrow);
    if (glu) launch_swiglu();
    return check_launch("grouped_w4a4_gemm_rac");
  }
  const size_t need_big = grouped_w4a4_gemm_rac_workspace_size(E, M_src, M_total, N, K, k);
  use_big = use_big && (k <= big::KMAX || big_streams_ws(k)) && K / big::BK <= big::KSTEPS_MAX &&
            ws_bytes >= need_big && (uint64_t)M_src * K * 2 < (1ULL << 32) &&
            (uint64_t)N * (uint64_t)K / 2 < (1ULL << 32) &&
            (uint64_t)(per_expert ? M_total : M_src) * k * 2 < (1ULL << 32);
  if (use_big) {
    uint16_t* img = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + img_offset(E));
    const int64_t chunks = M_src * (K / 8);
    int64_t nb = (chunks + 255) / 256;
    if (nb > 16LL * num_cus()) nb = 16LL * num_cus();
    k_decode_a<<<(unsigned)nb, 256, 0, s>>>(a_codes, a_scales, M_src, K, img);
    k_tile_prefix<<<1, 1024, 0, s>>>(expert_offsets, (int)E, M_total, big::BM, prefix);
    const int64_t nblk = (((m_tiles_big + 3) / 4) * 4 * n_tiles_big + 7) / 8 * 8;
    if (glu) a.glu_i = N / 2, a.h_amax = h_amax;
    // a problem that fills less than the chip: K slices, reduced in order
    const int ksplit = glu ? 1 : big_ksplit(M_total, N, K, k);
    const size_t part_off = img_offset(E) + round_up((size_t)M_src * (size_t)K * 2, 256);
    if (ksplit > 1 && ws_bytes >= part_off + split_bytes(M_total, N, K, k)) {
      a.ksplit = ksplit;
      a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + part_off);
      k_gemm_big<false, true><<<dim3((unsigned)nblk, (unsigned)ksplit), 512, 0, s>>>(
          a, reinterpret_cast<const uint8_t*>(img), (int)n_tiles_big, (int)m_tiles_big);
      const int64_t n8 = M_total * (N / 8);
      int64_t nb = (n8 + 255) / 256;
      if (nb > 8LL * num_cus()) nb = 8LL * num_cus();
      k_split_reduce<<<(unsigned)nb, 256, 0, s>>>(a.part, ksplit, M_total, N, expert_offsets,
                                                 (int)E, g_w, static_cast<uint16_t*>(y));
    } else {
      k_gemm_big<false><<<(unsigned)nblk, 512, 0, s>>>(a, reinterpret_cast<const uint8_t*>(img),
                                                      (int)n_tiles_big, (int)m_tiles_big);
    }
  } else {
    if (glu) a.y = glu_stage;
    k_tile_prefix<<<1, 1024, 0, s>>>(expert_offsets, (int)E, M_total, kBM, prefix);
    k_gemm_generic<<<dim3((unsigned)m_tiles, (unsigned)n_tiles), 256, 0, s>>>(a);
    if (glu) launch_swiglu();
  }
  return check_launch("grouped_w4a4_gemm_rac");
}

int grouped_w4a4_gemm_rac(const uint8_t* a_codes, const uint8_t* a_scales, const float* g_x,
                          const int32_t* a_rows, int64_t M_src, const void* R_S, const int32_t* S,
                          int64_t k, const uint8_t* w_codes, const uint8_t* w_scales,
                          const float* g_w, const int32_t* expert_offsets, int64_t E,
                          int64_t M_total, int64_t N, int64_t K, void* y, void* ws,
                          size_t ws_bytes, void* stream) {
  return gemm_rac(false, false, nullptr, a_codes, a_scales, g_x, a_rows, M_src, R_S, S, k, w_codes,
                  w_scales, g_w, expert_offsets, E, M_total, N, K, y, ws, ws_bytes, stream);
}

int grouped_w4a4_gemm_rac_per_expert(const uint8_t* a_codes, const uint8_t* a_scales,
                                     const float* g_x, const int32_t* a_rows, int64_t M_src,
                                     const void* R_P, const int32_t* S_E, int64_t k,
                                     const uint8_t* w_codes, const uint8_t* w_scales,
                                     const float* g_w, const int32_t* expert_offsets, int64_t E,
                                     int64_t M_total, int64_t N, int64_t K, void* y, void* ws,
                                     size_t ws_bytes, void* stream) {
  return gemm_rac(true, false, nullptr, a_codes, a_scales, g_x, a_rows, M_src, R_P, S_E, k,
                  w_codes, w_scales, g_w, expert_offsets, E, M_total, N, K, y, ws, ws_bytes,
                  stream);
}

size_t grouped_w4a4_gemm_rac_swiglu_workspace_size(int64_t E, int64_t M_src, int64_t M_total,
                                                   int64_t N, int64_t K, int64_t k) {
  return grouped_w4a4_gemm_rac_workspace_size(E, M_src, M_total, N, K, k) +
         round_up((size_t)(M_total > 0 ? M_total : 0) * (size_t)(N > 0 ? N : 0) * 2, 256);
}

int grouped_w4a4_gemm_rac_swiglu(const uint8_t* a_codes, const uint8_t* a_scales, const float* g_x,
                                 const int32_t* a_rows, int64_t M_src, const void* R_S,
                                 const int32_t* S, int64_t k, const uint8_t* w_codes,
                                 const uint8_t* w_scales, const float* g_w,
                                 const int32_t* expert_offsets, int64_t E, int64_t M_total,
                                 int64_t N, int64_t K, void* h, uint32_t* h_amax, void* ws,
                                 size_t ws_bytes, void* stream) {
  NV_REQUIRE(N % 32 == 0, NVFP4_ERR_SHAPE,
             "grouped_w4a4_gemm_rac_swiglu: N = 2 I needs N %% 32 == 0 (N=%lld)", (long long)N);
  NV_REQUIRE(aligned(h, 16), NVFP4_ERR_ALIGN, "grouped_w4a4_gemm_rac_swiglu: misaligned h");
  NV_REQUIRE(ws_bytes >= grouped_w4a4_gemm_rac_swiglu_workspace_size(E, M_src, M_total, N, K, k),
             NVFP4_ERR_WORKSPACE, "grouped_w4a4_gemm_rac_swiglu: workspace too small");
  NV_REQUIRE(aligned(h_amax, 4), NVFP4_ERR_ALIGN, "grouped_w4a4_gemm_rac_swiglu: misaligned h_amax");
  if (h_amax != nullptr) fill_u32(h_amax, 1, 0u, as_stream(stream));
  return gemm_rac(false, true, h_amax, a_codes, a_scales, g_x, a_rows, M_src, R_S, S, k, w_codes,
                  w_scales, g_w, expert_offsets, E, M_total, N, K, h, ws, ws_bytes, stream);
}

size_t grouped_w4a16_gemm_workspace_size(int64_t E) {
  return img_offset(E < 1 ? 1 : E);
}

int grouped_w4a16_gemm(const void* x, const int32_t* a_rows, int64_t M_src,
                       const uint8_t* w_codes, const uint8_t* w_scales, const float* g_w,
                       const int32_t* expert_offsets, int64_t E, int64_t M_total, int64_t N,
                       int64_t K, void* y, void* ws, size_t ws_bytes, void* stream) {
  NV_REQUIRE(E >= 1 && E <= 1024 && M_total >= 0 && N >= 16 && N % 16 == 0 && K >= 128 &&
                 K % 128 == 0 && K / big::BK <= big::KSTEPS_MAX && M_src >= 0,
             NVFP4_ERR_SHAPE,
             "grouped_w4a16_gemm: need 1 <= E <= 1024, N %% 16 == 0, K %% 128 == 0, K <= 16384 "
             "(E=%lld N=%lld K=%lld)",
             (long long)E, (long long)N, (long long)K);
  NV_REQUIRE(a_rows != nullptr || M_src >= M_total, NVFP4_ERR_SHAPE,
             "grouped_w4a16_gemm: without a_rows, M_src must be >= M_total");
  NV_REQUIRE(M_total == 0 || M_src >= 1, NVFP4_ERR_SHAPE, "grouped_w4a16_gemm: M_src == 0");
  NV_REQUIRE((uint64_t)M_src * (uint64_t)K * 2 < (1ULL << 32) &&
                 (uint64_t)N * (uint64_t)K / 2 < (1ULL << 32),
             NVFP4_ERR_UNSUPPORTED, "grouped_w4a16_gemm: x or one expert's codes exceed 4 GiB");
  NV_REQUIRE(w_codes && w_scales && g_w && expert_offsets && ws && (M_total == 0 || (x && y)),
             NVFP4_ERR_NULL, "grouped_w4a16_gemm: missing pointer");
  NV_REQUIRE(aligned(x, 16) && aligned(w_codes, 16) && aligned(w_scales, 8) && aligned(ws, 16) &&
                 aligned(y, 16),
             NVFP4_ERR_ALIGN, "grouped_w4a16_gemm: misaligned pointer");
  NV_REQUIRE(ws_bytes >= grouped_w4a16_gemm_workspace_size(E), NVFP4_ERR_WORKSPACE,
             "grouped_w4a16_gemm: workspace too small");
  if (M_total == 0) return ok();
  hipStream_t s = as_stream(stream);
  int32_t* prefix = static_cast<int32_t*>(ws);
  GemmArgs a{};
  a.a_rows = a_rows;
  a.w_codes = w_codes;
  a.w_scales = w_scales;
  a.g_w = g_w;
  a.offsets = expert_offsets;
  a.tile_prefix = prefix;
  a.y = static_cast<uint16_t*>(y);
  a.M_src = M_src;
  a.M_total = M_total;
  a.N = N;
  a.K = K;
  a.E = (int)E;
  a.k = 0;
  // few rows per expert (decode): stream each expert's weights once with
  // bf16 tokens (NVFP4RAC_GEMM=decode|big forces a kernel)
  const char* force = getenv("NVFP4RAC_GEMM");
  bool use_dec = M_total <= 48 * E;
  if (force && strcmp(force, "decode") == 0) use_dec = true;
  if (force && (strcmp(force, "big") == 0 || strcmp(force, "generic") == 0)) use_dec = false;
  use_dec = use_dec && K / dec::KC <= dec::CHUNKS_MAX;
  if (use_dec) {
    a.a_codes = static_cast<const uint8_t*>(x);
    const int64_t n_blocks = (N + dec::ROWS - 1) / dec::ROWS;
    const size_t lds = (size_t)kDecTokBytes;
    const int64_t slots = (int64_t)num_cus() * (2 * (lds + kDecStaticLds) <= kLdsPerCu ? 2 : 1);
    int64_t bpw = (E * n_blocks + slots - 1) / slots;
    bpw = bpw < 1 ? 1 : (bpw > n_blocks ? n_blocks : bpw);
    const int64_t groups = (n_blocks + bpw - 1) / bpw;
    k_gemm_decode<true><<<(unsigned)(E * groups), 256, lds, s>>>(a, (int)n_blocks, (int)bpw, 0, 0);
    return check_launch("grouped_w4a16_gemm");
  }
  const int64_t n_tiles = (N + big::BN - 1) / big::BN;
  const int64_t m_tiles = (M_total + big::BM - 1) / big::BM + E;
  k_tile_prefix<<<1, 1024, 0, s>>>(expert_offsets, (int)E, M_total, big::BM, prefix);
  const int64_t nblk = (((m_tiles + 3) / 4) * 4 * n_tiles + 7) / 8 * 8;
  k_gemm_big<true><<<(unsigned)nblk, 512, 0, s>>>(a, static_cast<const uint8_t*>(x), (int)n_tiles,
                                                  (int)m_tiles);
  return check_launch("grouped_w4a16_gemm");
}

size_t grouped_fp8_gemm_workspace_size(int64_t E) {
  return img_offset(E < 1 ? 1 : E);
}

int grouped_fp8_gemm(const uint8_t* a, const float* g_x, const int32_t* a_rows, int64_t M_src,
                     const uint8_t* w, const float* g_w, const int32_t* expert_offsets, int64_t E,
                     int64_t M_total, int64_t N, int64_t K, void* y, void* ws, size_t ws_bytes,
                     void* stream) {
  NV_REQUIRE(E >= 1 && E <= 1024 && M_total >= 0 && N >= 16 && N % 16 == 0 && K >= f8::BK &&
                 K % f8::BK == 0 && M_src >= 0,
             NVFP4_ERR_SHAPE,
             "grouped_fp8_gemm: need 1 <= E <= 1024, N %% 16 == 0, K %% 128 == 0 "
             "(E=%lld N=%lld K=%lld)",
             (long long)E, (long long)N, (long long)K);
  NV_REQUIRE(a_rows != nullptr || M_src >= M_total, NVFP4_ERR_SHAPE,
             "grouped_fp8_gemm: without a_rows, M_src must be >= M_total");
  NV_REQUIRE(M_total == 0 || M_src >= 1, NVFP4_ERR_SHAPE, "grouped_fp8_gemm: M_src == 0");
  NV_REQUIRE((uint64_t)M_src * (uint64_t)K < (1ULL << 32) &&
                 (uint64_t)N * (uint64_t)K < (1ULL << 32),
             NVFP4_ERR_UNSUPPORTED, "grouped_fp8_gemm: a or one expert's weights exceed 4 GiB");
  NV_REQUIRE(g_x && w && g_w && expert_offsets && ws && (M_total == 0 || (a && y)),
             NVFP4_ERR_NULL, "grouped_fp8_gemm: missing pointer");
  NV_REQUIRE(aligned(a, 16) && aligned(w, 16) && aligned(ws, 16) && aligned(y, 16),
             NVFP4_ERR_ALIGN, "grouped_fp8_gemm: misaligned pointer");
  NV_REQUIRE(ws_bytes >= grouped_fp8_gemm_workspace_size(E), NVFP4_ERR_WORKSPACE,
             "grouped_fp8_gemm: workspace too small");
  if (M_total == 0) return ok();
  hipStream_t s = as_stream(stream);
  int32_t* prefix = static_cast<int32_t*>(ws);
  Fp8Args p{};
  p.a = a;
  p.g_x = g_x;
  p.a_rows = a_rows;
  p.w = w;
  p.g_w = g_w;
  p.offsets = expert_offsets;
  p.tile_prefix = prefix;
  p.y = static_cast<uint16_t*>(y);
  p.M_src = M_src;
  p.M_total = M_total;
  p.N = N;
  p.K = K;
  p.E = (int)E;
  const int64_t n_tiles = (N + f8::BN - 1) / f8::BN;
  const int64_t m_tiles = (M_total + f8::BM - 1) / f8::BM + E;
  k_tile_prefix<<<1, 1024, 0, s>>>(expert_offsets, (int)E, M_total, f8::BM, prefix);
  const int64_t nblk = (((m_tiles + 3) / 4) * 4 * n_tiles + 7) / 8 * 8;
  k_gemm_fp8<<<(unsigned)nblk, 512, 0, s>>>(p, (int)n_tiles, (int)m_tiles);
  return check_launch("grouped_fp8_gemm");
}

}  // extern "C"
