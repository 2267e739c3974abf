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

// ------------------------------------------------------------------------
// Large tiles: 128 activation rows x 256 weight rows per workgroup of four
// waves, two workgroups on a CU, so one's epilogue and waits run under the
// other's products.  Wave w owns 64 weight rows (GLU: 32 gate rows and the
// same 32 up rows) and all of the tile's activation rows: 2 x 4 accumulators
// of 32x32.  K advances in steps of 128 through a ring of three LDS stages,
// filled two steps ahead by buffer loads straight into LDS.
//
// A stage's row is its 64 code bytes, four 16-byte pieces; piece c lies at
// place c ^ ((row >> 2) & 3), so that the 32 rows of a fragment read without
// bank conflicts.  Lane (r, q) of instruction s = 0, 1 takes piece 2 q + s of
// its row, both operands alike: which 32 of the 128 columns a lane of an
// instruction has does not matter for the sum, and so the scales of both
// instructions are two neighbouring bytes of the row's dword.
//
// Scales come straight to registers, three steps' (12 bytes of a row) at a
// time.
// ------------------------------------------------------------------------
namespace mxb {
constexpr int BM = 128, BN = 256, BK = 128;
constexpr int A_BYTES = BM * 64, STAGE = (BM + BN) * 64;
}  // namespace mxb

// The row tiles of all experts, in order: tiles[t] = {expert, first row, rows,
// 0}, and their number.  Every workgroup sums the experts' tiles for itself and
// writes a part of the list.
__global__ void __launch_bounds__(1024)
k_mx_tiles(MxGemmArgs p, int4* __restrict__ tiles, int32_t* __restrict__ n_tiles) {
  __shared__ int wsum[16];
  __shared__ int prefix[1025];
  const int tid = threadIdx.x;
  int v = 0;
  if (tid < p.E) {
    int64_t lo, hi;
    expert_rows(p, tid, lo, hi);
    v = (int)((hi - lo + mxb::BM - 1) / mxb::BM);
  }
  int incl = v;
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if ((tid & 63) >= o) incl += u;
  }
  if ((tid & 63) == 63) wsum[tid >> 6] = incl;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < (tid >> 6); ++w) base += wsum[w];
  prefix[tid] = base + incl - v;
  if (tid == 1023) prefix[1024] = base + incl;
  __syncthreads();
  const int total = prefix[1024];
  for (int t = blockIdx.x * 1024 + tid; t < total; t += gridDim.x * 1024) {
    int lo_e = 0, hi_e = p.E;                            // largest e with prefix[e] <= t
    while (hi_e - lo_e > 1) {
      const int mid = (lo_e + hi_e) >> 1;
      if (prefix[mid] <= t) lo_e = mid; else hi_e = mid;
    }
    int64_t lo, hi;
    expert_rows(p, lo_e, lo, hi);
    const int64_t p0 = lo + (int64_t)(t - prefix[lo_e]) * mxb::BM;
    tiles[t] = make_int4(lo_e, (int)p0, (int)(hi - p0 < mxb::BM ? hi - p0 : mxb::BM), 0);
  }
  if (blockIdx.x == 0 && tid == 0) *n_tiles = total;
}

// D += 2^(sa - 127 + sb - 127) A B over 64 k: lane (r = l % 32, q = l / 32)
// has 32 codes of row r in 16 bytes, byte SEL of sa / sb their scale
template <int SEL>
__device__ __forceinline__ f32x16_t mfma32_mx4(const u32x4& a, uint32_t sa, const u32x4& b,
                                               uint32_t sb, f32x16_t c) {
  const mx_i32x8 a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const mx_i32x8 b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

template <bool GLU>
__global__ void __launch_bounds__(256, 2)
k_mx_big(MxGemmArgs p, const int4* __restrict__ tiles, const int32_t* __restrict__ n_row_tiles,
         int n_tiles) {
  using namespace mxb;
  // separate objects, and the ring unrolled: each access names its stage, so
  // the compiler does not wait for loads into the others
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE], st1[STAGE], st2[STAGE];
  __shared__ int32_t rows_src[BM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 5, r32 = lane & 31;

  // groups of 8 row tiles x all column tiles; each XCD (workgroup b runs on
  // XCD b % 8) takes a contiguous range, so its L2 holds an expert's weights
  constexpr int G = 8;
  const int real_m = *n_row_tiles;
  const int total = real_m * n_tiles;
  const int per_xcd = (total + 7) / 8;
  const int loc = (int)blockIdx.x >> 3;
  if (loc >= per_xcd) return;
  const int v = ((int)blockIdx.x & 7) * per_xcd + loc;
  if (v >= total) return;
  const int gi = v / (G * n_tiles), gr = v - gi * G * n_tiles;
  const int gm = real_m - G * gi < G ? real_m - G * gi : G;
  const int nt = gr / gm;
  const int4 tile = tiles[G * gi + gr - nt * gm];
  const int e = tile.x, valid = tile.z;
  const int64_t p0 = tile.y;
  if (tid < BM) rows_src[tid] = (int32_t)source_row(p, p0 + (tid < valid ? tid : valid - 1));
  __syncthreads();

  const uint32_t KC = (uint32_t)(p.K / 2), KS = (uint32_t)(p.K / 32);
  const int nk = (int)(p.K / BK);
  const int64_t NO = GLU ? p.N / 2 : p.N;               // output columns
  constexpr int CW = GLU ? 32 : 64;                     // ... of a wave
  const int64_t n0 = (int64_t)nt * 4 * CW;
  // weight row of the tile's row r (wave r / 64, of which GLU: 32 gate, 32 up)
  auto w_row = [&](int r) -> uint32_t {
    int64_t n = n0 + (GLU ? (r >> 6) * 32 + (r & 31) : r);
    n = n < NO ? n : NO - 1;
    return (uint32_t)(GLU && (r & 32) ? n + NO : n);
  };
  const uint8_t* wc = p.w_codes + (int64_t)e * p.N * KC;
  const uint8_t* wsc = p.w_scales + (int64_t)e * p.N * KS;
  const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.a_codes), (short)0, (int)(uint32_t)(p.M_src * KC), kBufferRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs_w = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(wc), (short)0, (int)(uint32_t)(p.N * KC), kBufferRsrcWord3);

  // one load instruction fills 16 rows of 64 bytes: lane l's 16 bytes land at
  // row l / 4, place l % 4
  const int lr = lane >> 2, piece = (lane & 3) ^ ((lr >> 2) & 3);
  uint32_t off_a[2], off_w[4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    off_a[i] = (uint32_t)rows_src[(2 * wave + i) * 16 + lr] * KC + 16u * piece;
#pragma unroll
  for (int i = 0; i < 4; ++i) off_w[i] = w_row((4 * wave + i) * 16 + lr) * KC + 16u * piece;
  auto issue_loads = [&](uint8_t* st, int kt) {
    const uint32_t k0 = (uint32_t)kt * 64u;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(st + (2 * wave + i) * 1024), 16, off_a[i],
                                               k0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_w, lds_ptr(st + A_BYTES + (4 * wave + i) * 1024), 16,
                                               off_w[i], k0, 0, 0);
  };
  // scales: weight rows 64 wave + 32 i + r32, activation rows 32 j + r32
  uint32_t soff_w[2], soff_a[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) soff_w[i] = w_row(64 * wave + 32 * i + r32) * KS;
#pragma unroll
  for (int j = 0; j < 4; ++j) soff_a[j] = (uint32_t)rows_src[32 * j + r32] * KS;
  typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
  typedef u32x3 u32x3a __attribute__((aligned(4)));
  u32x3 sw[2], sa[4];
  auto load_scales = [&](int kt, auto full_c) {          // of steps kt .. kt + 2
    auto get = [&](const uint8_t* base, uint32_t off) -> u32x3 {
      const uint8_t* src = base + off + 4u * (uint32_t)kt;
      if (decltype(full_c)::value || kt + 3 <= nk) return *reinterpret_cast<const u32x3a*>(src);
      u32x3 s = {0, 0, 0};
      s.x = *reinterpret_cast<const uint32_t*>(src);
      if (kt + 1 < nk) s.y = *reinterpret_cast<const uint32_t*>(src + 4);
      return s;
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) sw[i] = get(wsc, soff_w[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) sa[j] = get(p.a_scales, soff_a[j]);
  };

  f32x16_t acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // (one offset per read: the compiler follows short address chains only when
  // it decides which loads into LDS a read has to wait for)
  const uint32_t place[2] = {(uint32_t)(r32 * 64 + (((2 * q) ^ ((r32 >> 2) & 3)) << 4)),
                             (uint32_t)(r32 * 64 + (((2 * q + 1) ^ ((r32 >> 2) & 3)) << 4))};
  const uint32_t w_place[2] = {place[0] + (uint32_t)(A_BYTES + 4096 * wave),
                               place[1] + (uint32_t)(A_BYTES + 4096 * wave)};
  auto ld = [&](const uint8_t* st, uint32_t off) -> u32x4 {
    return *reinterpret_cast<const u32x4*>(st + off);
  };

  auto run = [&](auto nv_c) {
    constexpr int NV = decltype(nv_c)::value;
    // FULL: the steps kt + 1 .. kt + 3 are there, and those whose scales are
    // loaded here
    auto step = [&](const uint8_t* st, uint8_t* next, int kt, auto sub_c, auto full_c) {
      constexpr int SUB = decltype(sub_c)::value;
      constexpr bool FULL = decltype(full_c)::value;
      // all but the newest stage's loads are there; every wave is past the
      // stage that is filled next
      if (FULL || kt + 1 < nk) asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      uint32_t tw[2], ta[NV];
#pragma unroll
      for (int i = 0; i < 2; ++i) tw[i] = sw[i][SUB] >> (16 * q);
#pragma unroll
      for (int j = 0; j < NV; ++j) ta[j] = sa[j][SUB] >> (16 * q);
      if (SUB == 2 && (FULL || kt + 1 < nk)) load_scales(kt + 1, full_c);
      asm volatile("" ::: "memory");                     // (older than the stage's loads)
      if (FULL || kt + 2 < nk) issue_loads(next, kt + 2);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u32x4 W[2], A[NV];
#pragma unroll
        for (int i = 0; i < 2; ++i) W[i] = ld(st, w_place[s] + 2048u * i);
#pragma unroll
        for (int j = 0; j < NV; ++j) A[j] = ld(st, place[s] + 2048u * j);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[i][j] = s == 0 ? mfma32_mx4<0>(W[i], tw[i], A[j], ta[j], acc[i][j])
                               : mfma32_mx4<1>(W[i], tw[i], A[j], ta[j], acc[i][j]);
      }
    };
    using c0 = std::integral_constant<int, 0>;
    using c1 = std::integral_constant<int, 1>;
    using c2 = std::integral_constant<int, 2>;
    using all = std::true_type;
    using some = std::false_type;
    load_scales(0, some{});
    issue_loads(st0, 0);
    if (nk > 1) issue_loads(st1, 1);
    int kt = 0;
    for (; kt + 5 < nk; kt += 3) {
      step(st0, st2, kt, c0{}, all{});
      step(st1, st0, kt + 1, c1{}, all{});
      step(st2, st1, kt + 2, c2{}, all{});
    }
    for (; kt < nk; kt += 3) {
      step(st0, st2, kt, c0{}, some{});
      if (kt + 1 < nk) step(st1, st0, kt + 1, c1{}, some{});
      if (kt + 2 < nk) step(st2, st1, kt + 2, c2{}, some{});
    }
    // lane (r, q) holds columns 8 g + 4 q .. + 3 of its row in registers 4 g ..
    // 4 g + 3: one exchange between the lane halves makes 16-byte pieces
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int row = 32 * j + r32;
      uint16_t* dst = p.y + (p0 + row) * NO;
#pragma unroll
      for (int i = 0; i < (GLU ? 1 : 2); ++i)
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
          uint32_t u[4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int x = 4 * (g + h) + 2 * c;
              u[2 * h + c] = GLU ? bf16x2_rne(silu_mul(acc[0][j][x], acc[1][j][x]),
                                              silu_mul(acc[0][j][x + 1], acc[1][j][x + 1]))
                                 : bf16x2_rne(acc[i][j][x], acc[i][j][x + 1]);
            }
          // lanes below 32 get all of columns 8 g .., the others of 8 (g + 1) ..
          const auto x0 = __builtin_amdgcn_permlane32_swap(u[0], u[2], false, false);
          const auto x1 = __builtin_amdgcn_permlane32_swap(u[1], u[3], false, false);
          const int64_t n = n0 + CW * wave + 32 * i + 8 * (g + q);
          if (row < valid && n < NO)
            *reinterpret_cast<uint4*>(dst + n) = make_uint4(x0[0], x1[0], x0[1], x1[1]);
        }
    }
  };
  if (valid > 96) run(std::integral_constant<int, 4>{});
  else if (valid > 64) run(std::integral_constant<int, 3>{});
  else if (valid > 32) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 1>{});
}

}  // namespace nvfp4

using namespace nvfp4;

// row tiles of 128 that the experts' rows can make
static int64_t mx_row_tiles(int64_t E, int64_t M_total) {
  return (M_total + mxb::BM - 1) / mxb::BM + E;
}

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
  if (M_total > 32 * E) {
    const int64_t n_tiles = (N + mxb::BN - 1) / mxb::BN, m_tiles = mx_row_tiles(E, M_total);
    NV_REQUIRE(m_tiles * n_tiles < (1 << 24), NVFP4_ERR_UNSUPPORTED, "%s: too many tiles", name);
    int32_t* count = static_cast<int32_t*>(ws);
    int4* tiles = reinterpret_cast<int4*>(static_cast<char*>(ws) + 256);
    const unsigned nb = (unsigned)((m_tiles * n_tiles + 7) / 8 * 8);
    const int64_t tb = (m_tiles + 1023) / 1024;
    k_mx_tiles<<<(unsigned)(tb < 256 ? tb : 256), 1024, 0, s>>>(p, tiles, count);
    if (glu)
      k_mx_big<true><<<nb, 256, 0, s>>>(p, tiles, count, (int)n_tiles);
    else
      k_mx_big<false><<<nb, 256, 0, s>>>(p, tiles, count, (int)n_tiles);
    return check_launch(name);
  }
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
  (void)N, (void)K;
  if (E < 1 || E > 1024 || M_total < 0 || M_total >= (1LL << 31)) return 256;
  return 256 + round_up((size_t)mx_row_tiles(E, M_total) * sizeof(int4), 256);
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
