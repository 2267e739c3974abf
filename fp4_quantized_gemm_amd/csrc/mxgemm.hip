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
__device__ __forceinline__ void clamp_rows(int M_total, int& lo, int& hi) {
  lo = max(0, min(lo, M_total));
  hi = max(lo, min(hi, M_total));
}
__device__ __forceinline__ void expert_rows(const MxGemmArgs& p, int e, int& lo, int& hi) {
  // (of the wave's one expert: scalar loads, that wait for no vector load or store)
  typedef const int32_t __attribute__((address_space(4))) * scalar_ptr;
  const scalar_ptr offsets = (scalar_ptr)p.offsets;
  lo = offsets[e];
  hi = offsets[e + 1];
  clamp_rows((int)p.M_total, lo, hi);
}

__device__ __forceinline__ int64_t source_row(const MxGemmArgs& p, int64_t row) {
  const int64_t t = p.a_rows ? (int64_t)p.a_rows[row] : row;
  return t < 0 ? 0 : (t >= p.M_src ? p.M_src - 1 : t);
}

// ------------------------------------------------------------------------
// Small products, without LDS: a wave owns 16 weight rows (GLU: 16 gate rows and
// the same 16 up rows) and multiplies all of K with a tile of 16 activation
// rows, operands straight from memory to registers.  K advances in chunks of
// 512, the next one under way while one is multiplied.  Lane (r, q) takes the
// 16-byte pieces 4 s + q, s = 0 .. 3, of its row's 256 bytes, and the chunk's 16
// scale bytes, of which byte q of dword s belongs to piece s.
//
// Bound by latency: a round trip per chunk, in as many workgroups as there are
// tiles (two tiles of rows per wave, weights read once: 128 rows of one
// 4096x1536 7.0 us against 8.2, but 32 rows for each of 4 of 1536x8192 43
// against 21, 64 rows of one of it 28.5 against 19.6).  Taken for at most 512
// tiles of 16 rows x 64 columns.  Times in a graph, against the large tiles: 64
// rows of one 512x512 3.2 us, 6.0; one row for each of 8 of 128 experts of
// 4096x1536 (512 tiles) 8.3, 11.2; 4 rows for each of 8 of it (512) 8.6, 10.8;
// 64 for each of 4 of 1536x2048 (432) 11.0, 11.5; beyond, 32 rows for each of 4
// of 4096x1536 (640) 11.7, 9.7; 16 for each of 8 of it (768) 12.3, 11.0.
// ------------------------------------------------------------------------
template <int R>
struct MxChunk {                                        // R: groups of 16 weight rows
  u32x4 w[R][4], sw[R], a[4], sa;
};

template <bool GLU>
__device__ __forceinline__ void mx_few_tile(const MxGemmArgs& p, int e, int64_t p0, int64_t hi) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  constexpr int R = GLU ? 2 : 1;
  const int64_t NO = GLU ? p.N / 2 : p.N;              // output columns
  const int64_t KC = p.K / 2, KS = p.K / 32;
  const int nd = (int)(p.K / 128), nch = (nd + 3) / 4;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * 16;
  const int64_t row = p0 + r16;
  const int64_t src = source_row(p, row < hi ? row : hi - 1);
  const uint8_t* const ac = p.a_codes + src * KC + 16 * q;
  const uint8_t* const asc = p.a_scales + src * KS;
  const uint8_t* wc[R];
  const uint8_t* wsc[R];
#pragma unroll
  for (int g = 0; g < R; ++g) {
    int64_t n = n0 + r16;
    n = n < NO ? n : NO - 1;
    if (g == 1) n += NO;
    wc[g] = p.w_codes + ((int64_t)e * p.N + n) * KC + 16 * q;
    wsc[g] = p.w_scales + ((int64_t)e * p.N + n) * KS;
  }
  typedef u32x4 u32x4a __attribute__((aligned(4)));     // (rows of scales are whole dwords)
  using Chunk = MxChunk<R>;
  auto load = [&](Chunk& k, int c) {
    const int m = nd - 4 * c;                           // pieces that are there, if fewer than 4
    const int64_t kc = 256 * c, ks = 16 * c;
    auto row = [&](u32x4* pieces, u32x4& scales, const uint8_t* codes, const uint8_t* bytes) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s < m) pieces[s] = *reinterpret_cast<const u32x4*>(codes + kc + 64 * s);
      if (m >= 4) {
        scales = *reinterpret_cast<const u32x4a*>(bytes + ks);
      } else {
#pragma unroll
        for (int s = 0; s < 3; ++s)
          if (s < m) scales[s] = reinterpret_cast<const uint32_t*>(bytes + ks)[s];
      }
    };
#pragma unroll
    for (int g = 0; g < R; ++g) row(k.w[g], k.sw[g], wc[g], wsc[g]);
    row(k.a, k.sa, ac, asc);
  };
  f32x4_t acc[R];
#pragma unroll
  for (int g = 0; g < R; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Chunk& k, int c) {
    const int m = nd - 4 * c;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (s < m) {
#pragma unroll
        for (int g = 0; g < R; ++g)
          acc[g] = mfma16_mx4(k.w[g][s], k.sw[g][s] >> (8 * q), k.a[s], k.sa[s] >> (8 * q), acc[g]);
      }
  };
  Chunk k0, k1;
  load(k0, 0);
  for (int c = 0; c < nch; c += 2) {
    if (c + 1 < nch) load(k1, c + 1);
    multiply(k0, c);
    if (c + 1 < nch) {
      if (c + 2 < nch) load(k0, c + 2);
      multiply(k1, c + 1);
    }
  }
  // lane (r, q): columns n0 + 4 q .. + 3 of row p0 + r
  const int64_t n = n0 + 4 * q;
  if (row >= hi || n >= NO) return;
  f32x4_t v = acc[0];
  if constexpr (GLU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = silu_mul(v[i], acc[1][i]);
  }
  *reinterpret_cast<uint2*>(p.y + row * NO + n) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
}

// Workgroup (x, y): columns 64 x .. 64 x + 63 of the y-th tile of 16 rows.  Every
// wave counts the experts' tiles, `per` experts to a lane, and looks its own up:
// a grid over the experts would have 8192 workgroups for one token's 8 of 128
// (11.1 us in a graph against 8.3; 0.5 us less for up to 8 experts).
template <bool GLU>
__global__ void __launch_bounds__(256, 2)
k_mx_few(MxGemmArgs p) {
  const int lane = threadIdx.x & 63, y = blockIdx.y;
  if (p.E == 1) {
    int lo, hi;
    expert_rows(p, 0, lo, hi);
    if (16 * y < hi - lo) mx_few_tile<GLU>(p, 0, lo + 16 * y, hi);
    return;
  }
  const int per = (p.E + 63) / 64;
  int n = 0;
  for (int i0 = 0; i0 < per; i0 += 4) {
    int off[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) off[i] = p.offsets[min(lane * per + min(i0 + i, per), p.E)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int lo = off[i], hi = off[i + 1];                 // (past the lane's last: the same)
      clamp_rows((int)p.M_total, lo, hi);
      n += (hi - lo + 15) / 16;
    }
  }
  int incl = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  const uint64_t mine = __ballot(incl > y);
  if (!mine) return;
  const int l = __builtin_ctzll(mine);
  int t = y - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l));
  const int last = min((l + 1) * per, p.E);
  for (int e = l * per; e < last; ++e) {
    int lo, hi;
    expert_rows(p, e, lo, hi);
    const int tiles = (hi - lo + 15) / 16;
    if (t < tiles) {
      mx_few_tile<GLU>(p, e, lo + 16 * t, hi);
      return;
    }
    t -= tiles;
  }
}

// ------------------------------------------------------------------------
// Large tiles: 128 activation rows x 256 weight rows per workgroup of four
// waves, two workgroups on a CU, so one's epilogue and waits run under the
// other's products; a workgroup goes from tile to tile, and the loads of the
// next tile's first step run under the last one's products.
//
// Wave w owns 64 weight rows (GLU: 32 gate rows and the same 32 up rows) and
// all of the tile's activation rows: 2 x 4 accumulators of 32x32.  K advances
// in steps of 256, so that a row of a step is a whole 128-byte line: the
// vector caches take as long for half a line (rows of 64 bytes reach 16 TB/s
// from L2 into LDS, rows of 128 bytes 33).  Activation rows go through two LDS
// stages, filled one step ahead by buffer loads straight into LDS; a weight
// row is read by one wave only, so the weights have one stage, which the wave
// empties into registers at the start of a step and fills again at once.
//
// A stage's row is its 128 code bytes, eight 16-byte pieces; piece c lies at
// place c ^ ((row >> 1) & 7), so that a fragment's 32 rows are spread over all
// banks.  (The scales' are not: rows 16 bytes apart, two to a bank.  Counted over
// the whole kernel, 29% of the cycles in which LDS is busy are conflicts.)  Lane
// (r, q) of instruction s = 0 .. 3 takes piece 4 q + s of its row, both operands
// alike: which 32 of the 256 columns a lane of an instruction has does not matter
// for the sum, and so the scales of the four are the bytes of one dword.  (A last
// step of 128 columns: s = 0, 1, piece 2 q + s.)  Scales take the same way
// through LDS, 16 bytes of a row for two steps.
//
// Measured: 131072 rows over 128 experts of 4096x1536 552 to 563 us, by card (2.9
// to 3.0 PFLOP/s, 1.6 GB), 32768 skewed rows over 128 of 1536x2048 with SwiGLU 89
// us, 2048 rows over 128 of 4096x1536 86 us (4.9 TB/s of weights), one 8192x8192
// with 16384 rows 545 us (4.0 PFLOP/s).  The first is bound by waits between loads, products and
// stores at 1.9 GHz: the matrix units are 39% busy; of 580 us on another card,
// 489 were left without the stores, 458 without the weights' loads, 338 for the
// products and LDS reads alone; on codes of zeros, which draw less power, it
// takes a fifth less.  64x256 tiles for up to 64 rows share the
// kernel.  Tried: one workgroup per CU with 256x256 tiles, of four waves 615 us,
// of eight with all loads two steps ahead 563 (10% faster for one 8192x8192, the
// same here); 1 to 16 row tiles to a group, staggered starts, loads between the
// products, touching the next tile's weights a tile ahead: no change.
// ------------------------------------------------------------------------
namespace mxb {
constexpr int BM = 128, BN = 256;
constexpr int A_BYTES = BM * 128, W_BYTES = BN * 128, SCALES = (BM + BN) * 16;
}  // namespace mxb

// D += 2^(sa - 127 + sb - 127) A B over 64 k: lane (r = l % 32, q = l / 32)
// has 32 codes of row r in 16 bytes, byte SEL of sa / sb their scale
template <int SEL>
__device__ __forceinline__ f32x16_t mfma32_mx4(const u32x4& a, uint32_t sa, const u32x4& b,
                                               uint32_t sb, f32x16_t c) {
  const mx_i32x8 a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const mx_i32x8 b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

// all but the newest N of the wave's loads and stores are done, and its reads
// of LDS; then every wave's
template <int N>
__device__ __forceinline__ void mx_wait() {
  // vmcnt(N) lgkmcnt(0), in a form that the compiler counts with
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | (7 << 4));
  asm volatile("" ::: "memory");
}
// all but the newest N of the wave's reads and writes of LDS are done (they
// end in the order in which they were issued)
template <int N>
__device__ __forceinline__ void mx_wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (N << 8));
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void mx_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_buffer(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes,
                                           kBufferRsrcWord3);
}

// N stores that go nowhere, behind what was issued before
template <int N>
__device__ __forceinline__ void mx_no_stores(uint16_t* y) {
  const __amdgpu_buffer_rsrc_t none = mx_buffer(y, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i)
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, none, 16u * i, 0, 2);
}

struct MxTile {
  int e, p0, valid, nt;
};

// prefix[e] = row tiles of the experts before e, for e = 0 .. 1024, at most cap:
// as many as offsets that never decrease can make; of others what goes beyond is
// left out.  scratch: 4 words.
__device__ __forceinline__ void mx_count_tiles(const MxGemmArgs& p, int cap, int32_t* prefix,
                                               int32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int off[5], n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) off[i] = p.offsets[min(4 * tid + i, p.E)];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int lo = off[i], hi = off[i + 1];
    clamp_rows((int)p.M_total, lo, hi);
    n[i] = 4 * tid + i < p.E ? (int)(((uint32_t)(hi - lo) + (mxb::BM - 1)) / mxb::BM) : 0;
    sum = min(sum + n[i], cap);
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl = min(incl + u, cap);
  }
  int before = __shfl_up(incl, 1);
  if (lane == 0) before = 0;
  if (lane == 63) scratch[wave] = incl;
  __syncthreads();
  for (int w = 0; w < wave; ++w) before = min(before + scratch[w], cap);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    prefix[4 * tid + i] = before;
    before = min(before + n[i], cap);
  }
  if (tid == 255) prefix[1024] = before;
  __syncthreads();
}

// Tile v in the order: groups of 8 row tiles x all column tiles, row tiles
// fastest.  The row tile's expert, the last whose prefix is not beyond it, is
// found in two steps of 64 and 16 lanes.
__device__ __forceinline__ MxTile mx_tile(const MxGemmArgs& p, const int32_t* prefix, int real_m,
                                          int n_tiles, int v) {
  constexpr int G = 8;
  const int gi = v / (G * n_tiles), gr = v - gi * G * n_tiles;
  const int gm = real_m - G * gi < G ? real_m - G * gi : G;
  const int nt = gr / gm, t = G * gi + gr - nt * gm;
  const int lane = threadIdx.x & 63;
  const uint64_t m1 = __ballot(16 * lane < p.E && prefix[16 * lane] <= t);
  const int e1 = 16 * (__builtin_popcountll(m1) - 1) + (lane & 15);
  const int at = prefix[e1];
  const uint64_t m2 = __ballot(lane < 16 && e1 < p.E && at <= t);
  const int l2 = __builtin_popcountll(m2) - 1;
  const int e = __builtin_amdgcn_readlane(e1, l2);
  int lo, hi;
  expert_rows(p, e, lo, hi);
  const int p0 = lo + (t - __builtin_amdgcn_readlane(at, l2)) * mxb::BM;
  return {e, p0, min(hi - p0, mxb::BM), nt};
}

// ND: K / 128 modulo 4, so what the last steps are
template <bool GLU, int ND>
__global__ void __launch_bounds__(256, 2)
k_mx_big(MxGemmArgs p, int32_t* __restrict__ taken, int max_m, int n_tiles) {
  using namespace mxb;
  // separate objects, each access naming its own: the compiler then does not
  // wait for loads into the others
  __shared__ __attribute__((aligned(16))) uint8_t sa0[A_BYTES], sa1[A_BYTES], sw[W_BYTES], ssc[SCALES];
  __shared__ int32_t rows[2][BM], prefix[1025];
  // written by one wave and read by all, once per tile, so by atomics: no plain
  // read of it may be taken out of the loop, whatever fences are there
  __shared__ int32_t next_v;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 5, r32 = lane & 31;

  // each XCD (workgroup b runs on XCD b % 8) takes a contiguous range of the
  // tiles, so its L2 holds an expert's weights; its workgroups take every
  // stride-th, or (taken: eight counters, 0 at first) after two each the next
  // that nobody has (which workgroup computes a tile does not show in it)
  mx_count_tiles(p, max_m, prefix, rows[0]);
  const int real_m = __builtin_amdgcn_readfirstlane(prefix[1024]);
  const int total = real_m * n_tiles;
  const int per_xcd = (total + 7) / 8;
  const int first = ((int)blockIdx.x & 7) * per_xcd;
  const int end = first + per_xcd < total ? first + per_xcd : total;
  const int stride = (int)gridDim.x >> 3;
  int v = first + ((int)blockIdx.x >> 3);
  if (v >= end) return;
  MxTile cur = mx_tile(p, prefix, real_m, n_tiles, v);
  v += stride;                                          // the next one
  // (an index that looks different per lane: of a common address the compiler
  // makes one atomic for the wave, and waits for it at once)
  uint32_t ticket_at = blockIdx.x & 7;
  asm volatile("" : "+v"(ticket_at));

  const uint32_t KC = (uint32_t)(p.K / 2), KS = (uint32_t)(p.K / 32);
  const int nd = (int)(p.K / 128);                      // dwords of a row's scales
  constexpr bool kHalf = ND % 2 == 1;                   // the last step is of 128 columns
  constexpr bool kOdd = ND == 1 || ND == 2;             // an odd number of steps
  const int ns = (nd + 1) / 2, M_last = (int)p.M_src - 1;
  const uint32_t NO = (uint32_t)(GLU ? p.N / 2 : p.N);  // output columns
  constexpr uint32_t CW = GLU ? 32 : 64;                // ... of a wave
  const __amdgpu_buffer_rsrc_t rs_a = mx_buffer(p.a_codes, (uint64_t)p.M_src * KC);
  const __amdgpu_buffer_rsrc_t rs_as = mx_buffer(p.a_scales, (uint64_t)p.M_src * KS);

  // ---- loads.  A tile's loads go through these; they are set for the next
  // tile when the current one's last are on their way.
  __amdgpu_buffer_rsrc_t rs_w, rs_s;
  uint32_t off_a[4], off_s[2];
  uint32_t w_row0, w_row1;                              // the wave's first 32 weight rows, the other 32
  // One load instruction fills 8 rows of 128 bytes: lane l's 16 bytes land at
  // row l / 8, place l % 8.  (The lane is taken afresh each time, so that what
  // follows from it is not kept in registers through the products.)
  auto aim = [&](const MxTile& t, const int32_t* src) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const uint32_t n0 = (uint32_t)t.nt * 4 * CW;
    auto a_row = [&](int r) -> uint32_t {
      const int s = p.a_rows ? src[r] : t.p0 + (r < t.valid ? r : t.valid - 1);
      return (uint32_t)max(0, min(s, M_last));
    };
    // (multiplied apart from the addition: a 64-bit multiply-add would hold a
    // pair of registers for each offset)
    auto times = [](uint32_t a, uint32_t b) {
      uint32_t m = a * b;
      asm volatile("" : "+v"(m));
      return m;
    };
    rs_w = mx_buffer(p.w_codes + (int64_t)t.e * p.N * KC, (uint64_t)p.N * KC);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (4 * wave + i) * 8 + (lane >> 3);
      off_a[i] = times(a_row(r), KC) + 16u * ((lane & 7) ^ ((r >> 1) & 7));
    }
    w_row0 = n0 + CW * wave;
    w_row1 = GLU ? w_row0 + NO : w_row0 + 32;
    // scales: wave 0 the activation rows', waves 1 and 2 the weight rows' (3:
    // the same as 2, so that every wave has as many loads in flight); the
    // tile's weight row r is wave r / 64's row r % 64
    rs_s = wave == 0 ? rs_as : mx_buffer(p.w_scales + (int64_t)t.e * p.N * KS, (uint64_t)p.N * KS);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (wave < 2 ? 0 : 128) + 64 * i + lane;
      uint32_t n = n0 + (uint32_t)(GLU ? (r >> 6) * 32 + (r & 31) : r);
      n = n < NO ? n : NO - 1;
      off_s[i] = times(wave == 0 ? a_row(r) : GLU && (r & 32) ? n + NO : n, KS);
    }
  };
  // A last step of 128 columns has rows of 64 bytes: the lanes of the pieces 4
  // to 7, the odd four of an even instruction, load 0 to 3 instead.
  auto cut = [&](int kt, int i) -> uint32_t {
    return kHalf && 2 * kt + 1 == nd && (((lane >> 2) ^ i) & 1) ? 64u : 0u;
  };
  auto issue_a = [&](uint8_t* st, int kt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t off = off_a[i] - cut(kt, i);
      const uint32_t k0 = 128u * (uint32_t)kt;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(st + (4 * wave + i) * 1024), 16, off, k0, 0, 0);
    }
  };
  // rows of the lanes of one instruction, and their places' pieces: of the even
  // instructions and of the odd
  const uint32_t w_lane = (uint32_t)(lane >> 3) * KC;
  const uint32_t off_w0 = w_lane + 16u * ((lane & 7) ^ (lane >> 4));
  const uint32_t off_w1 = w_lane + 16u * ((lane & 7) ^ (lane >> 4) ^ 4);
  auto issue_w = [&](int kt) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // (rows past the last: the last 8, of which nothing is stored)
      uint32_t r = (i < 4 ? w_row0 : w_row1) + 8u * (i & 3);
      r = r < (uint32_t)p.N - 8u ? r : (uint32_t)p.N - 8u;
      const uint32_t off = (i & 1 ? off_w1 : off_w0) - cut(kt, i);
      const uint32_t k0 = r * KC + 128u * (uint32_t)kt;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_w, lds_ptr(sw + (8 * wave + i) * 1024), 16, off, k0, 0, 0);
    }
  };
  // the scales of two steps (the last 16 bytes of a row, where fewer are left),
  // row after row; of rows of fewer bytes dword after dword
  auto issue_scales = [&](int kt) {
    const int r0 = 128 * (wave < 2 ? wave : 2);
    if (ND == 0 || nd >= 4) {
      const uint32_t s0 = 8u * kt < KS - 16u ? 8u * kt : KS - 16u;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_s, lds_ptr(ssc + (r0 + 64 * i) * 16), 16, off_s[i], s0,
                                                 0, 0);
    } else {
#pragma unroll 1
      for (int k = 0; k < nd; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_s, lds_ptr(ssc + (384 * k + r0 + 64 * i) * 4), 4,
                                                   off_s[i], 4u * k, 0, 0);
    }
  };
  // a tile's row list, straight to LDS
  auto issue_rows = [&](const MxTile& t, int32_t* dst) {
    if (wave < 2) {
      const int r = 64 * wave + lane;
      const __amdgpu_buffer_rsrc_t rs = mx_buffer(p.a_rows + t.p0, 4ull * t.valid);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, lds_ptr(dst + 64 * wave), 4,
                                               4u * (r < t.valid ? r : t.valid - 1), 0, 0, 0);
    }
  };
  // (one offset per read: the compiler follows short address chains only when
  // it decides which loads into LDS a read has to wait for)
  auto ld = [&](const uint8_t* st, uint32_t off) -> u32x4 {
    return *reinterpret_cast<const u32x4*>(st + off);
  };
  auto ld_scale = [&](uint32_t off) -> uint32_t {
    return *reinterpret_cast<const uint32_t*>(ssc + off);
  };

  int buf = 0;
  if (p.a_rows) {
    issue_rows(cur, rows[0]);
    mx_wait<0>();
    mx_barrier();
  }
  aim(cur, rows[0]);
  issue_scales(0);
  issue_a(sa0, 0);
  issue_w(0);

  // Every tile ends with as many stores, and one comes before the first tile
  // (those of rows that are not there go nowhere), so that a tile's first step
  // waits for what was loaded before them and not for them.
  constexpr int kStores = GLU ? 8 : 16;
  mx_no_stores<kStores>(p.y);
  bool odd = false;                                     // the tile's first step is in sa1
  for (;;) {
    const bool more = v < end;
    MxTile nxt = cur;
    int ticket;
    if (more) {
      nxt = mx_tile(p, prefix, real_m, n_tiles, v);
      if (p.a_rows) issue_rows(nxt, rows[buf ^ 1]);
      if (taken && tid == 0) ticket = atomicAdd(taken + ticket_at, 1);
    }

    // NV: blocks of 32 activation rows; x: the stage of the even steps
    auto run = [&](auto nv_c, uint8_t* const x, uint8_t* const y) __attribute__((always_inline)) {
      constexpr int NV = decltype(nv_c)::value;
      f32x16_t acc[2][NV];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
      uint32_t tw[2][2], ta[2][NV];                     // scales of a pair of steps
      // One step, from stage st; the next one's activation rows go to `other`.
      // U: the first or the second of a pair.  LAST: the tile's last, after
      // which comes the next tile's first; HALF: of 128 columns.
      auto step = [&](int kt, uint8_t* st, uint8_t* other, auto u_c, auto last_c, auto half_c) __attribute__((always_inline)) {
        constexpr int U = decltype(u_c)::value;
        constexpr bool LAST = decltype(last_c)::value, HALF = decltype(half_c)::value;
        constexpr int S = HALF ? 2 : 4;
        if (kt > 0 || ns == 1) mx_wait<0>();
        else mx_wait<kStores>();
        mx_barrier();
        if constexpr (U == 0) {
          // dword 2 u + q of the step u of the pair (HALF: 2 u, and two of its
          // bytes), behind those that a pair at the end of a row has before it
          const int left = nd - 2 * kt;                 // dwords of the pair that are there
          const bool wide = ND == 0 || nd >= 4;
          const uint32_t per_row = wide ? 16 : 4, per_dword = wide ? 4 : 1536;
          const uint32_t d0 = ND != 0 && wide && left < 4 ? (uint32_t)(4 - left) : 0u;
          auto get = [&](int u, bool half) {
            const uint32_t at = (d0 + 2u * u + (half ? 0u : (uint32_t)q)) * per_dword;
            const int sh = half ? 16 * q : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              tw[u][i] = ld_scale((uint32_t)(BM + 64 * wave + 32 * i + r32) * per_row + at) >> sh;
#pragma unroll
            for (int j = 0; j < NV; ++j) ta[u][j] = ld_scale((uint32_t)(32 * j + r32) * per_row + at) >> sh;
          };
          get(0, ND == 1 && left == 1);
          if (ND == 0 || left > 2) get(1, ND == 3 && left == 3);
        }
        uint32_t here = (uint32_t)(r32 * 128 + (((HALF ? 2 * q : 4 * q) ^ ((r32 >> 1) & 7)) << 4));
        asm volatile("" : "+v"(here));                   // (its sums are not kept in registers)
        if constexpr (!LAST) issue_a(other, kt + 1);
        u32x4 W[S][2], A[S][NV];
        auto read_a = [&](int s) {
#pragma unroll
          for (int j = 0; j < NV; ++j) A[s][j] = ld(st, (here ^ (16u * s)) + 4096u * j);
        };
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i) W[s][i] = ld(sw, (here ^ (16u * s)) + (uint32_t)(8192 * wave) + 4096u * i);
        // (the reads of the scales and the weights are issued before this, at least
        // the 2 NV of A[0] and A[1] after it)
        asm volatile("" ::: "memory");
        read_a(0);
        const bool ahead = !LAST || more;
        if (LAST && more) {
          aim(nxt, rows[buf ^ 1]);
          if (taken && tid == 0)
            __hip_atomic_store(&next_v, first + 2 * stride + ticket, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
          issue_a(other, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
          if (s + 1 < S) read_a(s + 1);
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (s == 0) acc[i][j] = mfma32_mx4<0>(W[s][i], tw[U][i], A[s][j], ta[U][j], acc[i][j]);
              if (s == 1) acc[i][j] = mfma32_mx4<1>(W[s][i], tw[U][i], A[s][j], ta[U][j], acc[i][j]);
              if (s == 2) acc[i][j] = mfma32_mx4<2>(W[s][i], tw[U][i], A[s][j], ta[U][j], acc[i][j]);
              if (s == 3) acc[i][j] = mfma32_mx4<3>(W[s][i], tw[U][i], A[s][j], ta[U][j], acc[i][j]);
            }
          __builtin_amdgcn_sched_barrier(0);
          if (s == 0 && ahead) {
            // Every read of the weights' stage, which only this wave reads, is done:
            // it is free.  (A wait of its own: the products above would wait for
            // it too, but the compiler may move them behind these loads.)  The
            // scales' stage is free one step later, or once every wave has read
            // the tile's last.
            mx_wait_lds<NV>();
            issue_w(LAST ? 0 : kt + 1);
            if (U == 1 || LAST) {
              if (U == 0) mx_barrier();
              issue_scales(LAST ? 0 : kt + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        // (the products belong here, not behind the next wait)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) asm volatile("" : "+v"(acc[i][j]));
      };
      using u0 = std::integral_constant<int, 0>;
      using u1 = std::integral_constant<int, 1>;
      using yes = std::true_type;
      using no = std::false_type;
      using half = std::integral_constant<bool, kHalf>;
      int kt = 0;
      for (; kt + 2 < ns; kt += 2) {
        step(kt, x, y, u0{}, no{}, no{});
        step(kt + 1, y, x, u1{}, no{}, no{});
      }
      if constexpr (kOdd) {
        step(kt, x, y, u0{}, yes{}, half{});
      } else {
        step(kt, x, y, u0{}, no{}, no{});
        step(kt + 1, y, x, u1{}, yes{}, half{});
      }

      // Rows of 128 bytes (GLU: 64) of the wave's columns, put together in 4 KB
      // of the stage that nobody reads any more.  Rows past the tile's last lie
      // past the buffer.
      mx_wait<63>();
      mx_barrier();
      const __amdgpu_buffer_rsrc_t rs_y =
          mx_buffer(p.y + (int64_t)cur.p0 * NO, (uint64_t)cur.valid * NO * 2);
      const uint32_t n0 = (uint32_t)cur.nt * 4 * CW + CW * wave;
      int l = threadIdx.x & 63;                          // (afresh, as in aim)
      asm volatile("" : "+v"(l));
      constexpr int LR = GLU ? 4 : 8;                   // lanes of a row of 16-byte pieces
      auto put = [&](uint8_t* const own) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int r = l & 31;
#pragma unroll
          for (int i = 0; i < (GLU ? 1 : 2); ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t u[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int e = 4 * g + 2 * c;
                u[c] = GLU ? bf16x2_rne(silu_mul(acc[0][j][e], acc[1][j][e]),
                                        silu_mul(acc[0][j][e + 1], acc[1][j][e + 1]))
                           : bf16x2_rne(acc[i][j][e], acc[i][j][e + 1]);
              }
              // (32 rows' 8 bytes cover all banks once)
              const int piece = GLU ? g ^ ((r >> 2) & 3) : (4 * i + g) ^ ((r >> 1) & 7);
              const int half = (l >> 5) ^ (r >> 4);
              *reinterpret_cast<uint2*>(own + (r * (16 * LR) + (piece << 4) + half * 8)) =
                  make_uint2(u[0], u[1]);
            }
          // (other lanes have written what is read next, and write over it for the
          // next 32 rows: a wave's accesses of LDS end in their order)
          asm volatile("" ::: "memory");
          u32x4 h[LR / 2];
#pragma unroll
          for (int t = 0; t < LR / 2; ++t) {
            const int row = (64 / LR) * t + l / LR, c = l % LR;
            h[t] = *reinterpret_cast<const u32x4*>(
                own + (row * (16 * LR) + ((GLU ? c ^ ((row >> 2) & 3) : c ^ ((row >> 1) & 7)) << 4)));
          }
          asm volatile("" ::: "memory");
#pragma unroll
          for (int t = 0; t < LR / 2; ++t) {
            const int row = (64 / LR) * t + l / LR, c = l % LR;
            // (rows 16 .. 31, the second half of the reads, have their halves swapped)
            const u32x4 o = t < LR / 4 ? h[t] : u32x4{h[t].z, h[t].w, h[t].x, h[t].y};
            const uint32_t n = n0 + 8 * c;
            __builtin_amdgcn_raw_buffer_store_b128(
                o, rs_y, n < NO ? ((uint32_t)(32 * j + row) * NO + n) * 2u : 0xFFFFFFF0u, 0, 2);
          }
        }
      };
      put((kOdd ? x : y) + 4096 * wave);
      mx_no_stores<(4 - NV) * (kStores / 4)>(p.y);
    };
    using n4 = std::integral_constant<int, 4>;
    using n2 = std::integral_constant<int, 2>;
    // (as functions of their own these would have their captures in memory)
    auto tile = [&](uint8_t* const x, uint8_t* const y) __attribute__((always_inline)) {
      if (cur.valid > 64) run(n4{}, x, y);
      else run(n2{}, x, y);
    };
    if (kOdd && odd) tile(sa1, sa0);
    else tile(sa0, sa1);
    if (!more) return;
    if (taken)
      v = __builtin_amdgcn_readfirstlane(__hip_atomic_load(&next_v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP));
    else
      v += stride;
    cur = nxt;
    buf ^= 1;
    odd = !odd;
  }
}

}  // namespace nvfp4

using namespace nvfp4;

// row tiles of 128 that the experts' rows can make
static int64_t mx_row_tiles(int64_t E, int64_t M_total) {
  return (M_total + mxb::BM - 1) / mxb::BM + E;
}

template <bool GLU>
static void mx_launch_big(unsigned nb, hipStream_t s, const MxGemmArgs& p, int32_t* taken, int max_m,
                          int n_tiles) {
  switch ((p.K / 128) % 4) {
    case 0: k_mx_big<GLU, 0><<<nb, 256, 0, s>>>(p, taken, max_m, n_tiles); break;
    case 1: k_mx_big<GLU, 1><<<nb, 256, 0, s>>>(p, taken, max_m, n_tiles); break;
    case 2: k_mx_big<GLU, 2><<<nb, 256, 0, s>>>(p, taken, max_m, n_tiles); break;
    default: k_mx_big<GLU, 3><<<nb, 256, 0, s>>>(p, taken, max_m, n_tiles); break;
  }
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
  // small: tiles of 16 rows (and half a one more for each expert that can have
  // rows) times 64 columns
  const int64_t blocks = (NO + 63) / 64, tiles16 = (M_total + 15) / 16;
  const int64_t active = M_total < E ? M_total : E;
  const int64_t likely = tiles16 + active / 2;
  if (blocks * (likely > active ? likely : active) > 512) {
    const int64_t n_tiles = (N + mxb::BN - 1) / mxb::BN, m_tiles = mx_row_tiles(E, M_total);
    NV_REQUIRE(m_tiles * n_tiles < (1 << 28), NVFP4_ERR_UNSUPPORTED, "%s: too many tiles", name);
    // two workgroups per CU, a multiple of the XCDs
    int64_t nb = (m_tiles * n_tiles + 7) / 8 * 8;
    if (nb > 2 * num_cus()) nb = (2 * num_cus() + 7) / 8 * 8;
    // Tiles taken as workgroups get free where one has more than 72 steps: 33
    // tiles of 6 steps each (128 experts of 4096x1536, 1024 rows each) 565 us
    // against 616, 5 of 16 (32 of 4096x4096, 512 rows) 198 against 205; 8 of 8
    // (8 of 4096x2048, 4096 rows, SwiGLU) 157 against 154, 4 of 6 (128 of
    // 4096x1536, 16 rows) 91 against 87.5, as the counters have to be cleared.
    int32_t* taken = nullptr;
    if (m_tiles * n_tiles * ((K + 255) / 256) > 72 * nb) {
      taken = static_cast<int32_t*>(ws);
      fill_u32(reinterpret_cast<uint32_t*>(taken), 8, 0u, s);
    }
    if (glu)
      mx_launch_big<true>((unsigned)nb, s, p, taken, (int)m_tiles, (int)n_tiles);
    else
      mx_launch_big<false>((unsigned)nb, s, p, taken, (int)m_tiles, (int)n_tiles);
    return check_launch(name);
  }
  // as many tiles of 16 rows as there can be
  const dim3 grid((unsigned)blocks, (unsigned)(M_total / 16 + active));
  if (glu)
    k_mx_few<true><<<grid, 256, 0, s>>>(p);
  else
    k_mx_few<false><<<grid, 256, 0, s>>>(p);
  return check_launch(name);
}

extern "C" {

size_t grouped_mxfp4_gemm_workspace_size(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  (void)E, (void)M_total, (void)N, (void)K;
  return 256;                                           // eight counters
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
