// Gradients of the W4A16 expert product y[p] = W~_e x[p] (asymmetric W4A16
// QAT: bf16 activations times the weights of the shared QDQ path, gist.science
// technical summary §2.2 A): the input gradient, a product with the same NVFP4
// weights contracted over their rows, and the weight gradient, contracted over
// each expert's own rows (the straight-through gradient of the master weight).
#include <type_traits>

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
  const int32_t* prefix;       // dgrad: whole tiles and tails before each expert
  uint16_t* dx;                // dgrad: [M_total][K] bf16
  void* dw;                    // wgrad: [E][N][K] f32 or bf16
  int64_t M_dy, M_x, M_total, N, K;
  int E;
  int dw_bf16, accumulate;
  int nsplit;                  // slices of the contraction
  float* part;                 // dgrad: their float32 parts [nsplit][M_total][K]
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

// ---------------------------------------------------------------------------
// Both gradients: 256x256 outputs per workgroup, eight waves (two rows of
// four) of 128x64 outputs each, bf16 32x32x16 matrix instructions.
//
// An operand whose contraction index is its slow one (both of the weight
// gradient's, the weights of the input gradient) lies in LDS as it does in
// memory, [contraction][256] bf16, and is read through the transposing LDS
// load: a group of 16 lanes reads 4 contraction rows of 16 columns and each
// lane gets its column's four values.  16-byte chunk c of contraction row r
// sits at c ^ swz(r): the four rows of a transposing load then lie in the four
// 64-byte parts of the 256-byte bank line, and 16 rows of one chunk (the order
// in which decoded weights are written) in 16 different 16-byte slots, eight
// rows in eight different ones of a 128-byte half, so neither conflicts.  bf16 operands go from memory to LDS directly; 4-bit
// weights and 8-bit activations are decoded (exactly) on the way, once per
// workgroup.
//
// LDS serves 128 bytes per clock: for 16 contraction rows the waves read 48 KB
// and 16 KB are filled, as many clocks as the matrix instructions take (512),
// so both have to run all the time: fragments are read one slice of 16 ahead
// of their products, in step with the matrix instructions, and the barrier
// that hands over a stage lies one slice before the stage's end.  Products are
// formed transposed (the column operand as matrix rows), so that a lane's four
// consecutive accumulators are four consecutive columns of its output row.
//
// Loads of a wave complete in order, and every step issues the same number of
// them (past the end too, where they return zeros), so a barrier waits until
// at most the loads issued after the wanted stage's are outstanding.
// ---------------------------------------------------------------------------
constexpr int kTile = 256;

// an offset past every buffer: such a load returns zeros, such a store is
// dropped.  (Rows are a multiple of 16 bytes, so a buffer below 4 GiB ends
// there at the latest.)
constexpr uint32_t kPastBuffer = 0xFFFFFFF0u;
constexpr uint64_t kMaxBytes = (1ULL << 32) - 1;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t* lds_tr_ptr;

__device__ __forceinline__ int swz(int r) {
  return ((r & 3) << 2) | ((r >> 1) & 2) | (((r >> 1) ^ (r >> 3)) & 1);
}

// 8 contraction values of one column: two transposing loads of 4 rows each
__device__ __forceinline__ u32x4 tr_frag(const uint8_t* lo, const uint8_t* hi) {
  const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_ptr)lo);
  const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_ptr)hi);
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Fragments of a [contraction][256] tile: lane i of a 16-lane group g reads
// row 8 (g / 2) + 4 h + i / 4 of a 16-row slice, columns 16 (g % 2) + 4 (i %
// 4) .. + 3 of the fragment's 32 (4 chunks); fragment f xors bits 2.. of the
// chunk.
struct TrLane {
  uint32_t off0, off1;
  __device__ __forceinline__ explicit TrLane(int lane) {
    const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    off0 = row * 512 + ((chunk ^ swz(row)) << 4) + (lane & 1) * 8;
    off1 = (row + 4) * 512 + ((chunk ^ swz(row + 4)) << 4) + (lane & 1) * 8;
  }
  __device__ __forceinline__ u32x4 at(const uint8_t* slice, int f) const {
    const uint32_t x = (uint32_t)f << 6;
    return tr_frag(slice + (off0 ^ x), slice + (off1 ^ x));
  }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes,
                                           kBufferRsrcWord3);
}

template <int N>
__device__ __forceinline__ void wait_for() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N < 63 ? N : 63) : "memory");
}

__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  wait_for<N>();
  barrier();
}

// Input gradient, one 32x64 block of a wave: sc * acc to columns k0 .. + 63 of
// rows r0 .. r0 + 31 of a matrix of `rows` rows of K at `out` (bf16, or the
// float32 part of a slice), through 4 KB of the wave's own LDS in 128-byte
// rows.  bf16 rows are stored nontemporally (131072 rows of 1536: 1.51 ->
// 1.50 ms); the parts of slices are read again at once.
template <typename T>
__device__ __forceinline__ void dgrad_out(uint8_t* own, const f32x16_t (&acc)[2], float sc, T* out,
                                          int64_t rows, uint32_t r0, uint32_t k0, uint32_t K) {
  constexpr bool kF32 = sizeof(T) == 4;
  const int lane = threadIdx.x & 63;
  const int kg = lane >> 5, r32 = lane & 31, lr = lane >> 3, lc = lane & 7;
  // (rows past the last lie past the buffer)
  const __amdgpu_buffer_rsrc_t rs = buffer_of(out, (uint64_t)rows * K * sizeof(T));
#pragma unroll
  for (int h = 0; h < (kF32 ? 2 : 1); ++h) {
    if constexpr (kF32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16_t& v = acc[h];
        *reinterpret_cast<f32x4*>(own + r32 * 128 + (((2 * q + kg) ^ (r32 & 7)) << 4)) =
            f32x4{v[4 * q] * sc, v[4 * q + 1] * sc, v[4 * q + 2] * sc, v[4 * q + 3] * sc};
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16_t& v = acc[j];
          *reinterpret_cast<uint2*>(own + r32 * 128 + (((4 * j + q) ^ (r32 & 7)) << 4) + kg * 8) =
              make_uint2(bf16x2_rne(v[4 * q] * sc, v[4 * q + 1] * sc),
                         bf16x2_rne(v[4 * q + 2] * sc, v[4 * q + 3] * sc));
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t r = 8 * q + lr;
      const u32x4 v = *reinterpret_cast<const u32x4*>(own + r * 128 + ((lc ^ (r & 7)) << 4));
      const uint32_t k = k0 + 32 * h + lc * (16 / sizeof(T));
      __builtin_amdgcn_raw_buffer_store_b128(
          v, rs, k < K ? ((r0 + r) * K + k) * (uint32_t)sizeof(T) : kPastBuffer, 0, kF32 ? 0 : 2);
    }
  }
}

// ---------------------------------------------------------------------------
// Input gradient.  Output rows are the experts' rows, columns k, contraction
// n, 64 at a time: dy as [256][64] in a ring of three LDS stages, filled three
// steps ahead (16-byte fragment reads, chunk c of row r at c ^ ((r >> 1) & 7)),
// the weights as [64][256] in two, decoded one step ahead from registers
// loaded two steps earlier.  Where the tiles fill less than the chip the
// contraction is split: each slice writes its float32 part (times g_w), and
// k_dgrad_join adds them.
//
// An expert's last 128 rows or fewer are a tail, multiplied with 64 (32 if at
// most 64) rows per wave and loading only the rows of dy that those read: it
// costs its weights' decode, not a full tile's products (2048 rows over 128
// experts 275 -> 207 us; 64 rows for each of 128 experts of 1536x2048, without
// the loads of rows that are not there, 124 -> 98 us); 129 to 192 rows likewise
// take 96 per wave (160 rows each: 169 -> 147 us).  Tails follow all whole
// tiles, so that every XCD has its share of both and the cheaper ones end the
// launch; an expert's weights are then read a second time, which costs less
// (32768 skewed rows 0.280 -> 0.261 ms, 16384 rows over 128 experts of
// 4096x1536 0.357 -> 0.308 ms).
//
// Measured: 131072 rows, 128 experts of 4096x1536, 1.43 to 1.48 ms = 1.13 PFLOP/s
// (1.50 on a slower card); 32768 rows, 128 experts of 1536x2048 (half the
// experts a tile and a tail), 0.25 ms.  Counters at the first: matrix units 60%
// busy, waves waiting for LDS 13% of their time, clock 1.84 GHz; operands of
// zeros take the same cycles at 2.38 GHz, 1.15 ms.  So the chip's power limit,
// then LDS and the weights' decode beside the products.  An earlier form of
// 1.53 ms was slower as one persistent workgroup per CU (1.57 ms, and 0.31
// against 0.28 on the second).
// ---------------------------------------------------------------------------
namespace dg {
constexpr int BC = 64;
constexpr int A_BYTES = kTile * BC * 2, B_BYTES = BC * kTile * 2;   // 32768 each
}  // namespace dg

// An expert's rows are whole tiles and, where 1 to 128 rows are left, a tail:
// prefix[e], prefix[E + 1 + e] = whole tiles and tails of the experts before e.
constexpr int kTail = 128;

__global__ void __launch_bounds__(1024)
k_dgrad_tiles(GradArgs p, int32_t* __restrict__ prefix) {
  __shared__ uint64_t wsum[16];
  const int tid = threadIdx.x, lane = tid & 63;
  uint64_t v = 0;   // whole tiles below, tails above
  if (tid < p.E) {
    int64_t lo, hi;
    expert_rows(p, tid, lo, hi);
    const int64_t left = (hi - lo) % kTile;
    v = (uint64_t)((hi - lo) / kTile + (left > kTail)) |
        (uint64_t)(left > 0 && left <= kTail) << 32;
  }
  uint64_t incl = v;
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) wsum[tid >> 6] = incl;
  __syncthreads();
  for (int w = 0; w < (tid >> 6); ++w) incl += wsum[w];
  if (tid >= p.E) return;
  const uint64_t before = incl - v;
  prefix[tid] = (int32_t)before;
  prefix[p.E + 1 + tid] = (int32_t)(before >> 32);
  if (tid == p.E - 1) {
    prefix[p.E] = (int32_t)incl;
    prefix[2 * p.E + 1] = (int32_t)(incl >> 32);
  }
}

__global__ void __launch_bounds__(512, 1)
k_dgrad(GradArgs p, int n_tiles) {
  using namespace dg;
  // separate objects, and the rings unrolled: each access names its stage, so
  // a fill in flight is not waited for before reads of another
  __shared__ __attribute__((aligned(16))) uint8_t sa0[A_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t sa1[A_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t sa2[A_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t sb0[B_BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t sb1[B_BYTES];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int kg = lane >> 5, r32 = lane & 31;
  uint8_t* const sa[3] = {sa0, sa1, sa2};
  uint8_t* const sb[2] = {sb0, sb1};

  // tile: whole row tiles first, then tails; of each, row tile by row tile, a
  // contiguous range of that order per XCD (workgroup b runs on XCD b % 8, each
  // with its own L2).  (Column tiles over groups of 2, 4 or 8 row tiles: 0.2%,
  // 1% and 1% slower at 131072 rows of 128 experts of 4096x1536, up to 2% either
  // way elsewhere.)
  int e, nt;
  int64_t lo, hi, a0;
  {
    const int n_whole = p.prefix[p.E] * n_tiles, n_tail = p.prefix[2 * p.E + 1] * n_tiles;
    const int per_whole = (n_whole + 7) / 8, per_tail = (n_tail + 7) / 8;
    int i = (int)blockIdx.x >> 3;
    const bool tail = i >= per_whole;
    if (tail) i -= per_whole;
    if (i >= (tail ? per_tail : per_whole)) return;
    const int v = ((int)blockIdx.x & 7) * (tail ? per_tail : per_whole) + i;
    if (v >= (tail ? n_tail : n_whole)) return;
    const int gt = v / n_tiles;
    nt = v - gt * n_tiles;
    const int32_t* const prefix = p.prefix + (tail ? p.E + 1 : 0);
    // the last expert whose first tile is at or before gt: 64 at a time
    int n = 0;
    for (int j = 0; j < p.E; j += 64)
      n += __builtin_popcountll(__ballot(j + lane < p.E && prefix[j + lane] <= gt));
    e = __builtin_amdgcn_readfirstlane(n - 1);
    expert_rows(p, e, lo, hi);
    a0 = lo + (tail ? (hi - lo) / kTile : gt - prefix[e]) * kTile;
  }
  const int64_t b0 = (int64_t)nt * kTile;
  // this slice's steps (all of them without a split)
  const int all = (int)((p.N + BC - 1) / BC);
  const int per = (all + p.nsplit - 1) / p.nsplit;
  const int u0 = (int)blockIdx.y * per, u1 = u0 + per < all ? u0 + per : all;

  // ---- loads -------------------------------------------------------------
  const uint32_t N2 = (uint32_t)(p.N * 2);
  const __amdgpu_buffer_rsrc_t rs_a = buffer_of(p.dy, (uint64_t)p.M_dy * N2);
  // of the 32 1-KB pieces (8 rows) of a dy stage, piece 8 i + wave; the lane
  // takes chunk a_c of row 64 i + 8 wave + lane / 8
  const uint32_t a_c = (uint32_t)((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
  uint32_t off_a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t pr = a0 + 64 * i + 8 * wave + (lane >> 3);
    off_a[i] = pr < hi ? (uint32_t)source_row(p.dy_rows, pr, p.M_dy) * N2 + 16u * a_c : kPastBuffer;
  }
  const __amdgpu_buffer_rsrc_t rs_w =
      buffer_of(p.w_codes + e * packed_codes_per_expert(p.N, p.K), (uint64_t)p.N * p.K / 2);
  const __amdgpu_buffer_rsrc_t rs_s =
      buffer_of(p.w_scales + e * packed_scales_per_expert(p.N, p.K), (uint64_t)p.N * p.K / 16);
  // weights: wave w takes the step's code tiles 2 w, 2 w + 1 (of 4 row blocks
  // x 4 column tiles), a lane one row's half tile: 16 bytes = 32 columns
  const int w_rb = (2 * wave + kg) >> 2, w_ct = (2 * wave + kg) & 3;
  const int w_half = (lane >> 4) & 1, w_row = lane & 15;
  const uint32_t k_tiles = (uint32_t)(p.K >> 6);
  const uint32_t kt = (uint32_t)(b0 >> 6) + w_ct;   // columns past K are never stored
  const uint32_t w_tile = w_rb * k_tiles + (kt < k_tiles ? kt : k_tiles - 1);
  const uint32_t off_w = w_tile * 512 + w_half * 256 + w_row * 16;
  const uint32_t off_ws = w_tile * 64 + w_row * 4 + w_half * 2;
  const uint32_t w_step = 4 * k_tiles * 512;
  u32x4 wcodes[2];
  uint32_t wscales[2];
  // (rows of the weights past N lie past the buffer)
  auto issue_w = [&](int set, int u) __attribute__((always_inline)) {
    const bool there = u < u1;
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs_w, there ? off_w : kPastBuffer,
                                                         there ? (uint32_t)u * w_step : 0, 0);
    wcodes[set] = u32x4{v[0], v[1], v[2], v[3]};
    wscales[set] = __builtin_amdgcn_raw_buffer_load_b16(
        rs_s, there ? off_ws : kPastBuffer, there ? (uint32_t)u * (w_step >> 3) : 0, 0);
  };
  using c0 = std::integral_constant<int, 0>;
  using c1 = std::integral_constant<int, 1>;
  using c2 = std::integral_constant<int, 2>;
  using c3 = std::integral_constant<int, 3>;
  using c4 = std::integral_constant<int, 4>;
  // (the first 64 NV rows of a stage: the waves read no others)
  auto issue_a = [&](uint8_t* st, int u, auto nv_c) __attribute__((always_inline)) {
    const bool there = u < u1 && (uint32_t)u * BC + 8 * a_c < (uint32_t)p.N;
    const uint32_t so = u < u1 ? (uint32_t)u * (2 * BC) : 0;
#pragma unroll
    for (int i = 0; i < decltype(nv_c)::value; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(st + (i * 8 + wave) * 1024), 16,
                                               there ? off_a[i] : kPastBuffer, so, 0, 0);
  };
  // chunk j (8 columns) of the lane's 32 into the weight stage
  const uint32_t f_row = 16 * w_rb + w_row, f_chunk = 8 * w_ct + 4 * w_half;
  auto fill = [&](uint8_t* st, int set, int j) __attribute__((always_inline)) {
    const float s = e4m3_decode(j < 2 ? wscales[set] & 0xFFu : wscales[set] >> 8);
    *reinterpret_cast<u32x4*>(st + f_row * 512 + (((f_chunk + j) ^ swz(w_row)) << 4)) =
        decode8_bf16(wcodes[set][j], s);
  };

  // ---- products ----------------------------------------------------------
  const TrLane tr(lane);
  const int a_sw = (r32 >> 1) & 7;
  issue_w(0, u0);
  issue_a(sa0, u0, c4{});
  issue_w(1, u0 + 1);
  issue_a(sa1, u0 + 1, c4{});
#pragma unroll
  for (int j = 0; j < 4; ++j) fill(sb0, 0, j);
  issue_w(0, u0 + 2);
  issue_a(sa2, u0 + 2, c4{});
  wait_and_barrier<12>();
  // the tile with NV 32-row blocks per row of waves; whole, so that no
  // accumulator is merged between variants
  auto whole = [&](auto nv_c) __attribute__((always_inline)) {
    constexpr int NV = decltype(nv_c)::value;
    f32x16_t acc[NV][2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const uint32_t a_row = (wm * 32 * NV + r32) * 128;
    u32x4 fa[2][NV], fb[2][2];   // by slice % 2
    auto read = [&](const uint8_t* a, const uint8_t* b, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[s & 1][j] = tr.at(b + s * 8192, 2 * wn + j);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        fa[s & 1][i] = *reinterpret_cast<const u32x4*>(a + a_row + 32 * i * 128 +
                                                       (((2 * s + kg) ^ a_sw) << 4));
    };
    auto multiply = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32_bf16(fb[s & 1][j], fa[s & 1][i], acc[i][j]);
      // a matrix instruction, then LDS reads, vector instructions, a load
#pragma unroll
      for (int i = 0; i < 2 * NV; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, NV == 4 ? 1 : NV == 2 ? 2 : 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x006, NV == 4 ? 5 : 10, 0);
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
      }
    };
    // step u: dy stage AU, weight stage BU
    auto step = [&](auto au_c, auto bu_c, int u) __attribute__((always_inline)) {
      constexpr int AU = decltype(au_c)::value, BU = decltype(bu_c)::value;
      read(sa[AU], sb[BU], 1);
      fill(sb[BU ^ 1], BU ^ 1, 0);
      fill(sb[BU ^ 1], BU ^ 1, 1);
      multiply(0);
      read(sa[AU], sb[BU], 2);
      fill(sb[BU ^ 1], BU ^ 1, 2);
      multiply(1);
      read(sa[AU], sb[BU], 3);
      fill(sb[BU ^ 1], BU ^ 1, 3);
      multiply(2);
      wait_and_barrier<2 + NV>();
      issue_w(BU ^ 1, u + 3);
      issue_a(sa[AU], u + 3, nv_c);
      read(sa[(AU + 1) % 3], sb[BU ^ 1], 0);
      multiply(3);
    };
    read(sa0, sb0, 0);
    for (int u = u0; u < u1;) {
      step(c0{}, c0{}, u);
      if (++u >= u1) break;
      step(c1{}, c1{}, u);
      if (++u >= u1) break;
      step(c2{}, c0{}, u);
      if (++u >= u1) break;
      step(c0{}, c1{}, u);
      if (++u >= u1) break;
      step(c1{}, c0{}, u);
      if (++u >= u1) break;
      step(c2{}, c1{}, u);
      if (++u >= u1) break;
    }
    wait_and_barrier<0>();

    const float sc = p.g_w[e];
    const int64_t rows = hi - a0 < kTile ? hi - a0 : kTile;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t r0 = 32 * (NV * wm + i), k0 = (uint32_t)b0 + 64 * wn;
      if (p.nsplit == 1)
        dgrad_out(sa0 + wave * 4096, acc[i], sc, p.dx + a0 * p.K, rows, r0, k0, (uint32_t)p.K);
      else
        dgrad_out(sa0 + wave * 4096, acc[i], sc,
                  p.part + ((int64_t)blockIdx.y * p.M_total + a0) * p.K, rows, r0, k0,
                  (uint32_t)p.K);
    }
  };
  const int nv = hi - a0 > 192 ? 4 : (int)(hi - a0 + 63) / 64;
  if (nv == 4) { whole(c4{}); return; }
  if (nv == 3) { whole(c3{}); return; }
  if (nv == 2) { whole(c2{}); return; }
  whole(c1{});
}

// ---------------------------------------------------------------------------
// Input gradient for few rows per expert: the weights' bytes bound it, so each
// wave streams a strip of 64 columns over its range of n by itself, without a
// barrier: the codes of 64 rows x 64 columns go from memory to registers two
// steps ahead, are decoded into the wave's own 8 KB of LDS and read back
// through the transposing load; dy's fragments come from memory (the four
// waves of a workgroup, four strips of one expert, share them in L1).  32 rows
// of the expert per pass; more re-stream the weights.
//
// Measured: 2048 rows over 128 experts of 4096x1536, evenly routed (26 rows in
// the longest expert), 115 us = 4.0 TB/s of weights (161 us tile by tile); one
// row of one such expert 20 us.  Bound by its vector instructions (two per
// decoded weight, 16 per 8) and their issue, with three waves per SIMD; with up
// to 64 rows per pass and two waves per SIMD 146 us.  The passes of an expert
// follow one another, about 55 us each there, so uneven routing costs: 216 us
// with 94 rows in the longest expert, 444 with 171, 1.9 ms with half of all
// rows in one, 3.6 with all.
// ---------------------------------------------------------------------------
namespace dgf {
constexpr int BC = 64;
}  // namespace dgf

__global__ void __launch_bounds__(256, 3)
k_dgrad_few(GradArgs p, int groups) {
  using namespace dgf;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * 8192];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = lane >> 5, r32 = lane & 31;
  uint8_t* const own = lds + wave * 8192;

  int b = (int)blockIdx.x;
  const int slice = b % p.nsplit;
  b /= p.nsplit;
  const int e = b / groups;
  const uint32_t k0 = (uint32_t)((b - e * groups) * 4 + wave) * 64;
  const uint32_t K = (uint32_t)p.K, N = (uint32_t)p.N;
  if (k0 >= K) return;
  int64_t lo, hi;
  expert_rows(p, e, lo, hi);
  if (lo >= hi) return;
  // this slice's steps
  const int all = (int)((p.N + BC - 1) / BC);
  const int per = (all + p.nsplit - 1) / p.nsplit;
  const int u0 = slice * per < all ? slice * per : all;
  const int u1 = u0 + per < all ? u0 + per : all;

  const uint32_t N2 = N * 2;
  const __amdgpu_buffer_rsrc_t rs_a = buffer_of(p.dy, (uint64_t)p.M_dy * N2);
  const __amdgpu_buffer_rsrc_t rs_w =
      buffer_of(p.w_codes + e * packed_codes_per_expert(p.N, p.K), (uint64_t)p.N * p.K / 2);
  const __amdgpu_buffer_rsrc_t rs_s =
      buffer_of(p.w_scales + e * packed_scales_per_expert(p.N, p.K), (uint64_t)p.N * p.K / 16);
  // load i of two: row block 2 i + kg of the step's four, one row's half tile
  const int w_half = (lane >> 4) & 1, w_row = lane & 15;
  const uint32_t k_tiles = K >> 6;
  const uint32_t w_step = 4 * k_tiles * 512;
  uint32_t off_w[2], off_ws[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t tile = (2 * i + kg) * k_tiles + (k0 >> 6);
    off_w[i] = tile * 512 + w_half * 256 + w_row * 16;
    off_ws[i] = tile * 64 + w_row * 4 + w_half * 2;
  }
  u32x4 wcodes[2][2];
  uint32_t wscales[2][2];
  // nontemporal: each code byte is read once (a line of scales serves two
  // strips)
  auto load_w = [&](int set, int u) __attribute__((always_inline)) {
    const uint32_t so = u < u1 ? (uint32_t)u * w_step : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto v =
          __builtin_amdgcn_raw_buffer_load_b128(rs_w, u < u1 ? off_w[i] : kPastBuffer, so, 2);
      wcodes[set][i] = u32x4{v[0], v[1], v[2], v[3]};
      wscales[set][i] = __builtin_amdgcn_raw_buffer_load_b16(
          rs_s, u < u1 ? off_ws[i] : kPastBuffer, so >> 3, 0);
    }
  };
  // the wave's [64][64] tile: 128-byte rows, chunk c of row r at c ^ wz(r):
  // four rows of a transposing load in four 64-byte bank parts, 16 rows of one
  // chunk (a write) in 16 slots
  auto wz = [](int r) __attribute__((always_inline)) {
    return ((r & 2) << 1) | ((r >> 1) & 2) | ((r ^ (r >> 3)) & 1);
  };
  auto fill = [&](int set) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s0 = e4m3_decode(wscales[set][i] & 0xFFu), s1 = e4m3_decode(wscales[set][i] >> 8);
      const int r = 16 * (2 * i + kg) + w_row;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<u32x4*>(own + r * 128 + (((4 * w_half + j) ^ wz(w_row)) << 4)) =
            decode8_bf16(wcodes[set][i][j], j < 2 ? s0 : s1);
    }
  };
  const int t_row = 8 * kg + ((lane & 15) >> 2);
  const int t_chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  const uint32_t t_off0 = t_row * 128 + ((t_chunk ^ wz(t_row)) << 4) + (lane & 1) * 8;
  const uint32_t t_off1 = (t_row + 4) * 128 + ((t_chunk ^ wz(t_row + 4)) << 4) + (lane & 1) * 8;
  const float sc = p.g_w[e];

  for (int64_t r0 = lo + 32 * (int64_t)blockIdx.y; r0 < hi; r0 += 32 * (int64_t)gridDim.y) {
    const int64_t pr = r0 + r32;
    const uint32_t off_a =
        pr < hi ? (uint32_t)source_row(p.dy_rows, pr, p.M_dy) * N2 + 16u * kg : kPastBuffer;
    f32x16_t acc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
    u32x4 fa[2][4];
    auto load_a = [&](int set, int u) __attribute__((always_inline)) {
      const uint32_t so = u < u1 ? (uint32_t)u * (2 * BC) : 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool there = u < u1 && (uint32_t)u * BC + 16 * s < N && off_a != kPastBuffer;
        const auto v =
            __builtin_amdgcn_raw_buffer_load_b128(rs_a, there ? off_a + 32 * s : kPastBuffer, so, 0);
        fa[set][s] = u32x4{v[0], v[1], v[2], v[3]};
      }
    };
    auto step = [&](auto set_c, int u) __attribute__((always_inline)) {
      constexpr int SET = decltype(set_c)::value;
      fill(SET);
      load_a(SET ^ 1, u + 1);
      load_w(SET, u + 2);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[j] = mfma32_bf16(tr_frag(own + s * 2048 + (t_off0 ^ (j << 6)),
                                       own + s * 2048 + (t_off1 ^ (j << 6))),
                               fa[SET][s], acc[j]);
    };
    load_a(0, u0);
    load_w(0, u0);
    load_w(1, u0 + 1);
    for (int u = u0; u < u1; u += 2) {
      step(std::integral_constant<int, 0>{}, u);
      if (u + 1 < u1) step(std::integral_constant<int, 1>{}, u + 1);
    }
    const int64_t rows = hi - r0 < 32 ? hi - r0 : 32;
    if (p.nsplit == 1)
      dgrad_out(own, acc, sc, p.dx + r0 * p.K, rows, 0, k0, K);
    else
      dgrad_out(own, acc, sc, p.part + ((int64_t)slice * p.M_total + r0) * p.K, rows, 0, k0, K);
  }
}

// Sum over the slices of four elements at q of parts of n each: G groups of
// 256 / G lanes take a G-th of the slices each, and their sums are added in
// order.  Group 0 gets the sum.  (One group over 64 slices of 5120 elements:
// 40 us, as its loads wait for one another.)
template <int G>
__device__ __forceinline__ f32x4 slice_sum(const float* __restrict__ part, int64_t q, int64_t n,
                                           int nsplit, bool there) {
  const int g = threadIdx.x / (256 / G), lane = threadIdx.x % (256 / G);
  const int per = (nsplit + G - 1) / G;
  const int end = (g + 1) * per < nsplit ? (g + 1) * per : nsplit;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (there) {
#pragma unroll 4
    for (int i = g * per; i < end; ++i) s += *reinterpret_cast<const f32x4*>(part + i * n + q);
  }
  if constexpr (G > 1) {
    __shared__ f32x4 sums[G][256 / G];
    sums[g][lane] = s;
    __syncthreads();
    s = sums[0][lane];
#pragma unroll
    for (int i = 1; i < G; ++i) s += sums[i][lane];
    __syncthreads();
  }
  return s;
}

// dx = sum of the slices' parts over the experts' rows; four columns per lane
template <int G>
__global__ void __launch_bounds__(256)
k_dgrad_join(const float* __restrict__ part, const int32_t* __restrict__ offsets, int E,
             int64_t M_total, int64_t K, int nsplit, uint16_t* __restrict__ dx) {
  constexpr int L = 256 / G;
  int64_t lo = offsets[0], hi = offsets[E];
  lo = lo < 0 ? 0 : lo;
  hi = (hi > M_total ? M_total : hi) * K;
  for (int64_t q0 = lo * K + blockIdx.x * (4LL * L); q0 < hi; q0 += gridDim.x * (4LL * L)) {
    const int64_t q = q0 + (threadIdx.x % L) * 4;
    const f32x4 s = slice_sum<G>(part, q, M_total * K, nsplit, q < hi);
    if (threadIdx.x < L && q < hi)
      *reinterpret_cast<uint2*>(dx + q) = make_uint2(bf16x2_rne(s.x, s.y), bf16x2_rne(s.z, s.w));
  }
}

// ---------------------------------------------------------------------------
// Weight gradient.  One workgroup per CU takes 256x256 output tiles (item:
// slice of the rows, expert, row tile, column tile) one after another, and the
// loads run on across them: contraction steps of 32 rows go through a ring of
// four LDS stages, filled three steps ahead, and a tile's outputs are stored
// while the next tile's first stages are in flight.  (A workgroup per tile
// waited for its first stage, and for its stores, once per tile: a tile of
// 1024 rows spent a third of its time there, one of 256 rows half.)
//
// Waits: stores complete in order with the loads, so the barrier of step
// s waits until at most the operations issued after stage s + 1's last fill
// are outstanding (two steps of kOps, plus the stores where a tile ended in
// between); each step issues the same number, past the last row too, where
// they return zeros, and an edge tile's stores are issued with an offset past
// the buffer.  Row lists are read two steps before the fill that uses them,
// 8-bit codes four steps before their stage and decoded two steps later.
// ---------------------------------------------------------------------------
namespace wg {
constexpr int BC = 32;
constexpr int A_BYTES = BC * kTile * 2;
constexpr int STAGE = 2 * A_BYTES;             // 32768
constexpr int OUT = 4096;                      // output staging of one wave
}  // namespace wg

// A contraction step's rows [p, hi) and its tile's first output row and column
struct WgStep {
  uint32_t p, hi, a0, b0;
};

// Measured: 131072 rows, 128 experts of 4096x1536, bf16 dw, 1.51 to 1.55 ms =
// 1.07 PFLOP/s.  Counters: matrix units 64% busy at 1.68 GHz; operands of zeros
// take 10% more cycles at 2.38 GHz, 1.18 ms: bound by the chip's power limit at
// real operands, then by waits.  There with float32 dw 1.71 to 1.73 ms, added to
// 2.14 to 2.17; 8-bit x the same within 3%.  32768 rows from 8-bit x, 128
// experts of 1536x2048, float32 dw (1.6 GB), 0.48 ms with new inputs each time
// (0.34 where they fit the Infinity Cache), added to 0.64: bound by the stores
// (5.5 TB/s with nothing else running) and operands that come from memory
// beside them.
// MX: x is an 8-bit checkpoint.  LA, LB: dy, x are gathered through a row list
// (without one a row is its step's own, and no per-row arithmetic is left).
template <bool MX, bool LA, bool LB>
__global__ void __launch_bounds__(512, 1)
k_wgrad(GradArgs p, int n_tiles, int m_tiles) {
  using namespace wg;
  // separate objects, and the ring unrolled by four: each access names its
  // stage, so a fill in flight is not waited for before reads of another
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st2[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st3[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t outb[8 * OUT];
  constexpr int kOps = (MX ? 6 : 4) + (LA ? 2 : 0) + (LB ? 2 : 0);
  constexpr int kStores = 16;   // of a bf16 tile; a float32 one has twice as many

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int kg = lane >> 5, r32 = lane & 31;
  uint8_t* const stage[4] = {st0, st1, st2, st3};

  // ---- items -------------------------------------------------------------
  // expert by expert, tile by tile, slice by slice
  const int per_tile = p.nsplit;
  const int per_e = n_tiles * m_tiles * per_tile;
  // Each XCD (workgroup b runs on XCD b % 8, each with its own L2) takes a
  // contiguous range of the items, so that its workgroups share operands in
  // L2, cut where an eighth of the work lies before it: an item costs its
  // expert's steps (of the slice) and its stores.  (Runs of 32 items dealt to
  // the XCDs in turn: 514 us against 492, 32768 rows over 128 experts, most
  // of them with 50 to 1400 rows, 1536x2048 float32.)
  int first, last;
  {
    int* const wsum = reinterpret_cast<int*>(outb);   // eight waves' sums, two cuts
    int mine[2], at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ex = 2 * tid + i;
      int64_t lo = 0, hi = 0;
      if (ex < p.E) expert_rows(p, ex, lo, hi);
      const int steps = (int)((hi - lo + BC - 1) / BC);
      mine[i] = ex < p.E ? (steps + p.nsplit - 1) / p.nsplit + (p.dw_bf16 ? 6 : 11) : 0;
    }
    int sum = mine[0] + mine[1];
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < 8; ++w) {
      const int u = wsum[w];
      if (w < wave) sum += u;
      all += u;
    }
    at[0] = sum - mine[0] - mine[1];
    at[1] = sum - mine[1];
    // the expert that holds the cut writes the cut's item
    const int x = (int)blockIdx.x & 7;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t cut = (int64_t)all * (x + c) / 8;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (mine[i] > 0 && cut >= at[i] && cut < at[i] + mine[i])
          wsum[8 + c] = (2 * tid + i) * per_e + (int)((cut - at[i]) * per_e / mine[i]);
    }
    if (tid == 0 && x == 7) wsum[9] = p.E * per_e;
    __syncthreads();
    first = __builtin_amdgcn_readfirstlane(wsum[8]);
    last = __builtin_amdgcn_readfirstlane(wsum[9]);
    __syncthreads();
  }
  const int loc = (int)blockIdx.x >> 3, per_xcd = (int)gridDim.x >> 3;
  // the workgroup's i-th item
  auto item_at = [&](int i) __attribute__((always_inline)) { return first + loc + i * per_xcd; };
  struct Item {
    uint32_t lo, hi, a0, b0;
    int e, slice, steps;
  };
  auto item_of = [&](int v) __attribute__((always_inline)) {
    Item t;
    t.e = v / per_e;
    v -= t.e * per_e;
    t.slice = v % per_tile;
    v /= per_tile;
    const int m = v / n_tiles;
    t.a0 = (uint32_t)m * kTile;
    t.b0 = (uint32_t)(v - m * n_tiles) * kTile;
    // scalar loads: the offsets do not change, and a vector load here would
    // wait for every fill in flight
    const __attribute__((address_space(4))) int32_t* off =
        (const __attribute__((address_space(4))) int32_t*)p.offsets;
    const int most = (int)p.M_total;
    int lo = off[t.e], hi = off[t.e + 1];
    lo = lo < 0 ? 0 : (lo > most ? most : lo);
    hi = hi < lo ? lo : (hi > most ? most : hi);
    if (p.nsplit > 1) {   // whole steps per slice
      const int per = ((hi - lo + BC - 1) / BC + p.nsplit - 1) / p.nsplit * BC;
      lo = lo + per * t.slice < hi ? lo + per * t.slice : hi;
      hi = lo + per < hi ? lo + per : hi;
    }
    t.lo = (uint32_t)lo;
    t.hi = (uint32_t)hi;
    // a tile's steps are rounded up to two; an added one loads and multiplies
    // zeros (a tile that may end after any step has branches in each, across
    // which instructions are not scheduled: 7% slower per step; rounding to
    // the ring's four adds 1.5 steps to an average tile)
    t.steps = (hi - lo + 2 * BC - 1) / (2 * BC) * 2;
    return t;
  };

  // ---- loads -------------------------------------------------------------
  // the step that the row lists are next read for
  int ahead_i = -1, ahead_s = 0;
  Item ahead;
  ahead.lo = ahead.hi = ahead.a0 = ahead.b0 = 0;
  ahead.steps = 0;
  auto next_step = [&](bool maybe_new) __attribute__((always_inline)) {
    ++ahead_s;
    while (maybe_new && ahead_s >= ahead.steps) {
      ahead_s = 0;
      const int v = item_at(++ahead_i);
      if (v >= last) {   // none left: rows that are not there
        ahead.lo = ahead.hi = 0;
        ahead.steps = 1 << 30;
      } else {
        ahead = item_of(v);
      }
    }
    return WgStep{ahead.lo + (uint32_t)ahead_s * BC, ahead.hi, ahead.a0, ahead.b0};
  };
  const uint32_t pitch_a = (uint32_t)(p.N * 2), pitch_b = (uint32_t)(p.K * (MX ? 1 : 2));
  // of the two 1-KB pieces (two rows) of a [32][256] tile that a wave fills,
  // piece i is rows 16 i + r16; the lane's slot in the row is lane % 32, which
  // holds chunk r32 ^ swz(row), columns col8 .. + 7
  const uint32_t r16 = 2 * wave + kg;
  const uint32_t col8 = 8u * (uint32_t)(r32 ^ swz(r16));
  constexpr uint32_t kBytesB = MX ? 1 : 2;
  const uint32_t at_a = r16 * pitch_a + col8 * 2, at_b = r16 * pitch_b + col8 * kBytesB;
  WgStep ring[4];                    // descriptors, row-list entries and codes by step % 4
  uint32_t ids_a[4][2], ids_b[4][2];
  uint32_t codes[4][2][2], scales[4][2];

  auto load_ids = [&](int u, const WgStep& d) __attribute__((always_inline)) {
    ring[u] = d;
    const uint64_t n = (uint64_t)p.M_total * 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t o = r16 * 4 + (d.p + 16 * i) * 4;
      if constexpr (LA)
        ids_a[u][i] = __builtin_amdgcn_raw_buffer_load_b32(buffer_of(p.dy_rows, n), o, 0, 0);
      if constexpr (LB)
        ids_b[u][i] = __builtin_amdgcn_raw_buffer_load_b32(buffer_of(p.x_rows, n), o, 0, 0);
    }
  };
  // Byte offset of the lane's chunk of row 16 i + r16, past the buffer for
  // rows and columns that are not there.
  auto chunk_at = [&](auto listed_c, uint32_t id, int i, const WgStep& d, uint32_t c0,
                      uint32_t cols, uint32_t rows, uint32_t pitch, uint32_t bytes,
                      uint32_t at) __attribute__((always_inline)) {
    const bool there = (r16 + 16 * i < d.hi - d.p) & (d.p < d.hi) & (col8 < cols - c0);
    uint32_t o;
    if constexpr (decltype(listed_c)::value)
      o = (id < rows ? id : rows - 1) * pitch + (col8 + c0) * bytes;
    else
      o = at + ((d.p + 16 * i) * pitch + c0 * bytes);
    return there ? o : kPastBuffer;
  };
  auto issue = [&](uint8_t* st, int u) __attribute__((always_inline)) {
    const WgStep d = ring[u];
    const __amdgpu_buffer_rsrc_t rs_a = buffer_of(p.dy, (uint64_t)p.M_dy * pitch_a);
    const __amdgpu_buffer_rsrc_t rs_b = buffer_of(p.x, (uint64_t)p.M_x * pitch_b);
    uint32_t oa[2], ob[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      oa[i] = chunk_at(std::integral_constant<bool, LA>{}, ids_a[u][i], i, d, d.a0, (uint32_t)p.N,
                       (uint32_t)p.M_dy, pitch_a, 2, at_a);
      ob[i] = chunk_at(std::integral_constant<bool, LB>{}, ids_b[u][i], i, d, d.b0, (uint32_t)p.K,
                       (uint32_t)p.M_x, pitch_b, kBytesB, at_b);
    }
    if constexpr (MX) {
      const __amdgpu_buffer_rsrc_t rs_s =
          buffer_of(p.x_scales, (uint64_t)p.M_x * (uint64_t)p.K / 32);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs_b, ob[i], 0, 0);
        codes[u][i][0] = v[0];
        codes[u][i][1] = v[1];
        scales[u][i] = __builtin_amdgcn_raw_buffer_load_b8(
            rs_s, ob[i] == kPastBuffer ? kPastBuffer : ob[i] >> 5, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint8_t* dst = st + (i * 8 + wave) * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(dst), 16, oa[i], 0, 0, 0);
      if constexpr (!MX)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, lds_ptr(dst + A_BYTES), 16, ob[i], 0, 0, 0);
    }
  };
  auto fill = [&](uint8_t* st, int u) __attribute__((always_inline)) {
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<u32x4*>(st + A_BYTES + (i * 8 + wave) * 1024 + lane * 16) =
            mx_decode8(make_uint2(codes[u][i][0], codes[u][i][1]), mx_scale(scales[u][i]));
    }
  };

  // ---- products ----------------------------------------------------------
  f32x16_t acc[4][2];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  };
  const TrLane tr(lane);
  u32x4 fa[2][4], fb[2][2];   // by half of the step
  auto read = [&](const uint8_t* st, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[half][j] = tr.at(st + A_BYTES + half * 8192, 2 * wn + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) fa[half][i] = tr.at(st + half * 8192, 4 * wm + i);
  };
  auto multiply = [&](int half) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma32_bf16(fb[half][j], fa[half][i], acc[i][j]);
    // a matrix instruction, then up to three LDS reads, four others, one load
    // (two and five: 3% slower)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
      __builtin_amdgcn_sched_group_barrier(0x006, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
  };

  // ---- outputs: through the wave's own LDS part, 128-byte rows ------------
  uint8_t* const ob = outb + wave * OUT;
  auto store = [&](const Item& t) __attribute__((always_inline)) {
    const int64_t nk = p.N * p.K;
    const uint32_t K = (uint32_t)p.K, N = (uint32_t)p.N;
    const int lr = lane >> 3, lc = lane & 7;
    // rows n0 + 8 q + lr, 16-byte chunk lc of the 128-byte piece at column k0
    auto rows_out = [&](const __amdgpu_buffer_rsrc_t& rs_o, uint32_t n0, uint32_t k0,
                        uint32_t bytes) __attribute__((always_inline)) {
      auto at = [&](int q) __attribute__((always_inline)) {
        const uint32_t n = n0 + 8 * q + lr, k = k0 + lc * (16 / bytes);
        return n < N && k < K ? (n * K + k) * bytes : kPastBuffer;
      };
      auto mine = [&](int q) __attribute__((always_inline)) {
        const int r = 8 * q + lr;
        return *reinterpret_cast<const u32x4*>(ob + r * 128 + ((lc ^ (r & 7)) << 4));
      };
      // nontemporal stores: dw is not read back soon, and its lines leave L2 to
      // the operands (wgrad of 32768 rows, 128 experts of 1536x2048: 0.52 ->
      // 0.37 ms)
      if (bytes == 4 && p.accumulate) {
        // all four loads before the first store, which none of them would be
        // moved across: 0.83 -> 0.65 ms there (a block further ahead spills)
        u32x4 was[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const auto w = __builtin_amdgcn_raw_buffer_load_b128(rs_o, at(q), 0, 0);
          was[q] = u32x4{w[0], w[1], w[2], w[3]};
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u32x4 v = mine(q);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[c] = __float_as_uint(__uint_as_float(v[c]) + __uint_as_float(was[q][c]));
          __builtin_amdgcn_raw_buffer_store_b128(v, rs_o, at(q), 0, 2);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          __builtin_amdgcn_raw_buffer_store_b128(mine(q), rs_o, at(q), 0, 2);
      }
    };
    if (p.dw_bf16) {
      const __amdgpu_buffer_rsrc_t rs_o =
          buffer_of(static_cast<uint16_t*>(p.dw) + t.e * nk, (uint64_t)nk * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& v = acc[i][j];
            *reinterpret_cast<uint2*>(ob + r32 * 128 + (((4 * j + q) ^ (r32 & 7)) << 4) + kg * 8) =
                make_uint2(bf16x2_rne(v[4 * q], v[4 * q + 1]),
                           bf16x2_rne(v[4 * q + 2], v[4 * q + 3]));
          }
        rows_out(rs_o, t.a0 + 128 * wm + 32 * i, t.b0 + 64 * wn, 2);
      }
    } else {
      const __amdgpu_buffer_rsrc_t rs_o =
          buffer_of(static_cast<float*>(p.dw) + ((int64_t)t.slice * p.E + t.e) * nk,
                    (uint64_t)nk * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& v = acc[i][j];
            *reinterpret_cast<f32x4*>(ob + r32 * 128 + (((2 * q + kg) ^ (r32 & 7)) << 4)) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          }
          rows_out(rs_o, t.a0 + 128 * wm + 32 * i, t.b0 + 64 * wn + 32 * j, 4);
        }
    }
  };

  // ---- the stream --------------------------------------------------------
#pragma unroll
  for (int u = 0; u < 4; ++u) load_ids(u, next_step(u % 2 == 0));
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    issue(stage[u], u);
    if (u < 2) fill(stage[u], u);
    if (u == 1) load_ids(0, next_step(true));    // step 4
    if (u == 2) load_ids(1, next_step(false));   // step 5
  }
  wait_and_barrier<2 * kOps>();
  read(st0, 0);
  int behind = 3;   // barriers since the last tile's stores
  int i = 0, n = 0, v = item_at(0);
  Item t;
  bool done = v >= last;
  if (!done) {
    t = item_of(v);
    n = t.steps;
  }
  clear();
  // store the tile that ended, and those after it that have no rows
  auto ended = [&]() __attribute__((always_inline)) {
    do {
      store(t);
      clear();
      behind = 0;
      v = item_at(++i);
      done = v >= last;
      if (done) break;
      t = item_of(v);
      n = t.steps;
    } while (n == 0);
  };
  if (!done && n == 0) ended();
  auto step = [&](auto j_c) __attribute__((always_inline)) {
    constexpr int j = decltype(j_c)::value, j1 = (j + 1) & 3, j2 = (j + 2) & 3;
    read(stage[j], 1);
    multiply(0);
    const WgStep next = next_step(j % 2 == 0);
    if (behind >= 3) wait_for<2 * kOps>();
    else if (p.dw_bf16) wait_for<2 * kOps + kStores>();
    else wait_for<2 * kOps + 2 * kStores>();
    barrier();
    ++behind;
    read(stage[j1], 0);
    issue(stage[j], j);
    load_ids(j2, next);
    fill(stage[j2], j2);
    multiply(1);
  };
  while (!done) {
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    if ((n -= 2) == 0) ended();
    if (done) break;
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
    if ((n -= 2) == 0) ended();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // fills past the end
}

// Sizes that a call takes.  Its workspace query asks the same first: the
// splits below divide by tile counts, which other sizes make zero or overflow.
static bool dgrad_sizes(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  return E >= 1 && E <= 1024 && M_total >= 0 && M_total < (1LL << 31) && N >= 16 && N % 16 == 0 &&
         N <= (1LL << 20) && K >= 64 && K % 64 == 0 && K <= (1LL << 20);
}
static bool wgrad_sizes(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  return E >= 1 && E <= 1024 && M_total >= 0 && M_total < (1LL << 30) && N >= 8 && N % 8 == 0 &&
         N <= (1LL << 20) && K >= 8 && K % 8 == 0 && K <= (1LL << 20);
}

// The input gradient's few-row kernel: up to 16 rows per expert on average
// (the host knows no more; the kernel's comment has what uneven rows cost),
// measured routed at random (128 experts of 1536x2048: 68 against 87 us at 16 rows, 97
// against 92 at 24, 119 against 101 at 32; 8 of 4096x4096: 35 against 34 at
// 16, 43 against 34 at 24), or 64 rows in all (one expert of 4096x1536, 64
// rows: 15 against 18 us, 100 rows 31 against 22).
static bool dgrad_few_rows(int64_t E, int64_t M_total) {
  return M_total <= 16 * E || M_total <= 64;
}

// Slices of n, at most 16, each of eight steps of 64 or more: for the few-row
// kernel, enough for four waves per SIMD of 256 CUs if every expert (at most
// one per row) has rows; for the tiled one, enough to give every CU a tile
// where the rows make less than one per two CUs.
static int dgrad_split(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  const int64_t steps = (N + 63) / 64;
  int64_t s;
  if (dgrad_few_rows(E, M_total)) {
    s = 4096 / ((E < M_total ? E : (M_total < 1 ? 1 : M_total)) * (K / 64));
  } else {
    // (an expert's last tile is half full on average, and every expert has one:
    // 256 rows over 8 experts of 4096x4096, 45 us with three slices, 35 with two)
    int64_t tiles = (M_total + kTile - 1) / kTile + E / 2;
    tiles = tiles < E ? E : tiles;
    s = 256 / (tiles * ((K + kTile - 1) / kTile));
  }
  s = s > steps / 8 ? steps / 8 : s;
  s = s < 1 ? 1 : (s > 16 ? 16 : s);
  const int64_t per = (steps + s - 1) / s;
  return (int)((steps + per - 1) / per);   // no slice is empty
}

// dw = sum of the slices' partial products; four elements per lane
template <int G, bool BF16>
__global__ void __launch_bounds__(256)
k_wgrad_reduce(const float* __restrict__ part, int64_t n, int nsplit, void* __restrict__ dw,
               int accumulate) {
  constexpr int L = 256 / G;
  for (int64_t q0 = blockIdx.x * (4LL * L); q0 < n; q0 += gridDim.x * (4LL * L)) {
    const int64_t q = q0 + (threadIdx.x % L) * 4;
    const f32x4 s = slice_sum<G>(part, q, n, nsplit, q < n);
    if (threadIdx.x >= L || q >= n) continue;
    if constexpr (BF16) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dw) + q) =
          make_uint2(bf16x2_rne(s.x, s.y), bf16x2_rne(s.z, s.w));
    } else {
      f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(dw) + q);
      *d = accumulate ? *d + s : s;
    }
  }
}

// workgroups of a slice sum over n elements with G groups
static unsigned join_grid(int64_t n, int G) {
  const int64_t per = 1024 / G, g = (n + per - 1) / per;
  return (unsigned)(g < 65536 ? g : 65536);
}

// Slices of each expert's rows for a weight gradient whose tiles fill less
// than the chip (sized for 256 CUs and rows spread evenly): each slice keeps
// four steps or more.
static int wgrad_split(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  const int64_t tiles = E * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
  const int64_t steps = (M_total / E + 63) / 64;
  int64_t s = 256 / tiles;
  s = s > steps / 4 ? steps / 4 : s;
  return (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

static size_t dgrad_prefix_bytes(int64_t E) { return round_up(2 * (size_t)(E + 1) * sizeof(int32_t), 256); }

size_t grouped_w4a16_dgrad_workspace_size(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  if (!dgrad_sizes(E, M_total, N, K)) return 256;   // the call refuses them
  const int sp = dgrad_split(E, M_total, N, K);
  return dgrad_prefix_bytes(E) +
         (sp > 1 ? round_up((size_t)sp * (size_t)M_total * (size_t)K * 4, 256) : 0);
}

int grouped_w4a16_dgrad(const void* dy, const int32_t* dy_rows, int64_t M_src,
                        const uint8_t* w_codes, const uint8_t* w_scales, const float* g_w,
                        const int32_t* expert_offsets, int64_t E, int64_t M_total, int64_t N,
                        int64_t K, void* dx, void* ws, size_t ws_bytes, void* stream) {
  NV_REQUIRE(dgrad_sizes(E, M_total, N, K) && M_src >= 0, NVFP4_ERR_SHAPE,
             "grouped_w4a16_dgrad: need 1 <= E <= 1024, M_total < 2^31, N %% 16 == 0, K %% 64 == 0, "
             "N and K up to 2^20 (E=%lld M_total=%lld N=%lld K=%lld)",
             (long long)E, (long long)M_total, (long long)N, (long long)K);
  NV_REQUIRE(dy_rows != nullptr || M_src >= M_total, NVFP4_ERR_SHAPE,
             "grouped_w4a16_dgrad: without dy_rows, M_src must be >= M_total");
  NV_REQUIRE(M_total == 0 || M_src >= 1, NVFP4_ERR_SHAPE, "grouped_w4a16_dgrad: M_src == 0");
  NV_REQUIRE((uint64_t)M_src <= kMaxBytes / (2 * (uint64_t)N) &&
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
  p.nsplit = dgrad_split(E, M_total, N, K);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + dgrad_prefix_bytes(E));
  if (dgrad_few_rows(E, M_total)) {
    const int64_t groups = (K + 255) / 256;
    const int64_t blocks = E * groups * p.nsplit;   // 2^22 at most, by the sizes and the split
    // (33 to 64 rows in all: the two passes an expert may need side by side)
    k_dgrad_few<<<dim3((unsigned)blocks, M_total > 32 && M_total <= 64 ? 2 : 1), 256, 0, s>>>(
        p, (int)groups);
  } else {
    const int64_t n_tiles = (K + kTile - 1) / kTile;
    const int64_t m_tiles = (M_total + kTile - 1) / kTile + E;   // the most there can be
    // (whole tiles and tails are each rounded up to 8 XCDs)
    const int64_t blocks = (m_tiles * n_tiles + 14) / 8 * 8;
    NV_REQUIRE(m_tiles * n_tiles + 14 < (1LL << 22), NVFP4_ERR_UNSUPPORTED,
               "grouped_w4a16_dgrad: 2^22 tiles of 256x256 or more");
    k_dgrad_tiles<<<1, 1024, 0, s>>>(p, static_cast<int32_t*>(ws));
    k_dgrad<<<dim3((unsigned)blocks, (unsigned)p.nsplit), 512, 0, s>>>(p, (int)n_tiles);
  }
  if (p.nsplit > 1) {
    if (p.nsplit >= 8)
      k_dgrad_join<4><<<join_grid(M_total * K, 4), 256, 0, s>>>(p.part, expert_offsets, (int)E,
                                                                M_total, K, p.nsplit, p.dx);
    else
      k_dgrad_join<1><<<join_grid(M_total * K, 1), 256, 0, s>>>(p.part, expert_offsets, (int)E,
                                                                M_total, K, p.nsplit, p.dx);
  }
  return check_launch("grouped_w4a16_dgrad");
}

size_t grouped_wgrad_workspace_size(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  if (!wgrad_sizes(E, M_total, N, K)) return 256;   // the call refuses them
  const int sp = wgrad_split(E, M_total, N, K);
  return sp > 1 ? round_up((size_t)sp * (size_t)E * (size_t)N * (size_t)K * 4, 256) : 256;
}

int grouped_wgrad(const void* dy, const int32_t* dy_rows, int64_t M_dy, const void* x,
                  const uint8_t* x_scales, const int32_t* x_rows, int64_t M_x,
                  const int32_t* expert_offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                  void* dw, int dw_bf16, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  NV_REQUIRE(wgrad_sizes(E, M_total, N, K) && M_dy >= 0 && M_x >= 0 &&
                 (x_scales == nullptr || K % 32 == 0),
             NVFP4_ERR_SHAPE,
             "grouped_wgrad: need 1 <= E <= 1024, M_total < 2^30, N %% 8 == 0, K %% 8 == 0 "
             "(K %% 32 == 0 for 8-bit x), N and K up to 2^20 (E=%lld M_total=%lld N=%lld K=%lld)",
             (long long)E, (long long)M_total, (long long)N, (long long)K);
  NV_REQUIRE((dy_rows != nullptr || M_dy >= M_total) && (x_rows != nullptr || M_x >= M_total),
             NVFP4_ERR_SHAPE, "grouped_wgrad: an operand without a row list needs M_total rows");
  NV_REQUIRE(M_total == 0 || (M_dy >= 1 && M_x >= 1), NVFP4_ERR_SHAPE,
             "grouped_wgrad: an operand has no rows");
  NV_REQUIRE((uint64_t)M_dy <= kMaxBytes / (2 * (uint64_t)N) &&
                 (uint64_t)M_x <= kMaxBytes / ((x_scales ? 1 : 2) * (uint64_t)K),
             NVFP4_ERR_UNSUPPORTED, "grouped_wgrad: dy or x exceeds 4 GiB");
  NV_REQUIRE((uint64_t)N * (uint64_t)K < (1ULL << 30), NVFP4_ERR_UNSUPPORTED,
             "grouped_wgrad: one expert's dw has 2^30 elements or more");
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
  p.accumulate = accumulate != 0;
  p.nsplit = wgrad_split(E, M_total, N, K);
  const int64_t n_tiles = (K + kTile - 1) / kTile, m_tiles = (N + kTile - 1) / kTile;
  const int64_t items = E * n_tiles * m_tiles * p.nsplit;
  NV_REQUIRE(items < (1LL << 30), NVFP4_ERR_UNSUPPORTED, "grouped_wgrad: more than 2^30 tiles");
  const int64_t cus = num_cus() / 8 * 8 > 0 ? num_cus() / 8 * 8 : 8;
  const int64_t want = (items + 7) / 8 * 8;
  const unsigned grid = (unsigned)(want < cus ? want : cus);
  const bool split = p.nsplit > 1;
  if (split) {
    p.dw = ws;
    p.accumulate = 0;
  }
  const int nt = (int)n_tiles, mt = (int)m_tiles;
  p.dw_bf16 = dw_bf16 && !split;
  const auto k = x_scales ? (dy_rows ? (x_rows ? k_wgrad<true, true, true> : k_wgrad<true, true, false>)
                                     : (x_rows ? k_wgrad<true, false, true> : k_wgrad<true, false, false>))
                          : (dy_rows ? (x_rows ? k_wgrad<false, true, true> : k_wgrad<false, true, false>)
                                     : (x_rows ? k_wgrad<false, false, true> : k_wgrad<false, false, false>));
  k<<<grid, 512, 0, s>>>(p, nt, mt);
  if (split) {
    const int64_t n = E * N * K;
    const float* part = static_cast<const float*>(ws);
    const int ns = p.nsplit, add = accumulate != 0;
    if (dw_bf16 && ns >= 8)
      k_wgrad_reduce<4, true><<<join_grid(n, 4), 256, 0, s>>>(part, n, ns, dw, 0);
    else if (dw_bf16)
      k_wgrad_reduce<1, true><<<join_grid(n, 1), 256, 0, s>>>(part, n, ns, dw, 0);
    else if (ns >= 8)
      k_wgrad_reduce<4, false><<<join_grid(n, 4), 256, 0, s>>>(part, n, ns, dw, add);
    else
      k_wgrad_reduce<1, false><<<join_grid(n, 1), 256, 0, s>>>(part, n, ns, dw, add);
  }
  return check_launch("grouped_wgrad");
}

}  // extern "C"
