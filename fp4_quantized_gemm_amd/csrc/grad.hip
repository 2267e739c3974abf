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
  const int32_t* prefix;       // dgrad: row tiles before each expert
  uint16_t* dx;                // dgrad: [M_total][K] bf16
  void* dw;                    // wgrad: [E][N][K] f32 or bf16
  int64_t M_dy, M_x, M_total, N, K;
  int E;
  int dw_bf16, accumulate;
  int run;                     // wgrad: log2 of the tiles an XCD takes in a row
  int nsplit;                  // wgrad: slices of the rows (blockIdx.y); dw holds their partials
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
// 256x256 outputs per workgroup, eight waves (two rows of four, 128x64 each:
// four by two 32x32 accumulators), contraction 64 at a time through two LDS
// stages.  "Rows" are dx rows (kDgrad) or dw rows n; columns are k.
//
// An operand whose contraction index is its slow one (both of wgrad's, the
// weights of dgrad) lies in LDS as it does in memory, [64][256] bf16, and is
// read through the transposing LDS load: a group of 16 lanes reads 4
// contraction rows of 16 columns and each lane gets its column's four values.
// 16-byte chunk c of contraction row r sits at c ^ swz(r): the four rows of a
// transposing load then lie in the four 64-byte parts of the 256-byte bank
// line, and 16 rows of one chunk (the order in which decoded weights are
// written) in 16 different 16-byte slots, so neither conflicts.
// dgrad's dy has the contraction fast: [256][64], 16-byte fragment reads,
// chunk c of row r at c ^ ((r >> 1) & 7).
// bf16 operands go from memory to LDS directly; 4-bit weights and 8-bit
// activations are decoded (exactly) on the way, once per workgroup.
// ---------------------------------------------------------------------------
namespace gr {
constexpr int BM = 256, BN = 256, BC = 64;
constexpr int A_BYTES = BM * BC * 2;
constexpr int STAGE = A_BYTES + BN * BC * 2;   // 65536
enum Mode { kDgrad, kWgrad, kWgradMx };
}  // namespace gr

// an offset past every buffer: such a load returns zeros
constexpr uint32_t kPastBuffer = 0xFFFFFFF0u;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t* lds_tr_ptr;

__device__ __forceinline__ int swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }

// 8 contraction values of one column: two transposing loads of 4 rows each
__device__ __forceinline__ u32x4 tr_frag(const uint8_t* lo, const uint8_t* hi) {
  const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_ptr)lo);
  const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_ptr)hi);
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes,
                                           kBufferRsrcWord3);
}

// MODE: which product.  BF16: the output is bf16, staged through LDS for
// 16-byte row stores (the product is formed transposed, so that a lane holds
// four consecutive columns); else float32, stored from the accumulators (32
// lanes write 128 consecutive bytes).
template <int MODE, bool BF16>
__global__ void __launch_bounds__(512, 1)
k_grad(GradArgs p, int n_tiles, int m_tiles) {
  using namespace gr;
  // two objects, and the loop unrolled by two: each access names its stage,
  // so the fill of one stage is not waited for before reads of the other
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
  __shared__ int32_t rows_src[MODE == kDgrad ? BM : 1];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int kg = lane >> 5, r32 = lane & 31;

  // tile order (workgroup b runs on XCD b % 8, each with its own L2)
  int e, nt;
  int64_t lo, hi, a0;
  {
    const int b = (int)blockIdx.x;
    if constexpr (MODE == kDgrad) {
      // groups of 4 row tiles x all column tiles, a contiguous range per XCD
      const int real_m = p.prefix[p.E];
      const int real_blocks = ((real_m + 3) / 4) * 4 * n_tiles;
      const int per_xcd = (real_blocks + 7) / 8;
      if ((b >> 3) >= per_xcd) return;
      const int v = (b & 7) * per_xcd + (b >> 3);
      if (v >= real_blocks) return;
      const int group = 4 * n_tiles;
      const int gi = v / group, g = v - gi * group;
      const int gm = real_m - 4 * gi < 4 ? real_m - 4 * gi : 4;
      const int gt = 4 * gi + g % gm;
      nt = g / gm;
      if (gt >= real_m || nt >= n_tiles) return;
      int l = 0, h = p.E;
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (p.prefix[mid] <= gt) l = mid; else h = mid;
      }
      e = l;
      expert_rows(p, e, lo, hi);
      a0 = lo + (int64_t)(gt - p.prefix[e]) * BM;
    } else {
      // runs of 2^run tiles of an expert go to the XCDs in turn
      const int per_e = n_tiles * m_tiles;
      const int total = per_e * p.E;
      const int loc = b >> 3, run = p.run;
      const int v = ((((loc >> run) << 3) + (b & 7)) << run) + (loc & ((1 << run) - 1));
      if (v >= total) return;
      e = v / per_e;
      const int t = v - e * per_e;
      nt = t % n_tiles;
      a0 = (int64_t)(t / n_tiles) * BM;
      expert_rows(p, e, lo, hi);
      if (p.nsplit > 1) {   // this slice's rows: whole steps
        const int64_t steps = (hi - lo + BC - 1) / BC;
        const int64_t per = (steps + p.nsplit - 1) / p.nsplit * BC;
        const int64_t l = lo + per * blockIdx.y;
        lo = l < hi ? l : hi;
        hi = lo + per < hi ? lo + per : hi;
      }
    }
  }
  const int64_t b0 = (int64_t)nt * BN;
  const int steps = MODE == kDgrad ? (int)((p.N + BC - 1) / BC) : (int)((hi - lo + BC - 1) / BC);

  // ---- loads -------------------------------------------------------------
  const uint32_t N2 = (uint32_t)(p.N * 2);
  const __amdgpu_buffer_rsrc_t rs_a = buffer_of(p.dy, (uint64_t)p.M_dy * (uint64_t)p.N * 2);
  // [64][256] tiles: lane's contraction row is 16 i + r16 of the step (i of
  // four), its slot in the row lane % 32, which holds chunk tr_c
  const int r16 = 2 * wave + kg;
  const int tr_c = r32 ^ swz(r16);
  uint32_t off_a[4];             // dgrad: byte offsets of the four loads at step 0
  uint32_t col_a = 0, col_b = 0; // wgrad: byte offset of the lane's chunk in a row
  uint32_t row_a[4], row_b[4];   // wgrad: the row lists' entries for the next loads
  uint32_t chunk_n[4];           // dgrad: first column of the chunk
  if constexpr (MODE == kDgrad) {
    if (tid < BM) {
      int64_t pr = a0 + tid;
      if (pr >= hi) pr = hi - 1;
      rows_src[tid] = (int32_t)source_row(p.dy_rows, pr, p.M_dy);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = (i * 8 + wave) * 64 + lane;
      const int r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
      off_a[i] = (uint32_t)rows_src[r] * N2 + 16u * c;
      chunk_n[i] = 8u * c;
    }
  } else {
    const int64_t n = a0 + 8 * tr_c, k = b0 + 8 * tr_c;
    col_a = n < p.N ? (uint32_t)n * 2 : kPastBuffer;
    col_b = k < p.K ? (uint32_t)k * (MODE == kWgrad ? 2 : 1) : kPastBuffer;
  }
  // A missing list is a buffer of no bytes: the load returns 0 and is not
  // used.  No branch surrounds these loads: a value merged after a branch
  // would be waited for there, and every fill in flight with it.
  const __amdgpu_buffer_rsrc_t rs_ra =
      buffer_of(p.dy_rows, MODE != kDgrad && p.dy_rows ? (uint64_t)p.M_total * 4 : 0);
  const __amdgpu_buffer_rsrc_t rs_rb =
      buffer_of(p.x_rows, MODE != kDgrad && p.x_rows ? (uint64_t)p.M_total * 4 : 0);
  const uint32_t p_lane = (uint32_t)lo + r16, p_hi = (uint32_t)hi;
  auto load_rows = [&](int step) __attribute__((always_inline)) {
    if constexpr (MODE != kDgrad) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t o = (p_lane + (uint32_t)step * BC + 16 * i) * 4;
        row_a[i] = __builtin_amdgcn_raw_buffer_load_b32(rs_ra, o, 0, 0);
        row_b[i] = __builtin_amdgcn_raw_buffer_load_b32(rs_rb, o, 0, 0);
      }
    }
  };
  // byte offset of the lane's chunk in row `listed` (or pr without a list),
  // past the buffer for rows and columns that are not there
  auto chunk_at = [&](bool has_list, uint32_t listed, uint32_t pr, int64_t M, uint32_t pitch,
                      uint32_t col) __attribute__((always_inline)) {
    const uint32_t t = has_list ? listed : pr;
    const uint32_t last = (uint32_t)(M - 1);
    const uint32_t row = (int32_t)t < 0 ? 0u : (t > last ? last : t);
    return pr < p_hi && col != kPastBuffer ? row * pitch + col : kPastBuffer;
  };
  const uint64_t x_bytes = (uint64_t)p.M_x * (uint64_t)p.K * (MODE == kWgrad ? 2 : 1);
  const __amdgpu_buffer_rsrc_t rs_b =
      MODE == kDgrad ? buffer_of(p.w_codes + e * packed_codes_per_expert(p.N, p.K),
                                 (uint64_t)p.N * p.K / 2)
                     : buffer_of(p.x, x_bytes);
  const __amdgpu_buffer_rsrc_t rs_s =
      MODE == kDgrad ? buffer_of(p.w_scales + e * packed_scales_per_expert(p.N, p.K),
                                 (uint64_t)p.N * p.K / 16)
                     : buffer_of(p.x_scales, (uint64_t)p.M_x * (uint64_t)p.K / 32);
  // dgrad weights: wave w takes the step's code tiles 2 w, 2 w + 1 (of 4 row
  // blocks x 4 column tiles), lane l one row's half tile: 16 bytes = 32 k
  const int w_rb = (2 * wave + kg) >> 2, w_ct = (2 * wave + kg) & 3;
  const int w_half = (lane >> 4) & 1, w_row = lane & 15;
  uint32_t off_w = 0, off_ws = 0;
  const uint32_t w_step = (uint32_t)(4 * (p.K >> 6) * 512);
  if constexpr (MODE == kDgrad) {
    int64_t kt = (b0 >> 6) + w_ct;
    if (kt >= (p.K >> 6)) kt = (p.K >> 6) - 1;   // columns past K are never stored
    const uint32_t tile = (uint32_t)(w_rb * (p.K >> 6) + kt);
    off_w = tile * 512 + w_half * 256 + w_row * 16;
    off_ws = tile * 64 + w_row * 4 + w_half * 2;
  }
  u32x4 wreg;
  uint32_t sreg[4];
  uint32_t creg[4][2];

  auto issue = [&](uint8_t* st, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint8_t* dst = st + (i * 8 + wave) * 1024;
      if constexpr (MODE == kDgrad) {
        const uint32_t n0 = (uint32_t)step * BC;
        const uint32_t o = n0 + chunk_n[i] < (uint32_t)p.N ? off_a[i] : kPastBuffer;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(dst), 16, o, n0 * 2, 0, 0);
      } else {
        const uint32_t pr = p_lane + (uint32_t)step * BC + 16 * i;
        const uint32_t o = chunk_at(p.dy_rows != nullptr, row_a[i], pr, p.M_dy, N2, col_a);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, lds_ptr(dst), 16, o, 0, 0, 0);
        const uint32_t ob = chunk_at(p.x_rows != nullptr, row_b[i], pr, p.M_x,
                                     (uint32_t)(p.K * (MODE == kWgrad ? 2 : 1)), col_b);
        if constexpr (MODE == kWgrad) {
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, lds_ptr(dst + A_BYTES), 16, ob, 0, 0, 0);
        } else {
          const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs_b, ob, 0, 0);
          creg[i][0] = v[0];
          creg[i][1] = v[1];
          sreg[i] = __builtin_amdgcn_raw_buffer_load_b8(
              rs_s, ob == kPastBuffer ? kPastBuffer : ob >> 5, 0, 0);
        }
      }
    }
    if constexpr (MODE == kDgrad) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs_b, off_w, (uint32_t)step * w_step, 0);
      wreg = u32x4{v[0], v[1], v[2], v[3]};
      sreg[0] = __builtin_amdgcn_raw_buffer_load_b16(rs_s, off_ws, (uint32_t)step * (w_step >> 3), 0);
    }
    load_rows(step + 1);
  };
  // decode what issue() left in registers into the stage
  auto fill = [&](uint8_t* st) __attribute__((always_inline)) {
    if constexpr (MODE == kDgrad) {
      const float s0 = e4m3_decode(sreg[0] & 0xFFu), s1 = e4m3_decode(sreg[0] >> 8);
      const int r = 16 * w_rb + w_row;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 8 * w_ct + 4 * w_half + j;
        *reinterpret_cast<u32x4*>(st + A_BYTES + r * 512 + ((c ^ swz(w_row)) << 4)) =
            decode8_bf16(wreg[j], j < 2 ? s0 : s1);
      }
    } else if constexpr (MODE == kWgradMx) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x4*>(st + A_BYTES + (i * 8 + wave) * 1024 + lane * 16) =
            mx_decode8(make_uint2(creg[i][0], creg[i][1]), mx_scale(sreg[i]));
    }
  };

  // ---- products ----------------------------------------------------------
  f32x16_t acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // transposing loads: lane i of a 16-lane group g reads row 8 (g / 2) + 4 h
  // + i / 4 of the 16-row slice, columns 16 (g % 2) + 4 (i % 4) .. + 3 of the
  // fragment's 32 (4 chunks)
  const int t_row = 8 * kg + ((lane & 15) >> 2);
  const int t_chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  const uint32_t t_off0 = t_row * 512 + ((t_chunk ^ swz(t_row)) << 4) + (lane & 1) * 8;
  const uint32_t t_off1 = (t_row + 4) * 512 + ((t_chunk ^ swz(t_row + 4)) << 4) + (lane & 1) * 8;
  // fragment f (32 columns = 4 chunks, 64 bytes): chunk bits 2.. are xored too
  auto tr_at = [&](const uint8_t* t, int slice, int f) __attribute__((always_inline)) {
    const uint32_t x = (uint32_t)f << 6;   // f < 8: bits 6..8 of the slot's byte offset
    return tr_frag(t + slice * 8192 + (t_off0 ^ x), t + slice * 8192 + (t_off1 ^ x));
  };
  const int sw = (r32 >> 1) & 7;
  auto compute = [&](const uint8_t* st, auto nv_c) __attribute__((always_inline)) {
    constexpr int NV = decltype(nv_c)::value;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 B[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) B[j] = tr_at(st + A_BYTES, s, 2 * wn + j);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        u32x4 A;
        if constexpr (MODE == kDgrad)
          A = *reinterpret_cast<const u32x4*>(st + (wm * 128 + 32 * i + r32) * 128 +
                                              (((2 * s + kg) ^ sw) << 4));
        else
          A = tr_at(st, s, 4 * wm + i);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = BF16 ? mfma32_bf16(B[j], A, acc[i][j]) : mfma32_bf16(A, B[j], acc[i][j]);
      }
    }
  };
  auto kstep = [&](const uint8_t* cur, uint8_t* nxt, int s, auto nv_c) __attribute__((always_inline)) {
    if (s + 1 < steps) issue(nxt, s + 1);
    compute(cur, nv_c);
    if (s + 1 < steps) fill(nxt);
    wait_vmem0();
    __syncthreads();
  };
  auto run = [&](auto nv_c) __attribute__((always_inline)) {
    int s = 0;
    for (; s + 1 < steps; s += 2) {
      kstep(st0, st1, s, nv_c);
      kstep(st1, st0, s + 1, nv_c);
    }
    if (s < steps) kstep(st0, st1, s, nv_c);
  };
  load_rows(0);
  if (steps > 0) {
    issue(st0, 0);
    fill(st0);
  }
  wait_vmem0();
  __syncthreads();
  if constexpr (MODE == kDgrad) {
    // rows of this wave inside the expert: only their 32-row blocks
    const int64_t vr = hi - a0 - wm * 128;
    if (vr > 64) run(std::integral_constant<int, 4>{});
    else if (vr > 32) run(std::integral_constant<int, 2>{});
    else if (vr > 0) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 0>{});
  } else {
    run(std::integral_constant<int, 4>{});
  }

  // ---- outputs -----------------------------------------------------------
  const float sc = MODE == kDgrad ? p.g_w[e] : 1.0f;
  if constexpr (BF16) {
    // row 32 i + r32 of the wave's half tile, columns 64 wn + 32 j + 8 q +
    // 4 kg .. + 3; 16-byte chunk c of row r at c ^ (r & 15)
    uint8_t* half = wm ? st1 : st0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 32 * i + r32, c = 8 * wn + 4 * j + q;
          const f32x16_t& v = acc[i][j];
          *reinterpret_cast<uint2*>(half + r * 512 + ((c ^ (r & 15)) << 4) + kg * 8) =
              make_uint2(bf16x2_rne(v[4 * q] * sc, v[4 * q + 1] * sc),
                         bf16x2_rne(v[4 * q + 2] * sc, v[4 * q + 3] * sc));
        }
    __syncthreads();
    const int64_t rows_end = MODE == kDgrad ? hi : p.N;
    uint16_t* out = MODE == kDgrad ? p.dx
                                   : static_cast<uint16_t*>(p.dw) + (int64_t)e * p.N * p.K;
#pragma unroll 4
    for (int q = tid; q < BM * 32; q += 512) {
      const int r = q >> 5, c = q & 31;
      const int64_t a = a0 + r, k = b0 + 8 * c;
      const uint8_t* src = (r < 128 ? st0 : st1) + (r & 127) * 512 + ((c ^ (r & 15)) << 4);
      if (a < rows_end && k < p.K)
        *reinterpret_cast<uint4*>(out + a * p.K + k) = *reinterpret_cast<const uint4*>(src);
    }
  } else {
    float* out = static_cast<float*>(p.dw) +
                 ((int64_t)(p.nsplit > 1 ? blockIdx.y : 0) * p.E + e) * p.N * p.K;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t k = b0 + 64 * wn + 32 * j + r32;
        if (k >= p.K) continue;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int64_t a = a0 + 128 * wm + 32 * i + 8 * (r >> 2) + 4 * kg + (r & 3);
          if (a >= p.N) continue;
          float* d = out + a * p.K + k;
          *d = p.accumulate ? *d + acc[i][j][r] : acc[i][j][r];
        }
      }
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
// Eight waves of 128x64 outputs.  LDS serves 128 bytes per clock: a step's
// 96 KB of fragment reads and 32 KB of fills take as many clocks as its matrix
// instructions (1024), so both have to run all the time: fragments are read
// half a step (16 rows) ahead of their products, in step with the matrix
// instructions, and the barrier that hands over a stage lies between a step's
// halves.
//
// Waits.  Loads and stores of a wave complete in order, so the barrier of step
// s waits until at most the operations issued after stage s + 1's last fill
// are outstanding (two steps of kOps, plus the stores where a tile ended in
// between); each step issues the same number, past the last row too, where
// they return zeros, and an edge tile's stores are issued with an offset past
// the buffer.  Row lists are read two steps before the fill that uses them,
// 8-bit codes four steps before their stage and decoded two steps later.
// ---------------------------------------------------------------------------
namespace wg {
constexpr int BM = 256, BN = 256, BC = 32;
constexpr int A_BYTES = BC * BM * 2;
constexpr int STAGE = A_BYTES + BC * BN * 2;   // 32768
constexpr int OUT = 4096;                      // output staging of one wave
}  // namespace wg

// A contraction step's rows [p, hi) and its tile's first output row and column
struct WgStep {
  uint32_t p, hi, a0, b0;
};

template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N < 63 ? N : 63) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

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
  constexpr int kStores = 16;   // bf16; float32 has 32, and waits for half of them

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int kg = lane >> 5, r32 = lane & 31;
  uint8_t* const stage[4] = {st0, st1, st2, st3};

  // ---- items -------------------------------------------------------------
  const int per_e = n_tiles * m_tiles;
  const int total = per_e * p.E;
  const int items = total * p.nsplit;
  const int xcd = (int)blockIdx.x & 7, loc = (int)blockIdx.x >> 3, per_xcd = (int)gridDim.x >> 3;
  // the workgroup's i-th item: runs of 2^run items go to the XCDs in turn
  // (workgroup b runs on XCD b % 8, each with its own L2), and an XCD's
  // workgroups take its items in turn
  auto item_at = [&](int i) __attribute__((always_inline)) {
    const int j = loc + i * per_xcd;
    return ((((j >> p.run) << 3) + xcd) << p.run) + (j & ((1 << p.run) - 1));
  };
  struct Item {
    uint32_t lo, hi, a0, b0;
    int e, slice, steps;
  };
  auto item_of = [&](int v) __attribute__((always_inline)) {
    Item t;
    t.slice = v / total;
    v -= t.slice * total;
    t.e = v / per_e;
    v -= t.e * per_e;
    const int m = v / n_tiles;
    t.a0 = (uint32_t)m * BM;
    t.b0 = (uint32_t)(v - m * n_tiles) * BN;
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
    // a tile's steps are rounded up to the ring's four; the added ones load
    // and multiply zeros
    t.steps = (hi - lo + 4 * BC - 1) / (4 * BC) * 4;
    return t;
  };

  // ---- loads -------------------------------------------------------------
  // the step that the row lists are next read for
  int ahead_i = -1, ahead_s = 0;
  Item ahead;
  ahead.lo = ahead.hi = ahead.a0 = ahead.b0 = 0;
  ahead.steps = 0;
  // (tiles begin at multiples of four: only there a new one can follow)
  auto next_step = [&](bool maybe_new) __attribute__((always_inline)) {
    ++ahead_s;
    while (maybe_new && ahead_s >= ahead.steps) {
      ahead_s = 0;
      const int v = item_at(++ahead_i);
      if (v >= items) {   // none left: rows that are not there
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
  // transposing loads: lane i of a 16-lane group g reads row 8 (g / 2) + 4 h
  // + i / 4 of the 16-row slice, columns 16 (g % 2) + 4 (i % 4) .. + 3 of the
  // fragment's 32 (4 chunks); fragment f xors bits 2.. of the chunk
  const int t_row = 8 * kg + ((lane & 15) >> 2);
  const int t_chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  const uint32_t t_off0 = t_row * 512 + ((t_chunk ^ swz(t_row)) << 4) + (lane & 1) * 8;
  const uint32_t t_off1 = (t_row + 4) * 512 + ((t_chunk ^ swz(t_row + 4)) << 4) + (lane & 1) * 8;
  auto tr_at = [&](const uint8_t* t, int f) __attribute__((always_inline)) {
    const uint32_t x = (uint32_t)f << 6;
    return tr_frag(t + (t_off0 ^ x), t + (t_off1 ^ x));
  };
  u32x4 fa[2][4], fb[2][2];   // by half of the step
  auto read = [&](const uint8_t* st, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) fb[half][j] = tr_at(st + A_BYTES + half * 8192, 2 * wn + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) fa[half][i] = tr_at(st + half * 8192, 4 * wm + i);
  };
  // formed transposed (x as the row operand), so that a lane's four
  // consecutive accumulators are four consecutive columns of its dw row
  auto multiply = [&](int half) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma32_bf16(fb[half][j], fa[half][i], acc[i][j]);
    // a matrix instruction, then up to two LDS reads, five others, one load
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x006, 5, 0);
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
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 8 * q + lr;
        u32x4 v = *reinterpret_cast<const u32x4*>(ob + r * 128 + ((lc ^ (r & 7)) << 4));
        const uint32_t n = n0 + r, k = k0 + lc * (16 / bytes);
        const uint32_t o = n < N && k < K ? (n * K + k) * bytes : kPastBuffer;
        if (bytes == 4 && p.accumulate) {
          const auto old = __builtin_amdgcn_raw_buffer_load_b128(rs_o, o, 0, 0);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[c] = __float_as_uint(__uint_as_float(v[c]) + __uint_as_float(old[c]));
        }
        // nontemporal: dw is not read back soon, and its lines leave L2 to the
        // operands (wgrad of 32768 rows, 128 experts of 1536x2048: 0.52 ->
        // 0.36 ms)
        __builtin_amdgcn_raw_buffer_store_b128(v, rs_o, o, 0, 2);
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
  load_ids(0, next_step(true));
  load_ids(1, next_step(false));
  load_ids(2, next_step(false));
  load_ids(3, next_step(false));
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    issue(stage[u], u);
    if (u < 2) fill(stage[u], u);
    if (u == 1) load_ids(0, next_step(true));    // step 4
    if (u == 2) load_ids(1, next_step(false));   // step 5
  }
  wait_and_barrier<2 * kOps>();
  read(st0, 0);
  bool stored = false;
  auto body = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      read(stage[j], 1);
      multiply(0);
      if (j < 3 && stored) wait_and_barrier<2 * kOps + kStores>();
      else wait_and_barrier<2 * kOps>();
      read(stage[(j + 1) & 3], 0);
      issue(stage[j], j);
      load_ids((j + 2) & 3, next_step(j == 2));
      fill(stage[(j + 2) & 3], (j + 2) & 3);
      multiply(1);
    }
    stored = false;
  };
  for (int i = 0;; ++i) {
    const int v = item_at(i);
    if (v >= items) break;
    const Item t = item_of(v);
    clear();
    for (int s = 0; s < t.steps; s += 4) body();
    store(t);
    stored = true;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // fills past the end
}

// dw = sum of the slices' partial products, in slice order; 4 per lane
template <bool BF16>
__global__ void __launch_bounds__(256)
k_wgrad_reduce(const float* __restrict__ part, int64_t n, int nsplit, void* __restrict__ dw,
               int accumulate) {
  for (int64_t q = (blockIdx.x * 256LL + threadIdx.x) * 4; q < n; q += gridDim.x * 1024LL) {
    f32x4 s = *reinterpret_cast<const f32x4*>(part + q);
    for (int i = 1; i < nsplit; ++i) s += *reinterpret_cast<const f32x4*>(part + i * n + q);
    if constexpr (BF16) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dw) + q) =
          make_uint2(bf16x2_rne(s.x, s.y), bf16x2_rne(s.z, s.w));
    } else {
      f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(dw) + q);
      *d = accumulate ? *d + s : s;
    }
  }
}

// Slices of each expert's rows for a weight gradient whose tiles fill less
// than the chip (sized for 256 CUs and rows spread evenly): each slice keeps
// four steps or more.
static int wgrad_split(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  const int64_t tiles = E * ((N + gr::BM - 1) / gr::BM) * ((K + gr::BN - 1) / gr::BN);
  const int64_t steps = (M_total / E + gr::BC - 1) / gr::BC;
  int64_t s = 256 / tiles;
  s = s > steps / 4 ? steps / 4 : s;
  return (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
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
  tile_prefix(expert_offsets, (int)E, M_total, gr::BM, static_cast<int32_t*>(ws), s);
  const int64_t n_tiles = (K + gr::BN - 1) / gr::BN;
  const int64_t m_tiles = (M_total + gr::BM - 1) / gr::BM + E;   // the most there can be
  const int64_t blocks = ((m_tiles + 3) / 4 * 4 * n_tiles + 7) / 8 * 8;
  NV_REQUIRE(blocks < (1LL << 22), NVFP4_ERR_UNSUPPORTED,
             "grouped_w4a16_dgrad: more than 2^22 tiles");
  k_grad<gr::kDgrad, true><<<(unsigned)blocks, 512, 0, s>>>(p, (int)n_tiles, (int)m_tiles);
  return check_launch("grouped_w4a16_dgrad");
}

size_t grouped_wgrad_workspace_size(int64_t E, int64_t M_total, int64_t N, int64_t K) {
  if (E < 1 || M_total < 0 || N < 1 || K < 1) return 256;
  const int sp = wgrad_split(E, M_total, N, K);
  return sp > 1 ? round_up((size_t)sp * (size_t)E * (size_t)N * (size_t)K * 4, 256) : 256;
}

int grouped_wgrad(const void* dy, const int32_t* dy_rows, int64_t M_dy, const void* x,
                  const uint8_t* x_scales, const int32_t* x_rows, int64_t M_x,
                  const int32_t* expert_offsets, int64_t E, int64_t M_total, int64_t N, int64_t K,
                  void* dw, int dw_bf16, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  NV_REQUIRE(E >= 1 && E <= 1024 && M_total >= 0 && M_total < (1LL << 30) && M_dy >= 0 &&
                 M_x >= 0 && N >= 8 && N % 8 == 0 && K >= 8 && K % 8 == 0 && N < (1LL << 31) &&
                 K < (1LL << 31) && (x_scales == nullptr || K % 32 == 0),
             NVFP4_ERR_SHAPE,
             "grouped_wgrad: need 1 <= E <= 1024, M_total < 2^30, N %% 8 == 0, K %% 8 == 0 "
             "(K %% 32 == 0 for 8-bit x) (E=%lld M_total=%lld N=%lld K=%lld)",
             (long long)E, (long long)M_total, (long long)N, (long long)K);
  NV_REQUIRE((dy_rows != nullptr || M_dy >= M_total) && (x_rows != nullptr || M_x >= M_total),
             NVFP4_ERR_SHAPE, "grouped_wgrad: an operand without a row list needs M_total rows");
  NV_REQUIRE(M_total == 0 || (M_dy >= 1 && M_x >= 1), NVFP4_ERR_SHAPE,
             "grouped_wgrad: an operand has no rows");
  NV_REQUIRE((uint64_t)M_dy < (1ULL << 32) / (2 * (uint64_t)N) &&
                 (uint64_t)M_x < (1ULL << 32) / ((x_scales ? 1 : 2) * (uint64_t)K),
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
  const int64_t n_tiles = (K + gr::BN - 1) / gr::BN, m_tiles = (N + gr::BM - 1) / gr::BM;
  const int64_t items = E * n_tiles * m_tiles * p.nsplit;
  NV_REQUIRE(items < (1LL << 30), NVFP4_ERR_UNSUPPORTED, "grouped_wgrad: more than 2^30 tiles");
  // 32 tiles in a row keep an XCD's workgroups on one expert; fewer where the
  // tiles would not reach every XCD a few times over
  while (p.run < 5 && (512LL << p.run) <= items) ++p.run;
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
    const int64_t g = (n + 1023) / 1024;
    const unsigned rg = (unsigned)(g < 65536 ? g : 65536);
    if (dw_bf16)
      k_wgrad_reduce<true><<<rg, 256, 0, s>>>(static_cast<float*>(ws), n, p.nsplit, dw, 0);
    else
      k_wgrad_reduce<false><<<rg, 256, 0, s>>>(static_cast<float*>(ws), n, p.nsplit, dw,
                                               accumulate != 0);
  }
  return check_launch("grouped_wgrad");
}

}  // extern "C"
