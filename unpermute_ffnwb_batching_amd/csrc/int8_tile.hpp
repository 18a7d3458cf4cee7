// Tiles of the INT8 products through LDS (matmul_int8.hip).
//
// A workgroup of WM x WN waves takes BM = 16 WM MF rows by 256 columns (SwiGLU: 128 gate columns
// and the 128 up columns that go with them, half and half in every wave), one 128-column block of K
// per step.  Both operands go from memory to LDS without passing through registers (16 bytes per
// lane).  A row of a block is 128 bytes, a whole line of the caches, 8 chunks of 16; chunk c of row r lies
// at position c ^ (r % 8), which spreads the 16 rows that a matrix operand reads at once over all
// banks.  The lanes of a copy write adjacent LDS addresses, so the permutation is applied to the
// addresses they read.
//
// Many rows are bound by the power that the matrix cores draw: 8191 rows by 7168 columns over 5120 take 249 us (2.41 POP/s;
// zeros in place of random codes 204), 4096 by 4096 over 8192 103 us (2.66), and by some us a round of tiles to fill the
// buffers and store, which do not overlap the next one.  Few rows of many experts are bound by memory: 4377 rows of
// 256 experts, 2048 columns over 7168, 636 us (5.8 TB/s).
#pragma once

#include <type_traits>

#include "fp8_block.hpp"
#include "internal.hpp"
#include "lds_copy.hpp"
#include "row_quant.hpp"
#include "row_tiles.hpp"

namespace ffnwb {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Mm8Args {
  int64_t K, N, F;             // F = outputs per row (N, or N / 2 with SwiGLU)
  int64_t xs, xss, ys, yss;    // row strides: bytes, elements, bytes, elements
  int32_t rows;
  int32_t kb;                  // 128-column blocks of K
  int32_t ntiles;              // column tiles
  int32_t ngroups, nexperts;
  bool vec;                    // four adjacent outputs are one aligned store
  const char* x;
  const float* x_scale;
  const char* w;
  const float* w_scale;
  char* y;
  float* y_scale;
  float* held_max;             // of a row that is held on its way to INT8 (Held): [rows][F / 16]
  const int64_t* groups;       // {expert, rows} pairs, or NULL for one dense product
  const int4* table;           // row tiles {expert, first row, rows, 0} of more than kWaveGroups groups
  const int32_t* count;        // [1] row tiles of the table
};

// 16 rows of A by 16 rows of B over 64 INT8 columns, added to c: exact.  Lane l holds columns of row l %
// 16; the order of the columns over lanes and registers only has to be the same for A and B.  The
// result lane holds B row lane % 16 and A rows 4 (lane / 16) + 0..3.
__device__ __forceinline__ i32x4 mul_int8(const u32x4& a, const u32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Scales of the channels n .. n + 3 of an expert (those past the last: the last one's).
__device__ __forceinline__ f32x4 channel_scales(const Mm8Args& a, int32_t expert, int64_t n) {
  const float* s = a.w_scale + static_cast<int64_t>(expert) * a.N;
  f32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = s[min(n + j, a.N - 1)];
  return v;
}

__device__ __forceinline__ f32x4 scaled(const i32x4& c, float xs, const f32x4& ws) {
  f32x4 p;
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = static_cast<float>(c[j]) * xs * ws[j];
  return p;
}

// Two results as one register of a 16-bit type, a lowest.
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <class T> __device__ __forceinline__ uint32_t narrow2(float a, float b);
template <> __device__ __forceinline__ uint32_t narrow2<TBF16>(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
template <> __device__ __forceinline__ uint32_t narrow2<TF16>(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}

// Registers of the lane groups g = lane / 16 of two fragments a, b, four columns each -> of 8
// adjacent columns: group 0 gets a's groups 0 and 1 (a first), group 1 a's 2 and 3, groups 2 and 3
// those of b.
__device__ __forceinline__ void join_columns(uint32_t& a, uint32_t& b) {
  const auto h = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  const auto q = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
  a = q[0], b = q[1];
}

// silu(g) * u as swiglu (fp8_block.hpp), with the hardware's exponential and reciprocal (2^-23 each): 7
// operations, or 12, instead of about 45 (131072 rows by 1024 outputs over 4096: 1189 -> 1130 us with 6).  The
// exponent of 2 is -g log2(e); its rounding is an error of |g| 2^-24 of the result, up to 6e-6, which is far
// below the rounding to 16 bits but not below that to FP32: there (kExact), and for rows on their way to
// INT8, the exponent is in two parts.  The hardware's reciprocal is 0 where it would be subnormal, for sums past
// 2^126 (g < -87.3): so it is taken of a 16th of the sum, and a 16th of it is rounded once there, 2^-22 of the
// result at most (the one operation more is within the noise at those rows).  exp overflows to infinity for g < -88.7, which gives the limit -0; g = -inf is NaN.
template <bool kExact>
__device__ __forceinline__ float swiglu_fast(float g, float u) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eRest = 1.925963033500011e-8f, kLn2 = 0.693147180559945f;
  constexpr float kPart = 0.0625f;
  const float x = -g * kLog2e;
  const float e = __builtin_amdgcn_exp2f(x);
  float part;  // (1 + exp(-g)) / 16
  if constexpr (kExact) {
    const float rest = __builtin_fmaf(-g, kLog2eRest, __builtin_fmaf(-g, kLog2e, -x));
    // at most 2^-16 where e matters; the bound is for g = inf, whose rest is NaN
    part = __builtin_fmaf(e, __builtin_fmaf(fminf(fmaxf(rest, -0.001f), 0.001f), kLn2 * kPart, kPart), kPart);
  } else {
    part = __builtin_fmaf(e, kPart, kPart);
  }
  return g * (__builtin_amdgcn_rcpf(part) * kPart) * u;
}

// The largest |v| of the 16 columns that the four lanes r, r + 16, .. hold, as FP32 bits (NaN largest).
__device__ __forceinline__ uint32_t fragment_max(const f32x4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  m = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  return max(b[0], b[1]);
}

// What a product writes: results of a type, or held rows.
template <class T> struct Scaled { static constexpr bool kHeld = false, kExact = T::kBytes == 4; using Out = T; };
struct Held { static constexpr bool kHeld = true, kExact = true; using Out = TF32; };

// Rows on their way to INT8 are held in FP32, with the largest |v| of each 16 columns beside them, so that
// the kernel that makes them INT8 knows a row's scale without reading the row first.  Held in 16 bits
// (whole numbers of 1 / 32767 of that largest value) they cost half the traffic, 16384 rows by 4096
// outputs over 1024 300 us instead of 335, but one element in some hundreds then lies on the other
// side of a rounding, 18 times the error of FP32 rows.
__device__ __forceinline__ void store_largest(const Mm8Args& a, const f32x4& v, int64_t row, int64_t n, bool in) {
  const uint32_t m = fragment_max(v);
  if (in && n % 16 == 0) a.held_max[row * (a.F / 16) + n / 16] = __uint_as_float(m);
}

template <int WM, int WN, int MF>
struct Tile8Shape {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kNF = 16 / WN;              // column fragments of a wave: 256 columns in all
  static constexpr int kBM = WM * MF * 16;
  static constexpr int kXCopies = kBM / 8 / (WM * WN), kWCopies = 256 / 8 / (WM * WN);  // of 8 rows
  static constexpr bool kAhead = MF >= 4;          // fragments are read half a step ahead (see mm8_tile)
  static constexpr int kXBuffers = kAhead ? 3 : 2, kWBuffers = 2;
  static constexpr int kLds = (kXBuffers * kBM + kWBuffers * 256) * kBlk;
  static_assert(kBM % (8 * WM * WN) == 0 && 256 % (8 * WM * WN) == 0, "every wave copies the same number of rows");
};

template <class T, int EPI, int WM, int WN, int MF>
__device__ __forceinline__ void mm8_tile(const Mm8Args& a, const RowTile& rt, int32_t c, char* lds) {
  using S = Tile8Shape<WM, WN, MF>;
  constexpr bool kSwiglu = EPI == FFNWB_EPI_SWIGLU;
  constexpr int NF = S::kNF, kWaves = WM * WN;
  const int32_t kb = a.kb;
  const int32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), r = lane % 16, g = lane / 16;
  const int32_t wm = wave / WN, wn = wave % WN;
  const int64_t c0 = static_cast<int64_t>(c) * (kSwiglu ? 128 : 256);  // first output column
  // weight row of LDS row q: of a wave's 16 NF columns the first half are gate, the rest up
  auto weight_row = [&](int32_t q) -> int64_t {
    if constexpr (kSwiglu) {
      const int32_t half = NF * 8, t = q % (2 * half);
      const int64_t f = min(c0 + q / (2 * half) * half + t % half, a.F - 1);
      return t < half ? f : a.F + f;
    } else {
      return min(c0 + q, a.N - 1);
    }
  };
  // Copy j of a wave takes 8 rows, one chunk per lane: 32-bit offsets from the tile's first rows
  // (256 rows of x, and of w as far as the up columns, are below 2^32 bytes in this kernel).
  const int64_t w0 = weight_row(0);
  const Buffer xbuf = make_buffer(a.x + rt.row0 * a.xs, (rt.rows - 1) * a.xs + a.K);
  const Buffer wbuf = make_buffer(a.w + (static_cast<int64_t>(rt.expert) * a.N + w0) * a.K, (a.N - w0) * a.K);
  const uint32_t chunk = ((lane % 8) ^ (lane / 8)) * 16;
  uint32_t xsrc[S::kXCopies], wsrc[S::kWCopies];
#pragma unroll
  for (int j = 0; j < S::kXCopies; ++j)
    xsrc[j] = chunk + static_cast<uint32_t>(min((j * kWaves + wave) * 8 + lane / 8, rt.rows - 1) * a.xs);
#pragma unroll
  for (int j = 0; j < S::kWCopies; ++j)
    wsrc[j] = chunk + static_cast<uint32_t>((weight_row((j * kWaves + wave) * 8 + lane / 8) - w0) * a.K);
  char* const xlds = lds;
  char* const wlds = lds + S::kXBuffers * S::kBM * kBlk;
  auto fetch_x = [&](int32_t b) {
    char* to = xlds + b % S::kXBuffers * S::kBM * kBlk;
#pragma unroll
    for (int j = 0; j < S::kXCopies; ++j) copy16_to_lds(xbuf, xsrc[j], b * kBlk, to + (j * kWaves + wave) * 1024);
  };
  auto fetch_w = [&](int32_t b) {
    char* to = wlds + b % S::kWBuffers * 256 * kBlk;
#pragma unroll
    for (int j = 0; j < S::kWCopies; ++j) copy16_to_lds(wbuf, wsrc[j], b * kBlk, to + (j * kWaves + wave) * 1024);
  };
  // fragments: 64 columns, the first (s = 0) or second half of a block
  const int32_t at = r * kBlk + (g ^ (r & 7)) * 16;
  auto read_x = [&](int32_t b, int s, int i) {
    return *reinterpret_cast<const u32x4*>(xlds + b % S::kXBuffers * S::kBM * kBlk + (wm * MF + i) * 16 * kBlk + (at ^ (s * 64)));
  };
  auto read_w = [&](int32_t b, int s, int f) {
    return *reinterpret_cast<const u32x4*>(wlds + b % S::kWBuffers * 256 * kBlk + (wn * NF + f) * 16 * kBlk + (at ^ (s * 64)));
  };
  // In the last block the columns past K (of the next row, or not there) count as zeros: clearing
  // them in x is enough.
  const int32_t left = static_cast<int32_t>(a.K) - (kb - 1) * kBlk - g * 16;
  auto clear_past = [&](int s, u32x4& v) {
    if (left <= s * 64) v = u32x4{0, 0, 0, 0};
  };

  // The scales of the wave's rows and columns: ahead of the first copies, among the last products where
  // registers are short, or behind them in tiles of 256 rows, which have none left (24 scales ahead of the last block took
  // 35 registers' way through memory: 131072 rows of 128 experts to INT8 1338 -> 1235 us, 40000 rows by 4096 columns over 512 184 -> 138).
  float xs[MF];
  f32x4 ws[NF];
  const int64_t n0 = c0 + wn * (kSwiglu ? NF * 8 : NF * 16) + g * 4;  // the lane's first column of fragment 0
  auto scales = [&] {
#pragma unroll
    for (int i = 0; i < MF; ++i) xs[i] = a.x_scale[(rt.row0 + min((wm * MF + i) * 16 + r, rt.rows - 1)) * a.xss];
#pragma unroll
    for (int f = 0; f < NF; ++f)
      ws[f] = channel_scales(a, rt.expert, kSwiglu && f >= NF / 2 ? a.F + n0 + (f - NF / 2) * 16 : n0 + f * 16);
  };
  if constexpr (!S::kAhead) scales();
  fetch_x(0);
  fetch_w(0);
  if (kb > 1) {
    fetch_x(1);
    if constexpr (S::kAhead) fetch_w(1);
  }
  i32x4 tot[MF][NF] = {};
  if constexpr (S::kAhead) {
    // A block's two halves are multiplied from fragments read before: w's in the half before, x's two
    // ahead.  Halfway through the first half every wave is done with block b - 1, and x of block b + 2 takes
    // its buffer; halfway through the second, w of block b is in registers, and w of block b + 2 takes its
    // buffer, once block b + 1 has landed for every wave.  So x has 1.5 steps to arrive and w one.
    u32x4 wv[2][NF], xv[3];
    copies_done<S::kXCopies + S::kWCopies>(kb > 1);
#pragma unroll
    for (int f = 0; f < NF; ++f) wv[0][f] = read_w(0, 0, f);
    xv[0] = read_x(0, 0, 0), xv[1] = read_x(0, 0, 1);
    auto block = [&](int32_t b, auto last) {
      constexpr bool kLast = decltype(last)::value;
#pragma unroll
      for (int n = 0; n < 2 * MF; ++n) {
        const int s = n / MF, i = n % MF;
        if (!kLast && n == MF / 2) {
          lds_barrier();
          if (b + 2 < kb) fetch_x(b + 2);
        }
        if (!kLast && n == MF + MF / 2) {
          copies_done<S::kXCopies>(b + 2 < kb);
          if (b + 2 < kb) fetch_w(b + 2);
        }
        if (n + 2 < 2 * MF) xv[2] = read_x(b, (n + 2) / MF, (n + 2) % MF);
        else if (!kLast) xv[2] = read_x(b + 1, 0, n + 2 - 2 * MF);
        if (kLast) clear_past(s, xv[0]);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          if (i == MF / 2) {
            if (s == 0) wv[1][f] = read_w(b, 1, f);
            else if (!kLast) wv[0][f] = read_w(b + 1, 0, f);
          }
          tot[i][f] = mul_int8(wv[s][f], xv[0], tot[i][f]);
        }
        xv[0] = xv[1], xv[1] = xv[2];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction,
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int32_t b = 0; b + 1 < kb; ++b) block(b, std::false_type{});
    if constexpr (MF < 8) scales();
    block(kb - 1, std::true_type{});
    if constexpr (MF >= 8) scales();
  } else {
    // w of the next block is on its way since the step before, x since the start of this one, and the
    // fragments of w go to registers first, which frees their buffer for the block after next.
    if (kb > 1) fetch_w(1);
    copies_done<S::kXCopies + S::kWCopies>(kb > 1);
    for (int32_t b = 0; b < kb; ++b) {
      u32x4 wv[2][NF];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int f = 0; f < NF; ++f) wv[s][f] = read_w(b, s, f);
      u32x4 xv[2][MF];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          xv[s][i] = read_x(b, s, i);
          if (b == kb - 1) clear_past(s, xv[s][i]);
        }
      if (b + 2 < kb) {
        lds_barrier();  // every wave has its fragments
        fetch_x(b + 2);
        fetch_w(b + 2);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int f = 0; f < NF; ++f) tot[i][f] = mul_int8(wv[s][f], xv[s][i], tot[i][f]);
      copies_done<S::kXCopies + S::kWCopies>(b + 2 < kb);
    }
  }

  // Results go from registers to memory: a lane holds 4 adjacent columns of a row, in 16-bit types 8 after
  // an exchange between two fragments, so that a store writes 64 adjacent bytes of 16 rows.
  constexpr int OF = kSwiglu ? NF / 2 : NF;  // result fragments of a wave
  const int64_t limit = kSwiglu ? a.F : a.N;
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    __builtin_amdgcn_sched_barrier(0);  // one row fragment after another: few registers
    const int32_t row = (wm * MF + i) * 16 + r;
    char* y = a.y + (rt.row0 + min(row, rt.rows - 1)) * a.ys;
    const bool in = row < rt.rows;
    using Out = typename T::Out;
    f32x4 v[OF];
#pragma unroll
    for (int f = 0; f < OF; ++f) {
      v[f] = scaled(tot[i][f], xs[i], ws[f]);
      if constexpr (kSwiglu) {
        const f32x4 up = scaled(tot[i][OF + f], xs[i], ws[OF + f]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[f][j] = swiglu_fast<T::kExact>(v[f][j], up[j]);
      }
    }
    if constexpr (Out::kBytes == 4) {
#pragma unroll
      for (int f = 0; f < OF; ++f) {
        const int64_t n = n0 + f * 16;
        char* to = y + n * 4;
        if constexpr (T::kHeld) store_largest(a, v[f], rt.row0 + row, n, in && n < limit);
        if (in && n + 4 <= limit) {
          *reinterpret_cast<u32x4_a4*>(to) = __builtin_bit_cast(u32x4, v[f]);
        } else if (in) {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (n + j < limit) reinterpret_cast<float*>(to)[j] = v[f][j];
        }
      }
    } else {
#pragma unroll
      for (int f = 0; f < OF; f += 2) {
        uint32_t p[2] = {narrow2<Out>(v[f][0], v[f][1]), narrow2<Out>(v[f][2], v[f][3])};
        uint32_t q[2] = {narrow2<Out>(v[f + 1][0], v[f + 1][1]), narrow2<Out>(v[f + 1][2], v[f + 1][3])};
        join_columns(p[0], q[0]);
        join_columns(p[1], q[1]);
        const int64_t n = n0 + f * 16 + g * 4;  // n0 holds 4 g, the lane's columns start at 8 g
        char* to = y + n * 2;
        if (in && n + 8 <= limit) {
          *reinterpret_cast<u32x4_a1*>(to) = u32x4{p[0], p[1], q[0], q[1]};
        } else if (in) {
          const uint32_t w[4] = {p[0], p[1], q[0], q[1]};
#pragma unroll
          for (int j = 0; j < 7; ++j)
            if (n + j < limit) reinterpret_cast<uint16_t*>(to)[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
        }
      }
    }
  }
}

// Tiles of at most half the rows (the last one of a group, the halves of find_tile) take half the
// fragments.  Two workgroups of 64 rows share a CU: 4 waves to a SIMD, 128 registers, for which 5 of the kernel
// with FP32 results pass through memory (24 bytes a lane; 16189 rows by 7922 columns over 1216, FP32: 319 us,
// 380 with 135 registers and none in memory).
template <class T, int EPI, int WM, int WN, int MF>
__global__ __launch_bounds__(WM* WN* kWave, MF == 2 && WM == 2 ? 4 : 2) void mm8_tile_kernel(Mm8Args a) {
  extern __shared__ __align__(16) char lds8[];
  constexpr int kBM = Tile8Shape<WM, WN, MF>::kBM;
  RowTile rt;
  int32_t c;
  if (!find_tile<(MF >= kHalvedFragments)>(a, kBM, rt, c)) return;
  if constexpr (MF >= kHalvedFragments) {
    if (rt.rows <= kBM / 2) {
      mm8_tile<T, EPI, WM, WN, MF / 2>(a, rt, c, lds8);
      return;
    }
  }
  mm8_tile<T, EPI, WM, WN, MF>(a, rt, c, lds8);
}

}  // namespace ffnwb
