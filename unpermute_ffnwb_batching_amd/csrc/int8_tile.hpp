// Tiles of the INT8 products through LDS (matmul_int8.hip).
//
// A workgroup of WM x WN waves takes BM = 16 WM MF rows by 256 columns (SwiGLU: 128 gate columns
// and the 128 up columns that go with them, half and half in every wave), 64 columns of K to a
// step.  Both operands go from memory to LDS without passing through registers (16 bytes per
// lane), kBuffers steps deep.  A row of a step is 64 bytes, 4 chunks of 16; chunk c of row r lies at
// position c ^ (r / 2 % 4), which spreads the 16 rows that a matrix operand reads at once over
// all banks.  The lanes of a copy write adjacent LDS addresses, so the permutation is applied to
// the addresses they read.
#pragma once

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
  int32_t parts, part_blocks;  // parts of K, each a workgroup's, and blocks of a part
  int64_t part_bytes;          // between the results of two parts
  int32_t ngroups, nexperts;
  bool vec;                    // four adjacent outputs are one aligned store
  int32_t unit;                // rows of y are whole aligned units of 16 or 4 bytes, or elements (0)
  const char* x;
  const float* x_scale;
  const char* w;
  const float* w_scale;
  char* y;
  float* y_scale;
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

// What a tile writes: whole-number sums, or scaled results of a type.
struct Whole { static constexpr bool kWhole = true; static constexpr int kBytes = 4; };
template <class T> struct Scaled { static constexpr bool kWhole = false; static constexpr int kBytes = T::kBytes; using Out = T; };

constexpr int kStep = 64;  // columns of K to a step

template <int WM, int WN, int MF>
struct Tile8Shape {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kNF = 16 / WN;              // column fragments of a wave: 256 columns in all
  static constexpr int kBM = WM * MF * 16;
  static constexpr int kRows = kBM + 256;          // rows of a buffer, x then w
  static constexpr int kXCopies = (kBM / 16 + WM * WN - 1) / (WM * WN), kWCopies = 256 / 16 / (WM * WN);  // of 16 rows
  static constexpr int kBuffers = 4;
  static constexpr int kLds = kBuffers * kRows * kStep;
  static_assert(kBM % 16 == 0 && 256 % (16 * WM * WN) == 0, "whole copies");
};

template <class T, int EPI, int WM, int WN, int MF>
__device__ __forceinline__ void mm8_tile(const Mm8Args& a, const RowTile& rt, int32_t c, char* lds) {
  using S = Tile8Shape<WM, WN, MF>;
  constexpr bool kSwiglu = EPI == FFNWB_EPI_SWIGLU;
  constexpr int NF = S::kNF, NB = S::kBuffers, kWaves = WM * WN;
  // this workgroup's part of K, in columns
  const int32_t part = c % a.parts, k0 = part * a.part_blocks * kBlk;
  const int32_t columns = min(static_cast<int32_t>(a.K) - k0, a.part_blocks * kBlk), steps = (columns + kStep - 1) / kStep;
  c /= a.parts;
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
  // Copy j of a wave takes 16 rows, one chunk per lane: 32-bit offsets from the tile's first rows
  // (256 rows of x, and of w as far as the up columns, are below 2^32 bytes in this kernel).
  const int64_t w0 = weight_row(0);
  const Buffer xbuf = make_buffer(a.x + rt.row0 * a.xs + k0, (rt.rows - 1) * a.xs + a.K - k0);
  const Buffer wbuf = make_buffer(a.w + (static_cast<int64_t>(rt.expert) * a.N + w0) * a.K + k0, (a.N - w0) * a.K - k0);
  const uint32_t chunk = ((lane % 4) ^ (lane / 8 % 4)) * 16;
  uint32_t xsrc[S::kXCopies], wsrc[S::kWCopies];
#pragma unroll
  for (int j = 0; j < S::kXCopies; ++j)
    xsrc[j] = chunk + static_cast<uint32_t>(min((j * kWaves + wave) % (S::kBM / 16) * 16 + lane / 4, rt.rows - 1) * a.xs);
#pragma unroll
  for (int j = 0; j < S::kWCopies; ++j)
    wsrc[j] = chunk + static_cast<uint32_t>((weight_row((j * kWaves + wave) * 16 + lane / 4) - w0) * a.K);
  // Waves that no rows of x are left for fetch the first rows once more, to where those lie: every
  // wave has the same number of copies on its way.
  auto fetch = [&](int32_t b) {
    char* to = lds + b % NB * S::kRows * kStep;
#pragma unroll
    for (int j = 0; j < S::kXCopies; ++j) copy16_to_lds(xbuf, xsrc[j], b * kStep, to + (j * kWaves + wave) % (S::kBM / 16) * 1024);
#pragma unroll
    for (int j = 0; j < S::kWCopies; ++j) copy16_to_lds(wbuf, wsrc[j], b * kStep, to + S::kBM * kStep + (j * kWaves + wave) * 1024);
  };
  constexpr int kCopies = S::kXCopies + S::kWCopies;
#pragma unroll
  for (int b = 0; b < NB - 1; ++b)
    if (b < steps) fetch(b);

  // Step b: once its operands have landed for every wave, which also means that every wave is done
  // with step b - 1, the buffer of that one takes step b + NB - 1.
  i32x4 tot[MF][NF] = {};
  for (int32_t b = 0; b < steps; ++b) {
    copies_done<(NB - 2) * kCopies>(b + NB - 2 < steps);
    if (b + NB - 1 < steps) fetch(b + NB - 1);
    const char* xb = lds + b % NB * S::kRows * kStep;
    const char* wb = xb + S::kBM * kStep;
    const int32_t at = r * kStep + (g ^ (r / 2 % 4)) * 16;
    u32x4 wv[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) wv[f] = *reinterpret_cast<const u32x4*>(wb + (wn * NF + f) * 16 * kStep + at);
    const bool past = b * kStep + g * 16 >= columns;  // columns past K: of the next row, or not there
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      u32x4 xv = *reinterpret_cast<const u32x4*>(xb + (wm * MF + i) * 16 * kStep + at);
      if (past) xv = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int f = 0; f < NF; ++f) tot[i][f] = mul_int8(wv[f], xv, tot[i][f]);
    }
  }
  __syncthreads();

  // Results go through LDS, so that memory sees whole lines: a matrix result is 16 rows by 4
  // adjacent columns per lane.  Row r of the tile is kPitch bytes, its 16-byte chunks at
  // position c ^ (r % 8).
  constexpr int kElt = T::kBytes;
  constexpr int kCols = kSwiglu ? 128 : 256, kPitch = kCols * kElt;
  constexpr int OF = kSwiglu ? NF / 2 : NF;  // result fragments of a wave
  const int64_t limit = kSwiglu ? a.F : a.N;
  // FP32 tiles of many rows are wider than the buffers: some of the waves' fragments at a time.
  constexpr int kParts = (S::kBM * kPitch + S::kLds - 1) / S::kLds <= 1 ? 1 : (S::kBM * kPitch + S::kLds - 1) / S::kLds <= 2 ? 2 : 4;
  constexpr int kPartF = MF / kParts, kPartRows = S::kBM / kParts;
  static_assert(MF % kParts == 0, "a part is some of the fragments of every wave");
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    if (p > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < kPartF; ++i) {
      const int32_t row = (wm * kPartF + i) * 16 + r;  // of the part
      float xs = 0.0f;
      if constexpr (!T::kWhole) xs = a.x_scale[(rt.row0 + min((wm * MF + p * kPartF + i) * 16 + r, rt.rows - 1)) * a.xss];
#pragma unroll
      for (int f = 0; f < OF; ++f) {
        const int32_t byte = ((wn * OF + f) * 16 + g * 4) * kElt;  // of the row
        char* to = lds + row * kPitch + ((byte / 16 ^ (row & 7)) * 16 + byte % 16);
        const i32x4& t = tot[p * kPartF + i][f];
        if constexpr (T::kWhole) {
          *reinterpret_cast<i32x4*>(to) = t;
        } else {
          const int64_t n = c0 + (wn * OF + f) * 16 + g * 4;
          f32x4 v = scaled(t, xs, channel_scales(a, rt.expert, n));
          if constexpr (kSwiglu) {
            const f32x4 up = scaled(tot[p * kPartF + i][OF + f], xs, channel_scales(a, rt.expert, a.F + n));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = swiglu(v[j], up[j]);
          }
          if constexpr (kElt == 2) {
            const float w[8] = {v[0], v[1], v[2], v[3], 0, 0, 0, 0};
            const u32x4 h = Chunk<typename T::Out>::narrow(w);
            *reinterpret_cast<u32x2*>(to) = u32x2{h[0], h[1]};
          } else {
            *reinterpret_cast<f32x4*>(to) = v;
          }
        }
      }
    }
    __syncthreads();
    const int32_t bytes = static_cast<int32_t>(min(limit - c0, int64_t{kCols})) * kElt;  // of a row
    // rows of a part: kPartF * 16 of every wave row
#pragma unroll
    for (int w = 0; w < (kParts == 1 ? 1 : WM); ++w) {
      const int32_t first = kParts == 1 ? 0 : w * MF * 16 + p * kPartF * 16;
      const int32_t rows = min(rt.rows - first, kParts == 1 ? S::kBM : kPartF * 16);
      char* y = a.y + part * a.part_bytes + (rt.row0 + first) * a.ys + c0 * kElt;
      const char* from = lds + (kParts == 1 ? 0 : w * kPartF * 16 * kPitch);
      if (a.unit == 16) copy_out<16, kPitch, S::kThreads>(from, y, a.ys, rows, bytes);
      else if (a.unit == 4) copy_out<4, kPitch, S::kThreads>(from, y, a.ys, rows, bytes);
      else copy_out<kElt, kPitch, S::kThreads>(from, y, a.ys, rows, bytes);
    }
  }
  (void)kPartRows;
}

// Tiles of at most half the rows (the last one of a group, the halves of find_tile) take half the
// fragments.
template <class T, int EPI, int WM, int WN, int MF>
__global__ __launch_bounds__(WM* WN* kWave) void mm8_tile_kernel(Mm8Args a) {
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
