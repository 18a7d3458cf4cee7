// Tiles of the experts' products through LDS (grouped_matmul.hip).
//
// A workgroup of WM x WN waves takes BM = 16 WM MF rows by 256 columns (SwiGLU: 128 gate columns
// and the 128 up columns that go with them, half and half in every wave), one 128-column block
// of K per step.  Both operands go from memory to LDS without passing through registers
// (16 bytes per lane), into the other of two buffers while one is being multiplied.  A row of a
// tile is 128 bytes, 8 chunks of 16; chunk c of row r lies at position c ^ (r % 8), which spreads the
// 16 rows a matrix operand reads at once over all banks.  The lanes of a copy write adjacent LDS
// addresses, so the permutation is applied to the addresses they read.
#pragma once

#include "fp8_block.hpp"

namespace ffnwb {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Over 128 e4m3 columns: D = A B.
__device__ __forceinline__ f32x4 mul_e4m3(const u32x4 (&a)[2], const u32x4 (&b)[2]) {
  const i32x8 av = {static_cast<int>(a[0][0]), static_cast<int>(a[0][1]), static_cast<int>(a[0][2]), static_cast<int>(a[0][3]),
                    static_cast<int>(a[1][0]), static_cast<int>(a[1][1]), static_cast<int>(a[1][2]), static_cast<int>(a[1][3])};
  const i32x8 bv = {static_cast<int>(b[0][0]), static_cast<int>(b[0][1]), static_cast<int>(b[0][2]), static_cast<int>(b[0][3]),
                    static_cast<int>(b[1][0]), static_cast<int>(b[1][1]), static_cast<int>(b[1][2]), static_cast<int>(b[1][3])};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

// 16 bytes per lane from `src` to LDS at `dst` + 16 * lane; `dst` is the same in all lanes.
__device__ __forceinline__ void copy16_to_lds(const char* src, char* dst) {
  __builtin_amdgcn_global_load_lds(reinterpret_cast<const __attribute__((address_space(1))) void*>(reinterpret_cast<uintptr_t>(src)),
                                   reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(dst)),
                                   16, 0, 0);
}

// All of this wave's copies have landed, then all waves' have.
__device__ __forceinline__ void copies_done() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

__device__ const u32x4 kZeroChunk = {0, 0, 0, 0};

template <int WM, int WN, int MF>
struct TileShape {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kNF = 16 / WN;              // column fragments of a wave: 256 columns in all
  static constexpr int kBM = WM * MF * 16;
  static constexpr int kRows = kBM + 256;          // rows of a buffer, x then w
  static constexpr int kCopies = kRows / 8 / (WM * WN);
  static constexpr int kScaleRuns = 8;             // blocks of the scales held at once
  static constexpr int kScales = kBM + 16;         // scales of a block: rows of x, then column fragments
  static constexpr int kScaleLoads = (kScales * kScaleRuns + kThreads - 1) / kThreads;
  static constexpr int kLds = 2 * kRows * kBlk + 2 * kScales * kScaleRuns * 4;
  static_assert(kRows % (8 * WM * WN) == 0, "every wave copies the same number of rows");
};

// kFast: e4m3 matrix instructions; else the operands are widened to BF16 (see fp8_block.hpp).
template <class T, int EPI, bool kQuant, bool kFast, int WM, int WN, int MF>
__global__ __launch_bounds__(WM* WN* kWave) void mm_tile_kernel(MmArgs a) {
  using S = TileShape<WM, WN, MF>;
  constexpr bool kSwiglu = EPI == FFNWB_EPI_SWIGLU;
  constexpr int NF = S::kNF;
  extern __shared__ __align__(16) char lds[];
  float* xsl = reinterpret_cast<float*>(lds + 2 * S::kRows * kBlk);  // [2][kScaleRuns][kScales]

  RowTile rt;
  int32_t c;
  if (!find_tile(a, S::kBM, rt, c)) return;
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
  // 32-bit offsets from the tile's first rows (256 rows of x are below 2^31 bytes)
  const char* xbase = a.x + rt.row0 * a.xs;
  const char* wbase = a.w + static_cast<int64_t>(rt.expert) * a.N * a.K;
  uint32_t src[S::kCopies];
#pragma unroll
  for (int j = 0; j < S::kCopies; ++j) {
    const int32_t row = (j * WM * WN + wave) * 8 + lane / 8;
    src[j] = ((lane % 8) ^ (lane / 8)) * 16 +
             static_cast<uint32_t>(row < S::kBM ? min(row, rt.rows - 1) * a.xs : weight_row(row - S::kBM) * a.K);
  }
  const int32_t tail = static_cast<int32_t>(a.K % kBlk);  // columns of a short last block
  auto fetch = [&](int32_t b) {
    char* to = lds + (b & 1) * S::kRows * kBlk;
    const int32_t k0 = b * kBlk;
    if (tail != 0 && b == a.kb - 1) {
      const bool cut = ((lane % 8) ^ (lane / 8)) * 16 >= tail;
#pragma unroll
      for (int j = 0; j < S::kCopies; ++j) {
        const char* p = ((j * WM * WN + wave) * 8 < S::kBM ? xbase : wbase) + k0 + src[j];
        copy16_to_lds(cut ? reinterpret_cast<const char*>(&kZeroChunk) : p, to + (j * WM * WN + wave) * 1024);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S::kCopies; ++j)
        copy16_to_lds(((j * WM * WN + wave) * 8 < S::kBM ? xbase : wbase) + k0 + src[j], to + (j * WM * WN + wave) * 1024);
    }
  };
  // The scales of 8 blocks at a time, 8 lanes per row of x or column fragment of w; they go
  // through registers to LDS 6 blocks later, held [block][row].  A fragment's 16 columns lie in
  // one block of w_scale.
  float scr[S::kScaleLoads];
  const float* scp[S::kScaleLoads];
#pragma unroll
  for (int j = 0; j < S::kScaleLoads; ++j) {
    const int32_t i = (j * S::kThreads + static_cast<int32_t>(threadIdx.x)) / S::kScaleRuns;
    scp[j] = i < S::kBM ? a.x_scale + (rt.row0 + min(i, rt.rows - 1)) * a.xss
                        : a.w_scale + (static_cast<int64_t>(rt.expert) * a.nb + weight_row(min(i - S::kBM, 15) * 16) / kBlk) * a.kb;
  }
  auto scales_load = [&](int32_t b0) {
    const int32_t b = min(b0 + static_cast<int32_t>(threadIdx.x) % S::kScaleRuns, a.kb - 1);
#pragma unroll
    for (int j = 0; j < S::kScaleLoads; ++j) scr[j] = scp[j][b];
  };
  auto scales_store = [&](int32_t b0) {
    float* to = xsl + ((b0 / S::kScaleRuns & 1) * S::kScaleRuns + threadIdx.x % S::kScaleRuns) * S::kScales;
#pragma unroll
    for (int j = 0; j < S::kScaleLoads; ++j) {
      const int32_t i = (j * S::kThreads + static_cast<int32_t>(threadIdx.x)) / S::kScaleRuns;
      if (i < S::kScales) to[i] = scr[j];
    }
  };

  fetch(0);
  scales_load(0);
  scales_store(0);
  copies_done();

  f32x4 tot[MF][NF] = {};
  for (int32_t b = 0; b < a.kb; ++b) {
    const int32_t turn = b % S::kScaleRuns, next = b - turn + S::kScaleRuns;
    if (turn == S::kScaleRuns - 2 && next < a.kb) scales_store(next);
    if (turn == 0 && next < a.kb) scales_load(next);
    if (b + 1 < a.kb) fetch(b + 1);
    // one stretch of code from here to the end of the step, in the order written
    const char* buf = lds + (b & 1) * S::kRows * kBlk;
    const float* scb = xsl + ((b / S::kScaleRuns & 1) * S::kScaleRuns + turn) * S::kScales;
    constexpr int NS = kSwiglu ? NF : 1;  // without SwiGLU a wave's columns lie in one block of 128
    float ws[NS];
#pragma unroll
    for (int f = 0; f < NS; ++f) ws[f] = scb[S::kBM + wn * NF + f];
    const int32_t ch0 = (g ^ (r & 7)) * 16, ch1 = ((4 + g) ^ (r & 7)) * 16;
    u32x4 wf[NF][kFast ? 2 : 4];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const char* row = buf + (S::kBM + (wn * NF + f) * 16 + r) * kBlk;
      const u32x4 v0 = *reinterpret_cast<const u32x4*>(row + ch0), v1 = *reinterpret_cast<const u32x4*>(row + ch1);
      if constexpr (kFast) {
        wf[f][0] = v0, wf[f][1] = v1;
      } else {
        wf[f][0] = widen8(v0[0], v0[1]), wf[f][1] = widen8(v0[2], v0[3]);
        wf[f][2] = widen8(v1[0], v1[1]), wf[f][3] = widen8(v1[2], v1[3]);
      }
    }
    // fragment i + 1 of x is read while i is multiplied; the other wave of the SIMD multiplies
    // while this one scales its sums
    u32x4 xv[2][2];
    auto read = [&](int i) {
      const char* row = buf + ((wm * MF + i) * 16 + r) * kBlk;
      xv[i & 1][0] = *reinterpret_cast<const u32x4*>(row + ch0);
      xv[i & 1][1] = *reinterpret_cast<const u32x4*>(row + ch1);
    };
    read(0);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if (i + 1 < MF) read(i + 1);
      const float xs = scb[(wm * MF + i) * 16 + r];
      f32x4 p[NF];
      const u32x4 v0 = xv[i & 1][0], v1 = xv[i & 1][1];
      if constexpr (kFast) {
        const u32x4 xf[2] = {v0, v1};
#pragma unroll
        for (int f = 0; f < NF; ++f) p[f] = mul_e4m3(wf[f], xf);
      } else {
        const u32x4 xf[4] = {widen8(v0[0], v0[1]), widen8(v0[2], v0[3]), widen8(v1[0], v1[1]), widen8(v1[2], v1[3])};
#pragma unroll
        for (int f = 0; f < NF; ++f) p[f] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int f = 0; f < NF; ++f) p[f] = Mat<TBF16>::mul(wf[f][s], xf[s], p[f]);
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const float s = xs * ws[kSwiglu ? f : 0];
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[i][f][j] = __builtin_fmaf(s, p[f][j], tot[i][f][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    copies_done();
  }

  if constexpr (!kSwiglu) {
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int32_t row = (wm * MF + i) * 16 + r;
      if (row >= rt.rows) continue;
      char* y = a.y + (rt.row0 + row) * a.ys;
#pragma unroll
      for (int f = 0; f < NF; ++f) store4<T>(y, c0 + (wn * NF + f) * 16 + g * 4, a.N, tot[i][f], a.vec);
    }
  } else {
    constexpr int HF = NF / 2;  // output fragments of a wave
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < HF; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[i][f][j] = swiglu(tot[i][f][j], tot[i][HF + f][j]);
    const int64_t f0 = c0 + wn * HF * 16 + g * 4;
    if constexpr (!kQuant) {
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int32_t row = (wm * MF + i) * 16 + r;
        if (row >= rt.rows) continue;
        char* y = a.y + (rt.row0 + row) * a.ys;
#pragma unroll
        for (int f = 0; f < HF; ++f) store4<T>(y, f0 + f * 16, a.F, tot[i][f], a.vec);
      }
    } else {
      // the row's largest |h| over the tile's 128 columns, one block: lanes, then waves
      uint32_t* amax = reinterpret_cast<uint32_t*>(lds);  // [kBM][WN]
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        uint32_t big = 0;
#pragma unroll
        for (int f = 0; f < HF; ++f)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (f0 + f * 16 < a.F) big = max(big, __float_as_uint(tot[i][f][j]) & 0x7fffffffu);
        big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 16)));
        big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 32)));
        if (g == 0) amax[((wm * MF + i) * 16 + r) * WN + wn] = big;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int32_t row = (wm * MF + i) * 16 + r;
        uint32_t big = 0;
#pragma unroll
        for (int w = 0; w < WN; ++w) big = max(big, amax[row * WN + w]);
        const float s = block_scale(big);
        if (row >= rt.rows) continue;
        char* y = a.y + (rt.row0 + row) * a.ys;
#pragma unroll
        for (int f = 0; f < HF; ++f) {
          float q[4] = {tot[i][f][0], tot[i][f][1], tot[i][f][2], tot[i][f][3]};
          block_quotients(q, s);
          const uint32_t v = pack_e4m3(q[0], q[1], q[2], q[3]);
          if (f0 + f * 16 >= a.F) continue;  // F is a multiple of 16
          char* to = y + f0 + f * 16;
          if (a.vec) {
            *reinterpret_cast<uint32_t*>(to) = v;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) to[j] = static_cast<char>((v >> (8 * j)) & 0xffu);
          }
        }
        if (wn == 0 && g == 0) a.y_scale[(rt.row0 + row) * a.yss + c] = s;
      }
    }
  }
}

}  // namespace ffnwb
