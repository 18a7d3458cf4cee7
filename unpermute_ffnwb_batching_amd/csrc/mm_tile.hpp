// Tiles of the experts' products through LDS (grouped_matmul.hip).
//
// A workgroup of WM x WN waves takes BM = 16 WM MF rows by 256 columns (SwiGLU: 128 gate columns
// and the 128 up columns that go with them, half and half in every wave), one 128-column block
// of K per step.  Both operands go from memory to LDS without passing through registers
// (16 bytes per lane), into the other of two buffers while one is being multiplied.  A row of a
// tile is 128 bytes, 8 chunks of 16; chunk c of row r lies at position c ^ (r % 8), which spreads the
// 16 rows a matrix operand reads at once over all banks.  The lanes of a copy write adjacent LDS
// addresses, so the permutation is applied to the addresses they read.
//
// What bounds it, measured on 256 rows: a step takes 1.64 to 1.73 us (4096 rows by 4096 columns, one
// round of tiles, over 1024 to 8192); its copies alone (64 KB a CU) 1.7, its arithmetic alone 1.5
// (2.86 PFLOP/s; a library's e4m3 product of 16384^3, without scales, runs at 3.1).  With weights
// fetched one step ahead instead of two, 128 rows took 16% and 64 rows 19% longer.  Besides its steps
// a call of one round takes 15 us: the launch, filling the buffers, storing the results.  8191 rows by
// 7168 columns over 5120: 297 to 304 us, 2.0 PFLOP/s.  Widened operands (FP32, e4m3 and exact results):
// the same product 530 us, 131072 rows by 2048 over 4096 2210 to 2250 us, 0.99 PFLOP/s; there the
// arithmetic alone takes 2170, without the conversions 1835.
// 256 groups of 17 rows (32-row tiles, two workgroups to a CU) run at 5.4 TB/s of weights.
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

// 16 bytes per lane, from a uniform base + lane offset + uniform offset, to LDS at `dst` + 16 *
// lane; `dst` is the same in all lanes.  Nothing is read from `bytes` past the base on.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer make_buffer(const char* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, static_cast<uint32_t>(min(bytes, int64_t{0xffffffff})),
                                           0x00027000);
}
__device__ __forceinline__ void copy16_to_lds(Buffer base, uint32_t lane_offset, uint32_t offset, char* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(dst)),
                                           16, lane_offset, offset, 0, 0);
}

// A barrier for the waves' LDS reads and writes, which leaves copies to LDS on their way:
// __syncthreads would wait for them too.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// This wave's copies have landed, all or (`some`, uniform) all but the last kLeft; then all
// waves' have.  The branch is inside the assembly: one in the compiler's sight would let it move
// the arithmetic of a step behind it, with every sum of the step held in registers until then.
template <int kLeft>
__device__ __forceinline__ void copies_done(bool some) {
  asm volatile("s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lsome%=\n\ts_waitcnt vmcnt(0)\n.Lsome%=:\n\ts_waitcnt vmcnt(%1)"
               ::"s"(uniform(static_cast<int32_t>(some))), "n"(kLeft) : "memory", "scc");
  lds_barrier();
}

template <int WM, int WN, int MF>
struct TileShape {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kNF = 16 / WN;              // column fragments of a wave: 256 columns in all
  static constexpr int kBM = WM * MF * 16;
  static constexpr int kRows = kBM + 256;          // rows of a buffer, x then w
  static constexpr int kXCopies = kBM / 8 / (WM * WN), kWCopies = 256 / 8 / (WM * WN);  // of 8 rows
  static constexpr int kScaleRuns = 8;             // blocks of the scales held at once
  static constexpr int kScales = kBM + 16;         // scales of a block: rows of x, then column fragments
  static constexpr int kScaleLoads = (kScales * kScaleRuns + kThreads - 1) / kThreads;
  static constexpr int kLds = 2 * kRows * kBlk + 2 * kScales * kScaleRuns * 4;
  static_assert(kBM % (8 * WM * WN) == 0 && 256 % (8 * WM * WN) == 0, "every wave copies the same number of rows");
};

// Rows of a tile from LDS to memory, U bytes per lane.
template <int U, int kPitch, int kThreads>
__device__ __forceinline__ void copy_out(const char* lds, char* y, int64_t stride, int32_t rows, int32_t bytes) {
  constexpr int kUnits = kPitch / U;
  for (int32_t i = threadIdx.x; i < rows * kUnits; i += kThreads) {
    const int32_t row = i / kUnits, at = i % kUnits * U;
    if (at >= bytes) continue;
    const char* from = lds + row * kPitch + ((at / 16 ^ (row & 7)) * 16 + at % 16);
    char* to = y + row * stride + at;
    if constexpr (U == 16) *reinterpret_cast<u32x4*>(to) = *reinterpret_cast<const u32x4*>(from);
    else if constexpr (U == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
    else if constexpr (U == 2) *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(from);
    else *to = *from;
  }
}

// kFast: e4m3 matrix instructions; else the operands are widened to BF16 (see fp8_block.hpp).
template <class T, int EPI, bool kQuant, bool kFast, int WM, int WN, int MF>
__device__ __forceinline__ void mm_tile(const MmArgs& a, const RowTile& rt, int32_t c, char* lds) {
  using S = TileShape<WM, WN, MF>;
  constexpr bool kSwiglu = EPI == FFNWB_EPI_SWIGLU;
  constexpr int NF = S::kNF;
  float* xsl = reinterpret_cast<float*>(lds + 2 * S::kRows * kBlk);  // [2][kScaleRuns][kScales]
  // this workgroup's part of K: kb blocks from block k0 on, all of them unless the product is split
  const int32_t part = c % a.parts, k0 = part * a.part_blocks, kb = min(a.kb - k0, a.part_blocks);
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
  // Copy j of a wave takes 8 rows, one chunk per lane: 32-bit offsets from the tile's first rows
  // (256 rows of x, and of w as far as the up columns, are below 2^32 bytes in this kernel).
  const int64_t w0 = weight_row(0);
  const int64_t kfirst = static_cast<int64_t>(k0) * kBlk;
  const Buffer xbuf = make_buffer(a.x + rt.row0 * a.xs + kfirst, (rt.rows - 1) * a.xs + a.K - kfirst);
  const Buffer wbuf = make_buffer(a.w + (static_cast<int64_t>(rt.expert) * a.N + w0) * a.K + kfirst, (a.N - w0) * a.K - kfirst);
  const uint32_t chunk = ((lane % 8) ^ (lane / 8)) * 16;
  uint32_t xsrc[S::kXCopies], wsrc[S::kWCopies];
#pragma unroll
  for (int j = 0; j < S::kXCopies; ++j)
    xsrc[j] = chunk + static_cast<uint32_t>(min((j * WM * WN + wave) * 8 + lane / 8, rt.rows - 1) * a.xs);
#pragma unroll
  for (int j = 0; j < S::kWCopies; ++j)
    wsrc[j] = chunk + static_cast<uint32_t>((weight_row((j * WM * WN + wave) * 8 + lane / 8) - w0) * a.K);
  // LDS: x of even and odd blocks, w of even and odd blocks, scales
  auto fetch_x = [&](int32_t b) {
    char* to = lds + (b & 1) * S::kBM * kBlk;
#pragma unroll
    for (int j = 0; j < S::kXCopies; ++j) copy16_to_lds(xbuf, xsrc[j], b * kBlk, to + (j * WM * WN + wave) * 1024);
  };
  auto fetch_w = [&](int32_t b) {
    char* to = lds + 2 * S::kBM * kBlk + (b & 1) * 256 * kBlk;
#pragma unroll
    for (int j = 0; j < S::kWCopies; ++j) copy16_to_lds(wbuf, wsrc[j], b * kBlk, to + (j * WM * WN + wave) * 1024);
  };
  // A short last block: the chunks past K (of the next row, or not there) become zeros.
  const int32_t full = k0 + kb == a.kb ? static_cast<int32_t>(a.K % kBlk) / 16 : 0;
  auto clear_tail = [&] {
    char* xb = lds + ((kb - 1) & 1) * S::kBM * kBlk;
    char* wb = lds + 2 * S::kBM * kBlk + ((kb - 1) & 1) * 256 * kBlk;
    for (int32_t i = threadIdx.x; i < S::kRows * (8 - full); i += S::kThreads) {
      const int32_t row = i / (8 - full), ch = full + i % (8 - full);
      char* at = row < S::kBM ? xb + row * kBlk : wb + (row - S::kBM) * kBlk;
      *reinterpret_cast<u32x4*>(at + (ch ^ (row & 7)) * 16) = u32x4{0, 0, 0, 0};
    }
    __syncthreads();
  };
  // The scales of 8 blocks at a time, 8 lanes per row of x or column fragment of w; they go
  // through registers to LDS 6 blocks later, held [block][row].  A fragment's 16 columns lie in
  // one block of w_scale.
  float scr[S::kScaleLoads];
  const float* scp[S::kScaleLoads];
#pragma unroll
  for (int j = 0; j < S::kScaleLoads; ++j) {
    const int32_t i = (j * S::kThreads + static_cast<int32_t>(threadIdx.x)) / S::kScaleRuns;
    scp[j] = i < S::kBM ? a.x_scale + (rt.row0 + min(i, rt.rows - 1)) * a.xss + k0
                        : a.w_scale + k0 + (static_cast<int64_t>(rt.expert) * a.nb + weight_row(min(i - S::kBM, 15) * 16) / kBlk) * a.kb;
  }
  auto scales_load = [&](int32_t b0) {
    const int32_t b = min(b0 + static_cast<int32_t>(threadIdx.x) % S::kScaleRuns, kb - 1);
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

  fetch_x(0);
  fetch_w(0);
  scales_load(0);
  scales_store(0);
  if (kb > 1) fetch_w(1);
  copies_done<S::kWCopies>(kb > 1);

  // Step b: x of block b + 1 is fetched from its start; the waves take their fragments of w into
  // registers, which frees that buffer for block b + 2.  So w has two steps to arrive and x one.
  f32x4 tot[MF][NF] = {};
  for (int32_t b = 0; b < kb; ++b) {
    const int32_t turn = b % S::kScaleRuns, next = b - turn + S::kScaleRuns;
    if (turn == S::kScaleRuns - 2 && next < kb) scales_store(next);
    if (turn == 0 && next < kb) scales_load(next);
    if (b + 1 < kb) fetch_x(b + 1);
    else if (full != 0) clear_tail();
    const char* xb = lds + (b & 1) * S::kBM * kBlk;
    const char* wb = lds + 2 * S::kBM * kBlk + (b & 1) * 256 * kBlk;
    const float* scb = xsl + ((b / S::kScaleRuns & 1) * S::kScaleRuns + turn) * S::kScales;
    constexpr int NS = kSwiglu ? NF : 1;  // without SwiGLU a wave's columns lie in one block of 128
    constexpr int kParts = kFast ? 2 : 4;  // registers of a fragment, in fours
    const int32_t ch0 = (g ^ (r & 7)) * 16, ch1 = ((4 + g) ^ (r & 7)) * 16;
    u32x4 wv[NF][2], xv[2][2];
    float ws[NS], xs[MF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const char* row = wb + ((wn * NF + f) * 16 + r) * kBlk;
      wv[f][0] = *reinterpret_cast<const u32x4*>(row + ch0);
      wv[f][1] = *reinterpret_cast<const u32x4*>(row + ch1);
    }
    auto read_x = [&](int i) {
      const char* row = xb + ((wm * MF + i) * 16 + r) * kBlk;
      xv[i & 1][0] = *reinterpret_cast<const u32x4*>(row + ch0);
      xv[i & 1][1] = *reinterpret_cast<const u32x4*>(row + ch1);
    };
    read_x(0);
#pragma unroll
    for (int f = 0; f < NS; ++f) ws[f] = scb[S::kBM + wn * NF + f];
#pragma unroll
    for (int i = 0; i < MF; ++i) xs[i] = scb[(wm * MF + i) * 16 + r];
    if constexpr (MF > 1) read_x(1);
    if (b + 2 < kb) {
      lds_barrier();  // every wave has its fragments of w
      fetch_w(b + 2);
    }
    // One stretch of code from here to the end of the step: a fragment of x is multiplied while the
    // sums of the one before are scaled and the one after next is read.
    u32x4 wf[NF][kParts], xf[2][kParts];
    f32x4 p[2][NF];
    auto widen = [](const u32x4 (&v)[2], u32x4 (&to)[kParts]) {
      if constexpr (kFast) {
        to[0] = v[0], to[1] = v[1];
      } else {
        to[0] = widen8(v[0][0], v[0][1]), to[1] = widen8(v[0][2], v[0][3]);
        to[2] = widen8(v[1][0], v[1][1]), to[3] = widen8(v[1][2], v[1][3]);
      }
    };
    auto scale = [&](int i) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const float s = xs[i] * ws[kSwiglu ? f : 0];
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[i][f][j] = __builtin_fmaf(s, p[i & 1][f][j], tot[i][f][j]);
      }
    };
#pragma unroll
    for (int f = 0; f < NF; ++f) widen(wv[f], wf[f]);
    widen(xv[0], xf[0]);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      if constexpr (kFast) {
#pragma unroll
        for (int f = 0; f < NF; ++f) p[i & 1][f] = mul_e4m3(wf[f], xf[i & 1]);
      } else {
#pragma unroll
        for (int f = 0; f < NF; ++f) p[i & 1][f] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int f = 0; f < NF; ++f) p[i & 1][f] = Mat<TBF16>::mul(wf[f][s], xf[i & 1][s], p[i & 1][f]);
      }
      if (i + 1 < MF) widen(xv[(i + 1) & 1], xf[(i + 1) & 1]);
      if (i + 2 < MF) read_x(i + 2);
      if (i > 0) scale(i - 1);
#pragma unroll
      for (int q = 0; q < (kFast ? NF : 4 * NF); ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);             // a matrix instruction,
        __builtin_amdgcn_sched_group_barrier(0x002, kFast ? 5 : 2, 0); // then vector ones
        if (q < 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // and a read
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    scale(MF - 1);
    copies_done<S::kWCopies>(b + 2 < kb);
  }

  // Results go through LDS, so that memory sees whole lines: a matrix result is 16 rows by 4
  // adjacent columns per lane.  Row r of the tile is kPitch bytes, its 16-byte chunks at
  // position c ^ (r % 8) as above.
  constexpr int kElt = kQuant ? 1 : T::kBytes;
  constexpr int kCols = kSwiglu ? 128 : 256, kPitch = kCols * kElt;
  constexpr int OF = kSwiglu ? NF / 2 : NF;  // result fragments of a wave
  const int64_t limit = kSwiglu ? a.F : a.N;
  if constexpr (kSwiglu) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int f = 0; f < OF; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[i][f][j] = swiglu(tot[i][f][j], tot[i][OF + f][j]);
  }
  float scale[kQuant ? MF : 1];
  if constexpr (kQuant) {
    // the row's largest |h| over the tile's 128 columns, one block: lanes, then waves
    uint32_t* amax = reinterpret_cast<uint32_t*>(xsl);  // [kBM][WN], in the scales' memory
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      uint32_t big = 0;
#pragma unroll
      for (int f = 0; f < OF; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + (wn * OF + f) * 16 < limit) big = max(big, __float_as_uint(tot[i][f][j]) & 0x7fffffffu);
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
      scale[i] = block_scale(big);
      if (wn == 0 && g == 0 && row < rt.rows) a.y_scale[(rt.row0 + row) * a.yss + c] = scale[i];
    }
  }
  // FP32 tiles of 128 rows are wider than the buffers: the waves of one half of the rows after
  // those of the other.
  constexpr int kParts = S::kBM * kPitch > 2 * S::kRows * kBlk ? 2 : 1;
  constexpr int kPartRows = S::kBM / kParts;
  static_assert(kParts == 1 || WM == 2, "a part is the rows of some of the waves");
#pragma unroll
  for (int half = 0; half < kParts; ++half) {
    if (half > 0) __syncthreads();
    if (kParts == 1 || wm == half) {
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int32_t row = ((kParts == 1 ? wm * MF : 0) + i) * 16 + r;
#pragma unroll
        for (int f = 0; f < OF; ++f) {
          const int32_t at = ((wn * OF + f) * 16 + g * 4) * kElt;  // byte of the row
          char* to = lds + row * kPitch + ((at / 16 ^ (row & 7)) * 16 + at % 16);
          if constexpr (kQuant) {
            float q[4] = {tot[i][f][0], tot[i][f][1], tot[i][f][2], tot[i][f][3]};
            block_quotients(q, scale[i]);
            *reinterpret_cast<uint32_t*>(to) = pack_e4m3(q[0], q[1], q[2], q[3]);
          } else if constexpr (kElt == 2) {
            const float v[8] = {tot[i][f][0], tot[i][f][1], tot[i][f][2], tot[i][f][3], 0, 0, 0, 0};
            const u32x4 h = Chunk<T>::narrow(v);
            *reinterpret_cast<u32x2*>(to) = u32x2{h[0], h[1]};
          } else {
            *reinterpret_cast<f32x4*>(to) = tot[i][f];
          }
        }
      }
    }
    __syncthreads();
    const int32_t rows = min(rt.rows - half * kPartRows, kPartRows);
    const int32_t bytes = static_cast<int32_t>(min(limit - c0, int64_t{kCols})) * kElt;  // of a row
    char* y = a.y + part * a.part_bytes + (rt.row0 + half * kPartRows) * a.ys + c0 * kElt;
    if (a.unit == 16) copy_out<16, kPitch, S::kThreads>(lds, y, a.ys, rows, bytes);
    else if (a.unit == 4) copy_out<4, kPitch, S::kThreads>(lds, y, a.ys, rows, bytes);
    else copy_out<kElt, kPitch, S::kThreads>(lds, y, a.ys, rows, bytes);
  }
}

// Tiles of at most half the rows (the last one of a group, the halves of find_tile) take half the
// fragments.
template <class T, int EPI, bool kQuant, bool kFast, int WM, int WN, int MF>
__global__ __launch_bounds__(WM* WN* kWave) void mm_tile_kernel(MmArgs a) {
  extern __shared__ __align__(16) char lds[];
  constexpr int kBM = TileShape<WM, WN, MF>::kBM;
  RowTile rt;
  int32_t c;
  if (!find_tile<(MF >= kHalvedFragments)>(a, kBM, rt, c)) return;
  if constexpr (MF >= kHalvedFragments) {
    if (rt.rows <= kBM / 2) {
      mm_tile<T, EPI, kQuant, kFast, WM, WN, MF / 2>(a, rt, c, lds);
      return;
    }
  }
  mm_tile<T, EPI, kQuant, kFast, WM, WN, MF>(a, rt, c, lds);
}

}  // namespace ffnwb
