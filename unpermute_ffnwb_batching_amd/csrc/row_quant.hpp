// Whole rows to 8 bits: INT8 with a scale for each row, and the device helpers of the kernels that
// make such rows.
//
// A row is taken by TR threads (16 lanes, a wave or a workgroup), thread t holding elements 8 t .. 8 t +
// 7 of every run of 8 TR.  Rows start at any element: gfx950 takes 16-byte accesses at any address, and
// the last elements of a row, fewer than 8, are read as the end of the 8 before the row's end.
#pragma once

#include "fp8_block.hpp"

namespace ffnwb {

typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));

// The bytes of 8 elements: one 16-byte register group, or two of FP32.
template <class T> struct Raw { u32x4 v[T::kBytes / 2]; };

// Elements h0 .. h0 + 7 of a row (h0 a multiple of 8, below hidden).  kTail: hidden may be no multiple of 8;
// the run that passes the row's end holds its last 8 elements instead, for widen_raw to shift.  kShort: hidden
// may be below 8; such rows are read one by one, zeros behind them.
template <class T, bool kTail, bool kShort>
__device__ __forceinline__ void load_raw(const char* row, int32_t h0, int32_t hidden, Raw<T>& out) {
  constexpr int W = T::kBytes * 2;  // registers of 8 elements
  if (kShort && hidden < 8) {
    uint32_t w[W] = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < hidden) {
        if constexpr (T::kBytes == 2) w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[i]) << (16 * (i % 2));
        else w[i] = reinterpret_cast<const uint32_t*>(row)[i];
      }
#pragma unroll
    for (int i = 0; i < W / 4; ++i) out.v[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    return;
  }
  const char* p = row + static_cast<int64_t>(kTail ? min(h0, hidden - 8) : h0) * T::kBytes;
#pragma unroll
  for (int i = 0; i < W / 4; ++i) out.v[i] = reinterpret_cast<const u32x4_a1*>(p)[i];
}

// The elements that load_raw read, zeros past the row's end.
template <class T, bool kTail, bool kShort>
__device__ __forceinline__ void widen_raw(const Raw<T>& r, int32_t h0, int32_t hidden, float (&f)[8]) {
  constexpr int W = T::kBytes * 2;
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = r.v[i / 4][i % 4];
  if (kTail && h0 + 8 > hidden && (!kShort || hidden >= 8)) {
    // the row's last 8, shifted down by those that the runs before hold: as many in every row
    const int32_t down = 8 - hidden % 8;
#pragma unroll
    for (int s = W / 2; s > 0; s >>= 1)  // by whole registers: s, s / 2, ... 1
      if (down * T::kBytes / 4 & s) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = i + s < W ? w[i + s] : 0;
      }
    if constexpr (T::kBytes == 2) {
      if (down & 1) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = w[i] >> 16 | (i + 1 < W ? w[i + 1] << 16 : 0);
      }
    }
  }
  if constexpr (T::kBytes == 2) {
    Chunk<T>::widen(u32x4{w[0], w[1], w[2], w[3]}, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
}

// W registers, at any address; the first `bytes` (the same for every row) of them where `part`.
template <bool kTail, int W>
__device__ __forceinline__ void store_raw(char* p, bool part, int32_t bytes, const uint32_t (&w)[W]) {
  if (!kTail || !part) {
    if constexpr (W == 2) {
      *reinterpret_cast<u32x2_a1*>(p) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        reinterpret_cast<u32x4_a1*>(p)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (bytes >= 4 * i + 4) {
      reinterpret_cast<u32_a1*>(p)[i] = w[i];
    } else if (bytes > 4 * i) {
      if (bytes & 2) *reinterpret_cast<u16_a1*>(p + 4 * i) = static_cast<uint16_t>(w[i]);
      if (bytes & 1) p[bytes - 1] = static_cast<char>(bytes & 2 ? w[i] >> 16 : w[i]);
    }
  }
}

// Elements h0 .. h0 + 7 of a row, those below hidden.
template <class T, bool kTail>
__device__ __forceinline__ void store_run(char* row, int32_t h0, int32_t hidden, const float (&f)[8]) {
  char* p = row + static_cast<int64_t>(h0) * T::kBytes;
  const bool part = h0 + 8 > hidden;
  const int32_t bytes = hidden % 8 * T::kBytes;
  if constexpr (T::kBytes == 2) {
    const u32x4 v = Chunk<T>::narrow(f);
    const uint32_t w[4] = {v[0], v[1], v[2], v[3]};
    store_raw<kTail>(p, part, bytes, w);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
    store_raw<kTail>(p, part, bytes, w);
  }
}

template <bool kTail>
__device__ __forceinline__ void store_bytes(char* row, int32_t h0, int32_t hidden, uint32_t lo, uint32_t hi) {
  const uint32_t w[2] = {lo, hi};
  store_raw<kTail>(row + h0, h0 + 8 > hidden, hidden % 8, w);
}

// ------------------------------------------------------------------ reductions
//
// Over 16 adjacent lanes in four steps of the data path (a lane's own neighbour, the pair beside, the
// mirrored half row, the mirrored row), then over rows of lanes by swapping registers: no LDS.  Every
// lane gets the same bits, for sums too: the two terms of a step are the same for both partners.

template <int kCtrl>
__device__ __forceinline__ uint32_t lane_dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xf, 0xf, false));
}

template <int kLanes, class Op>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, Op op) {
  v = op(v, lane_dpp<0xb1>(v));   // quad_perm [1, 0, 3, 2]
  v = op(v, lane_dpp<0x4e>(v));   // quad_perm [2, 3, 0, 1]
  v = op(v, lane_dpp<0x141>(v));  // row_half_mirror
  v = op(v, lane_dpp<0x140>(v));  // row_mirror
  if constexpr (kLanes == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(b[0], b[1]);
  }
  return v;
}

template <int kLanes>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_reduce<kLanes>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_reduce<kLanes>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

constexpr int kRowWaves = 16;  // most waves of a row

// Sum of ss (kSum) and maximum of m over a row's threads; every thread gets both.  kLanes: 16 or 64 lanes
// hold a row, or a workgroup does (0), which calls this with `turn` 0 and 1 alternately: one
// barrier to a call, then every 16 lanes take one wave's part each.
template <int kLanes, bool kSum>
__device__ __forceinline__ void row_reduce(float& ss, uint32_t& m, int32_t turn) {
  constexpr int kFirst = kLanes == 16 ? 16 : 64;
  m = lanes_max<kFirst>(m);
  if constexpr (kSum) ss = lanes_sum<kFirst>(ss);
  if constexpr (kLanes == 0) {
    __shared__ float2 part[2][kRowWaves];
    const int32_t waves = blockDim.x / kWave, at = threadIdx.x % 16;
    if (lane_id() == 0) part[turn][threadIdx.x / kWave] = float2{ss, __uint_as_float(m)};
    __syncthreads();
    const float2 p = at < waves ? part[turn][at] : float2{0.0f, 0.0f};
    m = lanes_max<16>(__float_as_uint(p.y));
    if constexpr (kSum) ss = lanes_sum<16>(p.x);
  }
}

// ------------------------------------------------------------------ values to codes

// The scale of a row whose largest |x| is `amax` (NaN and infinity reach it; see block_scale).
__device__ __forceinline__ float row_scale(float amax) {
  const float s = amax / 127.0f;
  return s < 1.17549435e-38f ? 1.17549435e-38f : s;
}

// The low bytes of four whole numbers, a's lowest.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(b, a, 0x0c0c0400u) | __builtin_amdgcn_perm(d, c, 0x04000c0cu);
}

// Eight values of a row -> INT8 bytes.  |x / s| is at most 127 (1 + 2^-23); 1.5 * 2^23 added to a
// quotient rounds it to a whole number, ties to even, whose low byte is the sum's.
__device__ __forceinline__ void quant_int8(float (&f)[8], float s, uint32_t& lo, uint32_t& hi) {
  block_quotients(f, s);
  const uint32_t keep = s < __builtin_inff() ? 0xffffffffu : 0u;  // scale NaN or inf: zeros
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(f[i] + 12582912.0f);
  lo = pack_bytes(u[0], u[1], u[2], u[3]) & keep;
  hi = pack_bytes(u[4], u[5], u[6], u[7]) & keep;
}

// quant_block (fp8_block.hpp) for a run in registers: the block is 16 adjacent lanes.
__device__ __forceinline__ float quant_e4m3(float (&f)[8], uint32_t& lo, uint32_t& hi) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  const float s = block_scale(lanes_max<16>(m));
  block_quotients(f, s);
  lo = pack_e4m3(f[0], f[1], f[2], f[3]);
  hi = pack_e4m3(f[4], f[5], f[6], f[7]);
  return s;
}

}  // namespace ffnwb
