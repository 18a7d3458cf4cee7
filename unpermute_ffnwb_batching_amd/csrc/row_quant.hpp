// Whole rows to 8 bits: INT8 with a scale for each row, and the device helpers of the kernels that
// make such rows.
//
// A row is taken by the TR threads of a wave or a workgroup, thread t holding elements 8 t .. 8 t + 7 of
// every run of 8 TR.
#pragma once

#include "fp8_block.hpp"

namespace ffnwb {

// 16- and 8-byte accesses at any address: gfx950 takes them from memory as they are.
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

// Elements h0 .. h0 + 7 of a row, zeros past its end.
template <class T>
__device__ __forceinline__ void load_run(const char* row, int32_t h0, int32_t hidden, float (&f)[8]) {
  const char* p = row + static_cast<int64_t>(h0) * T::kBytes;
  if (h0 + 8 <= hidden) {
    if constexpr (T::kBytes == 2) {
      const u32x4 v = *reinterpret_cast<const u32x4_a1*>(p);
      Chunk<T>::widen(v, f);
    } else {
      const u32x4 a = reinterpret_cast<const u32x4_a1*>(p)[0], b = reinterpret_cast<const u32x4_a1*>(p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(a[i]), f[4 + i] = __uint_as_float(b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = h0 + i < hidden ? load_elem<T>(p, i) : 0.0f;
  }
}

template <class T>
__device__ __forceinline__ void store_run(char* row, int32_t h0, int32_t hidden, const float (&f)[8]) {
  char* p = row + static_cast<int64_t>(h0) * T::kBytes;
  if (h0 + 8 <= hidden) {
    if constexpr (T::kBytes == 2) {
      *reinterpret_cast<u32x4_a1*>(p) = Chunk<T>::narrow(f);
    } else {
      reinterpret_cast<u32x4_a1*>(p)[0] = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
      reinterpret_cast<u32x4_a1*>(p)[1] = u32x4{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (h0 + i < hidden) store_elem<T>(p, i, f[i]);
  }
}

__device__ __forceinline__ void store_bytes(char* row, int32_t h0, int32_t hidden, uint32_t lo, uint32_t hi) {
  char* p = row + h0;
  if (h0 + 8 <= hidden) {
    *reinterpret_cast<u32x2_a1*>(p) = u32x2{lo, hi};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (h0 + i < hidden) p[i] = static_cast<char>((i < 4 ? lo >> (8 * i) : hi >> (8 * i - 32)) & 0xffu);
  }
}

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

constexpr int kRowWaves = 16;  // most waves of a row

// Sum of ss and maximum of m over a row's threads; every thread gets both.  The sums of the
// waves are added in order.  kOneWave: the row's threads are one wave; else they are the workgroup,
// which calls this with `turn` 0 and 1 alternately (one barrier to a call).
template <bool kOneWave>
__device__ __forceinline__ void row_reduce(float& ss, uint32_t& m, int32_t turn) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) {
    ss += __shfl_xor(ss, d);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  }
  if constexpr (!kOneWave) {
    __shared__ float2 part[2][kRowWaves];
    const int32_t wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
    if (lane_id() == 0) part[turn][wave] = float2{ss, __uint_as_float(m)};
    __syncthreads();
    ss = 0.0f, m = 0;
    for (int32_t w = 0; w < waves; ++w) {
      const float2 p = part[turn][w];
      ss += p.x;
      m = max(m, __float_as_uint(p.y));
    }
  }
}

}  // namespace ffnwb
