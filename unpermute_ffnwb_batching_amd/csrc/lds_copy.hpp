// Copies between memory and LDS that the products' tile kernels share.
#pragma once

#include "device_common.hpp"

namespace ffnwb {

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

}  // namespace ffnwb
