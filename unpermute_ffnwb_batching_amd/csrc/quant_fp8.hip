// Rows to e4m3 with an FP32 scale for each 128 elements.
//
// A block of 128 elements is taken by 16 lanes, 8 elements each: one 16-byte load per lane of
// 16-bit rows (two of FP32 rows), a maximum over the 16 lanes, 8 quotients, one 8-byte store.
// Blocks are numbered row by row, so a wave's 4 blocks are adjacent in memory whatever the row
// length.  Bound by memory: 4377 rows of 7168 BF16 take 19.7 us, 95 MB at 4.8 TB/s, which is what a
// plain copy moves; rows whose width or alignment allows no wide access go element by element, 4608
// of 7167 in 49 us.  The quotients by multiplication and FMA instead of division were worth 26%, and two
// or four blocks to a thread's lane group, one after another, gained nothing.
#include "fp8_block.hpp"
#include "internal.hpp"

namespace ffnwb {

constexpr int kQThreads = 256;
constexpr int kQGroups = kQThreads / 16;  // blocks a workgroup takes

struct QuantArgs {
  int64_t rows, hidden;
  int64_t xs, qs, ss;  // row strides: bytes, bytes, elements
  uint32_t nblk;       // blocks of a row
  const char* x;
  const int64_t* actual;
  char* q;
  float* scale;
};

template <class T, bool kVec>
__device__ __forceinline__ void load8(const char* row, int64_t h0, int64_t hidden, float (&f)[8]) {
  if constexpr (kVec) {
    const char* p = row + h0 * T::kBytes;
    if constexpr (T::kBytes == 2) {
      Chunk<T>::widen(*reinterpret_cast<const u32x4*>(p), f);
    } else {
      const u32x4 a = reinterpret_cast<const u32x4*>(p)[0], b = reinterpret_cast<const u32x4*>(p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) { f[i] = __uint_as_float(a[i]); f[4 + i] = __uint_as_float(b[i]); }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = h0 + i < hidden ? load_elem<T>(row, h0 + i) : 0.0f;
  }
}

// kVec: every row is 16-byte aligned and a multiple of 8 elements, every q row 8-byte aligned.
template <class T, bool kVec>
__global__ __launch_bounds__(kQThreads) void quant_fp8_kernel(QuantArgs a) {
  int64_t rows = a.rows;
  if (a.actual != nullptr) {
    const int64_t n = *a.actual;
    rows = n < 0 ? 0 : n < rows ? n : rows;
  }
  const uint32_t lane16 = threadIdx.x % 16;
  const uint32_t u = blockIdx.x * kQGroups + threadIdx.x / 16;
  const uint32_t row = u / a.nblk, b = u - row * a.nblk;
  const int64_t h0 = static_cast<int64_t>(b) * kBlk + lane16 * 8;
  const bool in = row < rows && h0 < a.hidden;
  float f[8] = {};
  if (in) load8<T, kVec>(a.x + static_cast<int64_t>(row) * a.xs, h0, a.hidden, f);
  uint32_t lo, hi;
  const float s = quant_block(f, lo, hi);
  if (!in) return;
  char* q = a.q + static_cast<int64_t>(row) * a.qs + h0;
  if constexpr (kVec) {
    *reinterpret_cast<u32x2*>(q) = u32x2{lo, hi};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (h0 + i < a.hidden) q[i] = static_cast<char>((i < 4 ? lo >> (8 * i) : hi >> (8 * i - 32)) & 0xffu);
  }
  if (lane16 == 0) a.scale[static_cast<int64_t>(row) * a.ss + b] = s;
}

// ------------------------------------------------------------------ host side

int plan_quant_fp8(const moe_quant_fp8_desc* d) {
  if (d == nullptr || d->x == nullptr || d->q == nullptr || d->scale == nullptr) return FFNWB_ERR_PARAM_NULLPTR;
  if (d->reserved0 != 0) return FFNWB_ERR_PARAM_INVALID;
  if (d->dtype != FFNWB_DT_FP16 && d->dtype != FFNWB_DT_BF16 && d->dtype != FFNWB_DT_FP32) return FFNWB_ERR_PARAM_INVALID;
  if (d->hidden <= 0 || d->hidden > (int64_t{1} << 20) || d->num_rows < 0) return FFNWB_ERR_PARAM_INVALID;
  const int64_t elt = d->dtype == FFNWB_DT_FP32 ? 4 : 2, nblk = (d->hidden + kBlk - 1) / kBlk;
  // one dimension of the grid: fewer than 2^32 threads, 16 to a block of elements
  if (d->num_rows > ((int64_t{1} << 28) - kQGroups) / nblk) return FFNWB_ERR_PARAM_INVALID;
  if (d->x_row_stride != 0 && (d->x_row_stride < d->hidden * elt || d->x_row_stride % elt != 0)) return FFNWB_ERR_PARAM_INVALID;
  if (d->q_row_stride != 0 && d->q_row_stride < d->hidden) return FFNWB_ERR_PARAM_INVALID;
  if (d->scale_row_stride != 0 && d->scale_row_stride < nblk) return FFNWB_ERR_PARAM_INVALID;
  // row * stride * 4 bytes stays inside 64 bits
  const int64_t far = d->num_rows > (1 << 20) ? (int64_t{1} << 60) / d->num_rows : int64_t{1} << 40;
  if (d->x_row_stride > far || d->q_row_stride > far || d->scale_row_stride > far) return FFNWB_ERR_PARAM_INVALID;
  if (reinterpret_cast<uintptr_t>(d->x) % elt != 0) return FFNWB_ERR_PARAM_INVALID;
  return FFNWB_OK;
}

template <class T>
static bool launch_t(const QuantArgs& a, bool vec, uint32_t grid, hipStream_t s, void* b, void* e) {
  return vec ? launch_bound(quant_fp8_kernel<T, true>, dim3(grid), dim3(kQThreads), 0, s, b, e, a)
             : launch_bound(quant_fp8_kernel<T, false>, dim3(grid), dim3(kQThreads), 0, s, b, e, a);
}

int launch_quant_fp8(const moe_quant_fp8_desc* d, hipStream_t s) {
  const int64_t elt = d->dtype == FFNWB_DT_FP32 ? 4 : 2;
  QuantArgs a{};
  a.rows = d->num_rows;
  a.hidden = d->hidden;
  a.nblk = static_cast<uint32_t>((d->hidden + kBlk - 1) / kBlk);
  a.xs = d->x_row_stride ? d->x_row_stride : d->hidden * elt;
  a.qs = d->q_row_stride ? d->q_row_stride : d->hidden;
  a.ss = d->scale_row_stride ? d->scale_row_stride : a.nblk;
  a.x = static_cast<const char*>(d->x);
  a.actual = d->actual_rows;
  a.q = static_cast<char*>(d->q);
  a.scale = d->scale;
  const int64_t units = d->num_rows * a.nblk;
  void *b = d->ev_quant_begin, *e = d->ev_quant_end;
  if (units == 0) return record_event(b, s) && record_event(e, s) ? FFNWB_OK : FFNWB_ERR_RUNTIME;
  const uint32_t grid = static_cast<uint32_t>((units + kQGroups - 1) / kQGroups);
  const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | static_cast<uintptr_t>(a.xs)) & 15) == 0 &&
                   ((reinterpret_cast<uintptr_t>(a.q) | static_cast<uintptr_t>(a.qs) | static_cast<uintptr_t>(a.hidden)) & 7) == 0;
  const bool ok = d->dtype == FFNWB_DT_FP16   ? launch_t<TF16>(a, vec, grid, s, b, e)
                  : d->dtype == FFNWB_DT_BF16 ? launch_t<TBF16>(a, vec, grid, s, b, e)
                                              : launch_t<TF32>(a, vec, grid, s, b, e);
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
}

}  // namespace ffnwb
