// Whole rows to 8 bits: moe_quant_int8, and moe_rmsnorm_quant with the residual's addition and the
// norm in the same pass.
//
// A row stays in registers between its reductions and its quotients.  The norm needs one round of
// reductions only: n = (s gamma) r with one r for the row, so the largest |n| is the largest
// |s gamma| times r (rounding is monotonic), and the sum of squares and that maximum travel together.
//
// Bound by memory, at the rate of a copy (4.9 TB/s read and written) or over it: 4608 rows of 7168 BF16
// with their residual take 46 us to INT8 and 49 us to e4m3 (231 MB), without a norm 21 us (99 MB; 17 with two
// sets of rows in turn, which the Infinity Cache holds in part); 16384 rows of 4096 with their residual 81 us
// (470 MB).  One row of 7168: 3.6 us, without a norm 2.4, most of it the launch.  What was worth it: all loads of a thread ahead of the first use, and registers few
// enough for 7 waves (gamma's type and rows of whole runs known to the compiler: 67 -> 46 us); reductions
// through the data path instead of LDS.
//
// Rows that are not whole runs of 8 elements start at any address: 4608 of 7167 BF16 take 63 us to INT8 and to
// e4m3, of 7164 (rows at multiples of 8 bytes) 51, without a norm both 18: the rest over 46 is the norm's six
// accesses a run that straddle lines.  The row's end is read where the run before it
// ends, without a branch: with one, the loads of a thread's runs waited for each other (64, 72 and 57 us; 16384 rows of
// 4095 129 instead of 108).
#include <type_traits>

#include "internal.hpp"
#include "row_quant.hpp"

namespace ffnwb {

struct RowArgs {
  int64_t rows;
  int32_t hidden;
  int64_t xs, rs, ros, ys, qs, ss;  // row strides: bytes, the last in elements
  float epsilon;
  const char* x;
  const char* residual;             // or NULL
  const char* gamma;
  const int64_t* actual;            // or NULL
  char* residual_out;
  char* y;                          // or NULL
  char* q;
  float* scale;
};

// C: runs of 8 elements that a thread holds; 0: the row is read twice instead.  kLanes: the lanes that
// hold a row, 256 / kLanes rows to a workgroup; 0: a row to a workgroup.  G: the type of gamma, void without a
// norm.  kTail: rows are not whole runs of 8.
template <class T, class G, bool kInt8, bool kTail, int C, int kLanes>
__global__ __launch_bounds__(kLanes > 0 ? 256 : 1024) void row_quant_kernel(RowArgs a) {
  constexpr int kHold = C > 0 ? C : 1;
  constexpr bool kNorm = !std::is_void<G>::value;
  using Gamma = typename std::conditional<kNorm, G, T>::type;
  int64_t rows = a.rows;
  if (a.actual != nullptr) {
    const int64_t n = *a.actual;
    rows = n < 0 ? 0 : n < rows ? n : rows;
  }
  const int32_t t = kLanes > 0 ? threadIdx.x % kLanes : threadIdx.x, tr = kLanes > 0 ? kLanes : blockDim.x;
  constexpr int kRows = kLanes > 0 ? 256 / kLanes : 1;  // of a workgroup
  constexpr bool kShort = kTail && kLanes == 16;        // rows below 8 elements take this shape only
  int32_t turn = 0;
  for (int64_t row = int64_t{blockIdx.x} * kRows + (kLanes == 64 ? uniform(threadIdx.x / kLanes) : kLanes > 0 ? threadIdx.x / kLanes : 0); row < rows;
       row += int64_t{gridDim.x} * kRows, turn ^= 1) {
    const char* x = a.x + row * a.xs;
    char* y = kNorm && a.y != nullptr ? a.y + row * a.ys : nullptr;
    char* q = a.q + row * a.qs;
    // The bytes of a run, all loads ahead of the first use.
    struct Run {
      Raw<T> x, res;
      Raw<Gamma> gamma;
    };
    auto load = [&](int32_t h0, Run& v) {
      if constexpr (kNorm) {
        load_raw<Gamma, kTail, kShort>(a.gamma, h0, a.hidden, v.gamma);
        if (a.residual != nullptr) load_raw<T, kTail, kShort>(a.residual + row * a.rs, h0, a.hidden, v.res);
      }
      load_raw<T, kTail, kShort>(x, h0, a.hidden, v.x);
    };
    // The values that r and the scale apply to, s gamma or x, with their part of the reductions.
    float ss = 0.0f;
    uint32_t m = 0;
    auto gather = [&](int32_t h0, const Run& v, float (&f)[8], bool store_sum) {
      widen_raw<T, kTail, kShort>(v.x, h0, a.hidden, f);
      if constexpr (kNorm) {
        float g[8];
        if (a.residual != nullptr) {
          widen_raw<T, kTail, kShort>(v.res, h0, a.hidden, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += g[i];
          if (store_sum) store_run<T, kTail>(a.residual_out + row * a.ros, h0, a.hidden, f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(f[i], f[i], ss);
        widen_raw<Gamma, kTail, kShort>(v.gamma, h0, a.hidden, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    };
    float r = 1.0f, scale = 0.0f;
    auto finish = [&](int32_t h0, float (&f)[8]) {  // every lane takes part, those past the end with zeros
      const bool in = h0 < a.hidden;
      uint32_t lo, hi;
      if constexpr (kNorm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= r;
        if (y != nullptr && in) store_run<T, kTail>(y, h0, a.hidden, f);
      }
      if constexpr (kInt8) {
        quant_int8(f, scale, lo, hi);
      } else {
        const float s = quant_e4m3(f, lo, hi);
        if (in && t % 16 == 0) a.scale[row * a.ss + h0 / kBlk] = s;
      }
      if (in) store_bytes<kTail>(q, h0, a.hidden, lo, hi);
    };
    float v[kHold][8] = {};
    if constexpr (C > 0) {
      Run run[kHold];
#pragma unroll
      for (int j = 0; j < kHold; ++j)
        if ((j * tr + t) * 8 < a.hidden) load((j * tr + t) * 8, run[j]);
#pragma unroll
      for (int j = 0; j < kHold; ++j)
        if ((j * tr + t) * 8 < a.hidden) gather((j * tr + t) * 8, run[j], v[j], true);
    } else {
      for (int32_t h0 = t * 8; h0 < a.hidden; h0 += tr * 8) {
        Run run;
        load(h0, run);
        gather(h0, run, v[0], false);
      }
    }
    row_reduce<kLanes, kNorm>(ss, m, turn);
    if constexpr (kNorm) r = 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.hidden) + a.epsilon);
    if constexpr (kInt8) {
      scale = row_scale(kNorm ? __uint_as_float(m) * r : __uint_as_float(m));
      if (t == 0) a.scale[row * a.ss] = scale;
    }
    if constexpr (C > 0) {
#pragma unroll
      for (int j = 0; j < kHold; ++j) finish((j * tr + t) * 8, v[j]);
    } else {
      for (int32_t base = 0; base < a.hidden; base += tr * 8) {
        const int32_t h0 = base + t * 8;
        float f[8] = {};
        if (h0 < a.hidden) {
          Run run;
          load(h0, run);
          gather(h0, run, f, true);
        }
        finish(h0, f);
      }
    }
  }
}

// ------------------------------------------------------------------ host side

constexpr int64_t kMostRows = int64_t{1} << 24;
constexpr int64_t kMostHidden = int64_t{1} << 20;
constexpr int64_t kFarStride = int64_t{1} << 32;

static int64_t float_size(int32_t dt) { return dt == FFNWB_DT_FP32 ? 4 : dt == FFNWB_DT_FP16 || dt == FFNWB_DT_BF16 ? 2 : 0; }

// A row stride of `bytes` per row or more, in steps of `elt`; 0 = dense.
static bool stride_ok(int64_t stride, int64_t bytes, int64_t elt) {
  return stride == 0 || (stride >= bytes && stride % elt == 0 && stride <= kFarStride);
}
static bool aligned(const void* p, int64_t elt) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elt) == 0; }

int plan_quant_int8(const moe_quant_int8_desc* d) {
  if (d == nullptr || d->x == nullptr || d->q == nullptr || d->scale == nullptr) return FFNWB_ERR_PARAM_NULLPTR;
  const int64_t elt = float_size(d->dtype);
  if (d->reserved0 != 0 || elt == 0) return FFNWB_ERR_PARAM_INVALID;
  if (d->num_rows < 0 || d->num_rows > kMostRows || d->hidden <= 0 || d->hidden > kMostHidden) return FFNWB_ERR_PARAM_INVALID;
  if (!stride_ok(d->x_row_stride, d->hidden * elt, elt) || !stride_ok(d->q_row_stride, d->hidden, 1) ||
      !stride_ok(d->scale_row_stride, 1, 1) || !aligned(d->x, elt) || !aligned(d->scale, 4))
    return FFNWB_ERR_PARAM_INVALID;
  return FFNWB_OK;
}

int plan_rmsnorm_quant(const moe_rmsnorm_quant_desc* d) {
  if (d == nullptr || d->x == nullptr || d->gamma == nullptr || d->q == nullptr || d->scale == nullptr) return FFNWB_ERR_PARAM_NULLPTR;
  if ((d->residual == nullptr) != (d->residual_out == nullptr)) return FFNWB_ERR_PARAM_NULLPTR;
  const int64_t elt = float_size(d->dtype), gelt = float_size(d->gamma_dtype);
  if (elt == 0 || (d->gamma_dtype != d->dtype && d->gamma_dtype != FFNWB_DT_FP32)) return FFNWB_ERR_PARAM_INVALID;
  if (d->q_dtype != FFNWB_DT_INT8 && d->q_dtype != FFNWB_DT_FP8_E4M3) return FFNWB_ERR_PARAM_INVALID;
  if (!(d->epsilon >= 0x1p-126f && d->epsilon < __builtin_inff())) return FFNWB_ERR_PARAM_INVALID;
  if (d->num_rows < 0 || d->num_rows > kMostRows || d->hidden <= 0 || d->hidden > kMostHidden) return FFNWB_ERR_PARAM_INVALID;
  const int64_t row = d->hidden * elt, scales = d->q_dtype == FFNWB_DT_INT8 ? 1 : (d->hidden + kBlk - 1) / kBlk;
  if (!stride_ok(d->x_row_stride, row, elt) || !stride_ok(d->residual_row_stride, row, elt) ||
      !stride_ok(d->residual_out_row_stride, row, elt) || !stride_ok(d->y_row_stride, row, elt) ||
      !stride_ok(d->q_row_stride, d->hidden, 1) || !stride_ok(d->scale_row_stride, scales, 1))
    return FFNWB_ERR_PARAM_INVALID;
  if (!aligned(d->x, elt) || !aligned(d->residual, elt) || !aligned(d->residual_out, elt) || !aligned(d->y, elt) ||
      !aligned(d->gamma, gelt) || !aligned(d->scale, 4))
    return FFNWB_ERR_PARAM_INVALID;
  const int64_t rs = d->residual_row_stride ? d->residual_row_stride : row, ros = d->residual_out_row_stride ? d->residual_out_row_stride : row;
  if (d->residual != nullptr && d->residual == d->residual_out && rs != ros) return FFNWB_ERR_PARAM_INVALID;
  return FFNWB_OK;
}

template <class T, class G, bool kInt8, bool kTail, int C, int kLanes>
static bool launch_rows(const RowArgs& a, int64_t threads, hipStream_t s, void* b, void* e) {
  constexpr int64_t kRows = kLanes > 0 ? 256 / kLanes : 1;
  const int64_t wgs = (a.rows + kRows - 1) / kRows, most = int64_t{1} << 21;  // rows past it by the kernel's loop
  return launch_bound(row_quant_kernel<T, G, kInt8, kTail, C, kLanes>, dim3(static_cast<uint32_t>(wgs < most ? wgs : most)),
                      dim3(static_cast<uint32_t>(threads)), 0, s, b, e, a);
}

// A thread holds two runs of a row, so that a workgroup of 7168 has 7 waves and a CU four of them; one in rows
// of the norm up to 4096 (16384 rows of 2048: 42.5 us with one, 44 with two; of 7168, 4608 rows: 50 and 46).
// Up to 512 elements a wave holds a row, up to 128 a quarter of one (8192 rows of 128: 3.2 us, 5.5 to 7 with
// a wave each).  Past 16384 elements a row is read twice (1024 rows of 20000: 38 us, in four runs to
// a thread 42; of 32768: 63 and 58).
template <class T, class G, bool kInt8, bool kTail>
static bool launch_shape(const RowArgs& a, hipStream_t s, void* b, void* e) {
  const int64_t runs = (a.hidden + 7) / 8;
  auto threads = [&](int64_t c) { return ((runs + c - 1) / c + kWave - 1) / kWave * kWave; };
  if (runs <= 16) return launch_rows<T, G, kInt8, kTail, 1, 16>(a, 256, s, b, e);
  if (runs <= 64) return launch_rows<T, G, kInt8, kTail, 1, 64>(a, 256, s, b, e);
  if constexpr (!std::is_void<G>::value) {
    if (runs <= 512) return launch_rows<T, G, kInt8, kTail, 1, 0>(a, threads(1), s, b, e);
  }
  if (runs <= 2048) return launch_rows<T, G, kInt8, kTail, 2, 0>(a, threads(2), s, b, e);
  return launch_rows<T, G, kInt8, kTail, 0, 0>(a, 1024, s, b, e);
}

template <class T, class G, bool kInt8>
static bool launch_tail(const RowArgs& a, hipStream_t s, void* b, void* e) {
  return a.hidden % 8 == 0 ? launch_shape<T, G, kInt8, false>(a, s, b, e) : launch_shape<T, G, kInt8, true>(a, s, b, e);
}

int launch_quant_int8(const moe_quant_int8_desc* d, hipStream_t s) {
  RowArgs a{};
  a.rows = d->num_rows;
  a.hidden = static_cast<int32_t>(d->hidden);
  a.xs = d->x_row_stride ? d->x_row_stride : d->hidden * float_size(d->dtype);
  a.qs = d->q_row_stride ? d->q_row_stride : d->hidden;
  a.ss = d->scale_row_stride ? d->scale_row_stride : 1;
  a.x = static_cast<const char*>(d->x);
  a.actual = d->actual_rows;
  a.q = static_cast<char*>(d->q);
  a.scale = d->scale;
  void *b = d->ev_quant_begin, *e = d->ev_quant_end;
  if (a.rows == 0) return record_event(b, s) && record_event(e, s) ? FFNWB_OK : FFNWB_ERR_RUNTIME;
  const bool ok = d->dtype == FFNWB_DT_FP16   ? launch_tail<TF16, void, true>(a, s, b, e)
                  : d->dtype == FFNWB_DT_BF16 ? launch_tail<TBF16, void, true>(a, s, b, e)
                                              : launch_tail<TF32, void, true>(a, s, b, e);
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
}

template <class T, class G>
static bool launch_norm(const RowArgs& a, bool int8, hipStream_t s, void* b, void* e) {
  return int8 ? launch_tail<T, G, true>(a, s, b, e) : launch_tail<T, G, false>(a, s, b, e);
}

int launch_rmsnorm_quant(const moe_rmsnorm_quant_desc* d, hipStream_t s) {
  const int64_t row = d->hidden * float_size(d->dtype);
  const bool int8 = d->q_dtype == FFNWB_DT_INT8;
  RowArgs a{};
  a.rows = d->num_rows;
  a.hidden = static_cast<int32_t>(d->hidden);
  a.xs = d->x_row_stride ? d->x_row_stride : row;
  a.rs = d->residual_row_stride ? d->residual_row_stride : row;
  a.ros = d->residual_out_row_stride ? d->residual_out_row_stride : row;
  a.ys = d->y_row_stride ? d->y_row_stride : row;
  a.qs = d->q_row_stride ? d->q_row_stride : d->hidden;
  a.ss = d->scale_row_stride ? d->scale_row_stride : int8 ? 1 : (d->hidden + kBlk - 1) / kBlk;
  a.epsilon = d->epsilon;
  a.x = static_cast<const char*>(d->x);
  a.residual = static_cast<const char*>(d->residual);
  a.gamma = static_cast<const char*>(d->gamma);
  a.actual = d->actual_rows;
  a.residual_out = static_cast<char*>(d->residual_out);
  a.y = static_cast<char*>(d->y);
  a.q = static_cast<char*>(d->q);
  a.scale = d->scale;
  void *b = d->ev_norm_begin, *e = d->ev_norm_end;
  if (a.rows == 0) return record_event(b, s) && record_event(e, s) ? FFNWB_OK : FFNWB_ERR_RUNTIME;
  const bool ok = d->dtype == FFNWB_DT_FP32   ? launch_norm<TF32, TF32>(a, int8, s, b, e)
                  : d->gamma_dtype == d->dtype ? (d->dtype == FFNWB_DT_FP16 ? launch_norm<TF16, TF16>(a, int8, s, b, e)
                                                                            : launch_norm<TBF16, TBF16>(a, int8, s, b, e))
                                               : (d->dtype == FFNWB_DT_FP16 ? launch_norm<TF16, TF32>(a, int8, s, b, e)
                                                                            : launch_norm<TBF16, TF32>(a, int8, s, b, e));
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
}

}  // namespace ffnwb
