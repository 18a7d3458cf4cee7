// Whole rows to 8 bits: moe_quant_int8, and moe_rmsnorm_quant with the residual's addition and the
// norm in the same pass.
//
// A row stays in registers between its reductions and its quotients.  The norm needs one round of
// reductions only: n = (s gamma) r with one r for the row, so the largest |n| is the largest
// |s gamma| times r (rounding is monotonic), and the sum of squares and that maximum travel together.
#include "internal.hpp"
#include "row_quant.hpp"

namespace ffnwb {

struct RowArgs {
  int64_t rows;
  int32_t hidden;
  int64_t xs, rs, ros, ys, qs, ss;  // row strides: bytes, the last in elements
  float epsilon;
  bool gamma32;                     // gamma in FP32, else in the type of x
  const char* x;
  const char* residual;             // or NULL
  const char* gamma;
  const int64_t* actual;            // or NULL
  char* residual_out;
  char* y;                          // or NULL
  char* q;
  float* scale;
};

// C: runs of 8 elements that a thread holds; 0: the row is read twice instead.  kOneWave: four rows to a
// workgroup, a wave each; else a row to a workgroup.
template <class T, int C, bool kOneWave, bool kNorm, bool kInt8>
__global__ __launch_bounds__(kOneWave ? 256 : 1024) void row_quant_kernel(RowArgs a) {
  int64_t rows = a.rows;
  if (a.actual != nullptr) {
    const int64_t n = *a.actual;
    rows = n < 0 ? 0 : n < rows ? n : rows;
  }
  const int32_t t = kOneWave ? threadIdx.x % kWave : threadIdx.x, tr = kOneWave ? kWave : blockDim.x;
  const int64_t first = kOneWave ? int64_t{blockIdx.x} * 4 + threadIdx.x / kWave : blockIdx.x;
  const int64_t step = kOneWave ? int64_t{gridDim.x} * 4 : gridDim.x;
  int32_t turn = 0;
  for (int64_t row = first; row < rows; row += step, turn ^= 1) {
    const char* x = a.x + row * a.xs;
    const char* res = kNorm && a.residual != nullptr ? a.residual + row * a.rs : nullptr;
    char* sum_out = kNorm && a.residual != nullptr ? a.residual_out + row * a.ros : nullptr;
    char* y = kNorm && a.y != nullptr ? a.y + row * a.ys : nullptr;
    char* q = a.q + row * a.qs;
    // the values that r and the scale apply to: s gamma, or x
    float ss = 0.0f;
    uint32_t m = 0;
    auto gather = [&](int32_t h0, float (&f)[8], bool store_sum) {
      load_run<T>(x, h0, a.hidden, f);
      if constexpr (kNorm) {
        if (res != nullptr) {
          float g[8];
          load_run<T>(res, h0, a.hidden, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += g[i];
          if (store_sum) store_run<T>(sum_out, h0, a.hidden, f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(f[i], f[i], ss);
        float g[8];
        if (a.gamma32) load_run<TF32>(a.gamma, h0, a.hidden, g);
        else load_run<T>(a.gamma, h0, a.hidden, g);
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
        if (y != nullptr && in) store_run<T>(y, h0, a.hidden, f);
      }
      if constexpr (kInt8) {
        quant_int8(f, scale, lo, hi);
      } else {
        const float s = quant_block(f, lo, hi);
        if (in && t % 16 == 0) a.scale[row * a.ss + h0 / kBlk] = s;
      }
      if (in) store_bytes(q, h0, a.hidden, lo, hi);
    };
    float v[C > 0 ? C : 1][8] = {};
    if constexpr (C > 0) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int32_t h0 = (j * tr + t) * 8;
        if (h0 < a.hidden) gather(h0, v[j], true);
      }
    } else {
      for (int32_t h0 = t * 8; h0 < a.hidden; h0 += tr * 8) gather(h0, v[0], false);
    }
    row_reduce<kOneWave>(ss, m, turn);
    if constexpr (kNorm) r = 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.hidden) + a.epsilon);
    if constexpr (kInt8) {
      scale = row_scale(kNorm ? __uint_as_float(m) * r : __uint_as_float(m));
      if (t == 0) a.scale[row * a.ss] = scale;
    }
    if constexpr (C > 0) {
#pragma unroll
      for (int j = 0; j < C; ++j) finish((j * tr + t) * 8, v[j]);
    } else {
      for (int32_t base = 0; base < a.hidden; base += tr * 8) {
        const int32_t h0 = base + t * 8;
        float f[8] = {};
        if (h0 < a.hidden) gather(h0, f, true);
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

template <class T, int C, bool kOneWave, bool kNorm, bool kInt8>
static bool launch_rows(const RowArgs& a, int64_t threads, hipStream_t s, void* b, void* e) {
  const int64_t wgs = kOneWave ? (a.rows + 3) / 4 : a.rows, most = int64_t{1} << 21;  // rows past it by the kernel's loop
  return launch_bound(row_quant_kernel<T, C, kOneWave, kNorm, kInt8>, dim3(static_cast<uint32_t>(wgs < most ? wgs : most)),
                      dim3(static_cast<uint32_t>(threads)), 0, s, b, e, a);
}

template <class T, bool kNorm, bool kInt8>
static bool launch_shape(const RowArgs& a, hipStream_t s, void* b, void* e) {
  const int64_t runs = (a.hidden + 7) / 8;
  auto threads = [&](int64_t c) { return ((runs + c - 1) / c + kWave - 1) / kWave * kWave; };
  if (runs <= 64) return launch_rows<T, 1, true, kNorm, kInt8>(a, 256, s, b, e);
  if (runs <= 128) return launch_rows<T, 2, true, kNorm, kInt8>(a, 256, s, b, e);
  if (runs <= 1024) return launch_rows<T, 1, false, kNorm, kInt8>(a, threads(1), s, b, e);
  if (runs <= 4096) return launch_rows<T, 4, false, kNorm, kInt8>(a, threads(4), s, b, e);
  return launch_rows<T, 0, false, kNorm, kInt8>(a, 1024, s, b, e);
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
  const bool ok = d->dtype == FFNWB_DT_FP16   ? launch_shape<TF16, false, true>(a, s, b, e)
                  : d->dtype == FFNWB_DT_BF16 ? launch_shape<TBF16, false, true>(a, s, b, e)
                                              : launch_shape<TF32, false, true>(a, s, b, e);
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
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
  a.gamma32 = d->gamma_dtype == FFNWB_DT_FP32;
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
  const bool ok = d->dtype == FFNWB_DT_FP16   ? (int8 ? launch_shape<TF16, true, true>(a, s, b, e) : launch_shape<TF16, true, false>(a, s, b, e))
                  : d->dtype == FFNWB_DT_BF16 ? (int8 ? launch_shape<TBF16, true, true>(a, s, b, e) : launch_shape<TBF16, true, false>(a, s, b, e))
                                              : (int8 ? launch_shape<TF32, true, true>(a, s, b, e) : launch_shape<TF32, true, false>(a, s, b, e));
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
}

}  // namespace ffnwb
