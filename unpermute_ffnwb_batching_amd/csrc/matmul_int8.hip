// The experts' products on INT8 rows, with a scale for each row of x and each row of w.
//
// As for e4m3 rows there are two kernels: few rows go straight from memory to registers
// (mm8_direct_kernel), more rows in tiles through LDS (mm8_tile_kernel).  The scales belong to whole
// rows, so the matrix cores carry the 32-bit totals over all of K, and the scaling is done once, at
// the end.  What a workgroup cannot finish by itself, mm8_join_kernel (parts of K) or mm8_rows_kernel
// (INT8 results, whose scale spans the row) does.
#include "int8_tile.hpp"

namespace ffnwb {

// ------------------------------------------------------------------ direct kernel
//
// For few rows, where the weights are read once and latency counts.  A workgroup takes MT * 16
// rows by 16 columns (SwiGLU: 16 gate and the 16 up columns that go with them); its waves take
// the 128-column blocks of K in turn, straight from memory to registers, a wave's next block
// ahead of its present one, and their totals are added in wave order.

template <class T, int EPI, int MT>
__global__ __launch_bounds__(MT == 1 ? 1024 : 512) void mm8_direct_kernel(Mm8Args a) {
  constexpr int NF = EPI == FFNWB_EPI_SWIGLU ? 2 : 1;
  extern __shared__ __align__(16) i32x4 red8[];  // [waves][NF * MT][lanes]
  RowTile rt;
  int32_t c;
  if (!find_tile(a, MT * 16, rt, c)) return;
  const int32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int32_t r = lane % 16, g = lane / 16;
  const int64_t n0 = int64_t{c} * 16;
  const char* wp[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
    wp[f] = a.w + (static_cast<int64_t>(rt.expert) * a.N + min(n0 + f * a.F + r, a.N - 1)) * a.K;
  const char* xp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xp[i] = a.x + static_cast<int64_t>(rt.row0 + min(i * 16 + r, rt.rows - 1)) * a.xs;
  // The scales: ahead of the blocks, where there are registers (MT = 4 would lose a wave of three).
  f32x4 ws[NF];
  float xs[MT];
  auto scales = [&] {
#pragma unroll
    for (int f = 0; f < NF; ++f) ws[f] = channel_scales(a, rt.expert, n0 + f * a.F + g * 4);
#pragma unroll
    for (int i = 0; i < MT; ++i) xs[i] = load_f32(a.x_scale + (rt.row0 + min(i * 16 + r, rt.rows - 1)) * a.xss);
  };
  if constexpr (MT < 4) scales();
  struct Block {
    u32x4 w[NF][2], x[MT][2];
  } blk[2];
  // A block's columns; past the end of K the row's last ones (no branch in the way of the loads),
  // which `multiply` clears in x.
  const int32_t last = static_cast<int32_t>(a.K) - 16;
  auto load = [&](Block& v, int32_t b) {
    if (b >= a.kb) return;
    const int32_t k0 = min(b * kBlk + g * 16, last), k1 = min(b * kBlk + 64 + g * 16, last);
#pragma unroll
    for (int f = 0; f < NF; ++f) v.w[f][0] = load16(wp[f] + k0), v.w[f][1] = load16(wp[f] + k1);
#pragma unroll
    for (int i = 0; i < MT; ++i) v.x[i][0] = load16(xp[i] + k0), v.x[i][1] = load16(xp[i] + k1);
  };
  i32x4 tot[NF][MT] = {};
  auto multiply = [&](Block& v, int32_t b) {
    if (b >= a.kb) return;
    if ((b + 1) * kBlk > a.K) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (b * kBlk + h * 64 + g * 16 > last) {
#pragma unroll
          for (int i = 0; i < MT; ++i) v.x[i][h] = u32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) tot[f][i] = mul_int8(v.w[f][h], v.x[i][h], tot[f][i]);
  };
  load(blk[0], wave);
  for (int32_t b = wave; b < a.kb; b += 2 * waves) {
    load(blk[1], b + waves);
    multiply(blk[0], b);
    load(blk[0], b + 2 * waves);
    multiply(blk[1], b + waves);
  }
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < MT; ++i) red8[(wave * NF * MT + f * MT + i) * kWave + lane] = tot[f][i];
  if constexpr (MT >= 4) scales();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i % waves != wave) continue;
    i32x4 s[NF] = {};
    for (int32_t w = 0; w < waves; ++w)
#pragma unroll
      for (int f = 0; f < NF; ++f) s[f] += red8[(w * NF * MT + f * MT + i) * kWave + lane];
    if (i * 16 + r >= rt.rows) continue;  // the four lanes of a row together
    const int64_t row = rt.row0 + i * 16 + r;
    f32x4 p[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) p[f] = scaled(s[f], xs[i], ws[f]);
    if constexpr (EPI == FFNWB_EPI_SWIGLU) {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[0][j] = swiglu_fast<T::kExact>(p[0][j], p[1][j]);
    }
    if constexpr (T::kHeld) store_largest(a, p[0], row, n0 + g * 4, true);
    store4<typename T::Out>(a.y + row * a.ys, n0 + g * 4, a.F, p[0], a.vec);
  }
}

// ------------------------------------------------------------------ joining a product
//
// Products split over K: whole-number sums [parts][R][N rounded up to 8], whose order does not
// matter.  16 lanes take 128 outputs of a row; a workgroup takes 16 such blocks of a row tile, so
// that rows of no expert stay as they were.

constexpr int kJoin8Threads = 256;

template <class T, bool kSwiglu>
__global__ __launch_bounds__(kJoin8Threads) void mm8_join_kernel(Mm8Args a, const int32_t* sums, int64_t pitch, int32_t parts, int32_t bm) {
  const int32_t fb = static_cast<int32_t>((a.F + kBlk - 1) / kBlk);
  RowTile rt;
  int32_t group;
  if (!find_tile(a, bm, rt, group)) return;
  const int32_t u = group * (kJoin8Threads / 16) + threadIdx.x / 16;
  const int32_t i = u / fb, b = u - i * fb;
  const int64_t row = rt.row0 + i, f0 = static_cast<int64_t>(b) * kBlk + threadIdx.x % 16 * 8;
  if (i >= rt.rows || f0 >= a.F) return;
  const float xs = a.x_scale[row * a.xss];
  auto sum = [&](int64_t n, f32x4 (&f)[2]) {  // columns n .. n + 7
    const int32_t* p = sums + row * pitch + n;
    i32x4 v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
#pragma unroll 4
    for (int32_t s = 0; s < parts; ++s, p += a.rows * pitch) {
      v0 += reinterpret_cast<const i32x4*>(p)[0];
      v1 += reinterpret_cast<const i32x4*>(p)[1];
    }
    f[0] = scaled(v0, xs, channel_scales(a, rt.expert, n));
    f[1] = scaled(v1, xs, channel_scales(a, rt.expert, n + 4));
  };
  f32x4 f[2];
  sum(f0, f);
  if constexpr (kSwiglu) {
    f32x4 up[2];
    sum(a.F + f0, up);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) f[h][j] = swiglu_fast<T::kExact>(f[h][j], up[h][j]);
  }
  char* y = a.y + row * a.ys;
  if constexpr (T::kHeld) {
    uint32_t m = 0;  // of the 16 columns of two lanes
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(f[h][j]) & 0x7fffffffu);
    m = max(m, lane_dpp<0xb1>(m));
    if (f0 % 16 == 0) a.held_max[row * (a.F / 16) + f0 / 16] = __uint_as_float(m);
  }
  store4<typename T::Out>(y, f0, a.F, f[0], a.vec);
  store4<typename T::Out>(y, f0 + 4, a.F, f[1], a.vec);
}

// ------------------------------------------------------------------ INT8 results
//
// Held rows (FP32 [R][F]) to INT8, with the row's scale: kLanes lanes to a row, 256 / kLanes rows of a row tile to a
// workgroup.  The row's largest value is that of its fragments, so its elements are read once,
// whatever the length.  131072 rows of 1024 take 127 us, 706 MB at the rate of a copy.

constexpr int kRows8Threads = 256;

template <int kLanes>
__global__ __launch_bounds__(kRows8Threads) void mm8_rows_kernel(Mm8Args a, const float* held, int32_t bm) {
  RowTile rt;
  int32_t group;
  if (!find_tile(a, bm, rt, group)) return;
  const int32_t i = group * (kRows8Threads / kLanes) + threadIdx.x / kLanes, t = threadIdx.x % kLanes;
  if (i >= rt.rows) return;
  const int64_t row = rt.row0 + i;
  const int32_t F = static_cast<int32_t>(a.F);
  const float* largest = a.held_max + row * (F / 16);
  uint32_t m = 0;
  for (int32_t f = t; f < F / 16; f += kLanes) m = max(m, __float_as_uint(largest[f]));
  const float s = row_scale(__uint_as_float(lanes_max<kLanes>(m)));
  if (t == 0) a.y_scale[row * a.yss] = s;
  const char* from = reinterpret_cast<const char*>(held + row * F);
  char* q = a.y + row * a.ys;
#pragma unroll 2
  for (int32_t h0 = t * 8; h0 < F; h0 += kLanes * 8) {
    Raw<TF32> raw;
    load_raw<TF32, false>(from, h0, F, raw);  // F is a multiple of 16
    float f[8];
    widen_raw(raw, f);
    uint32_t lo, hi;
    quant_int8(f, s, lo, hi);
    *reinterpret_cast<u32x2_a1*>(q + h0) = u32x2{lo, hi};
  }
}

// 16 lanes to a row of up to 512 elements (58010 rows of 208, the whole call: 37 us, 62 with a wave to a row).
static int64_t rows8_lanes(int64_t F) { return F <= 512 ? 16 : 64; }

// ------------------------------------------------------------------ host side

constexpr int64_t kCus8 = 256;
constexpr int64_t kListedTiles8 = 16 * kCus8;  // more tiles of grouped rows are listed by a launch of their own

static int64_t out_size8(int32_t dt) { return dt == FFNWB_DT_FP32 ? 4 : dt == FFNWB_DT_INT8 ? 1 : 2; }

// Waves of a direct workgroup: a block of K for each, four at most where there are enough
// workgroups to fill the chip.
static int direct_waves8(int64_t tiles, int64_t kb, int64_t bm) {
  int waves = 1;
  while (waves < (bm == 16 ? 16 : 8) && waves * 2 <= kb && (waves < 4 || tiles * waves < kCus8 * 16)) waves *= 2;
  return waves;
}

// Microseconds that a product takes with the given kernel and tile rows, as far as the choice
// between them needs it: rounds of workgroups that fit the chip together times what one needs for
// its blocks of K, or the time of the weights and results in memory if that is longer.  The figures
// are fitted so that the least of them picks the fastest shape, and are not those of the parts.
static double expected_us8(const Int8MatmulPlan& p, int64_t groups) {
  const int64_t some = groups < p.R ? groups : p.R, elt = p.quant || p.fp32 ? 4 : 2;
  const double mt = groups > 0 ? static_cast<double>(p.R) / p.bm + 0.7 * some : static_cast<double>((p.R + p.bm - 1) / p.bm);
  const double results = static_cast<double>(p.R * p.F * elt) / 2.42e6, wgs = mt * p.ntiles;
  auto rounds = [](double n, double together) { return n <= together ? 1.0 : __builtin_ceil(n / together); };
  double us = 2.6;
  if (groups > kWaveGroups || (groups > 0 && p.mtiles * p.ntiles > kListedTiles8)) us += 2.05;
  if (p.quant) us += 3.84 + static_cast<double>(p.R * p.F) / 1.24e6;
  if (p.tile) {
    const bool two = p.bm < 128 && wgs > kCus8;  // two workgroups share a CU
    const double block = p.bm == 256 ? 1.25 : p.bm == 128 ? 0.826 : p.bm == 64 ? (two ? 1.19 : 0.733) : (two ? 1.25 : 0.599);
    const double once = p.bm == 256 ? 6.9 : p.bm == 128 ? 2.0 : two ? 2.3 : 1.6;
    const double work = rounds(wgs, p.bm < 128 ? 2 * kCus8 : kCus8) * (p.part_blocks * block + once);
    const double memory = (groups > 0 ? 1.09 * some : 1.0) * p.N * p.K / 6.79e6 + results;
    if (p.parts > 1) us += 3.79 + static_cast<double>(p.parts * p.R * p.N) / 5.35e5;  // a launch, sums written and read
    return us + (work > memory ? work : memory);
  }
  const int waves = direct_waves8(p.mtiles * p.ntiles, p.kb, p.bm);
  const double fit = p.bm == 16 ? (p.swiglu ? 20 : 28) : p.bm == 32 ? (p.swiglu ? 12 : 20) : (p.swiglu ? 8 : 12);  // waves of a CU
  const double busy = wgs * waves / kCus8 < fit ? wgs * waves / kCus8 : fit;
  const double block = (p.bm == 64 ? 0.918 : p.bm == 32 ? 0.648 : 0.598) * (0.977 + 0.0956 * busy) * (p.swiglu ? 1.21 : 1.0);
  const double work = rounds(wgs, (fit > waves ? fit / waves : 1.0) * kCus8) * ((p.kb + waves - 1) / waves * block + 0.22 * (1 + 1.15 * (p.bm / 16 - 1)));
  const double memory = mt * p.N * p.K / 6.77e6 + results;  // the weights again for every row tile, from L2
  return us + (work > memory ? work : memory);
}

int plan_grouped_matmul_int8(const moe_grouped_matmul_int8_desc* d, Int8MatmulPlan* p) {
  if (d == nullptr || d->x == nullptr || d->x_scale == nullptr || d->w == nullptr || d->w_scale == nullptr || d->y == nullptr)
    return FFNWB_ERR_PARAM_NULLPTR;
  const bool quant = d->out_dtype == FFNWB_DT_INT8, swiglu = d->epilogue == FFNWB_EPI_SWIGLU;
  if (quant && d->y_scale == nullptr) return FFNWB_ERR_PARAM_NULLPTR;
  if (d->epilogue != FFNWB_EPI_NONE && !swiglu) return FFNWB_ERR_PARAM_INVALID;
  if (d->out_dtype != FFNWB_DT_FP16 && d->out_dtype != FFNWB_DT_BF16 && d->out_dtype != FFNWB_DT_FP32 && !(quant && swiglu))
    return FFNWB_ERR_PARAM_INVALID;
  if (d->num_rows < 0 || d->num_rows > (int64_t{1} << 24)) return FFNWB_ERR_PARAM_INVALID;
  // K * 128 * 128 stays below 2^31
  if (d->in_features <= 0 || d->in_features > 131056 || d->in_features % 16 != 0) return FFNWB_ERR_PARAM_INVALID;
  if (d->out_features <= 0 || d->out_features > (int64_t{1} << 18) || (swiglu && d->out_features % 32 != 0)) return FFNWB_ERR_PARAM_INVALID;
  if (d->num_experts < 1 || d->num_experts > kMaxExperts) return FFNWB_ERR_PARAM_INVALID;
  if (d->group_list != nullptr ? (d->num_groups < 1 || d->num_groups > kMaxExperts)
                               : (d->num_groups != 0 || d->num_experts != 1))
    return FFNWB_ERR_PARAM_INVALID;
  p->R = d->num_rows;
  p->K = d->in_features;
  p->N = d->out_features;
  p->F = swiglu ? d->out_features / 2 : d->out_features;
  p->kb = (p->K + 127) / 128;
  p->swiglu = swiglu;
  p->quant = quant;
  p->fp32 = d->out_dtype == FFNWB_DT_FP32;
  const int64_t elt = out_size8(d->out_dtype);
  p->xs = d->x_row_stride ? d->x_row_stride : p->K;
  p->xss = d->x_scale_stride ? d->x_scale_stride : 1;
  p->ys = d->y_row_stride ? d->y_row_stride : p->F * elt;
  p->yss = d->y_scale_stride ? d->y_scale_stride : 1;
  const int64_t far = int64_t{1} << 32;  // row * stride stays far inside 64 bits
  if (p->xs < p->K || p->xs % 16 != 0 || p->xs > far || p->xss < 1 || p->xss > far) return FFNWB_ERR_PARAM_INVALID;
  if (p->ys < p->F * elt || p->ys % elt != 0 || p->ys > far || p->yss < 1 || p->yss > far) return FFNWB_ERR_PARAM_INVALID;
  if ((reinterpret_cast<uintptr_t>(d->x) | reinterpret_cast<uintptr_t>(d->w)) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(d->y) % elt != 0 || (reinterpret_cast<uintptr_t>(d->x_scale) | reinterpret_cast<uintptr_t>(d->w_scale)) % 4 != 0 ||
      (quant && reinterpret_cast<uintptr_t>(d->y_scale) % 4 != 0))
    return FFNWB_ERR_PARAM_INVALID;
  const int64_t groups = d->group_list != nullptr ? d->num_groups : 1;
  auto shape = [&](int64_t bm, int64_t parts) {  // negative bm: direct; the result: workgroups, of the larger launch
    p->tile = bm > 0, p->bm = bm > 0 ? bm : -bm;
    p->part_blocks = (p->kb + parts - 1) / parts;
    p->parts = (p->kb + p->part_blocks - 1) / p->part_blocks;
    p->mtiles = (p->R + p->bm - 1) / p->bm + (d->group_list != nullptr ? (groups < p->R ? groups : p->R) : 0);
    p->ntiles = !p->tile ? (p->F + 15) / 16 : p->parts > 1 ? (p->N + 255) / 256 * p->parts : (p->F + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256);
    p->join = p->parts > 1;
    p->join_groups = p->join ? (p->bm * ((p->F + 127) / 128) + kJoin8Threads / 16 - 1) / (kJoin8Threads / 16) : 0;
    int64_t most = p->join_groups > p->ntiles ? p->join_groups : p->ntiles;
    const int64_t quant_groups = (p->bm * rows8_lanes(p->F) + kRows8Threads - 1) / kRows8Threads;
    if (quant && quant_groups > most) most = quant_groups;
    return p->mtiles * most;
  };
  // The kernel, the rows of its tiles and the parts of K: the least of the times expected.  On 1500
  // random sizes that the fit has not seen (1 to 65536 rows, K and N to 8192, 0 to 256 groups) the choice is
  // 2.0% slower than the best of the shapes on average, more than 10% in 103 of them and 1.85 times at
  // worst; on 700 with up to 4096 rows and K and N from 512 on, 2.6%, more than 10% in 62.  Parts are what fills the chip with a long K and few tiles: 256 rows by 2048 columns over 7168
  // take 32 us in the best shape without and 18 us in 4 parts.
  // 256 rows of x, and the gate rows of w, have to be inside the 32-bit offsets of the tile kernel.
  const bool near = p->xs <= (1 << 22) && (!swiglu || (p->F + 128) * p->K < (int64_t{1} << 32));
  const int64_t most = (int64_t{1} << 22) - 8;  // workgroups of a launch: fewer than 2^32 threads of at most 1024 a workgroup
  double best = 0;
  int64_t best_bm = 0, best_parts = 1;
  auto consider = [&](int64_t bm, int64_t parts) {
    if (shape(bm, parts) > most) return;
    const double t = expected_us8(*p, d->num_groups);
    if (best_bm == 0 || t < best) best = t, best_bm = bm, best_parts = p->parts;
  };
  for (const int64_t bm : {-16, -32, -64, 32, 64, 128, 256}) {
    if (bm > 0 && !near) continue;
    consider(bm, 1);
    if (bm < 0 || bm == 256) continue;
    // parts that fill the chip once, or half of it
    const int64_t last = d->num_groups < p->R ? d->num_groups : p->R, tiles = ((p->R + bm - 1) / bm + last * 6 / 10) * ((p->N + 255) / 256);
    const int64_t fill = (bm == 32 ? 2 : 1) * kCus8 / (tiles > 0 ? tiles : 1);
    for (const int64_t parts : {fill, fill / 2})
      if (parts > 1) consider(bm, parts < p->kb / 2 ? parts : p->kb / 2 > 1 ? p->kb / 2 : 1);
  }
  if (best_bm == 0) return FFNWB_ERR_PARAM_INVALID;
  shape(best_bm, best_parts);
  p->pitch = (p->N + 7) / 8 * 8;
  p->ws_bytes = 0;
  Carve c;
  p->table = p->R > 0 && (d->num_groups > kWaveGroups || (d->num_groups > 0 && p->mtiles * p->ntiles > kListedTiles8));
  if (p->table) {
    c.take<int32_t>(1);
    c.take<int4>(static_cast<size_t>(p->mtiles));
  }
  if (p->join) c.take<int32_t>(static_cast<size_t>(p->parts * p->R * p->pitch));
  if (p->quant) c.take<float>(static_cast<size_t>(p->R * p->F)), c.take<float>(static_cast<size_t>(p->R * p->F / 16));
  p->ws_bytes = c.off;
  return FFNWB_OK;
}

template <class T, int EPI, int MT>
static bool launch_direct8_rows(const Mm8Args& a, const Int8MatmulPlan& p, hipStream_t s, void* b, void* e) {
  const int waves = direct_waves8(p.mtiles * p.ntiles, p.kb, p.bm);
  const size_t lds = static_cast<size_t>(waves) * (EPI == FFNWB_EPI_SWIGLU ? 2 : 1) * MT * kWave * 16;
  auto kernel = mm8_direct_kernel<T, EPI, MT>;
  allow_large_lds(reinterpret_cast<const void*>(kernel), lds);
  return launch_bound(kernel, dim3(tile_grid(p.mtiles * p.ntiles)), dim3(static_cast<uint32_t>(waves * kWave)), lds, s, b, e, a);
}

template <class T, int EPI, int WM, int WN, int MF>
static bool launch_tile8_shape(const Mm8Args& a, const Int8MatmulPlan& p, hipStream_t s, void* b, void* e) {
  using S = Tile8Shape<WM, WN, MF>;
  auto kernel = mm8_tile_kernel<T, EPI, WM, WN, MF>;
  allow_large_lds(reinterpret_cast<const void*>(kernel), S::kLds);
  // halved tiles: up to half a round of workgroups more
  const int64_t more = MF >= kHalvedFragments ? kXcds * kXcdCus / 2 : 0;
  return launch_bound(kernel, dim3(tile_grid(p.mtiles * p.ntiles + more)), dim3(S::kThreads), S::kLds, s, b, e, a);
}

template <class T, int EPI>
static bool launch_product8(const Mm8Args& a, const Int8MatmulPlan& p, hipStream_t s, void* b, void* e) {
  if constexpr (!T::kWhole) {
    if (!p.tile)
      return p.bm == 16   ? launch_direct8_rows<T, EPI, 1>(a, p, s, b, e)
             : p.bm == 32 ? launch_direct8_rows<T, EPI, 2>(a, p, s, b, e)
                          : launch_direct8_rows<T, EPI, 4>(a, p, s, b, e);
  }
  return p.bm == 256   ? launch_tile8_shape<T, EPI, 2, 4, 8>(a, p, s, b, e)
         : p.bm == 128 ? launch_tile8_shape<T, EPI, 2, 4, 4>(a, p, s, b, e)
         : p.bm == 64  ? launch_tile8_shape<T, EPI, 2, 4, 2>(a, p, s, b, e)
                       : launch_tile8_shape<T, EPI, 1, 4, 2>(a, p, s, b, e);
}

int launch_grouped_matmul_int8(const moe_grouped_matmul_int8_desc* d, const Int8MatmulPlan& p, void* ws, hipStream_t s) {
  if (p.R == 0) return record_event(d->ev_matmul_begin, s) && record_event(d->ev_matmul_end, s) ? FFNWB_OK : FFNWB_ERR_RUNTIME;
  Mm8Args a{};
  a.rows = static_cast<int32_t>(p.R), a.K = p.K, a.N = p.N, a.F = p.F;
  a.xs = p.xs, a.xss = p.xss, a.ys = p.ys, a.yss = p.yss;
  a.kb = static_cast<int32_t>(p.kb);
  a.ngroups = static_cast<int32_t>(d->num_groups), a.nexperts = static_cast<int32_t>(d->num_experts);
  a.groups = d->group_list;
  a.x = static_cast<const char*>(d->x), a.x_scale = d->x_scale;
  a.w = static_cast<const char*>(d->w), a.w_scale = d->w_scale;
  a.y = static_cast<char*>(d->y), a.y_scale = d->y_scale;
  const int32_t bm = static_cast<int32_t>(p.bm);
  Carve c;
  c.base = static_cast<char*>(ws);
  if (p.table) {
    int32_t* count = c.take<int32_t>(1);
    int4* table = c.take<int4>(static_cast<size_t>(p.mtiles));
    hipLaunchKernelGGL(mm_table_kernel<Mm8Args>, dim3(1), dim3(kTableThreads), 0, s, a, bm, table, count);
    if (hipGetLastError() != hipSuccess) return FFNWB_ERR_RUNTIME;
    a.table = table, a.count = count;
  }
  int32_t* sums = p.join ? c.take<int32_t>(static_cast<size_t>(p.parts * p.R * p.pitch)) : nullptr;
  float* held = p.quant ? c.take<float>(static_cast<size_t>(p.R * p.F)) : nullptr;
  a.held_max = p.quant ? c.take<float>(static_cast<size_t>(p.R * p.F / 16)) : nullptr;
  void *b = d->ev_matmul_begin, *e = d->ev_matmul_end;
  // results in their own type, or rows held on their way to INT8
  Mm8Args out = a;
  const int32_t dt = d->out_dtype;
  const uint64_t elt = p.quant ? 4 : static_cast<uint64_t>(out_size8(dt));
  if (p.quant) out.y = reinterpret_cast<char*>(held), out.ys = p.F * 4;
  out.vec = ((reinterpret_cast<uintptr_t>(out.y) | static_cast<uint64_t>(out.ys)) & (4 * elt - 1)) == 0;
  void* out_end = p.quant ? nullptr : e;
  // the product: results, or whole-number sums for the join
  Mm8Args m = out;
  m.ntiles = static_cast<int32_t>(p.ntiles);
  m.parts = static_cast<int32_t>(p.parts), m.part_blocks = static_cast<int32_t>(p.part_blocks), m.part_bytes = p.R * p.pitch * 4;
  bool ok;
  if (p.join) {
    m.y = reinterpret_cast<char*>(sums), m.ys = p.pitch * 4, m.F = p.N;
    ok = launch_product8<Whole, FFNWB_EPI_NONE>(m, p, s, b, nullptr);
    if (ok) {
      out.ntiles = static_cast<int32_t>(p.join_groups);
      const int32_t parts = m.parts;
      const int64_t pitch = p.pitch;
      auto join = [&](auto kernel) {
        return launch_bound(kernel, dim3(tile_grid(p.mtiles * p.join_groups)), dim3(kJoin8Threads), 0, s, nullptr, out_end, out, sums, pitch, parts, bm);
      };
      ok = dt == FFNWB_DT_INT8   ? join(mm8_join_kernel<Held, true>)
           : dt == FFNWB_DT_FP16 ? (p.swiglu ? join(mm8_join_kernel<Scaled<TF16>, true>) : join(mm8_join_kernel<Scaled<TF16>, false>))
           : dt == FFNWB_DT_BF16 ? (p.swiglu ? join(mm8_join_kernel<Scaled<TBF16>, true>) : join(mm8_join_kernel<Scaled<TBF16>, false>))
                                 : (p.swiglu ? join(mm8_join_kernel<Scaled<TF32>, true>) : join(mm8_join_kernel<Scaled<TF32>, false>));
    }
  } else if (p.swiglu) {
    ok = dt == FFNWB_DT_INT8   ? launch_product8<Held, FFNWB_EPI_SWIGLU>(m, p, s, b, out_end)
         : dt == FFNWB_DT_FP16 ? launch_product8<Scaled<TF16>, FFNWB_EPI_SWIGLU>(m, p, s, b, out_end)
         : dt == FFNWB_DT_BF16 ? launch_product8<Scaled<TBF16>, FFNWB_EPI_SWIGLU>(m, p, s, b, out_end)
                               : launch_product8<Scaled<TF32>, FFNWB_EPI_SWIGLU>(m, p, s, b, out_end);
  } else {
    ok = dt == FFNWB_DT_FP16   ? launch_product8<Scaled<TF16>, FFNWB_EPI_NONE>(m, p, s, b, out_end)
         : dt == FFNWB_DT_BF16 ? launch_product8<Scaled<TBF16>, FFNWB_EPI_NONE>(m, p, s, b, out_end)
                               : launch_product8<Scaled<TF32>, FFNWB_EPI_NONE>(m, p, s, b, out_end);
  }
  if (ok && p.quant) {
    const int64_t lanes = rows8_lanes(p.F);
    a.ntiles = static_cast<int32_t>((p.bm * lanes + kRows8Threads - 1) / kRows8Threads);
    auto quant = [&](auto kernel) {
      return launch_bound(kernel, dim3(tile_grid(p.mtiles * a.ntiles)), dim3(kRows8Threads), 0, s, nullptr, e, a,
                          static_cast<const float*>(held), bm);
    };
    ok = lanes == 16 ? quant(mm8_rows_kernel<16>) : quant(mm8_rows_kernel<64>);
  }
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
}

}  // namespace ffnwb
