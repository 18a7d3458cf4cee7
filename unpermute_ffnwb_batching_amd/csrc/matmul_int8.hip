// The experts' products on INT8 rows, with a scale for each row of x and each row of w.
//
// As for e4m3 rows there are two kernels: few rows take small tiles whose waves split K
// (mm8_direct_kernel), more rows large ones whose waves share both operands (mm8_tile_kernel).  The scales
// belong to whole rows, so the matrix cores carry the 32-bit totals over all of K, and the scaling is
// done once, at the end.  INT8 results, whose scale spans the row, are finished by mm8_rows_kernel.
#include "int8_tile.hpp"

namespace ffnwb {

// ------------------------------------------------------------------ direct kernel
//
// For few rows, or few of each expert, where latency and the reading of the weights count.  A workgroup
// takes 16 MT rows by 16 NF columns (SwiGLU: half of them gate columns, half the up columns that go with
// them); its waves take the 128-column blocks of K in turn, each through two LDS buffers of its own, without
// barriers, and their totals are added at the end.
//
// Why through LDS although no wave shares its blocks: a matrix operand has 16 rows in adjacent lanes,
// and loads in that order move 38 GB/s per CU, a lane each cycle; copies of whole lines to LDS move 125 to
// 150.  More buffers gained nothing.  Over 7168: 1 row by 4096 columns 6.7 us (7.6 with loads to registers), which is
// 4.4 TB/s with the launch, 16 rows 7.1 us (9.3), 64 rows 8.5 us (21.4); 256 rows by 2048 11.3 us (33.8); 1024 rows 28.1 us,
// 61 GB/s of copies per CU.  What bounds the last two is not known: LDS reads are 11% to 18% of a CU's busy cycles, without
// bank conflicts, and waits for them few.

// Bytes of LDS of a wave, and the most waves of a workgroup.
constexpr int direct_lds(int mt, int nf) { return 2 * (mt + nf) * 2048; }
constexpr int direct_waves(int mt, int nf) { return mt + nf <= 2 ? 16 : mt + nf <= 4 ? 8 : 4; }

// This wave's copies have landed, all or (`some`, uniform) all but the last kLeft.
template <int kLeft>
__device__ __forceinline__ void own_copies_done(bool some) {
  asm volatile("s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lown%=\n\ts_waitcnt vmcnt(0)\n.Lown%=:\n\ts_waitcnt vmcnt(%1)"
               ::"s"(uniform(static_cast<int32_t>(some))), "n"(kLeft) : "memory", "scc");
}
template <class T, int EPI, int MT, int NF>
__global__ __launch_bounds__(direct_waves(MT, NF) * kWave) void mm8_direct_kernel(Mm8Args a) {
  constexpr bool kSwiglu = EPI == FFNWB_EPI_SWIGLU;
  constexpr int CF = kSwiglu ? NF / 2 : NF;  // fragments of results; SwiGLU: gate, then up
  constexpr int kFrags = NF + MT, kRegion = direct_lds(MT, NF);
  extern __shared__ __align__(16) char lds8[];
  RowTile rt;
  int32_t c;
  if (!find_tile(a, MT * 16, rt, c)) return;
  const int32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int32_t r = lane % 16, g = lane / 16;
  const int64_t n0 = int64_t{c} * 16 * CF;
  auto column = [&](int f) -> int64_t { return n0 + f % CF * 16 + f / CF * a.F; };
  const char* src[kFrags][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int32_t q = j * 8 + lane / 8;
#pragma unroll
    for (int f = 0; f < NF; ++f) src[f][j] = a.w + (static_cast<int64_t>(rt.expert) * a.N + min(column(f) + q, a.N - 1)) * a.K;
#pragma unroll
    for (int i = 0; i < MT; ++i) src[NF + i][j] = a.x + static_cast<int64_t>(rt.row0 + min(i * 16 + q, rt.rows - 1)) * a.xs;
  }
  f32x4 ws[NF];
  float xs[MT];
#pragma unroll
  for (int f = 0; f < NF; ++f) ws[f] = channel_scales(a, rt.expert, column(f) + g * 4);
#pragma unroll
  for (int i = 0; i < MT; ++i) xs[i] = load_f32(a.x_scale + (rt.row0 + min(i * 16 + r, rt.rows - 1)) * a.xss);
  // A block of a fragment: two copies of 8 rows, chunks permuted as in the tile kernel.  Chunks past the
  // end of K take the row's last one, which counts as zeros: clearing it in x is enough.
  char* const own = lds8 + wave * kRegion;
  const int32_t last = static_cast<int32_t>(a.K) - 16, chunk = ((lane % 8) ^ (lane / 8)) * 16;
  auto fetch = [&](int32_t b, int32_t stage) {
    const int32_t k = min(b * kBlk + chunk, last);
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src[f][j] + k),
                                         reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(own + (stage * kFrags + f) * 2048 + j * 1024)), 16, 0, 0);
  };
  const int32_t at = r * kBlk + (g ^ (r & 7)) * 16;
  i32x4 tot[NF][MT] = {};
#pragma unroll
  for (int st = 0; st < 2; ++st)
    if (wave + st * waves < a.kb) fetch(wave + st * waves, st);
  int32_t stage = 0;
  for (int32_t b = wave; b < a.kb; b += waves) {
    own_copies_done<kFrags * 2>(b + waves < a.kb);
    const char* p = own + stage * kFrags * 2048;
    u32x4 v[kFrags][2];
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h) v[f][h] = *reinterpret_cast<const u32x4*>(p + f * 2048 + (at ^ (h * 64)));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the fragments are in registers: their buffer is free
    if (b + 2 * waves < a.kb) fetch(b + 2 * waves, stage);
    if ((b + 1) * kBlk > a.K) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (b * kBlk + h * 64 + g * 16 > last) {
#pragma unroll
          for (int i = 0; i < MT; ++i) v[NF + i][h] = u32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) tot[f][i] = mul_int8(v[f][h], v[NF + i][h], tot[f][i]);
    stage ^= 1;
  }
  // Each wave's totals take the place of its own blocks, whose copies have all landed.
  auto red = [&](int32_t w, int k) -> i32x4& { return reinterpret_cast<i32x4*>(lds8 + w * kRegion)[k * kWave + lane]; };
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < MT; ++i) red(wave, f * MT + i) = tot[f][i];
  __syncthreads();
#pragma unroll
  for (int o = 0; o < MT * CF; ++o) {
    if (o % waves != wave) continue;
    constexpr int kParts = kSwiglu ? 2 : 1;
    const int i = o % MT, f = o / MT;
    i32x4 s[kParts] = {};
    for (int32_t w = 0; w < waves; ++w)
#pragma unroll
      for (int u = 0; u < kParts; ++u) s[u] += red(w, (f + u * CF) * MT + i);
    if (i * 16 + r >= rt.rows) continue;  // the four lanes of a row together
    const int64_t row = rt.row0 + i * 16 + r, n = n0 + f * 16 + g * 4;
    f32x4 p[kParts];
#pragma unroll
    for (int u = 0; u < kParts; ++u) p[u] = scaled(s[u], xs[i], ws[f + u * CF]);
    if constexpr (kSwiglu) {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[0][j] = swiglu_fast<T::kExact>(p[0][j], p[1][j]);
    }
    if constexpr (T::kHeld) store_largest(a, p[0], row, n, n < a.F);
    store4<typename T::Out>(a.y + row * a.ys, n, a.F, p[0], a.vec);
  }
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
    load_raw<TF32, false, false>(from, h0, F, raw);  // F is a multiple of 16
    float f[8];
    widen_raw<TF32, false, false>(raw, h0, F, f);
    uint32_t lo, hi;
    quant_int8(f, s, lo, hi);
    *reinterpret_cast<u32x2_a1*>(q + h0) = u32x2{lo, hi};
  }
}

// 16 lanes to a row of up to 512 elements (58010 rows of 208, the whole call: 38 us, 62 with a wave to a row).
static int64_t rows8_lanes(int64_t F) { return F <= 512 ? 16 : 64; }

// ------------------------------------------------------------------ host side

constexpr int64_t kCus8 = 256;
constexpr int64_t kListedTiles8 = 16 * kCus8;  // more tiles of grouped rows are listed by a launch of their own

static int64_t out_size8(int32_t dt) { return dt == FFNWB_DT_FP32 ? 4 : dt == FFNWB_DT_INT8 ? 1 : 2; }

// The direct kernel's tiles: MT row and NF column fragments (of w: SwiGLU has half of them as results).
struct Direct8 { int mt, nf; };
constexpr Direct8 kDirect8[] = {{1, 1}, {2, 1}, {2, 2}, {4, 2}, {4, 4}};
constexpr Direct8 kDirect8Swiglu[] = {{1, 2}, {2, 2}, {4, 2}, {4, 4}};

// Microseconds that a product takes with the given kernel and tile, as far as the choice
// between them needs it: rounds of workgroups that fit the chip together times what one needs for
// its blocks of K, and the time of the weights and results in memory; the longer one, and a part of
// the first, as they overlap in part.  The figures are fitted so that the least of them picks the fastest shape,
// and are not those of the parts.
static double expected_us8(const Int8MatmulPlan& p, int64_t groups) {
  const int64_t some = groups < p.R ? groups : p.R, elt = p.quant || p.fp32 ? 4 : 2;
  const double mt = groups > 0 ? static_cast<double>(p.R) / p.bm + 0.619 * some : static_cast<double>((p.R + p.bm - 1) / p.bm);
  const double weights = (groups > 0 ? 0.621 * some : 1.0) * p.N * p.K;
  const double results = static_cast<double>(p.R * p.F * elt) / 4.0e6, wgs = mt * p.ntiles;
  auto rounds = [](double n, double together) { return n <= together ? 1.0 : __builtin_ceil(n / together); };
  auto larger = [](double a, double b) { return a > b ? a : b; };
  auto lesser = [](double a, double b) { return a < b ? a : b; };
  double us = 2.46;
  if (p.table) us += 2.29;
  if (p.quant) us += 3.73 + static_cast<double>(p.R * p.F) / 6.74e5;
  if (p.tile) {
    const bool two = p.bm < 128 && wgs > kCus8;  // two workgroups share a CU
    const double block = p.bm == 256 ? 1.0 : p.bm == 128 ? 0.942 : p.bm == 64 ? (two ? 1.17 : 0.733) : (two ? 1.08 : 0.6);
    const double once = p.bm == 256 ? 4.0 : p.bm == 128 ? 2.91 : two ? 2.04 : 1.37;
    const double work = rounds(wgs, p.bm < 128 ? 2 * kCus8 : kCus8) * (p.kb * block + once);
    return us + larger(work, weights / 5.8e6 + results) + 0.43 * work;
  }
  const double m = p.bm / 16, n = p.cols / 16 * (p.swiglu ? 2 : 1);  // fragments
  const double fit = larger(1.0, __builtin_floor(lesser(160.0 * 1024 / (4096 * (m + n) * p.waves), 20.0 / p.waves)));  // workgroups of a CU
  const double busy = lesser(__builtin_ceil(wgs / kCus8), fit) * p.waves;                                              // waves of one
  const double block = 0.0481 * (m + n) + 0.00982 * busy * (m + n) + 0.00496 * busy * m * n;
  const double copies = wgs * p.kb * (m + n) / 6890 + 0.65;  // 2 KB each, mostly from L2
  const double work = larger(rounds(wgs, fit * kCus8) * ((p.kb + p.waves - 1) / p.waves * block + 0.798 + 0.0406 * busy * m * n), copies);
  return us + larger(work, weights / 8.07e6 + results) + 0.43 * work;
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
  auto shape = [&](bool tile, int64_t bm, int64_t cols, int64_t waves) {  // the result: workgroups, of the larger launch
    p->tile = tile, p->bm = bm, p->cols = cols, p->waves = waves;
    p->mtiles = (p->R + bm - 1) / bm + (d->group_list != nullptr ? (groups < p->R ? groups : p->R) : 0);
    p->ntiles = (p->F + cols - 1) / cols;
    p->table = p->R > 0 && (d->num_groups > kWaveGroups || (d->num_groups > 0 && p->mtiles * p->ntiles > kListedTiles8));
    const int64_t quant_groups = (bm * rows8_lanes(p->F) + kRows8Threads - 1) / kRows8Threads;
    return p->mtiles * (quant && quant_groups > p->ntiles ? quant_groups : p->ntiles);
  };
  // The kernel, its tiles and the waves of a direct workgroup: the least of the times expected.  On 1500
  // random sizes that the fit has not seen (up to 65536 rows, K and N to 8192, 0 to 256 groups; every other one
  // with K and N from 512 on) the choice is 2.2% slower than the best of all shapes on average, more than 10% in
  // 85 of them and 1.42 times at worst.  Either kernel alone would cost: 64 rows by 4096 columns over 7168 32 us in
  // tiles and 8.5 direct, 8191 rows by 7168 over 5120 249 us in tiles and more than twice that direct.
  // 256 rows of x, and the gate rows of w, have to be inside the 32-bit offsets of the tile kernel.
  const bool near = p->xs <= (1 << 22) && (!swiglu || (p->F + 128) * p->K < (int64_t{1} << 32));
  const int64_t most = (int64_t{1} << 22) - 8;  // workgroups of a launch: fewer than 2^32 threads of at most 1024 a workgroup
  double best = 0;
  Int8MatmulPlan chosen;
  auto consider = [&](bool tile, int64_t bm, int64_t cols, int64_t waves) {
    if (shape(tile, bm, cols, waves) > most) return;
    const double t = expected_us8(*p, d->num_groups);
    if (best == 0 || t < best) best = t, chosen = *p;
  };
  auto direct = [&](const Direct8& s) {
    for (int64_t waves = 1; waves <= direct_waves(s.mt, s.nf) && (waves == 1 || waves <= p->kb); waves *= 2)
      consider(false, s.mt * 16, (swiglu ? s.nf / 2 : s.nf) * 16, waves);
  };
  if (swiglu) for (const Direct8& s : kDirect8Swiglu) direct(s);
  else for (const Direct8& s : kDirect8) direct(s);
  if (near)
    for (const int64_t bm : {32, 64, 128, 256}) consider(true, bm, swiglu ? 128 : 256, 0);
  if (best == 0) return FFNWB_ERR_PARAM_INVALID;
  *p = chosen;
  p->ws_bytes = 0;
  Carve c;
  if (p->table) {
    c.take<int32_t>(1);
    c.take<int4>(static_cast<size_t>(p->mtiles));
  }
  if (p->quant) c.take<float>(static_cast<size_t>(p->R * p->F)), c.take<float>(static_cast<size_t>(p->R * p->F / 16));
  p->ws_bytes = c.off;
  return FFNWB_OK;
}

template <class T, int EPI, int MT, int NF>
static bool launch_direct8(const Mm8Args& a, const Int8MatmulPlan& p, hipStream_t s, void* b, void* e) {
  const size_t lds = static_cast<size_t>(p.waves) * direct_lds(MT, NF);
  auto kernel = mm8_direct_kernel<T, EPI, MT, NF>;
  allow_large_lds(reinterpret_cast<const void*>(kernel), lds);
  return launch_bound(kernel, dim3(tile_grid(p.mtiles * p.ntiles)), dim3(static_cast<uint32_t>(p.waves * kWave)), lds, s, b, e, a);
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
  if constexpr (EPI == FFNWB_EPI_SWIGLU) {
    if (!p.tile)
      return p.bm == 16     ? launch_direct8<T, EPI, 1, 2>(a, p, s, b, e)
             : p.bm == 32   ? launch_direct8<T, EPI, 2, 2>(a, p, s, b, e)
             : p.cols == 16 ? launch_direct8<T, EPI, 4, 2>(a, p, s, b, e)
                            : launch_direct8<T, EPI, 4, 4>(a, p, s, b, e);
  } else {
    if (!p.tile)
      return p.bm == 16     ? launch_direct8<T, EPI, 1, 1>(a, p, s, b, e)
             : p.bm == 32   ? (p.cols == 16 ? launch_direct8<T, EPI, 2, 1>(a, p, s, b, e) : launch_direct8<T, EPI, 2, 2>(a, p, s, b, e))
             : p.cols == 32 ? launch_direct8<T, EPI, 4, 2>(a, p, s, b, e)
                            : launch_direct8<T, EPI, 4, 4>(a, p, s, b, e);
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
  float* held = p.quant ? c.take<float>(static_cast<size_t>(p.R * p.F)) : nullptr;
  a.held_max = p.quant ? c.take<float>(static_cast<size_t>(p.R * p.F / 16)) : nullptr;
  void *b = d->ev_matmul_begin, *e = d->ev_matmul_end;
  // results in their own type, or rows held on their way to INT8
  Mm8Args m = a;
  m.ntiles = static_cast<int32_t>(p.ntiles);
  const int32_t dt = d->out_dtype;
  const uint64_t elt = p.quant ? 4 : static_cast<uint64_t>(out_size8(dt));
  if (p.quant) m.y = reinterpret_cast<char*>(held), m.ys = p.F * 4;
  m.vec = ((reinterpret_cast<uintptr_t>(m.y) | static_cast<uint64_t>(m.ys)) & (4 * elt - 1)) == 0;
  void* end = p.quant ? nullptr : e;
  bool ok = p.swiglu ? (dt == FFNWB_DT_INT8   ? launch_product8<Held, FFNWB_EPI_SWIGLU>(m, p, s, b, end)
                        : dt == FFNWB_DT_FP16 ? launch_product8<Scaled<TF16>, FFNWB_EPI_SWIGLU>(m, p, s, b, end)
                        : dt == FFNWB_DT_BF16 ? launch_product8<Scaled<TBF16>, FFNWB_EPI_SWIGLU>(m, p, s, b, end)
                                              : launch_product8<Scaled<TF32>, FFNWB_EPI_SWIGLU>(m, p, s, b, end))
                     : (dt == FFNWB_DT_FP16   ? launch_product8<Scaled<TF16>, FFNWB_EPI_NONE>(m, p, s, b, end)
                        : dt == FFNWB_DT_BF16 ? launch_product8<Scaled<TBF16>, FFNWB_EPI_NONE>(m, p, s, b, end)
                                              : launch_product8<Scaled<TF32>, FFNWB_EPI_NONE>(m, p, s, b, end));
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
