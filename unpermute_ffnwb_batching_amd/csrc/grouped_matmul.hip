// The experts' products on e4m3 rows with a scale for each 128 elements.
//
// Two kernels: few rows go straight from memory to registers (mm_direct_kernel), more rows in tiles
// through LDS (mm_tile_kernel); what their tiles cannot finish, mm_join_kernel does.  Every wave
// works out the row tiles of all groups by itself, or reads them from mm_table_kernel's list.  The
// products of a 128-column block start from zero, and its sum is added to the
// FP32 total times x_scale * w_scale: the scales differ from block to block, so the matrix
// cores cannot carry the total themselves.
#include "fp8_block.hpp"
#include "internal.hpp"
#include "row_tiles.hpp"

namespace ffnwb {

struct MmArgs {
  int64_t K, N, F;             // F = outputs per row (N, or N / 2 with SwiGLU)
  int64_t xs, xss, ys, yss;    // row strides: bytes, elements, bytes, elements
  int32_t rows;
  int32_t kb, nb;              // 128-blocks along K and N
  int32_t ntiles;              // column tiles
  int32_t parts, part_blocks;  // parts of K, each a workgroup's, and 128-blocks of a part
  int64_t part_bytes;          // between the results of two parts
  int32_t ngroups, nexperts;
  bool vec;                    // four adjacent outputs are one aligned store
  int32_t unit;                // rows of y are whole aligned units of 16 or 4 bytes, or elements (0)
  const char* x;
  const float* x_scale;
  const char* w;
  const float* w_scale;
  char* y;
  float* y_scale;
  const int64_t* groups;       // {expert, rows} pairs, or NULL for one dense product
  const int4* table;           // row tiles {expert, first row, rows, 0} of more than kWaveGroups groups
  const int32_t* count;        // [1] row tiles of the table
};

// ------------------------------------------------------------------ direct kernel
//
// For few rows, where the weights are read once and latency counts.  A workgroup takes MT * 16
// rows by 16 columns (SwiGLU: 16 gate and the 16 up columns that go with them); its waves take
// the 128-column blocks of K in turn, straight from memory to registers, a wave's next block
// ahead of its present one, and their totals are added in wave order.  One row by 4096 columns
// over 7168 takes 7.5 us, 3.9 TB/s of weights (a copy moves 4.8): three dependent loads (group,
// operands, scales), then the join of 16 waves.  With 64 columns and 4 waves to a workgroup
// it was 16.2 us: too few loads on their way.

template <class T, int EPI, int MT>
__global__ __launch_bounds__(MT == 1 ? 1024 : 512) void mm_direct_kernel(MmArgs a) {
  constexpr int NF = EPI == FFNWB_EPI_SWIGLU ? 2 : 1;
  extern __shared__ __align__(16) f32x4 red[];  // [waves][NF * MT][lanes]
  RowTile rt;
  int32_t c;
  if (!find_tile(a, MT * 16, rt, c)) return;
  const int32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int32_t r = lane % 16, g = lane / 16;
  const int64_t n0 = int64_t{c} * 16;
  const char* wp[NF];
  const float* wsp[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int64_t nf = n0 + f * a.F;  // the fragment's first weight row
    wp[f] = a.w + (static_cast<int64_t>(rt.expert) * a.N + min(nf + r, a.N - 1)) * a.K;
    wsp[f] = a.w_scale + (static_cast<int64_t>(rt.expert) * a.nb + nf / kBlk) * a.kb;
  }
  const char* xp[MT];
  const float* xsp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = rt.row0 + min(i * 16 + r, rt.rows - 1);
    xp[i] = a.x + row * a.xs;
    xsp[i] = a.x_scale + row * a.xss;
  }
  struct Block {
    u32x4 w[NF][2], x[MT][2];
    float ws[NF], xs[MT];
  } blk[2];
  // A block's columns; past the end of K the row's last ones (no branch in the way of the loads),
  // which `multiply` clears.
  const int32_t last = static_cast<int32_t>(a.K) - 16;
  auto load = [&](Block& v, int32_t b) {
    if (b >= a.kb) return;
    const int32_t k0 = min(b * kBlk + g * 16, last), k1 = min(b * kBlk + 64 + g * 16, last);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      v.w[f][0] = load16(wp[f] + k0);
      v.w[f][1] = load16(wp[f] + k1);
      v.ws[f] = load_f32(wsp[f] + b);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      v.x[i][0] = load16(xp[i] + k0);
      v.x[i][1] = load16(xp[i] + k1);
      v.xs[i] = load_f32(xsp[i] + b);
    }
  };
  f32x4 tot[NF][MT] = {};
  auto multiply = [&](Block& v, int32_t b) {
    if (b >= a.kb) return;
    if ((b + 1) * kBlk > a.K) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (b * kBlk + h * 64 + g * 16 > last) {
#pragma unroll
          for (int f = 0; f < NF; ++f) v.w[f][h] = u32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < MT; ++i) v.x[i][h] = u32x4{0, 0, 0, 0};
        }
    }
    f32x4 p[NF][MT] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // 8 columns of each lane
      u32x4 w8[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) w8[f] = widen8(v.w[f][s / 2][2 * (s % 2)], v.w[f][s / 2][2 * (s % 2) + 1]);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4 x8 = widen8(v.x[i][s / 2][2 * (s % 2)], v.x[i][s / 2][2 * (s % 2) + 1]);
#pragma unroll
        for (int f = 0; f < NF; ++f) p[f][i] = Mat<TBF16>::mul(w8[f], x8, p[f][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const float s = v.xs[i] * v.ws[f];
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[f][i][j] = __builtin_fmaf(s, p[f][i][j], tot[f][i][j]);
      }
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
    for (int i = 0; i < MT; ++i) red[(wave * NF * MT + f * MT + i) * kWave + lane] = tot[f][i];
  __syncthreads();
  for (int32_t i = wave; i < MT; i += waves) {
    f32x4 s[NF] = {};
    for (int32_t w = 0; w < waves; ++w)
#pragma unroll
      for (int f = 0; f < NF; ++f) s[f] += red[(w * NF * MT + f * MT + i) * kWave + lane];
    if (i * 16 + r >= rt.rows) continue;
    char* row = a.y + static_cast<int64_t>(rt.row0 + i * 16 + r) * a.ys;
    if constexpr (EPI == FFNWB_EPI_SWIGLU) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[0][j] = swiglu(s[0][j], s[1][j]);
    }
    store4<T>(row, n0 + g * 4, a.F, s[0], a.vec);
  }
}

}  // namespace ffnwb

#include "mm_tile.hpp"

namespace ffnwb {

// ------------------------------------------------------------------ joining a product
//
// For products whose tiles do not hold whole results: those split over K (FP32 sums [parts][R][N
// rounded up to 8]), and SwiGLU results of the direct kernel (FP32 h [R][F]) on their way to e4m3 rows,
// whose blocks are wider than its column tiles.  16 lanes take 128 outputs of a row, as in
// moe_quant_fp8; a workgroup takes 16 such blocks of a row tile, so that rows of no expert stay as
// they were.  The parts are added in order: the same bits on every run.

constexpr int kJoinThreads = 256;

template <class T, bool kSwiglu, bool kQuant>
__global__ __launch_bounds__(kJoinThreads) void mm_join_kernel(MmArgs a, const float* sums, int64_t pitch, int32_t parts, int32_t bm) {
  const int32_t fb = static_cast<int32_t>((a.F + kBlk - 1) / kBlk);
  RowTile rt;
  int32_t group;
  if (!find_tile(a, bm, rt, group)) return;
  const int32_t u = group * (kJoinThreads / 16) + threadIdx.x / 16;
  const int32_t i = u / fb, b = u - i * fb;
  const int64_t row = rt.row0 + i, f0 = static_cast<int64_t>(b) * kBlk + threadIdx.x % 16 * 8;
  const bool in = i < rt.rows && f0 < a.F;
  auto sum = [&](int64_t n, float (&f)[8]) {  // columns n .. n + 7
    const float* p = sums + row * pitch + n;
    f32x4 v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
#pragma unroll 4
    for (int32_t s = 0; s < parts; ++s, p += a.rows * pitch) {
      v0 += reinterpret_cast<const f32x4*>(p)[0];
      v1 += reinterpret_cast<const f32x4*>(p)[1];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = v0[j], f[4 + j] = v1[j];
  };
  float f[8] = {};
  if (in) {
    sum(f0, f);
    if constexpr (kSwiglu) {
      float up[8];
      sum(a.F + f0, up);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = swiglu(f[j], up[j]);
    }
  }
  if constexpr (kQuant) {  // F is a multiple of 16
    uint32_t lo, hi;
    const float s = quant_block(f, lo, hi);
    if (!in) return;
    char* q = a.y + row * a.ys + f0;
    if (((reinterpret_cast<uintptr_t>(a.y) | static_cast<uintptr_t>(a.ys)) & 7) == 0) {
      *reinterpret_cast<u32x2*>(q) = u32x2{lo, hi};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = static_cast<char>((j < 4 ? lo >> (8 * j) : hi >> (8 * j - 32)) & 0xffu);
    }
    if (threadIdx.x % 16 == 0) a.y_scale[row * a.yss + b] = s;
  } else {
    if (!in) return;
    char* y = a.y + row * a.ys;
    store4<T>(y, f0, a.F, f32x4{f[0], f[1], f[2], f[3]}, a.vec);
    store4<T>(y, f0 + 4, a.F, f32x4{f[4], f[5], f[6], f[7]}, a.vec);
  }
}

// ------------------------------------------------------------------ host side

constexpr int64_t kCus = 256;

static int64_t out_size(int32_t dt) { return dt == FFNWB_DT_FP32 ? 4 : dt == FFNWB_DT_FP8_E4M3 ? 1 : 2; }

// Waves of a direct workgroup: a block of K for each, four at most where there are enough
// workgroups to fill the chip.  (Four for a single block, three of them idle, took 12% longer on
// average over 136 sizes with K up to 384, up to twice as long.)
static int direct_waves(int64_t tiles, int64_t kb, int64_t bm) {
  int waves = 1;
  while (waves < (bm == 16 ? 16 : 8) && waves * 2 <= kb && (waves < 4 || tiles * waves < kCus * 16)) waves *= 2;
  return waves;
}

// Microseconds that a product takes with the given kernel and tile rows, as far as the choice
// between them needs it: rounds of workgroups that fit the chip together, times what one needs for
// its blocks of K.  The figures are fitted to the times of whole calls, and are not those of the
// parts (a round of 256-row tiles takes 15 us besides its blocks, the fit says 5.5).  A group's last tile is
// counted as 0.58 of one.  The launch that lists the row tiles is not counted.
static double expected_us(int64_t rows, int64_t N, int64_t K, int64_t F, int64_t groups, bool swiglu, bool quant, bool fast,
                          bool tile, int64_t bm, int64_t parts) {
  const int64_t kb = (K + 127) / 128, some = groups < rows ? groups : rows;
  const double mt = groups > 0 ? static_cast<double>(rows) / bm + 0.58 * some : static_cast<double>((rows + bm - 1) / bm);
  auto rounds = [](double wgs, int64_t together) { return wgs <= together ? 1.0 : __builtin_ceil(wgs / together); };
  if (tile) {
    const double tiles = parts > 1 ? mt * ((N + 255) / 256) * parts : mt * ((F + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256));
    const double join = parts > 1 ? 4.1 + parts * rows * N * 8 / 5430e3 : 0.0;  // a launch, sums written and read
    double us = fast ? (bm == 256 ? 1.53 : bm == 128 ? 0.98 : 0.79) : (bm == 128 ? 1.63 : 1.21);
    int64_t together = kCus;
    if (bm == 32) {  // two to a CU
      us = fast ? (tiles > kCus ? 1.2 : 0.65) : (tiles > kCus ? 1.68 : 0.83);
      together = 2 * kCus;
    }
    return 2.8 + rounds(tiles, together) * ((kb + parts - 1) / parts * us + 2.7) + join;
  }
  const int64_t nt = (F + 15) / 16;
  const int waves = direct_waves(((rows + bm - 1) / bm + some) * nt, kb, bm);
  // waves of a CU by the kernels' registers
  const int fit = bm == 16 ? (swiglu ? 20 : 28) : bm == 32 ? (swiglu ? 12 : 20) : (swiglu ? 8 : 12);
  const double wgs = mt * nt, us = (wgs * waves > 2048 ? 1.74 : 1.33) * (bm == 64 ? 1.63 : bm == 32 ? 1.27 : 1.0);
  const double work = rounds(wgs, fit / waves > 0 ? fit / waves * kCus : kCus) * ((kb + waves - 1) / waves * us + 0.7);
  const double weights = mt * N * K / 5120e3;  // read again for every row tile, from L2
  return 2.8 + (work > weights ? work : weights) + (quant ? 3.6 : 0.0);
}

int plan_grouped_matmul(const moe_grouped_matmul_fp8_desc* d, MatmulPlan* p) {
  if (d == nullptr || d->x == nullptr || d->x_scale == nullptr || d->w == nullptr || d->w_scale == nullptr || d->y == nullptr)
    return FFNWB_ERR_PARAM_NULLPTR;
  const int32_t epilogue = d->epilogue & ~FFNWB_EPI_EXACT;
  const bool quant = d->out_dtype == FFNWB_DT_FP8_E4M3, swiglu = epilogue == FFNWB_EPI_SWIGLU;
  if (quant && d->y_scale == nullptr) return FFNWB_ERR_PARAM_NULLPTR;
  if (epilogue != FFNWB_EPI_NONE && !swiglu) return FFNWB_ERR_PARAM_INVALID;
  if (d->out_dtype != FFNWB_DT_FP16 && d->out_dtype != FFNWB_DT_BF16 && d->out_dtype != FFNWB_DT_FP32 && !(quant && swiglu))
    return FFNWB_ERR_PARAM_INVALID;
  const int64_t big = int64_t{1} << 18;
  if (d->num_rows < 0 || d->num_rows > (int64_t{1} << 24)) return FFNWB_ERR_PARAM_INVALID;
  if (d->in_features <= 0 || d->in_features > big || d->in_features % 16 != 0) return FFNWB_ERR_PARAM_INVALID;
  if (d->out_features <= 0 || d->out_features > big || (swiglu && d->out_features % 32 != 0)) return FFNWB_ERR_PARAM_INVALID;
  if (d->num_experts < 1 || d->num_experts > kMaxExperts) return FFNWB_ERR_PARAM_INVALID;
  if (d->group_list != nullptr ? (d->num_groups < 1 || d->num_groups > kMaxExperts)
                               : (d->num_groups != 0 || d->num_experts != 1))
    return FFNWB_ERR_PARAM_INVALID;
  p->R = d->num_rows;
  p->K = d->in_features;
  p->N = d->out_features;
  p->F = swiglu ? d->out_features / 2 : d->out_features;
  p->kb = (p->K + 127) / 128;
  p->nb = (p->N + 127) / 128;
  const int64_t elt = out_size(d->out_dtype), fb = (p->F + 127) / 128;
  p->xs = d->x_row_stride ? d->x_row_stride : p->K;
  p->xss = d->x_scale_stride ? d->x_scale_stride : p->kb;
  p->ys = d->y_row_stride ? d->y_row_stride : p->F * elt;
  p->yss = d->y_scale_stride ? d->y_scale_stride : fb;
  const int64_t far = int64_t{1} << 32;  // row * stride stays far inside 64 bits
  if (p->xs < p->K || p->xs % 16 != 0 || p->xs > far || p->xss < p->kb || p->xss > far) return FFNWB_ERR_PARAM_INVALID;
  if (p->ys < p->F * elt || p->ys % elt != 0 || p->ys > far || (quant && (p->yss < fb || p->yss > far)))
    return FFNWB_ERR_PARAM_INVALID;
  if ((reinterpret_cast<uintptr_t>(d->x) | reinterpret_cast<uintptr_t>(d->w)) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(d->y) % elt != 0)
    return FFNWB_ERR_PARAM_INVALID;
  const int64_t groups = d->group_list != nullptr ? d->num_groups : 1;
  // The e4m3 instructions drop bits (fp8_block.hpp), mostly far below the rounding to 16 bits; FP32
  // results and the scales of e4m3 ones would show it, and a caller can refuse it.
  const bool fast = !quant && d->out_dtype != FFNWB_DT_FP32 && (d->epilogue & FFNWB_EPI_EXACT) == 0;
  auto shape = [&](int64_t bm, int64_t parts) {  // negative bm: direct; the result: workgroups, of the larger launch
    p->tile = bm > 0, p->bm = bm > 0 ? bm : -bm;
    p->part_blocks = (p->kb + parts - 1) / parts;
    p->parts = (p->kb + p->part_blocks - 1) / p->part_blocks;
    p->mtiles = (p->R + p->bm - 1) / p->bm + (d->group_list != nullptr ? (groups < p->R ? groups : p->R) : 0);
    p->ntiles = !p->tile ? (p->F + 15) / 16 : p->parts > 1 ? (p->N + 255) / 256 * p->parts : (p->F + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256);
    p->join = p->parts > 1 || (quant && !p->tile);
    p->join_groups = (p->bm * fb + kJoinThreads / 16 - 1) / (kJoinThreads / 16);
    return p->mtiles * (p->join && p->join_groups > p->ntiles ? p->join_groups : p->ntiles);
  };
  // The kernel, the rows of its tiles and the parts of K: the least of the times expected.  On 220
  // random sizes that the fit has not seen (1 to 16384 rows, K and N to 8192, 0 to 256 groups) the
  // choice is 3.6% slower than the best of the shapes on average, more than 10% in 22 of them and 1.7
  // times at worst; a fixed rule (the largest tile that the groups fill and that gives every CU one)
  // was 15%.  Parts are what fills the chip with a long K and few tiles: 256 rows by 2048 columns over
  // 7168 take 39.9 us in the best shape without and 17.7 us in 8 parts, 128 by 8192 over 8192 45.5 and
  // 24.3 us; with 1536 columns over 1536 they cost 0.2 to 3 us.  256 rows of x, and the gate rows of
  // w, have to be inside the 32-bit offsets of the tile kernel.  Tiles of 256 rows are for e4m3
  // instructions alone: with widened operands a wave has 67 to 76 registers too few for them.
  const bool near = p->xs <= (1 << 22) && (!swiglu || (p->F + 128) * p->K < (int64_t{1} << 32));
  const int64_t most = (int64_t{1} << 22) - 8;  // workgroups of a launch: fewer than 2^32 threads of at most 1024 a workgroup
  double best = 0;
  int64_t best_bm = 0, best_parts = 1;
  auto consider = [&](int64_t bm, int64_t parts) {
    if (shape(bm, parts) > most) return;
    const double t = expected_us(p->R, p->N, p->K, p->F, d->num_groups, swiglu, quant, fast, p->tile, p->bm, p->parts);
    if (best_bm == 0 || t < best) best = t, best_bm = bm, best_parts = p->parts;
  };
  for (const int64_t bm : {-16, -32, -64, 32, 64, 128, 256}) {
    if (bm > 0 && (!near || (bm == 256 && !fast))) continue;
    consider(bm, 1);
    if (bm < 0 || bm == 256) continue;
    // parts that fill the chip once, or half of it
    const int64_t last = d->num_groups < p->R ? d->num_groups : p->R, tiles = ((p->R + bm - 1) / bm + last * 6 / 10) * ((p->N + 255) / 256);
    const int64_t fill = (bm == 32 ? 2 : 1) * kCus / (tiles > 0 ? tiles : 1);
    for (const int64_t parts : {fill, fill / 2})
      if (parts > 1) consider(bm, parts < p->kb / 2 ? parts : p->kb / 2 > 1 ? p->kb / 2 : 1);
  }
  if (best_bm == 0) return FFNWB_ERR_PARAM_INVALID;
  shape(best_bm, best_parts);
  p->swiglu = swiglu;
  p->fast = p->tile && fast;
  p->pitch = p->parts > 1 ? (p->N + 7) / 8 * 8 : p->F;
  p->ws_bytes = 0;
  Carve c;
  // The list in every workgroup costs each about 1 us, two to a CU at a time; the launch 3 to 5 us with
  // 128 or 256 groups: 13119 rows of two groups by 78 columns over 80 take 9.1 us, in 820 row tiles of 16, where 64-row
  // tiles without the launch would take 6.4.
  p->table = p->R > 0 && (d->num_groups > kWaveGroups || (d->num_groups > 0 && p->mtiles * p->ntiles > 16 * kCus));
  if (p->table) {
    c.take<int32_t>(1);
    c.take<int4>(static_cast<size_t>(p->mtiles));
  }
  if (p->join) c.take<float>(static_cast<size_t>(p->parts * p->R * p->pitch));
  p->ws_bytes = c.off;
  return FFNWB_OK;
}

template <class T, int EPI, int MT>
static bool launch_direct_rows(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  const int waves = direct_waves(p.mtiles * p.ntiles, p.kb, p.bm);
  const size_t lds = static_cast<size_t>(waves) * (EPI == FFNWB_EPI_SWIGLU ? 2 : 1) * MT * kWave * 16;
  auto kernel = mm_direct_kernel<T, EPI, MT>;
  allow_large_lds(reinterpret_cast<const void*>(kernel), lds);
  return launch_bound(kernel, dim3(tile_grid(p.mtiles * p.ntiles)), dim3(static_cast<uint32_t>(waves * kWave)), lds, s, b, e, a);
}

template <class T, int EPI>
static bool launch_direct(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  return p.bm == 16   ? launch_direct_rows<T, EPI, 1>(a, p, s, b, e)
         : p.bm == 32 ? launch_direct_rows<T, EPI, 2>(a, p, s, b, e)
                      : launch_direct_rows<T, EPI, 4>(a, p, s, b, e);
}

template <class T, int EPI, bool kQuant, bool kFast, int WM, int WN, int MF>
static bool launch_tile_shape(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  using S = TileShape<WM, WN, MF>;
  auto kernel = mm_tile_kernel<T, EPI, kQuant, kFast, WM, WN, MF>;
  allow_large_lds(reinterpret_cast<const void*>(kernel), S::kLds);
  // halved tiles: up to half a round of workgroups more
  const int64_t more = MF >= kHalvedFragments ? kXcds * kXcdCus / 2 : 0;
  return launch_bound(kernel, dim3(tile_grid(p.mtiles * p.ntiles + more)), dim3(S::kThreads), S::kLds, s, b, e, a);
}

template <class T, int EPI, bool kQuant = false, bool kFast = false>
static bool launch_tile(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  if constexpr (T::kBytes == 2 && kFast) {
    if (p.bm == 256) return launch_tile_shape<T, EPI, kQuant, kFast, 2, 4, 8>(a, p, s, b, e);
  }
  return p.bm == 128  ? launch_tile_shape<T, EPI, kQuant, kFast, 2, 4, 4>(a, p, s, b, e)
         : p.bm == 64 ? launch_tile_shape<T, EPI, kQuant, kFast, 2, 4, 2>(a, p, s, b, e)
                      : launch_tile_shape<T, EPI, kQuant, kFast, 1, 4, 2>(a, p, s, b, e);
}

// 16-bit results.
template <class T, int EPI>
static bool launch_tile16(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  return p.fast ? launch_tile<T, EPI, false, true>(a, p, s, b, e) : launch_tile<T, EPI>(a, p, s, b, e);
}

int launch_grouped_matmul(const moe_grouped_matmul_fp8_desc* d, const MatmulPlan& p, void* ws, hipStream_t s) {
  if (p.R == 0) return record_event(d->ev_matmul_begin, s) && record_event(d->ev_matmul_end, s) ? FFNWB_OK : FFNWB_ERR_RUNTIME;
  MmArgs a{};
  a.rows = static_cast<int32_t>(p.R), a.K = p.K, a.N = p.N, a.F = p.F;
  a.xs = p.xs, a.xss = p.xss, a.ys = p.ys, a.yss = p.yss;
  a.kb = static_cast<int32_t>(p.kb), a.nb = static_cast<int32_t>(p.nb);
  a.ngroups = static_cast<int32_t>(d->num_groups), a.nexperts = static_cast<int32_t>(d->num_experts);
  a.groups = d->group_list;
  a.x = static_cast<const char*>(d->x), a.x_scale = d->x_scale;
  a.w = static_cast<const char*>(d->w), a.w_scale = d->w_scale;
  a.y = static_cast<char*>(d->y), a.y_scale = d->y_scale;
  Carve c;
  c.base = static_cast<char*>(ws);
  if (p.table) {
    int32_t* count = c.take<int32_t>(1);
    int4* table = c.take<int4>(static_cast<size_t>(p.mtiles));
    hipLaunchKernelGGL(mm_table_kernel<MmArgs>, dim3(1), dim3(kTableThreads), 0, s, a, static_cast<int32_t>(p.bm), table, count);
    if (hipGetLastError() != hipSuccess) return FFNWB_ERR_RUNTIME;
    a.table = table, a.count = count;
  }
  void *b = d->ev_matmul_begin, *e = d->ev_matmul_end;
  // the product: results, or sums for the join
  const int32_t dt = p.join ? static_cast<int32_t>(FFNWB_DT_FP32) : d->out_dtype;
  MmArgs m = a;
  m.ntiles = static_cast<int32_t>(p.ntiles);
  m.parts = static_cast<int32_t>(p.parts), m.part_blocks = static_cast<int32_t>(p.part_blocks), m.part_bytes = p.R * p.pitch * 4;
  float* sums = nullptr;
  if (p.join) {
    sums = c.take<float>(static_cast<size_t>(p.parts * p.R * p.pitch));
    m.y = reinterpret_cast<char*>(sums), m.ys = p.pitch * 4;
    m.vec = true, m.unit = 16;  // the units of a row's end may run into the rest of its pitch
    if (p.parts > 1) m.F = p.N;
  } else {
    const uint64_t at = reinterpret_cast<uintptr_t>(a.y) | static_cast<uint64_t>(p.ys), elt = static_cast<uint64_t>(out_size(dt));
    m.vec = (at & (4 * elt - 1)) == 0;
    m.unit = ((at | p.F * elt) & 15) == 0 ? 16 : ((at | p.F * elt) & 3) == 0 ? 4 : 0;
  }
  void* product_end = p.join ? nullptr : e;
  const bool swiglu = p.swiglu, quant = d->out_dtype == FFNWB_DT_FP8_E4M3;
  bool ok;
  if (p.parts > 1) {
    ok = p.fast ? launch_tile<TF32, FFNWB_EPI_NONE, false, true>(m, p, s, b, product_end)
                : launch_tile<TF32, FFNWB_EPI_NONE>(m, p, s, b, product_end);
  } else if (p.tile && swiglu) {
    ok = quant                ? launch_tile<TF32, FFNWB_EPI_SWIGLU, true>(m, p, s, b, e)
         : dt == FFNWB_DT_FP16 ? launch_tile16<TF16, FFNWB_EPI_SWIGLU>(m, p, s, b, e)
         : dt == FFNWB_DT_BF16 ? launch_tile16<TBF16, FFNWB_EPI_SWIGLU>(m, p, s, b, e)
                               : launch_tile<TF32, FFNWB_EPI_SWIGLU>(m, p, s, b, e);
  } else if (p.tile) {
    ok = dt == FFNWB_DT_FP16   ? launch_tile16<TF16, FFNWB_EPI_NONE>(m, p, s, b, e)
         : dt == FFNWB_DT_BF16 ? launch_tile16<TBF16, FFNWB_EPI_NONE>(m, p, s, b, e)
                               : launch_tile<TF32, FFNWB_EPI_NONE>(m, p, s, b, e);
  } else if (swiglu) {
    ok = dt == FFNWB_DT_FP16   ? launch_direct<TF16, FFNWB_EPI_SWIGLU>(m, p, s, b, product_end)
         : dt == FFNWB_DT_BF16 ? launch_direct<TBF16, FFNWB_EPI_SWIGLU>(m, p, s, b, product_end)
                               : launch_direct<TF32, FFNWB_EPI_SWIGLU>(m, p, s, b, product_end);
  } else {
    ok = dt == FFNWB_DT_FP16   ? launch_direct<TF16, FFNWB_EPI_NONE>(m, p, s, b, e)
         : dt == FFNWB_DT_BF16 ? launch_direct<TBF16, FFNWB_EPI_NONE>(m, p, s, b, e)
                               : launch_direct<TF32, FFNWB_EPI_NONE>(m, p, s, b, e);
  }
  if (ok && p.join) {
    a.ntiles = static_cast<int32_t>(p.join_groups);
    const int64_t quad = 4 * out_size(d->out_dtype);
    a.vec = ((reinterpret_cast<uintptr_t>(a.y) | static_cast<uintptr_t>(p.ys)) & (quad - 1)) == 0;
    const int64_t pitch = p.pitch;
    const int32_t parts = m.parts, bm = static_cast<int32_t>(p.bm);
    auto join = [&](auto kernel) {
      return launch_bound(kernel, dim3(tile_grid(p.mtiles * p.join_groups)), dim3(kJoinThreads), 0, s, nullptr, e, a, sums, pitch, parts, bm);
    };
    ok = quant && p.parts == 1                     ? join(mm_join_kernel<TF32, false, true>)
         : quant                                   ? join(mm_join_kernel<TF32, true, true>)
         : swiglu && d->out_dtype == FFNWB_DT_FP16 ? join(mm_join_kernel<TF16, true, false>)
         : swiglu && d->out_dtype == FFNWB_DT_BF16 ? join(mm_join_kernel<TBF16, true, false>)
         : swiglu                                  ? join(mm_join_kernel<TF32, true, false>)
         : d->out_dtype == FFNWB_DT_FP16           ? join(mm_join_kernel<TF16, false, false>)
         : d->out_dtype == FFNWB_DT_BF16           ? join(mm_join_kernel<TBF16, false, false>)
                                                   : join(mm_join_kernel<TF32, false, false>);
  }
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
}

}  // namespace ffnwb
