// The experts' products on e4m3 rows with a scale for each 128 elements.
//
// A tile table lists the row tiles of all groups (one launch over group_list); a dense product
// needs none.  The products of a 128-column block start from zero, and its sum is added to the
// FP32 total times x_scale * w_scale: the scales differ from block to block, so the matrix
// cores cannot carry the total themselves.
#include "fp8_block.hpp"
#include "internal.hpp"

namespace ffnwb {

struct MmArgs {
  int64_t rows, K, N, F;       // F = outputs per row (N, or N / 2 with SwiGLU)
  int64_t xs, xss, ys, yss;    // row strides: bytes, elements, bytes, elements
  int32_t kb, nb;              // 128-blocks along K and N
  int32_t mtiles, ntiles;      // row tiles of a dense product, column tiles
  bool vec;                    // four adjacent outputs are one aligned store
  const char* x;
  const float* x_scale;
  const char* w;
  const float* w_scale;
  char* y;
  float* y_scale;
  const int4* table;           // row tiles {expert, first row, rows, 0}, or NULL for a dense product
  const int32_t* count;        // [1] row tiles of the table
};

// ------------------------------------------------------------------ tile table

constexpr int kTableThreads = 1024;

// Row tiles of bm rows (a power of two) in group order.  Each thread takes a run of
// consecutive groups; sums over threads give every run its first row and first tile.
// Counts are clamped so that the rows never pass `rows`: the table then has at most
// ceil(rows / bm) + min(groups, rows) entries.
__global__ __launch_bounds__(kTableThreads) void mm_table_kernel(const int64_t* groups, int32_t ngroups, int64_t rows,
                                                                 int64_t nexperts, int32_t bm, int4* table, int32_t* count) {
  __shared__ int64_t sum_rows[kTableThreads];
  __shared__ int32_t sum_tiles[kTableThreads];
  const int32_t per = (ngroups + kTableThreads - 1) / kTableThreads;
  const int32_t g0 = threadIdx.x * per, g1 = min(g0 + per, ngroups);
  int64_t mine = 0;
  for (int32_t g = g0; g < g1; ++g) mine += min(max(groups[2 * g + 1], int64_t{0}), rows);
  sum_rows[threadIdx.x] = mine;
  __syncthreads();
  for (int d = 1; d < kTableThreads; d <<= 1) {
    const int64_t v = threadIdx.x >= static_cast<uint32_t>(d) ? sum_rows[threadIdx.x - d] : 0;
    __syncthreads();
    sum_rows[threadIdx.x] += v;
    __syncthreads();
  }
  const int64_t first = min(sum_rows[threadIdx.x] - mine, rows);
  int64_t at = first;
  int32_t tiles = 0;
  for (int32_t g = g0; g < g1; ++g) {
    const int64_t n = min(min(max(groups[2 * g + 1], int64_t{0}), rows), rows - at), key = groups[2 * g];
    if (key >= 0 && key < nexperts) tiles += static_cast<int32_t>((n + bm - 1) / bm);
    at += n;
  }
  sum_tiles[threadIdx.x] = tiles;
  __syncthreads();
  for (int d = 1; d < kTableThreads; d <<= 1) {
    const int32_t v = threadIdx.x >= static_cast<uint32_t>(d) ? sum_tiles[threadIdx.x - d] : 0;
    __syncthreads();
    sum_tiles[threadIdx.x] += v;
    __syncthreads();
  }
  int32_t t = sum_tiles[threadIdx.x] - tiles;
  if (threadIdx.x == kTableThreads - 1) *count = sum_tiles[threadIdx.x];
  at = first;
  for (int32_t g = g0; g < g1; ++g) {
    const int64_t n = min(min(max(groups[2 * g + 1], int64_t{0}), rows), rows - at), key = groups[2 * g];
    if (key >= 0 && key < nexperts) {
      for (int64_t r = 0; r < n; r += bm)
        table[t++] = int4{static_cast<int>(key), static_cast<int>(at + r), static_cast<int>(min(n - r, int64_t{bm})), 0};
    }
    at += n;
  }
}

// Row tile and column tile of a workgroup.  Workgroups go round the 8 XCDs, each with its own
// L2: XCD x gets the x-th eighth of the tiles, and walks it 8 row tiles by all column tiles at
// a time, row tiles first, so that workgroups running together share rows of x and of w.
__device__ __forceinline__ bool tile_of_block(const MmArgs& a, int32_t& m, int32_t& c) {
  constexpr int32_t kXcds = 8, kRun = 8;
  const int32_t mt = a.table != nullptr ? *a.count : a.mtiles, total = mt * a.ntiles;
  const int32_t per = (total + kXcds - 1) / kXcds, place = blockIdx.x / kXcds, t = blockIdx.x % kXcds * per + place;
  if (place >= per || t >= total) return false;
  const int32_t run = t / (kRun * a.ntiles), first = run * kRun, rows = min(kRun, mt - first), at = t - first * a.ntiles;
  m = first + at % rows;
  c = at / rows;
  return true;
}

struct RowTile { int32_t expert, row0, rows; };

// The row tile m, or rows = 0 past the last one.
__device__ __forceinline__ RowTile row_tile(const MmArgs& a, int32_t m, int32_t bm) {
  if (a.table == nullptr) {
    const int64_t r0 = static_cast<int64_t>(m) * bm;
    return RowTile{0, static_cast<int32_t>(r0), static_cast<int32_t>(min(a.rows - r0, int64_t{bm}))};
  }
  if (m >= *a.count) return RowTile{0, 0, 0};
  const int4 t = a.table[m];
  return RowTile{uniform(t.x), uniform(t.y), uniform(t.z)};
}

// Four adjacent outputs n .. n + 3 of one row, those below `end`.
template <class T>
__device__ __forceinline__ void store4(char* row, int64_t n, int64_t end, const f32x4& v, bool vec) {
  if (vec && n + 3 < end) {
    if constexpr (T::kBytes == 4) {
      *reinterpret_cast<f32x4*>(row + n * 4) = v;
    } else {
      const float f[8] = {v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      const u32x4 h = Chunk<T>::narrow(f);
      *reinterpret_cast<u32x2*>(row + n * 2) = u32x2{h[0], h[1]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < end) store_elem<T>(row, n + i, v[i]);
}

// ------------------------------------------------------------------ direct kernel
//
// A workgroup of 4 waves takes MT * 16 rows by 32 columns (SwiGLU: 16 gate and 16 up columns);
// each wave takes every fourth block along K straight from memory to registers, and the four
// totals are added in wave order.  The weights are read once per row tile.

constexpr int kDirectWaves = 4;

template <class T, int EPI, int MT>
__global__ __launch_bounds__(kDirectWaves* kWave) void mm_direct_kernel(MmArgs a) {
  __shared__ float red[kDirectWaves][2 * MT][kWave][4];
  const int32_t m = blockIdx.x / a.ntiles, c = blockIdx.x - m * a.ntiles;
  const RowTile rt = row_tile(a, m, MT * 16);
  if (rt.rows <= 0) return;
  const int32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int32_t r = lane % 16, g = lane / 16;
  // the two fragments' first weight rows
  const int64_t n0 = EPI == FFNWB_EPI_SWIGLU ? int64_t{c} * 16 : int64_t{c} * 32;
  const int64_t n1 = EPI == FFNWB_EPI_SWIGLU ? a.F + n0 : n0 + 16;
  const char* wp[2];
  const float* wsp[2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int64_t nf = f == 0 ? n0 : n1;
    wp[f] = a.w + (static_cast<int64_t>(rt.expert) * a.N + min(nf + r, a.N - 1)) * a.K;
    wsp[f] = a.w_scale + (static_cast<int64_t>(rt.expert) * a.nb + min(nf, a.N - 1) / kBlk) * a.kb;
  }
  const char* xp[MT];
  const float* xsp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = rt.row0 + min(i * 16 + r, rt.rows - 1);
    xp[i] = a.x + row * a.xs;
    xsp[i] = a.x_scale + row * a.xss;
  }
  f32x4 tot[2][MT] = {};
  const u32x4 zero = {0, 0, 0, 0};
  for (int32_t b = wave; b < a.kb; b += kDirectWaves) {
    const int64_t k0 = static_cast<int64_t>(b) * kBlk + g * 16, k1 = k0 + 64;
    const bool in0 = k0 < a.K, in1 = k1 < a.K;   // K is a multiple of 16
    u32x4 wv[2][2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      wv[f][0] = in0 ? *reinterpret_cast<const u32x4*>(wp[f] + k0) : zero;
      wv[f][1] = in1 ? *reinterpret_cast<const u32x4*>(wp[f] + k1) : zero;
    }
    f32x4 p[2][MT] = {};
    float xsc[MT];
    u32x4 xv[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      xsc[i] = xsp[i][b];
      xv[i][0] = in0 ? *reinterpret_cast<const u32x4*>(xp[i] + k0) : zero;
      xv[i][1] = in1 ? *reinterpret_cast<const u32x4*>(xp[i] + k1) : zero;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // 8 columns of each lane
      const u32x4 w0 = widen8(wv[0][s / 2][2 * (s % 2)], wv[0][s / 2][2 * (s % 2) + 1]);
      const u32x4 w1 = widen8(wv[1][s / 2][2 * (s % 2)], wv[1][s / 2][2 * (s % 2) + 1]);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4 x8 = widen8(xv[i][s / 2][2 * (s % 2)], xv[i][s / 2][2 * (s % 2) + 1]);
        p[0][i] = Mat<TBF16>::mul(w0, x8, p[0][i]);
        p[1][i] = Mat<TBF16>::mul(w1, x8, p[1][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const float s = xsc[i] * wsp[f][b];
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[f][i][j] = __builtin_fmaf(s, p[f][i][j], tot[f][i][j]);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(red[wave][f * MT + i][lane]) = tot[f][i];
  __syncthreads();
  for (int i = wave; i < MT; i += kDirectWaves) {
    f32x4 s[2] = {};
#pragma unroll
    for (int w = 0; w < kDirectWaves; ++w)
#pragma unroll
      for (int f = 0; f < 2; ++f) s[f] += *reinterpret_cast<const f32x4*>(red[w][f * MT + i][lane]);
    if (i * 16 + r >= rt.rows) continue;
    char* row = a.y + static_cast<int64_t>(rt.row0 + i * 16 + r) * a.ys;
    if constexpr (EPI == FFNWB_EPI_SWIGLU) {
      f32x4 h;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = swiglu(s[0][j], s[1][j]);
      store4<T>(row, n0 + g * 4, a.F, h, a.vec);
    } else {
      store4<T>(row, n0 + g * 4, a.N, s[0], a.vec);
      store4<T>(row, n1 + g * 4, a.N, s[1], a.vec);
    }
  }
}

}  // namespace ffnwb

#include "mm_tile.hpp"

namespace ffnwb {

// ------------------------------------------------------------------ quantising a product
//
// For the products whose column tiles are narrower than a block: SwiGLU results h [R, F] in
// FP32 to e4m3 rows, row tile by row tile so that rows of no expert stay as they were.
// 16 lanes take a block, as in moe_quant_fp8.

constexpr int kMqThreads = 256;

__global__ __launch_bounds__(kMqThreads) void mm_quant_kernel(MmArgs a, const float* h, int32_t bm) {
  const int32_t fb = static_cast<int32_t>((a.F + kBlk - 1) / kBlk);
  const int32_t per = (bm * fb * 16 + kMqThreads - 1) / kMqThreads;  // workgroups of a row tile
  const int32_t m = blockIdx.x / per;
  const RowTile rt = row_tile(a, m, bm);
  const int32_t u = (blockIdx.x - m * per) * (kMqThreads / 16) + threadIdx.x / 16;
  const int32_t i = u / fb, b = u - i * fb;
  const int64_t row = rt.row0 + i, f0 = static_cast<int64_t>(b) * kBlk + threadIdx.x % 16 * 8;
  const bool in = i < rt.rows && f0 < a.F;  // F is a multiple of 16
  float f[8] = {};
  if (in) {
    const f32x4* p = reinterpret_cast<const f32x4*>(h + row * a.F + f0);
    const f32x4 v0 = p[0], v1 = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = v0[j], f[4 + j] = v1[j];
  }
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
}

// ------------------------------------------------------------------ host side

constexpr int64_t kCus = 256;

static int64_t out_size(int32_t dt) { return dt == FFNWB_DT_FP32 ? 4 : dt == FFNWB_DT_FP8_E4M3 ? 1 : 2; }

int plan_grouped_matmul(const moe_grouped_matmul_fp8_desc* d, MatmulPlan* p) {
  if (d == nullptr || d->x == nullptr || d->x_scale == nullptr || d->w == nullptr || d->w_scale == nullptr || d->y == nullptr)
    return FFNWB_ERR_PARAM_NULLPTR;
  const bool quant = d->out_dtype == FFNWB_DT_FP8_E4M3, swiglu = d->epilogue == FFNWB_EPI_SWIGLU;
  if (quant && d->y_scale == nullptr) return FFNWB_ERR_PARAM_NULLPTR;
  if (d->epilogue != FFNWB_EPI_NONE && !swiglu) return FFNWB_ERR_PARAM_INVALID;
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
  const int64_t avg = (p->R + groups - 1) / groups;
  const bool fast = !quant && d->out_dtype != FFNWB_DT_FP32;
  auto shape = [&](bool tile, int64_t bm) {
    p->tile = tile, p->bm = bm;
    p->mtiles = (p->R + bm - 1) / bm + (d->group_list != nullptr ? (groups < p->R ? groups : p->R) : 0);
    p->ntiles = tile ? (swiglu ? (p->F + 127) / 128 : (p->N + 255) / 256) : (swiglu ? p->F / 16 : (p->N + 31) / 32);
    return p->mtiles * p->ntiles;
  };
  // Through LDS, with the largest tile that the groups fill on average and that leaves every CU
  // one; straight to registers where even the smallest tiles are few, and where 256 rows
  // of x pass the 32-bit offsets of the copies.
  int64_t bm = avg > 1024 && fast ? 256 : avg > 128 ? 128 : avg > 64 ? 64 : 32;
  while (bm > 32 && shape(true, bm) < kCus) bm /= 2;
  if (p->xs > (1 << 22) || shape(true, bm) < kCus / 2) shape(false, avg <= 16 ? 16 : avg <= 32 ? 32 : 64);
  // one dimension of the grid: fewer than 2^32 threads of at most 512 a workgroup
  if (p->mtiles * p->ntiles >= (int64_t{1} << 22)) return FFNWB_ERR_PARAM_INVALID;
  p->ws_bytes = 0;
  Carve c;
  if (d->group_list != nullptr && p->R > 0) {
    c.take<int32_t>(1);
    c.take<int4>(static_cast<size_t>(p->mtiles));
  }
  if (quant && !p->tile) c.take<float>(static_cast<size_t>(p->R * p->F));
  p->ws_bytes = c.off;
  return FFNWB_OK;
}

template <class T, int EPI>
static bool launch_direct(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  const dim3 grid(static_cast<uint32_t>(p.mtiles * p.ntiles)), block(kDirectWaves * kWave);
  return p.bm == 16   ? launch_bound(mm_direct_kernel<T, EPI, 1>, grid, block, 0, s, b, e, a)
         : p.bm == 32 ? launch_bound(mm_direct_kernel<T, EPI, 2>, grid, block, 0, s, b, e, a)
                     : launch_bound(mm_direct_kernel<T, EPI, 4>, grid, block, 0, s, b, e, a);
}

template <class T, int EPI, bool kQuant, bool kFast, int WM, int WN, int MF>
static bool launch_tile_shape(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  using S = TileShape<WM, WN, MF>;
  auto kernel = mm_tile_kernel<T, EPI, kQuant, kFast, WM, WN, MF>;
  allow_large_lds(reinterpret_cast<const void*>(kernel), S::kLds);
  const uint32_t grid = static_cast<uint32_t>((p.mtiles * p.ntiles + 7) / 8 * 8);
  return launch_bound(kernel, dim3(grid), dim3(S::kThreads), S::kLds, s, b, e, a);
}

template <class T, int EPI, bool kQuant = false>
static bool launch_tile(const MmArgs& a, const MatmulPlan& p, hipStream_t s, void* b, void* e) {
  constexpr bool kFast = !kQuant && T::kBytes == 2;
  if constexpr (kFast) {
    if (p.bm == 256) return launch_tile_shape<T, EPI, kQuant, kFast, 2, 4, 8>(a, p, s, b, e);
  }
  return p.bm == 128  ? launch_tile_shape<T, EPI, kQuant, kFast, 2, 4, 4>(a, p, s, b, e)
         : p.bm == 64 ? launch_tile_shape<T, EPI, kQuant, kFast, 2, 4, 2>(a, p, s, b, e)
                      : launch_tile_shape<T, EPI, kQuant, kFast, 1, 4, 2>(a, p, s, b, e);
}

int launch_grouped_matmul(const moe_grouped_matmul_fp8_desc* d, const MatmulPlan& p, void* ws, hipStream_t s) {
  if (p.R == 0) return FFNWB_OK;
  const bool quant = d->out_dtype == FFNWB_DT_FP8_E4M3;
  MmArgs a{};
  a.rows = p.R, a.K = p.K, a.N = p.N, a.F = p.F;
  a.xs = p.xs, a.xss = p.xss, a.ys = p.ys, a.yss = p.yss;
  a.kb = static_cast<int32_t>(p.kb), a.nb = static_cast<int32_t>(p.nb), a.ntiles = static_cast<int32_t>(p.ntiles);
  a.mtiles = static_cast<int32_t>(p.mtiles);
  a.x = static_cast<const char*>(d->x), a.x_scale = d->x_scale;
  a.w = static_cast<const char*>(d->w), a.w_scale = d->w_scale;
  a.y = static_cast<char*>(d->y), a.y_scale = d->y_scale;
  Carve c;
  c.base = static_cast<char*>(ws);
  if (d->group_list != nullptr) {
    int32_t* count = c.take<int32_t>(1);
    int4* table = c.take<int4>(static_cast<size_t>(p.mtiles));
    hipLaunchKernelGGL(mm_table_kernel, dim3(1), dim3(kTableThreads), 0, s, d->group_list, static_cast<int32_t>(d->num_groups),
                       p.R, d->num_experts, static_cast<int32_t>(p.bm), table, count);
    if (hipGetLastError() != hipSuccess) return FFNWB_ERR_RUNTIME;
    a.table = table, a.count = count;
  }
  const int64_t quad = 4 * out_size(d->out_dtype);
  a.vec = ((reinterpret_cast<uintptr_t>(a.y) | static_cast<uintptr_t>(p.ys)) & (quad - 1)) == 0;
  void *b = d->ev_matmul_begin, *e = d->ev_matmul_end;
  if (p.tile) {
    bool ok;
    if (d->epilogue == FFNWB_EPI_SWIGLU) {
      ok = quant                           ? launch_tile<TF32, FFNWB_EPI_SWIGLU, true>(a, p, s, b, e)
           : d->out_dtype == FFNWB_DT_FP16 ? launch_tile<TF16, FFNWB_EPI_SWIGLU>(a, p, s, b, e)
           : d->out_dtype == FFNWB_DT_BF16 ? launch_tile<TBF16, FFNWB_EPI_SWIGLU>(a, p, s, b, e)
                                           : launch_tile<TF32, FFNWB_EPI_SWIGLU>(a, p, s, b, e);
    } else {
      ok = d->out_dtype == FFNWB_DT_FP16   ? launch_tile<TF16, FFNWB_EPI_NONE>(a, p, s, b, e)
           : d->out_dtype == FFNWB_DT_BF16 ? launch_tile<TBF16, FFNWB_EPI_NONE>(a, p, s, b, e)
                                           : launch_tile<TF32, FFNWB_EPI_NONE>(a, p, s, b, e);
    }
    return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
  }
  float* h = quant ? c.take<float>(static_cast<size_t>(p.R * p.F)) : nullptr;
  if (quant) a.y = reinterpret_cast<char*>(h), a.ys = p.F * 4, a.vec = true;
  bool ok;
  if (d->epilogue == FFNWB_EPI_SWIGLU) {
    ok = d->out_dtype == FFNWB_DT_FP16   ? launch_direct<TF16, FFNWB_EPI_SWIGLU>(a, p, s, b, e)
         : d->out_dtype == FFNWB_DT_BF16 ? launch_direct<TBF16, FFNWB_EPI_SWIGLU>(a, p, s, b, e)
                                         : launch_direct<TF32, FFNWB_EPI_SWIGLU>(a, p, s, b, e);
  } else {
    ok = d->out_dtype == FFNWB_DT_FP16   ? launch_direct<TF16, FFNWB_EPI_NONE>(a, p, s, b, e)
         : d->out_dtype == FFNWB_DT_BF16 ? launch_direct<TBF16, FFNWB_EPI_NONE>(a, p, s, b, e)
                                         : launch_direct<TF32, FFNWB_EPI_NONE>(a, p, s, b, e);
  }
  if (!ok) return FFNWB_ERR_RUNTIME;
  if (quant) {
    a.y = static_cast<char*>(d->y), a.ys = p.ys;
    const int64_t bm = p.bm, fb = (p.F + 127) / 128, per = (bm * fb * 16 + kMqThreads - 1) / kMqThreads;
    hipLaunchKernelGGL(mm_quant_kernel, dim3(static_cast<uint32_t>(p.mtiles * per)), dim3(kMqThreads), 0, s, a, h,
                       static_cast<int32_t>(bm));
    if (hipGetLastError() != hipSuccess) return FFNWB_ERR_RUNTIME;
  }
  return FFNWB_OK;
}

}  // namespace ffnwb
