// Row tiles of the experts' products: which rows of x belong to which expert, cut into tiles of `bm`
// rows, and the tile that a workgroup takes.  Args: any of the products' argument structures, with the
// members rows, ntiles, ngroups, nexperts, groups, table and count.
#pragma once

#include "fp8_block.hpp"
#include "internal.hpp"

namespace ffnwb {

// Sums over the lanes up to and including this one, saturating at `cap` (terms are >= 0, so the
// order of the additions does not matter).
__device__ __forceinline__ int32_t wave_scan(int32_t v, int32_t cap) {
#define FFNWB_SCAN_STEP(ctrl, rows) v = min(v + __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xf, false), cap)
  FFNWB_SCAN_STEP(0x111, 0xf);  // within rows of 16 lanes: one lane below, two, four, eight
  FFNWB_SCAN_STEP(0x112, 0xf);
  FFNWB_SCAN_STEP(0x114, 0xf);
  FFNWB_SCAN_STEP(0x118, 0xf);
  FFNWB_SCAN_STEP(0x142, 0xa);  // lane 15 of a row into the next row, lane 31 into the upper half
  FFNWB_SCAN_STEP(0x143, 0xc);
#undef FFNWB_SCAN_STEP
  return v;
}

// Rows of a group that starts at row `at`, and whether they belong to an expert.
__device__ __forceinline__ int32_t group_rows(int64_t count, int32_t at, int32_t rows) {
  return static_cast<int32_t>(min(max(count, int64_t{0}), static_cast<int64_t>(rows - at)));
}

struct RowTile { int32_t expert, row0, rows; };

constexpr int kWaveGroups = 256;  // groups that one wave lists by itself, four to a lane

// The row tiles of all groups, as every wave of a product's kernel works them out for itself:
// for up to 256 groups that costs a kernel about 1 us, and a launch of its own 5 us.
struct WaveTiles {
  int32_t tiles = 0, first_tile = 0, first_row = 0;  // of this lane's groups
  int32_t total = 0;
  int32_t key[4], n[4];
  template <class Args>
  __device__ void list(const Args& a, int32_t bm) {
    const int32_t g0 = 4 * static_cast<int32_t>(lane_id());
    int64_t cnt[4];
    int32_t mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = g0 + j < a.ngroups;
      const int64_t k = in ? a.groups[2 * (g0 + j)] : -1;
      cnt[j] = in ? a.groups[2 * (g0 + j) + 1] : 0;
      key[j] = k >= 0 && k < a.nexperts ? static_cast<int32_t>(k) : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) mine = min(mine + group_rows(cnt[j], 0, a.rows), a.rows);
    const int32_t upto = wave_scan(mine, a.rows);
    // rows before this lane's: a saturated sum does not subtract, so take the neighbour's
    first_row = __shfl_up(upto, 1);
    if (g0 == 0) first_row = 0;
    int32_t at = first_row;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      n[j] = group_rows(cnt[j], at, a.rows);
      at += n[j];
      if (key[j] >= 0) tiles += (n[j] + bm - 1) / bm;
    }
    const int32_t incl = wave_scan(tiles, 0x7fffffff);
    first_tile = incl - tiles;
    total = __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  __device__ RowTile at(int32_t m, int32_t bm) const {
    const uint64_t has = wave_ballot(first_tile <= m && m < first_tile + tiles);
    const int32_t lane = __builtin_ctzll(has);
    int32_t t = m - first_tile, row = first_row;
    int4 f = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t here = key[j] >= 0 ? (n[j] + bm - 1) / bm : 0;
      if (t >= 0 && t < here) f = int4{key[j], row + t * bm, min(n[j] - t * bm, bm), 0};
      t -= here;
      row += n[j];
    }
    return RowTile{__builtin_amdgcn_readlane(f.x, lane), __builtin_amdgcn_readlane(f.y, lane), __builtin_amdgcn_readlane(f.z, lane)};
  }
};

constexpr int kTableThreads = 1024;

// The same list for more groups, in a launch of its own.  Each thread counts a run of consecutive
// groups and leaves their first rows and tiles in LDS; then the waves write the tiles, a group each at a
// time, 64 tiles at once (with a thread to a group, 820 tiles of two groups took 16 us).  The table
// has at most ceil(rows / bm) + min(groups, rows) entries.
template <class Args>
__global__ __launch_bounds__(kTableThreads) void mm_table_kernel(Args a, int32_t bm, int4* table, int32_t* count) {
  __shared__ int32_t wave_rows[kTableThreads / kWave], wave_tiles[kTableThreads / kWave];
  __shared__ int32_t first_row[kMaxExperts], first_tile[kMaxExperts];
  const int32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
  const int32_t per = (a.ngroups + kTableThreads - 1) / kTableThreads;
  const int32_t g0 = threadIdx.x * per, g1 = min(g0 + per, a.ngroups);
  int32_t mine = 0;
  for (int32_t g = g0; g < g1; ++g) mine = min(mine + group_rows(a.groups[2 * g + 1], 0, a.rows), a.rows);
  int32_t incl = wave_scan(mine, a.rows);
  int32_t first = __shfl_up(incl, 1);
  if (lane == 0) first = 0;
  if (lane == kWave - 1) wave_rows[wave] = incl;
  __syncthreads();
  for (int32_t w = 0; w < wave; ++w) first = min(first + wave_rows[w], a.rows);
  int32_t at = first, tiles = 0;
  for (int32_t g = g0; g < g1; ++g) {
    const int32_t n = group_rows(a.groups[2 * g + 1], at, a.rows);
    const int64_t key = a.groups[2 * g];
    first_row[g] = at;
    first_tile[g] = tiles;
    if (key >= 0 && key < a.nexperts) tiles += (n + bm - 1) / bm;
    at += n;
  }
  incl = wave_scan(tiles, 0x7fffffff);
  if (lane == kWave - 1) wave_tiles[wave] = incl;
  __syncthreads();
  int32_t t = incl - tiles;
  for (int32_t w = 0; w < wave; ++w) t += wave_tiles[w];
  if (threadIdx.x == kTableThreads - 1) *count = t + tiles;
  for (int32_t g = g0; g < g1; ++g) first_tile[g] += t;
  __syncthreads();
  // 64 groups of a wave: one to a lane, then lane by lane, all lanes to the group's tiles
  for (int32_t base = wave * kWave; base < a.ngroups; base += kTableThreads) {
    const int32_t g = base + lane;
    int32_t key = -1, row = 0, n = 0, tile = 0;
    if (g < a.ngroups) {
      const int64_t k = a.groups[2 * g];
      row = first_row[g];
      n = group_rows(a.groups[2 * g + 1], row, a.rows);
      tile = first_tile[g];
      if (k >= 0 && k < a.nexperts && n > 0) key = static_cast<int32_t>(k);
    }
    if (key >= 0) table[tile] = int4{key, row, min(n, bm), 0};
    for (uint64_t more = wave_ballot(key >= 0 && n > bm); more != 0; more &= more - 1) {
      const int32_t l = __builtin_ctzll(more);
      const int32_t k = __builtin_amdgcn_readlane(key, l), r0 = __builtin_amdgcn_readlane(row, l);
      const int32_t rows = __builtin_amdgcn_readlane(n, l), t0 = __builtin_amdgcn_readlane(tile, l);
      for (int32_t j = lane + 1; j * bm < rows; j += kWave) table[t0 + j] = int4{k, r0 + j * bm, min(rows - j * bm, bm), 0};
    }
  }
}

// The row tile and column tile of a workgroup; false for a workgroup without one.  Workgroups go
// round the 8 XCDs, each with its own L2: XCD x gets the x-th eighth of the tiles, and walks it
// 8 row tiles by all column tiles at a time, row tiles first, so that workgroups running
// together share rows of x and of w.  kHalve, for tiles of which a CU holds one: where the last
// round of tiles would leave half of the CUs idle, each of its tiles is two of half the rows (8191
// rows by 7168 columns over 5120, 3.5 rounds of 256 x 256: 316 us without, 291 us with, on one box;
// 4096 by 4096 over 4096, one full round, pays 0.8 of 68 us for the test).
constexpr int32_t kXcds = 8, kXcdCus = 32;
constexpr int kHalvedFragments = 4;  // least row fragments of a wave whose tiles are halved

template <bool kHalve = false, class Args>
__device__ __forceinline__ bool find_tile(const Args& a, int32_t bm, RowTile& rt, int32_t& c) {
  constexpr int32_t kRun = 8;
  WaveTiles wt;
  int32_t mt;
  if (a.groups == nullptr) mt = (a.rows + bm - 1) / bm;
  else if (a.table != nullptr) mt = *a.count;
  else wt.list(a, bm), mt = wt.total;
  const int32_t total = mt * a.ntiles;
  const int32_t per = (total + kXcds - 1) / kXcds;
  int32_t place = blockIdx.x / kXcds, half = -1;
  if constexpr (kHalve) {
    const int32_t rest = per % kXcdCus, whole = per - rest;
    if (2 * rest <= kXcdCus && place >= whole) half = (place - whole) % 2, place = whole + (place - whole) / 2;
  }
  const int32_t t = blockIdx.x % kXcds * per + place;
  if (place >= per || t >= total) return false;
  const int32_t run = t / (kRun * a.ntiles), first = run * kRun, rows = min(kRun, mt - first), in = t - first * a.ntiles;
  const int32_t m = first + in % rows;
  c = in / rows;
  if (a.groups == nullptr) {
    rt = RowTile{0, m * bm, min(a.rows - m * bm, bm)};
  } else if (a.table != nullptr) {
    const int4 v = a.table[m];
    rt = RowTile{uniform(v.x), uniform(v.y), uniform(v.z)};
  } else {
    rt = wt.at(m, bm);
  }
  if (kHalve && half >= 0) {
    const int32_t first = half * (bm / 2);
    rt.row0 += first;
    rt.rows = min(rt.rows - first, bm / 2);
  }
  return rt.rows > 0;
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

// Workgroups round the XCDs (find_tile): a multiple of 8.
inline uint32_t tile_grid(int64_t tiles) { return static_cast<uint32_t>((tiles + kXcds - 1) / kXcds * kXcds); }

}  // namespace ffnwb
