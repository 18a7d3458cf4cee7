// A whole expert layer for a few tokens, in two launches.
//
// With at most 64 tokens the layer is the reading of its distinct experts' weights, once each:
// everything else is small.  Launch 1 (gate and up products, SwiGLU) takes 16 columns of F of
// one distinct expert per workgroup; launch 2 (down product, weighted sum) takes 16 columns of
// H per workgroup and walks all experts, so the sum over a token's experts stays in one
// workgroup: no atomics, no third launch, the same bits on every run.
//
// Weights are the A operand of 16x16x32 matrix instructions (16 weight rows by 32 columns),
// straight from memory to registers; up to 16 tokens of the expert are the B operand.  e4m3
// weights become the 16-bit type of the activations exactly, and the total of each 128-column
// block is added to an FP32 sum times the block's scale.  h goes from launch 1 to launch 2 as a
// pair of BF16 numbers hi + lo (16 significant bits in the range of FP32): one BF16 would cost
// as much accuracy as the rounding of y itself, FP16 could overflow, and the second product is
// free while the weights are being read.
//
// Bound by memory: 16 tokens with 9 of 256 experts (hidden 7168, inter 1024) take 432 us, 5.0 TB/s;
// 64 with 8 of 64 in BF16 (4096, 1024) 327 us, 4.9; one token with 9 (7168, 2048) 79 us, 4.8.  64
// tokens with 8 of 64 in e4m3 (4096, 1024) take 253 us, 3.2 TB/s.  A toy layer takes 10 us, the two
// launches.
#include "fp8_block.hpp"
#include "internal.hpp"

namespace ffnwb {

constexpr int kLyMaxTokens = 64;
constexpr int kLyMaxSlots = 64;
constexpr int kUpMaxWaves = 8, kDownWaves = 8;

struct LayerArgs {
  int32_t T, K, E, H, F;
  int32_t hb, fb;             // 128-blocks of H and F
  int32_t nb13;               // 128-blocks of 2 F
  int32_t ctiles;             // 16-column tiles of F
  int32_t groups_max;         // most groups of launch 2
  int32_t id64;
  int32_t scale_dtype;
  int64_t xs, ys, is, ss, ms;
  const char* x;
  const void* ids;
  const void* scales;
  const uint8_t* mask;
  const char* w13;
  const float* w13s;
  const char* w2;
  const float* w2s;
  char* y;
  // workspace
  int32_t* groups;            // [1] groups of at most 16 tokens of one expert
  int32_t* expert;            // [groups] ascending ids
  int32_t* first;             // [groups + 1] first entry of each
  int32_t* slot;              // [T * K] entries: t * K + k, tokens ascending within an expert
  float* weight;              // [T * K] the token's weight for the expert
  char* hhi;                  // [T * K, F] BF16
  char* hlo;
  int32_t parts;              // workgroups of a column tile of launch 2
  int32_t* arrived;           // [H / 16] of them that are done (more than one part)
  float* partial;             // [H / 16, parts, T, 16]
};

// ------------------------------------------------------------------ operands

// One lane's share of 16 weight rows by 128 columns: four steps of 8 columns.  e4m3: a 16-byte
// load holds 16 columns, two steps; BF16: 8 columns, one step.
template <class T, bool kFp8>
struct Weights {
  static constexpr int kLoads = kFp8 ? 2 : 4;
  static constexpr int kElt = kFp8 ? 1 : 2;
  u32x4 v[kLoads];
  // column of step s, for the lanes of group g
  __device__ static int32_t col(int s, int32_t g) { return kFp8 ? (s / 2) * 64 + g * 16 + (s % 2) * 8 : s * 32 + g * 8; }
  // Columns c0 .. c0 + 127 of a row of `end`; past its end, the row's last columns (no branch in
  // the way of the loads), which `cut` clears.
  __device__ void load(const char* row, int32_t c0, int32_t g, int32_t end) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      v[i] = load16(row + static_cast<int64_t>(min(c0 + col(kFp8 ? 2 * i : i, g), end - 16 / kElt)) * kElt);
  }
  __device__ void cut(int32_t c0, int32_t g, int32_t end) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (c0 + col(kFp8 ? 2 * i : i, g) >= end) v[i] = u32x4{0, 0, 0, 0};
  }
  __device__ u32x4 step(int s) const {
    if constexpr (kFp8) {
      const uint32_t a = v[s / 2][2 * (s % 2)], b = v[s / 2][2 * (s % 2) + 1];
      return u32x4{Mat<T>::widen(a, false), Mat<T>::widen(a, true), Mat<T>::widen(b, false), Mat<T>::widen(b, true)};
    } else {
      return v[s];
    }
  }
};

// ------------------------------------------------------------------ routing

// The id of slot (t, k), or -1 when it takes no part.
__device__ __forceinline__ int32_t active_id(const LayerArgs& a, int32_t i) {
  const int32_t t = i / a.K, k = i - t * a.K;
  const int64_t at = t * a.is + k;
  const int64_t id = a.id64 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
  const bool on = a.mask == nullptr || a.mask[t * a.ms + k] != 0;
  return on && id >= 0 && id < a.E ? static_cast<int32_t>(id) : -1;
}

// All ids into LDS and one bit for each expert that occurs.
__device__ __forceinline__ void load_ids(const LayerArgs& a, int16_t* ids, uint32_t* bits) {
  for (int32_t i = threadIdx.x; i < kMaxExperts / 32; i += blockDim.x) bits[i] = 0;
  __syncthreads();
  for (int32_t i = threadIdx.x; i < a.T * a.K; i += blockDim.x) {
    const int32_t id = active_id(a, i);
    ids[i] = static_cast<int16_t>(id);  // below 8192
    if (id >= 0) atomicOr(&bits[id / 32], 1u << (id % 32));
  }
  __syncthreads();
}

// Bits set in the words below each lane's four (wave 0 holds all 256 words), and in all.
__device__ __forceinline__ int32_t bits_below(const uint32_t* bits, int32_t lane, int32_t& total) {
  int32_t mine = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) mine += __popc(bits[4 * lane + j]);
  int32_t incl = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int32_t v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  total = __shfl(incl, kWave - 1);
  return incl - mine;
}

__device__ __forceinline__ float slot_scale(const LayerArgs& a, int32_t t, int32_t k) {
  if (a.scales == nullptr) return 1.0f;
  const int64_t at = t * a.ss + k;
  return a.scale_dtype == FFNWB_DT_FP32   ? load_elem<TF32>(a.scales, at)
         : a.scale_dtype == FFNWB_DT_BF16 ? load_elem<TBF16>(a.scales, at)
                                          : load_elem<TF16>(a.scales, at);
}

// Workgroup 0 of launch 1: the experts, their tokens (in groups of up to 16, one matrix operand)
// and weights, for launch 2.  An expert's tokens are the bits of a mask, so that every slot finds
// its entry's place by counting bits; a token that names an expert twice has one entry, at its
// first slot, with the sum of the weights.
template <int kIds>
struct TableLds {
  int16_t ids[kIds];
  uint16_t first[kIds];      // [rank] first entry
  uint32_t mask[kIds][2];    // [rank] tokens
};

template <int kIds>
__device__ void build_table(const LayerArgs& a, TableLds<kIds>& s, const uint32_t* bits, int32_t* below) {
  const int32_t n = a.T * a.K, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  constexpr int kWords = kMaxExperts / 32;  // of the experts' bits, one to a thread (of at least as many)
  __shared__ int32_t sums[2][kUpMaxWaves];
  if (a.parts > 1)
    for (int32_t i = threadIdx.x; i < a.H / 16; i += blockDim.x) a.arrived[i] = 0;
  if (threadIdx.x < kWave) {
    int32_t total;
    int32_t at = bits_below(bits, lane, total);
    for (int j = 0; j < 4; ++j) {
      below[4 * lane + j] = at;
      at += __popc(bits[4 * lane + j]);
    }
    if (lane == 0) below[kMaxExperts / 32] = total;
  }
  __syncthreads();
  const int32_t ranks = below[kMaxExperts / 32];
  for (int32_t i = threadIdx.x; i < ranks; i += blockDim.x) s.mask[i][0] = s.mask[i][1] = 0;
  __syncthreads();
  auto rank = [&](int32_t e) { return below[e / 32] + __popc(bits[e / 32] & ((1u << (e % 32)) - 1)); };
  for (int32_t i = threadIdx.x; i < n; i += blockDim.x) {
    const int32_t t = i / a.K;
    if (s.ids[i] >= 0) atomicOr(&s.mask[rank(s.ids[i])][t / 32], 1u << (t % 32));
  }
  __syncthreads();
  // exclusive sums of entries and of groups over the experts
  const uint32_t word = threadIdx.x < kWords ? bits[threadIdx.x] : 0;
  const int32_t r0 = threadIdx.x < kWords ? below[threadIdx.x] : ranks, r1 = r0 + __popc(word);
  auto tokens = [&](int32_t r) { return __popc(s.mask[r][0]) + __popc(s.mask[r][1]); };
  int32_t mine = 0, mine_g = 0;
  for (int32_t r = r0; r < r1; ++r) mine += tokens(r), mine_g += (tokens(r) + 15) / 16;
  int32_t incl = mine, incl_g = mine_g;
  for (int d = 1; d < kWave; d <<= 1) {
    const int32_t v = __shfl_up(incl, d), vg = __shfl_up(incl_g, d);
    if (lane >= d) incl += v, incl_g += vg;
  }
  if (lane == kWave - 1) sums[0][wave] = incl, sums[1][wave] = incl_g;
  __syncthreads();
  int32_t at = incl - mine, group = incl_g - mine_g;
  for (int32_t w = 0; w < wave; ++w) at += sums[0][w], group += sums[1][w];
  uint32_t m = word;
  for (int32_t r = r0; r < r1; ++r, m &= m - 1) {
    s.first[r] = static_cast<uint16_t>(at);
    const int32_t c = tokens(r);
    for (int32_t i = 0; i < c; i += 16) {
      a.expert[group] = static_cast<int32_t>(threadIdx.x) * 32 + __builtin_ctz(m);
      a.first[group++] = at + i;
    }
    at += c;
  }
  if (threadIdx.x == blockDim.x - 1) {
    *a.groups = group;
    a.first[group] = at;
  }
  __syncthreads();
  for (int32_t i = threadIdx.x; i < n; i += blockDim.x) {
    const int32_t e = s.ids[i], t = i / a.K, t0 = t * a.K;
    if (e < 0) continue;
    bool head = true;
    for (int32_t j = t0; j < i; ++j) head = head && s.ids[j] != e;
    if (!head) continue;
    float w = 0.0f;
    for (int32_t j = i; j < t0 + a.K; ++j)
      if (s.ids[j] == e) w += slot_scale(a, t, j - t0);
    const int32_t r = rank(e);
    const uint32_t lo = t < 32 ? s.mask[r][0] & ((1u << t) - 1) : s.mask[r][0];
    const uint32_t hi = t < 32 ? 0u : s.mask[r][1] & ((1u << (t - 32)) - 1);
    const int32_t entry = s.first[r] + __popc(lo) + __popc(hi);
    a.slot[entry] = i;
    a.weight[entry] = w;
  }
}

// ------------------------------------------------------------------ launch 1: gate, up, SwiGLU

// h of 16 columns from f0 of expert e for its `count` tokens (at most MT * 16); list[j] is token
// j's slot.  The waves of a tile take the 128-blocks of H in turn; their totals are added in
// order.  With kSplit = 1 every wave has a tile of its own (f0 may then be past F).
template <class T, bool kFp8, int MT, int kSplit>
__device__ void up_tile(const LayerArgs& a, int32_t e, int32_t f0, int32_t count, const int32_t* list, float* red) {
  using W = Weights<T, kFp8>;
  const int32_t lane = threadIdx.x % kWave, r = lane % 16, g = lane / 16;
  const int32_t wave = kSplit == 1 ? 0 : uniform(threadIdx.x / kWave);
  if (kSplit == 1 && f0 >= a.F) return;
  const int64_t rowb = static_cast<int64_t>(a.H) * W::kElt;
  const char* wp[2] = {a.w13 + (static_cast<int64_t>(e) * 2 * a.F + f0 + r) * rowb,
                       a.w13 + (static_cast<int64_t>(e) * 2 * a.F + a.F + f0 + r) * rowb};
  const float* wsp[2] = {nullptr, nullptr};
  if constexpr (kFp8) {
    wsp[0] = a.w13s + (static_cast<int64_t>(e) * a.nb13 + f0 / kBlk) * a.hb;
    wsp[1] = a.w13s + (static_cast<int64_t>(e) * a.nb13 + (a.F + f0) / kBlk) * a.hb;
  }
  const char* xp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xp[i] = a.x + (list[min(i * 16 + r, count - 1)] / a.K) * a.xs;
  f32x4 tot[2][MT] = {};
  // the next block's weights (and, for up to 16 tokens, its activations) are on their way while
  // one is multiplied
  struct Block {
    W w[2];
    u32x4 x[MT == 1 ? 4 : 1];
  } blk[2];
  auto x_at = [&](int i, int32_t c) { return load16(xp[i] + static_cast<int64_t>(min(c, a.H - 8)) * 2); };
  auto load = [&](Block& v, int32_t b) {
    if (b >= a.hb) return;
    v.w[0].load(wp[0], b * kBlk, g, a.H);
    v.w[1].load(wp[1], b * kBlk, g, a.H);
    if constexpr (MT == 1) {
#pragma unroll
      for (int s = 0; s < 4; ++s) v.x[s] = x_at(0, b * kBlk + W::col(s, g));
    }
  };
  auto multiply = [&](Block& v, int32_t b) {
    if (b >= a.hb) return;
    const float s0 = kFp8 ? load_f32(wsp[0] + b) : 1.0f, s1 = kFp8 ? load_f32(wsp[1] + b) : 1.0f;
    const bool tail = (b + 1) * kBlk > a.H;
    if (tail) {
      v.w[0].cut(b * kBlk, g, a.H);
      v.w[1].cut(b * kBlk, g, a.H);
    }
    f32x4 p[2][MT] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const u32x4 w0 = v.w[0].step(s), w1 = v.w[1].step(s);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        u32x4 xv;
        if constexpr (MT == 1) xv = v.x[s];
        else xv = x_at(i, b * kBlk + W::col(s, g));
        if (tail && b * kBlk + W::col(s, g) >= a.H) xv = u32x4{0, 0, 0, 0};
        p[0][i] = Mat<T>::mul(w0, xv, p[0][i]);
        p[1][i] = Mat<T>::mul(w1, xv, p[1][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tot[0][i][j] = __builtin_fmaf(s0, p[0][i][j], tot[0][i][j]);
        tot[1][i][j] = __builtin_fmaf(s1, p[1][i][j], tot[1][i][j]);
      }
  };
  load(blk[0], wave);
  for (int32_t b = wave; b < a.hb; b += 2 * kSplit) {
    load(blk[1], b + kSplit);
    multiply(blk[0], b);
    load(blk[0], b + 2 * kSplit);
    multiply(blk[1], b + kSplit);
  }
  f32x4* rv = reinterpret_cast<f32x4*>(red);  // [wave][2 MT][lane]
  if constexpr (kSplit > 1) {
    __syncthreads();  // the ids share red's memory
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      rv[(wave * 2 * MT + i) * kWave + lane] = tot[0][i];
      rv[(wave * 2 * MT + MT + i) * kWave + lane] = tot[1][i];
    }
    __syncthreads();
  }
#pragma unroll
  for (int32_t i = 0; i < MT; ++i) {
    const int32_t j = i * 16 + r;
    if (j >= count || (kSplit > 1 && i % kSplit != wave)) continue;
    f32x4 gv = tot[0][i], uv = tot[1][i];
    if constexpr (kSplit > 1) {
      gv = uv = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int32_t w = 0; w < kSplit; ++w) {
        gv += rv[(w * 2 * MT + i) * kWave + lane];
        uv += rv[(w * 2 * MT + MT + i) * kWave + lane];
      }
    }
    u32x2 hi = {}, lo = {};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float h = swiglu(gv[q], uv[q]);
      const uint32_t hb16 = f32_to_bf16_rne(h);
      // an infinite or NaN h has no remainder
      const float rest = h - bf16_to_f32(hb16);
      const uint32_t lb16 = (hb16 & 0x7f80u) == 0x7f80u ? 0u : f32_to_bf16_rne(rest);
      hi[q / 2] |= hb16 << (16 * (q % 2));
      lo[q / 2] |= lb16 << (16 * (q % 2));
    }
    const int64_t at = (static_cast<int64_t>(list[j]) * a.F + f0 + g * 4) * 2;
    *reinterpret_cast<u32x2*>(a.hhi + at) = hi;
    *reinterpret_cast<u32x2*>(a.hlo + at) = lo;
  }
}

// h of one expert's tokens, 16 to an operand.
template <class T, bool kFp8, int kTokens, int kSplit>
__device__ __forceinline__ void up_tokens(const LayerArgs& a, int32_t e, int32_t f0, int32_t n, const int32_t* list, float* red) {
  if constexpr (kTokens == 16) {
    up_tile<T, kFp8, 1, kSplit>(a, e, f0, n, list, red);
  } else {
    if (n <= 16) up_tile<T, kFp8, 1, kSplit>(a, e, f0, n, list, red);
    else if (n <= 32) up_tile<T, kFp8, 2, kSplit>(a, e, f0, n, list, red);
    else up_tile<T, kFp8, 4, kSplit>(a, e, f0, n, list, red);
  }
}

// kTokens: the most tokens, 16 or 64.  The registers and LDS of 64 leave a CU 3 workgroups of 4
// waves, those of 16 leave it 4 (one token's layer of hidden 7168 and inter 2048, 1152 workgroups:
// 58 us with the former, 46 us with the latter).
template <class T, bool kFp8, int kTokens, int kSplit>
__global__ __launch_bounds__((kSplit == 1 ? 4 : kSplit) * kWave) void layer_up_kernel(LayerArgs a) {
  extern __shared__ __align__(16) char scratch[];  // the table's, then the waves' totals
  __shared__ uint32_t bits[kMaxExperts / 32];
  __shared__ int32_t below[kMaxExperts / 32 + 1];
  __shared__ int32_t lists[kUpMaxWaves][kLyMaxTokens];
  __shared__ int32_t chosen, count;
  using Table = TableLds<kTokens * kLyMaxSlots>;
  Table& table = *reinterpret_cast<Table*>(scratch);
  int16_t* ids = table.ids;
  float* red = reinterpret_cast<float*>(scratch);
  const int32_t per = kSplit == 1 ? (a.ctiles + 3) / 4 : a.ctiles;  // workgroups of an expert
  const int32_t rank = (static_cast<int32_t>(blockIdx.x) - 1) / per;
  const int32_t c = (static_cast<int32_t>(blockIdx.x) - 1 - rank * per) * (kSplit == 1 ? 4 : 1) +
                    (kSplit == 1 ? static_cast<int32_t>(threadIdx.x / kWave) : 0);
  const int32_t lane = threadIdx.x % kWave;
  if (blockIdx.x != 0 && a.T * a.K <= kWave) {
    // Up to 64 slots are one to a lane, and every wave finds the workgroup's expert (the rank-th
    // in the order of the slots) by itself: two barriers and a pass through LDS less.
    int32_t* list = lists[threadIdx.x / kWave];
    const int32_t id = lane < a.T * a.K ? active_id(a, lane) : -1;
    uint64_t rest = wave_ballot(id >= 0);
    for (int32_t k = 0; k < rank && rest != 0; ++k)
      rest &= ~wave_ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(rest)));
    if (rest == 0) return;
    const int32_t e = __builtin_amdgcn_readlane(id, __builtin_ctzll(rest));
    const uint64_t has = wave_ballot(id == e);
    const uint64_t before = (uint64_t{1} << lane) - 1, token = before & ~((uint64_t{1} << (lane / a.K * a.K)) - 1);
    const bool head = id == e && (has & token) == 0;  // the token's first slot with e
    const uint64_t heads = wave_ballot(head);
    if (head) list[count_below(heads)] = lane;
    wave_lds_sync();
    const int32_t n = __popcll(heads);
    up_tokens<T, kFp8, kTokens, kSplit>(a, e, c * 16, n, list, red);
    return;
  }
  int32_t* list = lists[0];
  load_ids(a, ids, bits);
  if (blockIdx.x == 0) {
    build_table(a, table, bits, below);
    return;
  }
  if (threadIdx.x < kWave) {
    int32_t total;
    const int32_t below4 = bits_below(bits, lane, total);
    if (lane == 0 && rank >= total) chosen = -1;
    int32_t left = rank - below4;  // the rank's place among this lane's bits
    for (int j = 0; j < 4; ++j) {
      uint32_t m = bits[4 * lane + j];
      const int32_t here = __popc(m);
      if (left >= 0 && left < here) {
        for (; left > 0; --left) m &= m - 1;
        chosen = (4 * lane + j) * 32 + __builtin_ctz(m);
        left = -1;
      } else {
        left -= here;
      }
    }
    wave_lds_sync();
    const int32_t e = chosen;
    int32_t slot = -1;
    if (e >= 0 && lane < a.T)
      for (int32_t k = a.K - 1; k >= 0; --k)
        if (ids[lane * a.K + k] == e) slot = lane * a.K + k;
    const uint64_t has = wave_ballot(slot >= 0);
    if (slot >= 0) list[count_below(has)] = slot;
    if (lane == 0) count = __popcll(has);
  }
  __syncthreads();
  const int32_t e = uniform(chosen), n = uniform(count);
  if (e < 0) return;
  up_tokens<T, kFp8, kTokens, kSplit>(a, e, c * 16, n, list, red);
}

// ------------------------------------------------------------------ launch 2: down, weighted sum

// 16 columns of H.  The 128-blocks of F of all groups are numbered in one row and dealt to the
// waves in turn; each wave adds its totals, times the tokens' weights, into sums of its own
// [T][16], which are added in wave order.  The table of experts and entries is copied to LDS
// first, so that only the loads of weights and h themselves go to memory in the loop, and those
// of a wave's next block are issued before its present one is multiplied.  A group of up to 8
// tokens takes the upper and lower parts of h as the two halves of one operand, which halves the
// loads of h: they cost more of the CU's load path than e4m3 weights do (16 tokens' layer of
// hidden 7168 519 -> 457 us).  BF16 weights are twice as many bytes, and their two blocks fill the
// registers: they always take the parts apart (64 tokens, hidden 4096: 131 us, with the choice 177).
template <class T, bool kFp8>
__global__ __launch_bounds__(kDownWaves* kWave, 4) void layer_down_kernel(LayerArgs a) {
  using W = Weights<TBF16, kFp8>;
  extern __shared__ __align__(16) float acc[];  // [waves][T][16], then the table
  const int32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave), r = lane % 16, g = lane / 16;
  const int32_t tile = blockIdx.x / a.parts, part = blockIdx.x - tile * a.parts, n0 = tile * 16;
  const int32_t groups = uniform(*a.groups);
  int32_t* le = reinterpret_cast<int32_t*>(acc + kDownWaves * a.T * 16);  // [groups] experts
  int32_t* lf = le + a.groups_max;                                        // [groups + 1] first entries
  int32_t* ls = lf + a.groups_max + 1;                                    // [entries] slots
  float* lw = reinterpret_cast<float*>(ls + a.T * a.K);                   // [entries] weights
  for (int32_t i = threadIdx.x; i < kDownWaves * a.T * 16; i += blockDim.x) acc[i] = 0.0f;
  for (int32_t i = threadIdx.x; i <= groups; i += blockDim.x) {
    if (i < groups) le[i] = a.expert[i];
    lf[i] = a.first[i];
  }
  for (int32_t i = threadIdx.x; i < a.T * a.K; i += blockDim.x) {  // past the last entry: not used
    ls[i] = a.slot[i];
    lw[i] = a.weight[i];
  }
  __syncthreads();
  f32x4* mine = reinterpret_cast<f32x4*>(acc) + wave * a.T * 4;
  const int64_t rowb = static_cast<int64_t>(a.F) * W::kElt;
  struct Block {
    W w;
    u32x4 h[4], lo[4];
    float s;
    bool both;       // the parts of h in operands of their own
    int32_t group;   // >= groups: none
    int32_t c0;
  } blk[2];
  int32_t group = 0, at = part * kDownWaves + wave;  // the next block to load
  auto load = [&](Block& v) {
    while (at >= a.fb && group < groups) at -= a.fb, ++group;
    v.group = group;
    if (group >= groups) return;
    const int32_t e = uniform(le[group]), first = lf[group], n = lf[group + 1] - first, c0 = at * kBlk;
    v.w.load(a.w2 + (static_cast<int64_t>(e) * a.H + n0 + r) * rowb, c0, g, a.F);
    v.s = kFp8 ? load_f32(a.w2s + (static_cast<int64_t>(e) * a.hb + n0 / kBlk) * a.fb + at) : 1.0f;
    v.c0 = c0;
    v.both = !kFp8 || uniform(n) > 8;
    const int64_t row = static_cast<int64_t>(ls[first + min(v.both ? r : r & 7, n - 1)]) * a.F;
    const char* h0 = v.both || r < 8 ? a.hhi : a.hlo;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v.h[s] = load16(h0 + (row + min(c0 + W::col(s, g), a.F - 8)) * 2);
    }
    if (v.both) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        v.lo[s] = load16(a.hlo + (row + min(c0 + W::col(s, g), a.F - 8)) * 2);
      }
    }
    at += a.parts * kDownWaves;
  };
  f32x4 tot = {0, 0, 0, 0};
  int32_t cur = -1;
  auto finish = [&] {  // the totals of a group's tokens into this wave's sums
    const int32_t first = lf[cur], n = lf[cur + 1] - first;
    if (kFp8 && n <= 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) tot[j] += __shfl_xor(tot[j], 8);  // the parts of h
    }
    if (r < n) {
      f32x4* to = mine + ls[first + r] / a.K * 4 + g;  // an expert's tokens are distinct
      const float c = lw[first + r];
      f32x4 v = *to;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(c, tot[j], v[j]);
      *to = v;
    }
    tot = f32x4{0, 0, 0, 0};
  };
  auto multiply = [&](Block& v) {
    if (v.group >= groups) return;
    if (cur != v.group) {
      if (cur >= 0) finish();
      cur = v.group;
    }
    if (v.c0 + kBlk > a.F) {
      v.w.cut(v.c0, g, a.F);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (v.c0 + W::col(s, g) >= a.F) v.h[s] = v.lo[s] = u32x4{0, 0, 0, 0};
    }
    f32x4 p = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const u32x4 wv = v.w.step(s);
      if (v.both) p = Mat<TBF16>::mul(wv, v.lo[s], p);
      p = Mat<TBF16>::mul(wv, v.h[s], p);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) tot[j] = __builtin_fmaf(v.s, p[j], tot[j]);
  };
  load(blk[0]);
  while (blk[0].group < groups) {
    load(blk[1]);
    multiply(blk[0]);
    load(blk[0]);
    multiply(blk[1]);
  }
  if (cur >= 0) finish();
  __syncthreads();
  float* out = a.partial + static_cast<int64_t>(tile) * a.parts * a.T * 16;
  for (int32_t i = threadIdx.x; i < a.T * 16; i += blockDim.x) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) v += acc[w * a.T * 16 + i];
    if (a.parts == 1) store_elem<T>(a.y + static_cast<int64_t>(i / 16) * a.ys, n0 + i % 16, v);
    else __hip_atomic_store(out + part * a.T * 16 + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.parts == 1) return;
  // The part that arrives last adds them all, in order, whichever it is.  The sums, the count and
  // the reading of the sums are atomics of device scope, which pass the L2 of the XCD by; a wave
  // counts itself only when its sums are there.  (A fence instead writes back the whole L2 of
  // the XCD, for every workgroup: 100 us.)
  __shared__ bool last;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(a.arrived + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.parts - 1;
  __syncthreads();
  if (!last) return;
  for (int32_t i = threadIdx.x; i < a.T * 16; i += blockDim.x) {
    float v = 0.0f;
    for (int32_t p0 = 0; p0 < a.parts; p0 += 8) {  // eight loads at a time
      float s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        s[j] = __hip_atomic_load(out + min(p0 + j, a.parts - 1) * a.T * 16 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int j = 0; j < 8; ++j) v += p0 + j < a.parts ? s[j] : 0.0f;
    }
    store_elem<T>(a.y + static_cast<int64_t>(i / 16) * a.ys, n0 + i % 16, v);
  }
}

// ------------------------------------------------------------------ host side

int plan_layer(const moe_layer_desc* d, LayerPlan* p) {
  if (d == nullptr || d->x == nullptr || d->expert_ids == nullptr || d->w13 == nullptr || d->w2 == nullptr || d->y == nullptr)
    return FFNWB_ERR_PARAM_NULLPTR;
  if (d->dtype != FFNWB_DT_FP16 && d->dtype != FFNWB_DT_BF16) return FFNWB_ERR_PARAM_INVALID;
  const bool fp8 = d->weight_dtype == FFNWB_DT_FP8_E4M3;
  if (!fp8 && !(d->weight_dtype == FFNWB_DT_BF16 && d->dtype == FFNWB_DT_BF16)) return FFNWB_ERR_PARAM_INVALID;
  if (fp8 != (d->w13_scale != nullptr) || fp8 != (d->w2_scale != nullptr)) return FFNWB_ERR_PARAM_INVALID;
  if (d->id_dtype != FFNWB_DT_INT32 && d->id_dtype != FFNWB_DT_INT64) return FFNWB_ERR_PARAM_INVALID;
  if (d->expert_scales != nullptr && d->scale_dtype != FFNWB_DT_FP16 && d->scale_dtype != FFNWB_DT_BF16 &&
      d->scale_dtype != FFNWB_DT_FP32)
    return FFNWB_ERR_PARAM_INVALID;
  if (d->num_tokens < 0 || d->num_tokens > kLyMaxTokens || d->slots <= 0 || d->slots > kLyMaxSlots) return FFNWB_ERR_PARAM_INVALID;
  if (d->hidden <= 0 || d->hidden > (1 << 18) || d->hidden % 16 != 0) return FFNWB_ERR_PARAM_INVALID;
  if (d->inter_size <= 0 || d->inter_size > (1 << 17) || d->inter_size % 16 != 0) return FFNWB_ERR_PARAM_INVALID;
  if (d->num_experts < 1 || d->num_experts > kMaxExperts) return FFNWB_ERR_PARAM_INVALID;
  p->T = d->num_tokens, p->K = d->slots, p->H = d->hidden, p->F = d->inter_size, p->E = d->num_experts;
  p->xs = d->x_row_stride ? d->x_row_stride : p->H * 2;
  p->ys = d->y_row_stride ? d->y_row_stride : p->H * 2;
  p->is = d->expert_ids_stride ? d->expert_ids_stride : p->K;
  p->ss = d->expert_scales_stride ? d->expert_scales_stride : p->K;
  p->ms = d->active_mask_stride ? d->active_mask_stride : p->K;
  const int64_t far = int64_t{1} << 40;  // row * stride stays inside 64 bits
  if (p->xs < p->H * 2 || p->xs % 16 != 0 || p->ys < p->H * 2 || p->ys % 2 != 0) return FFNWB_ERR_PARAM_INVALID;
  if (p->is < p->K || p->ss < p->K || p->ms < p->K) return FFNWB_ERR_PARAM_INVALID;
  if (p->xs > far || p->ys > far || p->is > far || p->ss > far || p->ms > far) return FFNWB_ERR_PARAM_INVALID;
  if ((reinterpret_cast<uintptr_t>(d->x) | reinterpret_cast<uintptr_t>(d->w13) | reinterpret_cast<uintptr_t>(d->w2)) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(d->y) % 2 != 0)
    return FFNWB_ERR_PARAM_INVALID;
  const int64_t n = p->T * p->K;
  p->ranks = n < p->E ? n : p->E;
  p->groups = p->ranks + n / 16 < n ? p->ranks + n / 16 : n;
  // one dimension of the grid: fewer than 2^32 threads
  if (p->ranks * (p->F / 16) >= (int64_t{1} << 32) / (kUpMaxWaves * kWave) - 1) return FFNWB_ERR_PARAM_INVALID;
  // Launch 1: four waves to a tile, eight where the tiles are few and H is long; a tile to each
  // wave where H has fewer blocks than four.
  const int64_t hb = (p->H + 127) / 128;
  p->up_tokens = p->T <= 16 ? 16 : 64;
  p->lanes = n <= kWave;
  p->split = hb < 4 ? 1 : hb >= 16 && p->ranks * (p->F / 16) < 1024 ? 8 : 4;
  Carve c;
  if (n > 0) {
    c.take<int32_t>(1);
    c.take<int32_t>(static_cast<size_t>(p->groups));
    c.take<int32_t>(static_cast<size_t>(p->groups) + 1);
    c.take<int32_t>(static_cast<size_t>(n));
    c.take<float>(static_cast<size_t>(n));
    c.take<uint16_t>(static_cast<size_t>(n * p->F));
    c.take<uint16_t>(static_cast<size_t>(n * p->F));
    // Launch 2 has H / 16 column tiles: below 256 their blocks of F are split over several
    // workgroups each, as long as every wave may have two (at most 32 workgroups).  5 tokens with 8 of 23
    // experts, hidden 576, inter 1024, BF16: 51 us by one workgroup a tile, 27 us by the 12 it gets.  One
    // token's 6 experts, hidden 2944, inter 496, whose waves have 3 blocks each: 14.1 us by the one it gets, 15.3 by
    // two.  Over 92 random layers the choice is 3% slower than the best count on average, 19% at most.
    const int64_t tiles = p->H / 16, blocks = p->groups * ((p->F + 127) / 128);
    p->parts = tiles >= 256 ? 1 : 512 / tiles < 32 ? 512 / tiles : 32;
    if (p->parts > blocks / (2 * kDownWaves)) p->parts = blocks / (2 * kDownWaves);
    if (p->parts < 1) p->parts = 1;
    if (p->parts > 1) {
      c.take<int32_t>(static_cast<size_t>(tiles));
      c.take<float>(static_cast<size_t>(tiles * p->parts * p->T * 16));
    }
  }
  p->ws_bytes = c.off;
  return FFNWB_OK;
}

template <class T, bool kFp8, int kTokens, int kSplit>
static bool launch_up(const LayerArgs& a, const LayerPlan& p, hipStream_t s, void* begin) {
  const uint32_t grid = static_cast<uint32_t>(1 + p.ranks * (kSplit == 1 ? (a.ctiles + 3) / 4 : a.ctiles));
  const size_t table = sizeof(TableLds<kTokens * kLyMaxSlots>), totals = size_t{kSplit} * 2 * (kTokens / 16) * kWave * 16;
  const size_t lds = table > totals ? table : totals;
  auto kernel = layer_up_kernel<T, kFp8, kTokens, kSplit>;
  allow_large_lds(reinterpret_cast<const void*>(kernel), lds);
  return launch_bound(kernel, dim3(grid), dim3((kSplit == 1 ? 4 : kSplit) * kWave), lds, s, begin, nullptr, a);
}

template <class T, bool kFp8, int kTokens>
static bool launch_up(const LayerArgs& a, const LayerPlan& p, hipStream_t s, void* begin) {
  return p.split == 1   ? launch_up<T, kFp8, kTokens, 1>(a, p, s, begin)
         : p.split == 4 ? launch_up<T, kFp8, kTokens, 4>(a, p, s, begin)
                        : launch_up<T, kFp8, kTokens, 8>(a, p, s, begin);
}

template <class T, bool kFp8>
static bool launch_t(const LayerArgs& a, const LayerPlan& p, hipStream_t s, void* begin, void* end) {
  if (!(p.up_tokens == 16 ? launch_up<T, kFp8, 16>(a, p, s, begin) : launch_up<T, kFp8, 64>(a, p, s, begin))) return false;
  const size_t lds = (kDownWaves * p.T * 16 + 2 * p.groups + 1 + 2 * p.T * p.K) * 4;
  allow_large_lds(reinterpret_cast<const void*>(layer_down_kernel<T, kFp8>), lds);
  return launch_bound(layer_down_kernel<T, kFp8>, dim3(static_cast<uint32_t>(p.H / 16 * p.parts)), dim3(kDownWaves * kWave), lds, s, nullptr,
                      end, a);
}

int launch_layer(const moe_layer_desc* d, const LayerPlan& p, void* ws, hipStream_t s) {
  if (p.T == 0) return record_event(d->ev_layer_begin, s) && record_event(d->ev_layer_end, s) ? FFNWB_OK : FFNWB_ERR_RUNTIME;
  LayerArgs a{};
  a.T = static_cast<int32_t>(p.T), a.K = static_cast<int32_t>(p.K), a.E = static_cast<int32_t>(p.E);
  a.H = static_cast<int32_t>(p.H), a.F = static_cast<int32_t>(p.F);
  a.hb = (a.H + kBlk - 1) / kBlk, a.fb = (a.F + kBlk - 1) / kBlk, a.nb13 = (2 * a.F + kBlk - 1) / kBlk;
  a.ctiles = a.F / 16;
  a.groups_max = static_cast<int32_t>(p.groups);
  a.id64 = d->id_dtype == FFNWB_DT_INT64;
  a.scale_dtype = d->scale_dtype;
  a.xs = p.xs, a.ys = p.ys, a.is = p.is, a.ss = p.ss, a.ms = p.ms;
  a.x = static_cast<const char*>(d->x), a.ids = d->expert_ids, a.scales = d->expert_scales, a.mask = d->active_mask;
  a.w13 = static_cast<const char*>(d->w13), a.w13s = d->w13_scale;
  a.w2 = static_cast<const char*>(d->w2), a.w2s = d->w2_scale;
  a.y = static_cast<char*>(d->y);
  const size_t n = static_cast<size_t>(p.T * p.K);
  Carve c;
  c.base = static_cast<char*>(ws);
  a.groups = c.take<int32_t>(1);
  a.expert = c.take<int32_t>(static_cast<size_t>(p.groups));
  a.first = c.take<int32_t>(static_cast<size_t>(p.groups) + 1);
  a.slot = c.take<int32_t>(n);
  a.weight = c.take<float>(n);
  a.hhi = reinterpret_cast<char*>(c.take<uint16_t>(n * p.F));
  a.hlo = reinterpret_cast<char*>(c.take<uint16_t>(n * p.F));
  a.parts = static_cast<int32_t>(p.parts);
  if (p.parts > 1) {
    a.arrived = c.take<int32_t>(static_cast<size_t>(p.H / 16));
    a.partial = c.take<float>(static_cast<size_t>(p.H * p.parts * p.T));
  }
  const bool fp8 = d->weight_dtype == FFNWB_DT_FP8_E4M3;
  void *b = d->ev_layer_begin, *e = d->ev_layer_end;
  const bool ok = d->dtype == FFNWB_DT_FP16 ? launch_t<TF16, true>(a, p, s, b, e)
                  : fp8                     ? launch_t<TBF16, true>(a, p, s, b, e)
                                            : launch_t<TBF16, false>(a, p, s, b, e);
  return ok ? FFNWB_OK : FFNWB_ERR_RUNTIME;
}

}  // namespace ffnwb
