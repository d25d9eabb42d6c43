// Internal declarations of the linear layers whose rows choose their own
// weights (mixtures of experts, adapters).  Not part of the public ABI.
#pragma once

#include "qlin_internal.hpp"

namespace qlin {

constexpr int kMostGroups = 1024;   // experts or adapters of one call

// A plan: the rows of a batch in the order of the weights they meet.  order
// [rows]: the row at each place; offsets [groups + 1]: where each group's run
// begins.  The rows of no group come last, from offsets[groups] on.
struct RowPlan {
  const int32_t* order;
  const int32_t* offsets;
  int groups;
  int rows;
};

// Sums and largest values over a wave's lanes by DPP moves (8 cycles a step,
// where a shuffle through LDS takes over 100): within rows of 16 lanes, then
// from row to row.  Lanes without a source take 0.
template <int kCtrl, int kRows>
__device__ __forceinline__ int dpp0(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kCtrl, kRows, 0xF, false);
}

// Inclusive prefix sum.
__device__ __forceinline__ int wave_prefix(int v) {
  v += dpp0<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v += dpp0<0x112, 0xF>(v);
  v += dpp0<0x114, 0xF>(v);
  v += dpp0<0x118, 0xF>(v);
  v += dpp0<0x142, 0xA>(v);   // lane 15 of a row to the next, rows 1 and 3
  v += dpp0<0x143, 0xC>(v);   // lane 31 to rows 2 and 3
  return v;
}

__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }

// The largest of unsigned values, the same for all lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, uint32_t(dpp0<0x111, 0xF>(int(v))));
  v = max(v, uint32_t(dpp0<0x112, 0xF>(int(v))));
  v = max(v, uint32_t(dpp0<0x114, 0xF>(int(v))));
  v = max(v, uint32_t(dpp0<0x118, 0xF>(int(v))));
  v = max(v, uint32_t(dpp0<0x142, 0xA>(int(v))));
  v = max(v, uint32_t(dpp0<0x143, 0xC>(int(v))));
  return uint32_t(last_lane(int(v)));
}

// A run of at most `tall` places of one group.
struct RowTile {
  int group;   // -1: no such tile; `groups`: rows without a group
  int first;   // its first place
  int count;   // 1 .. tall
};

// The places of a group (group == groups: those of no group).  Offsets are held
// to 0 .. rows, so that no plan makes a kernel leave its buffers.
struct GroupRun {
  int first, end;
};
__device__ __forceinline__ GroupRun run_of(const RowPlan& p, int g) {
  if (g > p.groups) return GroupRun{0, 0};
  const uint32_t most = uint32_t(p.rows);
  const int a = int(min(uint32_t(p.offsets[g]), most));
  const int b = g < p.groups ? int(min(uint32_t(p.offsets[g + 1]), most)) : p.rows;
  return GroupRun{a, max(a, b)};
}

// A plan's runs as a wave searches them: those of the first 192 groups are read
// once, at the same time (a read takes a microsecond where the plan was written
// by another XCD's blocks).
struct PlanRuns {
  static constexpr int kHeld = 3;
  const RowPlan& p;
  GroupRun held[kHeld];

  __device__ __forceinline__ explicit PlanRuns(const RowPlan& plan) : p(plan) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = run_of(p, i * 64 + (threadIdx.x & 63));
  }

  // f(first group, run of this lane's group) for each 64 groups, until it says true
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i * 64 <= p.groups && f(i * 64, held[i])) return;
    for (int g0 = kHeld * 64; g0 <= p.groups; g0 += 64)
      if (f(g0, run_of(p, g0 + (threadIdx.x & 63)))) return;
  }
};

// The tile of a number among those that tiles(group, run) counts for each group,
// in the order of the groups; a group's are its first ones, or its last one
// (kLast).  The search is a wave's: each lane takes a group of 64, a prefix sum
// over the lanes gives the tiles before it.  Not found: the number less what
// there is.
template <bool kLast, typename F>
__device__ __forceinline__ bool search_tiles(const PlanRuns& runs, int tall, int& number, RowTile& tile, F tiles) {
  bool found = false;
  runs.each([&](int g0, GroupRun run) {
    const int here = tiles(g0 + int(threadIdx.x & 63), run), sum = wave_prefix(here);
    const uint64_t past = __ballot(sum > number);
    if (!past) {
      number -= last_lane(sum);
      return false;
    }
    const int at = __builtin_ctzll(past);
    auto of = [&](int v) { return __builtin_amdgcn_readlane(v, at); };
    const int in_group = kLast ? (of(run.end) - of(run.first) - 1) / tall : number - of(sum) + of(here);
    const int first = of(run.first) + in_group * tall;
    tile = RowTile{g0 + at, first, min(of(run.end) - first, tall)};
    found = true;
    return true;
  });
  return found;
}

// All tiles: those of group 0, of group 1, ..., then those of the rows without a
// group.
__device__ __forceinline__ RowTile find_tile(const RowPlan& p, int tall, int number) {
  RowTile tile{-1, 0, 0};
  search_tiles<false>(PlanRuns(p), tall, number, tile,
                      [&](int, GroupRun run) { return (run.end - run.first + tall - 1) / tall; });
  return tile;
}

// How many tiles that counts.
template <typename F>
__device__ __forceinline__ int count_tiles(const PlanRuns& runs, F tiles) {
  int sum = 0;
  runs.each([&](int g0, GroupRun run) {
    sum += tiles(g0 + int(threadIdx.x & 63), run);
    return false;
  });
  return last_lane(wave_prefix(sum));
}

// The most tiles that a plan of so many rows and groups can have.
inline int64_t most_tiles(int64_t rows, int64_t groups, int64_t tall) {
  return rows / tall + (rows < groups + 1 ? rows : groups + 1);
}

// ---------------------------------------------------------------------------
// Launchers: arguments are checked by the caller.
// ---------------------------------------------------------------------------
size_t group_rows_ws_bytes(int64_t rows, int64_t top_k, int64_t groups);
hipError_t launch_group_rows(const int32_t* ids, int64_t rows, int groups, int32_t* order,
                             int32_t* where, int32_t* offsets, int32_t* ws, hipStream_t s);
hipError_t launch_moe_route(const void* logits, int dtype, int64_t tokens, int experts,
                            int64_t stride, int top_k, bool renormalize, int32_t* ids,
                            float* weights, int32_t* order, int32_t* where, int32_t* offsets,
                            int32_t* ws, hipStream_t s);
hipError_t launch_moe_combine(const void* rows, int x_dtype, const RowPlan& p, const int32_t* where,
                              const float* weights, int64_t tokens, int top_k, int64_t n, void* out,
                              int out_dtype, hipStream_t s);

struct MoeGemm {
  RowPlan plan;
  int top_k;              // with gather: the place's row of x is order / top_k
  bool gather, silu_mul;
  const uint8_t* experts; // blobs, `blob_stride` bytes apart
  int64_t blob_stride;
  int n, k;
  void* y;
  int y_dtype;
};
// W4A4: places of a tile, and the tiles of 256 weight rows that a launch has blocks
// for.  Tiles of 64 places up to 256 rows of an expert on average: 1362 rows over 8
// experts (gate and up of 4096 x 4096) 62 us, in tiles of 256 103; 2610 over 16
// (3840 x 1920) 53 and 77; 28000 over 128 (1536 x 2048) 244 and 252; but 9800
// over 32 (5120 x 1280) 185 and 179.
inline int w4a4_tall(int64_t rows, int64_t groups) { return rows <= 256 * groups ? 64 : 256; }
inline int64_t w4a4_tiles(int64_t rows, int64_t groups, int64_t n) {
  return most_tiles(rows, groups, w4a4_tall(rows, groups)) * ((n + 255) / 256);
}
hipError_t launch_moe_gemm_w4a16(const MoeGemm& g, const void* x, hipStream_t s);
hipError_t launch_moe_gemm_w4a4(const MoeGemm& g, const uint8_t* codes, const uint8_t* scales,
                                const float* a_ts, hipStream_t s);

struct LoraArgs {
  RowPlan plan;
  const void *x, *a, *b, *y;
  const float* scale;
  void* out;
  int64_t x_stride, y_stride, out_stride;
  int rank, n, k, y_dtype;
  float* part;            // [parts][rows][rank]
};
size_t lora_ws_bytes(int64_t rows, int64_t groups, int rank, int64_t k);
hipError_t launch_lora_add(const LoraArgs& a, hipStream_t s);

}  // namespace qlin
