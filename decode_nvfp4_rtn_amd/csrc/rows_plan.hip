// Which rows meet which weights: the choice of a token's experts, the plan
// that puts rows in the order of their weights, and the sum over a token's
// experts.
//
// Plan: a stable counting sort.  A block takes a run of rows and counts its
// groups; a second launch adds up the counts of the blocks before its own
// (every block for itself: at most 256 blocks' counts, read from L2), and
// writes each row's place.  Within a wave a row's rank among the rows of its
// group comes from ballots over the bits of the group's number.  One block's
// worth of rows takes one launch.  Whole numbers only, counted by integer
// atomics in LDS whose order does not show: the plan is the same every time.
//
// 16384 tokens, 8 of 256 experts, binary32 scores: the choice with its counts 16.4
// us (18.9 MB; the chain of choices in a wave bounds it: of their cycles its waves
// issue in 28 %, want to in 18 % and wait for a result in the rest), the places 8.3.
// 32 tokens, 8 of 128: 8.3, one block's chain.  Plans of given choices: 64 rows of 32
// groups 3.9 us, 8190 of 8 8.6, 300000 of 1024 26 (3.6 MB).  The sum of 8 rows of 4096 for 8192
// tokens: 118 us, 604 MB at 5.1 TB/s.
#include "moe.hpp"

#include <cmath>

namespace qlin {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int kMostBlocks = 256;

constexpr int kHeld = 1024;   // rows of a block whose choices stay in LDS

struct PlanSmem {
  int base[kMostGroups + 1];             // next place of each group
  int32_t held[kHeld];                   // the block's choices, where they fit
  __attribute__((aligned(4))) uint8_t wave_count[WAVES][kMostGroups + 1];
  int carry[WAVES];
};

// Counts of a block: rows of groups + 1 numbers, padded to whole 16 bytes.
__host__ __device__ constexpr int count_stride(int groups) { return (groups + 4) / 4 * 4; }

__device__ __forceinline__ int group_of(int32_t id, int groups) {
  return uint32_t(id) < uint32_t(groups) ? id : groups;
}

// base[g] = first place of group g (an exclusive sum of count over the
// groups); every thread of the block takes part.
__device__ __forceinline__ void scan_groups(PlanSmem& sm, int groups) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int before = 0;
  for (int g0 = 0; g0 <= groups; g0 += THREADS) {
    const int g = g0 + threadIdx.x;
    const int own = g <= groups ? sm.base[g] : 0;
    const int sum = wave_prefix(own);
    if (lane == 63) sm.carry[wave] = sum;
    __syncthreads();
    int at = before;
    for (int w = 0; w < wave; ++w) at += sm.carry[w];
    for (int w = 0; w < WAVES; ++w) before += sm.carry[w];
    if (g <= groups) sm.base[g] = at + sum - own;
    __syncthreads();
  }
}

// The choices of rows [begin, end) into LDS, where they fit (a barrier follows).
__device__ __forceinline__ void hold_rows(PlanSmem& sm, const int32_t* __restrict__ ids, int begin, int end) {
  if (end - begin <= kHeld)
    for (int r = begin + threadIdx.x; r < end; r += THREADS) sm.held[r - begin] = ids[r];
}

// Places of the rows [begin, end) from base on, which moves along.
__device__ __forceinline__ void place_rows(PlanSmem& sm, const int32_t* __restrict__ ids, int begin,
                                           int end, int groups, int32_t* __restrict__ order,
                                           int32_t* __restrict__ where) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bits = 32 - __clz(groups);   // groups itself is a number too
  const bool held = end - begin <= kHeld;
  for (int r0 = begin; r0 < end; r0 += THREADS) {
    static_assert(sizeof(sm.wave_count) % 4 == 0, "cleared by words");
    for (int i = threadIdx.x; i < int(sizeof(sm.wave_count) / 4); i += THREADS)
      reinterpret_cast<uint32_t*>(sm.wave_count)[i] = 0;
    __syncthreads();
    const int row = r0 + threadIdx.x;
    const bool live = row < end;
    const int g = live ? group_of(held ? sm.held[row - begin] : ids[row], groups) : 0;
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((g >> b) & 1);
      same &= (g >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (live && rank == 0) sm.wave_count[wave][g] = uint8_t(__popcll(same));
    __syncthreads();
    if (live) {
      int at = sm.base[g] + rank;
      for (int w = 0; w < wave; ++w) at += sm.wave_count[w][g];
      order[at] = row;
      where[row] = at;
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= groups; i += THREADS) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) sum += sm.wave_count[w][i];
      sm.base[i] += sum;
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void count_rows(PlanSmem& sm, const int32_t* __restrict__ ids, int begin,
                                           int end, int groups) {
  for (int i = threadIdx.x; i <= groups; i += THREADS) sm.base[i] = 0;
  __syncthreads();
  const bool held = end - begin <= kHeld;
  for (int r = begin + threadIdx.x; r < end; r += THREADS)
    atomicAdd(&sm.base[group_of(held ? sm.held[r - begin] : ids[r], groups)], 1);
  __syncthreads();
}

__device__ __forceinline__ void write_offsets(const PlanSmem& sm, int groups,
                                              int32_t* __restrict__ offsets) {
  for (int i = threadIdx.x; i <= groups; i += THREADS) offsets[i] = sm.base[i];
}

// What a block does once its rows' groups are known: the whole plan where it
// is the only block, or its counts.
__device__ __forceinline__ void finish_block(PlanSmem& sm, const int32_t* ids, int begin, int end,
                                             int groups, int32_t* order, int32_t* where,
                                             int32_t* offsets, int32_t* counts) {
  count_rows(sm, ids, begin, end, groups);
  if (gridDim.x > 1) {
    for (int i = threadIdx.x; i <= groups; i += THREADS)
      counts[blockIdx.x * count_stride(groups) + i] = sm.base[i];
    return;
  }
  scan_groups(sm, groups);
  write_offsets(sm, groups, offsets);
  __syncthreads();
  place_rows(sm, ids, begin, end, groups, order, where);
}

__global__ __launch_bounds__(THREADS) void group_count_kernel(const int32_t* __restrict__ ids, int rows,
                                                              int per_block, int groups,
                                                              int32_t* __restrict__ order,
                                                              int32_t* __restrict__ where,
                                                              int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ counts) {
  __shared__ PlanSmem sm;
  const int64_t begin = int64_t(blockIdx.x) * per_block, end = min(begin + per_block, int64_t(rows));
  hold_rows(sm, ids, int(begin), int(end));
  finish_block(sm, ids, int(begin), int(end), groups, order, where, offsets, counts);
}

__global__ __launch_bounds__(THREADS) void group_place_kernel(const int32_t* __restrict__ ids, int rows,
                                                              int per_block, int groups, int blocks,
                                                              const int32_t* __restrict__ counts,
                                                              int32_t* __restrict__ order,
                                                              int32_t* __restrict__ where,
                                                              int32_t* __restrict__ offsets) {
  __shared__ PlanSmem sm;
  __shared__ int before[kMostGroups + 1];   // of the blocks before this one
  const int own = blockIdx.x;
  for (int i = threadIdx.x; i <= groups; i += THREADS) sm.base[i] = before[i] = 0;
  __syncthreads();
  const int64_t begin = int64_t(own) * per_block, end = min(begin + per_block, int64_t(rows));
  hold_rows(sm, ids, int(begin), int(end));
  // a thread to four groups and a share of the blocks
  const int stride = count_stride(groups), quads = stride / 4, shares = THREADS / quads;
  const int g = threadIdx.x % quads * 4, share = threadIdx.x / quads;
  if (share < shares) {
    int all[4] = {0, 0, 0, 0}, mine[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int b = share; b < blocks; b += shares) {
      const int4 c = *reinterpret_cast<const int4*>(counts + b * stride + g);
      const int v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        all[i] += v[i];
        mine[i] += b < own ? v[i] : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (g + i <= groups) {   // past it: padding, never written
        atomicAdd(&sm.base[g + i], all[i]);
        atomicAdd(&before[g + i], mine[i]);
      }
  }
  __syncthreads();
  scan_groups(sm, groups);
  if (own == 0) write_offsets(sm, groups, offsets);
  __syncthreads();
  for (int i = threadIdx.x; i <= groups; i += THREADS) sm.base[i] += before[i];
  __syncthreads();
  place_rows(sm, ids, int(begin), int(end), groups, order, where);
}

// A number that orders binary32 values as unsigned integers do; +0 and -0 are
// one value, -infinity and NaN (an expert that may not be chosen) are 0.
__device__ __forceinline__ uint32_t rank_of(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t r) {
  return __uint_as_float(r & 0x80000000u ? r & 0x7FFFFFFFu : ~r);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// Two tokens at a time to a wave: lane l holds logits l, l + 64, ...; top_k times
// the largest is found (of equals the lowest expert) and taken out.  A choice is
// a chain of some twenty dependent steps; two tokens' chains fill each other's
// waits, and the next two tokens' logits are under way.  The softmax's terms
// are exp(l - largest); those of the largest are 1 whatever it is, so that
// infinities share the weight.
template <int PER, bool kBF16>
__global__ __launch_bounds__(THREADS) void route_kernel(
    const void* __restrict__ logits, int64_t stride, int tokens, int tokens_per_block, int experts,
    int top_k, bool renormalize, int32_t* __restrict__ ids, float* __restrict__ weights,
    int32_t* __restrict__ order, int32_t* __restrict__ where, int32_t* __restrict__ offsets,
    int32_t* __restrict__ counts) {
  constexpr int TOK = 2;
  __shared__ PlanSmem sm;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = int64_t(blockIdx.x) * tokens_per_block;
  const int64_t t1 = min(t0 + tokens_per_block, int64_t(tokens));
  float raw[TOK][PER];
  auto load = [&](int64_t t) {   // past the end: the last token again, not stored
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      const int64_t at = min(t + u * WAVES, t1 - 1) * stride;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = min(i * 64 + lane, experts - 1);
        if (kBF16)
          raw[u][i] = __uint_as_float(uint32_t(static_cast<const uint16_t*>(logits)[at + e]) << 16);
        else
          raw[u][i] = static_cast<const float*>(logits)[at + e];
      }
    }
  };
  if (t0 + wave < t1) load(t0 + wave);
  for (int64_t t = t0 + wave; t < t1; t += TOK * WAVES) {
    uint32_t rank[TOK][PER], top[TOK];
    float total[TOK];
#pragma unroll
    for (int u = 0; u < TOK; ++u)
#pragma unroll
      for (int i = 0; i < PER; ++i) rank[u][i] = i * 64 + lane < experts ? rank_of(raw[u][i]) : 0;
    load(t + TOK * WAVES);
    auto most = [&](int u) {
      uint32_t v = rank[u][0];
#pragma unroll
      for (int i = 1; i < PER; ++i) v = max(v, rank[u][i]);
      return wave_max(v);
    };
    auto term = [&](int u, uint32_t r) {
      return r == top[u] ? 1.0f : r ? expf(value_of(r) - value_of(top[u])) : 0.0f;
    };
    uint32_t chosen[TOK];   // lane j: the j-th choice
    int expert[TOK];
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      top[u] = most(u);
      chosen[u] = 0;
      expert[u] = -1;
      total[u] = 0.0f;
    }
    if (!renormalize) {
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
#pragma unroll
        for (int i = 0; i < PER; ++i) total[u] += top[u] ? term(u, rank[u][i]) : 0.0f;
        total[u] = wave_sum(total[u]);
      }
    }
    for (int j = 0; j < top_k; ++j) {
      uint32_t m[TOK];
      int e[TOK];
#pragma unroll
      for (int u = 0; u < TOK; ++u) m[u] = j == 0 ? top[u] : most(u);
      // the lowest expert of those with the largest rank: of the first register
      // that holds it the first lane
#pragma unroll
      for (int u = 0; u < TOK; ++u) {
        e[u] = -1;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
          const uint64_t with = __ballot(rank[u][i] == m[u]);
          e[u] = with ? i * 64 + __builtin_ctzll(with) : e[u];
        }
        if (m[u] == 0) e[u] = -1;   // none is left
#pragma unroll
        for (int i = 0; i < PER; ++i) rank[u][i] = i * 64 + lane == e[u] ? 0 : rank[u][i];
        if (lane == j) chosen[u] = m[u], expert[u] = e[u];
      }
    }
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      const int64_t at = t + u * WAVES;
      const float w = chosen[u] ? term(u, chosen[u]) : 0.0f;
      if (renormalize) total[u] = wave_sum(lane < top_k ? w : 0.0f);
      if (lane < top_k && at < t1) {
        ids[at * top_k + lane] = expert[u];
        const int in_block = int(at - t0) * top_k + lane;
        if (in_block < kHeld) sm.held[in_block] = expert[u];
        weights[at * top_k + lane] = chosen[u] ? w / total[u] : 0.0f;
      }
    }
  }
  __syncthreads();   // the block's choices, read back below
  finish_block(sm, ids, int(t0 * top_k), int(t1 * top_k), experts, order, where, offsets, counts);
}

// Rows of a block, whole tokens: one block up to kHeld rows, else blocks of
// about half as many (a CU each for a long prompt), at most kMostBlocks.
int64_t block_rows(int64_t rows, int64_t top_k) {
  const int64_t tokens = rows / top_k;
  const int64_t least = (rows <= kHeld ? kHeld : kHeld / 2) / top_k;
  const int64_t spread = (tokens + kMostBlocks - 1) / kMostBlocks;
  return (spread > least ? spread : least) * top_k;
}

template <bool kBF16>
hipError_t launch_route(const void* logits, int64_t tokens, int experts, int64_t stride, int top_k,
                        bool renormalize, int32_t* ids, float* weights, int32_t* order,
                        int32_t* where, int32_t* offsets, int32_t* ws, hipStream_t s) {
  const int64_t per = block_rows(tokens * top_k, top_k) / top_k;
  const int blocks = tokens ? int((tokens + per - 1) / per) : 1;   // no tokens: offsets of zero
  auto run = [&](auto kern) {
    kern<<<blocks, THREADS, 0, s>>>(logits, stride, int(tokens), int(per), experts, top_k, renormalize,
                                    ids, weights, order, where, offsets, ws);
    return hipGetLastError();
  };
  hipError_t e;
  if (experts <= 64) e = run(route_kernel<1, kBF16>);
  else if (experts <= 128) e = run(route_kernel<2, kBF16>);
  else if (experts <= 256) e = run(route_kernel<4, kBF16>);
  else if (experts <= 512) e = run(route_kernel<8, kBF16>);
  else e = run(route_kernel<16, kBF16>);
  if (e != hipSuccess || blocks == 1) return e;
  group_place_kernel<<<blocks, THREADS, 0, s>>>(ids, int(tokens * top_k), int(per * top_k), experts,
                                                blocks, ws, order, where, offsets);
  return hipGetLastError();
}

// Each token's weighted sum over its experts' rows, in binary32 and in the
// order of its choices.  A thread takes 8 columns; the rows of four choices
// are under way at once.  A place that is no expert's adds nothing and is not
// read.
template <bool kBF16In, bool kBF16Out>
__global__ __launch_bounds__(256) void combine_kernel(const void* __restrict__ rows,
                                                      const int32_t* __restrict__ where,
                                                      const float* __restrict__ weights,
                                                      const int32_t* __restrict__ offsets, int groups,
                                                      int n_rows, int top_k, int n,
                                                      void* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int col = (blockIdx.y * 256 + threadIdx.x) * 8;
  const int used = min(offsets[groups], n_rows);
  if (col >= n) return;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < top_k; j0 += 4) {
    uint4 v[4][kBF16In ? 1 : 2];
    float w[4];
    bool live[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int slot = min(j0 + j, top_k - 1);
      const int at = where[t * top_k + slot];
      live[j] = j0 + j < top_k && uint32_t(at) < uint32_t(max(used, 0));
      w[j] = weights[t * top_k + slot];
      const int64_t row = live[j] ? at : 0;
      if (live[j]) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(rows) +
                                                        (row * n + col) * (kBF16In ? 2 : 4));
        v[j][0] = p[0];
        if constexpr (!kBF16In) v[j][1] = p[1];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!live[j]) continue;
      float x[8];
      if constexpr (kBF16In) {
        const uint32_t d[4] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(d[i] << 16);
          x[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[4 * i] = __uint_as_float(v[j][i].x);
          x[4 * i + 1] = __uint_as_float(v[j][i].y);
          x[4 * i + 2] = __uint_as_float(v[j][i].z);
          x[4 * i + 3] = __uint_as_float(v[j][i].w);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], x[i], sum[i]);
    }
  }
  uint8_t* o = static_cast<uint8_t*>(out) + (t * n + col) * (kBF16Out ? 2 : 4);
  if constexpr (kBF16Out) {
    *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]),
                                              pack_bf16x2(sum[4], sum[5]), pack_bf16x2(sum[6], sum[7]));
  } else {
    reinterpret_cast<float4*>(o)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    reinterpret_cast<float4*>(o)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
  }
}

}  // namespace

size_t group_rows_ws_bytes(int64_t rows, int64_t top_k, int64_t groups) {
  const int64_t per = block_rows(rows, top_k);
  const int64_t blocks = (rows + per - 1) / per;
  return blocks > 1 ? size_t(blocks) * size_t(count_stride(int(groups))) * sizeof(int32_t) : 0;
}

hipError_t launch_group_rows(const int32_t* ids, int64_t rows, int groups, int32_t* order,
                             int32_t* where, int32_t* offsets, int32_t* ws, hipStream_t s) {
  const int per = int(block_rows(rows, 1));
  const int blocks = rows ? int((rows + per - 1) / per) : 1;   // no rows: offsets of zero
  group_count_kernel<<<blocks, THREADS, 0, s>>>(ids, int(rows), per, groups, order, where, offsets, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1) return e;
  group_place_kernel<<<blocks, THREADS, 0, s>>>(ids, int(rows), per, groups, blocks, ws, order, where,
                                                offsets);
  return hipGetLastError();
}

hipError_t launch_moe_route(const void* logits, int dtype, int64_t tokens, int experts,
                            int64_t stride, int top_k, bool renormalize, int32_t* ids,
                            float* weights, int32_t* order, int32_t* where, int32_t* offsets,
                            int32_t* ws, hipStream_t s) {
  return dtype == 1 ? launch_route<true>(logits, tokens, experts, stride, top_k, renormalize, ids,
                                         weights, order, where, offsets, ws, s)
                    : launch_route<false>(logits, tokens, experts, stride, top_k, renormalize, ids,
                                          weights, order, where, offsets, ws, s);
}

hipError_t launch_moe_combine(const void* rows, int x_dtype, const RowPlan& p, const int32_t* where,
                              const float* weights, int64_t tokens, int top_k, int64_t n, void* out,
                              int out_dtype, hipStream_t s) {
  const dim3 grid(unsigned(tokens), unsigned((n / 8 + 255) / 256));
  auto run = [&](auto kern) {
    kern<<<grid, 256, 0, s>>>(rows, where, weights, p.offsets, p.groups, p.rows, top_k, int(n), out);
    return hipGetLastError();
  };
  if (x_dtype == 1) return out_dtype == 1 ? run(combine_kernel<true, true>) : run(combine_kernel<true, false>);
  return out_dtype == 1 ? run(combine_kernel<false, true>) : run(combine_kernel<false, false>);
}

}  // namespace qlin
