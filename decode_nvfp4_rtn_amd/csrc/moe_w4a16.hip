// Products of rows with their experts' INT4 group-128 weights, bf16
// activations (the decode path of a mixture of experts).
//
//   y[p, :] = x[row(p), :] W_e^T      for the places p of expert e's run
//
// or, with silu_mul, silu(g) * u of the two halves g, u of that product.  A
// decode step meets most of its experts by a few rows each: what it costs is
// reading their weights once.
//
// A block takes up to 16 MT places of one expert (its tile, found on the
// device from the plan's offsets) and walks a part of the expert's 16-row
// weight tiles.  The tile's rows of x lie in LDS as MFMA fragments, written
// once; after that the waves share nothing: each streams weight tiles of its
// own, whose groups are contiguous in memory, two sets of W groups deep, and
// needs no barrier.  Operands are made as in the dense decode kernels: the
// bf16 values 128 + u of the codes u = q + 8, accumulators that begin at -136
// times the rows' sums (kept in LDS, one for each row and group) and the group
// scale in binary32 after each group's four MFMAs.
#include "moe.hpp"
#include "decode_ops.hpp"

namespace qlin {
namespace {

struct Args16 {
  RowPlan plan;
  const uint16_t* x;
  const uint8_t* experts;
  int64_t blob_stride, codes_off, sc_off;
  void* y;
  int top_k, gather, n, k, walkers, chunk;   // chunk: groups of x in LDS at a time
};

// LDS: fragments [chunk][MT][4][64] x 16 bytes, then sums [chunk][MT][16].
constexpr int frag_bytes(int mt) { return mt * 4096; }
constexpr int group_bytes(int mt) { return mt * (4096 + 64); }

// The slot of row r's 16-byte piece c (k 8 c of the group) within a group's
// 256 slots: piece 4 s + q of fragment s belongs to lanes of quarter q, which
// read 16 rows in 16 slots of their own; rows are XORed with the piece so
// that a row's 16 pieces, written together, fall on different banks.
__device__ __forceinline__ int piece_slot(int r, int c) { return c * 16 + (r ^ c); }

// NT weight tiles at a time: with silu_mul a gate tile and its up tile, else
// one tile or two neighbours.
template <int MT, int NT, int W, bool kSilu, bool kBF16Out>
__global__ __launch_bounds__(512, 2) void moe_w4a16_kernel(Args16 A) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int TALL = 16 * MT, WAVES = 8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int walker = blockIdx.x % A.walkers;
  const RowTile tile = find_tile(A.plan, TALL, blockIdx.x / A.walkers);
  if (tile.group < 0) return;
  const int G = A.k / 128, T = A.n / 16;
  const int n_out = kSilu ? A.n / 2 : A.n;
  const int units = kSilu ? T / 2 : (T + NT - 1) / NT;   // of NT weight tiles
  const int q = lane >> 4, r = lane & 15;

  if (tile.group == A.plan.groups) {   // rows without an expert: zeros
    const int64_t bytes = int64_t(n_out) * (kBF16Out ? 2 : 4);
    for (int i = 0; i < tile.count; ++i) {
      uint4* row = reinterpret_cast<uint4*>(static_cast<uint8_t*>(A.y) + (tile.first + i) * bytes);
      for (int64_t j = walker * 512 + threadIdx.x; j < bytes / 16; j += A.walkers * 512)
        row[j] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const uint8_t* blob = A.experts + tile.group * A.blob_stride;
  if (!blob_matches(blob, 1, A.n, A.k)) return;

  float* const sums = reinterpret_cast<float*>(smem + size_t(A.chunk) * frag_bytes(MT));
  // the rows of groups [c0, c1) into LDS: 16 lanes to a row's group
  auto stage = [&](int c0, int c1) {
    const int per_row = c1 - c0;
    const int rows = (tile.count + 3) / 4;
    for (int i = wave; i < rows * per_row; i += WAVES) {
      const int g = i / rows, row = 4 * (i % rows) + q;
      const int place = tile.first + min(row, tile.count - 1);
      int64_t from = place;
      if (A.gather) from = min(uint32_t(A.plan.order[place]), uint32_t(A.plan.rows - 1)) / uint32_t(A.top_k);
      const uint4 v = *reinterpret_cast<const uint4*>(A.x + from * A.k + (c0 + g) * 128 + 8 * r);
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s += __uint_as_float(d[j] << 16) + __uint_as_float(d[j] & 0xFFFF0000u);
#pragma unroll
      for (int m = 8; m; m /= 2) s += __shfl_xor(s, m);
      *reinterpret_cast<uint4*>(smem + g * frag_bytes(MT) + (row >> 4) * 4096 + piece_slot(row & 15, r) * 16) = v;
      if (r == 0) sums[(g * MT + (row >> 4)) * 16 + (row & 15)] = -136.0f * s;
    }
  };
  const uint32_t nib_mask = vconst(0x000F000Fu), bf16_128 = vconst(0x43004300u);
  const uint8_t* codes = blob + A.codes_off;
  const uint8_t* scales = blob + A.sc_off;

  struct Batch {
    uint4 w[W][NT];
    uint2 s[W][NT];
  };
  // first weight tile of unit u's strand j
  auto tile_of = [&](int u, int j) { return kSilu ? u + j * (T / 2) : min(u * NT + j, T - 1); };
  auto load = [&](Batch& B, int u, int g0, int g1) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t t = tile_of(u, j);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int64_t at = t * G + min(g0 + i, g1 - 1);
        B.w[i][j] = load_nt16(codes + at * 1024 + lane * 16);
        B.s[i][j] = *reinterpret_cast<const uint2*>(scales + at * 32 + 8 * q);
      }
    }
  };
  floatx4 tot[NT][MT];
  int off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) off[s] = piece_slot(r, 4 * s + q) * 16;
  auto compute = [&](const Batch& B, int g0, int g1, int c0) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (g0 + i >= g1) break;   // wave-uniform
      const uint8_t* fr = smem + (g0 + i - c0) * frag_bytes(MT);
      floatx4 acc[NT][MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float z = sums[((g0 + i - c0) * MT + m) * 16 + r];
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][m] = floatx4{z, z, z, z};
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8_t f[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          f[m] = as_bf16x8(*reinterpret_cast<const u32x4*>(fr + m * 4096 + off[s]));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t d = s == 0 ? B.w[i][j].x : s == 1 ? B.w[i][j].y : s == 2 ? B.w[i][j].z : B.w[i][j].w;
          const bf16x8_t op = int4_operand(d, nib_mask, bf16_128);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(op, f[m], acc[j][m], 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint2 sv = B.s[i][j];
        const float sc[4] = {__uint_as_float(sv.x << 16), __uint_as_float(sv.x & 0xFFFF0000u),
                             __uint_as_float(sv.y << 16), __uint_as_float(sv.y & 0xFFFF0000u)};
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) tot[j][m][e] = fmaf(sc[e], acc[j][m][e], tot[j][m][e]);
      }
    }
  };
  auto put = [&](int col, int m, floatx4 v) {
    const int place = 16 * m + r;
    if (place >= tile.count) return;
    uint8_t* o = static_cast<uint8_t*>(A.y) +
                 (int64_t(tile.first + place) * n_out + col) * (kBF16Out ? 2 : 4);
    if constexpr (kBF16Out)
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
      *reinterpret_cast<floatx4*>(o) = v;
  };
  auto finish = [&](int u) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (kSilu) {
        floatx4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = tot[0][m][e] / (1.0f + expf(-tot[0][m][e])) * tot[1][m][e];
        put(u * 16 + 4 * q, m, h);
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (u * NT + j < T) put((u * NT + j) * 16 + 4 * q, m, tot[j][m]);
      }
    }
  };

  const int rounds = (units + WAVES * A.walkers - 1) / (WAVES * A.walkers);
  const bool once = A.chunk >= G;
  if (once) {
    stage(0, G);
    __syncthreads();
  }
  for (int rd = 0; rd < rounds; ++rd) {
    const int u = (rd * A.walkers + walker) * WAVES + wave;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[j][m] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < G; c0 += A.chunk) {
      const int c1 = min(c0 + A.chunk, G);
      if (!once) {
        __syncthreads();   // the chunk before is read
        stage(c0, c1);
        __syncthreads();
      }
      if (u >= units) continue;
      Batch P, Q;
      load(P, u, c0, c1);
      for (int g0 = c0; g0 < c1; g0 += 2 * W) {
        load(Q, u, min(g0 + W, c1 - 1), c1);
        __builtin_amdgcn_sched_barrier(0);
        compute(P, g0, c1, c0);
        load(P, u, min(g0 + 2 * W, c1 - 1), c1);
        __builtin_amdgcn_sched_barrier(0);
        compute(Q, g0 + W, c1, c0);
      }
    }
    if (u < units) finish(u);
  }
}

template <int MT, int NT, int W, bool kSilu>
hipError_t launch16(const Args16& a, int y_dtype, int blocks, hipStream_t s) {
  const size_t lds = size_t(a.chunk) * group_bytes(MT);
  static std::atomic<int> done[2][64];
  auto run = [&](auto kern, std::atomic<int>* flag) {
    const hipError_t e = lds_limit_once(flag, reinterpret_cast<const void*>(kern), 160 * 1024);
    if (e != hipSuccess) return e;
    kern<<<blocks, 512, lds, s>>>(a);
    return hipGetLastError();
  };
  return y_dtype == 1 ? run(moe_w4a16_kernel<MT, NT, W, kSilu, true>, done[1])
                      : run(moe_w4a16_kernel<MT, NT, W, kSilu, false>, done[0]);
}

}  // namespace

hipError_t launch_moe_gemm_w4a16(const MoeGemm& g, const void* x, hipStream_t s) {
  const BlobLayout L = blob_layout(1, g.n, g.k);
  // the height of a tile: the rows that an expert has on average
  const int64_t mean = g.plan.rows / g.plan.groups;
  const int mt = mean > 32 ? 4 : mean > 12 ? 2 : 1;
  const int G = g.k / 128;
  Args16 a{};
  a.plan = g.plan;
  a.x = static_cast<const uint16_t*>(x);
  a.experts = g.experts;
  a.blob_stride = g.blob_stride;
  a.codes_off = int64_t(L.codes_off);
  a.sc_off = int64_t(L.aux_off);
  a.y = g.y;
  a.top_k = g.top_k;
  a.gather = g.gather;
  a.n = g.n;
  a.k = g.k;
  const int most = 160 * 1024 / group_bytes(mt);
  a.chunk = G < most ? G : most;
  const int64_t tiles = most_tiles(g.plan.rows, g.plan.groups, 16 * mt);
  const int cus = device_cu_count();
  const int64_t units = (g.n / 16 + 1) / 2;
  int64_t walkers = (2 * (cus > 0 ? cus : 256) + tiles - 1) / tiles;
  if (walkers > (units + 7) / 8) walkers = (units + 7) / 8;
  a.walkers = int(walkers);
  const int blocks = int(tiles * walkers);
  if (g.silu_mul) {
    if (mt == 1) return launch16<1, 2, 4, true>(a, g.y_dtype, blocks, s);
    if (mt == 2) return launch16<2, 2, 4, true>(a, g.y_dtype, blocks, s);
    return launch16<4, 2, 4, true>(a, g.y_dtype, blocks, s);
  }
  if (mt == 1) return launch16<1, 2, 4, false>(a, g.y_dtype, blocks, s);
  if (mt == 2) return launch16<2, 2, 4, false>(a, g.y_dtype, blocks, s);
  return launch16<4, 2, 4, false>(a, g.y_dtype, blocks, s);
}

}  // namespace qlin
