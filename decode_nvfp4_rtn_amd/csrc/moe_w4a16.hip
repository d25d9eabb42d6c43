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
// device from the plan's offsets) and a part of the expert's 16-row weight
// tiles.  The tile's rows of x lie in LDS as MFMA fragments, written once;
// after that the waves share nothing: each streams weight tiles of its own,
// two at a time and two sets of W groups deep, over the ends of tiles, and
// needs no barrier.  The first set is under way before x is.  Operands are the
// bf16 values 16 + u of the codes u = q + 8 (a code in the upper bits of the
// mantissa), accumulators begin at -24 times the rows' sums (kept in LDS, one
// for each row and group) and the group scale is applied in binary32 after each
// group's four MFMAs.  With 128 + u, one shift less for eight codes, the sums
// were five times as far off: 3e-6 of a result.
//
// Where there are few tiles and places (a single sequence's step) KS waves
// share a pair of weight tiles, a part of k each, and add up in LDS in a fixed
// order.
//
// 48 tokens that choose 8 of 128 experts of 2048 x 768: 19.7 us, 94.6 MB at 4.8
// TB/s, on weights that the Infinity Cache may hold; 23.9 us, 4.0 TB/s, on weights
// that it does not.  One token and 8 experts of 2048 x 4096: 10.2 us (11.4), 34.6 MB;
// a launch's start and one wave's chain are half of it.  509 tokens, 4 of 60 experts of
// 2816 x 2048 (34 rows each): 55 us, 186 MB at 3.4 TB/s; experts of more than 32
// rows have a second tile on another XCD, whose weights come past its L2 again
// (284 MB in all, 5.1 TB/s).
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

constexpr int NT = 2;
// Waves of a block: 16 where its rows fill the LDS of a CU.
constexpr int waves_of(int mt) { return mt == 1 ? 8 : 16; }
// LDS: fragments [chunk][MT][4 pieces][16 XR] x 16 bytes (XR rows to an
// m-tile: 16, or 4 where a tile holds at most 4 places), then sums
// [chunk][MT][XR], then (KS > 1) the waves' accumulators.
constexpr int frag_bytes(int mt, int xr) { return mt * 256 * xr; }
constexpr int group_bytes(int mt, int xr) { return mt * (256 * xr + 4 * xr); }
constexpr int red_bytes(int mt, int ks) { return ks > 1 ? waves_of(mt) * NT * mt * 1024 : 0; }

// The slot of row r's 16-byte piece c (k 8 c of the group) within a group's
// slots: piece 4 s + q of fragment s belongs to lanes of quarter q, which read
// XR rows in XR slots of their own; rows are XORed with the piece so that a
// row's pieces, written together, fall on different banks.
template <int XR>
__device__ __forceinline__ int piece_slot(int r, int c) { return c * XR + (r ^ (c & (XR - 1))); }

// dword of 8 nibbles (pairs at bits (4 j, 16 + 4 j)) -> bf16 (16 + u) x 8
__device__ __forceinline__ bf16x8_t operand16(uint32_t w, uint32_t mask, uint32_t bias) {
  u32x4 v;
  v[0] = ((w << 3) & mask) | bias;
  v[1] = ((w >> 1) & mask) | bias;
  v[2] = ((w >> 5) & mask) | bias;
  v[3] = ((w >> 9) & mask) | bias;
  return as_bf16x8(v);
}

// v of the lane N places on in the same row of 16 lanes
template <int N>
__device__ __forceinline__ float row_rotated(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xF, 0xF, false));
}

template <int MT, int XR, int KS, int W, bool kSilu, bool kBF16Out>
__global__ __launch_bounds__(waves_of(MT) * 64, 4) void moe_w4a16_kernel(Args16 A) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  static_assert(XR == 16 || MT == 1, "tiles of 4 places are one m-tile");
  constexpr int WAVES = waves_of(MT), TALL = MT == 1 ? XR : 16 * MT, FB = frag_bytes(MT, XR);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int walker = blockIdx.x % A.walkers;
  const RowTile tile = find_tile(A.plan, TALL, blockIdx.x / A.walkers);
  if (tile.group < 0) return;
  const int G = A.k / 128, T = A.n / 16;
  const int n_out = kSilu ? A.n / 2 : A.n;
  const int units = kSilu ? T / 2 : (T + 1) / 2;   // of two weight tiles
  const int q = lane >> 4, r = lane & 15;

  if (tile.group == A.plan.groups) {   // rows without an expert: zeros
    const int64_t bytes = int64_t(n_out) * (kBF16Out ? 2 : 4);
    for (int i = 0; i < tile.count; ++i) {
      uint4* row = reinterpret_cast<uint4*>(static_cast<uint8_t*>(A.y) + (tile.first + i) * bytes);
      for (int64_t j = walker * WAVES * 64 + threadIdx.x; j < bytes / 16; j += A.walkers * WAVES * 64)
        row[j] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const uint8_t* blob = A.experts + tile.group * A.blob_stride;
  const uint8_t* codes = blob + A.codes_off;
  const uint8_t* scales = blob + A.sc_off;

  // units of this wave: u0, u0 + step, ...; one at most where x comes in pieces, as
  // where waves share k
  const int u0 = KS > 1 ? walker * (WAVES / KS) + wave / KS : walker * WAVES + wave;
  const int step = A.walkers * WAVES;
  const int mine = u0 < units ? KS > 1 ? 1 : (units - u0 + step - 1) / step : 0;

  struct Batch {
    uint4 w[W][NT];
    uint2 s[W][NT];
  };
  // strand j of unit u: with silu_mul a gate tile and its up tile, else two
  // neighbours
  auto load = [&](Batch& B, int u, int g0, int g1) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int t = kSilu ? u + j * (T / 2) : min(u * NT + j, T - 1);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int64_t at = int64_t(t) * G + min(g0 + i, g1 - 1);
        B.w[i][j] = load_nt16(codes + at * 1024 + lane * 16);
        B.s[i][j] = *reinterpret_cast<const uint2*>(scales + at * 32 + 8 * q);
      }
    }
  };

  float* const sums = reinterpret_cast<float*>(smem + size_t(A.chunk) * FB);
  // the rows of groups [c0, c1) into LDS: 16 lanes to a row's group, a wave to
  // four rows and a share of the groups, four loads under way
  const int quads = (tile.count + 3) / 4, shares = WAVES / quads;
  const int row = 4 * (wave % quads) + q, share = wave / quads;
  const uint16_t* x_row;
  {
    const int place = tile.first + min(row, tile.count - 1);
    int64_t from = place;
    if (A.gather) from = min(uint32_t(A.plan.order[place]), uint32_t(A.plan.rows - 1)) / uint32_t(A.top_k);
    x_row = A.x + from * A.k + 8 * r;
  }
  auto stage = [&](int c0, int c1) {
    if (share >= shares) return;
    const int mt = XR == 16 ? row >> 4 : 0, rr = XR == 16 ? row & 15 : row;
    uint8_t* const to = smem + mt * (256 * XR) + piece_slot<XR>(rr, r) * 16;
    for (int g0 = c0 + share; g0 < c1; g0 += 4 * shares) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const uint4*>(x_row + min(g0 + i * shares, c1 - 1) * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = g0 + i * shares - c0;
        if (g >= c1 - c0) break;   // wave-uniform
        const uint32_t d[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s += __uint_as_float(d[j] << 16) + __uint_as_float(d[j] & 0xFFFF0000u);
        // over the row's 16 lanes
        s += row_rotated<8>(s);
        s += row_rotated<4>(s);
        s += row_rotated<2>(s);
        s += row_rotated<1>(s);
        *reinterpret_cast<uint4*>(to + g * FB) = v[i];
        if (r == 0) sums[(g * MT + mt) * XR + rr] = -24.0f * s;
      }
    }
  };
  const uint32_t nib_mask = vconst(0x00780078u), bf16_16 = vconst(0x41804180u);
  const int rl = XR == 16 ? r : min(r, XR - 1);   // lanes past a tile of 4 read its last row
  int off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) off[s] = piece_slot<XR>(rl, 4 * s + q) * 16;

  floatx4 tot[NT][MT];
  auto clear = [&]() {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) tot[j][m] = floatx4{0.f, 0.f, 0.f, 0.f};
  };
  auto compute = [&](const Batch& B, int g0, int g1, int c0) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (g0 + i >= g1) break;   // wave-uniform
      const uint8_t* fr = smem + (g0 + i - c0) * FB;
      floatx4 acc[NT][MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float z = sums[((g0 + i - c0) * MT + m) * XR + rl];
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][m] = floatx4{z, z, z, z};
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8_t f[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          f[m] = as_bf16x8(*reinterpret_cast<const u32x4*>(fr + m * (256 * XR) + off[s]));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t d = s == 0 ? B.w[i][j].x : s == 1 ? B.w[i][j].y : s == 2 ? B.w[i][j].z : B.w[i][j].w;
          const bf16x8_t op = operand16(d, nib_mask, bf16_16);
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

  Batch P, Q;
  const uint32_t hdr = header_word(blob);   // tested before the first store
  bool ok = false;
  clear();
  const int u_end = u0 + mine * step;
  for (int c0 = 0; c0 < G; c0 += A.chunk) {
    const int c1 = min(c0 + A.chunk, G);
    // this wave's part of the piece
    const int ga = KS > 1 ? c0 + (c1 - c0) * (wave % KS) / KS : c0;
    const int gb = KS > 1 ? c0 + (c1 - c0) * (wave % KS + 1) / KS : c1;
    const bool busy = mine > 0 && ga < gb;
    int u = u0, g = ga;                       // what P holds
    if (busy) load(P, u, g, gb);
    if (c0 > 0) __syncthreads();              // the piece before is read
    stage(c0, c1);
    __syncthreads();
    if (c0 == 0) ok = header_word_ok(hdr, 1, A.n, A.k);
    if (!busy) continue;
    // steps of W groups, the next one's loads under way, over tiles' ends
    auto walk = [&](const Batch& now, Batch& next) {
      int nu = u, ng = g + W;
      if (ng >= gb) nu += step, ng = ga;
      load(next, min(nu, u_end - step), ng, gb);
      __builtin_amdgcn_sched_barrier(0);
      compute(now, g, gb, c0);
      if (ng == ga && KS == 1 && c1 == G) {
        if (ok) finish(u);
        clear();
      }
      u = nu;
      g = ng;
    };
    while (u < u_end) {
      walk(P, Q);
      if (u >= u_end) break;
      walk(Q, P);
    }
  }
  if constexpr (KS > 1) {
    floatx4* const red = reinterpret_cast<floatx4*>(smem + size_t(A.chunk) * group_bytes(MT, XR));
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) red[((wave * NT + j) * MT + m) * 64 + lane] = tot[j][m];
    __syncthreads();
    if (wave % KS || !mine || !ok) return;
#pragma unroll
    for (int w = 1; w < KS; ++w)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) tot[j][m] += red[(((wave + w) * NT + j) * MT + m) * 64 + lane];
    finish(u0);
  }
}

template <int MT, int XR, int KS>
hipError_t launch16(Args16 a, const MoeGemm& g, hipStream_t s) {
  constexpr int W = 2, WAVES = waves_of(MT), TALL = MT == 1 ? XR : 16 * MT;
  const int G = g.k / 128, T = g.n / 16;
  const int most = (160 * 1024 - red_bytes(MT, KS)) / group_bytes(MT, XR);
  a.chunk = G < most ? G : most;
  const int64_t tiles = most_tiles(g.plan.rows, g.plan.groups, TALL);
  const int64_t units = g.silu_mul ? T / 2 : (T + 1) / 2;
  const int64_t widest = (units + WAVES / KS - 1) / (WAVES / KS);
  const int cus = device_cu_count();
  int64_t walkers = widest;
  // 16 waves to a CU, as far as there are units for them.  Where x passes through
  // LDS in pieces it does so for every unit of a wave, and one unit to a wave is
  // best (660 rows over 16 experts of 3840 x 3840: 73 -> 48 us).
  if (KS == 1 && a.chunk >= G) {
    walkers = (16 / WAVES * (cus > 0 ? cus : 256) + tiles - 1) / tiles;
    if (walkers > widest) walkers = widest;
    // Then as few blocks as do these units in the nearest whole number of rounds
    // (692 rows over 16 experts of 3840 x 1920: 36 -> 28 us; the others as before).
    const int64_t in_round = WAVES * walkers;
    const int64_t near = (2 * units + in_round) / (2 * in_round), rounds = near > 0 ? near : 1;
    walkers = (units + WAVES * rounds - 1) / (WAVES * rounds);
  }
  a.walkers = int(walkers);
  const size_t lds = size_t(a.chunk) * group_bytes(MT, XR) + red_bytes(MT, KS);
  static std::atomic<int> done[4][64];
  auto run = [&](auto kern, std::atomic<int>* flag) {
    const hipError_t e = lds_limit_once(flag, reinterpret_cast<const void*>(kern), 160 * 1024);
    if (e != hipSuccess) return e;
    kern<<<unsigned(tiles * walkers), WAVES * 64, lds, s>>>(a);
    return hipGetLastError();
  };
  if (g.silu_mul)
    return g.y_dtype == 1 ? run(moe_w4a16_kernel<MT, XR, KS, W, true, true>, done[0])
                          : run(moe_w4a16_kernel<MT, XR, KS, W, true, false>, done[1]);
  return g.y_dtype == 1 ? run(moe_w4a16_kernel<MT, XR, KS, W, false, true>, done[2])
                        : run(moe_w4a16_kernel<MT, XR, KS, W, false, false>, done[3]);
}

}  // namespace

hipError_t launch_moe_gemm_w4a16(const MoeGemm& g, const void* x, hipStream_t s) {
  const BlobLayout L = blob_layout(1, g.n, g.k);
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
  // Tiles of 4 places: up to 4 tokens (no expert has more rows, a token chooses
  // it once), or where experts have 2 rows on average, so that few take a second
  // tile.  x then leaves room in LDS for a second block on the CU.
  if (g.plan.rows <= 4 * g.top_k || g.plan.rows <= 2 * g.plan.groups) {
    // waves to a pair of weight tiles: until 8 waves to a CU have work, at
    // least 4 groups each
    const int cus = device_cu_count();
    const int64_t pairs = most_tiles(g.plan.rows, g.plan.groups, 4) * ((g.n / 16 + 1) / 2);
    int ks = 1;
    while (ks < 8 && pairs * ks < 8 * (cus > 0 ? cus : 256) && g.k / 128 >= 8 * ks) ks *= 2;
    if (ks == 8) return launch16<1, 4, 8>(a, g, s);
    if (ks == 4) return launch16<1, 4, 4>(a, g, s);
    if (ks == 2) return launch16<1, 4, 2>(a, g, s);
    return launch16<1, 4, 1>(a, g, s);
  }
  // the height of a tile: by the rows that an expert has on average
  if (g.plan.rows / g.plan.groups > 12) return launch16<2, 16, 1>(a, g, s);
  return launch16<1, 16, 1>(a, g, s);
}

}  // namespace qlin
