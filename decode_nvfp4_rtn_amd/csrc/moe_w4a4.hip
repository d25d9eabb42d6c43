// Products of rows with their experts' NVFP4 weights, NVFP4 activations (the
// prefill path of a mixture of experts).
//
//   y[p, :] = s_tA s_tW(e) sum_g sA sW sum_{k in g} E2M1(a[row(p), k]) E2M1(w_e[:, k])
//
// for the places p of expert e's run, or, with silu_mul, silu(g) * u of the two
// halves g, u of that product.  The arithmetic is that of the dense
// block-cooperative kernel: fp16 operands that hold E2M1 * E4M3 exactly,
// v_mfma_f32_16x16x32_f16, binary32 accumulation, every code dequantized once
// per block.
//
// Block 256 (weight rows) x up to 256 (places of one expert), 8 wavefronts; K
// advances 64 per stage, the fp16 tiles double buffered in LDS.  A thread
// dequantizes one weight row or one activation row, whose address it looks up
// once: activation rows come in the plan's order or through it from the
// tokens.  Codes are loaded 128 of k at a time (64 bytes of a row) into a ring
// of RING such pairs of stages, 2 RING - 3 stages before their dequantization.
//
// Experts' runs are ragged.  A tile of more than 128 places has its waves 2 x
// 4, each 128 x 64, as the dense kernel; a lower one 4 x 2, each 64 x 64, one
// of a run's first 64 places on each SIMD, so that half the products take half
// the time.  A wave whose 64 places lie past the run skips its products, one
// whose activation rows do their dequantization.  Low tiles do little for each
// weight and wait for memory: with their 64 accumulators the ring can be
// deeper.
//
// With silu_mul the 256 weight rows are 128 gate rows and their 128 up rows,
// alternating by 16, so that a wave holds both halves of an output in the same
// lane and the epilogue writes h: 4 n bytes a place less to memory and back
// than g and u.
//
// Few rows of an expert: a second kernel, tiles of 64 places, weights from memory
// to registers (below).
//
// 8192 tokens, 8 of 64 experts of 2048 x 4096: 977 - 995 us, 1105 - 1125 TFLOP/s
// (the dense kernel's rate for a tile; runs padded to whole 64s are 12 % of the
// products).  4095 tokens, 2 of 8 experts of 4096 x 2048: 147 - 153 us, 900 - 933
// TFLOP/s in 2.3 rounds of tiles.  1000 tokens, 4 of 60 experts of 2816 x 2048, by the
// second kernel: 71 - 75 us, 207 MB at 2.8 - 2.9 TB/s and 550 - 580 TFLOP/s (85 us on
// weights that the Infinity Cache does not hold); the first took 139.  313 MB come past
// the L2s: an expert's weights once for each of its tiles.
#include "moe.hpp"
#include "w4a4_ops.hpp"

namespace qlin {
namespace {

constexpr int TALL = 256, WIDE = 256, BK = 64, RS = 160, GROUP_M = 4;
constexpr int TILE_BYTES = 256 * RS;

struct Args4 {
  RowPlan plan;
  const uint8_t *codes, *scales;
  const float* a_ts;
  const uint8_t* experts;
  int64_t blob_stride, wc_off, ws_off;
  void* y;
  int top_k, gather, n, k, cus;
};

// Columns [n0, n0 + cols) of a tile's rows, zeroed: pairs without an expert.
template <bool kBF16Out>
__device__ __forceinline__ void zero_rows(void* y, const RowTile& tile, int n0, int cols, int n_out) {
  constexpr int size = kBF16Out ? 2 : 4;
  const int per = cols * size / 16;
  for (int i = threadIdx.x; i < tile.count * per; i += 512)
    reinterpret_cast<uint4*>(static_cast<uint8_t*>(y) +
                             (int64_t(tile.first + i / per) * n_out + n0) * size)[i % per] = make_uint4(0, 0, 0, 0);
}

// One tile.  WN wavefronts along the weight rows, TN x 16 of them each, and 8 /
// WN along the places, 64 each.  kAll: every wave has places (a branch around its
// products costs 4 % of a full tile's time).
template <int WN, int TN, int RING, bool kAll, bool kSilu, bool kBF16Out>
__device__ __forceinline__ void w4a4_tile(const Args4& A, const RowTile& tile, int n0, uint8_t* smem) {
  constexpr int TM = 4;                 // m-tiles of a wave
  constexpr int WROWS = WN * TN * 16;   // weight rows of the block
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = A.n, K = A.k, H = N / 2;
  const int n_out = kSilu ? H : N;
  const uint8_t* blob = A.experts + tile.group * A.blob_stride;
  if (!blob_matches(blob, 0, N, K)) return;   // before any barrier: uniform

  const int KT = K / 128;
  const __amdgpu_buffer_rsrc_t rcw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(blob + A.wc_off), 0, 0x7FFFFFFF, 0x00020000);
  const __amdgpu_buffer_rsrc_t rsw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(blob + A.ws_off), 0, 0x7FFFFFFF, 0x00020000);
  const __amdgpu_buffer_rsrc_t rcx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(A.codes), 0, 0x7FFFFFFF, 0x00020000);
  const __amdgpu_buffer_rsrc_t rsx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(A.scales), 0, 0x7FFFFFFF, 0x00020000);
  // this thread's row: four waves take the weight rows, four the places (low
  // tiles: the waves with products take places); past the weights' or the
  // run's end the last one (its products reach only outputs that are never
  // stored)
  const bool isw = WN == 2 ? wave < 4 : wave >= 4;
  const int lrow = tid & 255;
  uint32_t vc, vs;
  if (isw) {
    int wrow;
    if constexpr (kSilu) {
      const int col = min(n0 + (lrow >> 5) * 16 + (lrow & 15), H - 16 + (lrow & 15));
      wrow = ((lrow >> 4) & 1) * H + col;
    } else {
      wrow = min(n0 + lrow, N - 16 + (lrow & 15));
    }
    const uint32_t at = uint32_t(wrow >> 4) * uint32_t(KT) * 16u + uint32_t(wrow & 15);
    vc = at * 64u;
    vs = at * 8u;
  } else {
    const int place = tile.first + min(lrow, tile.count - 1);
    uint32_t from = uint32_t(place);
    if (A.gather) from = min(uint32_t(A.plan.order[place]), uint32_t(A.plan.rows - 1)) / uint32_t(A.top_k);
    vc = from * uint32_t(K / 2);
    vs = from * uint32_t(K / 16);
  }
  const int wn = wave & (WN - 1), wm = wave / WN;
  const bool multiplies = kAll || wm * 64 < tile.count;
  const bool dequantizes = kAll && WROWS == 256 ? true : (wave & 3) * 64 < (isw ? WROWS : tile.count);

  // codes and scales of 128 of k of this thread's row
  struct Regs {
    u32x4 c[4];
    uint32_t sc[2];
  };
  Regs ring[RING];
  const __amdgpu_buffer_rsrc_t rc = isw ? rcw : rcx, rs = isw ? rsw : rsx;
  const int cstep = isw ? 1024 : 64, sstep = isw ? 128 : 8;
  auto gload = [&](Regs& R, int p) {   // past the end: the last one again, never used
    p = min(p, KT - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) R.c[i] = __builtin_amdgcn_raw_buffer_load_b128(rc, vc, p * cstep + 16 * i, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) R.sc[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, vs, p * sstep + 4 * i, 0);
  };
  uint8_t* const own_row = smem + (isw ? 0 : TILE_BYTES) + lrow * RS;
  // eight values (of eight) of half `half` of a pair into LDS buffer `half`
  auto dq_store = [&](const Regs& R, int half, int d) {
    *reinterpret_cast<u32x4*>(own_row + half * 2 * TILE_BYTES + d * 16) =
        dequant8(R.c[2 * half + (d >> 2)][d & 3], scale_h2(R.sc[half], d >> 1));
  };

  floatx4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int i = 0; i < RING; ++i) {
    gload(ring[i], i);
    __builtin_amdgcn_sched_barrier(0);   // in this order, which the waits below count on
  }
  if (dequantizes) {
#pragma unroll
    for (int d = 0; d < 8; ++d) dq_store(ring[0], 0, d);
  }
  __syncthreads();

  const int r = lane & 15, q = lane >> 4;
  const int wbase = (wn * (TN * 16) + r) * RS + q * 16;
  const int xbase = (wm * 64 + r) * RS + q * 16;

  // one stage: MFMAs on LDS buffer `buf` while half `buf ^ 1` of `nxt` is
  // dequantized into the other buffer
  auto stage = [&](int buf, const Regs& nxt) {
    const uint8_t* wt = smem + buf * 2 * TILE_BYTES;
    const uint8_t* xt = wt + TILE_BYTES;
    if (!multiplies) {
      if (dequantizes) {
#pragma unroll
        for (int d = 0; d < 8; ++d) dq_store(nxt, buf ^ 1, d);
      }
      return;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      half8_t xf[TM];
#pragma unroll
      for (int j = 0; j < TM; ++j)
        xf[j] = *reinterpret_cast<const half8_t*>(xt + xbase + j * 16 * RS + s * 64);
      half8_t wf = *reinterpret_cast<const half8_t*>(wt + wbase + s * 64);
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        half8_t wn_f = wf;
        if (i + 1 < TN)
          wn_f = *reinterpret_cast<const half8_t*>(wt + wbase + (i + 1) * 16 * RS + s * 64);
#pragma unroll
        for (int j = 0; j < TM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf, xf[j], acc[i][j], 0, 0, 0);
        constexpr int ITS = 2 * TN;   // eight stores over them
#pragma unroll
        for (int d = (s * TN + i) * 8 / ITS; d < (s * TN + i + 1) * 8 / ITS; ++d) dq_store(nxt, buf ^ 1, d);
        wf = wn_f;
      }
    }
  };
  // pair p lies in ring[p % RING]; its second half is dequantized during its
  // first stage, after which its place in the ring is free.  On the last pair
  // the second stage writes the idle buffer, which nothing reads again.
  auto pair = [&](int p, int i) {
    stage(0, ring[i]);
    __syncthreads();
    gload(ring[i], p + RING);
    __builtin_amdgcn_sched_barrier(0);   // issue the loads here, not after the stage
    stage(1, ring[(i + 1) % RING]);
    __syncthreads();
  };
  int p = 0;
  for (; p + RING <= KT; p += RING) {
#pragma unroll
    for (int i = 0; i < RING; ++i) pair(p + i, i);
  }
#pragma unroll
  for (int i = 0; i < RING - 1; ++i)
    if (p + i < KT) pair(p + i, i);
  if (!multiplies) return;   // no barrier follows

  const float stv = A.a_ts[0] * reinterpret_cast<const BlobHeader*>(blob)->tensor_scale;
  static_assert(!kSilu || TN % 2 == 0, "a wave has whole pairs of gate and up");
  constexpr int TO = kSilu ? TN / 2 : TN;   // 16-column tiles of the wave's output
  if constexpr (kSilu) {
#pragma unroll
    for (int i = 0; i < TO; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        floatx4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float g = acc[2 * i][j][e] * stv, u = acc[2 * i + 1][j][e] * stv;
          h[e] = g / (1.0f + expf(-g)) * u;
        }
        acc[i][j] = h;
      }
  } else {
#pragma unroll
    for (int i = 0; i < TO; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = acc[i][j] * stv;
  }
  const int col0 = n0 + wn * (TO * 16);
  const int left = tile.count - wm * 64;   // places of this wave
  const int64_t row0 = int64_t(tile.first) + wm * 64;
  if constexpr (kBF16Out) {
    // through a private LDS region, so that whole rows are stored (a lane
    // holds four columns of one row); a wave's LDS operations stay in order
    constexpr int ORS = TO * 32 + 32, LPR = TO * 2;   // row bytes, lanes to a row
    static_assert(8 * 64 * ORS <= 4 * TILE_BYTES, "output staging fits in LDS");
    uint8_t* const ot = smem + wave * (64 * ORS);
#pragma unroll
    for (int i = 0; i < TO; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const floatx4 v = acc[i][j];
        *reinterpret_cast<uint2*>(ot + (16 * j + r) * ORS + (16 * i + 4 * q) * 2) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    __asm__ volatile("" ::: "memory");   // keep the reads below the writes
    const int n = col0 + 8 * (lane % LPR);
#pragma unroll
    for (int it = 0; it < LPR; ++it) {
      const int rr = (64 / LPR) * it + lane / LPR;
      const uint4 v = *reinterpret_cast<const uint4*>(ot + rr * ORS + 16 * (lane % LPR));
      if (rr < left && n < n_out)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.y) + (row0 + rr) * n_out + n) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < TO; ++i) {
      const int n = col0 + i * 16 + 4 * q;
      if (n >= n_out) continue;
#pragma unroll
      for (int j = 0; j < TM; ++j)
        if (16 * j + r < left)
          *reinterpret_cast<floatx4*>(static_cast<float*>(A.y) + (row0 + 16 * j + r) * n_out + n) = acc[i][j];
    }
  }
}

// A block to a CU at a time: what comes after the last whole round of tiles would
// take a round of its own with most CUs idle, so those tiles are cut into 2 or 4
// parts along the weight rows, as far as the CUs go.
template <bool kSilu, bool kBF16Out>
__global__ __launch_bounds__(512, 1) void moe_w4a4_kernel(Args4 A) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // [2][W tile, X tile]
  const int n_out = kSilu ? A.n / 2 : A.n;
  constexpr int OUT_WIDE = kSilu ? WIDE / 2 : WIDE;

  // Full tiles first: XCD-major (consecutive blocks go to different XCDs, so
  // each gets a contiguous run of tiles), in groups of GROUP_M row tiles with
  // the weight tiles in order, as the dense kernel's, so that an XCD's blocks
  // share panels in its L2.  Then the experts' ends, whose costs differ, spread
  // over the XCDs as they come.
  const int tiles_n = (n_out + OUT_WIDE - 1) / OUT_WIDE;
  const PlanRuns runs(A.plan);
  auto fulls = [](int, GroupRun run) { return (run.end - run.first) / TALL; };
  auto ends = [](int, GroupRun run) { return (run.end - run.first) % TALL ? 1 : 0; };
  // no plan has more than these, whatever the offsets hold
  const int full_m = min(count_tiles(runs, fulls), A.plan.rows / TALL);
  const int end_m = min(count_tiles(runs, ends), A.plan.groups + 1);
  const int full = full_m * tiles_n, total = full + end_m * tiles_n;
  const int whole = total / A.cus * A.cus, rest = total - whole;
  const int cut = 4 * rest <= A.cus ? 4 : 2 * rest <= A.cus ? 2 : 1;
  int t = blockIdx.x, part = 0, parts = 1;
  if (t >= whole) {
    part = (t - whole) % cut;
    t = whole + (t - whole) / cut;
    parts = cut;
  }
  if (t >= total) return;
  RowTile tile{-1, 0, 0};
  int at_n, at_m;
  if (t < full) {
    const int even = min(full, whole) & ~7;
    if (t < even) t = (t & 7) * (even >> 3) + (t >> 3);
    const int in_group = GROUP_M * tiles_n, first_m = t / in_group * GROUP_M, tall = min(full_m - first_m, GROUP_M);
    at_m = first_m + t % in_group % tall;
    at_n = t % in_group / tall;
    search_tiles<false>(runs, TALL, at_m, tile, fulls);
  } else {
    at_m = (t - full) / tiles_n;
    at_n = (t - full) % tiles_n;
    search_tiles<true>(runs, TALL, at_m, tile, ends);
  }
  if (tile.group < 0) return;
  const int wide = OUT_WIDE / parts, n0 = at_n * OUT_WIDE + part * wide;   // output columns
  if (n0 >= n_out) return;
  if (tile.group == A.plan.groups) {   // rows without an expert
    zero_rows<kBF16Out>(A.y, tile, n0, min(wide, n_out - n0), n_out);
    return;
  }
  const bool low = tile.count <= 128;
  if (parts == 1) {
    if (tile.count > 192) w4a4_tile<2, 8, 2, true, kSilu, kBF16Out>(A, tile, n0, smem);
    else if (low) w4a4_tile<4, 4, 4, false, kSilu, kBF16Out>(A, tile, n0, smem);
    else w4a4_tile<2, 8, 2, false, kSilu, kBF16Out>(A, tile, n0, smem);
  } else if (parts == 2) {
    if (low) w4a4_tile<4, 2, 4, false, kSilu, kBF16Out>(A, tile, n0, smem);
    else w4a4_tile<2, 4, 4, false, kSilu, kBF16Out>(A, tile, n0, smem);
  } else {
    w4a4_tile<2, 2, 4, false, kSilu, kBF16Out>(A, tile, n0, smem);
  }
}

// Short runs: tiles of 16 TM places, one m-tile of 16 for each of TM products of
// an operand, and weights that go from memory to a wave's registers and no
// further.
//
// Block 8 waves x 2 weight tiles of 16 rows (with silu_mul a gate tile and its
// up tile) x 16 TM places.  Of a weight tile's 128 of k a wave's load is one
// contiguous KB, lane (row r, quarter q) k 32 q .. 32 q + 31; dword s of it is
// the operand of step s, so step s contracts k 32 q + 8 s .. + 7 of each q, and
// the activations' fragments lie in LDS in that order: a thread that
// dequantizes 16 bytes of codes of a place stores one piece for each step,
// lane after lane.  Activations are dequantized PIECE pairs (128 of k each) at
// a time into the other of two buffers, one barrier to a piece; weights are
// loaded RING pairs ahead.  16 TM x 128 of k of products to an operand of 16 x
// 128: at 64 places the MFMAs take half the time of the weights' way from
// memory.
constexpr int PIECE = 2, FRAG = 1024;
constexpr int low_bytes(int tm) { return 2 * PIECE * tm * 4 * FRAG; }

template <int TM, bool kSilu, bool kBF16Out>
__device__ __forceinline__ void w4a4_low_tile(const Args4& A, const RowTile& tile, int n0, uint8_t* smem) {
  constexpr int RING = 4, LOW = 16 * TM;
  // smem: [2][PIECE][TM][4][64 lanes] x 16 bytes
  constexpr int BUF = PIECE * TM * 4 * FRAG;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_out = kSilu ? A.n / 2 : A.n;
  constexpr int OUT_WIDE = kSilu ? 128 : 256;
  const uint8_t* blob = A.experts + tile.group * A.blob_stride;
  if (!blob_matches(blob, 0, A.n, A.k)) return;   // before any barrier: uniform

  const int KT = A.k / 128, T = A.n / 16;
  const int r = lane & 15, q = lane >> 4;
  // this wave's weight tiles; past the last one again (not stored)
  const uint8_t *wc[2], *ws[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = kSilu ? min(n0 / 16 + wave, T / 2 - 1) + j * (T / 2) : min(n0 / 16 + 2 * wave + j, T - 1);
    wc[j] = blob + A.wc_off + int64_t(t) * KT * 1024 + r * 64 + q * 16;
    ws[j] = blob + A.ws_off + int64_t(t) * KT * 128 + r * 8 + q * 2;
  }
  struct Regs {
    uint4 c[2];
    uint32_t s[2];
  };
  Regs ring[RING];
  auto wload = [&](Regs& R, int p) {   // past the end: the last one again, not used
    p = min(p, KT - 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      R.c[j] = load_nt16(wc[j] + int64_t(p) * 1024);
      R.s[j] = *reinterpret_cast<const uint16_t*>(ws[j] + int64_t(p) * 128);
    }
  };
  // Activations: the units (pair, m-tile) of a piece go round the waves; a
  // unit is 16 bytes of codes of each of 16 places and 4 quarters.
  constexpr int UNITS = (PIECE * TM + 7) / 8;
  const uint8_t *xc[UNITS], *xs[UNITS];
  bool active[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int unit = wave + 8 * i, mt = unit % TM;
    active[i] = unit < PIECE * TM && 16 * mt < tile.count;   // wave-uniform
    const int place = tile.first + min(16 * mt + r, tile.count - 1);
    int64_t from = place;
    if (A.gather) from = min(uint32_t(A.plan.order[place]), uint32_t(A.plan.rows - 1)) / uint32_t(A.top_k);
    xc[i] = A.codes + from * (A.k / 2) + q * 16;
    xs[i] = A.scales + from * (A.k / 16) + q * 2;
  }
  struct XRegs {
    uint4 c[UNITS];
    uint32_t s[UNITS];
  };
  auto xload = [&](XRegs& R, int piece) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int64_t p = min(piece * PIECE + (wave + 8 * i) / TM % PIECE, KT - 1);
      R.c[i] = *reinterpret_cast<const uint4*>(xc[i] + p * 64);
      R.s[i] = *reinterpret_cast<const uint16_t*>(xs[i] + p * 8);
    }
  };
  auto xstore = [&](const XRegs& R, int buf) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      if (!active[i]) continue;
      uint8_t* to = smem + buf * BUF + (wave + 8 * i) * (4 * FRAG) + lane * 16;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        *reinterpret_cast<u32x4*>(to + s * FRAG) = dequant8(pick(R.c[i], s), scale_h2(R.s[i], s >> 1));
    }
  };

  floatx4 acc[2][TM];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[j][m] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Regs& R, int buf, int in_piece) {
    const uint8_t* x = smem + buf * BUF + in_piece * (TM * 4 * FRAG) + lane * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      half8_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = __builtin_bit_cast(half8_t, dequant8(pick(R.c[j], s), scale_h2(R.s[j], s >> 1)));
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const half8_t xf = *reinterpret_cast<const half8_t*>(x + (m * 4 + s) * FRAG);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[j], xf, acc[j][m], 0, 0, 0);
      }
    }
  };

  XRegs xa;
  xload(xa, 0);
#pragma unroll
  for (int i = 0; i < RING; ++i) {
    wload(ring[i], i);
    __builtin_amdgcn_sched_barrier(0);   // in this order, which the waits count on
  }
  xstore(xa, 0);
  xload(xa, 1);
  __syncthreads();
  // pieces two by two, so that ring and buffers have fixed places; pairs past
  // the end are skipped
  const int pieces = (KT + PIECE - 1) / PIECE;
  for (int c = 0; c < pieces; c += RING / PIECE) {
#pragma unroll
    for (int h = 0; h < RING / PIECE; ++h) {
      xstore(xa, (h & 1) ^ 1);
      xload(xa, c + h + 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < PIECE; ++i) {
        const int p = (c + h) * PIECE + i;
        if (p < KT) compute(ring[h * PIECE + i], h & 1, i);
        wload(ring[h * PIECE + i], p + RING);
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
    }
  }

  const float stv = A.a_ts[0] * reinterpret_cast<const BlobHeader*>(blob)->tensor_scale;
  // bf16 goes through LDS, so that whole rows are stored; [LOW places][OUT_WIDE]
  constexpr int ORS = OUT_WIDE * 2 + 16;
  static_assert(LOW * ORS <= low_bytes(4), "output staging fits in the launch's LDS");
  auto put = [&](int col, int m, floatx4 v) {   // col: within the block
    const int place = 16 * m + r;
    if constexpr (kBF16Out) {
      *reinterpret_cast<uint2*>(smem + place * ORS + col * 2) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else if (place < tile.count && n0 + col < n_out) {
      *reinterpret_cast<floatx4*>(static_cast<float*>(A.y) + int64_t(tile.first + place) * n_out + n0 + col) = v;
    }
  };
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    if constexpr (kSilu) {
      floatx4 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float g = acc[0][m][e] * stv, u = acc[1][m][e] * stv;
        h[e] = g / (1.0f + expf(-g)) * u;
      }
      put(wave * 16 + 4 * q, m, h);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) put((2 * wave + j) * 16 + 4 * q, m, acc[j][m] * stv);
    }
  }
  if constexpr (kBF16Out) {
    __syncthreads();
    constexpr int LPR = OUT_WIDE / 8;   // lanes to a row
    const int n = 8 * (threadIdx.x % LPR);
    for (int place = threadIdx.x / LPR; place < tile.count; place += 512 / LPR)
      if (n0 + n < n_out)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.y) + int64_t(tile.first + place) * n_out + n0 + n) =
            *reinterpret_cast<const uint4*>(smem + place * ORS + n * 2);
  }
}

template <bool kSilu, bool kBF16Out>
__global__ __launch_bounds__(512, 4) void moe_w4a4_low_kernel(Args4 A) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int n_out = kSilu ? A.n / 2 : A.n;
  constexpr int OUT_WIDE = kSilu ? 128 : 256;
  const int tiles_n = (n_out + OUT_WIDE - 1) / OUT_WIDE;
  const int n0 = (blockIdx.x % tiles_n) * OUT_WIDE;
  // tiles by their height, the highest first, so that the last blocks of the
  // launch are short ones; then the rows without an expert
  RowTile tile{-1, 0, 0};
  int number = blockIdx.x / tiles_n;
  const PlanRuns runs(A.plan);
  const int groups = A.plan.groups;
  bool found = search_tiles<false>(runs, 64, number, tile, [&](int g, GroupRun run) {
    return g < groups ? (run.end - run.first) / 64 : 0;
  });
  for (int low = 48; low >= 0 && !found; low -= 16)
    found = search_tiles<true>(runs, 64, number, tile, [&](int g, GroupRun run) {
      const int rows = (run.end - run.first) % 64;
      return g < groups && rows > low && rows <= low + 16 ? 1 : 0;
    });
  if (!found && !search_tiles<false>(runs, 64, number, tile, [&](int g, GroupRun run) {
        return g == groups ? (run.end - run.first + 63) / 64 : 0;
      }))
    return;
  if (tile.group == A.plan.groups)
    zero_rows<kBF16Out>(A.y, tile, n0, min(OUT_WIDE, n_out - n0), n_out);
  else if (tile.count > 48)
    w4a4_low_tile<4, kSilu, kBF16Out>(A, tile, n0, smem);
  else if (tile.count > 32)
    w4a4_low_tile<3, kSilu, kBF16Out>(A, tile, n0, smem);
  else if (tile.count > 16)
    w4a4_low_tile<2, kSilu, kBF16Out>(A, tile, n0, smem);
  else
    w4a4_low_tile<1, kSilu, kBF16Out>(A, tile, n0, smem);
}

}  // namespace

hipError_t launch_moe_gemm_w4a4(const MoeGemm& g, const uint8_t* codes, const uint8_t* scales,
                                const float* a_ts, hipStream_t s) {
  const BlobLayout L = blob_layout(0, g.n, g.k);
  Args4 a{};
  a.plan = g.plan;
  a.codes = codes;
  a.scales = scales;
  a.a_ts = a_ts;
  a.experts = g.experts;
  a.blob_stride = g.blob_stride;
  a.wc_off = int64_t(L.codes_off);
  a.ws_off = int64_t(L.aux_off);
  a.y = g.y;
  a.top_k = g.top_k;
  a.gather = g.gather;
  a.n = g.n;
  a.k = g.k;
  static_assert(TALL == 256 && WIDE == 256, "as w4a4_tall and w4a4_tiles count them");
  const int tall = w4a4_tall(g.plan.rows, g.plan.groups);
  const int64_t tiles = w4a4_tiles(g.plan.rows, g.plan.groups, g.n);
  static std::atomic<int> done[8][64];
  const int cus = device_cu_count();
  a.cus = cus > 0 ? cus : 256;
  auto run = [&](auto kern, std::atomic<int>* flag, size_t lds) {
    const hipError_t e = lds_limit_once(flag, reinterpret_cast<const void*>(kern), int(lds));
    if (e != hipSuccess) return e;
    // tiles of 256 places: with room for a last round of parts of tiles
    const int64_t blocks = tiles + (tall == TALL ? a.cus : 0);
    kern<<<unsigned(blocks), 512, lds, s>>>(a);
    return hipGetLastError();
  };
  const bool bf16 = g.y_dtype == 1;
  if (tall < TALL) {
    constexpr size_t lds = low_bytes(4);
    if (g.silu_mul)
      return bf16 ? run(moe_w4a4_low_kernel<true, true>, done[4], lds)
                  : run(moe_w4a4_low_kernel<true, false>, done[5], lds);
    return bf16 ? run(moe_w4a4_low_kernel<false, true>, done[6], lds)
                : run(moe_w4a4_low_kernel<false, false>, done[7], lds);
  }
  constexpr size_t lds = 2 * 2 * TILE_BYTES;
  if (g.silu_mul)
    return bf16 ? run(moe_w4a4_kernel<true, true>, done[0], lds)
                : run(moe_w4a4_kernel<true, false>, done[1], lds);
  return bf16 ? run(moe_w4a4_kernel<false, true>, done[2], lds)
              : run(moe_w4a4_kernel<false, false>, done[3], lds);
}

}  // namespace qlin
