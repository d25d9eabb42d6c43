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
// Block 256 (weight rows) x 256 (places of one expert), 8 wavefronts in 2 x 4,
// each 128 x 64; K advances 64 per stage, the fp16 tiles double buffered in
// LDS, the codes of stage s + 2 loaded at the start of stage s.  A thread
// dequantizes one weight row or one activation row, whose address it looks up
// once: activation rows come in the plan's order or through it from the
// tokens.  Experts' runs are ragged: a wave whose 64 places lie past the run
// skips its products (the block's waves then share fewer MFMAs, not fewer
// weights), and one whose 64 activation rows do skips their dequantization.
//
// With silu_mul the 256 weight rows are 128 gate rows and their 128 up rows,
// alternating by 16, so that a wave holds both halves of an output in the same
// lane and the product's epilogue writes h: a pass over 4 n bytes a place less
// than writing g and u and reading them again.
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
  int top_k, gather, n, k;
};

template <bool kSilu, bool kBF16Out>
__global__ __launch_bounds__(512, 1) void moe_w4a4_kernel(Args4 A) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // [2][W tile, X tile]
  constexpr int TN = 8, TM = 4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = A.n, K = A.k, H = N / 2;
  const int n_out = kSilu ? H : N;
  constexpr int OUT_WIDE = kSilu ? WIDE / 2 : WIDE;

  // tile: XCD-major over the tiles that there are, groups of GROUP_M row
  // tiles, weight tiles in order within a group
  const int tiles_n = (n_out + OUT_WIDE - 1) / OUT_WIDE;
  const int tiles_m = count_tiles(A.plan, TALL);
  const int total = tiles_m * tiles_n, per = (total + 7) / 8;
  const int in_xcd = blockIdx.x >> 3;
  const int t = (blockIdx.x & 7) * per + in_xcd;
  if (in_xcd >= per || t >= total) return;
  const int in_group = GROUP_M * tiles_n;
  const int first_m = (t / in_group) * GROUP_M;
  const int gsz = min(tiles_m - first_m, GROUP_M);
  const RowTile tile = find_tile(A.plan, TALL, first_m + (t % in_group) % gsz);
  const int n0 = ((t % in_group) / gsz) * OUT_WIDE;   // first output column
  if (tile.group < 0) return;

  if (tile.group == A.plan.groups) {   // rows without an expert: zeros
    const int cols = min(OUT_WIDE, n_out - n0) * (kBF16Out ? 2 : 4) / 16;
    for (int i = tid; i < tile.count * cols; i += 512)
      reinterpret_cast<uint4*>(static_cast<uint8_t*>(A.y) +
                               (int64_t(tile.first + i / cols) * n_out + n0) * (kBF16Out ? 2 : 4))[i % cols] =
          make_uint4(0, 0, 0, 0);
    return;
  }
  const uint8_t* blob = A.experts + tile.group * A.blob_stride;
  if (!blob_matches(blob, 0, N, K)) return;   // before any barrier: uniform

  const int KT = K / 128, S = K / BK;
  const __amdgpu_buffer_rsrc_t rcw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(blob + A.wc_off), 0, 0x7FFFFFFF, 0x00020000);
  const __amdgpu_buffer_rsrc_t rsw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(blob + A.ws_off), 0, 0x7FFFFFFF, 0x00020000);
  const __amdgpu_buffer_rsrc_t rcx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(A.codes), 0, 0x7FFFFFFF, 0x00020000);
  const __amdgpu_buffer_rsrc_t rsx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(A.scales), 0, 0x7FFFFFFF, 0x00020000);
  // this thread's row: weight rows on the first four waves, places on the
  // others; past the weights' or the run's end the last one (their products
  // reach only outputs that are never stored)
  const bool isw = wave < 4;
  const int lrow = tid & 255;
  uint32_t vc, vs;
  if (isw) {
    int wrow;
    if constexpr (kSilu) {
      const int col = min(n0 + (lrow >> 7) * 64 + ((lrow >> 5) & 3) * 16 + (lrow & 15), H - 16 + (lrow & 15));
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
  const int wn = wave & 1, wm = wave >> 1;
  const bool multiplies = wm * 64 < tile.count;
  const bool dequantizes = isw || (wave - 4) * 64 < tile.count;

  struct Regs {
    uint4 c[2];
    uint32_t sc;
  };
  Regs ra, rb;
  const __amdgpu_buffer_rsrc_t rc = isw ? rcw : rcx, rs = isw ? rsw : rsx;
  auto gload = [&](Regs& R, int st) {
    const int co = isw ? (st >> 1) * 1024 + (st & 1) * 32 : st * 32;
    const int so = isw ? (st >> 1) * 128 + (st & 1) * 4 : st * 4;
    const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(rc, vc, co, 0);
    const u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(rc, vc, co + 16, 0);
    R.c[0] = make_uint4(a[0], a[1], a[2], a[3]);
    R.c[1] = make_uint4(b[0], b[1], b[2], b[3]);
    R.sc = __builtin_amdgcn_raw_buffer_load_b32(rs, vs, so, 0);
  };
  uint8_t* const own_row = smem + (isw ? 0 : TILE_BYTES) + lrow * RS;
  auto dq_store = [&](const Regs& R, int buf, int d) {
    *reinterpret_cast<u32x4*>(own_row + buf * 2 * TILE_BYTES + d * 16) =
        dequant8(pick(R.c[d >> 2], d & 3), scale_h2(R.sc, d >> 1));
  };

  floatx4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  gload(ra, 0);
  if (dequantizes) {
#pragma unroll
    for (int d = 0; d < 8; ++d) dq_store(ra, 0, d);
  }
  gload(rb, 1);   // K is a multiple of 128: an even number of stages
  __syncthreads();

  const int r = lane & 15, q = lane >> 4;
  const int wbase = (wn * 128 + r) * RS + q * 16;
  const int xbase = (wm * 64 + r) * RS + q * 16;

  // one stage: MFMAs on LDS buffer `buf` while `nxt` (the next stage's codes)
  // is dequantized into the other buffer
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
        const int it = s * TN + i;
        if (it % 2 == 0) dq_store(nxt, buf ^ 1, it / 2);
        wf = wn_f;
      }
    }
  };
  // prefetches are unconditional, their stage clamped to the last
  for (int st = 0; st < S; st += 2) {
    gload(ra, min(st + 2, S - 1));
    __builtin_amdgcn_sched_barrier(0);
    stage(0, rb);
    __syncthreads();
    gload(rb, min(st + 3, S - 1));
    __builtin_amdgcn_sched_barrier(0);
    stage(1, ra);
    __syncthreads();
  }
  if (!multiplies) return;   // no barrier follows

  const float stv = A.a_ts[0] * reinterpret_cast<const BlobHeader*>(blob)->tensor_scale;
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
  const int64_t tiles = most_tiles(g.plan.rows, g.plan.groups, TALL) * ((g.n + WIDE - 1) / WIDE);
  const int blocks = int((tiles + 7) / 8 * 8);
  constexpr size_t lds = 2 * 2 * TILE_BYTES;
  static std::atomic<int> done[4][64];
  auto run = [&](auto kern, std::atomic<int>* flag) {
    const hipError_t e = lds_limit_once(flag, reinterpret_cast<const void*>(kern), int(lds));
    if (e != hipSuccess) return e;
    kern<<<blocks, 512, lds, s>>>(a);
    return hipGetLastError();
  };
  if (g.silu_mul)
    return g.y_dtype == 1 ? run(moe_w4a4_kernel<true, true>, done[0]) : run(moe_w4a4_kernel<true, false>, done[1]);
  return g.y_dtype == 1 ? run(moe_w4a4_kernel<false, true>, done[2]) : run(moe_w4a4_kernel<false, false>, done[3]);
}

}  // namespace qlin
