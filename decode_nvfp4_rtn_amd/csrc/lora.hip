// Low-rank adapters of many requests at once, beside a projection that all
// rows share:
//
//   out[t, :] = y[t, :] + scale_i B_i (A_i x_t),   i the adapter of row t
//
// with A_i [rank, k] and B_i [n, rank] in bf16.  Both products run over the
// runs of a plan, so that a tile of rows meets one adapter.
//
// Adapters of few rows and a low rank (a decode batch): one launch.  A block takes a tile of
// 16 places and a part of the columns; its waves share k, add their sums of
// u = A x in LDS in a fixed order, and make out = y + scale B u, each its own
// columns.  A and x are read once for each part of the columns.
//
// Other adapters (prompts): two launches.  "down" makes u: a block takes
// 64 places and a part of k, each wave 16 places and all of the rank; A passes
// through LDS, x goes from memory to registers.  u is stored in binary32, one
// buffer for each part of k.  "up" adds the parts in their order and makes out
// for 64 places and a part of the columns.
//
// u enters the second product as a sum of bf16 values, two beside a bf16 y (16
// bits of mantissa or more), three beside a binary32 one (all of it): that
// product is bound by reading y and writing out, so they cost nothing that shows.
//
// 64 tokens over 32 adapters of rank 16 beside 6144 x 4096: 9.2 us (10.5 with all of
// it from memory), one block's chain.  8190 tokens over 8 adapters of rank 64 beside 7168 x 5120: 28 us down (84
// MB of x at 3 TB/s) and 64 up (235 MB of y and out at 3.6 TB/s).
//
// Rows without an adapter come last in the plan: they are copied, or left
// alone where out is y.
#include "moe.hpp"
#include "decode_ops.hpp"

namespace qlin {
namespace {

__device__ __forceinline__ floatx4 mfma(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ u32x4 load16(const void* p) { return *static_cast<const u32x4*>(p); }

__device__ __forceinline__ int row_of(const RowPlan& p, int place) {
  return int(min(uint32_t(p.order[place]), uint32_t(p.rows - 1)));
}

// Eight binary32 values, each a sum of kTerms bf16 values: two keep 16 bits of
// the mantissa or more, three all of it.
template <int kTerms>
struct Split {
  bf16x8_t term[kTerms];
};
template <int kTerms>
__device__ __forceinline__ Split<kTerms> split(floatx4 a, floatx4 b) {
  Split<kTerms> s;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v = e < 4 ? a[e & 3] : b[e & 3];
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      s.term[t][e] = static_cast<__bf16>(v);
      v -= static_cast<float>(s.term[t][e]);
    }
  }
  return s;
}
constexpr int terms_of(bool bf16) { return bf16 ? 2 : 3; }

// Few rows: a step of 32 columns of the tile's rows, its y and the operand made
// of B.  The MFMA's rows are columns of out in an order that leaves each lane
// eight neighbours (lane quarter q: 8 q ..), so that y and out move in 16-byte
// pieces.  Columns past n and a rank past the last are clamped: the first are
// not stored, the second meet zeros of u.
template <int KT, bool kBF16>
struct Step {
  u32x4 b[2][KT];
  u32x4 y[kBF16 ? 1 : 2];
};

template <int KT, bool kBF16>
__device__ __forceinline__ void load_step(Step<KT, kBF16>& S, const LoraArgs& A, const uint16_t* b, int64_t y_at,
                                          int col0) {
  const int q = (threadIdx.x >> 4) & 3, r = threadIdx.x & 15;
  const uint8_t* p = static_cast<const uint8_t*>(A.y) + (y_at + min(col0 + 8 * q, A.n - 8)) * (kBF16 ? 2 : 4);
  S.y[0] = load16(p);
  if constexpr (!kBF16) S.y[1] = load16(p + 16);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t n = min(col0 + 8 * (r >> 2) + 4 * i + (r & 3), A.n - 1);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S.b[i][kt] = load16(b + n * A.rank + min(32 * kt + 8 * q, A.rank - 8));
  }
}

template <int KT, bool kBF16>
__device__ __forceinline__ void finish_step(const Step<KT, kBF16>& S, const LoraArgs& A, const Split<terms_of(kBF16)> (&u)[KT], float scale, int64_t out_at, int count, int col0) {
  const int q = (threadIdx.x >> 4) & 3, r = threadIdx.x & 15;
  floatx4 acc[2] = {floatx4{0.f, 0.f, 0.f, 0.f}, floatx4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < terms_of(kBF16); ++t) acc[i] = mfma(as_bf16x8(S.b[i][kt]), u[kt].term[t], acc[i]);
  const int col = col0 + 8 * q;
  if (col >= A.n || r >= count) return;   // n is a multiple of 16
  if constexpr (kBF16) {
    const u32x4 d = S.y[0];
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = pack_bf16x2(fmaf(scale, acc[e >> 1][2 * (e & 1)], __uint_as_float(d[e] << 16)),
                         fmaf(scale, acc[e >> 1][2 * (e & 1) + 1], __uint_as_float(d[e] & 0xFFFF0000u)));
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(A.out) + out_at + col) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      floatx4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fmaf(scale, acc[i][e], __uint_as_float(S.y[i][e]));
      *reinterpret_cast<floatx4*>(static_cast<float*>(A.out) + out_at + col + 4 * i) = o;
    }
  }
}

// Rows without an adapter: columns [c0, c1), copied by the block.
template <int kThreads, bool kBF16>
__device__ __forceinline__ void copy_rows(const LoraArgs& A, const RowTile& tile, int c0, int c1) {
  constexpr int size = kBF16 ? 2 : 4;
  const int per = (c1 - c0) * size / 16;
  for (int i = threadIdx.x; i < tile.count * per; i += kThreads) {
    const int64_t row = row_of(A.plan, tile.first + i / per), at = int64_t(c0) * size + i % per * 16;
    *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(A.out) + row * A.out_stride * size + at) =
        load16(static_cast<const uint8_t*>(A.y) + row * A.y_stride * size + at);
  }
}

// RT tiles of 16 of the rank (the last may be half), one m-tile of places.
template <int RT, bool kBF16>
__global__ __launch_bounds__(512) void lora_few_kernel(LoraArgs A, int col_parts) {
  constexpr int WAVES = 8, KT = (RT + 1) / 2;
  __shared__ union {
    __attribute__((aligned(16))) uint8_t stage[WAVES][4096];
    floatx4 red[WAVES][RT][64];   // the waves' sums
  } sm;
  __shared__ __attribute__((aligned(16))) float us[16][32 * KT + 4];   // u, zero past the rank
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.x % col_parts;
  const RowTile tile = find_tile(A.plan, 16, blockIdx.x / col_parts);
  if (tile.group < 0) return;
  const int steps = (A.n + 31) / 32;
  const int s0 = int(int64_t(steps) * part / col_parts), s1 = int(int64_t(steps) * (part + 1) / col_parts);
  if (tile.group == A.plan.groups) {
    if (A.out != A.y) copy_rows<512, kBF16>(A, tile, 32 * s0, min(32 * s1, A.n));
    return;
  }
  const int q = lane >> 4, r = lane & 15, G = A.k / 128;
  const int64_t row = row_of(A.plan, tile.first + min(r, tile.count - 1));
  // Rows of x and A are loaded whole (lane: row 4 i + q at k 8 r of a piece)
  // and become fragments in a wave-private LDS tile of 16 rows x 256 bytes: as
  // fragments straight from memory they cost the address unit two to four
  // times as much, and of x only the rows that there are would be wanted.
  const uint16_t* xr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    xr[i] = static_cast<const uint16_t*>(A.x) +
            row_of(A.plan, tile.first + min(4 * i + q, tile.count - 1)) * A.x_stride + 8 * r;
  const uint16_t* a = static_cast<const uint16_t*>(A.a) + int64_t(tile.group) * A.rank * A.k + 8 * r;
  struct Piece {
    u32x4 x[4], a[RT][4];
  };
  auto load = [&](Piece& P, int g) {   // past the end: the last piece again, not used
    g = min(g, G - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i == 0 || 4 * i < tile.count) P.x[i] = load16(xr[i] + g * 128);   // uniform
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) P.a[t][i] = load16(a + int64_t(min(16 * t + 4 * i + q, A.rank - 1)) * A.k + g * 128);
  };
  uint8_t* const stage = sm.stage[wave];
  auto slot = [](int row, int piece) { return row * 256 + 16 * (piece ^ row); };
  floatx4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Piece& P) {   // a wave's LDS operations stay in order
    u32x4 xf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i == 0 || 4 * i < tile.count) *reinterpret_cast<u32x4*>(stage + slot(4 * i + q, r)) = P.x[i];
#pragma unroll
    for (int s = 0; s < 4; ++s) xf[s] = load16(stage + slot(r, 4 * s + q));
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      __asm__ volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(stage + slot(4 * i + q, r)) = P.a[t][i];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        acc[t] = mfma(as_bf16x8(load16(stage + slot(r, 4 * s + q))), as_bf16x8(xf[s]), acc[t]);
    }
    __asm__ volatile("" ::: "memory");
  };
  Piece P, Q;
  load(P, wave);
  for (int g = wave; g < G; g += 2 * WAVES) {
    load(Q, g + WAVES);
    __builtin_amdgcn_sched_barrier(0);
    compute(P);
    load(P, g + 2 * WAVES);
    __builtin_amdgcn_sched_barrier(0);
    if (g + WAVES < G) compute(Q);
  }
  // the first step's y and B are under way while u is added up
  const uint16_t* b = static_cast<const uint16_t*>(A.b) + int64_t(tile.group) * A.n * A.rank;
  const int64_t y_at = row * A.y_stride, out_at = row * A.out_stride;
  Step<KT, kBF16> S;
  load_step<KT, kBF16>(S, A, b, y_at, 32 * min(s0 + wave, steps - 1));
  const float scale = A.scale ? A.scale[tile.group] : 1.0f;
  __syncthreads();   // the sums go where the rows were
#pragma unroll
  for (int i = 0; i < RT; ++i) sm.red[wave][i][lane] = acc[i];
  __syncthreads();
  for (int t = threadIdx.x; t < 2 * KT * 64; t += 512) {
    const int i = t / 64, ln = t % 64, j = 16 * i + 4 * (ln >> 4);
    floatx4 sum = floatx4{0.f, 0.f, 0.f, 0.f};
    if (j < A.rank) {   // the rank is a multiple of 8
      sum = sm.red[0][min(i, RT - 1)][ln];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum += sm.red[w][min(i, RT - 1)][ln];
    }
    *reinterpret_cast<floatx4*>(&us[ln & 15][j]) = sum;
  }
  __syncthreads();
  Split<terms_of(kBF16)> u[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
    u[kt] = split<terms_of(kBF16)>(*reinterpret_cast<const floatx4*>(&us[r][32 * kt + 8 * q]),
                  *reinterpret_cast<const floatx4*>(&us[r][32 * kt + 8 * q + 4]));
  for (int st = s0 + wave; st < s1; st += WAVES) {
    Step<KT, kBF16> next;
    load_step<KT, kBF16>(next, A, b, y_at, 32 * min(st + WAVES, steps - 1));
    finish_step<KT, kBF16>(S, A, u, scale, out_at, tile.count, 32 * st);
    S = next;
  }
}

constexpr int TALL = 64;

// the slot of row r's 16-byte piece c of 128 of k among a tile's 256: rows are
// XORed with the piece so that a row's pieces, written together, and a
// fragment's rows, read together, both fall on different banks
__device__ __forceinline__ int piece_slot(int r, int c) { return c * 16 + (r ^ c); }

template <int RT>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs A, int parts) {
  constexpr int BUF = RT * 4096;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];   // two pieces of A
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.x % parts;
  const RowTile tile = find_tile(A.plan, TALL, blockIdx.x / parts);
  if (tile.group < 0 || tile.group == A.plan.groups) return;
  const int q = lane >> 4, r = lane & 15;
  const int G = A.k / 128;
  const int g0 = int(int64_t(G) * part / parts), g1 = int(int64_t(G) * (part + 1) / parts);
  const bool busy = 16 * wave < tile.count;   // wave-uniform

  const uint16_t* xr = static_cast<const uint16_t*>(A.x) +
                       row_of(A.plan, tile.first + min(16 * wave + r, tile.count - 1)) * A.x_stride + 8 * q;
  // of a piece of A this thread moves one 16-byte piece of every 16th row
  const int ac = threadIdx.x & 15, an = threadIdx.x >> 4;
  const uint16_t* a = static_cast<const uint16_t*>(A.a) + int64_t(tile.group) * A.rank * A.k + 8 * ac;
  u32x4 av[RT];
  auto aload = [&](int g) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
      av[i] = load16(a + int64_t(min(16 * i + an, A.rank - 1)) * A.k + min(g, g1 - 1) * 128);
  };
  auto astore = [&](int buf) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *reinterpret_cast<u32x4*>(smem + buf * BUF + i * 4096 + piece_slot(an, ac) * 16) = av[i];
  };
  struct X {
    u32x4 v[4];
  };
  auto xload = [&](X& x, int g) {
#pragma unroll
    for (int s = 0; s < 4; ++s) x.v[s] = load16(xr + min(g, g1 - 1) * 128 + 32 * s);
  };
  int off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) off[s] = piece_slot(r, 4 * s + q) * 16;
  floatx4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const X& x, int buf) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < RT; ++i)
        acc[i] = mfma(as_bf16x8(load16(smem + buf * BUF + i * 4096 + off[s])), as_bf16x8(x.v[s]), acc[i]);
  };
  X P, Q;
  aload(g0);
  xload(P, g0);
  xload(Q, g0 + 1);
  __builtin_amdgcn_sched_barrier(0);
  astore(0);
  aload(g0 + 1);
  __syncthreads();
  // two pieces to a turn, so that buffers and registers have fixed places
  for (int g = g0; g < g1; g += 2) {
    astore(1);
    aload(g + 2);
    if (busy) compute(P, 0);
    xload(P, g + 2);
    __syncthreads();
    astore(0);
    aload(g + 3);
    if (busy && g + 1 < g1) compute(Q, 1);
    xload(Q, g + 3);
    __syncthreads();
  }
  const int place = 16 * wave + r;
  if (place < tile.count) {
    float* to = A.part + (int64_t(part) * A.plan.rows + tile.first + place) * A.rank;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (16 * i + 4 * q < A.rank) *reinterpret_cast<floatx4*>(to + 16 * i + 4 * q) = acc[i];
  }
}

// KT pieces of 32 of the rank.  The block's waves take 16 places each and share
// the columns, 64 at a time: B's rows of them, contiguous in memory, pass
// through LDS a step ahead (fragments loaded from memory, 64 bytes of each of 16
// rows, cost the address unit twice as much and took 11 us of the 85 that this
// product took of 8190 rows beside 7168 columns).  u stays in registers.  The
// sums pass through an LDS region of the wave's own, so that y and out move in
// whole lines, 128 bytes of 8 rows an instruction.
template <int KT, bool kBF16>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs A, int parts, int col_parts) {
  constexpr int NB = 4, WIDE = 16 * NB;                             // columns of a step
  constexpr int EPL = kBF16 ? 8 : 4;                                // a lane's columns
  constexpr int LPR = WIDE / EPL, RPI = 64 / LPR, ITS = 16 / RPI;   // lanes to a row, rows and instructions
  constexpr int BROW = 64 * KT + 16;                                // bytes of a row of B in LDS, at most
  __shared__ __attribute__((aligned(16))) uint8_t bs[2][WIDE * BROW];
  __shared__ __attribute__((aligned(16))) float st[4][16][WIDE + 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile tile = find_tile(A.plan, TALL, blockIdx.x / col_parts);
  if (tile.group < 0) return;
  const int part = blockIdx.x % col_parts, steps = (A.n + WIDE - 1) / WIDE;
  const int s0 = int(int64_t(steps) * part / col_parts), s1 = int(int64_t(steps) * (part + 1) / col_parts);
  if (tile.group == A.plan.groups) {
    if (A.out != A.y) copy_rows<256, kBF16>(A, tile, WIDE * s0, min(WIDE * s1, A.n));
    return;
  }
  const int q = lane >> 4, r = lane & 15;
  const int first = 16 * wave, count = tile.count - first;   // this wave's places of the tile
  const int lr = lane / LPR, lc = lane % LPR * EPL;          // this lane's row and first column of a piece
  int64_t y_at[ITS], out_at[ITS];
#pragma unroll
  for (int it = 0; it < ITS; ++it) {
    const int64_t row = row_of(A.plan, tile.first + min(first + RPI * it + lr, tile.count - 1));
    y_at[it] = row * A.y_stride * (kBF16 ? 2 : 4);
    out_at[it] = (row * A.out_stride + lc) * (kBF16 ? 2 : 4);
  }
  struct Y {
    u32x4 v[ITS];
  };
  auto yload = [&](Y& y, int step) {   // columns past n are clamped, and not stored
    const int col = min(step * WIDE + lc, A.n - EPL) * (kBF16 ? 2 : 4);
#pragma unroll
    for (int it = 0; it < ITS; ++it) y.v[it] = load16(static_cast<const uint8_t*>(A.y) + y_at[it] + col);
  };
  // B: pieces of 16 bytes, 8 rank of them a step; a rank past the last meets
  // zeros of u, so its place in LDS is clamped
  const uint8_t* b = static_cast<const uint8_t*>(A.b) + int64_t(tile.group) * A.n * A.rank * 2;
  const int pieces = 8 * A.rank, in_row = A.rank / 8, row_bytes = 2 * A.rank + 16;
  int b_to[KT];
#pragma unroll
  for (int i = 0; i < KT; ++i) {
    const int p = threadIdx.x + 256 * i;
    b_to[i] = p / in_row * row_bytes + p % in_row * 16;
  }
  u32x4 bq[KT];
  auto bload = [&](int step) {
    const int64_t end = int64_t(A.n) * A.rank * 2 - 16;
#pragma unroll
    for (int i = 0; i < KT; ++i)
      bq[i] = load16(b + min(int64_t(step) * pieces * 16 + (threadIdx.x + 256 * i) * 16, end));
  };
  auto bstore = [&](int buf) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
      if (int(threadIdx.x) + 256 * i < pieces) *reinterpret_cast<u32x4*>(bs[buf] + b_to[i]) = bq[i];
  };
  int b_at[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) b_at[kt] = r * row_bytes + 2 * min(32 * kt + 8 * q, A.rank - 8);

  Y P, Q;
  yload(P, s0);
  bload(s0);
  yload(Q, min(s0 + 1, steps - 1));
  // u of the wave's places: the parts of k in their order
  Split<terms_of(kBF16)> u[KT];
  {
    const int place = tile.first + min(first + r, tile.count - 1);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int j = 32 * kt + 8 * q;
      floatx4 v[2] = {floatx4{0.f, 0.f, 0.f, 0.f}, floatx4{0.f, 0.f, 0.f, 0.f}};
      if (j < A.rank) {
        const float* p = A.part + int64_t(place) * A.rank + j;
        for (int s = 0; s < parts; ++s, p += int64_t(A.plan.rows) * A.rank) {
          v[0] += *reinterpret_cast<const floatx4*>(p);
          v[1] += *reinterpret_cast<const floatx4*>(p + 4);
        }
      }
      u[kt] = split<terms_of(kBF16)>(v[0], v[1]);
    }
  }
  const float scale = A.scale ? A.scale[tile.group] : 1.0f;
  bstore(0);
  bload(min(s0 + 1, steps - 1));
  __syncthreads();

  auto work = [&](Y& y, int step, int buf) {
    floatx4 d[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) d[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (count > 0) {   // wave-uniform
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const bf16x8_t bf = as_bf16x8(load16(bs[buf] + 16 * i * row_bytes + b_at[kt]));
#pragma unroll
          for (int t = 0; t < terms_of(kBF16); ++t) d[i] = mfma(bf, u[kt].term[t], d[i]);
        }
    }
    bstore(buf ^ 1);   // read by nobody since the last barrier
    bload(min(step + 2, steps - 1));
    if (count > 0) {
      // a wave's LDS operations stay in order
#pragma unroll
      for (int i = 0; i < NB; ++i) *reinterpret_cast<floatx4*>(&st[wave][r][16 * i + 4 * q]) = d[i];
      __asm__ volatile("" ::: "memory");
      const int64_t col = int64_t(step) * WIDE * (kBF16 ? 2 : 4);
      const bool inside = step * WIDE + lc < A.n;
#pragma unroll
      for (int it = 0; it < ITS; ++it) {
        const u32x4 v = y.v[it];
        const floatx4 a0 = *reinterpret_cast<const floatx4*>(&st[wave][RPI * it + lr][lc]);
        u32x4 o;
        if constexpr (kBF16) {
          const floatx4 a1 = *reinterpret_cast<const floatx4*>(&st[wave][RPI * it + lr][lc + 4]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = pack_bf16x2(fmaf(scale, e < 2 ? a0[2 * e] : a1[2 * e - 4], __uint_as_float(v[e] << 16)),
                               fmaf(scale, e < 2 ? a0[2 * e + 1] : a1[2 * e - 3], __uint_as_float(v[e] & 0xFFFF0000u)));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(fmaf(scale, a0[e], __uint_as_float(v[e])));
        }
        if (inside && RPI * it + lr < count)
          *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(A.out) + out_at[it] + col) = o;
      }
      yload(y, min(step + 2, steps - 1));
    }
    __syncthreads();
  };
  for (int step = s0; step < s1; step += 2) {
    work(P, step, 0);
    if (step + 1 < s1) work(Q, step + 1, 1);
  }
}

int cus_or(int otherwise) {
  const int cus = device_cu_count();
  return cus > 0 ? cus : otherwise;
}

// Adapters of few rows, less than 48 on average over all that the call is given, met
// or not (how many are met only the device knows): one launch, which makes u again
// for each part of the columns.  Of long runs it reads A and B again for every 16
// rows: 8000 rows over 8 adapters of rank 16 beside 7168 x 5120 take 84 us where the
// call is given 200 adapters, and 72 - 74 in two launches where it is given up to 100.  It pays up to a rank of 32 (64 tokens over 32
// adapters of rank 16 beside 6144 x 4096: 9 us, in two launches 13; 18 tokens
// over 60 of rank 64: 20 and 15).
bool few_rows(int64_t rows, int64_t groups, int rank) { return rank <= 32 && rows < 48 * groups; }

// Parts of k of the first product: a block to a CU, at least 512 of k each.
int parts_of(int64_t rows, int64_t groups, int rank, int64_t k) {
  if (few_rows(rows, groups, rank)) return 0;
  const int64_t tiles = most_tiles(rows, groups, TALL);
  int64_t parts = (cus_or(256) + tiles - 1) / tiles;
  if (parts > k / 512) parts = k / 512;
  return parts < 1 ? 1 : int(parts);
}

// Parts of the columns: as many as give a CU `each` blocks, at least one step
// of `wide` columns for each of `waves` waves.
int col_parts_of(int64_t tiles, int64_t n, int each, int waves, int wide) {
  int64_t parts = each * cus_or(256) / tiles;
  const int64_t most = ((n + wide - 1) / wide + waves - 1) / waves;
  return int(parts < 1 ? 1 : parts < most ? parts : most);
}

template <int RT>
hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const bool bf16 = a.y_dtype == 1;
  if constexpr (RT <= 2) if (few_rows(a.plan.rows, a.plan.groups, a.rank)) {
    const int64_t tiles = most_tiles(a.plan.rows, a.plan.groups, 16);
    const int cols = col_parts_of(tiles, a.n, 1, 8, 32);
    if (bf16) lora_few_kernel<RT, true><<<unsigned(tiles * cols), 512, 0, s>>>(a, cols);
    else lora_few_kernel<RT, false><<<unsigned(tiles * cols), 512, 0, s>>>(a, cols);
    return hipGetLastError();
  }
  const int64_t tiles = most_tiles(a.plan.rows, a.plan.groups, TALL);
  const int parts = parts_of(a.plan.rows, a.plan.groups, a.rank, a.k);
  lora_down_kernel<RT><<<unsigned(tiles * parts), 256, 2 * RT * 4096, s>>>(a, parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int KT = (RT + 1) / 2;
  const int cols = col_parts_of(tiles, a.n, 8, 1, 256);
  if (bf16) lora_up_kernel<KT, true><<<unsigned(tiles * cols), 256, 0, s>>>(a, parts, cols);
  else lora_up_kernel<KT, false><<<unsigned(tiles * cols), 256, 0, s>>>(a, parts, cols);
  return hipGetLastError();
}

}  // namespace

size_t lora_ws_bytes(int64_t rows, int64_t groups, int rank, int64_t k) {
  return size_t(parts_of(rows, groups, rank, k)) * size_t(rows) * size_t(rank) * sizeof(float);
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t s) {
  if (a.rank <= 16) return launch_lora<1>(a, s);
  if (a.rank <= 32) return launch_lora<2>(a, s);
  if (a.rank <= 64) return launch_lora<4>(a, s);
  return launch_lora<8>(a, s);
}

}  // namespace qlin
