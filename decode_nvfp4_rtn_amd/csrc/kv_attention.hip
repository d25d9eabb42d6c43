// Attention of a sequence's newest tokens (one, a chain or a tree of drafts)
// over the paged, possibly quantized key/value cache: kv_attention
// (include/qlin.h).
//
// One block takes up to 16 MT query rows (a row: one new token and one of the
// n_q / n_kv query heads that share a kv head) of one sequence and kv head,
// and one chunk of its keys; its four waves take the chunk's 32-key tiles in
// turn.  A tile needs two products, computed transposed so that no operand
// moves between lanes:
//   S^T = K Q^T   A: 16 keys (lane % 16), 8 elements of d (lane / 16) per step
//   O^T += V^T P^T  A: 16 elements of d (lane % 16), 8 keys (lane / 16)
// S^T leaves lane (n, g) the scores of query row n and keys 4 g .. 4 g + 3 of
// each 16-key block.  The contraction index of the second product may run
// over keys in any order as long as both operands agree: with index 8 g + j
// standing for key 4 g + j % 4 of block j / 4, the probabilities already are
// the B operand, and the cache keeps V so that a lane's registers are the A
// operand (kv_cache.hpp).  Each row's statistics live in the four lanes of its
// column, the accumulator is rescaled in place.
//
// Quantized rows.  K's row scale 2^ke multiplies the row's score after the
// product.  V's, 2^ve, joins the exponent: with z the score in units of
// log 2 the weight that enters the product is 2^(z + ve - m), m a running
// maximum of z + ve, and the sum of weights takes 2^(z + ve - m) 2^-ve.  So the
// weights of the product are at most 2^8 however the rows' scales differ, and
// codes (and NVFP4 codes times their group scales, at most 6 significant
// bits) enter it exactly in fp16.  Queries are scaled by a power of two for
// each row to fit fp16.  The weights' rounding to fp16 (relative 2^-12) is
// below that of the bf16 result; a bf16 cache takes bf16 operands and its
// weights as the sum of two bf16 values (16 bits).
#include "kv_cache.hpp"

namespace qlin {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kTile = 32;               // keys per tile
constexpr float kLowest = -3.0e38f;     // running maximum before the first key
constexpr float kSlack = 8.0f;          // growth of the maximum that is let pass (weights <= 2^8)
constexpr float kLog2e = 1.44269504088896340736f;

template <int FMT>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (FMT == QL_KV_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Reductions over the four lanes of a column (16 apart).
__device__ __forceinline__ float column_max(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, int hi) {   // two E4M3 codes -> fp16
  const f16x2 v = hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(w), 1.0f, true)
                     : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(w), 1.0f, false);
  return __builtin_bit_cast(uint32_t, v);
}
template <int B>
__device__ __forceinline__ f16x2 fp4_pair(uint32_t w) {              // byte B's two E2M1 codes
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, B);
}
__device__ __forceinline__ uint32_t times(f16x2 a, f16x2 s) {        // exact: 2 x 4 bits
  return __builtin_bit_cast(uint32_t, a * s);
}

// The raw bytes of one 32-key tile that a lane holds: two 16-key blocks.
template <int FMT, int D>
struct Tile {
  using L = KvLayout<FMT, D>;
  static constexpr int W = L::kLoad / 4;      // words per load
  uint32_t k[2][L::kLoads * W], v[2][L::kLoads * W];
  uint32_t ks[2][L::kLoads], vs[2][L::kLoads];   // NVFP4 group scales
  uint32_t ke[2], ve[2];                         // row exponents of keys 4 g .. 4 g + 3

  __device__ __forceinline__ void load(int t, const uint8_t* codes, const uint8_t* scales, int lane) {
    auto words = [&](const uint8_t* p, uint32_t* w) {
      if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
      }
    };
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      words(codes + (64 * i + lane) * L::kLoad, &k[t][i * W]);
      words(codes + 16 * L::kRow + (64 * i + lane) * L::kLoad, &v[t][i * W]);
    }
    if constexpr (FMT == QL_KV_NVFP4) {
#pragma unroll
      for (int i = 0; i < L::kLoads; ++i) {
        const uint8_t* p = scales + (64 * i + lane) * L::kGPC;
        if constexpr (L::kGPC == 2) ks[t][i] = *reinterpret_cast<const uint16_t*>(p);
        else ks[t][i] = *p;
        const int group = i * L::kDC + (lane & 15) * L::kDC / 16;
        vs[t][i] = *reinterpret_cast<const uint32_t*>(scales + D + group * 16 + (lane >> 4) * 4);
      }
    }
    if constexpr (FMT != QL_KV_BF16) {
      const uint2 e = *reinterpret_cast<const uint2*>(scales + L::kExp + (lane >> 4) * 8);
      ke[t] = e.x, ve[t] = e.y;
    }
  }

  // K operand of block t, step s (elements d of a lane: see q_element).
  __device__ __forceinline__ u32x4 k_operand(int t, int s) const {
    u32x4 r;
    if constexpr (FMT == QL_KV_BF16) {
      for (int x = 0; x < 4; ++x) r[x] = k[t][4 * s + x];
    } else if constexpr (FMT == QL_KV_E4M3) {
      const uint32_t a = k[t][2 * s], b = k[t][2 * s + 1];
      r[0] = fp8_pair(a, 0), r[1] = fp8_pair(a, 1), r[2] = fp8_pair(b, 0), r[3] = fp8_pair(b, 1);
    } else {
      constexpr int per = L::kEC / 8;   // steps per load
      const f16x2 sc = __builtin_bit_cast(f16x2, fp8_pair(ks[t][s / per], 0));
      const _Float16 g = sc[s % per * 8 / 16];
      const uint32_t a = k[t][s];
      const f16x2 gg = {g, g};
      r[0] = times(fp4_pair<0>(a), gg), r[1] = times(fp4_pair<1>(a), gg);
      r[2] = times(fp4_pair<2>(a), gg), r[3] = times(fp4_pair<3>(a), gg);
    }
    return r;
  }

  // V operands of one load i: its kDC d-tiles, keys of both blocks.
  __device__ __forceinline__ void v_operands(int i, u32x4 (&r)[L::kDC]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (FMT == QL_KV_BF16) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          r[q][2 * t] = v[t][4 * i + 2 * q];
          r[q][2 * t + 1] = v[t][4 * i + 2 * q + 1];
        }
      } else if constexpr (FMT == QL_KV_E4M3) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          r[q][2 * t] = fp8_pair(v[t][4 * i + q], 0);
          r[q][2 * t + 1] = fp8_pair(v[t][4 * i + q], 1);
        }
      } else {
        const f16x2 lo = __builtin_bit_cast(f16x2, fp8_pair(vs[t][i], 0));
        const f16x2 hi = __builtin_bit_cast(f16x2, fp8_pair(vs[t][i], 1));
#pragma unroll
        for (int q = 0; q < W; ++q) {
          // bytes (key 0..3) of a pair of elements -> bytes of two keys each:
          // (d0: keys 0, 1), (d1: keys 0, 1), (d0: keys 2, 3), (d1: keys 2, 3)
          const uint32_t x = v[t][W * i + q];
          const uint32_t y = (x & 0xF00FF00Fu) | ((x << 4) & 0x0F000F00u) | ((x >> 4) & 0x00F000F0u);
          r[2 * q][2 * t] = times(fp4_pair<0>(y), lo);
          r[2 * q + 1][2 * t] = times(fp4_pair<1>(y), lo);
          r[2 * q][2 * t + 1] = times(fp4_pair<2>(y), hi);
          r[2 * q + 1][2 * t + 1] = times(fp4_pair<3>(y), hi);
        }
      }
    }
  }

  // Clears the V rows of block t's keys from `keys` (0..4 of this lane's
  // quad) on: what lies there is not part of the sequence.
  __device__ __forceinline__ void clear_v(int t, int keys) {
    if constexpr (FMT == QL_KV_BF16) {
      const uint32_t a = keys >= 2 ? ~0u : keys == 1 ? 0xFFFFu : 0u;
      const uint32_t b = keys >= 4 ? ~0u : keys == 3 ? 0xFFFFu : 0u;
#pragma unroll
      for (int x = 0; x < L::kLoads * W; ++x) v[t][x] &= x & 1 ? b : a;
    } else {
      const uint32_t m = keys >= 4 ? ~0u : (1u << (8 * keys)) - 1u;
#pragma unroll
      for (int x = 0; x < L::kLoads * W; ++x) v[t][x] &= m;
      if constexpr (FMT == QL_KV_NVFP4) {
#pragma unroll
        for (int i = 0; i < L::kLoads; ++i) vs[t][i] &= m;
      }
    }
  }
};

// Element of d that lane group g's operand element 0 of step s stands for.
template <int FMT, int D>
__device__ __forceinline__ int q_element(int s, int g) {
  constexpr int EC = KvLayout<FMT, D>::kEC, per = EC / 8;
  return (s / per * 4 + g) * EC + s % per * 8;
}

template <int FMT>
__device__ __forceinline__ bool non_finite(u32x4 v) {
  constexpr uint32_t e = FMT == QL_KV_BF16 ? 0x7F80u : 0x7C00u;
  bool r = false;
#pragma unroll
  for (int x = 0; x < 4; ++x) r |= (v[x] & e) == e || (v[x] >> 16 & e) == e;
  return r;
}

template <int FMT, int D, int MT>
struct State {
  static constexpr int KS = D / 32;     // steps of the first product
  static constexpr int DT = D / 16;     // d-tiles of the second
  u32x4 q[MT][KS];
  f32x4 o[MT][DT];
  float qs[MT];                         // scale * log2(e) * the row's power of two
  float m[MT], l[MT];
};

// Which keys a lane's row (column) sees in a masked tile, per m-tile.
struct RowMask {
  int last;          // chain: last visible position
  uint64_t bits;     // tree: visible new tokens
};

// One tile.  MASKED: some key of it is hidden from some row: `base` its first
// position, `n0`, `n1` how many of each block's 16 positions are there.
template <bool MASKED, int FMT, int D, int MT>
__device__ __forceinline__ void attend(State<FMT, D, MT>& st, Tile<FMT, D>& tile, int base, int n0,
                                       int n1, int ctx, bool tree, const RowMask (&rm)[MT],
                                       int lane) {
  using L = KvLayout<FMT, D>;
  constexpr int KS = State<FMT, D, MT>::KS;
  const int g = lane >> 4;
  f32x4 s[MT][2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) s[mt][t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const u32x4 a = tile.k_operand(t, k);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][t] = mma<FMT>(a, st.q[mt][k], s[mt][t]);
    }
  }

  // row scales of the lane's eight keys
  float kf[2][4], vb[2][4], iv[2][4];
  if constexpr (FMT != QL_KV_BF16) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t kb = tile.ke[t] >> (8 * r) & 0xFFu, b = tile.ve[t] >> (8 * r) & 0xFFu;
        kf[t][r] = __uint_as_float(kb << 23);
        vb[t][r] = static_cast<float>(b);
        iv[t][r] = __uint_as_float((254u - b) << 23);
      }
  }

  u32x4 p[MT], p_lo[MT];
  uint32_t seen[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float z[2][4];
    seen[mt] = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v;
        if constexpr (FMT == QL_KV_BF16) v = s[mt][t][r] * st.qs[mt];
        else v = __builtin_fmaf(s[mt][t][r] * kf[t][r], st.qs[mt], vb[t][r]);
        if constexpr (MASKED) {
          const int in = 4 * g + r, pos = base + 16 * t + in, node = pos - ctx;
          bool vis = in < (t ? n1 : n0);
          if (tree) vis = vis && (node < 0 || (node < 64 && (rm[mt].bits >> (node & 63) & 1)));
          else vis = vis && pos <= rm[mt].last;
          if (!vis) v = -__builtin_inff();
          seen[mt] |= vis ? 1u << (4 * t + r) : 0u;
        }
        z[t][r] = v;
      }
    float mx = z[0][0];
#pragma unroll
    for (int x = 1; x < 8; ++x) mx = __builtin_fmaxf(mx, z[x >> 2][x & 3]);
    mx = column_max(mx);
    if (__any(mx > st.m[mt] + kSlack)) {
      const float mn = __builtin_fmaxf(st.m[mt], mx);
      const float f = __builtin_amdgcn_exp2f(st.m[mt] - mn);
      st.m[mt] = mn;
      st.l[mt] *= f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) st.o[mt][d] *= f;
    }
    float w[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      w[x] = __builtin_amdgcn_exp2f(z[x >> 2][x & 3] - st.m[mt]);
      float add = w[x];
      if constexpr (FMT != QL_KV_BF16) {
        add *= iv[x >> 2][x & 3];
        if constexpr (MASKED) add = seen[mt] >> x & 1 ? add : 0.0f;   // iv may be anything there
      }
      st.l[mt] += add;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if constexpr (FMT == QL_KV_BF16) {
        p[mt][x] = pack_bf16x2(w[2 * x], w[2 * x + 1]);
        p_lo[mt][x] = pack_bf16x2(w[2 * x] - __uint_as_float(p[mt][x] << 16),
                                  w[2 * x + 1] - __uint_as_float(p[mt][x] & 0xFFFF0000u));
      } else {
        const f32x2 v = {w[2 * x], w[2 * x + 1]};
        p[mt][x] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
      }
    }
  }

  if constexpr (MASKED) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int left = (t ? n1 : n0) - 4 * g;
      tile.clear_v(t, left < 0 ? 0 : left > 4 ? 4 : left);
    }
  }
#pragma unroll
  for (int i = 0; i < L::kLoads; ++i) {
    u32x4 v[L::kDC];
    tile.v_operands(i, v);
#pragma unroll
    for (int q = 0; q < L::kDC; ++q) {
      const int d = i * L::kDC + q;
      if constexpr (MASKED) {
        if (__any(non_finite<FMT>(v[q]))) {
          // A zero weight does not hide a NaN or infinity in the product, so
          // the keys enter one by one, each only in the rows that see it.
          for (int x = 0; x < 32; ++x) {
            const int gk = x >> 3, j = x & 7;
            const uint32_t half = j & 1 ? 0xFFFF0000u : 0xFFFFu;
            u32x4 one, sel;
            for (int y = 0; y < 4; ++y) sel[y] = g == gk && y == j >> 1 ? half : 0u;
            one = v[q] & sel;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              f32x4 c = mma<FMT>(one, p[mt] & sel, st.o[mt][d]);
              if constexpr (FMT == QL_KV_BF16) c = mma<FMT>(one, p_lo[mt] & sel, c);
              const bool vis = __shfl(seen[mt], gk * 16 + (lane & 15), 64) >> j & 1;
#pragma unroll
              for (int y = 0; y < 4; ++y) st.o[mt][d][y] = vis ? c[y] : st.o[mt][d][y];
            }
          }
          continue;
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        st.o[mt][d] = mma<FMT>(v[q], p[mt], st.o[mt][d]);
        if constexpr (FMT == QL_KV_BF16) st.o[mt][d] = mma<FMT>(v[q], p_lo[mt], st.o[mt][d]);
      }
    }
  }
}

// Keys of one split of a sequence of `len` keys: the planned chunk, or more
// where the sequence is longer than the plan's splits cover.
__device__ __forceinline__ int chunk_of(int len, int chunk, int splits) {
  const int need = (len + splits - 1) / splits;
  return need <= chunk ? chunk : (need + 127) / 128 * 128;
}
// Splits that hold keys (at least one, so that every row is written).
__device__ __forceinline__ int splits_of(int len, int chunk) {
  return len > chunk ? (len + chunk - 1) / chunk : 1;
}

struct Seq {
  int q0, nodes, rows_q, len, ctx;   // rows_q: its queries that lie in q and y
};
__device__ __forceinline__ Seq sequence(const KvAttnArgs& a, int b) {
  Seq s;
  s.q0 = a.cu_q[b];
  s.nodes = a.cu_q[b + 1] - s.q0;
  const int64_t room = a.tokens - s.q0;
  s.rows_q = s.q0 < 0 || s.nodes < 0 || room <= 0 ? 0 : room < s.nodes ? int(room) : s.nodes;
  if (s.rows_q > a.max_q) s.rows_q = a.max_q;
  const int64_t cap = a.table_cols << a.g.page_shift;
  const int len = a.kv_lens[b];
  s.len = len < 0 ? 0 : len < cap ? len : int(cap);
  s.ctx = s.len > s.nodes ? s.len - s.nodes : 0;
  return s;
}

template <int FMT, int D, int MT>
__global__ __launch_bounds__(64 * kWaves) void kv_attention_kernel(KvAttnArgs a, int row_blocks) {
  using L = KvLayout<FMT, D>;
  constexpr int KS = D / 32, DT = D / 16;
  constexpr int DCH = D < 128 ? D : 128;        // elements of d merged at a time
  __shared__ float sm_m[kWaves][16 * MT], sm_l[kWaves][16 * MT];
  __shared__ __align__(16) float sm_o[kWaves][16][DCH + 4];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  const int rb = id % row_blocks;
  id /= row_blocks;
  const int split = id % a.splits;
  id /= a.splits;
  const int head = id % a.g.n_kv, b = id / a.g.n_kv;
  const int group = a.n_q / a.g.n_kv;
  const Seq sq = sequence(a, b);
  const int64_t rows = int64_t(sq.rows_q) * group, row0 = int64_t(rb) * (16 * MT);
  if (row0 >= rows) return;
  const int chunk = chunk_of(sq.len, a.chunk, a.splits), nsplit = splits_of(sq.len, chunk);
  if (split >= nsplit) return;
  const int k0 = split * chunk;
  int k1 = sq.len - k0 < chunk ? sq.len : k0 + chunk;
  if (!a.tree) {
    // no row of this block sees past its last token
    const int64_t last = (row0 + 16 * MT < rows ? row0 + 16 * MT : rows) - 1;
    const int64_t lim = int64_t(sq.ctx) + last / group + 1;
    if (lim < k1) k1 = int(lim);
  }

  State<FMT, D, MT> st;
  RowMask rm[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int64_t r = row0 + 16 * mt + n;
    const bool in = r < rows;
    const int node = in ? int(r / group) : 0;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + int64_t(sq.q0 + node) * a.q_stride +
                        int64_t(head * group + (in ? int(r % group) : 0)) * D;
    rm[mt].last = sq.ctx + node;
    rm[mt].bits = a.tree ? a.tree[sq.q0 + node] : 0;
    u32x4 w[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      w[s] = u32x4{0, 0, 0, 0};
      if (in) w[s] = *reinterpret_cast<const u32x4*>(q + q_element<FMT, D>(s, g));
    }
    st.qs[mt] = a.scale * kLog2e;
    if constexpr (FMT == QL_KV_BF16) {
#pragma unroll
      for (int s = 0; s < KS; ++s) st.q[mt][s] = w[s];
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(w[s][x] << 16)));
          amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(w[s][x] & 0xFFFF0000u)));
        }
      amax = column_max(amax);
      // the row's largest value goes to [2^14, 2^15)
      int e = int(__float_as_uint(amax) >> 23);
      e = e < 40 ? 40 : e > 254 ? 254 : e;
      const float down = __uint_as_float(uint32_t(254 + 14 - e) << 23);   // 2^(14 - (e - 127))
      st.qs[mt] *= __uint_as_float(uint32_t(e - 14) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const f32x2 v = {__uint_as_float(w[s][x] << 16) * down,
                           __uint_as_float(w[s][x] & 0xFFFF0000u) * down};
          st.q[mt][s][x] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
        }
    }
    st.m[mt] = kLowest;
    st.l[mt] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) st.o[mt][d] = f32x4{0, 0, 0, 0};
  }

  // tiles first, first + 4, ... of the split
  const int first = k0 / kTile + wave;
  const int tiles = (k1 + kTile - 1) / kTile;
  const int count = tiles > first ? (tiles - first + kWaves - 1) / kWaves : 0;
  const int per_page = a.g.page_shift - 4;             // log2(blocks of a page)
  const int32_t* table = a.table + int64_t(b) * a.table_stride;
  int pages = -1;   // of 32 iterations' two blocks, one per lane
  auto fetch_pages = [&](int it) {
    const int block = 2 * (first + kWaves * (it + (lane >> 1))) + (lane & 1);
    pages = -1;
    if (int64_t(block) * 16 < k1) {
      pages = table[block >> per_page];
      if (pages >= a.g.n_pages) pages = -1;
    }
  };
  auto load = [&](int it, Tile<FMT, D>& tile, int& p0, int& p1) {
    if ((it & 31) == 0) fetch_pages(it);
    const int block = 2 * (first + kWaves * it);
    p0 = __builtin_amdgcn_readlane(pages, 2 * (it & 31));
    p1 = __builtin_amdgcn_readlane(pages, 2 * (it & 31) + 1);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int page = t ? p1 : p0;
      const int64_t at = kv_block(a.g, page < 0 ? 0 : page, head, (block + t) & ((1 << per_page) - 1));
      tile.load(t, a.g.codes + at * L::kCodes, a.g.scales + at * L::kScales, lane);
    }
  };
  if (count > 0) {
    Tile<FMT, D> cur, nxt;
    int c0, c1, x0 = 0, x1 = 0;
    load(0, cur, c0, c1);
    for (int it = 0; it < count; ++it) {
      if (it + 1 < count) load(it + 1, nxt, x0, x1);
      const int base = (first + kWaves * it) * kTile;
      if (base + kTile > sq.ctx || base + kTile > k1 || (c0 | c1) < 0) {
        const int left = k1 - base;
        const int n0 = c0 < 0 ? 0 : left, n1 = c1 < 0 ? 0 : left - 16;
        attend<true, FMT, D, MT>(st, cur, base, n0, n1, sq.ctx, a.tree != nullptr, rm, lane);
      } else {
        attend<false, FMT, D, MT>(st, cur, base, 16, 16, sq.ctx, false, rm, lane);
      }
      cur = nxt;
      c0 = x0, c1 = x1;
    }
  }

  // the four waves' parts, in wave order
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    st.l[mt] = column_sum(st.l[mt]);
    if (g == 0) sm_m[wave][16 * mt + n] = st.m[mt], sm_l[wave][16 * mt + n] = st.l[mt];
  }
  __syncthreads();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float top = sm_m[0][16 * mt + n];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = __builtin_fmaxf(top, sm_m[w][16 * mt + n]);
    const float f = __builtin_amdgcn_exp2f(st.m[mt] - top);
#pragma unroll
    for (int part = 0; part < D / DCH; ++part) {
      // lane (n, g) holds, of each load i, the 4 kDC elements from
      // 16 kDC i + 4 kDC g on: element kDC r + q is row r of d-tile kDC i + q
#pragma unroll
      for (int i = 0; i < L::kLoads; ++i) {
        const int d0 = 16 * L::kDC * i;
        if (d0 / DCH != part) continue;
#pragma unroll
        for (int x = 0; x < 4 * L::kDC; x += 4) {
          f32x4 v;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            v[y] = st.o[mt][L::kDC * i + (x + y) % L::kDC][(x + y) / L::kDC] * f;
          *reinterpret_cast<f32x4*>(&sm_o[wave][n][d0 % DCH + 4 * L::kDC * g + x]) = v;
        }
      }
      __syncthreads();
      constexpr int kCols = DCH / 8;      // threads per row, 8 elements each
      const int row = threadIdx.x / kCols, c = threadIdx.x % kCols * 8;
      const int64_t r = row0 + 16 * mt + row;
      if (row < 16 && r < rows) {
        float tm = sm_m[0][16 * mt + row];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) tm = __builtin_fmaxf(tm, sm_m[w][16 * mt + row]);
        float l = 0.0f, v[8] = {};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          l += sm_l[w][16 * mt + row] * __builtin_amdgcn_exp2f(sm_m[w][16 * mt + row] - tm);
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] += sm_o[w][row][c + x];
        }
        const int64_t out = int64_t(sq.q0 + int(r / group)) * a.n_q + head * group + int(r % group);
        if (nsplit == 1) {
          uint32_t y[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            y[x] = l == 0.0f ? 0u : pack_bf16x2(v[2 * x] / l, v[2 * x + 1] / l);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + out * D + part * DCH + c) =
              make_uint4(y[0], y[1], y[2], y[3]);
        } else {
          const int64_t at = int64_t(split) * a.tokens * a.n_q + out;
          float4* o = reinterpret_cast<float4*>(a.part_o + at * D + part * DCH + c);
          o[0] = make_float4(v[0], v[1], v[2], v[3]);
          o[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (part == 0 && c == 0) a.part_ml[2 * at] = tm, a.part_ml[2 * at + 1] = l;
        }
      }
      __syncthreads();
    }
  }
}

// Joins the splits of every row that has more than one, in split order: a
// wave per row.
template <int D>
__global__ __launch_bounds__(64 * kWaves) void kv_attention_join_kernel(KvAttnArgs a) {
  constexpr int N = D / 64;
  const int lane = threadIdx.x & 63, b = blockIdx.y;
  const int64_t r = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);   // token of the sequence, head
  const Seq sq = sequence(a, b);
  if (r >= int64_t(sq.rows_q) * a.n_q) return;
  const int nsplit = splits_of(sq.len, chunk_of(sq.len, a.chunk, a.splits));
  if (nsplit == 1) return;
  const int64_t row = int64_t(sq.q0) * a.n_q + r, step = a.tokens * a.n_q;
  float top = kLowest;
  for (int s = 0; s < nsplit; ++s) top = __builtin_fmaxf(top, a.part_ml[2 * (s * step + row)]);
  float l = 0.0f, v[N] = {};
  for (int s = 0; s < nsplit; ++s) {
    const int64_t at = s * step + row;
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * at] - top);
    l += a.part_ml[2 * at + 1] * f;
#pragma unroll
    for (int x = 0; x < N; ++x) v[x] = __builtin_fmaf(a.part_o[at * D + lane * N + x], f, v[x]);
  }
  uint16_t* y = static_cast<uint16_t*>(a.y) + row * D + lane * N;
#pragma unroll
  for (int x = 0; x < N; ++x) y[x] = l == 0.0f ? uint16_t(0) : to_bf16(v[x] / l);
}

}  // namespace

KvAttnPlan kv_attention_plan(int fmt, int d, int n_q, int n_kv, int64_t n_seqs, int64_t max_q,
                             int64_t max_kv) {
  (void)fmt;
  KvAttnPlan p;
  const int64_t rows = max_q * (n_q / n_kv);
  const int most = d == 256 ? 2 : 4;
  p.mt = rows <= 16 ? 1 : rows <= 32 || most == 2 ? 2 : 4;
  p.row_blocks = (rows + 16 * p.mt - 1) / (16 * p.mt);
  // enough blocks for two on each compute unit, and at least 256 keys in one
  const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
  const int64_t blocks = n_seqs * n_kv * p.row_blocks;
  int64_t splits = (2 * cus + blocks - 1) / blocks;
  const int64_t most_splits = (max_kv + 255) / 256;
  if (splits > most_splits) splits = most_splits;
  if (splits < 1) splits = 1;
  if (splits > 256) splits = 256;
  const int64_t chunk = ((max_kv + splits - 1) / splits + 127) / 128 * 128;
  p.chunk = chunk > 128 ? int(chunk) : 128;
  p.splits = int((max_kv + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  return p;
}

size_t kv_attention_ws_bytes(const KvAttnPlan& p, int64_t tokens, int n_q, int d) {
  if (p.splits < 2) return 0;
  return size_t(p.splits) * size_t(tokens) * size_t(n_q) * size_t(d + 2) * sizeof(float);
}

hipError_t launch_kv_attention(int fmt, int d, const KvAttnPlan& p, KvAttnArgs a, hipStream_t s) {
  const int64_t blocks = int64_t(a.n_seqs) * a.g.n_kv * p.row_blocks * p.splits;
  const hipError_t e = kv_dispatch(fmt, d, [&](auto f, auto n) {
    constexpr int FMT = decltype(f)::value, D = decltype(n)::value;
    const dim3 grid(static_cast<unsigned>(blocks));
    const int rb = int(p.row_blocks);
    if (p.mt == 1) {
      kv_attention_kernel<FMT, D, 1><<<grid, 64 * kWaves, 0, s>>>(a, rb);
    } else if (p.mt == 2) {
      kv_attention_kernel<FMT, D, 2><<<grid, 64 * kWaves, 0, s>>>(a, rb);
    } else if constexpr (D != 256) {
      kv_attention_kernel<FMT, D, 4><<<grid, 64 * kWaves, 0, s>>>(a, rb);
    }
    return hipGetLastError();
  });
  if (e != hipSuccess || p.splits < 2) return e;
  const dim3 grid(unsigned((int64_t(a.max_q) * a.n_q + kWaves - 1) / kWaves), unsigned(a.n_seqs));
  switch (d) {
    case 64: kv_attention_join_kernel<64><<<grid, 64 * kWaves, 0, s>>>(a); break;
    case 128: kv_attention_join_kernel<128><<<grid, 64 * kWaves, 0, s>>>(a); break;
    default: kv_attention_join_kernel<256><<<grid, 64 * kWaves, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace qlin
