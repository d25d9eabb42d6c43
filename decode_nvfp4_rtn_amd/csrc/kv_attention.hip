// Attention of a sequence's newest tokens (one, a chain or a tree of drafts)
// over the paged, possibly quantized key/value cache: kv_attention
// (include/qlin.h).
//
// A row is one new token and one of the n_q / n_kv query heads that share a
// kv head.  A block takes some rows of one sequence and kv head and one part of
// its keys, 32 at a time, with the running maximum and sum of a softmax.
// Both products of such a tile run transposed, so that no operand moves
// between lanes:
//   S^T = K Q^T     A: 16 keys (lane % 16), 8 elements of d (lane / 16) a step
//   O^T += V^T P^T  A: 16 elements of d (lane % 16), 8 keys (lane / 16)
// S^T leaves lane (n, g) the scores of query row n and keys 4 g .. 4 g + 3 of
// each 16-key block.  The contraction index of the second product may run
// over the keys in any order as long as both operands agree: with index
// 8 g + j standing for key 4 g + j % 4 of block j / 4, the weights already are
// the B operand, and the cache keeps V so that a lane's registers are the A
// operand (kv_cache.hpp).  A row's statistics live in the four lanes of its
// column, and the accumulator is rescaled in place.
//
// Three kernels share this.
// narrow (up to 16 rows): each of four waves takes tiles of its own straight
//   from memory into registers and the four results are joined at the end;
//   bound by the cache's bytes (32 sequences of 2048 to 8192 keys, 32 / 8
//   128-wide heads, with the join: bf16 130 us, 685 MB at 5.3 TB/s; 8-bit
//   71 us, 4.9 TB/s), at 4 bits by each wave's chain of loads, unpacking,
//   products and softmax (52 us, 195 MB at 3.8 TB/s; the vector unit issues in
//   46 % of the cycles).
// pair (more rows, 64- and 128-wide heads): as narrow with 32 rows, so that a
//   tile's operands serve two products each; bound by the chain of a tile as
//   well (16 sequences of 63 drafts over up to 2000 8-bit 128-wide keys, 32 / 8
//   heads: 53 us; a prompt's 4096 tokens over 8-bit keys 246 us, bf16 255, of 110
//   for the operations).
// wide (256-wide heads, whose 32 rows do not fit the registers, and mostly more
//   than 32 rows over 4-bit 128-wide keys, whose unpacking counts for more): four
//   waves share each tile.  Each turns a quarter of it into matrix operands in
//   LDS, once for all, and takes 16 rows of its own; bound by what a tile takes
//   a wave from barrier to barrier: operands made and stored, LDS reads,
//   products, softmax (4 sequences of 6893 to 16063 4-bit 256-wide keys, 63
//   drafts, 15 / 5 heads: 109 us with the join, 47 GFLOP; a prompt's 4096 tokens
//   over 4-bit 128-wide keys 278 us).  A wave issues 44 % of that time; when the
//   trees took 107 us, they took 76 without the operands' making and storing, 101
//   without LDS reads, 99 without the softmax.
//
// Quantized rows.  K's row scale 2^ke goes into the bf16 operand where that
// is free (narrow, NVFP4: it multiplies the score).  V's, 2^ve, joins the
// exponent: with z the score in units of log 2 the weight that enters the
// product is w = 2^(z + ve - m), m + 7 a running maximum of z + ve, and the
// sum of weights takes w 2^-ve.  So the weights are at most 2^15 however the
// rows' scales differ, and V's codes (NVFP4: times their group scales, at most
// 6 significant bits) enter in fp16 exactly.  The weights' rounding to fp16
// (relative 2^-12, and of weights below 2^-21 of the largest a multiple of at
// most 2^-31 of it) is below that of the bf16 result.  A bf16 cache takes bf16
// operands and its weights as the sum of two bf16 values (16 bits), because
// one of 8 bits would add as much error as the rounding of the result.
#include "kv_cache.hpp"

namespace qlin {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kTile = 32;               // keys per tile
constexpr float kLowest = -3.0e38f;     // running maximum before the first key
// Weights are 2^(z - m).  The largest is 2^kUp when m is set, and m is set anew
// when one would pass 2^kMost: fp16 ends at 2^16, and the further up the
// weights are the fewer fall below its normal range.
constexpr float kUp = 7.0f, kMost = 15.0f;
// The sum of weights of quantized rows is kept times 2^-7: 2^-ve reaches 2^100.
constexpr float kUnit = 1.0f / 128;
constexpr float kLog2e = 1.44269504088896340736f;

template <bool HALF>   // fp16 operands, or bf16
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
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
// two E4M3 codes times a power of two -> bf16
__device__ __forceinline__ uint32_t fp8_pair_bf16(uint32_t w, float p, int hi) {
  const bf16x2 v = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(w), p, true)
                      : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(w), p, false);
  return __builtin_bit_cast(uint32_t, v);
}
template <int B>
__device__ __forceinline__ f16x2 fp4_pair(uint32_t w) {              // byte B's two E2M1 codes
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, B);
}
__device__ __forceinline__ uint32_t times(f16x2 a, f16x2 s) {        // exact: 2 x 4 bits
  return __builtin_bit_cast(uint32_t, a * s);
}
// byte B's two E2M1 codes times a power of two and a group scale -> bf16
template <int B>
__device__ __forceinline__ uint32_t fp4_pair_bf16(uint32_t w, float p, float s) {
  const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, p, B);
  return pack_bf16x2(v[0] * s, v[1] * s);
}
__device__ __forceinline__ float power(uint32_t b) {                 // 2^(b - 127)
  return __uint_as_float(b << 23);
}

// Top bit of each half / byte that is a bf16 infinity or NaN / an E4M3 NaN.
__device__ __forceinline__ uint32_t bad_halves(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t bad_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
// In the upper two bits of each byte: not 0 where the row exponent lies outside
// of [64, 127], that is of 2^-63 .. 1.
__device__ __forceinline__ uint32_t far_bits(uint32_t w) { return w ^ 0x40404040u; }
// 0xFF in byte k for bit k.
__device__ __forceinline__ uint32_t byte_mask(uint32_t bits) {
  return ((bits & 15u) * 0x00204081u & 0x01010101u) * 0xFFu;
}
template <int CTRL>
__device__ __forceinline__ uint32_t row_or(uint32_t v) {   // another lane of the same 16
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xF, 0xF, true));
}

// A block's codes and scales as buffer resources: the base is uniform, so a
// lane's address is one 32-bit offset.
struct Source {
  __amdgpu_buffer_rsrc_t codes, scales;
};
template <int FMT, int D>
__device__ __forceinline__ Source source(const KvGeom& g, int64_t block) {
  using L = KvLayout<FMT, D>;
  constexpr int kWord3 = 0x00020000;      // raw buffer
  Source s;
  s.codes = __builtin_amdgcn_make_buffer_rsrc(g.codes + block * L::kCodes, 0, L::kCodes, kWord3);
  s.scales = __builtin_amdgcn_make_buffer_rsrc(g.scales + block * L::kScales, 0, L::kScales, kWord3);
  return s;
}
__device__ __forceinline__ uint32_t load32(__amdgpu_buffer_rsrc_t r, int at) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
}

// One block's (16 keys') K or V bytes that a lane holds.
template <int FMT, int D>
struct Block {
  using L = KvLayout<FMT, D>;
  static constexpr int W = L::kLoad / 4;      // words per load
  typedef uint32_t Words __attribute__((ext_vector_type(W)));
  Words w[L::kLoads];
  uint32_t sc[L::kLoads];                     // NVFP4 group scales (K: of the lane's key, V: of its quad)

  __device__ __forceinline__ Words words(const Source& s, int at) {
    if constexpr (W == 4) return __builtin_amdgcn_raw_buffer_load_b128(s.codes, at, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b64(s.codes, at, 0, 0);
  }
  __device__ __forceinline__ void load_k(const Source& s, int lane) {
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      w[i] = words(s, lane * L::kLoad + 64 * i * L::kLoad);
      if constexpr (FMT == QL_KV_NVFP4) {
        // whole words: a narrower load's result is extended at once, and waited for
        sc[i] = load32(s.scales, (lane * L::kGPC & ~3) + 64 * i * L::kGPC);
      }
    }
  }
  __device__ __forceinline__ void load_v(const Source& s, int lane) {
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      w[i] = words(s, lane * L::kLoad + (16 * L::kRow + 64 * i * L::kLoad));
      if constexpr (FMT == QL_KV_NVFP4)      // group i kDC + (lane % 16) kDC / 16
        sc[i] = load32(s.scales, (lane & 15) * L::kDC / 16 * 16 + (lane >> 4) * 4 +
                                     (D + i * L::kDC * 16));
    }
  }
  // K operand of step s (its elements of d: q_element), bf16 with the row
  // scale p; HALF (NVFP4): fp16 without it.
  template <bool HALF>
  __device__ __forceinline__ u32x4 k_operand(int s, float p, int lane) const {
    constexpr int per = L::kEC / 8;           // steps per load
    if constexpr (FMT == QL_KV_BF16) {
      return w[s];
    } else if constexpr (FMT == QL_KV_E4M3) {
      const uint32_t a = w[s / per][s % per * 2], b = w[s / per][s % per * 2 + 1];
      return u32x4{fp8_pair_bf16(a, p, 0), fp8_pair_bf16(a, p, 1), fp8_pair_bf16(b, p, 0),
                   fp8_pair_bf16(b, p, 1)};
    } else {
      const uint32_t a = w[s / per][s % per];
      const uint32_t groups = sc[s / per] >> 8 * (lane * L::kGPC & 3);
      if constexpr (HALF) {
        const f16x2 two = __builtin_bit_cast(f16x2, fp8_pair(groups, 0));
        const _Float16 g = two[s % per / 2];
        const f16x2 gg = {g, g};
        return u32x4{times(fp4_pair<0>(a), gg), times(fp4_pair<1>(a), gg),
                     times(fp4_pair<2>(a), gg), times(fp4_pair<3>(a), gg)};
      } else {
        const float g = s % per / 2 ? __builtin_amdgcn_cvt_f32_fp8(int(groups), 1)
                                    : __builtin_amdgcn_cvt_f32_fp8(int(groups), 0);
        return u32x4{fp4_pair_bf16<0>(a, p, g), fp4_pair_bf16<1>(a, p, g),
                     fp4_pair_bf16<2>(a, p, g), fp4_pair_bf16<3>(a, p, g)};
      }
    }
  }

  // This block's half (4 of a lane's 8 keys) of the V operands of kPer d-tiles
  // from kPer j on: bf16 values, or fp16 codes (NVFP4: times group scales).
  static constexpr int kPer = FMT == QL_KV_E4M3 ? 1 : 2;
  __device__ __forceinline__ void v_operands(int j, uint2 (&r)[kPer]) const {
    constexpr int per = L::kDC / kPer;        // such pieces of a load
    const int i = j / per, q = j % per;
    if constexpr (FMT == QL_KV_BF16) {
      r[0] = make_uint2(w[i][0], w[i][1]);
      r[1] = make_uint2(w[i][2], w[i][3]);
    } else if constexpr (FMT == QL_KV_E4M3) {
      r[0] = make_uint2(fp8_pair(w[i][q], 0), fp8_pair(w[i][q], 1));
    } else {
      const f16x2 lo = __builtin_bit_cast(f16x2, fp8_pair(sc[i], 0));
      const f16x2 hi = __builtin_bit_cast(f16x2, fp8_pair(sc[i], 1));
      // bytes (key 0..3) of a pair of elements -> bytes of two keys each:
      // (d0: keys 0, 1), (d1: keys 0, 1), (d0: keys 2, 3), (d1: keys 2, 3)
      const uint32_t x = w[i][q];
      uint32_t y = (x & ~0x0F000F00u) | ((x << 4) & 0x0F000F00u);
      y = (y & ~0x00F000F0u) | ((x >> 4) & 0x00F000F0u);
      r[0] = make_uint2(times(fp4_pair<0>(y), lo), times(fp4_pair<2>(y), hi));
      r[1] = make_uint2(times(fp4_pair<1>(y), lo), times(fp4_pair<3>(y), hi));
    }
  }

  // V: clears the keys of the lane's quad from `keys` (0..4) on; what lies
  // there is not part of the sequence.
  __device__ __forceinline__ void clear_v(int keys) {
    if constexpr (FMT == QL_KV_BF16) {
      const uint32_t a = keys >= 2 ? ~0u : keys == 1 ? 0xFFFFu : 0u;
      const uint32_t b = keys >= 4 ? ~0u : keys == 3 ? 0xFFFFu : 0u;
#pragma unroll
      for (int x = 0; x < L::kLoads * W; ++x) w[x / W][x % W] &= x & 1 ? b : a;
    } else {
      const uint32_t m = keys >= 4 ? ~0u : (1u << (8 * keys)) - 1u;
#pragma unroll
      for (int i = 0; i < L::kLoads; ++i) {
        w[i] &= m;
        if constexpr (FMT == QL_KV_NVFP4) sc[i] &= m;
      }
    }
  }

  // V: non-zero where a value that the lane holds is a NaN or an infinity.
  __device__ __forceinline__ uint32_t non_finite() const {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      if constexpr (FMT == QL_KV_NVFP4) {
        r |= bad_bytes(sc[i]);
      } else {
#pragma unroll
        for (int x = 0; x < W; ++x) r |= FMT == QL_KV_BF16 ? bad_halves(w[i][x]) : bad_bytes(w[i][x]);
      }
    }
    return r;
  }
  // V: clears them (NVFP4: their groups); bit k of the result: key k of the
  // lane's quad had one, in an element of any of the 16 lanes that hold it.
  __device__ __forceinline__ uint32_t clear_non_finite() {
    uint32_t b = 0, c = 0, r;     // BF16: keys 0, 1 and keys 2, 3; others: b, a byte a key
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      if constexpr (FMT == QL_KV_NVFP4) {
        const uint32_t m = bad_bytes(sc[i]);
        b |= m;
        sc[i] &= ~((m >> 7) * 0xFFu);
      } else {
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const uint32_t m = FMT == QL_KV_BF16 ? bad_halves(w[i][x]) : bad_bytes(w[i][x]);
          if (FMT == QL_KV_BF16 && (x & 1)) c |= m;
          else b |= m;
          w[i][x] &= FMT == QL_KV_BF16 ? ~((m >> 15) * 0xFFFFu) : ~((m >> 7) * 0xFFu);
        }
      }
    }
    if constexpr (FMT == QL_KV_BF16)
      r = (b >> 15 & 1u) | (b >> 30 & 2u) | (c >> 13 & 4u) | (c >> 28 & 8u);
    else
      r = (b >> 7 & 1u) | (b >> 14 & 2u) | (b >> 21 & 4u) | (b >> 28 & 8u);
    r |= row_or<0xB1>(r);
    r |= row_or<0x4E>(r);
    r |= row_or<0x141>(r);
    r |= row_or<0x140>(r);
    return r;
  }
};

// Element of d that lane group g's operand element 0 of step s stands for.
template <int FMT, int D>
__device__ __forceinline__ int q_element(int s, int g) {
  constexpr int EC = KvLayout<FMT, D>::kEC, per = EC / 8;
  return (s / per * 4 + g) * EC + s % per * 8;
}

// ---------------------------------------------------------------------------
// Sequences, rows, splits
// ---------------------------------------------------------------------------
// Keys of sequence b that its row of the table reaches.
__device__ __forceinline__ int length(const KvAttnArgs& a, int b) {
  const int64_t cap = a.table_cols << a.g.page_shift;
  const int len = a.kv_lens[b];
  return len < 0 ? 0 : len < cap ? len : int(cap);
}

struct Seq {
  int q0, rows_q;   // rows_q: its queries that lie in q and y
  int len;          // its keys, as far as the table goes
  int ctx;          // of all its keys, those before the new tokens' (may pass len)
};
__device__ __forceinline__ Seq sequence(const KvAttnArgs& a, int b) {
  Seq s;
  s.q0 = a.cu_q[b];
  const int nodes = a.cu_q[b + 1] - s.q0;
  const int64_t room = a.tokens - s.q0;
  s.rows_q = s.q0 < 0 || nodes < 0 || room <= 0 ? 0 : room < nodes ? int(room) : nodes;
  if (s.rows_q > a.max_q) s.rows_q = a.max_q;
  s.len = length(a, b);
  const int all = a.kv_lens[b] > 0 ? a.kv_lens[b] : 0;
  s.ctx = nodes < 0 ? all : all > nodes ? all - nodes : 0;
  return s;
}

// Sum over the wave, in every lane.
__device__ __forceinline__ uint32_t wave_sum(uint32_t v) {
  v += row_or<0xB1>(v);
  v += row_or<0x4E>(v);
  v += row_or<0x141>(v);
  v += row_or<0x140>(v);
  auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = r[0] + r[1];
  r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return r[0] + r[1];
}

// The keys of all sequences are cut into at most a.parts parts, every sequence
// into pieces of one length, which is the shortest (nearly) that does: so the
// parts are even however uneven the sequences are, and the grid, which is
// planned without the lengths, is full.  (Against parts planned by the longest
// sequence alone: 32 sequences of 2260 to 8193 4-bit keys 51 us for 56, 16 of
// up to 8192 8-bit 256-wide ones 40 for 49.)
struct Part {
  int b, split, nsplit, keys;    // sequence (none if < 0), place in it, its parts, keys of one
};
// Part u; every wave works it out alone, with a sequence to a lane.
__device__ __forceinline__ Part part_of(const KvAttnArgs& a, int u) {
  if (a.parts == a.n_seqs) return {u, 0, 1, 0x7FFFFFFF};
  const int lane = threadIdx.x & 63;
  // in steps of 128 keys
  auto steps_of = [&](int b) { return b < a.n_seqs ? (uint32_t(length(a, b)) + 127) >> 7 : 0u; };
  const uint32_t mine = steps_of(lane);
  uint64_t total = wave_sum(mine);
  for (int b = 64; b < a.n_seqs; b += 64) total += wave_sum(steps_of(b + lane));
  // parts that a sequence of w steps needs at c steps each: one at least, so
  // that every row is written
  auto need = [&](uint32_t w, uint32_t c) { return w > c ? (w + c - 1) / c : 1u; };
  auto fits = [&](uint32_t c) {
    uint32_t n = lane < a.n_seqs ? need(mine, c) : 0u;
    for (int b = 64 + lane; b < a.n_seqs; b += 64) n += need(steps_of(b), c);
    return __builtin_amdgcn_readfirstlane(wave_sum(n)) <= uint32_t(a.parts);
  };
  // between the mean part and what surely fits; 256 keys at least
  const uint32_t spare = uint32_t(a.parts - a.n_seqs);
  uint64_t least = (total + a.parts - 1) / uint32_t(a.parts), most = (total + spare - 1) / spare;
  uint32_t lo = least < 2 ? 2u : uint32_t(least), hi = most > 1u << 24 ? 1u << 24 : uint32_t(most);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi < lo ? lo : hi);
  if (fits(lo)) hi = lo;
  for (int i = 0; i < 6 && lo < hi; ++i) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (fits(mid)) hi = mid;
    else lo = mid + 1;
  }
  Part p = {-1, 0, 1, hi >> 24 ? 0x7FFFFFFF : int(hi) << 7};
  uint32_t before = 0;
  for (int b0 = 0; b0 < a.n_seqs; b0 += 64) {
    const uint32_t n = b0 + lane < a.n_seqs ? need(b0 ? steps_of(b0 + lane) : mine, hi) : 0u;
    uint32_t upto = n;
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
      const uint32_t v = __shfl_up(upto, off, 64);
      if (lane >= off) upto += v;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 64 && b0 + lane < a.n_seqs) {
      a.first[b0 + lane] = int(before + upto - n);
      if (b0 + lane == a.n_seqs - 1) a.first[a.n_seqs] = int(before + upto);
    }
    const int ahead = __popcll(__ballot(before + upto <= uint32_t(u)));   // lanes whose parts come first
    if (p.b < 0 && ahead < 64 && b0 + ahead < a.n_seqs) {
      p.b = b0 + ahead;
      p.nsplit = __builtin_amdgcn_readlane(n, ahead);
      p.split = u - int(before + __builtin_amdgcn_readlane(upto, ahead) - p.nsplit);
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return p;
}

// What a thread block works on.
struct Work {
  Seq sq;
  int part, head, split, nsplit, group;
  int b;
  int rows, row0;
  int k0, k1;            // its keys
  bool any;
};
// Row blocks of one unit (split, sequence, head) read the same keys: their ids
// are 8 apart, so that they run on one XCD and share its L2.  Heads come
// fastest, so that what is not used at the end spreads over all XCDs.
template <int ROWS>
__device__ __forceinline__ Work work_of(const KvAttnArgs& a) {
  Work w;
  const uint32_t id = blockIdx.y * gridDim.x + blockIdx.x;
  const int slot = int(id >> 3);
  int unit = slot / a.row_blocks * 8 + int(id & 7);
  w.row0 = slot % a.row_blocks * ROWS;
  w.any = unit < a.units;
  if (!w.any) return w;
  w.head = unit % a.g.n_kv;
  w.part = unit / a.g.n_kv;
  const Part p = part_of(a, w.part);
  w.any = p.b >= 0;
  if (!w.any) return w;
  w.b = p.b, w.split = p.split, w.nsplit = p.nsplit;
  w.group = a.n_q / a.g.n_kv;
  w.sq = sequence(a, w.b);
  w.rows = w.sq.rows_q * w.group;
  w.any = w.row0 < w.rows;
  w.k0 = w.split * p.keys;
  w.k1 = w.sq.len - w.k0 < p.keys ? w.sq.len : w.k0 + p.keys;
  if (!a.tree) {
    // of a chain, no row sees past the block's last token
    const int last = (w.row0 + ROWS < w.rows ? w.row0 + ROWS : w.rows) - 1;
    const int lim = w.sq.ctx + last / w.group + 1;
    if (lim < w.k1) w.k1 = lim;
  }
  return w;
}
// Tiles that hold `keys` keys (up to 2^31 - 16 of them).
__device__ __forceinline__ int tiles_of(int keys) { return int((uint32_t(keys) + kTile - 1) / kTile); }
// Positions that every row from `row0` on sees.
__device__ __forceinline__ int open_to(const KvAttnArgs& a, const Work& w, int row0) {
  const int o = a.tree ? w.sq.ctx : w.sq.ctx + row0 / w.group + 1;
  return o < w.k1 ? o : w.k1;
}

// Which new tokens a row sees.
struct RowMask {
  int last;          // chain: last visible position
  uint64_t bits;     // tree: visible new tokens
};
// Bit 4 t + r: the row sees key 4 g + r of block t of the tile at `base`.
__device__ __forceinline__ uint32_t visible(const RowMask& rm, bool tree, int base, int ctx, int g) {
  uint32_t seen = 0;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int pos = base + 16 * (x >> 2) + 4 * g + (x & 3), node = pos - ctx;
    const bool vis = tree ? node < 0 || (node < 64 && (rm.bits >> (node & 63) & 1)) : pos <= rm.last;
    seen |= vis ? 1u << x : 0u;
  }
  return seen;
}

// A row's query operands; HALF: scaled by a power of two to fit fp16.
template <int FMT, int D, bool HALF>
__device__ __forceinline__ void load_query(const KvAttnArgs& a, const Work& w, int row, int g,
                                           u32x4 (&q)[D / 32], float& qs, RowMask& rm) {
  constexpr int KS = D / 32;
  const bool in = row < w.rows;
  const int node = in ? row / w.group : 0, sub = in ? row - node * w.group : 0;
  const uint16_t* p = static_cast<const uint16_t*>(a.q) + int64_t(w.sq.q0 + node) * a.q_stride +
                      int64_t(w.head * w.group + sub) * D;
  rm.last = w.sq.ctx + node;
  rm.bits = a.tree ? a.tree[w.sq.q0 + node] : 0;
  qs = a.scale * kLog2e;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    q[s] = u32x4{0, 0, 0, 0};
    if (in) q[s] = *reinterpret_cast<const u32x4*>(p + q_element<FMT, D>(s, g));
  }
  if constexpr (HALF) {
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(q[s][x] << 16)));
        amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(q[s][x] & 0xFFFF0000u)));
      }
    amax = column_max(amax);
    // the row's largest value goes to [2^14, 2^15)
    int e = int(__float_as_uint(amax) >> 23);
    e = e < 40 ? 40 : e > 254 ? 254 : e;
    const float down = power(254 + 14 - e);               // 2^(14 - (e - 127))
    qs *= power(e - 14);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const f32x2 v = {__uint_as_float(q[s][x] << 16) * down,
                         __uint_as_float(q[s][x] & 0xFFFF0000u) * down};
        q[s][x] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
      }
  }
}

// ---------------------------------------------------------------------------
// One row tile's softmax step over a tile of keys
// ---------------------------------------------------------------------------
template <int D>
struct Rows {
  f32x4 o[D / 16];
  float m, l;
  __device__ __forceinline__ void clear() {
    m = kLowest, l = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[d] = f32x4{0, 0, 0, 0};
  }
};

// From z (scores, V's row exponent added) to the weights' operand p (BF16:
// and p_lo); iv: 2 2^-ve (its sign does not count if far).  MASKED: `seen` says which keys count.
// The sum of weights takes w 2^-ve.  Where row exponents are at most 63 apart
// (far_bits), a w below 2^-126, which is 0, has less than 2^-70 of the weights.
// Otherwise (far: in this tile or an earlier one of this wave) it may have any
// share, and the terms are made from their exponents, 8 more exponentials.  They
// are as large as 2^116 or as small as 2^-112, whatever o is: l is rescaled in
// two steps.  Telling the two apart costs 0 to 5 %; with all rows far the 4-bit
// batch takes 8 % more, 16 trees of 63 drafts over 8-bit keys 20 %.
template <int FMT, int D, bool MASKED, bool IV>
__device__ __forceinline__ void softmax_step(Rows<D>& r, float (&z)[8], const float (&iv)[8],
                                             bool far, uint32_t seen, u32x4& p, u32x4& p_lo) {
  if constexpr (MASKED) {
#pragma unroll
    for (int x = 0; x < 8; ++x) z[x] = seen >> x & 1 ? z[x] : -__builtin_inff();
  }
  float mx = z[0];
#pragma unroll
  for (int x = 1; x < 8; ++x) mx = __builtin_fmaxf(mx, z[x]);
  mx = column_max(mx);
  float l_far = 0.0f;
  const bool anew = __any(mx > r.m + kMost);
  // one way round for both: two would cut the step in three for the scheduler
  if (anew || (IV && far)) {
    if (anew) {
      const float mn = __builtin_fmaxf(r.m, mx - kUp);
      const float h = __builtin_amdgcn_exp2f(0.5f * (r.m - mn)), f = h * h;
      r.m = mn;
      r.l = r.l * h * h;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) r.o[d] *= f;
    }
    if (IV && far) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float e = static_cast<float>(int(__float_as_uint(iv[x]) >> 23 & 0xFFu) - 127);
        const float t = iv[x] != iv[x] ? iv[x] : __builtin_amdgcn_exp2f(z[x] - r.m + e);
        l_far += !MASKED || (seen >> x & 1) ? t : 0.0f;
      }
    }
  }
  float w[8], l = 0.0f;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    w[x] = __builtin_amdgcn_exp2f(z[x] - r.m);
    if constexpr (IV) {
      if constexpr (MASKED) l += seen >> x & 1 ? w[x] * iv[x] : 0.0f;   // iv may be NaN
      else l = __builtin_fmaf(w[x], iv[x], l);
    } else {
      l += w[x];
    }
  }
  if (IV && far) l = l_far;
  r.l = FMT == QL_KV_BF16 ? r.l + l : __builtin_fmaf(l, kUnit / 2, r.l);   // iv: 2 2^-ve
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if constexpr (FMT == QL_KV_BF16) {
      p[x] = pack_bf16x2(w[2 * x], w[2 * x + 1]);
      p_lo[x] = pack_bf16x2(w[2 * x] - __uint_as_float(p[x] << 16),
                            w[2 * x + 1] - __uint_as_float(p[x] & 0xFFFF0000u));
    } else {
      const f32x2 v = {w[2 * x], w[2 * x + 1]};
      p[x] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    }
  }
}

// Operands are made right before the product that takes them: made further
// ahead (as the compiler would) they cost registers, and so waves.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

template <int FMT>
__device__ __forceinline__ f32x4 weigh(u32x4 v, u32x4 p, u32x4 p_lo, f32x4 o) {
  o = mma<FMT != QL_KV_BF16>(v, p, o);
  if constexpr (FMT == QL_KV_BF16) o = mma<false>(v, p_lo, o);
  return o;
}

// 1 / (sum of weights), from the sum as it is kept (in units of 1 / unit); 0
// for a row that sees nothing, whose result is zero.
__device__ __forceinline__ float reciprocal(float l, float unit) {
  return l == 0.0f ? 0.0f : unit / l;
}
constexpr float unit_of(int fmt) { return fmt == QL_KV_BF16 ? 1.0f : kUnit; }

// Row `row`'s place in y, or among the partial results of a split sequence.
__device__ __forceinline__ int64_t out_row(const KvAttnArgs& a, const Work& w, int row) {
  const int node = row / w.group, head = w.head * w.group + (row - node * w.group);
  return w.nsplit == 1 ? int64_t(w.sq.q0 + node) * a.n_q + head
                       : (int64_t(w.part) * a.max_q + node) * a.n_q + head;
}

// ---------------------------------------------------------------------------
// narrow: 16 rows, keys split over the waves
// ---------------------------------------------------------------------------
template <int FMT, int D>
struct Tile {
  using L = KvLayout<FMT, D>;
  Block<FMT, D> k[2], v[2];
  uint32_t ke[2];      // row exponents: E4M3 of the four keys around key lane % 16,
                       // NVFP4 of keys 4 g .. 4 g + 3
  uint32_t ve[2];      // of keys 4 g .. 4 g + 3
  __device__ __forceinline__ void load(int t, const Source& s, int lane) {
    k[t].load_k(s, lane);
    v[t].load_v(s, lane);
    if constexpr (FMT == QL_KV_E4M3) {
      ke[t] = load32(s.scales, L::k_exp(lane & 12));
      ve[t] = load32(s.scales, L::v_exp(lane >> 4 << 2));
    } else if constexpr (FMT == QL_KV_NVFP4) {
      const auto e = __builtin_amdgcn_raw_buffer_load_b64(s.scales, L::k_exp(lane >> 4 << 2), 0, 0);
      ke[t] = e[0], ve[t] = e[1];
    }
  }
  // Whether a V row (MASKED: of the keys in some lane's `seen`) has an exponent
  // far from the usual.
  template <bool MASKED>
  __device__ __forceinline__ bool any_far(uint32_t seen) const {
    uint32_t out = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      out |= MASKED ? far_bits(ve[t]) & byte_mask(seen >> (4 * t)) : far_bits(ve[t]);
    return __any((out & 0xC0C0C0C0u) != 0);
  }
};

// One tile.  n0, n1: how many of each block's 16 keys are there.  MASKED: some
// are hidden from some row, or missing; otherwise n0 or n1 is 0 only where a
// block's page is absent, and the tile holds the other block in its place.
template <int FMT, int D, bool MASKED>
__device__ __forceinline__ void narrow_tile(Rows<D>& r, const u32x4 (&sm_q)[D / 32][64], float qs,
                                            Tile<FMT, D>& tile, int n0, int n1, uint32_t seen,
                                            bool& far, int lane) {
  constexpr bool HALF = FMT == QL_KV_NVFP4;
  const int g = lane >> 4;
  // read again for every tile: held in registers they would cost waves
  asm volatile("" ::: "memory");
  u32x4 q[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) q[k] = sm_q[k][lane];
  f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  float kp[2] = {1.0f, 1.0f};
  if constexpr (FMT == QL_KV_E4M3) {
#pragma unroll
    for (int t = 0; t < 2; ++t) kp[t] = power(tile.ke[t] >> 8 * (lane & 3) & 0xFFu);
  }
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      s[t] = mma<HALF>(tile.k[t].template k_operand<HALF>(k, kp[t], lane), q[k], s[t]);
    in_order();
  }
  const float hide0 = MASKED || n0 ? 0.0f : -__builtin_inff();
  const float hide1 = MASKED || n1 ? 0.0f : -__builtin_inff();
  float z[8], iv[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int t = x >> 2, k = x & 3;
    const float hide = t ? hide1 : hide0;
    if constexpr (FMT == QL_KV_BF16) {
      z[x] = __builtin_fmaf(s[t][k], qs, hide);
    } else {
      const uint32_t b = tile.ve[t] >> (8 * k) & 0xFFu;
      iv[x] = power(~tile.ve[t] >> (8 * k) & 0xFFu);   // 2^(128 - b)
      float v = s[t][k];
      if constexpr (HALF) v *= power(tile.ke[t] >> (8 * k) & 0xFFu);
      z[x] = __builtin_fmaf(v, qs, static_cast<float>(b) + hide);
    }
  }
  if constexpr (MASKED) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int left = (t ? n1 : n0) - 4 * g, keys = left < 0 ? 0 : left > 4 ? 4 : left;
      seen &= ~(0xFu << (4 * t)) | ((1u << keys) - 1u) << (4 * t);
      tile.v[t].clear_v(keys);
    }
  }
  if constexpr (FMT != QL_KV_BF16) far = far || tile.template any_far<MASKED>(seen);
  u32x4 p, p_lo;
  softmax_step<FMT, D, MASKED, FMT != QL_KV_BF16>(r, z, iv, far, seen, p, p_lo);
  if constexpr (MASKED) {
    // A zero weight does not hide a NaN or an infinity in the product: they
    // are cleared, and the sum of weights of a row that sees one is made NaN.
    if (__any((tile.v[0].non_finite() | tile.v[1].non_finite()) != 0)) {
      const uint32_t bad = tile.v[0].clear_non_finite() | tile.v[1].clear_non_finite() << 4;
      if (seen & bad) r.l = __builtin_nanf("");
    }
  }
  constexpr int per = Block<FMT, D>::kPer;
#pragma unroll
  for (int j = 0; j < D / 16 / per; ++j) {
    uint2 a[per], b[per];
    tile.v[0].v_operands(j, a);
    tile.v[1].v_operands(j, b);
#pragma unroll
    for (int x = 0; x < per; ++x) {
      f32x4& o = r.o[j * per + x];
      o = weigh<FMT>(u32x4{a[x].x, a[x].y, b[x].x, b[x].y}, p, p_lo, o);
    }
    in_order();
  }
}

// Waves per SIMD that the register budget is set for: what fits without
// spills that matter.  It is the number of waves, not loads under way in each,
// that covers the memory's latency: with the next tile's loads issued ahead,
// and half the waves for want of registers, 16 sequences of up to 8192 8-bit
// 256-wide keys took 62 us instead of 49, 64 of up to 1024 128-wide ones 22.6
// instead of 21.8.
constexpr int narrow_waves(int fmt, int d) {
  return d == 64 ? 5 : d == 128 ? (fmt == QL_KV_BF16 ? 3 : 4) : 2;
}

// The tiles that one wave takes of a block's keys: first, first + 4, ..., the
// last first, so that those with hidden keys come before those that every row
// sees.
template <int FMT, int D>
struct Walk {
  const KvAttnArgs& a;
  const Work& w;
  int lane, first, count, partly;      // tiles; of them, the first `partly` with hidden keys
  int per_page;                        // log2(blocks of a page)
  const int32_t* table;
  int pages = -1;                      // of 32 tiles' two blocks, one per lane
  __device__ __forceinline__ Walk(const KvAttnArgs& args, const Work& work, int wave, int ln)
      : a(args), w(work), lane(ln) {
    first = w.k0 / kTile + wave;
    const int tiles = tiles_of(w.k1);
    count = tiles > first ? (tiles - first + kWaves - 1) / kWaves : 0;
    const int open = open_to(a, w, w.row0) / kTile;
    partly = count - (open > first ? (open - first + kWaves - 1) / kWaves : 0);
    per_page = a.g.page_shift - 4;
    table = a.table + int64_t(w.b) * a.table_stride;
  }
  __device__ __forceinline__ int tile_of(int i) const { return first + kWaves * (count - 1 - i); }
  // Reads tile i; p0, p1: its blocks' pages, negative if absent.  An absent
  // block is read from the tile's other block.
  __device__ __forceinline__ void load(int i, Tile<FMT, D>& tile, int& p0, int& p1) {
    if ((i & 31) == 0) {
      const int mine = i + (lane >> 1) < count ? 2 * tile_of(i + (lane >> 1)) + (lane & 1) : -1;
      pages = -1;
      if (mine >= 0 && int64_t(mine) * 16 < w.k1) {
        pages = table[mine >> per_page];
        if (pages >= a.g.n_pages) pages = -1;
      }
    }
    const int block = 2 * tile_of(i);
    p0 = __builtin_amdgcn_readlane(pages, 2 * (i & 31));
    p1 = __builtin_amdgcn_readlane(pages, 2 * (i & 31) + 1);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int own = t ? p1 : p0, other = t ? p0 : p1;
      const int page = own >= 0 ? own : other >= 0 ? other : 0;
      const int in = (own >= 0 ? block + t : block + 1 - t) & ((1 << per_page) - 1);
      tile.load(t, source<FMT, D>(a.g, kv_block(a.g, page, w.head, in)), lane);
    }
  }
};

// Joins the four waves' parts of 16 rows, in wave order, and stores them.
template <int FMT, int D, int DCH>
__device__ __forceinline__ void finish(const KvAttnArgs& a, const Work& w, Rows<D>& r, int row0,
                                       float (&sm_m)[kWaves][16], float (&sm_l)[kWaves][16],
                                       float (&sm_o)[kWaves][16][DCH + 4]) {
  using L = KvLayout<FMT, D>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  r.l = column_sum(r.l);
  if (g == 0) sm_m[wave][n] = r.m, sm_l[wave][n] = r.l;
  __syncthreads();
  float top = sm_m[0][n];
#pragma unroll
  for (int x = 1; x < kWaves; ++x) top = __builtin_fmaxf(top, sm_m[x][n]);
  const float f = __builtin_amdgcn_exp2f(r.m - top);
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
        for (int y = 0; y < 4; ++y) v[y] = r.o[L::kDC * i + (x + y) % L::kDC][(x + y) / L::kDC] * f;
        *reinterpret_cast<f32x4*>(&sm_o[wave][n][d0 % DCH + 4 * L::kDC * g + x]) = v;
      }
    }
    __syncthreads();
    constexpr int kCols = DCH / 8;      // threads per row, 8 elements each
    const int row = threadIdx.x / kCols, c = threadIdx.x % kCols * 8;
    if (row < 16 && row0 + row < w.rows) {
      float tm = sm_m[0][row];
#pragma unroll
      for (int x = 1; x < kWaves; ++x) tm = __builtin_fmaxf(tm, sm_m[x][row]);
      float l = 0.0f, v[8] = {};
#pragma unroll
      for (int x = 0; x < kWaves; ++x) {
        const float h = __builtin_amdgcn_exp2f(0.5f * (sm_m[x][row] - tm));
        l += sm_l[x][row] * h * h;     // in two steps, as in softmax_step
#pragma unroll
        for (int y = 0; y < 8; ++y) v[y] += sm_o[x][row][c + y];
      }
      const int64_t out = out_row(a, w, row0 + row);
      if (w.nsplit == 1) {
        const float inv = reciprocal(l, unit_of(FMT));
        uint32_t y[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] = pack_bf16x2(v[2 * x] * inv, v[2 * x + 1] * inv);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + out * D + part * DCH + c) =
            make_uint4(y[0], y[1], y[2], y[3]);
      } else {
        float4* o = reinterpret_cast<float4*>(a.part_o + out * D + part * DCH + c);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
        if (part == 0 && c == 0) a.part_ml[2 * out] = tm, a.part_ml[2 * out + 1] = l;
      }
    }
    __syncthreads();
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(64 * kWaves, narrow_waves(FMT, D)) void kv_attention_narrow_kernel(
    KvAttnArgs a) {
  using L = KvLayout<FMT, D>;
  constexpr int DCH = D < 128 ? D : 128;        // elements of d joined at a time
  __shared__ float sm_m[kWaves][16], sm_l[kWaves][16];
  __shared__ __align__(16) float sm_o[kWaves][16][DCH + 4];
  __shared__ u32x4 sm_q[D / 32][64];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const Work w = work_of<16>(a);
  if (!w.any) return;
  float qs;
  RowMask rm;
  {
    u32x4 q[D / 32];
    load_query<FMT, D, FMT == QL_KV_NVFP4>(a, w, w.row0 + n, g, q, qs, rm);
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
      if (k % kWaves == wave) sm_q[k][lane] = q[k];
  }
  __syncthreads();
  Rows<D> r;
  r.clear();

  Walk<FMT, D> walk(a, w, wave, lane);
  Tile<FMT, D> tile;
  bool far = false;
  int p0, p1;
  for (int i = 0; i < walk.partly; ++i) {
    walk.load(i, tile, p0, p1);
    const int base = walk.tile_of(i) * kTile, left = w.k1 - base;
    narrow_tile<FMT, D, true>(r, sm_q, qs, tile, p0 < 0 ? 0 : left, p1 < 0 ? 0 : left - 16,
                              visible(rm, a.tree != nullptr, base, w.sq.ctx, g), far, lane);
  }
  for (int i = walk.partly; i < walk.count; ++i) {
    walk.load(i, tile, p0, p1);
    if (p0 >= 0 || p1 >= 0)
      narrow_tile<FMT, D, false>(r, sm_q, qs, tile, p0 >= 0, p1 >= 0, 0, far, lane);
  }

  finish<FMT, D, DCH>(a, w, r, w.row0, sm_m, sm_l, sm_o);
}

// ---------------------------------------------------------------------------
// pair: 32 rows, keys split over the waves
// ---------------------------------------------------------------------------
// Waves per SIMD: 64 elements of o and two blocks' bytes of 128-wide heads fill
// the registers of two (with three they spill: 51 us become 126); of 64-wide
// heads four fit, three at 8 bits (32 sequences of up to 4096 keys, 4 drafts,
// 60 / 12 heads: 4 bits 40 us, and 43 with three; 8 bits 37 us either way, 16
// sequences of up to 8192 22 us and 24 with four).
constexpr int pair_waves(int fmt, int d) {
  return d == 128 ? 2 : fmt == QL_KV_E4M3 ? 3 : 4;
}

// One tile for two row tiles; arguments as narrow_tile.
template <int FMT, int D, bool MASKED>
__device__ __forceinline__ void pair_tile(Rows<D> (&r)[2], const u32x4 (&sm_q)[2][D / 32][64],
                                          const float (&qs)[2], Tile<FMT, D>& tile, int n0, int n1,
                                          uint32_t (&seen)[2], bool& far, int lane) {
  constexpr bool HALF = FMT == QL_KV_NVFP4;
  const int g = lane >> 4;
  // read again for every tile: held in registers they would cost waves
  asm volatile("" ::: "memory");
  f32x4 s[2][2] = {};
  float kp[2] = {1.0f, 1.0f};
  if constexpr (FMT == QL_KV_E4M3) {
#pragma unroll
    for (int t = 0; t < 2; ++t) kp[t] = power(tile.ke[t] >> 8 * (lane & 3) & 0xFFu);
  }
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    u32x4 q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) q[i] = sm_q[i][k][lane];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const u32x4 a = tile.k[t].template k_operand<HALF>(k, kp[t], lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) s[i][t] = mma<HALF>(a, q[i], s[i][t]);
    }
    in_order();
  }
  const float hide0 = MASKED || n0 ? 0.0f : -__builtin_inff();
  const float hide1 = MASKED || n1 ? 0.0f : -__builtin_inff();
  if constexpr (MASKED) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int left = (t ? n1 : n0) - 4 * g, keys = left < 0 ? 0 : left > 4 ? 4 : left;
#pragma unroll
      for (int i = 0; i < 2; ++i) seen[i] &= ~(0xFu << (4 * t)) | ((1u << keys) - 1u) << (4 * t);
      tile.v[t].clear_v(keys);
    }
  }
  if constexpr (FMT != QL_KV_BF16) far = far || tile.template any_far<MASKED>(seen[0] | seen[1]);
  u32x4 p[2], p_lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float z[8], iv[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int t = x >> 2, k = x & 3;
      const float hide = t ? hide1 : hide0;
      if constexpr (FMT == QL_KV_BF16) {
        z[x] = __builtin_fmaf(s[i][t][k], qs[i], hide);
      } else {
        const uint32_t b = tile.ve[t] >> (8 * k) & 0xFFu;
        iv[x] = power(~tile.ve[t] >> (8 * k) & 0xFFu);   // 2^(128 - b)
        float v = s[i][t][k];
        if constexpr (HALF) v *= power(tile.ke[t] >> (8 * k) & 0xFFu);
        z[x] = __builtin_fmaf(v, qs[i], static_cast<float>(b) + hide);
      }
    }
    softmax_step<FMT, D, MASKED, FMT != QL_KV_BF16>(r[i], z, iv, far, seen[i], p[i], p_lo[i]);
    in_order();
  }
  if constexpr (MASKED) {
    // A zero weight does not hide a NaN or an infinity in the product: they
    // are cleared, and the sum of weights of a row that sees one is made NaN.
    if (__any((tile.v[0].non_finite() | tile.v[1].non_finite()) != 0)) {
      const uint32_t bad = tile.v[0].clear_non_finite() | tile.v[1].clear_non_finite() << 4;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (seen[i] & bad) r[i].l = __builtin_nanf("");
    }
  }
  constexpr int per = Block<FMT, D>::kPer;
#pragma unroll
  for (int j = 0; j < D / 16 / per; ++j) {
    uint2 a[per], b[per];
    tile.v[0].v_operands(j, a);
    tile.v[1].v_operands(j, b);
#pragma unroll
    for (int x = 0; x < per; ++x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f32x4& o = r[i].o[j * per + x];
        o = weigh<FMT>(u32x4{a[x].x, a[x].y, b[x].x, b[x].y}, p[i], p_lo[i], o);
      }
    }
    in_order();
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(64 * kWaves, pair_waves(FMT, D)) void kv_attention_pair_kernel(
    KvAttnArgs a) {
  constexpr int DCH = D < 128 ? D : 128;
  __shared__ float sm_m[kWaves][16], sm_l[kWaves][16];
  __shared__ __align__(16) float sm_o[kWaves][16][DCH + 4];
  __shared__ u32x4 sm_q[2][D / 32][64];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const Work w = work_of<32>(a);
  if (!w.any) return;
  float qs[2];
  RowMask rm[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    u32x4 q[D / 32];
    load_query<FMT, D, FMT == QL_KV_NVFP4>(a, w, w.row0 + 16 * x + n, g, q, qs[x], rm[x]);
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
      if (k % kWaves == wave) sm_q[x][k][lane] = q[k];
  }
  __syncthreads();
  Rows<D> r[2];
  r[0].clear();
  r[1].clear();
  Walk<FMT, D> walk(a, w, wave, lane);
  Tile<FMT, D> tile;
  bool far = false;
  int p0, p1;
  uint32_t seen[2] = {0, 0};
  for (int i = 0; i < walk.partly; ++i) {
    walk.load(i, tile, p0, p1);
    const int base = walk.tile_of(i) * kTile, left = w.k1 - base;
#pragma unroll
    for (int x = 0; x < 2; ++x) seen[x] = visible(rm[x], a.tree != nullptr, base, w.sq.ctx, g);
    pair_tile<FMT, D, true>(r, sm_q, qs, tile, p0 < 0 ? 0 : left, p1 < 0 ? 0 : left - 16, seen, far,
                            lane);
  }
  for (int i = walk.partly; i < walk.count; ++i) {
    walk.load(i, tile, p0, p1);
    if (p0 >= 0 || p1 >= 0)
      pair_tile<FMT, D, false>(r, sm_q, qs, tile, p0 >= 0, p1 >= 0, seen, far, lane);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) finish<FMT, D, DCH>(a, w, r[x], w.row0 + 16 * x, sm_m, sm_l, sm_o);
}

// ---------------------------------------------------------------------------
// wide: 64 rows, 16 for each wave; tiles shared through LDS
// ---------------------------------------------------------------------------
template <int FMT, int D>
struct Shared {        // one tile's operands
  u32x4 k[2][D / 32][64];
  u32x4 v[D / 16][64];
  float ve[kTile];     // V's row exponent + 127; -inf: the key is missing
  float iv[kTile];     // 2 2^-that exponent, negative if it is far from the usual
                       // (far_bits); NaN: the row holds a NaN or an infinity
};

// The quarter of a tile that a wave turns into operands: block t's K or V.
template <int FMT, int D>
struct Quarter {
  using L = KvLayout<FMT, D>;
  Block<FMT, D> x;
  uint32_t e;          // row exponents of the four keys around key lane % 16
  int keys;            // keys of the block that are there

  __device__ __forceinline__ void load(const Source& s, bool is_v, int lane) {
    if (is_v) x.load_v(s, lane);
    else x.load_k(s, lane);
    if constexpr (FMT != QL_KV_BF16) e = load32(s.scales, L::k_exp(lane & 12) + (is_v ? 4 : 0));
  }
  // check: keys of this tile may be hidden from some row.
  __device__ __forceinline__ void store(Shared<FMT, D>& sh, int t, bool is_v, bool check, int lane) {
    const int n = lane & 15, g = lane >> 4;
    uint32_t mine = 0;
    if constexpr (FMT != QL_KV_BF16) mine = e >> 8 * (n & 3) & 0xFFu;
    if (!is_v) {
      float p = 1.0f;
      if constexpr (FMT != QL_KV_BF16) p = power(mine);
      const uint32_t keep = n < keys ? ~0u : 0u;
#pragma unroll
      for (int s = 0; s < D / 32; ++s)
        sh.k[t][s][lane] = x.template k_operand<false>(s, p, lane) & keep;
    } else {
      uint32_t bad = 0;
      if (keys < 16) {
        const int left = keys - 4 * g;
        x.clear_v(left < 0 ? 0 : left > 4 ? 4 : left);
      }
      if (check && __any(x.non_finite() != 0)) {
        // as in narrow_tile; lane n's key is in quad n / 4
        bad = x.clear_non_finite();
        bad = __shfl(bad, (n >> 2) * 16, 64) >> (n & 3) & 1u;
      }
      constexpr int per = Block<FMT, D>::kPer;
#pragma unroll
      for (int j = 0; j < D / 16 / per; ++j) {
        uint2 r[per];
        x.v_operands(j, r);
#pragma unroll
        for (int q = 0; q < per; ++q) reinterpret_cast<uint2*>(&sh.v[j * per + q][lane])[t] = r[q];
      }
      if (g == 0) {
        float ve = 0.0f, iv = 1.0f;
        if constexpr (FMT != QL_KV_BF16) {
          ve = static_cast<float>(mine), iv = power(255u - mine);
          iv = far_bits(mine) & 0xC0u ? -iv : iv;
        }
        sh.ve[16 * t + n] = n < keys ? ve : -__builtin_inff();
        sh.iv[16 * t + n] = n >= keys ? 0.0f : bad ? __builtin_nanf("") : iv;
      }
    }
  }
};

template <int FMT, int D, bool MASKED>
__device__ __forceinline__ void wide_tile(Rows<D>& r, const u32x4 (&q)[D / 32], float qs,
                                          const Shared<FMT, D>& sh, uint32_t seen, bool& far, int lane) {
  const int g = lane >> 4;
  f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
#pragma unroll
    for (int t = 0; t < 2; ++t) s[t] = mma<false>(sh.k[t][k][lane], q[k], s[t]);
    if (k % 2) in_order();
  }
  float z[8], iv[8];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(&sh.ve[16 * t + 4 * g]);
    const f32x4 b = *reinterpret_cast<const f32x4*>(&sh.iv[16 * t + 4 * g]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      z[4 * t + k] = __builtin_fmaf(s[t][k], qs, a[k]);
      iv[4 * t + k] = b[k];
    }
  }
  if constexpr (FMT != QL_KV_BF16) {
    uint32_t signs = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) signs |= __float_as_uint(iv[x]);
    far = far || __any(int(signs) < 0);
  }
  u32x4 p, p_lo;
  softmax_step<FMT, D, MASKED, true>(r, z, iv, far, seen, p, p_lo);
#pragma unroll
  for (int d = 0; d < D / 16; ++d) {
    r.o[d] = weigh<FMT>(sh.v[d][lane], p, p_lo, r.o[d]);
    if (d % 4 == 3) in_order();
  }
}

// 16 rows to a wave, and so two or three waves on a SIMD, beat 32: a tile is a
// chain of LDS reads, products and the softmax that takes a wave more than
// twice the cycles it issues, so it is the other waves that fill the SIMD.
// (Measured with 8-bit 128-wide keys before those had the pair kernel, 16
// sequences of 63 drafts over 2000 keys: 56 us, with 32 rows to a wave 77, with
// eight waves to a block 78.)
template <int FMT, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_attention_wide_kernel(KvAttnArgs a) {
  using L = KvLayout<FMT, D>;
  constexpr int P = 2;      // tiles whose bytes are under way, and buffers in LDS
  extern __shared__ __align__(16) uint8_t lds[];
  Shared<FMT, D>* sh = reinterpret_cast<Shared<FMT, D>*>(lds);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const Work w = work_of<64>(a);
  if (!w.any) return;
  const int row0 = w.row0 + wave * 16;
  const bool active = row0 < w.rows;
  u32x4 q[D / 32];
  float qs;
  RowMask rm;
  load_query<FMT, D, false>(a, w, row0 + n, g, q, qs, rm);
  Rows<D> r;
  r.clear();
  bool far = false;

  // The tiles in the order they are taken: the last ones, of which some key is
  // hidden from some row, before those that every row sees.
  const int first = w.k0 / kTile, tiles = tiles_of(w.k1);
  const int open = open_to(a, w, w.row0) / kTile;
  const int count = tiles > first ? tiles - first : 0;
  int partly = open > first ? tiles - open : count;
  partly = partly + partly % P < count ? partly + partly % P : count;
  auto tile_of = [&](int i) { return i < partly ? tiles - partly + i : first + i - partly; };
  const int t = wave & 1;
  const bool is_v = wave >> 1;
  const int per_page = a.g.page_shift - 4;
  const int32_t* table = a.table + int64_t(w.b) * a.table_stride;
  int pages = -1;   // of block t of 64 tiles, one per lane
  auto load = [&](int i, Quarter<FMT, D>& x) {
    if (i >= count) i = count - 1;      // once more: a load that may not happen costs a move
    if ((i & 63) == 0) {
      const int ahead = 2 * tile_of(i + lane) + t;
      pages = -1;
      if (i + lane < count && int64_t(ahead) * 16 < w.k1) {
        pages = table[ahead >> per_page];
        if (pages >= a.g.n_pages) pages = -1;
      }
    }
    const int block = 2 * tile_of(i) + t;
    const int page = __builtin_amdgcn_readlane(pages, i & 63);
    const int left = w.k1 - 16 * block;
    x.keys = page < 0 || left < 0 ? 0 : left < 16 ? left : 16;
    x.load(source<FMT, D>(a.g, kv_block(a.g, page < 0 ? 0 : page, w.head,
                                        block & ((1 << per_page) - 1))), is_v, lane);
  };
  // Tile i's bytes are in x[i % P] and its operands in sh[i % P]; the loops go
  // P tiles at a time, because registers that are loaded must not be moved
  // (the move would wait for the load).
  Quarter<FMT, D> x[P];
  if (count > 0) {
#pragma unroll
    for (int y = 0; y < P; ++y) load(y, x[y]);
  }
  // Makes tile i's operands (y = i % P).  Every wave has left that buffer,
  // which held tile i - P, before the last barrier.
  auto prepare = [&](int i, int y) {
    if (i < count) x[y].store(sh[y], t, is_v, i < partly, lane);
    load(i + P, x[y]);
  };
  if (count > 0) prepare(0, 0);
  __syncthreads();
  // A loop for each kind of tile: where two ways meet, the accumulators would
  // be copied.  No way out of a loop but its end: where one in the middle met
  // the others, the compiler would wait for all loads on every turn.
  auto hidden = [&](int i, int y) {
    prepare(i + 1, (y + 1) % P);
    if (active) {
      const uint32_t seen = visible(rm, a.tree != nullptr, tile_of(i) * kTile, w.sq.ctx, g);
      in_order();
      wide_tile<FMT, D, true>(r, q, qs, sh[y], seen, far, lane);
    }
    __syncthreads();
  };
  auto open_tile = [&](int i, int y) {
    prepare(i + 1, (y + 1) % P);
    if (active) wide_tile<FMT, D, false>(r, q, qs, sh[y], 0, far, lane);
    __syncthreads();
  };
  int i = 0;
  for (; i + P <= partly; i += P) {
#pragma unroll
    for (int y = 0; y < P; ++y) hidden(i + y, y);
  }
  if (i < partly) hidden(i, 0);      // then partly == count
  for (i = partly; i + P <= count; i += P) {
#pragma unroll
    for (int y = 0; y < P; ++y) open_tile(i + y, y);
  }
  if (i < count) open_tile(i, 0);
  const int row = row0 + n;
  const float l = column_sum(r.l), inv = reciprocal(l, unit_of(FMT));
  if (row >= w.rows) return;
  const int64_t out = out_row(a, w, row);
  if (w.nsplit > 1 && g == 0) a.part_ml[2 * out] = r.m, a.part_ml[2 * out + 1] = l;
#pragma unroll
  for (int i = 0; i < L::kLoads; ++i)
#pragma unroll
    for (int x8 = 0; x8 < 4 * L::kDC; x8 += 8) {
      const int d = 16 * L::kDC * i + 4 * L::kDC * g + x8;
      float v[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) v[y] = r.o[L::kDC * i + (x8 + y) % L::kDC][(x8 + y) / L::kDC];
      if (w.nsplit == 1) {
        uint32_t y[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] = pack_bf16x2(v[2 * z] * inv, v[2 * z + 1] * inv);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + out * D + d) =
            make_uint4(y[0], y[1], y[2], y[3]);
      } else {
        float4* o = reinterpret_cast<float4*>(a.part_o + out * D + d);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
}

// Joins the splits of every row that has more than one, in a fixed order.
// D / 4 lanes (4 elements each) take one of `parts` shares of a row's splits,
// every parts-th split; the shares are then added in order.
template <int D>
__global__ __launch_bounds__(256) void kv_attention_join_kernel(KvAttnArgs a, int parts,
                                                                     float unit) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
  __shared__ f32x4 sm_o[kGroups][kLanes];
  __shared__ float sm_l[kGroups];
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int b = blockIdx.y, part = group % parts;
  const Seq sq = sequence(a, b);
  const int first = a.first[b], nsplit = a.first[b + 1] - first;
  if (nsplit == 1) return;
  const int64_t r = int64_t(blockIdx.x) * (kGroups / parts) + group / parts;   // token, head
  const bool in = r < int64_t(sq.rows_q) * a.n_q;
  const int64_t step = int64_t(a.max_q) * a.n_q, row = first * step + r;
  float l = 0.0f;
  f32x4 v = {0, 0, 0, 0};
  if (in) {
    float top = kLowest;
    for (int s = lane; s < nsplit; s += kLanes) top = __builtin_fmaxf(top, a.part_ml[2 * (s * step + row)]);
#pragma unroll
    for (int off = 1; off < kLanes; off *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, off, 64));
    for (int s = part; s < nsplit; s += parts) {
      const int64_t at = s * step + row;
      const float h = __builtin_amdgcn_exp2f(0.5f * (a.part_ml[2 * at] - top)), f = h * h;
      l = __builtin_fmaf(a.part_ml[2 * at + 1] * h, h, l);     // in two steps, as in softmax_step
      v += *reinterpret_cast<const f32x4*>(a.part_o + at * D + 4 * lane) * f;
    }
  }
  if (parts > 1) {
    sm_o[group][lane] = v;
    if (lane == 0) sm_l[group] = l;
    __syncthreads();
    if (part) return;
    for (int x = 1; x < parts; ++x) v += sm_o[group + x][lane], l += sm_l[group + x];
  }
  if (!in) return;
  v *= reciprocal(l, unit);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + (int64_t(sq.q0) * a.n_q + r) * D + 4 * lane) =
      make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

}  // namespace

// Whether the kernel of 64 rows is built for a format and head.
static constexpr bool wide_fits(int fmt, int d) {
  return d == 256 || (fmt == QL_KV_NVFP4 && d == 128);
}

KvAttnPlan kv_attention_plan(int fmt, int d, int n_q, int n_kv, int64_t n_seqs, int64_t max_q,
                             int64_t max_kv) {
  KvAttnPlan p;
  const int64_t rows = max_q * (n_q / n_kv);
  // 32 rows straight from memory, or 64 through LDS (8-bit keys, 128-wide heads:
  // 16 sequences of 63 drafts over up to 2000 keys 51 us, and 59; a 512-token
  // chunk of a prompt 25 and 41; 4-bit: 32 drafts over 60000 keys 79 and 72, 8
  // sequences of up to 8192 and 8 drafts in 5 heads 39 and 36; but a chunk of a
  // prompt whose blocks of 64 rows would not fill a round, which is not split
  // either, 33 and 44 at 512 tokens over 1000; at 4096 tokens 291 and 259)
  const int64_t cus = device_cu_count() > 0 ? device_cu_count() : 256;
  const bool few = max_q > 64 && n_seqs * n_kv * ((rows + 63) / 64) <= 3 * cus;
  const bool wide = wide_fits(fmt, d) && (d == 256 || (rows > 32 && !few));
  p.rows = rows <= 16 ? 16 : wide ? 64 : 32;
  p.row_blocks = (rows + p.rows - 1) / p.rows;
  // Parts of all keys together.  A second launch joins those of one sequence (3
  // to 10 us), and a block takes about as long as 128 keys of a narrow wave to
  // start, so up to 512 keys stay whole (500 keys, one sequence: 8 us against
  // 12), and no part of a longer one is planned under 256 keys.
  auto parts_for = [&](int64_t per_cu, int64_t least) {
    const int64_t most = max_kv <= 512 ? n_seqs : n_seqs * ((max_kv + least - 1) / least);
    // what each XCD's eighth of the units leaves room for in one round
    const int64_t n = per_cu * (cus / 8) / p.row_blocks * 8 / n_kv;
    return n > most ? most : n < n_seqs ? n_seqs : n;
  };
  if (p.rows >= 32) {
    // as many blocks as run at once where the parts stay over 512 keys, two on a
    // compute unit otherwise (4-bit 128-wide keys through LDS, three run: 16
    // sequences of 63 drafts over up to 2000 keys 67 us, and 70 with two; 8 of
    // 16 drafts over up to 4096 keys 31 us, and 28 with two)
    const int at_once = p.rows == 32 ? pair_waves(fmt, d) : d == 256 ? 2 : 3;
    const int64_t all = parts_for(at_once, 512);
    p.parts = parts_for(2, 256);
    if (p.parts < all) p.parts = all;
  } else {
    // two on a compute unit (one sequence of 131072 8-bit keys: 57 us, with
    // four 62); of rows of at most 64 bytes, whose instructions count for more
    // than their bytes, up to four while the parts are long (32 sequences of up
    // to 8192 4-bit 128-wide keys: 51 us, with two 61; 8-bit 64-wide: 60 and 69;
    // but 8-bit 128-wide: 71 and 70)
    p.parts = parts_for(2, 256);
    const int row_bytes = fmt == QL_KV_BF16 ? 2 * d : fmt == QL_KV_E4M3 ? d : d / 2;
    if (row_bytes <= 64) {
      const int64_t four = parts_for(4, 256), need = n_seqs * ((max_kv + 2047) / 2048);
      if (p.parts < need) p.parts = need < four ? need : four;
    }
  }
  return p;
}

size_t kv_attention_ws_bytes(const KvAttnPlan& p, int64_t n_seqs, int64_t max_q, int n_q, int d) {
  if (p.parts == n_seqs) return 0;
  return size_t(p.parts) * size_t(max_q) * size_t(n_q) * size_t(d + 2) * sizeof(float) +
         (size_t(n_seqs) + 1) * sizeof(int32_t);
}

template <int FMT, int D>
static hipError_t launch_wide(const KvAttnArgs& a, dim3 blocks, hipStream_t s) {
  constexpr int bytes = 2 * sizeof(Shared<FMT, D>);
  if constexpr (bytes > 64 * 1024) {
    static std::atomic<int> done[64];
    const hipError_t e = lds_limit_once(
        done, reinterpret_cast<const void*>(kv_attention_wide_kernel<FMT, D>), bytes);
    if (e != hipSuccess) return e;
  }
  kv_attention_wide_kernel<FMT, D><<<blocks, 64 * kWaves, bytes, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_attention(int fmt, int d, const KvAttnPlan& p, KvAttnArgs a, hipStream_t s) {
  const int64_t units = p.parts * a.g.n_kv;
  a.units = int(units);
  a.row_blocks = int(p.row_blocks);
  // up to 2^30 (api_kv.cpp), while a grid has less than 2^32 threads along x; x is
  // a multiple of 8, so that a block's number tells its XCD
  const unsigned all = unsigned((units + 7) / 8 * 8 * p.row_blocks), most = 1u << 23;
  const dim3 blocks(all < most ? all : most, (all + most - 1) / most);
  const hipError_t e = kv_dispatch(fmt, d, [&](auto f, auto n) {
    constexpr int FMT = decltype(f)::value, D = decltype(n)::value;
    if constexpr (wide_fits(FMT, D)) {
      if (p.rows == 64) return launch_wide<FMT, D>(a, blocks, s);
    }
    if constexpr (D < 256) {
      if (p.rows == 32) kv_attention_pair_kernel<FMT, D><<<blocks, 64 * kWaves, 0, s>>>(a);
    }
    if (p.rows == 16) kv_attention_narrow_kernel<FMT, D><<<blocks, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
  });
  if (e != hipSuccess || p.parts == a.n_seqs) return e;
  // shares of a row: all of a block's groups where there are many splits
  const int groups = 1024 / d, splits = int(p.parts / a.n_seqs);
  const int parts = splits >= 2 * groups ? groups : splits >= 4 ? 2 : 1;
  const int64_t rows = int64_t(a.max_q) * a.n_q, per_block = groups / parts;
  const dim3 grid(unsigned((rows + per_block - 1) / per_block), unsigned(a.n_seqs));
  switch (d) {
    case 64: kv_attention_join_kernel<64><<<grid, 256, 0, s>>>(a, parts, unit_of(fmt)); break;
    case 128: kv_attention_join_kernel<128><<<grid, 256, 0, s>>>(a, parts, unit_of(fmt)); break;
    default: kv_attention_join_kernel<256><<<grid, 256, 0, s>>>(a, parts, unit_of(fmt)); break;
  }
  return hipGetLastError();
}

}  // namespace qlin
